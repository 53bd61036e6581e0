"""More segments in a block than it keeps records of in shared memory (32): the
others' are read from global memory."""
import numpy as np
import pytest
import torch

from step_ref import tree_rows
from tree_common import TreeBatch

pytestmark = pytest.mark.gpu


def _most(b):
    m = b.plan.metadata()
    ptr = m[int(m[12]):int(m[12]) + int(m[6]) + 1]
    return int(np.diff(ptr).max())


@pytest.mark.parametrize("q,kv,d", [("bf16", "e4m3fn", 128), ("f16", "e5m2", 64), ("bf16", "bf16", 128)])
@pytest.mark.parametrize("num_ctas", [1, 3])
def test_few_blocks_over_many_requests(cuda_device, q, kv, d, num_ctas):
    r = np.random.default_rng(num_ctas)
    kv_lens = [int(x) for x in r.integers(20, 300, 45)]
    b = TreeBatch(kv_lens, [int(x) for x in r.integers(1, 9, 45)], 8, 4, d=d, q=q, kv=kv, num_ctas=num_ctas, seed=num_ctas)
    assert _most(b) > 32
    b.check(*b.run())


def test_a_batch_of_a_thousand(cuda_device):
    """A batch that leaves every block of the whole device more than 32."""
    r = np.random.default_rng(7)
    kv_lens = [int(x) for x in r.integers(5, 200, 1021)]
    qo_lens = [min(int(x), n) for x, n in zip(r.integers(0, 6, 1021), kv_lens)]
    b = TreeBatch(kv_lens, qo_lens, 16, 8, seed=7)
    assert _most(b) > 32
    o, lse = b.run()
    b.check(o, lse)
    # A few requests row by row.  o: P and o are off by half a step each (2^-8), P's f16 by 2^-11 and the logits by
    # 2^-10 at most (2^-17 of the row's largest times the sum of |k|: 2^-17 4.5 90 / 11.3 = 2.7e-4, and 2e-4 of fp32
    # sums), together 0.0103 of the largest value.
    for i in list(range(0, 1021, 97)) + [1020]:
        t, n, r0 = qo_lens[i], kv_lens[i], int(b.qo_indptr[i])
        seen = torch.ones(t, n, dtype=torch.bool)
        seen[:, n - t:] = torch.from_numpy(b.seen[i])
        for h in range(16):
            k, v = b.k[i][:, h // 2].double() * b.ks, b.v[i][:, h // 2].double() * b.vs
            ro, rl = tree_rows(b.q[r0:r0 + t, h].double(), k, v, seen, sm_scale=128 ** -0.5)
            off_o = (o[r0:r0 + t, h].double() - ro).abs()
            off_l = (lse[r0:r0 + t, h].double() - rl).abs()
            assert off_o.numel() == 0 or float(off_o.max()) <= 2.0 ** -6 * float(v.abs().max())
            assert off_l.numel() == 0 or float(off_l.max()) <= 2.0 ** -10
