"""Tree attention under memory load: many ragged requests whose lengths end
inside a tile, launch after launch, on rings of every depth a cache type gets
(two stages for a 2-byte cache at head_dim 128, three or more otherwise)."""
import numpy as np
import pytest
import torch

from tree_common import TreeBatch

pytestmark = pytest.mark.gpu


def _ragged(seed, batch, lo, hi, new):
    r = np.random.default_rng(seed)
    kv = [int(x) for x in r.integers(lo, hi, batch)]
    return [n + 1 if n % 128 == 0 else n for n in kv], [int(x) for x in r.integers(1, new + 1, batch)]


def _same_every_time(b, launches):
    """Launches back to back, every output compared on the device with the first's."""
    o, lse = b.run()
    size = torch.int16
    first_o, first_l = b.o.view(size).clone(), b.lse.view(torch.int32).clone()
    differ = torch.zeros((), dtype=torch.int64, device=b.device)
    for _ in range(launches):
        b.o.fill_(7.0)
        b.call()
        differ += (b.o.view(size) != first_o).sum() + (b.lse.view(torch.int32) != first_l).sum()
    b.plan.device_status(b.ws)
    assert int(differ) == 0, f"{int(differ)} elements differed over {launches} launches"
    b.check(o, lse)


@pytest.mark.parametrize("q,kv", [("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("new,layout,page_size", [(8, "HND", 16), (16, "NHD", 16), (5, "NHD", 48)])
def test_two_stages(cuda_device, q, kv, new, layout, page_size):
    kv_lens, qo_lens = _ragged(new, 40, 130, 2600, new)
    _same_every_time(TreeBatch(kv_lens, qo_lens, 16, 4, q=q, kv=kv, layout=layout, page_size=page_size, seed=new), 200)


@pytest.mark.parametrize("q,kv,d", [("bf16", "e4m3fn", 128), ("f16", "e5m2", 128), ("e4m3fn", "e4m3fn", 64), ("bf16", "bf16", 64)])
def test_more_stages(cuda_device, q, kv, d):
    kv_lens, qo_lens = _ragged(3, 40, 130, 2600, 16)
    _same_every_time(TreeBatch(kv_lens, qo_lens, 16, 4, d=d, q=q, kv=kv, seed=3), 100)


def test_short_requests_one_after_the_other(cuda_device):
    """Every tile is a request's last: the group waits for V at each of them."""
    kv_lens, qo_lens = _ragged(4, 600, 5, 250, 4)
    _same_every_time(TreeBatch(kv_lens, [min(a, b) for a, b in zip(qo_lens, kv_lens)], 8, 8, q="bf16", kv="bf16", seed=4), 100)
