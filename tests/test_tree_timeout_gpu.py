"""Tree attention with waits that give up at any point of a run: the call ends
at once, the status says so or the outputs are right, and the next call is clean."""
import time

import pytest
import torch

import paged_attention_fp8_gb300 as pa
from tree_common import TreeBatch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(), dict(d=64), dict(q="f16"), dict(q="e4m3fn"), dict(kv="bf16"), dict(d=64, kv="bf16"),
                                dict(qo=1)])
def test_waits_that_give_up_in_the_middle(cuda_device, monkeypatch, kw):
    kw = dict(kw)
    qo = kw.pop("qo", 12)
    b = TreeBatch([6000, 2500, 40, 900], [qo] * 4, 16, 4, num_ctas=24, seed=15, **kw)
    o, lse = b.run()
    expired, longest = 0, 0.0
    for limit in (1, 100, 300, 600, 1000, 1500, 2000, 2500, 3000, 4000, 5000, 7000, 10000, 20000, 50000):
        monkeypatch.setenv("PAFP8_WAIT_CYCLES", str(limit))
        torch.cuda.synchronize()
        began = time.monotonic()
        b.o.fill_(7.0)
        b.call()
        try:
            b.plan.device_status(b.ws)
            assert torch.equal(b.o[:b.n].cpu(), o)
        except pa.Pafp8Error as e:
            assert e.status_name == "ERR_TIMEOUT"
            expired += 1
        longest = max(longest, time.monotonic() - began)
    monkeypatch.delenv("PAFP8_WAIT_CYCLES")
    b.call()
    b.plan.device_status(b.ws)
    assert torch.equal(b.o[:b.n].cpu(), o) and torch.equal(b.lse[:b.n].cpu(), lse)
    assert expired >= 2
    # A wait for a phase that has passed would last the full bound of about a second.
    assert longest < 0.25, f"a call took {longest:.2f} s to wind down"
