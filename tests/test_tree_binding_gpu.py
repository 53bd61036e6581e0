"""pafp8_run_tree's refusals of device arrays, and that what it passes on still runs."""
import pytest
import torch

from tree_common import TreeBatch

pytestmark = pytest.mark.gpu


def test_scales_and_indices_of_another_type_or_place(cuda_device):
    b = TreeBatch([100, 60], [4, 4], 8, 2, q="e4m3fn", head_scales=True, seed=14)
    o, lse = b.run()
    good = [b.dq, b.kc, b.vc, b.ids, b.mask, b.o, b.lse, b.ws]
    scales = dict(q_scales=b.qs_h.cuda(), k_scales=b.ks_h.cuda(), v_scales=b.vs_h.cuda())
    for name in scales:
        for bad, match in ((scales[name].cpu(), f"{name} is on cpu"), (scales[name].double(), f"{name} has dtype"),
                           (scales[name].repeat_interleave(2)[::2], f"{name} .*not contiguous")):
            with pytest.raises(ValueError, match=match):
                b.plan.run_tree(*good, **{**scales, name: bad})
    for at, bad, match in ((3, b.ids.long(), "kv_indices has dtype"), (6, b.lse.double(), "lse has dtype"),
                           (6, b.lse.bfloat16(), "lse has dtype")):
        args = list(good)
        args[at] = bad
        with pytest.raises(ValueError, match=match):
            b.plan.run_tree(*args, **scales)
    b.o.fill_(7.0)
    b.plan.run_tree(*good, **scales)
    b.plan.device_status(b.ws)
    assert torch.equal(b.o[:b.n].cpu(), o) and torch.equal(b.lse[:b.n].cpu(), lse)
