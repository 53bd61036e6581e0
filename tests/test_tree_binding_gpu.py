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


def test_arrays_that_are_too_small_for_the_plan(cuda_device):
    b = TreeBatch([100, 60], [4, 4], 8, 2, seed=16, layout="HND", page_size=32)
    o, lse = b.run()
    good = [b.dq, b.kc, b.vc, b.ids, b.mask, b.o, b.lse, b.ws]
    kw = dict(k_scale=b.ks, v_scale=b.vs)
    for at, bad, match in ((0, b.dq[:7], "q .* the plan needs"), (5, b.o[:7], "o .* the plan needs"), (6, b.lse[:7], "lse .* the plan"),
                           (3, b.ids[:-1], "kv_indices .* the plan"), (1, b.kc[:-1], "k_cache .* the plan"),
                           (2, b.vc.transpose(1, 2).contiguous(), "v_cache .* pages"), (4, b.mask[:7], "tree_mask")):
        args = list(good)
        args[at] = bad
        with pytest.raises(ValueError, match=match):
            b.plan.run_tree(*args, **kw)
    # padded rows, and the caches and the query as bytes
    b.o.fill_(7.0)
    wide = torch.cat([b.dq, b.dq[:2]])
    b.plan.run_tree(wide, b.kc.view(torch.uint8), b.vc.view(torch.uint8), b.ids, b.mask, b.o, b.lse, b.ws, k_dtype="e4m3fn",
                    v_dtype="e4m3fn", **kw)
    b.plan.device_status(b.ws)
    assert torch.equal(b.o[:b.n].cpu(), o) and bool((b.o[b.n:] == 7).all())
