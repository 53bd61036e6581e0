"""K scales so small that the softmax scale they are folded into underflows: the logits are zero, and hidden keys stay hidden
(minus infinity times a factor of zero would be NaN)."""
import pytest
import torch

from window_ref import Batch

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -149  # fp32's smallest number


@pytest.mark.parametrize("new", [None, [70, 33]])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("kw", [
    dict(), dict(q="e4m3fn", d=64), dict(scales="head"), dict(scales="head", q="f16", kv="f16"),
    dict(scales="head", q="bf16", kv="bf16", d=64), dict(scales="block"), dict(scales="block", q="e5m2"),
    dict(scales="block", q="f16", d=64, page_size=48, layout="HND")])
def test_a_softmax_scale_that_underflows(cuda_device, new, window, kw):
    b = Batch([333, 150], new, window=window, sinks=3 if window else 0, num_ctas=6, **kw)
    if b.scales == "tensor":
        b.k_scale = TINY
    else:  # every other head, or page
        b.ks[::2] = TINY
    b.upload()
    b.run()
    b.plan.device_status(b.ws)
    b.check()
