"""Calls that start early (programmatic launches) after work on two streams that was joined, eagerly and captured: they wait
for all of it."""
import pytest
import torch

import paged_attention_fp8_gb300 as pa
from blocks_ref import in_layout, raw
from window_ref import Batch

pytestmark = pytest.mark.gpu

KINDS = [dict(scales="block"), dict(window=150, sinks=9), dict(window=150, sinks=9, kv="bf16"), dict(scales="block", window=100)]


class Late:
    """A batch whose inputs arrive on two streams, each behind some tens of microseconds of other work."""

    def __init__(self, new, kw):
        self.b = Batch([333, 48, 700], new, num_ctas=30, **kw).upload()
        self.o = Batch([333, 48, 700], new, num_ctas=30, seed=5, **kw)
        self.side = torch.cuda.Stream()
        o, b = self.o, self.b
        self.src = [o.q.cuda(), *(in_layout(x, b.layout).cuda() for x in (o.k, o.v)),
                    *((o.ks.cuda(), o.vs.cuda()) if o.scales == "block" else ())]
        self.dst = [b.q_d, b.k_d, b.v_d, *((b.ks_d, b.vs_d) if o.scales == "block" else ())]

    def step(self):
        here = torch.cuda.current_stream()
        self.side.wait_stream(here)
        with torch.cuda.stream(self.side):
            torch.cuda._sleep(100000)
            for d, s in list(zip(self.dst, self.src))[::2]:
                raw(d).copy_(raw(s))
            torch.add(raw(self.dst[0]), 0, out=raw(self.dst[0]))  # (a kernel last, not a copy)
        torch.cuda._sleep(50000)
        for d, s in list(zip(self.dst, self.src))[1::2]:
            raw(d).copy_(raw(s))
        torch.add(raw(self.dst[1]), 0, out=raw(self.dst[1]))
        here.wait_stream(self.side)
        self.b.run()

    def forget(self):
        for d in self.dst:
            raw(d).zero_()
        self.b.o.fill_(7)
        self.b.lse.fill_(7)

    def check(self):
        b, o = self.b, self.o
        b.plan.device_status(b.ws)
        b.q, b.k, b.v, b.ks, b.vs = o.q, o.k, o.v, o.ks, o.vs
        b.check()


@pytest.mark.parametrize("new", [None, [60, 9, 200]])
@pytest.mark.parametrize("kw", KINDS)
def test_inputs_of_two_joined_streams(cuda_device, new, kw):
    x = Late(new, kw)
    if x.o.scales == "tensor":  # the plan's scales are arguments of the call
        x.b.k_scale, x.b.v_scale = x.o.k_scale, x.o.v_scale
    for _ in range(3):
        x.forget()
        x.step()
        x.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.step()
    for _ in range(3):
        x.forget()
        g.replay()
        x.check()


def test_pod_with_a_windowed_phase_captured(cuda_device):
    """Windowed decode on the POD call's side stream, in a graph, after writes of the cache on the caller's."""
    p = Batch([900, 45, 0, 300], [300, 45, 0, 1], num_ctas=60).upload()
    d = Batch([900, 45, 0, 300], window=200, sinks=3, num_ctas=60).upload()
    d.k, d.v, d.k_d, d.v_d, d.ids, d.ids_d, d.k_scale, d.v_scale = p.k, p.v, p.k_d, p.v_d, p.ids, p.ids_d, p.k_scale, p.v_scale
    keep_k, keep_v = p.k_d.clone(), p.v_d.clone()

    def step():
        torch.cuda._sleep(50000)
        raw(p.k_d).copy_(raw(keep_k))
        raw(p.v_d).copy_(raw(keep_v))
        torch.add(raw(p.v_d), 0, out=raw(p.v_d))
        pa.pafp8_run_pod(p.plan.handle, p.q_d, p.ids_d, p.o, p.lse, p.ws, d.plan.handle, d.q_d, d.ids_d, d.o, d.lse, d.ws, p.k_d, p.v_d,
                         k_scale=p.k_scale, v_scale=p.v_scale)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for t in (p.k_d, p.v_d):
            raw(t).zero_()
        for t in (p.o, p.lse, d.o, d.lse):
            t.fill_(7)
        g.replay()
        for x in (p, d):
            x.plan.device_status(x.ws)
            x.check()
