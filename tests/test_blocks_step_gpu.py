"""A server's steps over a cache with block scales and a sliding window: page
tables, norm + rotation into plain rows, the quantizing append, attention over
the cache, rows read back; and waits that expire in the new kernels."""
import numpy as np
import pytest
import torch

import paged_attention_fp8_gb300 as pa
from blocks_ref import TORCH, Cache, as_tokens, raw, table
from window_ref import OUT, Batch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Server:
    """Requests that grow: a pool with block scales, a block table and a free list on the device."""

    def __init__(self, batch, *, hq=8, hkv=2, d=128, kv="e4m3fn", layout="NHD", page_size=16, window=0, sinks=0, pool=160):
        self.hq, self.hkv, self.d, self.kv, self.layout, self.ps = hq, hkv, d, kv, layout, page_size
        self.window, self.sinks, self.pool, self.batch = window, sinks, pool, batch
        self.gen = torch.Generator().manual_seed(9)
        i = dict(dtype=torch.int32, device="cuda")
        shape = (pool, page_size, hkv, d) if layout == "NHD" else (pool, hkv, page_size, d)
        self.k, self.v = (torch.zeros(shape, device="cuda").to(TORCH[kv]) for _ in range(2))
        # The pool's scales are whatever was there: blocks without tokens are not read.
        self.ks, self.vs = (torch.full((pool, page_size // 16, hkv), float("nan"), device="cuda") for _ in range(2))
        self.table = torch.full((batch, pool), -1, **i)
        self.free = torch.randperm(pool, generator=self.gen).to(torch.int32).cuda()
        self.used, self.lens = torch.zeros(1, **i), [0] * batch
        ang = torch.rand(4096, d // 2, generator=self.gen, dtype=torch.float64) * 6.3
        self.cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
        self.w = (1 + 0.1 * torch.randn(d, generator=self.gen)).to(BF).cuda()
        zero = np.zeros((pool, page_size, hkv, d))
        self.rk, self.rv = (Cache(zero, np.ones((pool, page_size // 16, hkv)), kv) for _ in range(2))

    def step(self, new, mode, pad=0, stream=None):
        n, tokens = sum(new), sum(new) + pad
        pages = sum(-(-(c + m) // self.ps) for c, m in zip(self.lens, new))
        t = pa.StepTables(batch=self.batch, max_pages=pages + 1, max_tokens=tokens, page_size=self.ps, num_pages=self.pool)
        cached, fresh = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (self.lens, new))
        qkv = torch.randn(tokens, self.hq + 2 * self.hkv, self.d, generator=self.gen)
        qkv = (qkv * 2.0 ** torch.randint(-2, 3, (tokens, 1, 1), generator=self.gen)).to(BF).cuda()
        t.build(cached, fresh, self.table, self.free, self.used)
        self.used.copy_(t.free_used)
        # Norm and rotation into plain rows: a 2-byte pool whose slots are the tokens in order.
        rows = torch.zeros(-(-tokens // 16), 16, self.hkv, self.d, dtype=BF, device="cuda")
        vals, q = torch.zeros_like(rows), torch.zeros(tokens, self.hq, self.d, dtype=BF, device="cuda")
        order = torch.where(t.slots >= 0, torch.arange(tokens, device="cuda"), -1)
        pa.pafp8_norm_rope_append(qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.hkv], qkv[:, self.hq + self.hkv:], self.w, self.w,
                                  self.cs, t.positions, order, q, rows, vals)
        k_new, v_new = (x.view(-1, self.hkv, self.d)[:tokens] for x in (rows, vals))
        pa.pafp8_append_kv_blocks(k_new, v_new, t.qo_indptr, cached, t.kv_indptr, t.kv_indices, self.k, self.v, self.ks, self.vs,
                                  kv_layout=self.layout, status=t.status)
        lens = [c + m for c, m in zip(self.lens, new)]
        b = Batch.__new__(Batch)
        b.lens, b.new, b.hq, b.hkv, b.d, b.ps = lens, new if mode == "prefill" else None, self.hq, self.hkv, self.d, self.ps
        b.kv_type, b.window, b.sinks, b.scales, b.qs, b.q_scale, b.sm_scale = self.kv, self.window, self.sinks, "block", None, 1.0, self.d ** -0.5
        b.o_type, b.rows = OUT["bf16"], np.concatenate([[0], np.cumsum(new)])
        plan = pa.Plan(mode=mode, num_qo_heads=self.hq, num_kv_heads=self.hkv, num_pages=self.pool, q_dtype="bf16", kv_dtype=self.kv,
                       kv_indptr=np.concatenate([[0], np.cumsum([-(-x // self.ps) for x in lens])]),
                       last_page_len=[x - (-(-x // self.ps) - 1) * self.ps if x else 0 for x in lens],
                       qo_indptr=b.rows if mode == "prefill" else None, head_dim=self.d, page_size=self.ps, kv_layout=self.layout,
                       window=self.window, sinks=self.sinks)
        ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        plan.upload(ws)
        o, lse = torch.zeros(n, self.hq, self.d, dtype=BF, device="cuda"), torch.zeros(n, self.hq, device="cuda")
        plan.run_block_scales(q[:n], self.k, self.v, t.kv_indices, o, lse, ws, k_scales=self.ks, v_scales=self.vs)
        torch.cuda.synchronize()
        plan.device_status(ws)
        assert int(t.status) == 0
        # The cache, number for number, then the attention over it.
        ptr, ids = t.kv_indptr.cpu().numpy(), t.kv_indices.cpu().numpy()
        for ref, x in ((self.rk, k_new), (self.rv, v_new)):
            ref.append(x.double().cpu().numpy(), b.rows, self.lens, ptr, ids)
        self.lens = lens
        b.ptr, b.ids, b.q = ptr, ids, q[:n].cpu()
        b.k, b.v = (x.cpu() if self.layout == "NHD" else raw(x.cpu()).transpose(1, 2).contiguous().view(x.dtype) for x in (self.k, self.v))
        b.ks, b.vs = self.ks.cpu(), self.vs.cpu()
        b.check(o, lse)
        self.t, self.b = t, b
        return t

    def check_cache(self):
        used = np.unique(self.b.ids[:self.b.ptr[-1]])
        for got, scales, ref in ((self.k, self.ks, self.rk), (self.v, self.vs, self.rv)):
            got, scales = as_tokens(got, self.layout), scales.double().cpu().numpy()
            for b, n in enumerate(self.lens):
                pos = np.arange(n)
                page, slot = self.b.ids[self.b.ptr[b] + pos // self.ps], pos % self.ps
                np.testing.assert_array_equal(got[page, slot], ref.values[page, slot])
                np.testing.assert_array_equal(scales[page, slot // 16], ref.scales[page, slot // 16])
        free = np.setdiff1d(np.arange(self.pool), used)
        assert np.isnan(self.ks.cpu().numpy()[free]).all() and not as_tokens(self.k, self.layout)[free].any()

    def check_read(self):
        """Every request's tokens in plain rows: the reference's numbers times its scales, exactly (powers of two)."""
        n = sum(self.lens)
        ptr = torch.tensor(np.concatenate([[0], np.cumsum(self.lens)]), dtype=torch.int32, device="cuda")
        ko, vo = (torch.zeros(n, self.hkv, self.d, device="cuda") for _ in range(2))
        pa.pafp8_read_kv(self.k, self.v, ptr, torch.zeros(self.batch, dtype=torch.int32, device="cuda"), self.t.kv_indptr,
                         self.t.kv_indices, ko, vo, k_scales=self.ks, v_scales=self.vs, kv_layout=self.layout, status=self.t.status)
        assert int(self.t.status) == 0
        for out, ref in ((ko, self.rk), (vo, self.rv)):
            want = []
            for b, m in enumerate(self.lens):
                pos = np.arange(m)
                page, slot = self.b.ids[self.b.ptr[b] + pos // self.ps], pos % self.ps
                want.append(ref.values[page, slot] * ref.scales[page, slot // 16][:, :, None])
            np.testing.assert_array_equal(out.double().cpu().numpy(), np.concatenate(want))


@pytest.mark.parametrize("kw", [
    dict(batch=4, window=60, sinks=5), dict(batch=3, d=64, hq=12, hkv=3, kv="e5m2", layout="HND", page_size=32, window=33, sinks=0),
    dict(batch=2, hq=4, hkv=1, page_size=48)])
def test_prompts_then_tokens(cuda_device, kw):
    s = Server(**kw)
    n = kw["batch"]
    s.step([70, 1, 130, 17][:n], "prefill")
    for _ in range(18):
        s.step([1] * n, "decode")
    s.step([5, 20, 1, 3][:n], "prefill", pad=6)  # a padded batch
    s.step([1] * n, "decode")
    s.check_cache()
    s.check_read()


def test_two_batches_on_two_streams(cuda_device):
    bs = [Batch([500 + 9 * i for i in range(20)], window=200, sinks=6, scales="block", num_ctas=30).upload(),
          Batch([700, 33], [300, 20], window=150, sinks=9, scales="block", num_ctas=30).upload()]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, st in zip(bs, streams):
            b.run(stream=st)
    torch.cuda.synchronize()
    for b in bs:
        b.plan.device_status(b.ws)
        b.check()


@pytest.mark.parametrize("new", [None, [90, 33, 200]])
@pytest.mark.parametrize("scales", ["tensor", "block"])
def test_each_call_sees_the_work_before_it(cuda_device, scales, new):
    """The attention kernels launch early and waits in the kernel: every input is rewritten right before a call -- by copies, kernels and
    the append -- and right after it, eager and captured with the plan's upload, forty times over one workspace."""
    bs = [Batch([700, 33, 260], new, window=300, sinks=5, scales=scales, num_ctas=40, seed=i).upload() for i in range(2)]
    a = bs[0]
    want = []
    for b in bs:
        b.run()
        b.check()
        want.append((raw(b.o).clone(), b.lse.clone()))
    held = [[raw(t).clone() for t in (b.q_d, b.k_d, b.v_d)] + [b.ids_d.clone()] +
            ([b.ks_d.clone(), b.vs_d.clone()] if scales == "block" else []) for b in bs]
    into = [raw(a.q_d), raw(a.k_d), raw(a.v_d), a.ids_d] + ([a.ks_d, a.vs_d] if scales == "block" else [])
    scal = [(b.k_scale, b.v_scale) if scales == "tensor" else (1.0, 1.0) for b in bs]
    got = []

    def step(i):
        for x, y in zip(into, held[i]):
            x.copy_(y)
        if scales == "tensor":
            a.k_scale, a.v_scale = scal[i]
        a.run()
        out = raw(a.o).clone(), a.lse.clone()
        for x in into[:1] + into[3:4]:
            x.zero_()
        a.o.fill_(7)
        return out

    for k in range(40):
        got.append((k % 2, *step(k % 2)))
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(0)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    outs = []
    with torch.cuda.graph(g):
        for k in range(6):
            a.plan.upload(a.ws)
            outs.append((k % 2, *step(k % 2)))
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        got += [(i, o.clone(), l.clone()) for i, o, l in outs]
    torch.cuda.synchronize()
    for i, o, l in got:
        assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


@pytest.mark.parametrize("kw", [
    dict(lens=[9000, 40], scales="block"), dict(lens=[9000, 40], window=8000, sinks=4), dict(lens=[300, 60], new=[129, 40], scales="block"),
    dict(lens=[300, 60], new=[129, 40], scales="block", q="e4m3fn", window=100, sinks=4),
    dict(lens=[300, 60], new=[129, 40], window=100, sinks=4), dict(lens=[1900], new=[300], window=800, sinks=4, q="bf16", kv="bf16")])
def test_expired_wait_is_reported_and_the_next_run_is_clean(cuda_device, monkeypatch, kw):
    """(Decode: 60 pages and more a block, through a ring of 8, so that its producer has to wait for a page's use.)"""
    b = Batch(num_ctas=8, **kw).upload()
    monkeypatch.delenv("PAFP8_DEBUG", raising=False)
    monkeypatch.setenv("PAFP8_WAIT_CYCLES", "1")
    b.run()
    with pytest.raises(pa.Pafp8Error) as e:
        b.plan.device_status(b.ws)
    assert e.value.status == 6
    monkeypatch.delenv("PAFP8_WAIT_CYCLES")
    b.o.fill_(float("nan"))
    b.lse.fill_(float("nan"))
    b.run()
    b.plan.device_status(b.ws)
    b.check()


def test_appends_and_reads_one_after_the_other(cuda_device):
    """Both launch early and wait in the kernel: forty rounds of new rows (written right before the call and over right after
    it), the append and the read-back of the whole cache, against rows kept aside."""
    g = torch.Generator().manual_seed(3)
    lens, hkv, d = [130, 47, 64], 2, 128
    ptr, ids, pool = table(lens, 16, g)
    i32 = dict(dtype=torch.int32, device="cuda")
    ptr_d, ids_d = torch.as_tensor(ptr, **i32), torch.as_tensor(ids, **i32)
    rows = torch.as_tensor(np.concatenate([[0], np.cumsum(lens)]), **i32)
    zero = torch.zeros(3, **i32)
    n = sum(lens)
    kc, vc = (torch.zeros(pool, 16, hkv, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.ones(pool, 1, hkv, device="cuda") for _ in range(2))
    # Numbers of few bits, so that a code holds them exactly under their block's power of two.
    kept = [(torch.randint(-7, 8, (n, hkv, d), generator=g).float() * 2.0 ** (i % 5)).to(torch.bfloat16).cuda() for i in range(8)]
    x, y = torch.zeros_like(kept[0]), torch.zeros_like(kept[0])
    a, b = torch.zeros_like(x), torch.zeros_like(x)
    got = []
    for i in range(40):
        x.copy_(kept[i % 8])
        y.copy_(kept[(i + 3) % 8])
        pa.pafp8_append_kv_blocks(x, y, rows, zero, ptr_d, ids_d, kc, vc, ks, vs)
        x.fill_(float("nan"))
        y.fill_(float("nan"))
        pa.pafp8_read_kv(kc, vc, rows, zero, ptr_d, ids_d, a, b, k_scales=ks, v_scales=vs)
        got.append((a.clone(), b.clone()))
        a.fill_(7)
        b.fill_(7)
    for i, (p, q) in enumerate(got):
        assert torch.equal(p, kept[i % 8]) and torch.equal(q, kept[(i + 3) % 8])
