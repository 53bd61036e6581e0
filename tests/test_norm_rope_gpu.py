"""pafp8_norm_rope_append against the formulas in float64."""
import pytest
import torch

import paged_attention_fp8_gb300 as pa
from step_ref import FP8_MAX, assert_rounded, norm_rope

pytestmark = pytest.mark.gpu
E4, E5, BF, HF = torch.float8_e4m3fn, torch.float8_e5m2, torch.bfloat16, torch.float16


def _scale(dt, amax):
    return amax / FP8_MAX[dt] if dt in FP8_MAX else 1.0


class Case:
    def __init__(self, n, hq, hkv, d, src, kv, q_out, layout="NHD", page_size=16, axes=1, rot=None, interleaved=False,
                 norm="qk", packed=True, seed=0, std=1.5):
        g = torch.Generator().manual_seed(seed)
        rot = d if rot is None else rot
        self.n, self.hq, self.hkv, self.d, self.layout, self.ps = n, hq, hkv, d, layout, page_size
        self.interleaved, self.rot, self.eps = interleaved, rot, 1e-5
        x = (torch.randn(n, hq + 2 * hkv, d, generator=g) * std).to(src)
        self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        dev = x.cuda()
        if packed:
            self.dq, self.dk, self.dv = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
        else:
            self.dq, self.dk, self.dv = (t.contiguous() for t in (dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]))
        w = lambda: (1 + 0.3 * torch.randn(d, generator=g)).to(src)  # noqa: E731
        self.qw, self.kw = (w() if "q" in norm else None), (w() if "k" in norm else None)
        limit = 513
        ang = torch.rand(limit, rot // 2, generator=g, dtype=torch.float64) * 6.3
        self.cs = torch.cat([ang.cos(), ang.sin()], 1).float()
        self.pos = torch.randint(0, limit, (axes, n), generator=g, dtype=torch.int32)
        self.axis = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.uint8)
        pages = -(-n // page_size) + 3
        self.slots = torch.randperm(pages * page_size, generator=g)[:n].contiguous()
        shape = (pages, page_size, hkv, d) if layout == "NHD" else (pages, hkv, page_size, d)
        size = {1: torch.uint8, 2: torch.int16}[torch.empty(0, dtype=kv).element_size()]
        self.fill = [torch.randint(0, 100, shape, generator=g).to(size) for _ in range(2)]
        self.kc, self.vc = (f.cuda().view(kv) for f in self.fill)
        self.size, self.kv = size, kv
        self.ks, self.vs, self.qs = _scale(kv, 3.9), _scale(kv, 4.1), _scale(q_out, 4.3)
        self.out = torch.full((n, hq, d), 7.0).to(q_out).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, **kw):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        args = dict(pair_axis=c(self.axis) if self.pos.shape[0] > 1 else None, interleaved=self.interleaved, eps=self.eps,
                    q_scale=self.qs, k_scale=self.ks, v_scale=self.vs, kv_layout=self.layout, status=self.status)
        args.update(kw)
        pos = self.pos if self.pos.shape[0] > 1 else self.pos[0]
        pa.pafp8_norm_rope_append(self.dq, self.dk, self.dv, c(self.qw), c(self.kw), c(self.cs), c(pos), c(self.slots),
                                  self.out, self.kc, self.vc, **args)
        torch.cuda.synchronize()

    def rows(self, cache):
        """(rows at the tokens' slots, all other bytes, the filler's other bytes)."""
        flat = cache.cpu().view(self.size)
        if self.layout == "HND":
            flat = flat.transpose(1, 2)
        return flat.reshape(-1, self.hkv, self.d)

    def check(self, rows=None):
        axis = self.axis if self.pos.shape[0] > 1 else torch.zeros_like(self.axis)
        keep = torch.ones(self.n, dtype=torch.bool) if rows is None else rows
        q, qm = norm_rope(self.q, self.qw, self.eps, self.cs, self.pos, axis, self.interleaved)
        k, km = norm_rope(self.k, self.kw, self.eps, self.cs, self.pos, axis, self.interleaved)
        v = self.v.double()
        raw = self.out.cpu().view(torch.uint8).view(self.n, self.hq, -1)  # fp8 tensors cannot be indexed on the CPU
        assert_rounded(raw[keep].view(self.out.dtype), q[keep], qm[keep], self.qs, "q")
        for cache, fill, ref, mag, s, what in ((self.kc, self.fill[0], k, km, self.ks, "k"),
                                               (self.vc, self.fill[1], v, v.abs(), self.vs, "v")):
            got, was = self.rows(cache), self.rows(fill)
            at = self.slots[keep]
            assert_rounded(got[at].contiguous().view(self.kv), ref[keep], mag[keep], s, what)
            rest = torch.ones(got.shape[0], dtype=torch.bool)
            rest[at] = False
            assert torch.equal(got[rest], was[rest]), f"{what}: rows of no token were written"


@pytest.mark.parametrize("kw", [
    dict(n=1, hq=1, hkv=1, d=128, src=BF, kv=E4, q_out=BF), dict(n=1, hq=32, hkv=8, d=128, src=BF, kv=E4, q_out=BF),
    dict(n=37, hq=8, hkv=2, d=128, src=BF, kv=E4, q_out=BF, packed=False),
    dict(n=64, hq=32, hkv=8, d=128, src=HF, kv=E5, q_out=HF), dict(n=33, hq=7, hkv=7, d=64, src=BF, kv=BF, q_out=BF),
    dict(n=50, hq=28, hkv=4, d=128, src=HF, kv=HF, q_out=E4), dict(n=131, hq=5, hkv=1, d=64, src=HF, kv=E4, q_out=E5),
    dict(n=9, hq=70, hkv=14, d=128, src=BF, kv=E4, q_out=BF), dict(n=2500, hq=2, hkv=1, d=128, src=BF, kv=E4, q_out=BF)])
@pytest.mark.parametrize("variant", [dict(), dict(interleaved=True, layout="HND", page_size=32),
                                     dict(axes=3, norm="k", page_size=48), dict(axes=2, rot=32, interleaved=True, norm=""),
                                     dict(rot=48, norm="q", layout="HND")])
def test_against_the_formulas(cuda_device, kw, variant):
    c = Case(**{**kw, **variant}, seed=kw["n"])
    c.run()
    c.check()
    assert int(c.status) == 0


def test_padding_bad_slots_and_bad_positions(cuda_device):
    c = Case(n=40, hq=8, hkv=2, d=128, src=BF, kv=E4, q_out=BF)
    pages = c.kc.shape[0]
    before = c.out.clone()
    c.slots[5] = c.slots[17] = -1          # padding
    c.run()
    assert int(c.status) == 0
    keep = torch.ones(40, dtype=torch.bool)
    keep[[5, 17]] = False
    c.check(keep)
    assert torch.equal(c.out[[5, 17]], before[[5, 17]])
    for slot in (pages * 16, -2, 1 << 40):  # outside the pool: the query alone
        c = Case(n=40, hq=8, hkv=2, d=128, src=BF, kv=E4, q_out=BF)
        c.slots[7] = slot
        c.run()
        assert int(c.status) == 1
        keep = torch.ones(40, dtype=torch.bool)
        keep[7] = False
        c.check(keep)
        assert not torch.equal(c.out[7].cpu(), before[7].cpu())
    for pos in (-1, 513):                    # outside the table: nothing
        c = Case(n=40, hq=8, hkv=2, d=128, src=BF, kv=E4, q_out=BF, axes=3)
        c.pos[1, 30] = pos
        c.run()
        assert int(c.status) == 1
        keep = torch.ones(40, dtype=torch.bool)
        keep[30] = False
        c.pos[1, 30] = 0
        c.check(keep)
        assert torch.equal(c.out[30], before[30])


def test_query_in_place_and_empty(cuda_device):
    c = Case(n=21, hq=4, hkv=2, d=64, src=HF, kv=E4, q_out=HF, packed=False)
    c.out = c.dq
    c.run()
    c.check()
    none = torch.empty(0, 4, 64, dtype=HF, device="cuda")
    kv = torch.empty(0, 2, 64, dtype=HF, device="cuda")
    pa.pafp8_norm_rope_append(none, kv, kv, None, None, c.cs.cuda(), torch.empty(0, dtype=torch.int32, device="cuda"),
                              torch.empty(0, dtype=torch.int64, device="cuda"), none, c.kc, c.vc, k_scale=c.ks, v_scale=c.vs)


def test_zero_rows_large_values_and_other_streams(cuda_device):
    c = Case(n=6, hq=4, hkv=2, d=128, src=BF, kv=E4, q_out=BF, packed=False)
    for t in (c.q, c.k):
        t[0] = 0
        t[1] *= 2.0 ** 50   # the sum of squares stays below fp32's largest value
        t[2] *= 2.0 ** -50  # eps decides
    c.v[3] *= 1e6           # saturates
    c.dq, c.dk, c.dv = c.q.contiguous().cuda(), c.k.contiguous().cuda(), c.v.contiguous().cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run()
    c.check()


def test_byte_equal_to_append_kv(cuda_device):
    """With the identity rotation and no norm the caches are pafp8_append_kv's."""
    c = Case(n=100, hq=8, hkv=8, d=128, src=BF, kv=E4, q_out=BF, norm="", page_size=32, layout="HND")
    c.cs[:, :64], c.cs[:, 64:] = 1.0, 0.0
    c.run()
    pages = c.kc.shape[0]
    kc, vc = (f.cuda().view(E4) for f in c.fill)
    ident = torch.arange(pages, dtype=torch.int32, device="cuda")
    pa.pafp8_append_kv(c.dk.contiguous(), c.dv.contiguous(), torch.zeros(100, dtype=torch.int32, device="cuda"),
                       c.slots.int().cuda(), torch.tensor([0, pages], dtype=torch.int32, device="cuda"), ident, kc, vc,
                       k_scale=c.ks, v_scale=c.vs, kv_layout="HND")
    assert torch.equal(kc.view(torch.uint8), c.kc.view(torch.uint8))
    assert torch.equal(vc.view(torch.uint8), c.vc.view(torch.uint8))


@pytest.mark.parametrize("variant", [dict(), dict(axes=3, layout="HND", page_size=48), dict(rot=32, interleaved=True, hq=9)])
def test_skipped_tokens_among_many(cuda_device, variant):
    """More tokens than blocks: what a skipped token leaves must not reach the next one of its block."""
    c = Case(**{**dict(n=6001, hq=3, hkv=1, d=128, src=BF, kv=E4, q_out=BF, seed=3), **variant})
    before = c.out.clone()
    skip = torch.arange(6001) % 7 == 2
    lost = torch.arange(6001) % 11 == 5
    c.slots[skip] = -1
    good = c.pos.clone()
    c.pos[0, lost] = 513
    c.run()
    c.pos = good
    c.check(~(skip | lost))
    assert int(c.status) == 1 and torch.equal(c.out[(skip | lost).cuda()], before[(skip | lost).cuda()])
