"""The append that gives every 16-token block and head a scale, and the read-back,
against their definitions in 64 bits, number for number: scales are powers of
two, so products with them are exact and every code has one right value."""
import numpy as np
import pytest
import torch

import paged_attention_fp8_gb300 as pa
from blocks_ref import BLOCK, TOP, TORCH, Cache, as_tokens, in_layout, random_cache, raw, table

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Setup:
    """A pool with cached tokens, its page table and reference caches; rows come per step."""

    def __init__(self, lens, *, heads=3, d=128, fmt="e4m3fn", layout="NHD", page_size=16, seed=0, spare=3):
        self.gen = torch.Generator().manual_seed(seed)
        self.heads, self.d, self.fmt, self.layout, self.ps = heads, d, fmt, layout, page_size
        self.ptr, self.ids, self.pool = table(lens, page_size, self.gen, spare)
        self.k, self.ks = random_cache(self.pool, page_size, heads, d, fmt, self.gen)
        self.v, self.vs = random_cache(self.pool, page_size, heads, d, fmt, self.gen)
        self.rk, self.rv = Cache(self.k.double(), self.ks, fmt), Cache(self.v.double(), self.vs, fmt)
        self.k, self.v = (in_layout(x, layout).cuda() for x in (self.k, self.v))
        self.ks, self.vs = self.ks.cuda(), self.vs.cuda()
        self.ptr_d, self.ids_d = ints(self.ptr), ints(self.ids)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def rows(self, n, src, packed=False, big=1.0):
        x = torch.randn(n, 2, self.heads, self.d, generator=self.gen) * big
        x = (x * 2.0 ** torch.randint(-5, 6, (n, 2, 1, 1), generator=self.gen)).to(TORCH[src]).cuda()
        return (x[:, 0], x[:, 1]) if packed else (x[:, 0].contiguous(), x[:, 1].contiguous())

    def append(self, k, v, qo, cached, stream=None):
        pa.pafp8_append_kv_blocks(k, v, qo, cached, self.ptr_d, self.ids_d, self.k, self.v, self.ks, self.vs,
                                  kv_layout=self.layout, status=self.status, stream=stream)

    def expect(self, k, v, qo, cached):
        for ref, x in ((self.rk, k), (self.rv, v)):
            ref.append(x.double().cpu().numpy(), qo, cached, self.ptr, self.ids)

    def check(self, status=0):
        assert int(self.status) == status
        for got, scales, ref in ((self.k, self.ks, self.rk), (self.v, self.vs, self.rv)):
            np.testing.assert_array_equal(scales.double().cpu().numpy(), ref.scales)
            np.testing.assert_array_equal(as_tokens(got, self.layout), ref.values)


CASES = [
    # cached, new: one token, block borders on both sides, requests without new tokens, long ones
    ([0], [1]), ([5], [1]), ([15], [1]), ([16], [1]), ([15], [2]), ([31], [33]), ([0, 7, 16, 40], [16, 0, 17, 5]),
    ([3, 0, 90, 1, 1], [0, 0, 200, 1, 0]), ([100] * 9, [1] * 9), ([0, 0], [0, 0]), ([12, 700], [321, 77])]


@pytest.mark.parametrize("cached,new", CASES)
@pytest.mark.parametrize("heads,d,fmt,layout,page_size,src,packed", [
    (3, 128, "e4m3fn", "NHD", 16, "bf16", True), (2, 64, "e5m2", "HND", 48, "f16", False),
    (1, 128, "e5m2", "NHD", 64, "f32", True), (5, 64, "e4m3fn", "HND", 16, "f32", False), (8, 128, "e4m3fn", "HND", 32, "bf16", False)])
def test_one_step(cuda_device, cached, new, heads, d, fmt, layout, page_size, src, packed):
    s = Setup([c + n for c, n in zip(cached, new)], heads=heads, d=d, fmt=fmt, layout=layout, page_size=page_size)
    qo = np.concatenate([[0], np.cumsum(new)])
    k, v = s.rows(int(qo[-1]), src, packed)
    s.append(k, v, ints(qo), ints(cached))
    s.expect(k, v, qo, cached)
    s.check()


@pytest.mark.parametrize("batch,low,high", [(40, 1, 8), (300, 1, 3), (300, 4, 7), (300, 8, 15), (120, 16, 40)])
@pytest.mark.parametrize("src", ["bf16", "f32"])
def test_requests_of_like_lengths(cuda_device, batch, low, high, src):
    """Requests of like lengths: a warp looks through 1, 2, 4, 8 or 16 tokens, with borders of requests and blocks anywhere in them."""
    gen = np.random.default_rng(batch + high)
    cached, new = gen.integers(0, 50, batch), gen.integers(low, high + 1, batch)
    s = Setup(cached + new, heads=4, seed=high)
    qo = np.concatenate([[0], np.cumsum(new)])
    k, v = s.rows(int(qo[-1]), src)
    s.append(k, v, ints(qo), ints(cached))
    s.expect(k, v, qo, cached)
    s.check()


@pytest.mark.parametrize("fmt,layout", [("e4m3fn", "NHD"), ("e5m2", "HND")])
def test_token_by_token_while_values_grow_and_shrink(cuda_device, fmt, layout):
    """Forty steps of one token: a block's scale follows its largest value, its earlier codes are written anew."""
    s = Setup([40, 53], fmt=fmt, layout=layout, page_size=32)
    for t in range(40):
        k, v = s.rows(2, "bf16", big=2.0 ** [0, 9, -9, 3, 14][t % 5])
        s.append(k, v, ints([0, 1, 2]), ints([t, t + 13]))
        s.expect(k, v, [0, 1, 2], [t, t + 13])
    s.check()


def test_a_token_written_again(cuda_device):
    """A rejected draft's positions are written by a later step: the block keeps the larger scale."""
    s = Setup([60])
    for at, n, big in ((20, 9, 1e4), (22, 3, 1.0), (20, 1, 1e-3), (16, 20, 1e-2)):
        k, v = s.rows(n, "bf16", big=big)
        s.append(k, v, ints([0, n]), ints([at]))
        s.expect(k, v, [0, n], [at])
        s.check()


@pytest.mark.parametrize("fmt,src", [("e4m3fn", "f32"), ("e5m2", "bf16")])
def test_scales_that_are_not_powers_of_two(cuda_device, fmt, src):
    """A cache whose blocks have other scales (another writer's): a larger one is kept, a smaller one grows to a power of two."""
    s = Setup([16 * i + 9 for i in range(60)], fmt=fmt)
    for t, ref in ((s.ks, s.rk), (s.vs, s.rv)):
        t.mul_(1 + torch.rand(t.shape, generator=s.gen).cuda())
        ref.scales = t.double().cpu().numpy()
    cached = [16 * i + 5 for i in range(60)]
    k, v = s.rows(240, src, big=8.0)
    s.append(k, v, ints(np.arange(0, 241, 4)), ints(cached))
    s.expect(k, v, np.arange(0, 241, 4), cached)
    s.check()
    frac = np.frexp(np.stack([s.rk.scales[s.ids[s.ptr[b] + b], 0] for b in range(60)]))[0]
    assert (frac != 0.5).any() and (frac == 0.5).any()  # both happened


@pytest.mark.parametrize("fmt", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
def test_special_values(cuda_device, fmt, src):
    """Zeros, NaN, infinities, the type's largest and smallest numbers, and the border between two scales."""
    s = Setup([16 * 14], heads=1, fmt=fmt)
    x = torch.zeros(16 * 14, 1, 128)
    inf, nan = float("inf"), float("nan")
    top = torch.finfo(TORCH[src]).max
    tiny = torch.finfo(TORCH[src]).smallest_normal
    x[16, 0, 0] = nan                                   # block 1: NaN alone
    x[32, 0, 1], x[33, 0, 2] = inf, -inf                # block 2: infinities alone
    x[48, 0, 0], x[49, 0, 5], x[50, 0, 6] = 3.0, nan, -inf
    x[64, 0, 0], x[65, 0, 1] = top, -top
    x[80, 0, 0], x[81, 0, 1] = tiny, -tiny / 2
    x[96, 0, 3] = 1.75                                  # the largest value at its scale
    x[112, 0, 3] = 1.7578125 if src != "f32" else 1.75 + 2.0 ** -22  # a little more: the next scale
    x[128:144, 0] = -0.0
    x[144:160, 0] = torch.linspace(-500, 500, 16 * 128).view(16, 128)
    x[160, 0, 0], x[161, 0, 1] = 2.0 ** -64 * TOP[fmt] if src == "f32" else 0.0, 2.0 ** -66 if src == "f32" else 0.0
    x[176:192, 0] = 2.0 ** -9 * torch.arange(16 * 128).view(16, 128).float() / 7
    x = x.to(TORCH[src]).cuda()
    s.append(x, x, ints([0, len(x)]), ints([0]))
    s.expect(x, x, [0, len(x)], [0])
    s.check()
    codes = as_tokens(s.k, "NHD")[s.ids[8], :, 0]
    assert np.all(codes == 0) and np.all(np.signbit(codes))  # -0 keeps its sign


def test_padded_rows_and_slots_behind_stay(cuda_device):
    """Rows from qo_indptr[batch] on are not read (they hold NaN here), other pages and slots not written."""
    s = Setup([21, 3])
    before = raw(s.k).clone()
    k, v = s.rows(12, "bf16")
    k[7:], v[7:] = float("nan"), float("nan")
    s.append(k, v, ints([0, 4, 7]), ints([17, 0]))
    s.expect(k, v, [0, 4, 7], [17, 0])
    s.check()
    free = np.setdiff1d(np.arange(s.pool), s.ids)
    assert torch.equal(raw(s.k)[free], before[free])


def test_what_lies_outside_is_skipped_and_reported(cuda_device):
    s = Setup([64, 20, 30], spare=0)
    ids = s.ids.copy()
    ids[s.ptr[0] + 1] = s.pool  # request 0's second page is not in the pool
    s.ids_d = ints(ids)
    k, v = s.rows(34, "bf16")
    # Request 0: tokens 10 .. 39, of which 16 .. 31 have no page; 1: a negative length; 2: past its table's end.
    qo = [0, 30, 32, 34]
    s.append(k, v, ints(qo), ints([10, -3, 31]))
    for ref, x in ((s.rk, k), (s.rv, v)):
        x = x.double().cpu().numpy()
        ref.append(x[:6], [0, 6], [10], s.ptr, s.ids)
        ref.append(x[22:30], [0, 8], [32], s.ptr, s.ids)
        ref.append(x[32:33], [0, 1], [31], s.ptr[2:], s.ids)
    s.check(status=1)


def test_more_rows_said_than_there_are(cuda_device):
    s = Setup([50])
    k, v = s.rows(20, "bf16")
    s.append(k, v, ints([0, 40]), ints([3]))
    s.expect(k, v, [0, 20], [3])
    s.check(status=1)


def test_many_requests(cuda_device):
    """More requests than one step of the search looks at, tokens spread unevenly."""
    new = [(7 * i) % 5 for i in range(1500)]
    cached = [(11 * i) % 37 for i in range(1500)]
    s = Setup([c + n for c, n in zip(cached, new)], heads=1, d=64)
    qo = np.concatenate([[0], np.cumsum(new)])
    k, v = s.rows(int(qo[-1]), "bf16")
    s.append(k, v, ints(qo), ints(cached))
    s.expect(k, v, qo, cached)
    s.check()


def test_captured_with_other_lengths_and_on_another_stream(cuda_device):
    s = Setup([200, 200])
    k, v = s.rows(40, "bf16")
    qo, cached = ints([0, 3, 5]), ints([0, 0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.append(k, v, qo, cached)
    torch.cuda.current_stream().wait_stream(side)
    s.expect(k, v, [0, 3, 5], [0, 0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.append(k, v, qo, cached)
    for lens, at in (([0, 30, 40], [3, 2]), ([0, 0, 1], [33, 12]), ([0, 16, 17], [48, 13])):
        qo.copy_(ints(lens))
        cached.copy_(ints(at))
        k2, v2 = s.rows(40, "bf16", big=4.0)
        k.copy_(k2)
        v.copy_(v2)
        g.replay()
        s.expect(k, v, lens, at)
        s.check()


def test_pages_past_two_gib(cuda_device):
    """A pool of more than 2^31 codes and the pages at its end."""
    heads, d, pool = 8, 128, 140000
    k = torch.zeros(pool, 16, heads, d, dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.zeros_like(k)
    ks, vs = (torch.ones(pool, 1, heads, device="cuda") for _ in range(2))
    ids = [pool - 1, 7, pool - 2]
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(40, 2, heads, d, generator=gen).to(torch.bfloat16).cuda()
    pa.pafp8_append_kv_blocks(x[:, 0], x[:, 1], ints([0, 40]), ints([0]), ints([0, 3]), ints(ids), k, v, ks, vs)
    zero = np.zeros((3, 16, heads, d))
    for got, scales, rows in ((k, ks, x[:, 0]), (v, vs, x[:, 1])):
        ref = Cache(zero, np.ones((3, 1, heads)), "e4m3fn")
        ref.append(rows.double().cpu().numpy(), [0, 40], [0], [0, 3], [0, 1, 2])
        at = torch.tensor(ids, device="cuda")
        np.testing.assert_array_equal(got.view(torch.uint8)[at].view(got.dtype).double().cpu().numpy(), ref.values)
        np.testing.assert_array_equal(scales[at].double().cpu().numpy(), ref.scales)
    out = torch.zeros(40, heads, d, device="cuda")
    out2 = torch.zeros_like(out)
    pa.pafp8_read_kv(k, v, ints([0, 40]), ints([0]), ints([0, 3]), ints(ids), out, out2, k_scales=ks, v_scales=vs)
    got = k.view(torch.uint8)[torch.tensor(ids, device="cuda")].view(k.dtype).float().view(48, heads, d)[:40]
    assert torch.equal(out, got * ks[torch.tensor(ids, device="cuda")].repeat_interleave(16, 0).view(48, heads, 1)[:40])


# ---- reading back: one fp32 product rounded once, so torch's own arithmetic is the reference, bit for bit

def read_ref(s, which, starts, counts, scale=None):
    cache, scales = (s.k, s.ks) if which == "k" else (s.v, s.vs)
    tok = torch.from_numpy(np.ascontiguousarray(as_tokens(cache, s.layout))).float()
    by = scales.cpu().repeat_interleave(BLOCK, 1)[..., None] if scale is None else torch.tensor(scale, dtype=torch.float32)
    val = (tok * by).view(-1, s.heads, s.d)
    out = []
    for b, (a, n) in enumerate(zip(starts, counts)):
        pos = np.arange(a, a + n)
        out.append(val[s.ids[s.ptr[b] + pos // s.ps] * s.ps + pos % s.ps])
    return torch.cat(out)


@pytest.mark.parametrize("starts,counts", [([0], [1]), ([15], [2]), ([0, 3, 0, 20], [40, 0, 16, 17]), ([1] * 40, [3] * 40),
                                           ([0, 511], [500, 1300])])
@pytest.mark.parametrize("heads,d,fmt,layout,page_size,out,blocks", [
    (3, 128, "e4m3fn", "NHD", 16, "bf16", True), (2, 64, "e5m2", "HND", 48, "f16", True), (8, 128, "e4m3fn", "HND", 32, "f32", True),
    (1, 64, "e4m3fn", "NHD", 64, "bf16", False), (5, 128, "e5m2", "NHD", 16, "f32", False)])
def test_read_back(cuda_device, starts, counts, heads, d, fmt, layout, page_size, out, blocks):
    s = Setup([a + n for a, n in zip(starts, counts)], heads=heads, d=d, fmt=fmt, layout=layout, page_size=page_size)
    if blocks:  # any scales, not powers of two alone
        s.ks.mul_(1 + torch.rand(s.ks.shape, device="cuda"))
        s.vs.mul_(1 + torch.rand(s.vs.shape, device="cuda"))
    n = sum(counts)
    ko, vo = (torch.full((n + 5, heads, d), 7.0, dtype=TORCH[out], device="cuda") for _ in range(2))
    kw = dict(k_scales=s.ks, v_scales=s.vs) if blocks else dict(k_scale=0.37, v_scale=1.9)
    pa.pafp8_read_kv(s.k, s.v, ints(np.concatenate([[0], np.cumsum(counts)])), ints(starts), s.ptr_d, s.ids_d, ko, vo,
                     kv_layout=layout, status=s.status, **kw)
    assert int(s.status) == 0
    for got, name, sc in ((ko, "k", 0.37), (vo, "v", 1.9)):
        ref = read_ref(s, name, starts, counts, None if blocks else sc).to(TORCH[out])
        assert torch.equal(raw(got[:n].cpu()), raw(ref))
        assert bool((got[n:] == 7).all())  # rows behind the last request's


def test_read_of_nan_and_infinite_codes(cuda_device):
    s = Setup([16], fmt="e5m2", heads=1)
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(8)
    raw(s.k).view(-1)[int(s.ids[0]) * 2048:][:2048] = codes
    ko, vo = (torch.zeros(16, 1, 128, dtype=torch.float16, device="cuda") for _ in range(2))
    pa.pafp8_read_kv(s.k, s.v, ints([0, 16]), ints([0]), s.ptr_d, s.ids_d, ko, vo, k_scale=3.0)
    ref = (codes.view(torch.float8_e5m2).float() * 3).to(torch.float16)
    assert torch.equal(torch.nan_to_num(ko.view(-1), nan=1.5), torch.nan_to_num(ref, nan=1.5))


def test_read_outside_is_skipped_and_reported(cuda_device):
    s = Setup([40, 10], spare=0)
    ids = s.ids.copy()
    ids[1] = -1
    ko, vo = (torch.full((30, 3, 128), 7.0, device="cuda") for _ in range(2))
    # Request 0: tokens 10 .. 33 (16 .. 31 without a page); 1: from 14 on, past its table's end; more rows said than there are.
    pa.pafp8_read_kv(s.k, s.v, ints([0, 24, 99]), ints([10, 14]), s.ptr_d, ints(ids), ko, vo, k_scales=s.ks, v_scales=s.vs,
                     status=s.status)
    assert int(s.status) == 1
    ref = read_ref(s, "k", [10, 14], [24, 2])
    good = torch.tensor(list(range(6)) + list(range(22, 24)) + [24, 25])
    assert torch.equal(ko.cpu()[good], ref[good])
    rest = [i for i in range(30) if i not in good.tolist()]
    assert bool((ko[rest] == 7).all()) and bool((vo[rest] == 7).all())


def test_written_then_read_then_written(cuda_device):
    """A sequence moved to other pages through plain rows: powers of two lose nothing on the way."""
    a, b = Setup([77], seed=1), Setup([77], seed=2)
    k, v = a.rows(77, "bf16")
    a.append(k, v, ints([0, 77]), ints([0]))
    ko, vo = (torch.zeros(77, 3, 128, device="cuda") for _ in range(2))
    pa.pafp8_read_kv(a.k, a.v, ints([0, 77]), ints([0]), a.ptr_d, a.ids_d, ko, vo, k_scales=a.ks, v_scales=a.vs)
    b.append(ko, vo, ints([0, 77]), ints([0]))
    k2, v2 = torch.zeros_like(ko), torch.zeros_like(vo)
    pa.pafp8_read_kv(b.k, b.v, ints([0, 77]), ints([0]), b.ptr_d, b.ids_d, k2, v2, k_scales=b.ks, v_scales=b.vs)
    assert torch.equal(ko, k2) and torch.equal(vo, v2)
