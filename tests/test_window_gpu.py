"""Attention with a sliding window and sinks, and over block scales, against
the definition in 64 bits, with bounds derived from the roundings (window_ref)."""
import numpy as np
import pytest
import torch

import paged_attention_fp8_gb300 as pa
from blocks_ref import BLOCK, in_layout, raw
from window_ref import Batch, run

pytestmark = pytest.mark.gpu

LENS = [0, 1, 2, 15, 16, 17, 31, 33, 100, 127, 128, 129, 300, 777]
WINDOWS = [(1, 0), (1, 1), (2, 1), (16, 16), (17, 4), (15, 33), (100, 20), (128, 0), (129, 129), (500, 4), (4000, 7), (3, 5000),
           (2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("kw", [
    dict(q="bf16", kv="e4m3fn"), dict(q="f16", kv="bf16", layout="HND", d=64, hq=15, hkv=3),
    dict(q="e5m2", kv="e5m2", scales="head", page_size=48, layout="HND"), dict(q="bf16", kv="e4m3fn", scales="block", hq=5, hkv=1, d=64),
    dict(q="f16", kv="e5m2", scales="block", page_size=64, hq=24, hkv=6, layout="HND")])
def test_decode_window(cuda_device, window, sinks, kw):
    run(LENS, window=window, sinks=sinks, num_ctas=19, seed=window % 97 + sinks % 89, **kw)


PROMPTS = [([1], [1]), ([33], [33]), ([200, 0, 16, 333], [1, 0, 16, 70]), ([700, 129], [300, 129]), ([1000], [17])]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("kw", [
    dict(q="bf16", kv="e4m3fn"), dict(q="e4m3fn", kv="e5m2", layout="HND", page_size=32, hq=12, hkv=2),
    dict(q="f16", kv="f16", hq=6, hkv=2), dict(q="bf16", kv="bf16", d=64, layout="HND", page_size=48, hq=4, hkv=4),
    dict(q="f16", kv="e5m2", scales="head", hq=16, hkv=1), dict(q="bf16", kv="e4m3fn", scales="block", page_size=48, hq=9, hkv=3),
    dict(q="e5m2", kv="e4m3fn", scales="block", layout="HND", d=64)])
def test_prefill_window(cuda_device, window, sinks, kw):
    for lens, new in PROMPTS:
        run(lens, new, window=window, sinks=sinks, num_ctas=13, seed=window % 97 + sinks % 89, **kw)


@pytest.mark.parametrize("window", [100, 1600, 0])
@pytest.mark.parametrize("kv,d,scales", [("e4m3fn", 128, "tensor"), ("e5m2", 64, "head"), ("e5m2", 128, "block")])
def test_bf16_queries_beyond_f16(cuda_device, window, kv, d, scales):
    """Rows of 2^18 and of 2^-20 times the others, under windows and without one."""
    b = Batch([2000, 129], [300, 129], window=window, sinks=4 if window else 0, q="bf16", kv=kv, d=d, scales=scales, num_ctas=13)
    b.q[::3] *= 2.0 ** 18
    b.q[1::3] *= 2.0 ** -20
    b.upload()
    b.run()
    b.plan.device_status(b.ws)
    b.check()


@pytest.mark.parametrize("window", [600, 767, 895, 896, 900])
@pytest.mark.parametrize("kv", ["bf16", "f16"])
def test_prefill_window_on_pairs(cuda_device, window, kv):
    """A 2-byte cache at head_dim 128: windows on both sides of the rule that picks CTA pairs."""
    for lens, new in (([2100, 5, 900], [1500, 5, 100]), ([1024], [3])):
        run(lens, new, window=window, sinks=4, q=kv, kv=kv, hq=8, hkv=2, num_ctas=12)


@pytest.mark.parametrize("kw", [
    dict(q="bf16", kv="e4m3fn"), dict(q="f16", kv="e5m2", d=64, hq=12, hkv=6, layout="HND"),
    dict(q="e4m3fn", kv="e4m3fn", page_size=64, hq=64, hkv=8), dict(q="bf16", kv="e5m2", hq=1, hkv=1, page_size=48)])
def test_block_scales(cuda_device, kw):
    run(LENS, scales="block", num_ctas=23, **kw)
    for lens, new in PROMPTS + [([300, 40], [300, 8])]:
        run(lens, new, scales="block", num_ctas=13, **kw)


def test_block_scales_of_very_unlike_size(cuda_device):
    """V scales 2^36 apart, K scales 2^6: the largest products carry the result, small blocks keep their probability mass."""
    for new in (None, [90, 33]):
        b = Batch([400, 65], new, scales="block", spread=6, num_ctas=7)
        e = torch.randint(-18, 19, b.vs.shape, generator=torch.Generator().manual_seed(1))
        b.vs = b.vs * 2.0 ** e
        b.upload()
        b.run()
        b.check()


def test_all_zero_blocks(cuda_device):
    """Blocks of zeros carry the append's smallest scale and still count in the softmax's sum."""
    for new in (None, [70]):
        b = Batch([200], new, scales="block")
        page = b.ids[[0, 3, 5]]
        for c, s in ((b.k, b.ks), (b.v, b.vs)):
            raw(c)[page] = 0
            s[page] = 2.0 ** -64
        b.upload()
        b.run()
        b.check()


@pytest.mark.parametrize("scales", ["tensor", "block"])
@pytest.mark.parametrize("new", [None, [40]])
@pytest.mark.parametrize("kv", ["e4m3fn", "bf16"])
def test_what_no_row_sees_does_not_matter(cuda_device, scales, new, kv):
    """NaN keys, values and scales in the tokens between the sinks and the first window, and behind the end, and page ids
    there that are not in the pool."""
    if kv == "bf16" and scales == "block":
        pytest.skip("block scales go with an fp8 cache")
    length, window, sinks = 500, 90, 5
    b = Batch([length], new, window=window, sinks=sinks, scales=scales, kv=kv, layout="HND")
    low = length - (new[0] if new else 1) - window + 1
    pos = np.r_[sinks:low, length:-(-length // 16) * 16]
    page, slot = torch.as_tensor(b.ids[pos // 16]), torch.as_tensor(pos % 16)
    bits = 0x7F if kv == "e4m3fn" else 0x7FC0
    for c in (b.k, b.v):
        raw(c)[page, slot] = bits
    whole = np.arange(-(-sinks // 16), low // 16)
    if scales == "block":
        b.ks[b.ids[whole]], b.vs[b.ids[whole]] = float("nan"), float("inf")
    b.ids = b.ids.copy()
    real = b.ids.copy()
    b.ids[whole[1:]] = b.pool + 12345
    b.upload()
    b.run()
    b.plan.device_status(b.ws)  # the pages of the gap are not looked at
    b.ids = real
    b.check()


def test_bad_page_is_reported(cuda_device):
    for scales in ("tensor", "block"):
        for new in (None, [30]):
            b = Batch([300], new, window=64, sinks=4, scales=scales)
            b.ids[-1] = b.pool
            b.upload()
            b.run()
            with pytest.raises(pa.Pafp8Error, match="ERR_BOUNDS"):
                b.plan.device_status(b.ws)


@pytest.mark.parametrize("split", [dict(fixed_split_pages=3), dict(disable_split_kv=True), dict(num_ctas=1), dict(num_ctas=152)])
@pytest.mark.parametrize("scales", ["tensor", "block"])
def test_decode_splits(cuda_device, split, scales):
    run([2000, 37, 0, 1500], window=900, sinks=30, scales=scales, **split)


def test_many_requests_take_chunks_at_run_time(cuda_device):
    """Enough pages a CTA that the plan hands the last of each row out at run time; launched again and again."""
    for scales in ("tensor", "block"):
        b = Batch([400 + 7 * i for i in range(40)], window=333, sinks=20, scales=scales, num_ctas=16, hq=16, hkv=4).upload()
        first = None
        for _ in range(3):
            b.run()
            b.check()
            first = b.o.clone() if first is None else first
        assert torch.equal(raw(first), raw(b.o))


def test_window_over_everything_is_the_plain_result(cuda_device):
    """A window at least as long as the sequence changes nothing, bit for bit."""
    for new in (None, [100, 7]):
        for kw in (dict(q="bf16", kv="e4m3fn"), dict(q="e4m3fn", kv="e4m3fn"), dict(q="bf16", kv="bf16")):
            a = run([300, 41], new, num_ctas=9, **kw)
            b = run([300, 41], new, num_ctas=9, window=300, sinks=2, **kw)
            assert torch.equal(raw(a.o), raw(b.o)) and torch.equal(a.lse, b.lse)


def test_equal_power_of_two_scales_agree_with_one(cuda_device):
    """A cache whose blocks all have the scale that the tensor has: the same logits, bit for bit (powers of two)."""
    for new in (None, [64, 9]):
        a = Batch([500, 33], new, num_ctas=5)
        a.k_scale, a.v_scale = 2.0 ** -6, 2.0 ** -5
        a.upload()
        a.run()
        b = Batch([500, 33], new, num_ctas=5, scales="block")
        b.q, b.k, b.v, b.ids = a.q, a.k, a.v, a.ids
        b.ks, b.vs = torch.full_like(b.ks, 2.0 ** -6), torch.full_like(b.vs, 2.0 ** -5)
        b.upload()
        b.run()
        b.check()
        if new is None:
            assert torch.equal(a.lse, b.lse)


def test_host_buffers_stages_noalloc_and_pod(cuda_device):
    """The other run calls take windowed plans as they are."""
    b = run([900, 45, 0, 300], window=200, sinks=17, num_ctas=11)
    want_o, want_l = b.o.clone(), b.lse.clone()
    kw = dict(q_scale=b.q_scale, k_scale=b.k_scale, v_scale=b.v_scale)

    def same():
        torch.cuda.synchronize()
        assert torch.equal(raw(b.o), raw(want_o)) and torch.equal(b.lse, want_l)
        b.o.fill_(7)
        b.lse.fill_(7)

    for stage in (1, 2):
        b.plan.run_stage(stage, *b.args(), **kw)
    same()
    pa.pafp8_run_decode_noalloc(b.plan.handle, *b.args()[:-1], **kw)
    same()
    ws = torch.empty(b.plan.host_workspace_bytes("bf16"), dtype=torch.uint8, device="cuda")
    o_h, l_h = torch.empty(b.o.shape, dtype=b.o.dtype).pin_memory(), torch.empty(b.lse.shape).pin_memory()
    b.plan.run_host(b.q.pin_memory(), b.k_d, b.v_d, torch.as_tensor(b.ids, dtype=torch.int32).pin_memory(), o_h, l_h, ws, **kw)
    torch.cuda.synchronize()
    assert torch.equal(raw(o_h), raw(want_o.cpu())) and torch.equal(l_h, want_l.cpu())
    # A windowed prefill beside an unwindowed decode of the same pool.
    p = Batch([900, 45, 0, 300], [300, 45, 0, 1], window=100, sinks=3, num_ctas=20).upload()
    d = Batch([900, 45, 0, 300], num_ctas=20).upload()
    for x in (p, d):
        x.k, x.v, x.k_d, x.v_d, x.ids, x.ids_d, x.k_scale, x.v_scale = b.k, b.v, b.k_d, b.v_d, b.ids, b.ids_d, b.k_scale, b.v_scale
    pa.pafp8_run_pod(p.plan.handle, p.q_d, p.ids_d, p.o, p.lse, p.ws, d.plan.handle, d.q_d, d.ids_d, d.o, d.lse, d.ws, b.k_d, b.v_d,
                     k_scale=b.k_scale, v_scale=b.v_scale)
    torch.cuda.synchronize()
    p.check()
    d.check()


@pytest.mark.parametrize("new", [None, [60, 9]])
@pytest.mark.parametrize("scales", ["tensor", "block"])
def test_captured_and_on_another_stream(cuda_device, new, scales):
    b = Batch([333, 48], new, window=150, sinks=9, scales=scales, num_ctas=10).upload()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    b.run()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        b.run()
    # Other queries, keys, values and scales in the same buffers.
    o = Batch([333, 48], new, window=150, sinks=9, scales=scales, num_ctas=10, seed=5)
    b.q, b.k, b.v = o.q, o.k, o.v
    b.q_d.copy_(o.q)
    raw(b.k_d).copy_(raw(in_layout(o.k, b.layout)))
    raw(b.v_d).copy_(raw(in_layout(o.v, b.layout)))
    if scales == "block":
        b.ks, b.vs = o.ks, o.vs
        b.ks_d.copy_(o.ks)
        b.vs_d.copy_(o.vs)
    b.o.fill_(7)
    g.replay()
    b.check()
    b.o.fill_(7)
    side.wait_stream(torch.cuda.current_stream())
    b.run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    b.check()


def test_long_context(cuda_device):
    """70000 keys, a window in their middle scales: sums of many tiles."""
    run([70000], window=20000, sinks=64, scales="block", hq=8, hkv=1)
    run([70000, 3], [5, 3], window=30000, sinks=130, scales="block", hq=4, hkv=1)


def test_scales_past_two_gib_of_codes(cuda_device):
    """Pages at the end of a pool whose codes pass 2^31: the scale lookups count in 64 bits."""
    heads, d, pool = 8, 128, 140000
    k, v = (torch.zeros(pool, 16, heads, d, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(pool, 1, heads, device="cuda") for _ in range(2))
    small = Batch([100], scales="block", hq=16, hkv=heads)
    at = torch.tensor([pool - 1 - 3 * i for i in range(len(small.ids))])
    for big, sc, c, s in ((k, ks, small.k, small.ks), (v, vs, small.v, small.vs)):
        raw(big)[at.cuda()] = raw(c)[small.ids].cuda()
        sc[at.cuda()] = s[small.ids].cuda()
    plan = pa.Plan(mode="decode", num_qo_heads=16, num_kv_heads=heads, num_pages=pool, kv_indptr=[0, 7], last_page_len=[4],
                   q_dtype="bf16", kv_dtype="e4m3fn")
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    plan.upload(ws)
    o, lse = torch.zeros(1, 16, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 16, device="cuda")
    plan.run_block_scales(small.q.cuda(), k, v, at.to(torch.int32).cuda(), o, lse, ws, k_scales=ks, v_scales=vs)
    small.check(o, lse)


@pytest.mark.parametrize("window,sinks", [(900, 0), (900, 4), (1000, 40), (300, 40), (17, 130)])
@pytest.mark.parametrize("kv,layout,page_size", [("bf16", "NHD", 32), ("f16", "HND", 48), ("bf16", "HND", 16), ("f16", "NHD", 64)])
def test_2_byte_prefill_with_a_gap_in_larger_pages(cuda_device, window, sinks, kv, layout, page_size):
    """Pages of several 16-token blocks and sinks over several of them, with lengths well past the window, so that items leave
    pages out; windows on both sides of the rule that picks CTA pairs."""
    run([2500, 40, 1700], [900, 40, 33], window=window, sinks=sinks, q=kv, kv=kv, hq=8, hkv=2, num_ctas=12, layout=layout,
        page_size=page_size)


@pytest.mark.parametrize("new", [None, [150]])
@pytest.mark.parametrize("kv,q", [("e4m3fn", "bf16"), ("e5m2", "e4m3fn")])
def test_zero_blocks_beside_the_largest_values_they_go_with(cuda_device, new, kv, q):
    """V scales 2^90 apart, as the append writes them for blocks of zeros (2^-64) and for values of 2^26 times the type's
    largest: the border that the header states, with the zeros first, between and last, keys of zeros and others."""
    b = Batch([333], new, scales="block", q=q, kv=kv, num_ctas=3)
    b.vs = b.vs / b.vs.max() * 2.0 ** 26  # within a factor of 8 of one another
    for i, at in enumerate((0, 1, 7, 12, 20)):
        page = int(b.ids[at])
        raw(b.v)[page] = 0
        b.vs[page] = 2.0 ** -64
        if i % 2:
            raw(b.k)[page] = 0
            b.ks[page] = 2.0 ** -64
    b.upload()
    b.run()
    b.plan.device_status(b.ws)
    b.check()


@pytest.mark.parametrize("new", [None, [120]])
@pytest.mark.parametrize("kv,q", [("e4m3fn", "bf16"), ("e5m2", "e4m3fn")])
def test_small_blocks_carry_the_output_where_the_large_ones_weigh_little(cuda_device, new, kv, q):
    """V scales 2^12 apart and logits that leave the large blocks next to nothing.  Below f16's normal range a probability loses
    at most 2^-25 of the largest one, and itself (decode), or the product with its V scale 2^-25 of the largest such product
    (prefill): the bound counts that in place of 2^-25 of the largest V scale."""
    b = Batch([300], new, scales="block", q=q, kv=kv, num_ctas=4)
    big = torch.as_tensor(b.ids[::3])
    b.q = b.q.double().abs().to(b.q.dtype)
    for pages, sign in ((torch.arange(b.pool), 1), (big, -1)):  # keys of large blocks point away from every query
        x = b.k.view(torch.uint8)[pages] & 0x7F
        b.k.view(torch.uint8)[pages] = x | (0x80 if sign < 0 else 0)
    b.vs = b.vs / 2.0 ** 12
    b.vs[big] *= 2.0 ** 12
    b.upload()
    b.run()
    b.check()
    o, _, tol, _ = b.expect()
    key, qs = b.dense("k", 0), b.q_scale
    page = torch.as_tensor(b.ids[np.arange(300) // 16])
    group, rows = b.hq // b.hkv, len(b.q)
    z = torch.einsum("uhgd,jhd->uhgj", (b.q.double() * qs).view(rows, b.hkv, group, b.d), key) * b.sm_scale
    w = torch.softmax(z.masked_fill(~b.visible(0)[:, None, None], -np.inf), -1)
    top = 448.0 if kv == "e4m3fn" else 57344.0
    scale = b.vs.double()[page, 0].T[None, :, None]
    if new is None:
        lost = (torch.minimum(w, 2.0 ** -25 * w.amax(-1, keepdim=True)) * scale).sum(-1)
    else:
        lost = b.visible(0).sum(-1)[:, None, None] * 2.0 ** -25 * (w * scale).amax(-1)
    counted = b.visible(0).sum(-1)[:, None] * 2.0 ** -25 * float(b.vs.max())
    tight = tol - (counted - lost.view(rows, b.hq))[..., None] * top * (1 + torch.finfo(b.o.dtype).eps / 2)
    over = (b.o.double().cpu() - o).abs() - tight
    assert over.max() <= 0, float(over.max())
    assert (tight < o.abs() / 8).double().mean() > 0.5  # an output of zero would not pass
