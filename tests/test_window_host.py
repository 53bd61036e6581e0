"""Windowed plans and block-scale runs on the host: refusals, and what the plans
make of a window (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import paged_attention_fp8_gb300 as pa

A = 0x10000


def plan(mode="decode", lens=(100, 0, 33), new=None, *, window=0, sinks=0, page_size=16, q="bf16", kv="e4m3fn", **kw):
    n = [-(-x // page_size) for x in lens]
    return pa.Plan(mode=mode, num_qo_heads=8, num_kv_heads=2, num_pages=sum(n) + 1, kv_indptr=np.concatenate([[0], np.cumsum(n)]),
                   last_page_len=[x - (m - 1) * page_size if x else 0 for x, m in zip(lens, n)],
                   qo_indptr=None if new is None else np.concatenate([[0], np.cumsum(new)]), q_dtype=q, kv_dtype=kv,
                   page_size=page_size, window=window, sinks=sinks, num_ctas=8, **kw)


@pytest.mark.parametrize("kw,match", [
    (dict(window=-1), "window -1"), (dict(window=4, sinks=-2), "sinks -2"), (dict(sinks=3), "sinks 3 given without a window"),
    (dict(mode="tree", new=[1, 0, 2], window=5), "tree plan takes no window")])
def test_window_refusals(kw, match):
    with pytest.raises(pa.Pafp8Error, match=match):
        plan(**kw)


@pytest.mark.parametrize("kw", [dict(window=2 ** 31), dict(window=2 ** 32 + 5), dict(window=4, sinks=2 ** 32), dict(window=-2 ** 33),
                                dict(window=0.5), dict(window=float("inf"))])
def test_the_binding_does_not_wrap_or_cut_numbers(kw):
    with pytest.raises((ValueError, OverflowError)):
        plan(**kw)
    plan(window=2 ** 31 - 1, sinks=2 ** 31 - 1)


def test_window_length_limit():
    pages = (2 ** 31 - 1) // 16
    a = dict(mode="decode", num_qo_heads=1, num_kv_heads=1, num_pages=1, kv_indptr=[0, pages], last_page_len=[16], q_dtype="bf16",
             kv_dtype="e4m3fn", num_ctas=1, disable_split_kv=True)
    with pytest.raises(pa.Pafp8Error, match="a window goes with up to 2147483519"):
        pa.Plan(**a, window=10)
    assert pa.Plan(**{**a, "kv_indptr": [0, pages - 8]}, window=10).metadata()[8] == 0  # no merge


META = dict(segs=13, num_segs=7, off_chunk=23, num_chunks=22, num_tiles=18, off_tile=19)


def seen_pages(length, window, sinks):
    """16-token pages of a decode row that hold a visible key."""
    j = np.arange(length)
    vis = (j >= length - window) | (j < sinks) if window else j >= 0
    return len(np.unique(j[vis] // 16))


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 16), (40, 17), (90, 3), (2 ** 31 - 1, 5), (5, 2 ** 31 - 1)])
def test_decode_plans_count_the_pages_that_are_seen(window, sinks):
    lens = [100, 0, 33, 512, 16, 1]
    m = plan(lens=lens, window=window, sinks=sinks, disable_split_kv=True).metadata()
    segs = m[m[META["segs"]]:][:4 * m[META["num_segs"]]].reshape(-1, 4)
    got = {int(s[0]): int(s[2] - s[1]) for s in segs}
    assert got == {b: seen_pages(n, window, sinks) if n else 0 for b, n in enumerate(lens)}


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 5), (128, 128), (333, 20), (2 ** 31 - 1, 0), (4, 2 ** 31 - 1)])
@pytest.mark.parametrize("kv", ["e4m3fn", "bf16"])
def test_prefill_items_cover_what_their_rows_see(window, sinks, kv):
    """Every item's pages are those of its rows' visible keys, and its tiles hold them."""
    lens, new = [700, 40, 300], [500, 40, 3]
    m = plan("prefill", lens, new, window=window, sinks=sinks, kv=kv).metadata()
    tiles = m[m[META["off_tile"]]:][:8 * m[META["num_tiles"]]].reshape(-1, 8)
    span = 64 * (2 if kv == "bf16" and window >= 896 else 1)
    rows = {}
    for gap, hk, t0, nkv, qo0, qo_len, kv_len, page0 in tiles.tolist():
        b = [0, 500, 540].index(qo0)
        length = lens[b]
        assert kv_len == length - 16 * gap and qo_len == new[b]
        t = np.arange(t0, min(t0 + span, qo_len)) + length - qo_len
        j = np.arange(length)
        vis = (j[None] <= t[:, None]) & ((j[None] > t[:, None] - window) | (j[None] < sinks))
        pages = np.unique(j[vis.any(0)] // 16)
        head = -(-min(sinks, length) // 16)
        numbered = [p if p < head else p - gap for p in pages]
        assert min(numbered) >= 0 and 16 * max(numbered) < min(kv_len, 128 * nkv)
        assert len(set(numbered)) == len(numbered)
        if gap:  # nothing that is left out is seen
            assert not np.isin(pages, np.arange(head, head + gap)).any()
        rows.setdefault((b, hk), []).append(t0)
    for (b, hk), t0s in rows.items():
        assert sorted(t0s) == list(range(0, new[b], span))


def blocks(p, **kw):
    a = dict(q_dtype=pa.BF16, q=A, k_dtype=pa.E4M3FN, k=A, v_dtype=pa.E4M3FN, v=A, idx=A, q_scale=1.0, ks=A, vs=A, o_dtype=pa.BF16,
             o=A, lse=A, ws=A, n=1 << 20)
    a.update(kw)
    return pa.lib().pafp8_run_block_scales(p, a["q_dtype"], a["q"], a["k_dtype"], a["k"], a["v_dtype"], a["v"], a["idx"], a["q_scale"],
                                           a["ks"], a["vs"], a["o_dtype"], a["o"], a["lse"], a["ws"], a["n"], None)


def test_block_run_refusals():
    p, t = plan(), plan("tree", new=[1, 0, 2])
    assert blocks(None) == 3
    assert blocks(t.handle) == 8 and "tree plans" in pa.pafp8_last_error()
    assert blocks(p.handle) == 4 and "not the one" in pa.pafp8_last_error()
    assert blocks(p.handle, k_dtype=pa.E5M2) == 1 and blocks(p.handle, q_scale=2.0) == 3
    assert blocks(plan(kv="bf16").handle, k_dtype=pa.BF16, v_dtype=pa.BF16) in (1, 4)


HQ, HKV, D, POOL = 8, 2, 128, 11


@pytest.fixture(params=["decode", "prefill"])
def call(monkeypatch, request):
    p = plan(request.param, new=[4, 0, 3] if request.param == "prefill" else None)
    rows = 7 if request.param == "prefill" else 3
    calls = []
    real = pa.lib()

    class Recorder:
        def __getattr__(self, name):
            if name == "pafp8_run_block_scales":
                return lambda *a: calls.append(a) or 0
            return getattr(real, name)

    recorder = Recorder()
    monkeypatch.setattr(pa, "lib", lambda: recorder)
    monkeypatch.setattr(pa, "_device_of", lambda t, name: -1)
    e4 = dict(dtype=torch.float8_e4m3fn)
    good = dict(q=torch.zeros(rows, HQ, D, dtype=torch.bfloat16), k_cache=torch.zeros(POOL, 16, HKV, D, **e4),
                v_cache=torch.zeros(POOL, 16, HKV, D, **e4), kv_indices=torch.zeros(10, dtype=torch.int32),
                o=torch.zeros(rows, HQ, D, dtype=torch.bfloat16), lse=torch.zeros(rows, HQ),
                workspace=torch.zeros(p.workspace_bytes, dtype=torch.uint8), k_scales=torch.ones(POOL, 1, HKV),
                v_scales=torch.ones(POOL, 1, HKV))

    def go(**kw):
        a = {**good, **kw}
        n = len(calls)
        p.run_block_scales(a.pop("q"), a.pop("k_cache"), a.pop("v_cache"), a.pop("kv_indices"), a.pop("o"), a.pop("lse"),
                           a.pop("workspace"), stream=1, **a)
        assert len(calls) == n + 1

    go.plan, go.good, go.calls = p, good, calls
    return go


def test_binding_passes_on_what_fits(call):
    call()
    call(lse=None)
    call(kv_indices=torch.zeros(50, dtype=torch.int32))


def test_binding_refuses(call):
    g = call.good
    for kw, match in [
            (dict(q=g["q"][:-1]), "do not fit"), (dict(o=torch.zeros(3, 8, 64, dtype=torch.bfloat16)), "do not fit"),
            (dict(lse=g["lse"].double()), "lse has dtype"), (dict(lse=g["lse"][:-1]), "do not fit"),
            (dict(k_cache=g["k_cache"][:-1]), "do not fit"), (dict(v_cache=g["v_cache"].view(torch.float8_e5m2)), "v_cache has dtype"),
            (dict(kv_indices=g["kv_indices"].long()), "kv_indices has dtype"), (dict(kv_indices=g["kv_indices"][:9]), "do not fit"),
            (dict(k_scales=None), "k_scales None is not"), (dict(k_scales=torch.ones(POOL, HKV)), "k_scales .* is not"), (dict(v_scales=torch.ones(POOL, 2, HKV)), "v_scales .* is not"),
            (dict(k_scales=g["k_scales"].double()), "k_scales has dtype"), (dict(q=g["q"].transpose(0, 1)), "contiguous"),
            (dict(k_scales=torch.ones(POOL, 1, 2 * HKV)[..., ::2]), "contiguous")]:
        with pytest.raises(ValueError, match=match):
            call(**kw)
    assert not call.calls


def test_binding_refuses_other_plans():
    t = plan("tree", new=[1, 0, 2])
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    if not torch.cuda.is_available():
        with pytest.raises(ValueError, match="q is on cpu"):
            t.run_block_scales(q, q, q, None, q, None, q, k_scales=q, v_scales=q)
    p = plan()
    h = p.handle
    assert h in pa._SIZES
    del p
    assert h not in pa._SIZES


def test_the_plain_plan_call_is_unchanged():
    a, b = plan(), plan()
    assert np.array_equal(a.metadata(), b.metadata())
    out = ctypes.c_void_p()
    ptr, last = np.array([0, 7, 7, 10], np.int32), np.array([4, 0, 1], np.int32)
    assert pa.lib().pafp8_plan_create_window(ctypes.byref(a.desc), 0, 0, ptr.ctypes.data, last.ctypes.data, None,
                                             ctypes.byref(out)) == 0
    assert np.array_equal(pa.pafp8_plan_metadata(out.value), a.metadata())
    pa.lib().pafp8_plan_destroy(out)


def test_a_tree_plan_without_a_window_keeps_its_checks(monkeypatch):
    """pafp8_plan_create_window with a window of 0 makes every plan that pafp8_plan_create makes, tree plans too: their run
    call knows their sizes and refuses arrays that are too small."""
    desc = pa.plan_desc(mode=pa.MODE_TREE, batch=1, num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, num_pages=6,
                        q_dtype=pa.BF16, kv_dtype=pa.E4M3FN, o_dtype=pa.BF16, num_ctas=8)
    calls = []

    class Recorder:
        @staticmethod
        def pafp8_run_tree(*a):
            calls.append(a)
            return 0

        def __getattr__(self, name):
            return getattr(real, name)

    real, recorder = pa.lib(), Recorder()
    monkeypatch.setattr(pa, "lib", lambda: recorder)
    monkeypatch.setattr(pa, "_device_of", lambda t, name: -1)
    for make in (lambda: pa.pafp8_plan_create(desc, [0, 3], [5], [0, 4]), lambda: pa.pafp8_plan_create_window(desc, 0, 0, [0, 3], [5], [0, 4])):
        plan = make()
        try:
            args = [torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(6, 16, 2, 128, dtype=torch.float8_e4m3fn),
                    torch.zeros(6, 16, 2, 128, dtype=torch.float8_e4m3fn), torch.zeros(3, dtype=torch.int32),
                    torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(4, 8),
                    torch.zeros(pa.pafp8_workspace_bytes(plan), dtype=torch.uint8)]
            pa.pafp8_run_tree(plan, *args, stream=1)
            n = len(calls)
            for at in (1, 3, 4, 5, 6):  # a cache, page ids, mask rows, o, lse: one element or row less
                short = list(args)
                short[at] = args[at][:-1].contiguous()
                with pytest.raises(ValueError):
                    pa.pafp8_run_tree(plan, *short, stream=1)
            assert len(calls) == n
            with pytest.raises(ValueError, match="decode or prefill plan"):
                pa.pafp8_run_block_scales(plan, *args[:4], *args[5:], k_scales=None, v_scales=None, stream=1)
        finally:
            pa.pafp8_plan_destroy(plan)
        assert plan not in pa._TREE_SIZES and plan not in pa._SIZES
