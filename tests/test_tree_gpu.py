"""pafp8_run_tree against a float64 reference."""
import numpy as np
import pytest
import torch

import paged_attention_fp8_gb300 as pa
from tree_common import TreeBatch

pytestmark = pytest.mark.gpu


def _check(*a, **kw):
    b = TreeBatch(*a, **kw)
    b.check(*b.run())
    return b


@pytest.mark.parametrize("q,kv,o", [("bf16", "e4m3fn", None), ("bf16", "e5m2", None), ("f16", "e4m3fn", None),
                                    ("f16", "e5m2", "bf16"), ("bf16", "e4m3fn", "f16"), ("e4m3fn", "e4m3fn", None),
                                    ("e5m2", "e4m3fn", "f16"), ("e4m3fn", "e5m2", None), ("bf16", "bf16", None),
                                    ("f16", "f16", None), ("f16", "f16", "bf16")])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("hq,hkv,qo", [(8, 2, [5, 3, 8]), (4, 4, [40, 1, 17]), (16, 2, [11, 16, 9])])
def test_types_and_head_sizes(cuda_device, q, kv, o, d, hq, hkv, qo):
    """32, 64 and 128 rows a tile (4, 2 and 1 copies)."""
    _check([45, 300, 129], qo, hq, hkv, d=d, q=q, kv=kv, o=o, seed=d + hq)


@pytest.mark.parametrize("kv_len", [1, 2, 15, 16, 17, 31, 127, 128, 129, 143, 255, 256, 257, 1000, 2049])
@pytest.mark.parametrize("qo", [1, 7])
def test_lengths(cuda_device, kv_len, qo):
    qo = min(qo, kv_len)
    _check([kv_len], [qo], 8, 2, seed=kv_len)
    _check([kv_len, 5, kv_len], [qo, 0, 1], 4, 1, d=64, kv="e5m2", layout="HND", page_size=48, seed=kv_len + 1)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 16, 33, 71, 128])
def test_groups_and_row_tiles(cuda_device, group):
    """Row tiles of 128 // group tokens, some drafts longer than one tile."""
    _check([200, 333, 64], [max(1, 150 // group), 3, min(64, 2 * (128 // group))], 2 * group, 2, seed=group)


@pytest.mark.parametrize("mask", ["tree", "causal", "full", "random", "none", "some_empty"])
@pytest.mark.parametrize("ctx", [0, 1, 100, 511])
@pytest.mark.parametrize("T", [3, 33, 130])
def test_masks(cuda_device, mask, ctx, T):
    """Rows that see nothing, bits behind the last token, drafts across key tiles."""
    b = _check([ctx + T, T], [T, T], 2, 1, mask=mask, words=-(-T // 32) + 1, seed=T + ctx)
    if mask == "none" and ctx == 0:
        assert bool((b.o[:b.n] == 0).all()) and bool(torch.isneginf(b.lse[:b.n]).all())


@pytest.mark.parametrize("num_ctas", [1, 2, 7, 40, 152])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_splits(cuda_device, num_ctas, hkv):
    """Long and short lines over few and many CTAs: partial states and their merge."""
    _check([1500, 16, 700, 130], [4, 1, 9, 20], 2 * hkv, hkv, num_ctas=num_ctas, seed=num_ctas)


@pytest.mark.parametrize("page_size", [16, 32, 48, 64, 128, 256])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("kv", ["e4m3fn", "bf16"])
def test_pages_and_layouts(cuda_device, page_size, layout, kv):
    _check([333, 70], [6, 4], 8, 2, kv=kv, page_size=page_size, layout=layout, seed=page_size)


@pytest.mark.parametrize("q,kv", [("bf16", "e4m3fn"), ("e4m3fn", "e4m3fn"), ("f16", "f16")])
def test_head_scales(cuda_device, q, kv):
    _check([333, 70], [6, 4], 8, 2, q=q, kv=kv, head_scales=True, seed=4)


@pytest.mark.parametrize("spread", [0.0, 1e-3, 30.0])
def test_flat_and_peaked_rows(cuda_device, spread):
    """Equal weights (zero query) and rows where one key takes all."""
    _check([900, 70], [6, 4], 8, 2, spread=spread, seed=6)
    _check([900, 70], [6, 4], 8, 2, q="f16", spread=spread, seed=6)


def test_rising_maxima(cuda_device):
    """Keys that grow along the sequence: every tile raises the maximum."""
    b = TreeBatch([1024], [8], 8, 2, kv="bf16", seed=8)
    for q, kv in (("bf16", "bf16"), ("bf16", "e4m3fn"), ("f16", "e4m3fn")):
        b = TreeBatch([1024], [8], 8, 2, q=q, kv=kv, seed=8)
        ramp = torch.linspace(0.05, 3.0, 1024)[:, None, None]
        up = torch.ones(128) * 0.7
        b.q = (b.q.float() * 0.1 + up).to(b.q.dtype)
        rows = (b.k[0].float() * 0.1 + ramp * up).to(b.k[0].dtype)
        b.k[0] = rows
        raw = torch.uint8 if kv == "e4m3fn" else torch.int16
        host = b.kc.cpu().view(raw)
        for p in range(64):
            host[int(b.ids[p])] = rows.view(raw)[16 * p:16 * p + 16]
        b.kc = host.cuda().view(b.kc.dtype)
        b.check(*b.run())


def test_non_finite_queries_stay_in_their_row(cuda_device):
    b = TreeBatch([200], [6], 8, 2, seed=9)
    ro, rl = b.run()
    b.q[2, 3, 5] = float("inf")
    b.q[4, 1, 0] = float("nan")
    o, lse = b.run()
    for u, h in ((2, 3), (4, 1)):
        assert bool(torch.isnan(o[u, h]).all()) and bool(torch.isnan(lse[u, h]))
        o[u, h], lse[u, h] = ro[u, h], rl[u, h]
    assert torch.equal(o, ro) and torch.equal(lse, rl)


def test_bad_page_is_reported(cuda_device):
    b = TreeBatch([100, 60], [4, 4], 8, 2, seed=10)
    b.run()
    b.ids[3] = b.pool
    b.call()
    with pytest.raises(pa.Pafp8Error) as e:
        b.plan.device_status(b.ws)
    assert e.value.status_name == "ERR_BOUNDS"


def test_repeats_graphs_and_streams_are_bit_identical(cuda_device):
    b = TreeBatch([1500, 300, 16], [9, 4, 16], 8, 2, seed=11)
    o, lse = b.run()
    b.o.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.call()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.o[:b.n].cpu(), o) and torch.equal(b.lse[:b.n].cpu(), lse)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b.o.zero_()
        b.call()
    side.synchronize()
    assert torch.equal(b.o[:b.n].cpu(), o)


def test_single_token_chain_is_decode(cuda_device):
    """One drafted token a request: the decode kernel's outputs within both kernels' roundings."""
    b = TreeBatch([700, 33, 256], [1, 1, 1], 8, 2, mask="causal", seed=12)
    o, lse = b.run()
    dec = pa.Plan(mode="decode", num_qo_heads=8, num_kv_heads=2, num_pages=b.pool, kv_indptr=b.kv_indptr,
                  last_page_len=b.last, q_dtype="bf16", kv_dtype="e4m3fn")
    ws = torch.empty(dec.workspace_bytes, dtype=torch.uint8, device="cuda")
    dec.upload(ws)
    od, ld = torch.empty_like(b.o[:3]), torch.empty_like(b.lse[:3])
    kc, vc = (torch.nan_to_num(c.float()).to(c.dtype) for c in (b.kc, b.vc))
    dec.run(b.dq, kc, vc, b.ids, od, ld, ws, k_scale=b.ks, v_scale=b.vs)
    assert float((od.cpu().float() - o.float()).abs().max()) < 0.02
    assert float((ld.cpu() - lse).abs().max()) < 1e-3


def test_expired_wait_is_reported_and_the_context_stays_usable(cuda_device, monkeypatch):
    b = TreeBatch([4000, 300], [9, 4], 8, 2, seed=13)
    o, lse = b.run()
    monkeypatch.setenv("PAFP8_WAIT_CYCLES", "1")
    b.call()
    with pytest.raises(pa.Pafp8Error) as e:
        b.plan.device_status(b.ws)
    assert e.value.status_name == "ERR_TIMEOUT"
    monkeypatch.delenv("PAFP8_WAIT_CYCLES")
    b.call()
    b.plan.device_status(b.ws)
    assert torch.equal(b.o[:b.n].cpu(), o) and torch.equal(b.lse[:b.n].cpu(), lse)


def test_arrays_that_cannot_be_read_as_they_are_refused(cuda_device):
    b = TreeBatch([100, 60], [4, 4], 8, 2, seed=14)
    b.run()
    good = (b.dq, b.kc, b.vc, b.ids, b.mask, b.o, b.lse, b.ws)
    for at, bad, match in ((0, b.dq.transpose(0, 1), "q .*not contiguous"), (0, b.dq.cpu(), "q is on cpu"),
                           (1, b.kc.cpu(), "k_cache is on cpu"), (3, b.ids.cpu(), "kv_indices is on cpu"),
                           (4, b.mask.float(), "tree_mask"), (4, b.mask.t(), "tree_mask"), (4, b.mask[:3], "tree_mask"),
                           (5, b.o.transpose(0, 1), "o .*not contiguous"), (6, b.lse.t(), "lse .*not contiguous")):
        args = list(good)
        args[at] = bad
        with pytest.raises(ValueError, match=match):
            b.plan.run_tree(*args, k_scale=b.ks, v_scale=b.vs)
    b.plan.run_tree(*good[:6], None, b.ws, k_scale=b.ks, v_scale=b.vs)  # lse may be left out
    b.plan.device_status(b.ws)
