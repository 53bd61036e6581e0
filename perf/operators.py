"""The operators of a verification step over the paged cache, as timed work.

A serving loop that verifies drafted tokens (a tree of candidates for each
request, a single token being the smallest tree) runs three operators a step:

* ``tables``  block tables and slot maps on the GPU from request lengths: new
  pages from the free list, the CSR page table, every token's request,
  position and cache slot, the tree's rotary positions and ancestor masks;
* ``rope``    per-head RMS norm of q and k with the rotary rotation (one
  position axis, or time / height / width), k and v written into the paged
  cache at their slots in the cache's own type;
* ``tree``    attention of the drafted tokens over the cache: a request's
  cached context in full, its drafted tokens by the ancestor masks.

``run`` computes them in plain torch operations where ``own`` is false and
calls the library's entry points where it is true.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8_MAX = {"e4m3fn": 448.0, "e5m2": 57344.0}
BYTES = {"bf16": 2, "f16": 2, "e4m3fn": 1, "e5m2": 1}


def listed():
    return [
        # One chat request that takes one new token: the call's latency alone.
        dict(name="tables_one", op="tables", batch=1, kv_min=1000, kv_max=1000, new_min=1, new_max=1, page_size=16, lens=1),
        # The serving batch (64 requests of 512-4096 tokens) with 16 drafted tokens each.
        dict(name="tables_serving", op="tables", batch=64, kv_min=512, kv_max=4096, new_min=16, new_max=16,
             page_size=16, lens=2),
        # A large pool of long requests with ragged drafts: the page lists are what moves.
        dict(name="tables_long", op="tables", batch=1021, kv_min=0, kv_max=32768, new_min=0, new_max=33, page_size=16,
             lens=3),
        # One decode step of 64 tokens: latency.
        dict(name="rope_decode", op="rope", tokens=64, hq=32, hkv=8, d=128, src="bf16", kv="e4m3fn", q_out="bf16",
             layout="NHD", page_size=16, axes=1, rot=128, interleaved=False, norm=True),
        # The new tokens of the ragged prefill batch.
        dict(name="rope_prefill", op="rope", tokens=8838, hq=32, hkv=8, d=128, src="bf16", kv="e4m3fn", q_out="bf16",
             layout="NHD", page_size=16, axes=1, rot=128, interleaved=False, norm=True),
        # Image and video tokens: three position axes, head-major pages, head_dim 64, odd count.
        dict(name="rope_axes", op="rope", tokens=5003, hq=24, hkv=6, d=64, src="f16", kv="e5m2", q_out="f16",
             layout="HND", page_size=32, axes=3, rot=64, interleaved=False, norm=True),
        # A long prompt whose query goes on in fp8; half the head rotates, in neighbouring pairs.
        dict(name="rope_long", op="rope", tokens=32768, hq=32, hkv=8, d=128, src="bf16", kv="e4m3fn", q_out="e4m3fn",
             layout="NHD", page_size=16, axes=1, rot=64, interleaved=True, norm=True),
        # One short request with five drafted tokens: latency.
        dict(name="tree_one", op="tree", batch=1, kv_min=333, kv_max=333, new_min=5, new_max=5, hq=8, hkv=2, d=128,
             q="bf16", kv="e4m3fn", layout="NHD", page_size=16, lens=4),
        # The serving batch with 16 drafted tokens a request (64 rows a KV head).
        dict(name="tree_serving", op="tree", batch=64, kv_min=512, kv_max=4096, new_min=16, new_max=16, hq=32, hkv=8,
             d=128, q="bf16", kv="e4m3fn", layout="NHD", page_size=16, lens=5),
        # Long context, few drafted tokens, f16 over e5m2.
        dict(name="tree_long", op="tree", batch=8, kv_min=32768, kv_max=32768, new_min=4, new_max=4, hq=64, hkv=8, d=128,
             q="f16", kv="e5m2", layout="NHD", page_size=16, lens=6),
        # Wide ragged trees: up to 61 drafted tokens, several row tiles a request.
        dict(name="tree_wide", op="tree", batch=24, kv_min=500, kv_max=4096, new_min=17, new_max=61, hq=32, hkv=8, d=128,
             q="bf16", kv="e4m3fn", layout="NHD", page_size=32, lens=7),
        # A 2-byte cache of the query's own type, head-major.
        dict(name="tree_bf16_cache", op="tree", batch=32, kv_min=512, kv_max=4096, new_min=1, new_max=12, hq=32, hkv=8,
             d=128, q="bf16", kv="bf16", layout="HND", page_size=16, lens=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "rope", "tree", "tree", "tree"])
    lens = rng.randrange(1 << 30)
    page_size = rng.choice([16, 16, 32, 64, 48])
    if op == "tables":
        batch = _log(rng, 1, 1021)
        top = _log(rng, 16, 32768)
        new = _log(rng, 1, 64)
        return dict(op=op, batch=batch, kv_min=rng.choice([0, top // 8]), kv_max=top, new_min=rng.choice([0, 1, new]),
                    new_max=new, page_size=page_size, lens=lens)
    layout = rng.choice(["NHD", "HND"])
    d = rng.choice([128, 128, 64])
    hkv = rng.choice([1, 2, 4, 6, 8])
    if op == "rope":
        src = rng.choice(["bf16", "f16"])
        return dict(op=op, tokens=_log(rng, 1, 20000), hq=hkv * rng.choice([1, 2, 4]), hkv=hkv, d=d, src=src,
                    kv=rng.choice(["e4m3fn", "e5m2", src]), q_out=rng.choice([src, src, "e4m3fn"]), layout=layout,
                    page_size=page_size, axes=rng.choice([1, 3]), rot=rng.choice([d, d, d // 2]),
                    interleaved=rng.choice([False, True]), norm=rng.choice([True, True, False]))
    q = rng.choice(["bf16", "bf16", "f16", "e4m3fn"])
    kv = rng.choice(["e4m3fn", "e4m3fn", "e5m2"] + ([q] if q != "e4m3fn" else []))
    group = rng.choice([1, 2, 4, 5, 8])
    new = _log(rng, 1, 48)
    top = max(_log(rng, 64, 32768), 2 * new)
    # At most the largest listed case's keys, rows and products.
    most = min(1 << 17, int(1.4e7 / (new * group * hkv)) * (128 // d))
    batch = max(1, min(64, most // top))
    top = max(2 * new, min(top, most // batch))
    return dict(op=op, batch=batch, kv_min=max(new, top // 8), kv_max=top, new_min=rng.choice([1, new]), new_max=new,
                hq=hkv * group, hkv=hkv, d=d, q=q, kv=kv, layout=layout, page_size=page_size, lens=lens)


def _lengths(case):
    """Every request's (length before the step, new tokens), from the case alone."""
    r = random.Random(case["lens"])
    kv = [r.randint(case["kv_min"], case["kv_max"]) for _ in range(case["batch"])]
    new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["batch"])]
    return kv, new


def _ceil(a, b):
    return -(-a // b)


def _scan(xs):
    out = [0]
    for x in xs:
        out.append(out[-1] + x)
    return out


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _int(xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


def _codes(shape, fmt, scale, g):
    """Normal values in the type `fmt`, fp8 ones as codes of value / scale."""
    x = torch.randn(shape, device="cuda", generator=g)
    if fmt in FP8_MAX:
        x = (x / scale).clamp_(-FP8_MAX[fmt], FP8_MAX[fmt])
    return x.to(DTYPES[fmt])


def _parents(counts, g):
    """Random trees: a request's first drafted token is the root (-1), the others hang on an earlier one."""
    n = sum(counts)
    u = torch.tensor([i for c in counts for i in range(c)], dtype=torch.float64, device="cuda")
    p = (torch.rand(n, device="cuda", generator=g, dtype=torch.float64) * u).floor().to(torch.int32)
    return torch.where(u == 0, torch.full_like(p, -1), p)


def _scale(fmt):
    return 5.5 / FP8_MAX[fmt] if fmt in FP8_MAX else 1.0


# ---- inputs ---------------------------------------------------------------

def _inputs(case, seed):
    return {"tables": _inputs_tables, "rope": _inputs_rope, "tree": _inputs_tree}[case["op"]](case, _generator(seed))


def _inputs_tables(c, g):
    kv, new = _lengths(c)
    ps = c["page_size"]
    have = [_ceil(a, ps) for a in kv]
    total = [_ceil(a + b, ps) for a, b in zip(kv, new)]
    width = max(total) + 3
    pool = sum(total) + 37
    perm = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    held = sum(have)
    used = 5
    table = torch.full((c["batch"], width), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(width, device="cuda")
    table[at[None] < _int(have)[:, None]] = perm[:held]
    tokens = sum(new)
    cap = _ceil(tokens + 1, 64) * 64
    parents = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    if tokens:
        parents[:tokens] = _parents(new, g)
    return dict(case=c, cached_lens=_int(kv), new_lens=_int(new), block_table=table,
                free_pages=torch.cat([perm[held:held + 2].repeat(3)[:used], perm[held:]]).contiguous(),
                free_used=_int([used]), parents=parents, pool=pool, max_pages=sum(total) + 11, max_tokens=cap,
                words=_ceil(max(1, c["new_max"]), 32), new_max=max(1, c["new_max"]))


def _inputs_rope(c, g):
    n, d, half = c["tokens"], c["d"], c["rot"] // 2
    heads = c["hq"] + 2 * c["hkv"]
    ps = c["page_size"]
    pages = _ceil(n, ps) + 2
    qkv = (torch.randn(n, heads, d, device="cuda", generator=g) * 1.7).to(DTYPES[c["src"]])
    qw = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(DTYPES[c["src"]])
    kw = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(DTYPES[c["src"]])
    limit = 40960
    angle = torch.arange(limit, device="cuda", dtype=torch.float64)[:, None] * \
        (1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half))[None]
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
    pos = torch.randint(0, limit, (c["axes"], n), device="cuda", generator=g).to(torch.int32)
    # Time, height and width share the pairs in runs of a quarter, three eighths and the rest.
    axis = torch.zeros(half, dtype=torch.uint8, device="cuda")
    if c["axes"] == 3:
        axis[half // 4:] = 1
        axis[half // 4 + 3 * half // 8:] = 2
    slots = torch.randperm(pages * ps, device="cuda", generator=g)[:n].contiguous()
    shape = (pages, ps, c["hkv"], d) if c["layout"] == "NHD" else (pages, c["hkv"], ps, d)
    sc = _scale(c["kv"])
    # The caches' other slots hold what earlier steps wrote.
    return dict(case=c, qkv=qkv, q_weight=qw if c["norm"] else None, k_weight=kw if c["norm"] else None, cos_sin=cos_sin,
                positions=pos, pair_axis=axis if c["axes"] > 1 else None, slots=slots,
                k_cache=_codes(shape, c["kv"], sc, g), v_cache=_codes(shape, c["kv"], sc, g), k_scale=sc, v_scale=sc,
                q_scale=_scale(c["q_out"]), eps=1e-6,
                q_out=torch.zeros(n, c["hq"], d, device="cuda", dtype=DTYPES[c["q_out"]]))


def _inputs_tree(c, g):
    kv, new = _lengths(c)
    kv = [max(a, b) for a, b in zip(kv, new)]  # lengths with the drafted tokens in the cache
    ps = c["page_size"]
    npages = [_ceil(a, ps) for a in kv]
    pool = sum(npages) + 5
    tokens = sum(new)
    shape = (pool, ps, c["hkv"], c["d"]) if c["layout"] == "NHD" else (pool, c["hkv"], ps, c["d"])
    sc = _scale(c["kv"])
    qsc = _scale(c["q"])
    words = _ceil(max(1, c["new_max"]), 32)
    kv_indptr, qo_indptr = _scan(npages), _scan(new)
    q = _codes((tokens, c["hq"], c["d"]), c["q"], qsc, g)
    k, v = _codes(shape, c["kv"], sc, g), _codes(shape, c["kv"], sc, g)
    ids = torch.randperm(pool, device="cuda", generator=g)[:kv_indptr[-1]].to(torch.int32)
    return dict(case=c, q=q, k_cache=k, v_cache=v, kv_indices=ids, kv_lens=kv, qo_lens=new, kv_indptr_h=kv_indptr,
                last_page_len_h=[a - (p - 1) * ps if p else 0 for a, p in zip(kv, npages)], qo_indptr_h=qo_indptr,
                kv_indptr=_int(kv_indptr), qo_indptr=_int(qo_indptr), kv_len=_int(kv), pool=pool,
                mask=_masks(_parents(new, g), _int(qo_indptr), tokens, max(1, c["new_max"]), words), q_scale=qsc, k_scale=sc,
                v_scale=sc, sm_scale=1.0 / math.sqrt(c["d"]),
                o=torch.zeros(tokens, c["hq"], c["d"], device="cuda", dtype=DTYPES["bf16" if c["q"] in FP8_MAX else c["q"]]),
                lse=torch.zeros(tokens, c["hq"], device="cuda"))


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import paged_attention_fp8_gb300 as pa
        s["pa"] = pa
        if case["op"] == "tables":
            s["tables"] = pa.StepTables(batch=case["batch"], max_pages=s["max_pages"], max_tokens=s["max_tokens"],
                                        mask_words=s["words"], page_size=case["page_size"], num_pages=s["pool"],
                                        device="cuda")
        elif case["op"] == "tree":
            s["plan"] = pa.Plan(mode="tree", num_qo_heads=case["hq"], num_kv_heads=case["hkv"], num_pages=s["pool"],
                                kv_indptr=s["kv_indptr_h"], last_page_len=s["last_page_len_h"], qo_indptr=s["qo_indptr_h"],
                                q_dtype=case["q"], kv_dtype=case["kv"], head_dim=case["d"], page_size=case["page_size"],
                                kv_layout=case["layout"])
            s["workspace"] = torch.empty(s["plan"].workspace_bytes, dtype=torch.uint8, device="cuda")
            s["plan"].upload(s["workspace"])
    return s


# ---- one pass -------------------------------------------------------------

def run(s):
    return {"tables": _tables, "rope": _rope, "tree": _tree}[s["case"]["op"]](s)


def _tables(s):
    if own:
        t = s["tables"]
        t.build(s["cached_lens"], s["new_lens"], s["block_table"], s["free_pages"], s["free_used"], parents=s["parents"])
        return dict(block_table=s["block_table"], free_used=t.free_used, kv_indptr=t.kv_indptr, last_page_len=t.last_page_len,
                    kv_indices=t.kv_indices, qo_indptr=t.qo_indptr, batch_indices=t.batch_indices, positions=t.positions,
                    slots=t.slots, rope_positions=t.rope_positions, tree_mask=t.tree_mask)
    ps, batch = s["case"]["page_size"], s["case"]["batch"]
    cached, new, table = s["cached_lens"].long(), s["new_lens"].long(), s["block_table"]
    dev = table.device
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    have, total = (cached + ps - 1) // ps, (cached + new + ps - 1) // ps
    need = torch.cat([zero, (total - have).cumsum(0)])
    kv_indptr, qo_indptr = torch.cat([zero, total.cumsum(0)]), torch.cat([zero, new.cumsum(0)])
    col = torch.arange(table.shape[1], device=dev)[None]
    fresh = (col >= have[:, None]) & (col < total[:, None])
    taken = s["free_used"].long() + need[:-1, None] + col - have[:, None]
    pages = s["free_pages"].numel()
    got = torch.where(taken < pages, s["free_pages"][taken.clamp(0, pages - 1)], -1)
    table = torch.where(fresh, got.to(torch.int32), table)
    # The CSR page list, entry by entry.
    e = torch.arange(s["max_pages"], device=dev)
    row = (torch.searchsorted(kv_indptr, e, right=True) - 1).clamp(max=batch - 1)
    at = (e - kv_indptr[row]).clamp(0, table.shape[1] - 1)
    kv_indices = torch.where(e < kv_indptr[-1], table[row, at], 0).to(torch.int32)
    # The tokens.
    t = torch.arange(s["max_tokens"], device=dev)
    inside = t < qo_indptr[-1]
    req = (torch.searchsorted(qo_indptr, t, right=True) - 1).clamp(max=batch - 1)
    pos = cached[req] + t - qo_indptr[req]
    page = table[req, (pos // ps).clamp(0, table.shape[1] - 1)].long()
    slots = torch.where(inside & (page >= 0), page * ps + pos % ps, -1)
    mask = _masks(s["parents"], qo_indptr, s["max_tokens"], s["new_max"], s["words"])
    depth = _bits(mask).sum(1) - 1
    last = torch.where(cached + new > 0, cached + new - (total - 1) * ps, 0)
    return dict(block_table=table, free_used=(s["free_used"] + need[-1]).to(torch.int32), kv_indptr=kv_indptr.to(torch.int32),
                last_page_len=last.to(torch.int32), kv_indices=kv_indices, qo_indptr=qo_indptr.to(torch.int32),
                batch_indices=torch.where(inside, req, -1).to(torch.int32),
                positions=torch.where(inside, pos, 0).to(torch.int32), slots=slots,
                rope_positions=torch.where(inside, cached[req] + depth, 0).to(torch.int32), tree_mask=mask)


def _bits(mask):
    """[n, 32 words] truth values of an int32 mask."""
    sh = torch.arange(32, device=mask.device, dtype=torch.int32)
    return ((mask[:, :, None] >> sh) & 1).flatten(1)


def _masks(parents, qo_indptr, tokens, widest, words):
    """Ancestor masks [tokens, words] (bit w of row u: drafted token w is u or an ancestor of it)."""
    dev = parents.device
    qo_indptr = qo_indptr.long()
    batch = qo_indptr.numel() - 1
    t = torch.arange(tokens, device=dev)
    inside = t < qo_indptr[-1]
    req = (torch.searchsorted(qo_indptr, t, right=True) - 1).clamp(max=batch - 1)
    u = torch.where(inside, t - qo_indptr[req], 0)
    # step[b, u, w] = 1 where w is u's parent; (1 - step)^-1 adds up all its powers, the ancestors.
    par = parents[:tokens].long()
    linked = inside & (par >= 0)
    step = torch.zeros(batch, widest, widest + 1, device=dev)
    step[req, u, torch.where(linked, par, widest)] = 1.0
    step = step[:, :, :widest]
    eye = torch.eye(widest, device=dev).expand(batch, -1, -1)
    reach = torch.linalg.solve_triangular(eye - step, eye, upper=False, unitriangular=True)
    row = torch.zeros(tokens, 32 * words, device=dev, dtype=torch.int64)
    row[:, :widest] = torch.where(inside[:, None], reach[req, u].round().long(), 0)
    word = (row.view(tokens, words, 32) << torch.arange(32, device=dev)).sum(2)
    return torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)


def _round_fp8(x, fmt):
    return x.clamp(-FP8_MAX[fmt], FP8_MAX[fmt]).to(DTYPES[fmt]) if fmt in FP8_MAX else x.to(DTYPES[fmt])


def _rope(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    q, k, v = s["qkv"][:, :hq], s["qkv"][:, hq:hq + hkv], s["qkv"][:, hq + hkv:]
    if own:
        s["pa"].pafp8_norm_rope_append(
            q, k, v, s["q_weight"], s["k_weight"], s["cos_sin"], s["positions"], s["slots"], s["q_out"], s["k_cache"],
            s["v_cache"], eps=s["eps"], pair_axis=s["pair_axis"], interleaved=c["interleaved"], q_scale=s["q_scale"],
            k_scale=s["k_scale"], v_scale=s["v_scale"], kv_layout=c["layout"])
        return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    half = c["rot"] // 2
    pos = s["positions"].long()
    if s["pair_axis"] is None:
        cos, sin = s["cos_sin"][pos[0], :half], s["cos_sin"][pos[0], half:]
    else:
        pair = torch.arange(half, device=pos.device)
        at = pos.t()[:, s["pair_axis"].long()]
        cos, sin = s["cos_sin"][at, pair], s["cos_sin"][at, half + pair]
    q = _turn(_normed(q.float(), s["q_weight"], s["eps"]), cos[:, None], sin[:, None], c["interleaved"])
    k = _turn(_normed(k.float(), s["k_weight"], s["eps"]), cos[:, None], sin[:, None], c["interleaved"])
    _put(s["k_cache"], k * torch.tensor(1.0 / s["k_scale"], dtype=torch.float32), s["slots"], c)
    _put(s["v_cache"], v.float() * torch.tensor(1.0 / s["v_scale"], dtype=torch.float32), s["slots"], c)
    return dict(q=_round_fp8(q * torch.tensor(1.0 / s["q_scale"], dtype=torch.float32), c["q_out"]), k_cache=s["k_cache"],
                v_cache=s["v_cache"])


def _normed(x, w, eps):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()


def _turn(x, cos, sin, interleaved):
    half = cos.shape[-1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y, z], -1).flatten(-2) if interleaved else torch.cat([y, z], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _put(cache, x, slots, c):
    """Rows x [n, heads, d] to the cache's slots, rounded to its type."""
    size = {1: torch.uint8, 2: torch.int16}[cache.element_size()]
    rows = _round_fp8(x, c["kv"]).view(size)
    page, at = slots // c["page_size"], slots % c["page_size"]
    if c["layout"] == "NHD":
        cache.view(size)[page, at] = rows
    else:
        cache.view(size)[page, :, at] = rows


def _tree(s):
    c = s["case"]
    if own:
        s["plan"].run_tree(s["q"], s["k_cache"], s["v_cache"], s["kv_indices"], s["mask"], s["o"], s["lse"], s["workspace"],
                           q_scale=s["q_scale"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return dict(o=s["o"], lse=s["lse"])
    batch, hq, hkv, d, ps = c["batch"], c["hq"], c["hkv"], c["d"], c["page_size"]
    group = hq // hkv
    top, widest = max(s["kv_lens"]), max(1, max(s["qo_lens"]))
    pages = _ceil(top, ps)
    length = pages * ps
    dev = s["q"].device
    kv_indptr, qo_indptr = s["kv_indptr"].long(), s["qo_indptr"].long()
    at = kv_indptr[:-1, None] + torch.arange(pages, device=dev)
    ids = s["kv_indices"][at.clamp(max=s["kv_indices"].numel() - 1)].long()
    ids = torch.where(at < kv_indptr[1:, None], ids, 0)
    k, v = _gathered(s["k_cache"], ids, c), _gathered(s["v_cache"], ids, c)  # [batch, hkv, length, d]
    n = s["q"].shape[0]
    t = torch.arange(n, device=dev)
    req = torch.searchsorted(qo_indptr, t, right=True) - 1
    u = t - qo_indptr[req]
    q = torch.zeros(batch, widest, hq, d, device=dev)
    q[req, u] = s["q"].float()
    q = q.view(batch, widest, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(batch, hkv, widest * group, d)
    logits = (q @ k.transpose(2, 3)).mul_(s["sm_scale"] * s["q_scale"] * s["k_scale"]).view(batch, hkv, widest, group, length)
    # Visible keys of every drafted token: the context, then the mask's bits.
    j = torch.arange(length, device=dev)
    new = qo_indptr[1:] - qo_indptr[:-1]
    w = j[None] - (s["kv_len"].long() - new)[:, None]
    bits = torch.zeros(batch, widest, 32 * s["mask"].shape[1], device=dev, dtype=torch.int32)
    bits[req, u] = _bits(s["mask"])
    seen = bits.gather(2, w.clamp(0, bits.shape[2] - 1)[:, None].expand(-1, widest, -1)) > 0
    seen = (seen | (w < 0)[:, None]) & (j[None] < s["kv_len"][:, None])[:, None]
    logits = logits.masked_fill_(~seen[:, None, :, None], -math.inf)
    m = logits.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    p = logits.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(batch, hkv, widest * group, length) @ v).view(batch, hkv, widest, group, d)
    o = torch.where(total > 0, o / total, 0.0) * s["v_scale"]
    lse = (total.log() + m).squeeze(-1)
    o = o.permute(0, 2, 1, 3, 4).reshape(batch, widest, hq, d)[req, u].to(s["o"].dtype)
    return dict(o=o, lse=lse.permute(0, 2, 1, 3).reshape(batch, widest, hq)[req, u])


def _gathered(cache, ids, c):
    """The requests' keys or values in fp32, [batch, hkv, length, d]."""
    rows = cache.view({1: torch.uint8, 2: torch.int16}[cache.element_size()])[ids].view(cache.dtype).float()
    if c["layout"] == "NHD":
        return rows.flatten(1, 2).transpose(1, 2)
    return rows.transpose(1, 2).flatten(2, 3)


# ---- what a pass cannot do without ----------------------------------------

def work(case):
    c = case
    if c["op"] == "tables":
        kv, new = _lengths(c)
        ps = c["page_size"]
        pages = sum(_ceil(a + b, ps) for a, b in zip(kv, new))
        fresh = pages - sum(_ceil(a, ps) for a in kv)
        words = _ceil(max(1, c["new_max"]), 32)
        # Lengths; page ids in and out (fresh ones into the block table too); per token its parent, request,
        # position, slot, rotary position and mask.
        return {"bytes": 8 * c["batch"] + 12 * c["batch"] + 8 * pages + 4 * fresh + sum(new) * (4 + 4 + 4 + 8 + 4 + 4 * words),
                "flops": pages + sum(new)}
    if c["op"] == "rope":
        row = c["d"] * ((c["hq"] + 2 * c["hkv"]) * BYTES[c["src"]] + c["hq"] * BYTES[c["q_out"]] +
                        2 * c["hkv"] * BYTES[c["kv"]])
        return {"bytes": c["tokens"] * (row + 4 * c["axes"] + 8 + 4 * c["rot"]),
                "flops": c["tokens"] * (c["hq"] + c["hkv"]) * (4 * c["d"] + 3 * c["rot"])}
    kv, new = _lengths(c)
    kv = [max(a, b) for a, b in zip(kv, new)]
    keys = sum(a for a, b in zip(kv, new) if b)
    rows = sum(new) * c["hq"]
    return {"bytes": 2 * keys * c["hkv"] * c["d"] * BYTES[c["kv"]] + rows * (c["d"] * (BYTES[c["q"]] + 2) + 4) +
            4 * sum(_ceil(a, c["page_size"]) for a in kv) + 4 * sum(new) * _ceil(max(1, c["new_max"]), 32),
            "flops": 4 * c["d"] * c["hq"] * sum(a * b for a, b in zip(kv, new))}


# ---- the definitions in 64 bits -------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    return {"tables": _exact_tables, "rope": _exact_rope, "tree": _exact_tree}[case["op"]](s, case)


def _exact_tables(s, c):
    return None  # whole numbers: the plain form's are the definition's


def _exact_rope(s, c):
    hq, hkv, half = c["hq"], c["hkv"], c["rot"] // 2
    x = s["qkv"].double()
    first = [2 * i if c["interleaved"] else i for i in range(half)]
    second = [2 * i + 1 if c["interleaved"] else half + i for i in range(half)]
    axis = [0] * half if s["pair_axis"] is None else s["pair_axis"].tolist()
    angles = s["cos_sin"].double()
    pos = s["positions"].long()
    for lo, hi, w in ((0, hq, s["q_weight"]), (hq, hq + hkv, s["k_weight"])):
        part = x[:, lo:hi]
        if w is not None:
            part = part / (part.pow(2).sum(-1, keepdim=True) / c["d"] + s["eps"]).sqrt() * w.double()
        done = part.clone()
        for i in range(half):
            cos, sin = angles[pos[axis[i]], i][:, None], angles[pos[axis[i]], half + i][:, None]
            a, b = part[..., first[i]], part[..., second[i]]
            done[..., first[i]], done[..., second[i]] = a * cos - b * sin, a * sin + b * cos
        x[:, lo:hi] = done
    out = dict(q=x[:, :hq] / s["q_scale"], k_cache=None, v_cache=None)
    if c["q_out"] in FP8_MAX:
        out["q"] = out["q"].clamp(-FP8_MAX[c["q_out"]], FP8_MAX[c["q_out"]])
    if c["kv"] == "e5m2":
        return out  # two bits of mantissa: the type's own rounding (5 %) would hide every error of the arithmetic
    for name, part, scale in (("k_cache", x[:, hq:hq + hkv], s["k_scale"]), ("v_cache", x[:, hq + hkv:], s["v_scale"])):
        cache = s[name].double()
        flat = cache if c["layout"] == "NHD" else cache.transpose(1, 2).contiguous()
        shape = flat.shape
        flat = flat.reshape(-1, *shape[2:])
        flat[s["slots"]] = part / scale
        flat = flat.view(shape)
        out[name] = flat if c["layout"] == "NHD" else flat.transpose(1, 2).contiguous()
        if c["kv"] in FP8_MAX:
            out[name] = out[name].clamp(-FP8_MAX[c["kv"]], FP8_MAX[c["kv"]])
    return out


def _exact_tree(s, c):
    if work(c)["flops"] > 1.5e12:
        return None
    hkv, group, d, ps = c["hkv"], c["hq"] // c["hkv"], c["d"], c["page_size"]
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for b, (length, new) in enumerate(zip(s["kv_lens"], s["qo_lens"])):
        if not new:
            continue
        ids = s["kv_indices"][s["kv_indptr_h"][b]:s["kv_indptr_h"][b + 1]].tolist()
        r0 = s["qo_indptr_h"][b]
        words = [[x & 0xFFFFFFFF for x in row] for row in s["mask"][r0:r0 + new].tolist()]
        hidden = torch.tensor([[not (row[w // 32] >> (w % 32)) & 1 for w in range(new)] for row in words], device="cuda")
        raw_k = torch.stack([s["k_cache"][i] for i in ids]).double()
        raw_v = torch.stack([s["v_cache"][i] for i in ids]).double()
        for h in range(hkv):
            if c["layout"] == "NHD":
                k, v = raw_k[:, :, h], raw_v[:, :, h]
            else:
                k, v = raw_k[:, h], raw_v[:, h]
            k, v = k.reshape(-1, d)[:length] * s["k_scale"], v.reshape(-1, d)[:length] * s["v_scale"]
            q = s["q"][r0:r0 + new, h * group:(h + 1) * group].double() * s["q_scale"]
            z = torch.einsum("ugd,jd->ugj", q, k) * s["sm_scale"]
            z[:, :, length - new:].masked_fill_(hidden[:, None], -math.inf)
            lse[r0:r0 + new, h * group:(h + 1) * group] = torch.logsumexp(z, -1)
            weight = torch.nan_to_num(torch.softmax(z, -1), nan=0.0)
            o[r0:r0 + new, h * group:(h + 1) * group] = torch.einsum("ugj,jd->ugd", weight, v)
    return dict(o=o, lse=lse)
