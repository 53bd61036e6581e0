"""The operators of a paged fp8 cache with a scale for each block of tokens and
head, and of attention with a sliding window, as timed work.

* ``append``  new tokens quantised into the cache as they are written: every
  16-token block of every KV head has its own power-of-two scale, which grows
  with what is written (the block's earlier codes are then written anew);
* ``read``    ranges of a request's tokens read back into plain rows, from a
  cache with block scales or with one scale per tensor;
* ``attn``    decode or causal prefill attention over such a cache, over the
  whole context or over a sliding window and a few first tokens that stay
  visible, the window also over a cache with one scale per tensor and over a
  2-byte one.

``run`` computes them in plain torch operations where ``own`` is false and
calls the library's entry points where it is true.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3fn": torch.float8_e4m3fn,
          "e5m2": torch.float8_e5m2}
FP8_MAX = {"e4m3fn": 448.0, "e5m2": 57344.0}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3fn": 1, "e5m2": 1}
BLOCK = 16  # tokens that share a scale


def listed():
    return [
        # One decode step of the serving batch (a token a request): latency.
        dict(name="append_step", op="append", batch=64, kv_min=512, kv_max=4096, new_min=1, new_max=1, hkv=8, d=128,
             src="bf16", kv="e4m3fn", layout="NHD", page_size=16, packed=True, lens=1),
        # The new tokens of the ragged prefill batch.
        dict(name="append_prefill", op="append", batch=16, kv_min=0, kv_max=2048, new_min=128, new_max=1024, hkv=8, d=128,
             src="bf16", kv="e4m3fn", layout="NHD", page_size=16, packed=True, lens=2),
        # Long prompts into head-major pages of 32 tokens, head_dim 64, e5m2, contiguous rows, odd lengths.
        dict(name="append_long", op="append", batch=5, kv_min=0, kv_max=999, new_min=5001, new_max=8191, hkv=6, d=64,
             src="f16", kv="e5m2", layout="HND", page_size=32, packed=False, lens=3),
        # One short request's prefix, to move it: latency.
        dict(name="read_one", op="read", batch=1, kv_min=333, kv_max=333, all=False, hkv=8, d=128, kv="e4m3fn", out="bf16",
             blocks=True, layout="NHD", page_size=16, lens=4),
        # The whole serving batch's cache in bf16, for a step that wants plain rows.
        dict(name="read_serving", op="read", batch=64, kv_min=512, kv_max=4096, all=True, hkv=8, d=128, kv="e4m3fn",
             out="bf16", blocks=True, layout="NHD", page_size=16, lens=5),
        # One short request's decode step: latency.
        dict(name="blocks_one", op="attn", mode="decode", batch=1, kv_min=333, kv_max=333, new_min=1, new_max=1, hq=8, hkv=2,
             d=128, q="bf16", kv="e4m3fn", blocks=True, window=0, sinks=0, layout="NHD", page_size=16, lens=6),
        # The serving decode batch over block scales.
        dict(name="blocks_serving", op="attn", mode="decode", batch=64, kv_min=512, kv_max=4096, new_min=1, new_max=1, hq=32,
             hkv=8, d=128, q="bf16", kv="e4m3fn", blocks=True, window=0, sinks=0, layout="NHD", page_size=16, lens=7),
        # The ragged prefill batch over block scales.
        dict(name="blocks_prefill", op="attn", mode="prefill", batch=16, kv_min=0, kv_max=2048, new_min=128, new_max=1024,
             hq=32, hkv=8, d=128, q="bf16", kv="e4m3fn", blocks=True, window=0, sinks=0, layout="NHD", page_size=16, lens=8),
        # Decode of long chats whose layer sees the last 4096 tokens and the first 4.
        dict(name="window_serving", op="attn", mode="decode", batch=64, kv_min=1000, kv_max=32768, new_min=1, new_max=1,
             hq=32, hkv=8, d=128, q="bf16", kv="e4m3fn", blocks=False, window=4096, sinks=4, layout="NHD", page_size=16,
             lens=9),
        # A long prompt through such a layer with a window of 1024.
        dict(name="window_prefill", op="attn", mode="prefill", batch=1, kv_min=2000, kv_max=2000, new_min=16384,
             new_max=16384, hq=32, hkv=8, d=128, q="bf16", kv="e4m3fn", blocks=False, window=1024, sinks=4, layout="NHD",
             page_size=16, lens=10),
        # Both together: long context, e5m2, head-major pages of 32, an odd window.
        dict(name="window_blocks", op="attn", mode="decode", batch=8, kv_min=32768, kv_max=32768, new_min=1, new_max=1,
             hq=64, hkv=8, d=128, q="f16", kv="e5m2", blocks=True, window=5001, sinks=20, layout="HND", page_size=32,
             lens=11),
        # A 2-byte cache and a short odd window, ragged prompts.
        dict(name="window_bf16_cache", op="attn", mode="prefill", batch=9, kv_min=0, kv_max=1500, new_min=100, new_max=2500,
             hq=16, hkv=4, d=128, q="bf16", kv="bf16", blocks=False, window=333, sinks=7, layout="NHD", page_size=16,
             lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "attn", "attn", "attn", "attn"])
    c = dict(op=op, lens=rng.randrange(1 << 30), layout=rng.choice(["NHD", "HND"]), page_size=rng.choice([16, 16, 32, 48, 64]),
             d=rng.choice([128, 128, 64]), hkv=rng.choice([1, 2, 4, 6, 8]))
    if op == "append":
        total = _log(rng, 1, 30000)
        batch = min(total, _log(rng, 1, 128))
        top = total // batch
        return dict(c, batch=batch, kv_min=0, kv_max=_log(rng, 1, 4096), new_min=rng.choice([0, 1, top]), new_max=top,
                    src=rng.choice(["bf16", "bf16", "f16", "f32"]), kv=rng.choice(["e4m3fn", "e4m3fn", "e5m2"]),
                    packed=rng.choice([False, True]))
    if op == "read":
        total = _log(rng, 1, 60000)
        batch = min(total, _log(rng, 1, 128))
        top = total // batch
        return dict(c, batch=batch, kv_min=rng.choice([0, top // 2, top]), kv_max=top, all=rng.choice([False, True]),
                    kv=rng.choice(["e4m3fn", "e5m2"]), out=rng.choice(["bf16", "f16", "f32"]), blocks=rng.choice([True, True, False]))
    mode = rng.choice(["decode", "prefill"])
    blocks = rng.choice([False, True])
    q = rng.choice(["bf16", "bf16", "f16", "e4m3fn", "e5m2"])
    kinds = ["e4m3fn", "e4m3fn", "e5m2"]
    if not blocks and q in ("bf16", "f16"):
        kinds += [q] if mode == "prefill" else ["bf16", "f16"]
    kv = rng.choice(kinds)
    group = rng.choice([1, 2, 4, 5, 8] if mode == "decode" else [1, 2, 3, 4, 8, 16])
    c.update(mode=mode, blocks=blocks, q=q, kv=kv, hq=c["hkv"] * group)
    window = 0 if blocks and rng.random() < 0.5 else _log(rng, 1, 8192)
    c.update(window=window, sinks=rng.choice([0, 1, 4, 16, 77]) if window else 0)
    if mode == "decode":
        # At most the keys of the listed decode batches.
        top = _log(rng, 1, 32768)
        seen = top if not window else min(top, window + c["sinks"])
        batch = max(1, min(_log(rng, 1, 128), (1 << 17) // seen, (1 << 20) // top))
        return dict(c, batch=batch, kv_min=rng.choice([0, top // 8, top]), kv_max=top, new_min=1, new_max=1)
    # At most the products of the listed prompts: rows x keys x query heads x head_dim.
    rows = _log(rng, 1, 8192)
    cached = rng.choice([0, _log(rng, 1, 4096)])
    seen = cached + rows if not window else min(cached + rows, window + c["sinks"] + 128)
    most = int(2.0e10 / (seen * c["hq"] * c["d"]))
    rows = max(1, min(rows, most))
    batch = max(1, min(_log(rng, 1, 16), most // rows))
    return dict(c, batch=batch, kv_min=0, kv_max=cached, new_min=rng.choice([0, 1, rows]), new_max=rows)


def _lengths(case):
    """Every request's (tokens before the step, new tokens), from the case alone."""
    r = random.Random(case["lens"])
    kv = [r.randint(case["kv_min"], case["kv_max"]) for _ in range(case["batch"])]
    if case["op"] == "read":
        # (first token read, tokens read): all of them, or an inner part.
        part = [(0, a) if case["all"] else (r.randint(0, a // 4), a) for a in kv]
        return [a for a, _ in part], [b - a for a, b in part]
    if case["op"] == "attn" and case["mode"] == "decode":
        return [max(0, a - 1) for a in kv], [min(1, a) for a in kv]
    return kv, [r.randint(case["new_min"], case["new_max"]) for _ in range(case["batch"])]


def _ceil(a, b):
    return -(-a // b)


def _scan(xs):
    out = [0]
    for x in xs:
        out.append(out[-1] + x)
    return out


def _int(xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


def _power(amax, fmt):
    """The smallest power of two, 2^-64 at least, that brings amax into the type's range."""
    m, e = torch.frexp(amax)
    e = e - {"e4m3fn": 9, "e5m2": 16}[fmt] + (m > 0.875).to(e.dtype)  # 448 = 0.875 * 2^9, 57344 = 0.875 * 2^16
    return (torch.where(amax > 0, e, -64).clamp(min=-64) + 127 << 23).view(torch.float32)


def _round_to(x, fmt):
    return x.clamp(-FP8_MAX[fmt], FP8_MAX[fmt]).to(DTYPES[fmt]) if fmt in FP8_MAX else x.to(DTYPES[fmt])


def _raw(t):
    """The tensor as integers of its size (indexing is not defined for every 8-bit type)."""
    return t.view({1: torch.uint8, 2: torch.int16}[t.element_size()])


# ---- inputs ---------------------------------------------------------------

def _cache(c, pool, g):
    """One pool of pages in the case's layout, and its scales: fp8 codes with a scale for each block and
    head (heads and blocks of unlike magnitude; powers of two, as the append writes them) or one for the tensor."""
    ps, hkv, d, per = c["page_size"], c["hkv"], c["d"], c["page_size"] // BLOCK
    size = 2.0 ** (0.7 * torch.randn(pool, per, 1, hkv, 1, device="cuda", generator=g))
    x = torch.empty(pool, per, BLOCK, hkv, d, device="cuda", dtype=DTYPES[c["kv"]])
    step = max(1, (1 << 28) // (ps * hkv * d))
    scales = torch.empty(pool, per, hkv, device="cuda")
    for at in range(0, pool, step):
        part = torch.randn(min(step, pool - at), per, BLOCK, hkv, d, device="cuda", generator=g)
        if c["kv"] not in FP8_MAX:
            x[at:at + step] = part.to(x.dtype)
        elif c["op"] == "append" or c["blocks"]:
            part *= size[at:at + step]
            s = _power(part.abs().amax((2, 4)), c["kv"])
            scales[at:at + step] = s
            _raw(x)[at:at + step] = _raw(_round_to(part / s[:, :, None, :, None], c["kv"]))
        else:
            _raw(x)[at:at + step] = _raw(_round_to(part / _scale(c["kv"]), c["kv"]))
    x = x.view(pool, ps, hkv, d)
    if c["layout"] == "HND":
        x = _raw(x).transpose(1, 2).contiguous().view(x.dtype)
    return x, scales


def _scale(fmt):
    return 5.5 / FP8_MAX[fmt] if fmt in FP8_MAX else 1.0


def _inputs(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(int(seed))
    first, count = _lengths(c)
    ps, hkv, d = c["page_size"], c["hkv"], c["d"]
    lens = [a + b for a, b in zip(first, count)]
    npages = [_ceil(n, ps) for n in lens]
    pool, kv_indptr, rows = sum(npages) + 5, _scan(npages), _scan(count)
    ids = torch.randperm(pool, device="cuda", generator=g)[:max(1, kv_indptr[-1])].to(torch.int32)
    k, ks = _cache(c, pool, g)
    v, vs = _cache(c, pool, g)
    n = rows[-1]
    s = dict(case=c, k_cache=k, v_cache=v, k_scales=ks, v_scales=vs, kv_indices=ids, first=_int(first), lens=lens,
             kv_indptr=_int(kv_indptr), rows=_int(rows), kv_indptr_h=kv_indptr, rows_h=rows, pool=pool, n=n,
             k_scale=_scale(c["kv"]), v_scale=_scale(c["kv"]))
    if c["op"] == "append":
        # The projection's output: keys and values of a token side by side, or two tensors; a few large channels.
        x = torch.randn(n, 2, hkv, d, device="cuda", generator=g) * (1 + 6 * (torch.rand(d, device="cuda", generator=g) > 0.97))
        x = (x * 2.0 ** (0.7 * torch.randn(n, 2, 1, 1, device="cuda", generator=g))).to(DTYPES[c["src"]])
        begun = [b for b in range(c["batch"]) if count[b] and first[b] % BLOCK]
        s["begun"] = torch.tensor(begun, dtype=torch.int64, device="cuda")
        s["live"] = torch.tensor([(i, t) for i, b in enumerate(begun) for t in range(first[b] % BLOCK)], dtype=torch.int64,
                                 device="cuda").view(-1, 2)
        s["k_new"], s["v_new"] = (x[:, 0], x[:, 1]) if c["packed"] else (x[:, 0].contiguous(), x[:, 1].contiguous())
    elif c["op"] == "read":
        s["k_out"] = torch.zeros(n, hkv, d, device="cuda", dtype=DTYPES[c["out"]])
        s["v_out"] = torch.zeros_like(s["k_out"])
    else:
        s["q_scale"], s["sm_scale"] = _scale(c["q"]), 1.0 / math.sqrt(d)
        # A decode batch has a row for every request, one without tokens too.
        n = c["batch"] if c["mode"] == "decode" else n
        s["q"] = _round_to(torch.randn(n, c["hq"], d, device="cuda", generator=g) / s["q_scale"], c["q"])
        s["o"] = torch.zeros(n, c["hq"], d, device="cuda", dtype=DTYPES["bf16" if c["q"] in FP8_MAX else c["q"]])
        s["lse"] = torch.zeros(n, c["hq"], device="cuda")
        s["blocks_of_rows"] = _row_blocks(c, first, count, lens)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import paged_attention_fp8_gb300 as pa
        s["pa"] = pa
        if case["op"] == "attn":
            ps = case["page_size"]
            s["plan"] = pa.Plan(mode=case["mode"], num_qo_heads=case["hq"], num_kv_heads=case["hkv"], num_pages=s["pool"],
                                kv_indptr=s["kv_indptr_h"],
                                last_page_len=[a - (_ceil(a, ps) - 1) * ps if a else 0 for a in s["lens"]],
                                qo_indptr=s["rows_h"] if case["mode"] == "prefill" else None, q_dtype=case["q"],
                                kv_dtype=case["kv"], head_dim=case["d"], page_size=ps, kv_layout=case["layout"],
                                window=case["window"], sinks=case["sinks"])
            s["workspace"] = torch.empty(s["plan"].workspace_bytes, dtype=torch.uint8, device="cuda")
            s["plan"].upload(s["workspace"])
    return s


# ---- one pass -------------------------------------------------------------

def run(s):
    return {"append": _append, "read": _read, "attn": _attn}[s["case"]["op"]](s)


def _token_slots(s):
    """Page and slot in it of every row of the step (rows s["rows"][b] .. of request b, from its token s["first"][b])."""
    ps = s["case"]["page_size"]
    t = torch.arange(s["n"], device="cuda")
    rows = s["rows"].long()
    req = torch.searchsorted(rows, t, right=True) - 1
    pos = s["first"].long()[req] + t - rows[req]
    return s["kv_indices"].long()[s["kv_indptr"].long()[req] + pos // ps], pos % ps


def _append(s):
    c = s["case"]
    if own:
        s["pa"].pafp8_append_kv_blocks(s["k_new"], s["v_new"], s["rows"], s["first"], s["kv_indptr"], s["kv_indices"],
                                       s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], kv_layout=c["layout"])
    elif s["n"]:
        page, at = _token_slots(s)
        ps, per = c["page_size"], c["page_size"] // BLOCK
        block = page * per + at // BLOCK
        # The block that a request's first new token finds begun, if it does: its tokens before that one stay.
        first = s["first"].long()[s["begun"]]
        old_page = s["kv_indices"].long()[s["kv_indptr"].long()[s["begun"]] + first // ps]
        old_block = old_page * per + first % ps // BLOCK
        which, tok = s["live"].unbind(1)
        live = (which, old_page[which], (first % ps // BLOCK * BLOCK)[which] + tok)
        for name in ("k", "v"):
            _append_one(s[name + "_new"].float(), s[name + "_cache"], s[name + "_scales"].view(-1, c["hkv"]), c, page, at, block,
                        old_block, live)
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"], k_scales=s["k_scales"], v_scales=s["v_scales"])


def _append_one(x, cache, scales, c, page, at, block, old_block, live):
    """Rows x to their places; block: the block of scales of each row, old_block: the begun ones; live: the earlier
    tokens of those (which begun block, page, slot)."""
    size = torch.zeros(len(scales), BLOCK, c["hkv"], device=x.device)
    size[block, at % BLOCK] = x.abs().amax(-1)
    fresh = _power(size.amax(1), c["kv"])
    was = scales[old_block]
    fresh[old_block] = torch.maximum(was, fresh[old_block])
    scales[block] = fresh[block]
    raw = _raw(cache) if c["layout"] == "NHD" else _raw(cache).transpose(1, 2)  # [page, token, head, d] either way
    which, old_page, tok = live
    old = raw[old_page, tok].view(cache.dtype).float() * (was / fresh[old_block])[which][:, :, None]
    raw[old_page, tok] = _raw(_round_to(old, c["kv"]))
    raw[page, at] = _raw(_round_to(x / fresh[block][:, :, None], c["kv"]))


def _read(s):
    c = s["case"]
    if own:
        scales = dict(k_scales=s["k_scales"], v_scales=s["v_scales"]) if c["blocks"] else \
            dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
        s["pa"].pafp8_read_kv(s["k_cache"], s["v_cache"], s["rows"], s["first"], s["kv_indptr"], s["kv_indices"], s["k_out"],
                              s["v_out"], kv_layout=c["layout"], **scales)
        return dict(k=s["k_out"], v=s["v_out"])
    page, at = _token_slots(s)
    out = {}
    for name in ("k", "v"):
        scale = s[name + "_scales"][page, at // BLOCK][:, :, None] if c["blocks"] else s[name + "_scale"]
        out[name] = (_tokens(s[name + "_cache"], page, at, c) * scale).to(DTYPES[c["out"]])
    return out


def _tokens(cache, page, at, c):
    """The cache's rows [..., hkv, d] at these pages and slots, in 32 bits and without their scales."""
    raw = _raw(cache) if c["layout"] == "NHD" else _raw(cache).transpose(1, 2)
    return raw[page, at].contiguous().view(cache.dtype).float()


def _row_blocks(c, first, count, lens):
    """The query rows in blocks of up to `most` rows of one request: per block its request, first row in
    it, rows, and the first key past the sinks that one of its rows sees."""
    most = 1 if c["mode"] == "decode" else min(128, max(1, max(count)))
    out = []
    for b in range(c["batch"]):
        for r in range(0, count[b], most):
            low = first[b] + r - c["window"] + 1 if c["window"] else 0
            out.append((b, r, min(most, count[b] - r), max(low, min(c["sinks"], lens[b]))))
    keys = max(lens) if not c["window"] else min(max(lens), c["sinks"] + c["window"] + most)
    return dict(most=most, keys=max(1, keys), table=torch.tensor(out or [(0, 0, 0, 0)], device="cuda"), any=bool(out))


def _attn(s):
    c = s["case"]
    if own:
        if c["blocks"]:
            s["plan"].run_block_scales(s["q"], s["k_cache"], s["v_cache"], s["kv_indices"], s["o"], s["lse"], s["workspace"],
                                       q_scale=s["q_scale"], k_scales=s["k_scales"], v_scales=s["v_scales"])
        else:
            s["plan"].run(s["q"], s["k_cache"], s["v_cache"], s["kv_indices"], s["o"], s["lse"], s["workspace"],
                          q_scale=s["q_scale"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return dict(o=s["o"], lse=s["lse"])
    hq, hkv, d, ps = c["hq"], c["hkv"], c["d"], c["page_size"]
    group, how = hq // hkv, s["blocks_of_rows"]
    o = torch.zeros(s["o"].shape, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, device="cuda")
    if not how["any"]:
        return dict(o=o.to(s["o"].dtype), lse=lse)
    req, r0, rows, low = how["table"].unbind(1)
    blocks, most = len(req), how["most"]
    end = s["first"].long()[req] + s["rows"].long()[req + 1] - s["rows"].long()[req]
    # The keys a block of rows may see: the sinks, then a run from `low` on.
    col = torch.arange(how["keys"], device="cuda")[None]
    sinks = torch.minimum(torch.full_like(end, c["sinks"]), end)[:, None]
    pos = torch.where(col < sinks, col, low[:, None] + col - sinks)
    real = pos < end[:, None]
    pos = torch.where(real, pos, 0)
    page = s["kv_indices"].long()[s["kv_indptr"].long()[req][:, None] + pos // ps]
    k, v = (_tokens(s[name + "_cache"], page, pos % ps, c) * (
        s[name + "_scales"][page, pos % ps // BLOCK][..., None] if c["blocks"] else s[name + "_scale"])
        for name in ("k", "v"))
    k, v = k.transpose(1, 2), v.transpose(1, 2)  # [blocks, hkv, keys, d]
    u = torch.arange(most, device="cuda")[None]
    mine = u < rows[:, None]
    row = (torch.arange(c["batch"], device="cuda") if c["mode"] == "decode" else s["rows"].long())[req][:, None] + r0[:, None] + u
    row = torch.where(mine, row, 0)
    q = (s["q"].float() * s["q_scale"])[row].view(blocks, most, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(
        blocks, hkv, most * group, d)
    z = (q @ k.transpose(2, 3)).mul_(s["sm_scale"]).view(blocks, hkv, most, group, -1)
    at = (s["first"].long()[req] + r0)[:, None] + u  # the rows' own positions
    seen = real[:, None] & (pos[:, None] <= at[:, :, None])
    if c["window"]:
        seen &= (pos[:, None] < c["sinks"]) | (pos[:, None] > at[:, :, None] - c["window"])
    z = z.masked_fill_(~seen[:, None, :, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    p = z.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(blocks, hkv, most * group, -1) @ v).view(blocks, hkv, most, group, d)
    out = (out / total).permute(0, 2, 1, 3, 4).reshape(blocks, most, hq, d)
    logs = (total.log() + m).squeeze(-1).permute(0, 2, 1, 3).reshape(blocks, most, hq)
    o[row[mine]], lse[row[mine]] = out[mine], logs[mine]
    return dict(o=o.to(s["o"].dtype), lse=lse)


# ---- what a pass cannot do without ----------------------------------------

def _pairs(c, first, count):
    """(query row, key) pairs that a window and causality leave, and the keys that some row sees."""
    pairs = keys = 0
    for a, n in zip(first, count):
        w, sinks = c["window"], c["sinks"]
        if not w:
            pairs += n * a + n * (n + 1) // 2
            keys += a + n if n else 0
            continue
        # Row p sees p + 1 keys while all are in its window or among the sinks, window + sinks of them after.
        full = w + sinks
        short = max(0, min(n, full - 1 - a))  # rows whose p + 1 < full
        pairs += short * a + short * (short + 1) // 2 + (n - short) * full
        keys += (a + n if a + 1 <= full else n + full - 1) if n else 0
    return pairs, keys


def work(case):
    c = case
    first, count = _lengths(c)
    n, d, hkv = sum(count), c["d"], c["hkv"]
    ids = 4 * sum(_ceil(a + b, c["page_size"]) for a, b in zip(first, count))
    if c["op"] == "append":
        blocks = sum(_ceil(a + b, BLOCK) - a // BLOCK for a, b in zip(first, count) if b)
        begun = sum(1 for a, b in zip(first, count) if b and a % BLOCK)
        return {"bytes": 2 * hkv * (n * d * (BYTES[c["src"]] + 1) + 4 * blocks + 4 * begun), "flops": 4 * n * hkv * d}
    if c["op"] == "read":
        blocks = sum(_ceil(a + b, BLOCK) - a // BLOCK for a, b in zip(first, count) if b) if c["blocks"] else 0
        return {"bytes": 2 * hkv * (n * d * (BYTES[c["out"]] + 1) + 4 * blocks), "flops": 2 * n * hkv * d}
    pairs, keys = _pairs(c, first, count)
    ids = min(ids, 4 * _ceil(keys, c["page_size"]) + 8 * c["batch"])
    return {"bytes": 2 * keys * hkv * d * BYTES[c["kv"]] + (8 * hkv * _ceil(keys, BLOCK) if c["blocks"] else 0) + ids +
            n * c["hq"] * (d * (BYTES[c["q"]] + 2) + 4), "flops": 4 * d * c["hq"] * pairs}


# ---- the definitions in 64 bits -------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attn": _exact_attn}[case["op"]](s, case)


def _exact_rows(s, c, name, b):
    """Request b's codes [tokens, hkv, d] and the places (page, token) they lie at."""
    ps = c["page_size"]
    ids = s["kv_indices"][s["kv_indptr_h"][b]:s["kv_indptr_h"][b + 1]].long()
    codes = s[name + "_cache"][ids].double() if s[name + "_cache"].element_size() > 1 else \
        s[name + "_cache"].view(torch.uint8)[ids].view(s[name + "_cache"].dtype).double()
    if c["layout"] == "HND":
        codes = codes.permute(0, 2, 1, 3)
    return ids, codes.reshape(len(ids) * ps, c["hkv"], c["d"])


def _exponent(x):
    """The binary exponents of |x|."""
    return ((x.abs().view(torch.int64) >> 52) & 2047) - 1023


def _two_to(e):
    return (e + 1023 << 52).view(torch.float64)


def _grid(x, fmt):
    """x to the nearest number of the type, ties to even, in 64 bits."""
    bits, low = {"e4m3fn": (3, -6), "e5m2": (2, -14)}[fmt]
    unit = _two_to(_exponent(x).clamp(min=low) - bits)
    return (torch.round(x / unit) * unit).clamp(-FP8_MAX[fmt], FP8_MAX[fmt])


def _exact_append(s, c):
    out = {}
    ps, per = c["page_size"], c["page_size"] // BLOCK
    for name in ("k", "v"):
        cache, scales = s[name + "_cache"], s[name + "_scales"].double().clone()
        values = cache.double() if c["layout"] == "NHD" else cache.double().transpose(1, 2).contiguous()
        x = s[name + "_new"].double()
        for b in range(c["batch"]):
            a, r0, r1 = int(s["first"][b]), s["rows_h"][b], s["rows_h"][b + 1]
            if r0 == r1:
                continue
            end = a + r1 - r0
            lo, hi = a // BLOCK * BLOCK, _ceil(end, BLOCK) * BLOCK
            # The blocks touched, whole, as numbers; what the step does not write keeps its code.
            t = torch.arange(lo, hi, device="cuda")
            page, at = s["kv_indices"][s["kv_indptr_h"][b] + t // ps].long(), t % ps
            rows = torch.zeros(hi - lo, c["hkv"], c["d"], dtype=torch.float64, device="cuda")
            rows[a - lo:end - lo] = x[r0:r1]
            top = rows.view(-1, BLOCK, c["hkv"], c["d"]).abs().amax((1, 3))
            s2 = _two_to(_exponent(top / FP8_MAX[c["kv"]]).clamp(min=-64))
            s2 = torch.where(top > s2 * FP8_MAX[c["kv"]], 2 * s2, s2)
            p0, q0 = page[::BLOCK], at[::BLOCK] // BLOCK
            before = scales[p0, q0]
            if a > lo:
                s2[0] = torch.maximum(s2[0], before[0])
                values[page[:a - lo], at[:a - lo]] = _grid(values[page[:a - lo], at[:a - lo]] * (before[0] / s2[0])[None, :, None],
                                                           c["kv"])
            scales[p0, q0] = s2
            each = s2.repeat_interleave(BLOCK, 0)[a - lo:end - lo]
            values[page[a - lo:end - lo], at[a - lo:end - lo]] = _grid(x[r0:r1] / each[:, :, None], c["kv"])
        out[name + "_cache"] = values if c["layout"] == "NHD" else values.transpose(1, 2).contiguous()
        out[name + "_scales"] = scales
    return out


def _exact_read(s, c):
    out = {"k": [], "v": []}
    for name in ("k", "v"):
        for b in range(c["batch"]):
            ids, codes = _exact_rows(s, c, name, b)
            if c["blocks"]:
                codes = codes * s[name + "_scales"].double()[ids].reshape(-1, c["hkv"]).repeat_interleave(BLOCK, 0)[:, :, None]
            else:
                codes = codes * s[name + "_scale"]
            a = int(s["first"][b])
            out[name].append(codes[a:a + s["rows_h"][b + 1] - s["rows_h"][b]])
    return {name: torch.cat(x) for name, x in out.items()}


def _exact_attn(s, c):
    if work(c)["flops"] > 1.5e12:
        return None
    hq, hkv, group = c["hq"], c["hkv"], c["hq"] // c["hkv"]
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["lens"]):
        n, a = s["rows_h"][b + 1] - s["rows_h"][b], int(s["first"][b])
        if not n:
            continue
        kv = []
        for name in ("k", "v"):
            ids, codes = _exact_rows(s, c, name, b)
            codes = codes[:length]
            if c["blocks"]:
                kv.append(codes * s[name + "_scales"].double()[ids].reshape(-1, hkv).repeat_interleave(BLOCK, 0)[:length, :, None])
            else:
                kv.append(codes * s[name + "_scale"])
        k, v = kv
        r0 = b if c["mode"] == "decode" else s["rows_h"][b]
        for u in range(0, n, 256):
            rows = torch.arange(u, min(n, u + 256), device="cuda")
            p = a + rows
            keys = torch.arange(length, device="cuda")
            if c["window"]:
                keys = keys[(keys < c["sinks"]) | (keys > a + u - c["window"])]
            keys = keys[keys <= a + int(rows[-1])]
            hidden = keys[None] > p[:, None]
            if c["window"]:
                hidden |= (keys[None] >= c["sinks"]) & (keys[None] <= p[:, None] - c["window"])
            q = s["q"][r0 + u:r0 + u + len(rows)].double().view(len(rows), hkv, group, -1) * s["q_scale"]
            z = torch.einsum("uhgd,jhd->hugj", q, k[keys]) * s["sm_scale"]
            z = z.masked_fill(hidden[None, :, None], -math.inf)
            lse[r0 + u:r0 + u + len(rows)] = torch.logsumexp(z, -1).permute(1, 0, 2).reshape(len(rows), hq)
            o[r0 + u:r0 + u + len(rows)] = torch.einsum("hugj,jhd->uhgd", torch.softmax(z, -1), v[keys]).reshape(
                len(rows), hq, -1)
    return dict(o=o, lse=lse)
