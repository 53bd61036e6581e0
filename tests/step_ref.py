"""Plain restatements of the step operators (tables, norm + rotation + append,
tree attention) for tests: Python loops and float64, no library code."""
from __future__ import annotations

import math

import numpy as np
import torch

FP8_MAX = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
# Half a step relative to the value, and half the smallest step.
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float8_e4m3fn: 2.0 ** -4,
        torch.float8_e5m2: 2.0 ** -3}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float8_e4m3fn: 2.0 ** -10,
        torch.float8_e5m2: 2.0 ** -17}


def tables(cached, new, table, free, used, *, page_size, num_pages, max_pages, max_tokens, parents=None, words=0):
    """The outputs of one step's tables; table is a [batch, width] array.
    Entries the operator leaves alone are 0."""
    table = np.array(table)
    out = dict(kv_indptr=[0], qo_indptr=[0], last_page_len=[], block_table=table,
               kv_indices=np.zeros(max_pages, np.int64), batch_indices=np.full(max_tokens, -1),
               positions=np.zeros(max_tokens, np.int64), slots=np.full(max_tokens, -1),
               rope_positions=np.zeros(max_tokens, np.int64), tree_mask=np.zeros((max_tokens, max(1, words)), np.uint32))
    take, bad = used, False
    for b, (c, n) in enumerate(zip(cached, new)):
        have, total = -(-c // page_size), -(-(c + n) // page_size)
        row = []
        for j in range(total):
            if j < have:
                page = int(table[b, j]) if j < table.shape[1] else -1
            else:
                page = int(free[take]) if take < len(free) and j < table.shape[1] else -1
                take += 1
                if j < table.shape[1]:
                    table[b, j] = page
            bad |= not 0 <= page < num_pages
            row.append(page)
        k0, t0 = out["kv_indptr"][-1], out["qo_indptr"][-1]
        for j, page in enumerate(row):
            if k0 + j < max_pages:
                out["kv_indices"][k0 + j] = page
            else:
                bad = True
        for u in range(n):
            t = t0 + u
            if t >= max_tokens:
                bad = True
                continue
            pos = c + u
            page = row[pos // page_size]
            out["batch_indices"][t], out["positions"][t] = b, pos
            out["slots"][t] = page * page_size + pos % page_size if 0 <= page < num_pages else -1
            chain, a = [u], u
            while True:
                up = (a - 1 if parents is None else int(parents[t0 + a]))
                if not 0 <= up < a:
                    bad |= up != -1
                    break
                chain.append(up)
                a = up
            out["rope_positions"][t] = c + len(chain) - 1
            for a in chain:
                if a < 32 * words:
                    out["tree_mask"][t, a // 32] |= np.uint32(1 << (a % 32))
            bad |= words > 0 and u >= 32 * words
        out["kv_indptr"].append(k0 + total)
        out["qo_indptr"].append(t0 + n)
        out["last_page_len"].append(c + n - (total - 1) * page_size if total else 0)
    out["free_used"] = [min(take, max(len(free), used))]
    return out, bad


def norm_rope(x, w, eps, cos_sin, positions, axis, interleaved):
    """x [n, heads, D] -> (normed and rotated rows, what their terms amount to
    without cancellation), float64."""
    x = x.double()
    n, heads, d = x.shape
    rot = cos_sin.shape[1]
    half = rot // 2
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    y, mag = x.clone(), x.abs()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        at = positions[int(axis[i])].long()
        c, s = cos_sin[at, i].double()[:, None], cos_sin[at, half + i].double()[:, None]
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, mag


def assert_rounded(got, ref, mag, scale, what, arithmetic=2.0 ** -20):
    """got (a tensor of its type) is ref / scale rounded once, saturating, after
    fp32 arithmetic that is off by `arithmetic` of mag / scale at most."""
    dt = got.dtype
    v = ref / scale
    if dt in FP8_MAX:
        v = v.clamp(-FP8_MAX[dt], FP8_MAX[dt])
    slack = mag / scale * arithmetic
    tol = (v.abs() + slack) * HALF[dt] + TINY[dt] + slack
    err = (got.double() - v).abs() - tol
    assert float(err.max()) <= 0, f"{what}: off by {float((got.double() - v).abs().max())}, {float(err.max())} too much"


def tree_rows(q, k, v, visible, *, sm_scale):
    """One (request, KV head): q [rows, D], k and v [keys, D] in float64 and
    visible [rows, keys] -> (o, lse); a row that sees nothing gives 0, -inf."""
    o = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64)
    lse = torch.full((q.shape[0],), -math.inf, dtype=torch.float64)
    z = (q @ k.t()) * sm_scale
    for r in range(q.shape[0]):
        seen = visible[r].nonzero().flatten()
        if len(seen):
            zz = z[r, seen]
            m = zz.max()
            e = (zz - m).exp()
            o[r] = (e[:, None] * v[seen]).sum(0) / e.sum()
            lse[r] = m + e.sum().log()
    return o, lse
