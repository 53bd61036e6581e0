"""Batches for the tree attention tests and their float64 reference."""
from __future__ import annotations

import math

import numpy as np
import torch

import paged_attention_fp8_gb300 as pa
from step_ref import HALF

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8 = ("e4m3fn", "e5m2")
NAN_CODE = {"e4m3fn": 0x7F, "e5m2": 0x7E, "bf16": 0x7FC0, "f16": 0x7E00}


def tree_masks(qo_lens, kind, r, words):
    """uint32 [nnz, words] masks of a kind, and truth values per request."""
    rows, seen = [], []
    for n in qo_lens:
        m = np.zeros((n, n), bool)
        for u in range(n):
            if kind == "tree":
                p = int(r.integers(-1, u)) if u else -1
                if p >= 0:
                    m[u] = m[p]
                m[u, u] = True
            elif kind == "causal":
                m[u, :u + 1] = True
            elif kind == "full":
                m[u] = True
            elif kind == "random":
                m[u] = r.random(n) < 0.4
        if kind == "some_empty" and n:
            m[::2] = r.random((len(m[::2]), n)) < 0.5
        seen.append(m)
        w = np.zeros((n, words), np.uint32)
        for u in range(n):
            for j in range(n):
                if m[u, j]:
                    w[u, j // 32] |= np.uint32(1 << (j % 32))
            for j in range(n, 32 * words):  # bits behind the last token: ignored
                w[u, j // 32] |= np.uint32(1 << (j % 32))
        rows.append(w)
    return np.concatenate(rows + [np.zeros((0, words), np.uint32)]), seen


class TreeBatch:
    def __init__(self, kv_lens, qo_lens, hq, hkv, *, d=128, q="bf16", kv="e4m3fn", o=None, layout="NHD", page_size=16,
                 mask="tree", words=None, seed=0, num_ctas=0, head_scales=False, spread=1.0, device="cuda"):
        r = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.kv_lens, self.qo_lens, self.hq, self.hkv, self.d = list(kv_lens), list(qo_lens), hq, hkv, d
        self.qt, self.kt, self.ot = q, kv, o or ("bf16" if q in FP8 else q)
        self.layout, self.ps = layout, page_size
        npages = [-(-n // page_size) for n in kv_lens]
        pool = sum(npages) + 3
        self.kv_indptr = np.concatenate([[0], np.cumsum(npages)]).astype(np.int32)
        self.qo_indptr = np.concatenate([[0], np.cumsum(qo_lens)]).astype(np.int32)
        self.last = np.array([n - (p - 1) * page_size if p else 0 for n, p in zip(kv_lens, npages)], np.int32)
        ids = r.permutation(pool)[:sum(npages)].astype(np.int32)
        n = int(self.qo_indptr[-1])
        self.q = (torch.randn(n, hq, d, generator=g) * spread).to(DT[q])
        self.k, self.v = [], []
        self.q_scale = 0.8 if q in FP8 else 1.0
        self.ks, self.vs = (0.7, 1.3) if kv in FP8 else (1.0, 1.0)
        self.head_scales = head_scales
        if head_scales:
            self.qs_h = torch.rand(hq, generator=g) + 0.5
            self.ks_h, self.vs_h = torch.rand(hkv, generator=g) + 0.5, torch.rand(hkv, generator=g) + 0.5
        es = 1 if kv in FP8 else 2
        raw = torch.uint8 if es == 1 else torch.int16
        caches = []
        for _ in range(2):
            c = torch.full((pool, page_size, hkv, d), NAN_CODE[kv], dtype=torch.int32).to(raw)  # no token's slot is read
            rows = []
            for b, length in enumerate(kv_lens):
                x = (torch.randn(length, hkv, d, generator=g)).to(DT[kv])
                rows.append(x)
                for p in range(npages[b]):
                    part = x.view(raw)[p * page_size:(p + 1) * page_size]
                    c[int(ids[self.kv_indptr[b] + p]), :len(part)] = part
            (self.k if not self.k and _ == 0 else self.v).extend(rows)
            if layout == "HND":
                c = c.transpose(1, 2).contiguous()
            caches.append(c.to(device).view(DT[kv]))
        self.kc, self.vc = caches
        widest = max(list(qo_lens) + [1])
        words = words or -(-widest // 32)
        bits, self.seen = tree_masks(qo_lens, mask, r, words)
        self.mask = torch.from_numpy(bits.astype(np.int64)).to(torch.int64)
        self.mask = torch.where(self.mask >= 1 << 31, self.mask - (1 << 32), self.mask).to(torch.int32).to(device)
        self.ids = torch.from_numpy(ids).to(device)
        self.pool = pool
        self.plan = pa.Plan(mode="tree", num_qo_heads=hq, num_kv_heads=hkv, num_pages=pool, kv_indptr=self.kv_indptr,
                            last_page_len=self.last, qo_indptr=self.qo_indptr, q_dtype=q, kv_dtype=kv, o_dtype=self.ot,
                            head_dim=d, page_size=page_size, kv_layout=layout, num_ctas=num_ctas)
        self.device = device
        self.n = n

    def run(self, stream=None):
        dev = self.device
        self.ws = torch.empty(self.plan.workspace_bytes, dtype=torch.uint8, device=dev)
        self.plan.upload(self.ws)
        self.o = torch.full((self.n + 1, self.hq, self.d), 7.0, dtype=DT[self.ot], device=dev)
        self.lse = torch.full((self.n + 1, self.hq), 7.0, device=dev)
        self.dq = self.q.to(dev)
        self.call()
        self.plan.device_status(self.ws)
        assert bool((self.o[self.n] == 7).all()) and bool((self.lse[self.n] == 7).all()), "rows behind the last were written"
        return self.o[:self.n].cpu(), self.lse[:self.n].cpu()

    def call(self):
        kw = dict(q_scale=self.q_scale, k_scale=self.ks, v_scale=self.vs)
        if self.head_scales:
            dev = self.device
            kw = dict(q_scales=self.qs_h.to(dev) if self.qt in FP8 else None, k_scales=self.ks_h.to(dev),
                      v_scales=self.vs_h.to(dev))
        self.plan.run_tree(self.dq, self.kc, self.vc, self.ids, self.mask, self.o, self.lse, self.ws, **kw)

    def check(self, o, lse):
        g = self.hq // self.hkv
        sm = 1 / math.sqrt(self.d)
        pieces = 1 if self.qt in FP8 or self.kt not in FP8 else 2 if self.qt == "bf16" else 3
        # P's rounding: f16's (2^-11), which three e4m3 pieces hold exactly and of which
        # two leave 2^-8 (hi leaves up to 2^-4 of its binade, whose e5m2 below that
        # value has steps of 2^-7), or the cache's type.
        p_half = HALF[DT[self.kt]] if self.kt not in FP8 else 2.0 ** -11 if self.ot == "f16" else 2.0 ** -8 + 2.0 ** -11
        for b, (L, T) in enumerate(zip(self.kv_lens, self.qo_lens)):
            if T == 0:
                continue
            vis = torch.ones(T, L, dtype=torch.bool)
            vis[:, L - T:] = torch.from_numpy(self.seen[b])
            r0 = int(self.qo_indptr[b])
            for hk in range(self.hkv):
                ks = float(self.ks_h[hk]) if self.head_scales else self.ks
                vs = float(self.vs_h[hk]) if self.head_scales else self.vs
                k, v = self.k[b][:, hk].double() * ks, self.v[b][:, hk].double() * vs
                for h in range(hk * g, hk * g + g):
                    qs = (float(self.qs_h[h]) if self.qt in FP8 else 1.0) if self.head_scales else self.q_scale
                    q = self.q[r0:r0 + T, h].double() * qs
                    z = (q @ k.t()) * sm
                    z = z.masked_fill(~vis, -math.inf)
                    m = z.amax(1, keepdim=True)
                    e = (z - torch.where(torch.isinf(m), 0.0, m)).exp()
                    tot = e.sum(1, keepdim=True)
                    w = torch.where(tot > 0, e / tot, 0.0)
                    ro = w @ v
                    rl = (tot.log() + m).squeeze(1)
                    # Logit error: query pieces (2^-18 of the row's largest), fp32
                    # accumulation of d products a piece.
                    dz = (q.abs() @ k.abs().t()) * sm * self.d * pieces * 2.0 ** -23
                    if pieces > 1:
                        dz = dz + q.abs().amax(1, keepdim=True) * k.abs().sum(1)[None] * sm * 2.0 ** -18
                    dz = torch.where(vis, dz, 0.0).amax(1, keepdim=True)
                    # exp2, the sums and the fold of the scale: 2^-20 together
                    rel = p_half + 2 * dz + 2.0 ** -20
                    # Small probabilities, the row's maximum being at 2^5: half the last
                    # piece's smallest step, e4m3's 2^-10 / 32 (2^-20 of it; e5m2's 2^-17
                    # and an f16's are smaller).  With two pieces hi is a multiple of
                    # 2^-9 below 2^-6 and leaves less than 2^-10, whose e5m2 steps are
                    # 2^-13: 2^-14 off, 2^-19 of it.
                    tail = L * 2.0 ** (-19 if p_half > 2.0 ** -8 else -20) * v.abs().max() / tot.clamp(min=1.0)
                    if self.kt == "bf16":
                        tail = 0.0
                    slack = (w @ v.abs()) * rel + tail
                    tol = slack + HALF[DT[self.ot]] * (ro.abs() + slack) + 2.0 ** -24
                    got = o[r0:r0 + T, h].double()
                    bad = (got - ro).abs() - tol
                    assert float(bad.max()) <= 0, (f"request {b} head {h}: o off by {float((got - ro).abs().max())}, "
                                                   f"{float(bad.max())} too much at {divmod(int(bad.argmax()), self.d)}")
                    gl = lse[r0:r0 + T, h].double()
                    assert torch.equal(torch.isinf(gl), torch.isinf(rl)), f"request {b} head {h}: lse finiteness"
                    fin = torch.isfinite(rl)
                    off = ((gl - rl).abs() - (dz.squeeze(1) + 2.0 ** -18 + rl.abs() * 2.0 ** -22))[fin]
                    assert off.numel() == 0 or float(off.max()) <= 0, f"request {b} head {h}: lse off {float(off.max())} too much"
