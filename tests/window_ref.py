"""Attention with a sliding window, sinks and block scales in 64 bits, with
bounds on what the kernels may differ by (tests only)."""
import math

import numpy as np
import torch

import paged_attention_fp8_gb300 as pa
from blocks_ref import BLOCK, TOP, TORCH, in_layout, raw, table

OUT = {"bf16": "bf16", "f16": "f16", "e4m3fn": "bf16", "e5m2": "bf16"}


class Batch:
    """A paged batch with values of every kind the kernels take.

    scales: "tensor", "head" or "block"; new None means decode."""

    def __init__(self, lens, new=None, *, hq=8, hkv=2, d=128, q="bf16", kv="e4m3fn", layout="NHD", page_size=16, window=0,
                 sinks=0, scales="tensor", seed=0, spread=3, **plan):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.new, self.hq, self.hkv, self.d = lens, new, hq, hkv, d
        self.q_type, self.kv_type, self.layout, self.ps = q, kv, layout, page_size
        self.window, self.sinks, self.scales = window, sinks, scales
        self.ptr, self.ids, self.pool = table(lens, page_size, g)
        self.rows = np.arange(len(lens) + 1) if new is None else np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        n, per = int(self.rows[-1]), page_size // BLOCK
        fp8 = kv in TOP

        def cache():
            x = torch.randn(self.pool, page_size, hkv, d, generator=g)
            return (x * (TOP[kv] / 6)).clamp(-TOP[kv], TOP[kv]).to(TORCH[kv]) if fp8 else x.to(TORCH[kv])

        self.k, self.v = cache(), cache()  # token-major codes
        unit = 6 / TOP[kv] if fp8 else 1.0

        def some(*shape):
            # Scales of unlike size: any numbers, not powers of two alone.
            return unit * 2.0 ** ((torch.rand(shape, generator=g) - 0.5) * spread)

        self.q_scale = 6 / TOP[q] if q in TOP else 1.0
        self.qs = None
        if scales == "tensor":
            self.ks = self.vs = None
            self.k_scale, self.v_scale = (float(some(1)) if fp8 else 1.0 for _ in range(2))
        else:
            shape = (hkv,) if scales == "head" else (self.pool, per, hkv)
            self.ks, self.vs = some(*shape), some(*shape)
            if scales == "head" and q in TOP:
                self.qs = self.q_scale * 2.0 ** (torch.rand(hq, generator=g) - 0.5)
        x = torch.randn(n, hq, d, generator=g)
        self.q = (x / self.q_scale).clamp(-TOP[q], TOP[q]).to(TORCH[q]) if q in TOP else x.to(TORCH[q])
        self.sm_scale = 1 / math.sqrt(d)
        self.o_type = OUT[q]
        self.plan = pa.Plan(mode="decode" if new is None else "prefill", num_qo_heads=hq, num_kv_heads=hkv, num_pages=self.pool,
                            kv_indptr=self.ptr, last_page_len=[x - (-(-x // page_size) - 1) * page_size if x else 0 for x in lens],
                            qo_indptr=None if new is None else self.rows, q_dtype=q, kv_dtype=kv, head_dim=d,
                            page_size=page_size, kv_layout=layout, window=window, sinks=sinks, **plan)

    # ---- the kernels' side
    def upload(self):
        n = int(self.rows[-1])
        self.k_d, self.v_d = (in_layout(x, self.layout).cuda() for x in (self.k, self.v))
        self.q_d, self.ids_d = self.q.cuda(), torch.as_tensor(self.ids, dtype=torch.int32).cuda()
        self.o = torch.full((n, self.hq, self.d), 7.0, dtype=TORCH[self.o_type], device="cuda")
        self.lse = torch.full((n, self.hq), 7.0, device="cuda")
        self.ws = torch.empty(self.plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        self.plan.upload(self.ws)
        if self.ks is not None:
            self.ks_d, self.vs_d = self.ks.cuda(), self.vs.cuda()
        return self

    def args(self):
        return self.q_d, self.k_d, self.v_d, self.ids_d, self.o, self.lse, self.ws

    def run(self, **kw):
        if self.scales == "block":
            self.plan.run_block_scales(*self.args(), q_scale=self.q_scale, k_scales=self.ks_d, v_scales=self.vs_d, **kw)
        elif self.scales == "head":
            self.plan.run_head_scales(*self.args(), q_scales=None if self.qs is None else self.qs.cuda(), k_scales=self.ks_d,
                                      v_scales=self.vs_d, **kw)
        else:
            self.plan.run(*self.args(), q_scale=self.q_scale, k_scale=self.k_scale, v_scale=self.v_scale, **kw)

    # ---- the reference
    def dense(self, name, b):
        """Request b's keys or values [len, hkv, d] in 64 bits."""
        n = self.lens[b]
        pos = np.arange(n)
        page = torch.as_tensor(self.ids[self.ptr[b] + pos // self.ps])
        slot = torch.as_tensor(pos % self.ps)
        cache, s = (self.k, self.ks) if name == "k" else (self.v, self.vs)
        x = raw(cache)[page, slot].view(cache.dtype).double()
        if self.scales == "tensor":
            return x * (self.k_scale if name == "k" else self.v_scale)
        by = s.double()[None, :, None] if self.scales == "head" else s.double()[page, slot // BLOCK][:, :, None]
        return x * by

    def visible(self, b):
        """[rows, keys] truth values of request b."""
        n = self.lens[b]
        m = int(self.rows[b + 1] - self.rows[b]) if self.new is not None else 1
        t = torch.arange(n - m, n)[:, None] if n else torch.zeros(m, 1)
        j = torch.arange(n)[None]
        seen = j <= t
        return seen & ((j > t - self.window) | (j < self.sinks)) if self.window else seen

    def expect(self):
        """(o, lse, bound on o, bound on lse).  Bounds, with A = sum of weight x |v|: the output's rounding, half a step
        (eps / 2 of its value); each probability's rounding, half a step of f16 (2^-11; bf16 probabilities over a bf16 cache:
        2^-8) and, below f16's normal range, 2^-25 of the largest; sums of n terms in fp32, n 2^-23 of A at most; a weight's
        relative error, the error of its logit: d + 2 roundings of sum |q k| (2^-23 each), of the exponent's argument and
        of exp2 itself (2^-22 each, on |logit| log2 e)."""
        n = int(self.rows[-1])
        o, lse = torch.zeros(n, self.hq, self.d, dtype=torch.float64), torch.full((n, self.hq), -math.inf, dtype=torch.float64)
        tol_o, tol_l = torch.zeros_like(o), torch.zeros_like(lse)
        half = torch.finfo(TORCH[self.o_type]).eps / 2
        p_half = 2.0 ** -8 if self.kv_type == "bf16" else 2.0 ** -11
        group = self.hq // self.hkv
        qs = self.q_scale if self.qs is None else self.qs.double()[None, :, None]
        for b, length in enumerate(self.lens):
            r0, r1 = int(self.rows[b]), int(self.rows[b + 1])
            if not length or r0 == r1:
                continue
            k, v = self.dense("k", b), self.dense("v", b)
            seen = self.visible(b)
            nan = torch.isnan(v).any(-1).any(-1) | torch.isnan(k).any(-1).any(-1)
            assert not (nan[None] & seen).any()
            k, v = torch.nan_to_num(k), torch.nan_to_num(v)
            q = (self.q[r0:r1].double() * qs).view(r1 - r0, self.hkv, group, self.d)
            z = torch.einsum("uhgd,jhd->uhgj", q, k) * self.sm_scale
            mag = torch.einsum("uhgd,jhd->uhgj", q.abs(), k.abs()) * self.sm_scale
            hid = ~seen[:, None, None]
            z = z.masked_fill(hid, -math.inf)
            w = torch.softmax(z, -1)
            l2 = torch.logsumexp(z, -1)
            mag = mag.masked_fill(hid, 0).amax(-1)
            big = z.abs().masked_fill(hid, 0).amax(-1)
            delta = (self.d + 2) * 2.0 ** -23 * mag + 2.0 ** -21 * (1.5 * big + 32)
            out = torch.einsum("uhgj,jhd->uhgd", w, v)
            A = torch.einsum("uhgj,jhd->uhgd", w, v.abs())
            cnt = seen.sum(-1)[:, None, None]
            top = v.abs().amax()
            if self.scales == "block":  # a probability is rounded after its V scale has joined it: its code alone follows
                top = float(self.vs[torch.isfinite(self.vs)].max()) * TOP[self.kv_type]
            tol = A * (p_half + 2 * delta[..., None] + cnt[..., None] * 2.0 ** -23) + cnt[..., None] * 2.0 ** -25 * top
            o[r0:r1], lse[r0:r1] = out.reshape(r1 - r0, self.hq, self.d), l2.reshape(r1 - r0, self.hq)
            tol_o[r0:r1] = tol.reshape(r1 - r0, self.hq, self.d) * (1 + half) + half * o[r0:r1].abs() + 2.0 ** -25
            tol_l[r0:r1] = (delta + cnt * 2.0 ** -23 + 2.0 ** -20).reshape(r1 - r0, self.hq)
        return o, lse, tol_o, tol_l

    def check(self, o=None, lse=None):
        o, lse = (self.o if o is None else o).double().cpu(), (self.lse if lse is None else lse).double().cpu()
        ro, rl, to, tl = self.expect()
        assert torch.isfinite(o).all()
        over = (o - ro).abs() - to
        assert over.max() <= 0, f"o off by {float((o - ro).abs().max())}, {float(over.max())} over its bound"
        assert torch.equal(torch.isinf(lse), torch.isinf(rl))
        fin = torch.isfinite(rl)
        if fin.any():
            over = (lse - rl).abs()[fin] - tl[fin]
            assert over.max() <= 0, f"lse {float(over.max())} over its bound"


def run(*a, **kw):
    b = Batch(*a, **kw).upload()
    b.run()
    b.plan.device_status(b.ws)
    b.check()
    return b
