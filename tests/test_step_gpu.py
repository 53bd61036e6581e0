"""A verification step of speculative decoding, as a server runs it: tables,
then norm + rotation + append, then tree attention over the cache."""
import numpy as np
import pytest
import torch

import paged_attention_fp8_gb300 as pa
from step_ref import assert_rounded, norm_rope
from step_ref import tables as ref_tables
from tree_common import TreeBatch

pytestmark = pytest.mark.gpu
E4, BF, HF = torch.float8_e4m3fn, torch.bfloat16, torch.float16


class Step:
    def __init__(self, cached, new, *, hq, hkv, d, src, kv, layout, page_size, chain=False, pad_tokens=3):
        self.cached, self.new, self.hq, self.hkv, self.d = cached, new, hq, hkv, d
        self.src, self.kv, self.layout, self.ps, self.chain = src, kv, layout, page_size, chain
        total = [-(-(c + n) // page_size) for c, n in zip(cached, new)]
        self.have = [-(-c // page_size) for c in cached]
        self.n, self.pages, self.width = sum(new), sum(total), max(total) + 1
        self.tokens, self.pool = self.n + pad_tokens, sum(total) + 9
        self.words = max(1, -(-max(new) // 32))
        i = dict(dtype=torch.int32, device="cuda")
        self.cl, self.nl = torch.tensor(cached, **i), torch.tensor(new, **i)
        self.table, self.free, self.used = torch.zeros(len(cached), self.width, **i), torch.zeros(self.pool, **i), torch.ones(1, **i)
        self.parents = None if chain else torch.zeros(self.tokens, **i)
        self.qkv = torch.zeros(self.tokens, hq + 2 * hkv, d, dtype=src, device="cuda")
        g = torch.Generator().manual_seed(5)
        self.qw, self.kw = ((1 + 0.2 * torch.randn(d, generator=g)).to(src).cuda() for _ in range(2))
        ang = torch.rand(2048, d // 2, generator=g, dtype=torch.float64) * 6.3
        self.cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
        shape = (self.pool, page_size, hkv, d) if layout == "NHD" else (self.pool, hkv, page_size, d)
        self.kc, self.vc = (torch.zeros(shape, dtype=src, device="cuda").to(kv) for _ in range(2))
        self.ks, self.vs = (0.01, 0.012) if kv is E4 else (1.0, 1.0)
        self.t = pa.StepTables(batch=len(cached), max_pages=self.pages + 2, max_tokens=self.tokens, page_size=page_size,
                               num_pages=self.pool, mask_words=self.words)
        self.q_out = torch.full((self.tokens, hq, d), 7.0, dtype=src, device="cuda")
        self.o, self.lse = torch.full_like(self.q_out, 7.0), torch.full((self.tokens, hq), 7.0, device="cuda")
        np_ = [int(x) for x in total]
        names = {BF: "bf16", HF: "f16", E4: "e4m3fn"}
        self.names = names[src], names[kv]
        self.plan = pa.Plan(
            mode="tree", num_qo_heads=hq, num_kv_heads=hkv, num_pages=self.pool, q_dtype=self.names[0], kv_dtype=self.names[1],
            kv_indptr=np.concatenate([[0], np.cumsum(np_)]).astype(np.int32),
            last_page_len=np.array([c + n - (p - 1) * page_size if p else 0 for c, n, p in zip(cached, new, np_)], np.int32),
            qo_indptr=np.concatenate([[0], np.cumsum(new)]).astype(np.int32), head_dim=d, page_size=page_size, kv_layout=layout)
        self.ws = torch.empty(self.plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        self.plan.upload(self.ws)

    def fill(self, seed):
        """New tokens, pages, drafts and cached keys and values, in place."""
        g, r = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
        ids = r.permutation(self.pool)
        at, table = 0, np.full((len(self.cached), self.width), -1)
        for b, h in enumerate(self.have):
            table[b, :h] = ids[at:at + h]
            at += h
        free = np.zeros(self.pool, np.int64)
        free[1:1 + self.pool - at] = ids[at:]
        self.free_h = free[:1 + self.pool - at]
        par = np.full(self.tokens, -1)
        t0 = 0
        for n in self.new:
            for u in range(1, n):
                par[t0 + u] = r.integers(-1, u)
            t0 += n
        self.table_h, self.par_h = table, None if self.chain else par
        self.table.copy_(torch.from_numpy(table))
        self.free.copy_(torch.from_numpy(free))
        if not self.chain:
            self.parents.copy_(torch.from_numpy(par))
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=g).to(self.src))
        for c in (self.kc, self.vc):
            x = torch.randn(c.shape, generator=g) / (0.01 if self.kv is E4 else 1.0)
            c.copy_(x.clamp(-448, 448).to(self.src).to(self.kv))  # past 464 an e4m3 cast gives NaN

    def run(self):
        t, hq, hkv = self.t, self.hq, self.hkv
        t.build(self.cl, self.nl, self.table, self.free[:len(self.free_h)], self.used, parents=self.parents)
        pa.pafp8_norm_rope_append(self.qkv[:, :hq], self.qkv[:, hq:hq + hkv], self.qkv[:, hq + hkv:], self.qw, self.kw,
                                  self.cs, t.rope_positions, t.slots, self.q_out, self.kc, self.vc, k_scale=self.ks,
                                  v_scale=self.vs, kv_layout=self.layout, status=t.status)
        self.plan.run_tree(self.q_out, self.kc, self.vc, t.kv_indices, t.tree_mask, self.o, self.lse, self.ws,
                           k_scale=self.ks, v_scale=self.vs)

    def cached_rows(self, cache, slots):
        raw = cache.cpu().view(torch.uint8 if self.kv is E4 else torch.int16)
        if self.layout == "HND":
            raw = raw.transpose(1, 2)
        return raw.reshape(-1, self.hkv, self.d)[torch.as_tensor(slots, dtype=torch.int64)].contiguous().view(self.kv)

    def check(self):
        torch.cuda.synchronize()
        self.plan.device_status(self.ws)
        assert int(self.t.status) == 0
        n, hq, hkv = self.n, self.hq, self.hkv
        ref, bad = ref_tables(self.cached, self.new, self.table_h, self.free_h, 1, page_size=self.ps, num_pages=self.pool,
                              max_pages=self.pages + 2, max_tokens=self.tokens, parents=self.par_h, words=self.words)
        assert not bad
        for name in ("kv_indptr", "qo_indptr", "last_page_len", "slots", "rope_positions", "free_used"):
            assert np.array_equal(getattr(self.t, name).cpu().numpy(), np.array(ref[name])), name
        assert np.array_equal(self.t.kv_indices.cpu().numpy()[:self.pages], ref["kv_indices"][:self.pages])
        assert np.array_equal(self.t.tree_mask.cpu().numpy().view(np.uint32), ref["tree_mask"])
        x, pos = self.qkv[:n].cpu(), torch.from_numpy(ref["rope_positions"][:n])[None]
        axis = torch.zeros(self.d // 2, dtype=torch.uint8)
        args = (1e-6, self.cs.cpu(), pos, axis, False)
        q, qm = norm_rope(x[:, :hq], self.qw.cpu(), *args)
        k, km = norm_rope(x[:, hq:hq + hkv], self.kw.cpu(), *args)
        v = x[:, hq + hkv:].double()
        got_q = self.q_out.cpu()
        assert_rounded(got_q[:n], q, qm, 1.0, "q")
        assert_rounded(self.cached_rows(self.kc, ref["slots"][:n]), k, km, self.ks, "k")
        assert_rounded(self.cached_rows(self.vc, ref["slots"][:n]), v, v.abs(), self.vs, "v")
        # the attention, over what the cache holds now
        b = TreeBatch.__new__(TreeBatch)
        b.kv_lens, b.qo_lens = [c + m for c, m in zip(self.cached, self.new)], self.new
        b.hq, b.hkv, b.d, (b.qt, b.kt), b.ot = hq, hkv, self.d, self.names, self.names[0]
        b.ks, b.vs, b.q_scale, b.head_scales, b.q, b.k, b.v, b.seen = self.ks, self.vs, 1.0, False, got_q[:n], [], [], []
        b.qo_indptr = np.array(ref["qo_indptr"])
        for i, length in enumerate(b.kv_lens):
            p0 = ref["kv_indptr"][i]
            j = np.arange(length)
            slots = ref["kv_indices"][p0 + j // self.ps] * self.ps + j % self.ps if length else j
            b.k.append(self.cached_rows(self.kc, slots))
            b.v.append(self.cached_rows(self.vc, slots))
            rows = ref["tree_mask"][b.qo_indptr[i]:b.qo_indptr[i + 1]]
            w = np.arange(self.new[i])
            b.seen.append((rows[:, w // 32] >> (w % 32).astype(np.uint32) & 1).astype(bool))
        b.check(self.o[:n].cpu(), self.lse[:n].cpu())
        for t in (self.o, self.lse):
            assert bool((t[n:] == 7).all()), "rows behind the last request were written"
        assert bool((self.q_out[n:] == 7).all())


STEPS = [
    dict(cached=[37, 0, 500, 128, 15], new=[5, 3, 16, 1, 33], hq=8, hkv=2, d=128, src=BF, kv=E4, layout="NHD", page_size=16),
    dict(cached=[260, 63, 0], new=[7, 2, 1], hq=12, hkv=3, d=64, src=HF, kv=E4, layout="HND", page_size=32),
    dict(cached=[90, 1000], new=[4, 9], hq=4, hkv=4, d=128, src=BF, kv=BF, layout="NHD", page_size=16, chain=True),
    dict(cached=[31], new=[1], hq=6, hkv=1, d=64, src=HF, kv=HF, layout="HND", page_size=16, pad_tokens=0)]


@pytest.mark.parametrize("kw", STEPS)
def test_a_step(cuda_device, kw):
    s = Step(**kw)
    s.fill(1)
    s.run()
    s.check()


@pytest.mark.parametrize("kw", STEPS[:2])
def test_a_captured_step_takes_the_next_inputs(cuda_device, kw):
    s = Step(**kw)
    s.fill(1)
    s.run()
    torch.cuda.synchronize()
    s.fill(2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for seed in (2, 3):
        s.fill(seed)
        s.o[:s.n].zero_()
        graph.replay()
        s.check()


def test_two_steps_on_two_streams(cuda_device):
    steps, streams = [Step(**kw) for kw in STEPS[:2]], [torch.cuda.Stream() for _ in range(2)]
    for i, s in enumerate(steps):
        s.fill(10 + i)
    torch.cuda.synchronize()
    for _ in range(3):  # every launch of one may overlap those of the other
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s.table.copy_(torch.from_numpy(s.table_h))
                s.run()
    torch.cuda.synchronize()
    for s in steps:
        s.check()
