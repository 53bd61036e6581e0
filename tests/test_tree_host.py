"""The tree plan's partition and refusals (no GPU needed)."""
import ctypes

import numpy as np
import pytest

import paged_attention_fp8_gb300 as pa

SEG, MERGE = 12, 8


def _plan(kv_lens, qo_lens, hq=8, hkv=2, page_size=16, num_ctas=152, **kw):
    pages = [-(-n // page_size) for n in kv_lens]
    indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    last = np.array([n - (p - 1) * page_size if p else 0 for n, p in zip(kv_lens, pages)], np.int32)
    qo = np.concatenate([[0], np.cumsum(qo_lens)]).astype(np.int32)
    kw = {**dict(q_dtype="bf16", kv_dtype="e4m3fn"), **kw}
    return pa.Plan(mode="tree", num_qo_heads=hq, num_kv_heads=hkv, num_pages=max(1, sum(pages)), kv_indptr=indptr,
                   last_page_len=last, qo_indptr=qo, page_size=page_size, num_ctas=num_ctas, **kw)


def _parts(plan):
    m = plan.metadata()
    off_cta, off_seg, off_merge = int(m[12]), int(m[13]), int(m[19])
    ctas, nseg, nmerge, npart = int(m[6]), int(m[7]), int(m[9]), int(m[8])
    ptr = m[off_cta:off_cta + ctas + 1]
    segs = m[off_seg:off_seg + SEG * nseg].reshape(nseg, SEG)
    merges = m[off_merge:off_merge + MERGE * nmerge].reshape(nmerge, MERGE)
    assert off_seg % 4 == 0 and off_merge % 4 == 0
    assert nseg == 0 or (int(ptr[0]) == 0 and int(ptr[-1]) == nseg and (np.diff(ptr) >= 0).all())
    return ctas, ptr, segs, merges, npart


@pytest.mark.parametrize("seed", range(40))
def test_every_tile_of_every_line_is_in_one_segment(seed):
    r = np.random.default_rng(seed)
    hkv = int(r.choice([1, 2, 3, 4, 6, 8, 12, 16, 40]))
    group = int(r.choice([1, 2, 4, 5, 8, 16, 100]))
    batch = int(r.integers(0, 30))
    kv = [int(x) for x in r.integers(1, int(r.choice([20, 500, 6000])), batch)]
    qo = [int(r.integers(0, min(n, 70) + 1)) for n in kv]
    num_ctas = int(r.choice([1, 3, 20, 152]))
    plan = _plan(kv, qo, hq=hkv * group, hkv=hkv, num_ctas=num_ctas)
    ctas, ptr, segs, merges, npart = _parts(plan)
    assert ctas <= num_ctas
    R = 32 if max(qo + [0]) * group <= 32 else 64
    want = {(b, hk, r0) for b in range(batch) for hk in range(hkv) for r0 in range(0, qo[b] * group, R)}
    qo0 = np.concatenate([[0], np.cumsum(qo)])
    page0 = np.concatenate([[0], np.cumsum([-(-n // 16) for n in kv])])
    got, slots = {}, {}
    first = {(int(qo0[b]), qo[b], kv[b], int(page0[b])): b for b in range(batch) if qo[b]}
    for s in segs:
        hk, r0, a, e, slot = (int(x) for x in s[:5])
        b = first[tuple(int(x) for x in s[5:9])]
        assert a < e
        got.setdefault((b, hk, r0), []).append((a, e, slot))
        if slot >= 0:
            assert slot not in slots
            slots[slot] = (b, hk, r0, a)
    assert set(got) == want
    split = {}
    for key, parts in got.items():
        parts.sort()
        nt = -(-kv[key[0]] // 128)
        assert [p[0] for p in parts] == [0] + [p[1] for p in parts[:-1]] and parts[-1][1] == nt
        if len(parts) == 1:
            assert parts[0][2] == -1
        else:
            assert [p[2] for p in parts] == list(range(parts[0][2], parts[0][2] + len(parts)))
            split[(int(qo0[key[0]]), key[2], key[1])] = (parts[0][2], parts[-1][2] + 1, min(R, qo[key[0]] * group - key[2]))
    assert len(slots) == npart and set(slots) == set(range(npart))
    assert {(int(x[2]), int(x[5]), int(x[3])): (int(x[0]), int(x[1]), int(x[4])) for x in merges} == split
    if npart:
        rows = max(min(R, n * group) for n in qo)
        assert plan.workspace_bytes >= npart * rows * (128 + 1) * 4


def test_equal_requests_are_balanced():
    plan = _plan([4096] * 64, [16] * 64, hq=32, hkv=8)
    ctas, ptr, segs, _, _ = _parts(plan)
    # tiles, and five for each segment's start
    cost = [int((segs[ptr[i]:ptr[i + 1], 3] - segs[ptr[i]:ptr[i + 1], 2] + 5).sum()) for i in range(ctas)]
    assert ctas == 152 and max(cost) <= 1.02 * sum(cost) / ctas
    # the heads of one range are neighbours
    assert [int(segs[ptr[i], 0]) for i in range(8)] == list(range(8))


@pytest.mark.parametrize("kw,status,words", [
    (dict(kv_dtype="f16"), 1, "tree attention takes a 2-byte cache only"), (dict(kv_dtype="int8"), 1, "int8"),
    (dict(q_dtype="e4m3fn", kv_dtype="bf16"), 1, "fp8 query"), (dict(hq=258, hkv=2), 8, "tree attention serves up to 128"),
    (dict(head_dim=96), 8, "head_dim 96"), (dict(o_dtype="e4m3fn"), 1, "o_data_type")])
def test_plan_refusals(kw, status, words):
    with pytest.raises(pa.Pafp8Error) as e:
        _plan([40], [4], **kw)
    assert e.value.status == status and words in str(e.value)
    with pytest.raises(pa.Pafp8Error, match="qo_len 5 > kv_len 4"):
        _plan([4], [5])
    with pytest.raises(pa.Pafp8Error, match="tree attention needs the qo_indptr"):
        pa.Plan(mode="tree", num_qo_heads=8, num_kv_heads=2, num_pages=4, kv_indptr=[0, 1], last_page_len=[3],
                q_dtype="bf16", kv_dtype="e4m3fn", num_ctas=4)


A = 0x10000


def _run(plan, **kw):
    a = dict(plan=plan.handle, q_dtype=pa.BF16, q=A, k_dtype=pa.E4M3FN, k=A, v_dtype=pa.E4M3FN, v=A, idx=A, mask=A, words=1,
             q_scale=1.0, k_scale=1.0, v_scale=1.0, q_scales=None, k_scales=None, v_scales=None, o_dtype=pa.BF16, o=A, lse=A,
             ws=A, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return pa.lib().pafp8_run_tree(*a.values())


@pytest.mark.parametrize("kw,status,words", [
    (dict(q_dtype=pa.F16), 1, "plan was made for"), (dict(k_dtype=pa.E5M2), 1, "v_cache has"),
    (dict(o_dtype=pa.F16), 1, "o_data_type"), (dict(q_scale=2.0), 3, "q_scale"), (dict(k_scale=-1.0), 3, "scales"),
    (dict(k_scales=A, v_scales=A, k_scale=2.0), 3, "replace"), (dict(v_scales=A), 3, "both"), (dict(k_scales=A), 3, "both"),
    (dict(), 4, "uploaded")])
def test_run_refusals(kw, status, words):
    plan = _plan([40], [4])
    assert _run(plan, **kw) == status
    assert words in pa.pafp8_last_error()


def test_tree_and_other_plans_do_not_mix():
    tree = _plan([40], [4])
    other = pa.Plan(mode="prefill", num_qo_heads=8, num_kv_heads=2, num_pages=3, kv_indptr=[0, 3], last_page_len=[8],
                    qo_indptr=[0, 4], q_dtype="bf16", kv_dtype="e4m3fn", num_ctas=4)
    assert _run(other) == 3 and "tree plans only" in pa.pafp8_last_error()
    L = pa.lib()
    common = (pa.BF16, A, pa.E4M3FN, A, pa.E4M3FN, A, A, 1.0, 1.0, 1.0, pa.BF16, A, A)
    assert L.pafp8_run(tree.handle, *common, A, 1 << 30, None) == 3 and "pafp8_run_tree" in pa.pafp8_last_error()
    assert L.pafp8_run_decode_noalloc(tree.handle, *common, None) == 3
    ph = pa.pod_phase(tree.handle, A, A, A, A, A, 1 << 20)
    assert L.pafp8_run_pod(ctypes.byref(ph), ctypes.byref(ph), pa.BF16, pa.E4M3FN, A, pa.E4M3FN, A, 1.0, 1.0, 1.0, pa.BF16,
                           None) == 3
    assert "is a tree plan" in pa.pafp8_last_error()


def test_pieces_of_the_probabilities():
    """Every f16 in (0, 256], the largest at 2^5 or above: what its fp8 pieces leave."""
    import torch

    def e4m3(x):
        return x.to(torch.float8_e4m3fn).float()

    half = torch.arange(1, 0x5C01, dtype=torch.int32).to(torch.int16).view(torch.float16)
    x = half.float()
    hi = e4m3(x)
    left = (x - hi).half()
    assert torch.equal(left.float(), x - hi)
    bits = (left.view(torch.int16).int() + 0x80) & 0xFF00
    lo = torch.where(bits > 0x7FFF, bits - 0x10000, bits).to(torch.int16).view(torch.float16).float()
    two = (x - hi - lo).abs()
    assert (two <= torch.where(x >= 2.0 ** -6, x * 2.0 ** -8, torch.tensor(2.0 ** -14))).all()
    scaled = 32 * (x - hi)
    l1 = e4m3(scaled)
    three = (x - hi - (l1 + e4m3(scaled - l1)) / 32).abs()
    assert (three <= torch.where(x >= 2.0 ** -4, 0.0, 2.0 ** -15)).all()
