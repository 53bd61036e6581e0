"""Refusals of the step operators (no GPU needed: every check is on the host,
before any launch)."""
import ctypes

import pytest
import torch

import paged_attention_fp8_gb300 as pa

A = 0x10000  # an aligned address that no refused call reads


def tables(**kw):
    a = dict(batch=2, page_size=16, num_pages=8, cached_lens=A, new_lens=A, block_table=A, block_stride=4, block_width=4,
             free_pages=A, num_free=3, free_used=A, free_used_out=A + 64, max_pages=8, max_tokens=8, kv_indptr=A,
             last_page_len=A, kv_indices=A, qo_indptr=A, batch_indices=A, positions=A, slots=A, parents=None,
             rope_positions=A, tree_mask=A, mask_words=1, status=None, stream=None)
    a.update(kw)
    stream = a.pop("stream")
    return pa.lib().pafp8_build_tables(ctypes.byref(pa.tables_desc(**a)), stream)


@pytest.mark.parametrize("kw,status,words", [
    (dict(batch=-1), 2, "negative"), (dict(num_free=-1), 2, "negative"), (dict(max_tokens=-1), 2, "negative"),
    (dict(page_size=24), 8, "page_size 24"), (dict(page_size=0), 8, "page_size 0"), (dict(block_stride=3), 2, "block_stride 3"),
    (dict(max_pages=1 << 31), 2, "2^31"), (dict(mask_words=0), 2, "mask_words 0"), (dict(free_used=None), 3, "free_used"),
    (dict(free_used_out=A), 3, "must not be free_used"), (dict(cached_lens=None), 3, "cached_lens"),
    (dict(block_table=None), 3, "block_table"), (dict(free_pages=None), 3, "free_pages"), (dict(kv_indices=None), 3, "kv_indices"),
    (dict(slots=None), 3, "slots"), (dict(slots=A + 4), 3, "aligned"), (dict(parents=A + 2), 3, "aligned"),
    (dict(kv_indptr=None), 3, "kv_indptr")])
def test_tables_refusals(kw, status, words):
    assert tables(**kw) == status
    assert words in pa.pafp8_last_error()


def rope(**kw):
    a = dict(src_dtype=pa.BF16, nnz=4, num_qo_heads=8, num_kv_heads=2, head_dim=128, q=A, q_stride=1024, k=A, k_stride=256, v=A, v_stride=256,
             q_weight=None, k_weight=None, eps=1e-6, cos_sin=A, max_position=64, rot_dim=128, interleaved=0, positions=A,
             num_axes=1, pos_stride=4, pair_axis=None, slots=A, q_out_dtype=pa.BF16, q_out=A + 4096, q_scale=1.0,
             kv_dtype=pa.E4M3FN, kv_layout=0, k_cache=A, v_cache=A, num_pages=8, page_size=16, k_scale=0.5, v_scale=0.5,
             status=None, stream=None)
    a.update(kw)
    stream = a.pop("stream")
    return pa.lib().pafp8_norm_rope_append(ctypes.byref(pa.rope_desc(**a)), stream)


@pytest.mark.parametrize("kw,status,words", [
    (dict(src_dtype=pa.F32), 1, "float32"), (dict(src_dtype=pa.E4M3FN), 1, "float8_e4m3fn"),
    (dict(q_out_dtype=pa.F16), 1, "q_out"), (dict(kv_dtype=pa.F16), 1, "cache of dtype float16"),
    (dict(kv_dtype=pa.INT8), 1, "int8"), (dict(kv_layout=2), 3, "kv_layout"), (dict(nnz=-1), 2, "nnz -1"),
    (dict(num_qo_heads=0), 2, "head counts"), (dict(head_dim=96), 8, "head_dim 96"), (dict(rot_dim=24), 8, "rot_dim 24"),
    (dict(rot_dim=144), 8, "rot_dim 144"), (dict(rot_dim=0), 8, "rot_dim 0"), (dict(page_size=8), 8, "page_size 8"),
    (dict(num_axes=4), 2, "num_axes 4"), (dict(num_axes=0), 2, "num_axes 0"), (dict(max_position=0), 2, "max_position"),
    (dict(eps=-1.0), 3, "eps"), (dict(eps=float("nan")), 3, "eps"), (dict(k_scale=0.0), 3, "scales"),
    (dict(v_scale=float("inf")), 3, "scales"), (dict(q_scale=2.0), 3, "q_scale 2"),
    (dict(kv_dtype=pa.BF16), 3, "as they are"), (dict(q=None), 3, "non-NULL"), (dict(slots=None), 3, "non-NULL"),
    (dict(q_stride=1016), 2, "strides"), (dict(v_stride=128), 2, "strides"), (dict(num_axes=2, pos_stride=3), 2, "pos_stride"),
    (dict(q=A + 8), 3, "16-byte"), (dict(cos_sin=A + 4), 3, "16-byte"), (dict(q_stride=1028), 3, "multiples of 8"),
    (dict(slots=A + 4), 3, "aligned"), (dict(q_out=A, q_out_dtype=pa.E4M3FN), 3, "q_out may be q"),
    (dict(q_out=A, q_stride=2048), 3, "q_out may be q")])
def test_norm_rope_refusals(kw, status, words):
    assert rope(**kw) == status
    assert words in pa.pafp8_last_error()


def test_no_tokens_is_ok():
    assert rope(nnz=0, q=None, slots=None) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    z = torch.zeros
    i = z(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="cached_lens is on cpu"):
        pa.pafp8_build_tables(i, i, i.view(1, 2), i, i, i, i, i, i, i, i, i, z(2, dtype=torch.int64), page_size=16, num_pages=2)
    q, kv = z(3, 4, 128, dtype=torch.bfloat16), z(3, 2, 128, dtype=torch.bfloat16)
    cache = z(2, 16, 2, 128, dtype=torch.bfloat16)
    args = [q, kv, kv, None, None, z(8, 128), z(3, dtype=torch.int32), z(3, dtype=torch.int64), q, cache, cache]
    with pytest.raises(ValueError, match="q is on cpu"):
        pa.pafp8_norm_rope_append(*args)
    with pytest.raises(ValueError, match="are not"):
        pa.pafp8_norm_rope_append(*args[:1], kv[:2], *args[2:])
    with pytest.raises(ValueError, match="different dtypes"):
        pa.pafp8_norm_rope_append(*args[:1], kv.half(), *args[2:])


def test_null_descriptions_are_refused():
    assert pa.lib().pafp8_build_tables(None, None) == 3 and pa.lib().pafp8_norm_rope_append(None, None) == 3


def test_packed_descriptions_are_the_structures():
    """The binding packs its descriptions by format; the formats lay the fields
    out as the structures do."""
    for fmt, cls in ((pa._TABLES, pa.tables_desc), (pa._ROPE, pa.rope_desc)):
        vals = [float(i + 1) if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(cls._fields_)]
        raw = fmt.pack(*vals)
        d = cls.from_buffer_copy(raw.ljust(ctypes.sizeof(cls), b"\0"))
        assert [getattr(d, n) for n, _ in cls._fields_] == vals
        assert ctypes.sizeof(cls) == fmt.size


def test_step_tables_keep_their_arrays():
    import torch

    t = pa.StepTables(batch=2, max_pages=4, max_tokens=8, page_size=16, num_pages=4, mask_words=1, device="cpu")
    with pytest.raises(AttributeError, match="slots"):
        t.slots = torch.zeros(8, dtype=torch.int64)
    with pytest.raises(AttributeError, match="batch"):
        t.batch = 3
    assert t.tree_mask.shape == (8, 1) and t.slots.dtype is torch.int64
