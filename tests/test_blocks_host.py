"""Refusals of the block-scale append and the read-back (no GPU needed: every
check is on the host, before any launch), and the reference's own rounding."""
import ctypes

import numpy as np
import pytest
import torch

import paged_attention_fp8_gb300 as pa
from blocks_ref import TOP, TORCH, grid, own_scale

A = 0x10000  # an aligned address that no refused call reads


def append(**kw):
    a = dict(k=A, v=A + 512, qo_indptr=A, cached_lens=A, kv_indptr=A, kv_indices=A, k_cache=A, v_cache=A + 4096, k_scales=A,
             v_scales=A + 4096, status=None, nnz=4, k_stride=512, v_stride=512, batch=2, src_dtype=pa.BF16, kv_dtype=pa.E4M3FN,
             kv_layout=0, num_kv_heads=2, head_dim=128, num_pages=8, page_size=16)
    a.update(kw)
    return pa.lib().pafp8_append_kv_blocks(ctypes.byref(pa.block_append_desc(**a)), None)


def read(**kw):
    a = dict(k_cache=A, v_cache=A, out_indptr=A, starts=A, kv_indptr=A, kv_indices=A, k_out=A, v_out=A, k_scales=A, v_scales=A,
             status=None, nnz=4, batch=2, kv_dtype=pa.E5M2, out_dtype=pa.BF16, kv_layout=1, num_kv_heads=2, head_dim=64,
             num_pages=8, page_size=32, k_scale=1.0, v_scale=1.0)
    a.update(kw)
    return pa.lib().pafp8_read_kv(ctypes.byref(pa.read_desc(**a)), None)


SHARED = [
    (dict(kv_dtype=pa.BF16), 1, "bfloat16"), (dict(kv_dtype=pa.INT8), 1, "int8"), (dict(kv_layout=2), 3, "kv_layout 2"),
    (dict(nnz=-1), 2, "nnz -1"), (dict(nnz=1 << 31), 2, "below 2^31"), (dict(batch=-1), 2, "batch -1"),
    (dict(num_pages=-1), 2, "num_pages -1"), (dict(num_kv_heads=0), 2, "num_kv_heads 0"),
    (dict(num_kv_heads=65537), 2, "num_kv_heads 65537"), (dict(head_dim=96), 8, "head_dim 96"),
    (dict(page_size=24), 8, "page_size 24"), (dict(page_size=0), 8, "page_size 0"), (dict(k_cache=None), 3, "non-NULL"),
    (dict(kv_indptr=None), 3, "non-NULL"), (dict(kv_indices=None), 3, "non-NULL"), (dict(k_cache=A + 8), 3, "16-byte"),
    (dict(k_scales=A + 2), 3, "4-byte"), (dict(kv_indices=A + 1), 3, "4-byte"), (dict(status=A + 2), 3, "4-byte")]


@pytest.mark.parametrize("kw,status,words", SHARED + [
    (dict(src_dtype=pa.E4M3FN), 1, "float8_e4m3fn"), (dict(k=None), 3, "non-NULL"), (dict(v_scales=None), 3, "non-NULL"),
    (dict(cached_lens=None), 3, "non-NULL"), (dict(k_stride=248), 2, "strides"), (dict(v_stride=0), 2, "strides"),
    (dict(k_stride=516), 3, "multiples of 8"), (dict(v=A + 8), 3, "16-byte"), (dict(v_cache=A), 3, "a cache and scales each"),
    (dict(v_scales=A), 3, "a cache and scales each")])
def test_append_refusals(kw, status, words):
    assert append(**kw) == status
    assert words in pa.pafp8_last_error()


@pytest.mark.parametrize("kw,status,words", SHARED + [
    (dict(out_dtype=pa.E5M2), 1, "float8_e5m2"), (dict(k_scales=None), 3, "both k_scales and v_scales"),
    (dict(k_scale=2.0), 3, "must then be 1"), (dict(k_scales=None, v_scales=None, v_scale=0.0), 3, "finite and > 0"),
    (dict(k_out=None), 3, "non-NULL"), (dict(starts=None), 3, "non-NULL"), (dict(v_out=A + 4), 3, "16-byte")])
def test_read_refusals(kw, status, words):
    assert read(**kw) == status
    assert words in pa.pafp8_last_error()


def test_nothing_to_do_is_ok():
    assert append(nnz=0, k=None, k_cache=None) == 0
    assert read(nnz=0, k_out=None, k_cache=None) == 0
    assert pa.lib().pafp8_append_kv_blocks(None, None) == 3 and pa.lib().pafp8_read_kv(None, None) == 3


@pytest.fixture
def on_cpu(monkeypatch):
    """The binding with the library's two calls recorded and the CPU standing for the device."""
    calls = []
    real = pa.lib()

    class Recorder:
        def __getattr__(self, name):
            if name in ("pafp8_append_kv_blocks", "pafp8_read_kv"):
                return lambda *a: calls.append(a) or 0
            return getattr(real, name)

    monkeypatch.setattr(pa, "lib", lambda: Recorder())
    monkeypatch.setattr(pa, "_device_of", lambda t, name: -1)
    return calls


def z(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


BF, E4, F = torch.bfloat16, torch.float8_e4m3fn, torch.float32


def append_args():
    return dict(k_new=z(7, 2, 128, dtype=BF), v_new=z(7, 2, 128, dtype=BF), qo_indptr=z(4), cached_lens=z(3), kv_indptr=z(4),
                kv_indices=z(9), k_cache=z(6, 32, 2, 128, dtype=E4), v_cache=z(6, 32, 2, 128, dtype=E4), k_scales=z(6, 2, 2, dtype=F),
                v_scales=z(6, 2, 2, dtype=F))


@pytest.mark.parametrize("kw,match", [
    (dict(k_new=z(7, 256, dtype=BF)), r"\[n, Hkv, D\]"), (dict(v_new=z(6, 2, 128, dtype=BF)), r"\[n, Hkv, D\]"),
    (dict(v_new=z(7, 2, 128, dtype=F)), "one dtype"), (dict(k_new=z(7, 128, 2, dtype=BF).transpose(1, 2)), "heads of a token"),
    (dict(k_new=z(7, 4, 128, dtype=BF)[:, ::2]), "heads of a token"), (dict(cached_lens=z(2)), "cached_lens"),
    (dict(cached_lens=z(3, dtype=torch.int64)), "cached_lens has dtype"), (dict(kv_indptr=z(3)), "kv_indptr"),
    (dict(qo_indptr=z(0)), "qo_indptr is empty"), (dict(kv_indices=z(18)[::2]), "kv_indices"),
    (dict(k_cache=z(6, 2, 32, 128, dtype=E4)), "do not hold"), (dict(v_cache=z(5, 32, 2, 128, dtype=E4)), "do not hold"),
    (dict(v_cache=z(6, 32, 2, 128, dtype=torch.float8_e5m2)), "v_cache has dtype"),
    (dict(k_cache=z(6, 32, 4, 128, dtype=E4)[:, :, :2]), "k_cache .* is not contiguous"),
    (dict(k_scales=z(6, 2, dtype=F)), "k_scales"), (dict(v_scales=z(6, 1, 2, dtype=F)), "v_scales"),
    (dict(k_scales=z(6, 2, 2, dtype=torch.float64)), "k_scales has dtype"), (dict(status=z(0)), "status"),
    (dict(kv_layout="HND"), "do not hold")])
def test_binding_refuses_for_the_append(on_cpu, kw, match):
    with pytest.raises(ValueError, match=match):
        pa.pafp8_append_kv_blocks(**{**append_args(), **kw}, stream=1)
    assert not on_cpu


def test_binding_passes_on_what_fits(on_cpu):
    a = append_args()
    pa.pafp8_append_kv_blocks(**a, stream=1)
    a["k_new"], a["v_new"] = z(7, 4, 128, dtype=BF)[:, :2], z(7, 4, 128, dtype=BF)[:, 2:]
    pa.pafp8_append_kv_blocks(**a, stream=1)
    a["k_cache"], a["v_cache"] = (z(6, 2, 32, 128, dtype=E4) for _ in range(2))
    pa.pafp8_append_kv_blocks(**a, kv_layout="HND", status=z(1), stream=1)
    assert len(on_cpu) == 3
    got = pa.block_append_desc.from_buffer_copy(on_cpu[1][0])
    assert (got.nnz, got.k_stride, got.batch, got.head_dim, got.page_size, got.num_pages) == (7, 512, 3, 128, 32, 6)


def read_args():
    a = append_args()
    return dict(k_cache=a["k_cache"], v_cache=a["v_cache"], out_indptr=z(4), starts=z(3), kv_indptr=z(4), kv_indices=z(9),
                k_out=z(7, 2, 128, dtype=BF), v_out=z(7, 2, 128, dtype=BF))


@pytest.mark.parametrize("kw,match", [
    (dict(k_out=z(7, 256, dtype=BF)), r"\[n, Hkv, D\]"), (dict(v_out=z(8, 2, 128, dtype=BF)), r"\[n, Hkv, D\]"),
    (dict(v_out=z(7, 2, 128, dtype=F)), "v_out has dtype"), (dict(k_out=z(7, 4, 128, dtype=BF)[:, :2]), "k_out .* is not contiguous"),
    (dict(starts=z(2)), "starts"), (dict(out_indptr=z(0)), "out_indptr is empty"), (dict(kv_indptr=z(4, dtype=torch.int64)), "kv_indptr"),
    (dict(k_scales=z(6, 2, 3, dtype=F)), "k_scales"), (dict(k_cache=z(6, 32, 2, 64, dtype=E4)), "do not hold")])
def test_binding_refuses_for_the_read(on_cpu, kw, match):
    with pytest.raises(ValueError, match=match):
        pa.pafp8_read_kv(**{**read_args(), **kw}, stream=1)
    assert not on_cpu


def test_host_tensors_are_refused():
    if not torch.cuda.is_available():
        with pytest.raises(ValueError, match="is on cpu"):
            pa.pafp8_append_kv_blocks(**append_args())
        with pytest.raises(ValueError, match="is on cpu"):
            pa.pafp8_read_kv(**read_args())


@pytest.mark.parametrize("fmt", ["e4m3fn", "e5m2"])
def test_reference_rounding_is_the_types(fmt):
    """grid() against torch's own cast of values within range, and own_scale() at its borders."""
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(4000, generator=g) * s for s in (1e-3, 0.1, 3.0, TOP[fmt] / 8)]).clamp(-TOP[fmt], TOP[fmt])
    np.testing.assert_array_equal(grid(x.double().numpy(), fmt), x.to(TORCH[fmt]).double().numpy())
    assert own_scale([TOP[fmt]], fmt) == 1 and own_scale([TOP[fmt] * (1 + 2 ** -20)], fmt) == 2
    assert own_scale([0.0], fmt) == own_scale([float("nan"), float("inf")], fmt) == 2.0 ** -64
