"""paged_attention_fp8_gb300 -- Python binding of libpafp8.

Paged attention of a bf16/f16 (or fp8) query against a KV cache stored in
fp8 (e4m3fn/e5m2) with per-tensor scales, on GB300 (sm_103a).  Every step of
the computation runs in the CUDA library ``libpafp8.so``; this module only
marshals arguments through its C ABI (``include/pafp8.h``) with ctypes.  The
functions carry the C names.  There is no fallback: if the library is not
built, every call raises.

Typical use::

    plan = Plan(mode="decode", num_qo_heads=32, num_kv_heads=8, num_pages=...,
                kv_indptr=..., last_page_len=..., q_dtype=torch.bfloat16,
                kv_dtype=torch.float8_e4m3fn)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    plan.upload(ws)
    plan.run(q, k_cache, v_cache, kv_indices, o, lse, ws, k_scale=..., v_scale=...)
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpafp8.so")

# dtype codes of include/pafp8.h
DTYPE_DEFAULT, F16, BF16, E4M3FN, E5M2, F32, INT8, UINT8 = range(8)
MODE_DECODE, MODE_PREFILL, MODE_TREE = 0, 1, 2
_MODES = {"decode": MODE_DECODE, "prefill": MODE_PREFILL, "tree": MODE_TREE}
LAYOUT_NHD, LAYOUT_HND = 0, 1
_LAYOUTS = {"NHD": LAYOUT_NHD, "HND": LAYOUT_HND}
STATUS = {0: "OK", 1: "ERR_DTYPE", 2: "ERR_SHAPE", 3: "ERR_ARG", 4: "ERR_WORKSPACE", 5: "ERR_CUDA",
          6: "ERR_TIMEOUT", 7: "ERR_BOUNDS", 8: "ERR_UNSUPPORTED"}
_NAME_CODES = {"default": DTYPE_DEFAULT, "f16": F16, "float16": F16, "bf16": BF16, "bfloat16": BF16,
               "e4m3fn": E4M3FN, "float8_e4m3fn": E4M3FN, "e5m2": E5M2, "float8_e5m2": E5M2,
               "f32": F32, "float32": F32, "int8": INT8, "uint8": UINT8}

# Every entry point include/pafp8.h declares.
EXPORTS = ("pafp8_abi_version", "pafp8_last_error", "pafp8_plan_create", "pafp8_plan_destroy",
           "pafp8_workspace_bytes", "pafp8_plan_metadata", "pafp8_plan_upload", "pafp8_run",
           "pafp8_run_stage", "pafp8_device_status", "pafp8_run_decode_noalloc", "pafp8_append_kv",
           "pafp8_run_head_scales", "pafp8_run_pod", "pafp8_host_workspace_bytes", "pafp8_run_host",
           "pafp8_build_tables", "pafp8_norm_rope_append", "pafp8_run_tree")


class Pafp8Error(RuntimeError):
    """A non-OK status from libpafp8, with its sentence."""

    def __init__(self, status: int, message: str):
        self.status = status
        self.status_name = STATUS.get(status, str(status))
        super().__init__(f"{self.status_name}: {message}")


class plan_desc(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("num_qo_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("q_dtype", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("o_dtype", ctypes.c_int32),
                ("sm_scale", ctypes.c_float), ("fixed_split_pages", ctypes.c_int32),
                ("disable_split_kv", ctypes.c_int32), ("num_ctas", ctypes.c_int32),
                ("kv_layout", ctypes.c_int32)]


class pod_phase(ctypes.Structure):
    _fields_ = [("plan", ctypes.c_void_p), ("q", ctypes.c_void_p), ("kv_indices", ctypes.c_void_p),
                ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class tables_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "cached_lens", "new_lens", "block_table", "free_pages", "free_used", "free_used_out", "kv_indptr",
        "last_page_len", "kv_indices", "qo_indptr", "batch_indices", "positions", "slots", "parents", "rope_positions",
        "tree_mask", "status")] + \
        [(n, ctypes.c_int64) for n in ("block_stride", "max_pages", "max_tokens")] + \
        [(n, ctypes.c_int32) for n in ("batch", "page_size", "num_pages", "num_free", "block_width", "mask_words")]


class rope_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "q", "k", "v", "q_weight", "k_weight", "cos_sin", "positions", "pair_axis", "slots", "q_out", "k_cache",
        "v_cache", "status")] + \
        [(n, ctypes.c_int64) for n in ("nnz", "q_stride", "k_stride", "v_stride", "pos_stride")] + \
        [(n, ctypes.c_int32) for n in (
            "src_dtype", "q_out_dtype", "kv_dtype", "kv_layout", "num_qo_heads", "num_kv_heads", "head_dim", "rot_dim",
            "interleaved", "num_axes", "max_position", "num_pages", "page_size")] + \
        [(n, ctypes.c_float) for n in ("eps", "q_scale", "k_scale", "v_scale")]


# The same two structures as struct formats: packing one costs a third of a
# microsecond, filling a ctypes structure field by field five.
_TABLES = struct.Struct("@17P3q6i")
_ROPE = struct.Struct("@13P5q13i4f0q")

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libpafp8.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libpafp8.so is not built ({LIB_PATH} missing); run "
                           "paged_attention_fp8_gb300.build.build() first")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    L.pafp8_abi_version.argtypes, L.pafp8_abi_version.restype = [], i32
    L.pafp8_last_error.argtypes, L.pafp8_last_error.restype = [], ctypes.c_char_p
    L.pafp8_plan_create.argtypes = [ctypes.POINTER(plan_desc), vp, vp, vp, ctypes.POINTER(vp)]
    L.pafp8_plan_create.restype = i32
    L.pafp8_plan_destroy.argtypes, L.pafp8_plan_destroy.restype = [vp], None
    L.pafp8_workspace_bytes.argtypes, L.pafp8_workspace_bytes.restype = [vp], sz
    L.pafp8_plan_metadata.argtypes = [vp, ctypes.POINTER(ctypes.POINTER(ctypes.c_int32)),
                                      ctypes.POINTER(sz)]
    L.pafp8_plan_metadata.restype = i32
    L.pafp8_plan_upload.argtypes, L.pafp8_plan_upload.restype = [vp, vp, sz, vp], i32
    L.pafp8_run.argtypes = [vp, i32, vp, i32, vp, i32, vp, vp, f32, f32, f32, i32, vp, vp, vp, sz, vp]
    L.pafp8_run.restype = i32
    L.pafp8_run_stage.argtypes = [vp, i32, i32, vp, i32, vp, i32, vp, vp, f32, f32, f32, i32, vp, vp,
                                  vp, sz, vp]
    L.pafp8_run_stage.restype = i32
    L.pafp8_host_workspace_bytes.argtypes, L.pafp8_host_workspace_bytes.restype = [vp, i32], sz
    L.pafp8_run_host.argtypes = [vp, i32, vp, i32, vp, i32, vp, vp, f32, f32, f32, i32, vp, vp, vp, sz, vp]
    L.pafp8_run_host.restype = i32
    L.pafp8_device_status.argtypes, L.pafp8_device_status.restype = [vp, vp, vp], i32
    L.pafp8_run_decode_noalloc.argtypes = [vp, i32, vp, i32, vp, i32, vp, vp, f32, f32, f32, i32, vp,
                                           vp, vp]
    L.pafp8_run_decode_noalloc.restype = i32
    L.pafp8_append_kv.argtypes = [i32, vp, vp, ctypes.c_int64, i32, i32, vp, vp, i32, vp, vp, i32, i32, vp,
                                  vp, i32, i32, f32, f32, vp, vp]
    L.pafp8_append_kv.restype = i32
    L.pafp8_run_head_scales.argtypes = [vp, i32, vp, i32, vp, i32, vp, vp, vp, vp, vp, i32, vp, vp, vp, sz, vp]
    L.pafp8_run_head_scales.restype = i32
    L.pafp8_run_pod.argtypes = [ctypes.POINTER(pod_phase), ctypes.POINTER(pod_phase), i32, i32, vp, i32, vp,
                                f32, f32, f32, i32, vp]
    L.pafp8_run_pod.restype = i32
    L.pafp8_run_tree.argtypes = [vp, i32, vp, i32, vp, i32, vp, vp, vp, i32, f32, f32, f32, vp, vp, vp, i32, vp, vp, vp,
                                 sz, vp]
    L.pafp8_run_tree.restype = i32
    # Their descriptions come packed (_TABLES, _ROPE) or as the structures above.
    L.pafp8_build_tables.argtypes, L.pafp8_build_tables.restype = [vp, vp], i32
    L.pafp8_norm_rope_append.argtypes, L.pafp8_norm_rope_append.restype = [vp, vp], i32
    _lib = L
    return L


_T = None  # the torch module, once a step call has used it: importing this module does not import torch


def _torch():
    """torch (an import statement in every call would cost it half a microsecond)."""
    global _T
    if _T is None:
        import torch
        _T = torch
    return _T


_OBJ_CODES = {}  # dtype objects seen before -> code (the run calls pass torch dtypes)


def dtype_code(x) -> int:
    """int32 dtype code for a torch dtype, a name or a code."""
    if isinstance(x, int):
        return x
    if isinstance(x, str):
        return _NAME_CODES[x]
    code = _OBJ_CODES.get(x)
    if code is not None:
        return code
    name = str(x).replace("torch.", "")
    if name not in _NAME_CODES:
        raise ValueError(f"no libpafp8 dtype code for {x}")
    _OBJ_CODES[x] = _NAME_CODES[name]
    return _NAME_CODES[name]


def _check(status: int) -> None:
    if status != 0:
        raise Pafp8Error(status, pafp8_last_error())


def _i32_host(a):
    """A host int32 array: a contiguous CPU int32 tensor as it is (its
    data_ptr is passed), anything else as a contiguous numpy int32 array."""
    if a is None:
        return None
    if hasattr(a, "cpu"):
        if a.device.type == "cpu" and str(a.dtype) == "torch.int32" and a.is_contiguous():
            return a
        a = a.cpu().numpy()
    return np.ascontiguousarray(a, dtype=np.int32)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


# ---- the C entry points, same names --------------------------------------

def pafp8_abi_version() -> int:
    return int(lib().pafp8_abi_version())


def pafp8_last_error() -> str:
    return lib().pafp8_last_error().decode()


# What pafp8_run_tree needs of its arrays, by the handles of the tree plans that
# exist: the shapes of q and o, of the caches and of lse, page ids, mask rows, KV heads.
_TREE_SIZES = {}
_ITEM = {F16: 2, BF16: 2, E4M3FN: 1, E5M2: 1}  # bytes of an element; the library refuses other types


def _tree_sizes(desc, kv_indptr, qo_indptr):
    rows = int(qo_indptr[-1]) if desc.batch > 0 else 0
    hq, hkv, ps, d = desc.num_qo_heads, desc.num_kv_heads, desc.page_size, desc.head_dim
    page = (hkv, ps, d) if desc.kv_layout == LAYOUT_HND else (ps, hkv, d)
    return (rows, hq, d), (desc.num_pages, *page), (rows, hq), int(kv_indptr[-1]) if desc.batch > 0 else 0, rows, hkv


def _tree_fits(sizes, arrays, kv_indices, lse) -> None:
    """ValueError for an array with fewer bytes than the plan's shapes take
    (larger and differently shaped ones are taken as they lie), or a cache
    whose pages are shaped otherwise.  arrays: (tensor, name, dtype code, shape)."""
    for t, name, code, shape in (*arrays, (kv_indices, "kv_indices", None, (sizes[3],)), (lse, "lse", None, sizes[2])):
        need = (4 if code is None else _ITEM.get(code, 0)) * int(np.prod(shape, dtype=np.int64))
        if t is not None and t.nbytes < need:
            raise ValueError(f"{name} {tuple(t.shape)} of {t.dtype} has {t.nbytes} bytes; the plan needs {need}")
        if shape is sizes[1] and t.dim() == 4 and tuple(t.shape[1:]) != shape[1:]:
            raise ValueError(f"{name} {tuple(t.shape)} has pages of {tuple(t.shape[1:])}; the plan's are {shape[1:]}")


def pafp8_plan_create(desc: plan_desc, kv_indptr, last_page_len, qo_indptr=None) -> int:
    kv_indptr, last_page_len, qo_indptr = _i32_host(kv_indptr), _i32_host(last_page_len), _i32_host(qo_indptr)
    out = ctypes.c_void_p()
    _check(lib().pafp8_plan_create(ctypes.byref(desc), _ptr(kv_indptr), _ptr(last_page_len),
                                   _ptr(qo_indptr), ctypes.byref(out)))
    if desc.mode == MODE_TREE:
        _TREE_SIZES[out.value] = _tree_sizes(desc, kv_indptr, qo_indptr)
    return out.value


def pafp8_plan_destroy(handle: int) -> None:
    _TREE_SIZES.pop(handle, None)
    lib().pafp8_plan_destroy(handle)


def pafp8_workspace_bytes(handle: int) -> int:
    return int(lib().pafp8_workspace_bytes(handle))


def pafp8_plan_metadata(handle: int) -> np.ndarray:
    words = ctypes.POINTER(ctypes.c_int32)()
    n = ctypes.c_size_t()
    _check(lib().pafp8_plan_metadata(handle, ctypes.byref(words), ctypes.byref(n)))
    return np.ctypeslib.as_array(words, shape=(n.value,)).copy()


def pafp8_plan_upload(handle: int, workspace, stream=None) -> None:
    _check(lib().pafp8_plan_upload(handle, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _stream(stream)))


def pafp8_run(handle: int, q, k_cache, v_cache, kv_indices, o, lse, workspace, *, q_scale=1.0,
              k_scale=1.0, v_scale=1.0, q_dtype=None, k_dtype=None, v_dtype=None, o_dtype=None,
              stream=None) -> None:
    """Dtype codes default to the tensors' own dtypes."""
    _check(lib().pafp8_run(
        handle, dtype_code(q_dtype if q_dtype is not None else q.dtype), _ptr(q),
        dtype_code(k_dtype if k_dtype is not None else k_cache.dtype), _ptr(k_cache),
        dtype_code(v_dtype if v_dtype is not None else v_cache.dtype), _ptr(v_cache),
        _ptr(kv_indices), float(q_scale), float(k_scale), float(v_scale),
        dtype_code(o_dtype if o_dtype is not None else o.dtype), _ptr(o), _ptr(lse),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def pafp8_host_workspace_bytes(handle: int, q_dtype) -> int:
    return int(lib().pafp8_host_workspace_bytes(handle, dtype_code(q_dtype)))


def pafp8_run_host(handle: int, q_h, k_cache, v_cache, kv_indices_h, o_h, lse_h, workspace, *, q_scale=1.0,
                   k_scale=1.0, v_scale=1.0, q_dtype=None, k_dtype=None, v_dtype=None, o_dtype=None,
                   stream=None) -> None:
    """One step from and to host memory (q_h, kv_indices_h, o_h, lse_h: CPU
    tensors, preferably pinned); dtype codes default to the tensors' own."""
    _check(lib().pafp8_run_host(
        handle, dtype_code(q_dtype if q_dtype is not None else q_h.dtype), _ptr(q_h),
        dtype_code(k_dtype if k_dtype is not None else k_cache.dtype), _ptr(k_cache),
        dtype_code(v_dtype if v_dtype is not None else v_cache.dtype), _ptr(v_cache),
        _ptr(kv_indices_h), float(q_scale), float(k_scale), float(v_scale),
        dtype_code(o_dtype if o_dtype is not None else o_h.dtype), _ptr(o_h), _ptr(lse_h),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def pafp8_run_stage(handle: int, stage: int, q, k_cache, v_cache, kv_indices, o, lse, workspace, *,
                    q_scale=1.0, k_scale=1.0, v_scale=1.0, q_dtype=None, k_dtype=None, v_dtype=None,
                    o_dtype=None, stream=None) -> None:
    """pafp8_run limited to stage 1 (attention kernel) or 2 (merge); 0 = all."""
    _check(lib().pafp8_run_stage(
        handle, int(stage), dtype_code(q_dtype if q_dtype is not None else q.dtype), _ptr(q),
        dtype_code(k_dtype if k_dtype is not None else k_cache.dtype), _ptr(k_cache),
        dtype_code(v_dtype if v_dtype is not None else v_cache.dtype), _ptr(v_cache),
        _ptr(kv_indices), float(q_scale), float(k_scale), float(v_scale),
        dtype_code(o_dtype if o_dtype is not None else o.dtype), _ptr(o), _ptr(lse),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def pafp8_run_head_scales(handle: int, q, k_cache, v_cache, kv_indices, o, lse, workspace, *, q_scales=None,
                          k_scales, v_scales, q_dtype=None, k_dtype=None, v_dtype=None, o_dtype=None,
                          stream=None) -> None:
    """pafp8_run with per-head scale tensors (device float32: q_scales [Hq] or
    None, k_scales and v_scales [Hkv])."""
    _check(lib().pafp8_run_head_scales(
        handle, dtype_code(q_dtype if q_dtype is not None else q.dtype), _ptr(q),
        dtype_code(k_dtype if k_dtype is not None else k_cache.dtype), _ptr(k_cache),
        dtype_code(v_dtype if v_dtype is not None else v_cache.dtype), _ptr(v_cache),
        _ptr(kv_indices), _ptr(q_scales), _ptr(k_scales), _ptr(v_scales),
        dtype_code(o_dtype if o_dtype is not None else o.dtype), _ptr(o), _ptr(lse),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def pafp8_run_tree(handle: int, q, k_cache, v_cache, kv_indices, tree_mask, o, lse, workspace, *, q_scale=1.0,
                   k_scale=1.0, v_scale=1.0, q_scales=None, k_scales=None, v_scales=None, q_dtype=None, k_dtype=None,
                   v_dtype=None, o_dtype=None, stream=None) -> None:
    """Attention of a tree of drafted tokens (a plan of mode "tree"): tree_mask
    [nnz_qo, words] of int32 (bits), as StepTables holds it; per-head scale
    tensors (device float32: q_scales [Hq] or None, k_scales and v_scales
    [Hkv]) instead of the per-tensor ones when k_scales is given.  Arrays are
    contiguous; kv_indices is int32, lse float32 or None."""
    T = _torch()
    dev = _device_of(q, "q")
    qt, kt, vt, ot, i32, f32 = q.dtype, k_cache.dtype, v_cache.dtype, o.dtype, T.int32, T.float32
    for t, name, dtype in ((q, "q", qt), (k_cache, "k_cache", kt), (v_cache, "v_cache", vt), (kv_indices, "kv_indices", i32),
                           (o, "o", ot), (lse, "lse", f32), (workspace, "workspace", workspace.dtype)):
        if t is not None and (t.get_device() != dev or t.dtype is not dtype or not t.is_contiguous()):
            _refuse(t, name, dtype, dev)
    code = _OBJ_CODES.get
    qc = code(qt) or dtype_code(qt) if q_dtype is None else dtype_code(q_dtype)
    oc = code(ot) or dtype_code(ot) if o_dtype is None else dtype_code(o_dtype)
    kc = code(kt) or dtype_code(kt) if k_dtype is None else dtype_code(k_dtype)
    vc = code(vt) or dtype_code(vt) if v_dtype is None else dtype_code(v_dtype)
    sizes = _TREE_SIZES.get(handle)
    if sizes is None:
        hq, hkv, n_rows = 0, 0, q.shape[0]
    else:
        rows_of, pool, lse_of, n_index, n_rows, hkv = sizes
        hq = rows_of[1]
        if q.shape != rows_of or o.shape != rows_of or k_cache.shape != pool or v_cache.shape != pool or \
                (lse is not None and lse.shape != lse_of) or (kv_indices is not None and kv_indices.numel() < n_index) or \
                q_dtype is not None or o_dtype is not None or k_dtype is not None or v_dtype is not None:
            _tree_fits(sizes, ((q, "q", qc, rows_of), (o, "o", oc, rows_of), (k_cache, "k_cache", kc, pool),
                               (v_cache, "v_cache", vc, pool)), kv_indices, lse)
    scales = (0, 0, 0) if q_scales is k_scales is v_scales is None else (
        _addr(q_scales, "q_scales", hq, f32, dev), _addr(k_scales, "k_scales", hkv, f32, dev),
        _addr(v_scales, "v_scales", hkv, f32, dev))
    rows, words = tree_mask.shape if tree_mask.dim() == 2 else (-1, 0)
    if rows < n_rows or tree_mask.get_device() != dev or not tree_mask.is_contiguous() or \
            (tree_mask.dtype is not i32 and (tree_mask.element_size() != 4 or tree_mask.is_floating_point())):
        raise ValueError(f"tree_mask {tuple(tree_mask.shape)} of {tree_mask.dtype} on {tree_mask.device} is not a "
                         f"contiguous int32 [{n_rows}, words] tensor on the query's device")
    _check(lib().pafp8_run_tree(
        handle, qc, q.data_ptr(), kc, k_cache.data_ptr(), vc, v_cache.data_ptr(), _ptr(kv_indices), tree_mask.data_ptr(), words,
        q_scale, k_scale, v_scale, *scales, oc, o.data_ptr(), _ptr(lse), workspace.data_ptr(), workspace.nbytes,
        _stream_on(dev, stream)))


def pafp8_device_status(handle: int, workspace, stream=None) -> None:
    _check(lib().pafp8_device_status(handle, _ptr(workspace), _stream(stream)))


def pafp8_run_decode_noalloc(handle: int, q, k_cache, v_cache, kv_indices, o, lse, *, q_scale=1.0,
                             k_scale=1.0, v_scale=1.0, q_dtype=None, k_dtype=None, v_dtype=None,
                             o_dtype=None, stream=None) -> None:
    """Decode with the library's built-in scratch instead of a workspace, for
    callers that may not allocate device memory (see include/pafp8.h)."""
    _check(lib().pafp8_run_decode_noalloc(
        handle, dtype_code(q_dtype if q_dtype is not None else q.dtype), _ptr(q),
        dtype_code(k_dtype if k_dtype is not None else k_cache.dtype), _ptr(k_cache),
        dtype_code(v_dtype if v_dtype is not None else v_cache.dtype), _ptr(v_cache),
        _ptr(kv_indices), float(q_scale), float(k_scale), float(v_scale),
        dtype_code(o_dtype if o_dtype is not None else o.dtype), _ptr(o), _ptr(lse), _stream(stream)))


def _phase(handle, q, kv_indices, o, lse, workspace) -> pod_phase:
    return pod_phase(handle, _ptr(q), _ptr(kv_indices), _ptr(o), _ptr(lse), _ptr(workspace),
                     workspace.numel() * workspace.element_size())


def pafp8_run_pod(prefill_handle: int, prefill_q, prefill_kv_indices, prefill_o, prefill_lse, prefill_workspace,
                  decode_handle: int, decode_q, decode_kv_indices, decode_o, decode_lse, decode_workspace,
                  k_cache, v_cache, *, q_scale=1.0, k_scale=1.0, v_scale=1.0, q_dtype=None, k_dtype=None,
                  v_dtype=None, o_dtype=None, stream=None) -> None:
    """A prefill plan's phase and a decode plan's phase over one cache in one
    call, side by side on the SMs their plans' num_ctas give (see
    include/pafp8.h).  Dtype codes default to the prefill tensors' dtypes."""
    pre = _phase(prefill_handle, prefill_q, prefill_kv_indices, prefill_o, prefill_lse, prefill_workspace)
    dec = _phase(decode_handle, decode_q, decode_kv_indices, decode_o, decode_lse, decode_workspace)
    _check(lib().pafp8_run_pod(
        ctypes.byref(pre), ctypes.byref(dec), dtype_code(q_dtype if q_dtype is not None else prefill_q.dtype),
        dtype_code(k_dtype if k_dtype is not None else k_cache.dtype), _ptr(k_cache),
        dtype_code(v_dtype if v_dtype is not None else v_cache.dtype), _ptr(v_cache),
        float(q_scale), float(k_scale), float(v_scale),
        dtype_code(o_dtype if o_dtype is not None else prefill_o.dtype), _stream(stream)))


def pafp8_append_kv(k_new, v_new, batch_indices, positions, kv_indptr, kv_indices, k_cache, v_cache, *,
                    k_scale=1.0, v_scale=1.0, status=None, src_dtype=None, kv_dtype=None,
                    kv_layout="NHD", num_pages=None, stream=None) -> None:
    """Quantize new tokens k_new/v_new [nnz, Hkv, D] into the paged fp8 cache
    (see include/pafp8.h).  Index arrays are device int32; dtype codes,
    head counts and sizes default to what the tensors say."""
    nnz, hkv, d = k_new.shape
    layout = _LAYOUTS[kv_layout] if isinstance(kv_layout, str) else int(kv_layout)
    page_size = int(k_cache.shape[2] if layout == LAYOUT_HND else k_cache.shape[1])
    _check(lib().pafp8_append_kv(
        dtype_code(src_dtype if src_dtype is not None else k_new.dtype), _ptr(k_new), _ptr(v_new), int(nnz),
        int(hkv), int(d), _ptr(batch_indices), _ptr(positions), int(kv_indptr.numel() - 1), _ptr(kv_indptr),
        _ptr(kv_indices), dtype_code(kv_dtype if kv_dtype is not None else k_cache.dtype), layout,
        _ptr(k_cache), _ptr(v_cache), int(num_pages if num_pages is not None else k_cache.shape[0]),
        page_size, float(k_scale), float(v_scale), _ptr(status), _stream(stream)))


def _refuse(t, name, dtype, dev) -> None:
    """The sentence for an array that _bad found wanting."""
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on the current CUDA device")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, not {dtype}")
    raise ValueError(f"{name} (shape {tuple(t.shape)}, strides {t.stride()}) is not contiguous or too small")


def _addr(t, name, n, dtype, dev) -> int:
    """The address of a contiguous tensor of `dtype` on device `dev` with n
    elements at least (None: 0); ValueError otherwise."""
    if t is None:
        return 0
    if t.get_device() != dev or t.dtype is not dtype or not t.is_contiguous() or t.numel() < n:
        _refuse(t, name, dtype, dev)
    return t.data_ptr()


def _stream_on(dev, stream) -> Optional[int]:
    """`stream`, or the current stream of device `dev`: _stream without the
    torch.cuda.Stream object that it makes, a tenth of a small step's call."""
    if stream is None:
        return _torch()._C._cuda_getCurrentRawStream(dev)
    return getattr(stream, "cuda_stream", stream)


def _device_of(t, name) -> int:
    """The current CUDA device, which `t` must be on."""
    dev = _torch().cuda.current_device() if t.is_cuda else -2
    if t.get_device() != dev:
        _refuse(t, name, t.dtype, dev)
    return dev


def pafp8_build_tables(cached_lens, new_lens, block_table, free_pages, free_used, free_used_out, kv_indptr,
                       last_page_len, kv_indices, qo_indptr, batch_indices, positions, slots, *, page_size, num_pages,
                       parents=None, rope_positions=None, tree_mask=None, status=None, stream=None) -> None:
    """Block tables and slot maps of one step from request lengths, on the
    device (see include/pafp8.h; StepTables owns the outputs).  Arrays are
    contiguous device int32 tensors, slots int64; block_table is
    [batch, width] with contiguous rows; tree_mask is [tokens, words]."""
    i32 = _torch().int32
    dev = _device_of(cached_lens, "cached_lens")
    batch, tokens = cached_lens.numel(), slots.numel()
    words = 0
    if tree_mask is not None:
        if tree_mask.dim() != 2:
            raise ValueError(f"tree_mask has shape {tuple(tree_mask.shape)}, not [tokens, words]")
        words = tree_mask.shape[1]
    _build_tables(
        dev, cached_lens, new_lens, block_table, free_pages, free_used, parents,
        (_addr(free_used_out, "free_used_out", 1, i32, dev), _addr(kv_indptr, "kv_indptr", batch + 1, i32, dev),
         _addr(last_page_len, "last_page_len", batch, i32, dev), _addr(kv_indices, "kv_indices", 0, i32, dev),
         _addr(qo_indptr, "qo_indptr", batch + 1, i32, dev), _addr(batch_indices, "batch_indices", tokens, i32, dev),
         _addr(positions, "positions", tokens, i32, dev), _addr(slots, "slots", tokens, _T.int64, dev)),
        (_addr(rope_positions, "rope_positions", tokens, i32, dev),
         _addr(tree_mask, "tree_mask", tokens * words, i32, dev), _addr(status, "status", 1, i32, dev)),
        kv_indices.numel(), tokens, words, page_size, num_pages, stream)


def _build_tables(dev, cached_lens, new_lens, block_table, free_pages, free_used, parents, outs, tree_outs, max_pages,
                  tokens, words, page_size, num_pages, stream) -> None:
    """The call itself, its outputs given as addresses."""
    i32, batch = _torch().int32, cached_lens.numel()
    rows, width = block_table.shape
    if rows < batch or block_table.dtype is not i32 or block_table.get_device() != dev or \
            (width > 1 and block_table.stride(1) != 1):
        raise ValueError(f"block_table {tuple(block_table.shape)} of {block_table.dtype} on {block_table.device} is not "
                         f"an int32 [batch {batch}, width] device tensor with contiguous rows")
    _check(lib().pafp8_build_tables(_TABLES.pack(
        _addr(cached_lens, "cached_lens", batch, i32, dev), _addr(new_lens, "new_lens", batch, i32, dev),
        block_table.data_ptr(), _addr(free_pages, "free_pages", 0, i32, dev), _addr(free_used, "free_used", 1, i32, dev),
        *outs, _addr(parents, "parents", tokens, i32, dev), *tree_outs,
        block_table.stride(0) if rows > 1 else width, max_pages, tokens, batch, page_size, num_pages, free_pages.numel(),
        width, words), _stream_on(dev, stream)))


def pafp8_norm_rope_append(q, k, v, q_weight, k_weight, cos_sin, positions, slots, q_out, k_cache, v_cache, *,
                           eps=1e-6, pair_axis=None, interleaved=False, q_scale=1.0, k_scale=1.0, v_scale=1.0,
                           kv_layout="NHD", status=None, stream=None) -> None:
    """Per-head RMS norm of q [n, Hq, D] and k [n, Hkv, D], rotary rotation,
    and the append of k and v to the paged cache at `slots`, in one pass (see
    include/pafp8.h).  q, k and v may be slices of one packed projection (any
    token stride); positions is int32 [n] or [axes, n], slots int64 [n],
    cos_sin float32 [max_position, rot_dim].  Types come from the tensors."""
    T = _torch()
    i32 = T.int32
    shape, kshape, cshape, dt = q.shape, k.shape, k_cache.shape, q.dtype
    n, hq, d = shape
    _, hkv, _ = kshape
    layout = _LAYOUTS[kv_layout] if kv_layout in _LAYOUTS else int(kv_layout)
    if kshape != (n, hkv, d) or v.shape != kshape or q_out.shape != shape:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)} and q_out {tuple(q_out.shape)} are "
                         "not [n, Hq, D], [n, Hkv, D], [n, Hkv, D] and [n, Hq, D]")
    if k.dtype is not dt or v.dtype is not dt:
        raise ValueError(f"q, k and v have different dtypes ({dt}, {k.dtype}, {v.dtype})")
    dev = _device_of(q, "q")
    (qs, qh, q1), (ks, kh, k1), (vs, vh, v1) = q.stride(), k.stride(), v.stride()
    if k.get_device() != dev or v.get_device() != dev or q1 != 1 or k1 != 1 or v1 != 1 or \
            (hq > 1 and qh != d) or (hkv > 1 and (kh != d or vh != d)):
        raise ValueError(f"q, k and v (on {q.device}, {k.device}, {v.device}; strides {q.stride()}, {k.stride()}, "
                         f"{v.stride()}) must lie on the current CUDA device with the heads of a token contiguous")
    axes, stride = 1, n
    if positions.dim() == 2:
        axes = positions.shape[0]
        if axes > 1:
            stride = positions.stride(0)
    if positions.dtype is not i32 or positions.get_device() != dev or positions.dim() > 2 or \
            positions.shape[-1] != n or (n > 1 and positions.stride(-1) != 1):
        raise ValueError(f"positions {tuple(positions.shape)} of {positions.dtype} on {positions.device} is not an int32 "
                         f"[{n}] or [axes, {n}] device tensor with contiguous rows")
    limit, rot = cos_sin.shape
    pages, ps, heads, cd = cshape
    if layout == LAYOUT_HND:
        ps, heads = heads, ps
    if heads != hkv or cd != d or v_cache.shape != cshape:
        raise ValueError(f"k_cache {tuple(k_cache.shape)} and v_cache {tuple(v_cache.shape)} do not hold {hkv} heads of "
                         f"{d} in layout {kv_layout}")
    kt, qt = k_cache.dtype, q_out.dtype
    # (the shapes of these four are known by now)
    for t, name, dtype in ((cos_sin, "cos_sin", T.float32), (q_out, "q_out", qt), (k_cache, "k_cache", kt),
                           (v_cache, "v_cache", kt)):
        if t.get_device() != dev or t.dtype is not dtype or not t.is_contiguous():
            _refuse(t, name, dtype, dev)
    _check(lib().pafp8_norm_rope_append(_ROPE.pack(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _addr(q_weight, "q_weight", d, dt, dev),
        _addr(k_weight, "k_weight", d, dt, dev), cos_sin.data_ptr(), positions.data_ptr(),
        _addr(pair_axis, "pair_axis", rot // 2, T.uint8, dev), _addr(slots, "slots", n, T.int64, dev), q_out.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), _addr(status, "status", 1, i32, dev), n, qs, ks, vs, stride, dtype_code(dt),
        dtype_code(qt), dtype_code(kt), layout, hq, hkv, d, rot, 1 if interleaved else 0, axes, limit, pages, ps, eps,
        q_scale, k_scale, v_scale), _stream_on(dev, stream)))


class StepTables:
    """Owns the device arrays that pafp8_build_tables fills for a step of up
    to `batch` requests, `max_pages` pages and `max_tokens` new tokens:
    kv_indptr, last_page_len, kv_indices, qo_indptr, batch_indices, positions,
    slots, free_used, and, with mask_words > 0, rope_positions and tree_mask
    (int32 words).  The arrays keep their addresses, so a step that uses them
    can be captured into a graph; they cannot be replaced by others."""

    def __init__(self, *, batch: int, max_pages: int, max_tokens: int, page_size: int, num_pages: int,
                 mask_words: int = 0, device="cuda"):
        import torch
        def ints(*shape, dtype=torch.int32):
            return torch.zeros(shape, dtype=dtype, device=device)

        own = dict(free_used=ints(1), kv_indptr=ints(batch + 1), last_page_len=ints(batch), kv_indices=ints(max_pages),
                   qo_indptr=ints(batch + 1), batch_indices=ints(max_tokens), positions=ints(max_tokens),
                   slots=ints(max_tokens, dtype=torch.int64))
        tree = dict(rope_positions=ints(max_tokens) if mask_words > 0 else None,
                    tree_mask=ints(max_tokens, mask_words) if mask_words > 0 else None, status=ints(1))
        addresses = [tuple(0 if t is None else t.data_ptr() for t in d.values()) for d in (own, tree)]
        self.__dict__.update(own, **tree, page_size=int(page_size), num_pages=int(num_pages), _batch=batch,
                             _dev=own["slots"].get_device(), _addresses=addresses,
                             _sizes=(int(max_pages), int(max_tokens), max(0, int(mask_words))))

    def __setattr__(self, name, value):
        raise AttributeError(f"{name}: a StepTables keeps the arrays that it was made with")

    def build(self, cached_lens, new_lens, block_table, free_pages, free_used, *, parents=None, stream=None) -> None:
        """Fill the arrays (and block_table's new entries) for these lengths;
        self.free_used holds the free list's entries taken after the step."""
        dev = _device_of(cached_lens, "cached_lens")
        if dev != self._dev:
            _refuse(self.slots, "this StepTables", self.slots.dtype, dev)
        if cached_lens.numel() > self._batch:
            raise ValueError(f"{cached_lens.numel()} requests in a StepTables made for {self._batch}")
        _build_tables(dev, cached_lens, new_lens, block_table, free_pages, free_used, parents, *self._addresses,
                      *self._sizes, self.page_size, self.num_pages, stream)


# ---- convenience owner of a plan ---------------------------------------

class Plan:
    """Owns one pafp8_plan.  Shapes served: head_dim 128 or 64,
    page_size a multiple of 16 in either layout."""

    def __init__(self, *, mode: str, num_qo_heads: int, num_kv_heads: int, num_pages: int,
                 kv_indptr, last_page_len, qo_indptr=None, q_dtype, kv_dtype, o_dtype=None,
                 head_dim: int = 128, page_size: int = 16, sm_scale: float = 0.0,
                 fixed_split_pages: int = 0, disable_split_kv: bool = False, num_ctas: int = 0,
                 kv_layout: str = "NHD"):
        kv_indptr_h = _i32_host(kv_indptr)
        self.desc = plan_desc(
            mode=_MODES.get(mode, MODE_PREFILL), batch=len(kv_indptr_h) - 1,
            num_qo_heads=num_qo_heads, num_kv_heads=num_kv_heads, head_dim=head_dim,
            page_size=page_size, num_pages=num_pages, q_dtype=dtype_code(q_dtype),
            kv_dtype=dtype_code(kv_dtype),
            o_dtype=DTYPE_DEFAULT if o_dtype is None else dtype_code(o_dtype),
            sm_scale=float(sm_scale), fixed_split_pages=int(fixed_split_pages),
            disable_split_kv=int(bool(disable_split_kv)), num_ctas=int(num_ctas),
            kv_layout=_LAYOUTS[kv_layout] if isinstance(kv_layout, str) else int(kv_layout))
        self.handle = None
        self.handle = pafp8_plan_create(self.desc, kv_indptr_h, last_page_len, qo_indptr)

    def __del__(self):
        if getattr(self, "handle", None):
            pafp8_plan_destroy(self.handle)
            self.handle = None

    @property
    def workspace_bytes(self) -> int:
        return pafp8_workspace_bytes(self.handle)

    def metadata(self) -> np.ndarray:
        return pafp8_plan_metadata(self.handle)

    def upload(self, workspace, stream=None) -> None:
        pafp8_plan_upload(self.handle, workspace, stream)

    def run(self, q, k_cache, v_cache, kv_indices, o, lse, workspace, **kw) -> None:
        pafp8_run(self.handle, q, k_cache, v_cache, kv_indices, o, lse, workspace, **kw)

    def host_workspace_bytes(self, q_dtype) -> int:
        return pafp8_host_workspace_bytes(self.handle, q_dtype)

    def run_host(self, q_h, k_cache, v_cache, kv_indices_h, o_h, lse_h, workspace, **kw) -> None:
        pafp8_run_host(self.handle, q_h, k_cache, v_cache, kv_indices_h, o_h, lse_h, workspace, **kw)

    def run_head_scales(self, q, k_cache, v_cache, kv_indices, o, lse, workspace, **kw) -> None:
        pafp8_run_head_scales(self.handle, q, k_cache, v_cache, kv_indices, o, lse, workspace, **kw)

    def run_tree(self, q, k_cache, v_cache, kv_indices, tree_mask, o, lse, workspace, **kw) -> None:
        pafp8_run_tree(self.handle, q, k_cache, v_cache, kv_indices, tree_mask, o, lse, workspace, **kw)

    def run_stage(self, stage, q, k_cache, v_cache, kv_indices, o, lse, workspace, **kw) -> None:
        pafp8_run_stage(self.handle, stage, q, k_cache, v_cache, kv_indices, o, lse, workspace, **kw)

    def device_status(self, workspace, stream=None) -> None:
        pafp8_device_status(self.handle, workspace, stream)
