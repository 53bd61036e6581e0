"""What pafp8_run_tree refuses before it passes addresses on: arrays of another
type or too few elements would be read or written out of range (no GPU needed:
the library call is recorded, the device is the CPU's ordinal)."""
import numpy as np
import pytest
import torch

import paged_attention_fp8_gb300 as pa

HQ, HKV, D, PAGES, NNZ, POOL = 8, 2, 128, 5, 7, 6


@pytest.fixture
def call(monkeypatch):
    plan = pa.Plan(mode="tree", num_qo_heads=HQ, num_kv_heads=HKV, num_pages=POOL, kv_indptr=[0, 3, PAGES], last_page_len=[5, 16],
                   qo_indptr=[0, 4, NNZ], q_dtype="e4m3fn", kv_dtype="e4m3fn", num_ctas=8)
    calls = []

    class Recorder:
        @staticmethod
        def pafp8_run_tree(*a):
            calls.append(a)
            return 0

        def __getattr__(self, name):
            return getattr(real, name)

    real, recorder = pa.lib(), Recorder()
    monkeypatch.setattr(pa, "lib", lambda: recorder)
    monkeypatch.setattr(pa, "_device_of", lambda t, name: -1)
    fp8 = dict(dtype=torch.float8_e4m3fn)
    good = dict(q=torch.zeros(NNZ, HQ, D, **fp8), k_cache=torch.zeros(POOL, 16, HKV, D, **fp8),
                v_cache=torch.zeros(POOL, 16, HKV, D, **fp8), kv_indices=torch.zeros(PAGES, dtype=torch.int32),
                tree_mask=torch.zeros(NNZ, 1, dtype=torch.int32), o=torch.zeros(NNZ, HQ, D, dtype=torch.bfloat16),
                lse=torch.zeros(NNZ, HQ), workspace=torch.zeros(plan.workspace_bytes, dtype=torch.uint8))
    scales = dict(q_scales=torch.ones(HQ), k_scales=torch.ones(HKV), v_scales=torch.ones(HKV))

    def run(head_scales=False, **kw):
        a = {**good, **(scales if head_scales else {}), **kw}
        n = len(calls)
        plan.run_tree(a.pop("q"), a.pop("k_cache"), a.pop("v_cache"), a.pop("kv_indices"), a.pop("tree_mask"), a.pop("o"),
                      a.pop("lse"), a.pop("workspace"), stream=1, **a)
        assert len(calls) == n + 1

    run.plan = plan
    return run


def test_what_fits_is_passed_on(call):
    call()
    call(head_scales=True)
    call(lse=None)
    call(head_scales=True, q_scales=None)


@pytest.mark.parametrize("kw,match", [
    (dict(kv_indices=torch.zeros(PAGES, dtype=torch.int64)), "kv_indices has dtype torch.int64"),
    (dict(kv_indices=torch.zeros(PAGES, dtype=torch.int16)), "kv_indices has dtype torch.int16"),
    (dict(kv_indices=torch.zeros(PAGES)), "kv_indices has dtype torch.float32"),
    (dict(lse=torch.zeros(NNZ, HQ, dtype=torch.float64)), "lse has dtype torch.float64"),
    (dict(lse=torch.zeros(NNZ, HQ, dtype=torch.bfloat16)), "lse has dtype torch.bfloat16"),
    (dict(head_scales=True, k_scales=torch.ones(HKV, dtype=torch.float64)), "k_scales has dtype torch.float64"),
    (dict(head_scales=True, v_scales=torch.ones(HKV, dtype=torch.float16)), "v_scales has dtype torch.float16"),
    (dict(head_scales=True, q_scales=torch.ones(HQ, dtype=torch.bfloat16)), "q_scales has dtype torch.bfloat16"),
    (dict(head_scales=True, q_scales=torch.ones(2 * HQ)[::2]), "q_scales .* not contiguous"),
    (dict(head_scales=True, k_scales=torch.ones(2 * HKV)[::2]), "k_scales .* not contiguous")])
def test_types(call, kw, match):
    with pytest.raises(ValueError, match=match):
        call(**kw)


FP8 = dict(dtype=torch.float8_e4m3fn)


@pytest.mark.parametrize("kw,match", [
    (dict(q=torch.zeros(NNZ - 1, HQ, D, **FP8)), "q "), (dict(q=torch.zeros(NNZ, HQ // 2, D, **FP8)), "q "),
    (dict(q=torch.zeros(NNZ, HQ, D // 2, **FP8)), "q "), (dict(o=torch.zeros(NNZ - 1, HQ, D, dtype=torch.bfloat16)), "o "),
    (dict(o=torch.zeros(NNZ, HQ, D, dtype=torch.uint8), o_dtype="bf16"), "o "),
    (dict(lse=torch.zeros(NNZ - 1, HQ)), "lse "), (dict(lse=torch.zeros(NNZ)), "lse "),
    (dict(kv_indices=torch.zeros(PAGES - 1, dtype=torch.int32)), "kv_indices "),
    (dict(k_cache=torch.zeros(POOL - 1, 16, HKV, D, **FP8)), "k_cache "),
    (dict(v_cache=torch.zeros(POOL - 1, 16, HKV, D, **FP8)), "v_cache "),
    (dict(v_cache=torch.zeros(POOL * 16 * HKV * D - 1, **FP8)), "v_cache "),
    (dict(k_cache=torch.zeros(POOL, HKV, 16, D, **FP8)), "k_cache "),
    (dict(v_cache=torch.zeros(POOL, 32, HKV // 2, D, **FP8)), "v_cache "),
    (dict(tree_mask=torch.zeros(NNZ - 1, 1, dtype=torch.int32)), "tree_mask "),
    (dict(tree_mask=torch.zeros(NNZ - 1, 1, dtype=torch.int32), q=torch.zeros(NNZ - 1, HQ, D, **FP8)), "(tree_mask|q) "),
    (dict(head_scales=True, q_scales=torch.ones(HQ - 1)), "q_scales "), (dict(head_scales=True, k_scales=torch.ones(1)), "k_scales "),
    (dict(head_scales=True, v_scales=torch.ones(1)), "v_scales ")])
def test_sizes(call, kw, match):
    with pytest.raises(ValueError, match="^" + match):
        call(**kw)


def test_larger_arrays_are_taken(call):
    """A batch padded to more rows, a longer page list, a larger pool and wider mask rows, other shapes of as many elements."""
    call(q=torch.zeros(NNZ + 3, HQ, D, **FP8), o=torch.zeros(NNZ + 1, HQ, D, dtype=torch.bfloat16), lse=torch.zeros(NNZ + 2, HQ),
         tree_mask=torch.zeros(NNZ + 3, 2, dtype=torch.int32), kv_indices=torch.zeros(PAGES + 4, dtype=torch.int32),
         k_cache=torch.zeros(POOL + 2, 16, HKV, D, **FP8), v_cache=torch.zeros(POOL + 2, 16, HKV, D, **FP8))
    call(q=torch.zeros(NNZ, HQ * D, **FP8), o=torch.zeros(NNZ * HQ * D, dtype=torch.bfloat16), lse=torch.zeros(NNZ * HQ),
         k_cache=torch.zeros(POOL * 16 * HKV * D, **FP8), q_dtype="e4m3fn")
    call(q=torch.zeros(NNZ, HQ, D, dtype=torch.uint8), q_dtype="e4m3fn")


def test_sizes_go_with_their_plan(call):
    """A plan's handle that is destroyed takes its sizes along: the next plan may get the same address."""
    other = pa.Plan(mode="tree", num_qo_heads=2, num_kv_heads=2, num_pages=1, kv_indptr=[0, 1], last_page_len=[5], qo_indptr=[0, 2],
                    q_dtype="bf16", kv_dtype="bf16", num_ctas=8)
    handle = other.handle
    assert handle in pa._TREE_SIZES and call.plan.handle in pa._TREE_SIZES
    pa.pafp8_plan_destroy(handle)
    other.handle = None
    assert handle not in pa._TREE_SIZES
    empty = pa.Plan(mode="tree", num_qo_heads=2, num_kv_heads=2, num_pages=0, kv_indptr=[0], last_page_len=[], qo_indptr=[0],
                    q_dtype="bf16", kv_dtype="bf16", num_ctas=8)
    none = dict(dtype=torch.bfloat16)
    pa.pafp8_run_tree(empty.handle, torch.zeros(0, 2, 128, **none), torch.zeros(0, 16, 2, 128, **none), torch.zeros(0, 16, 2, 128, **none),
                      torch.zeros(0, dtype=torch.int32), torch.zeros(0, 1, dtype=torch.int32), torch.zeros(0, 2, 128, **none),
                      torch.zeros(0, 2), torch.zeros(empty.workspace_bytes, dtype=torch.uint8), stream=1)
