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
