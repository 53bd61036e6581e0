"""The longest requests a tree plan takes (no GPU needed)."""
import numpy as np
import pytest

import paged_attention_fp8_gb300 as pa

SEG = 12
LONGEST = (1 << 31) - 1 - 128  # the end of a request's last 128-key tile is an int


def _plan(kv_len, page_size=1 << 20):
    pages = -(-kv_len // page_size)
    return pa.Plan(mode="tree", num_qo_heads=4, num_kv_heads=1, num_pages=1, kv_indptr=[0, pages],
                   last_page_len=[kv_len - (pages - 1) * page_size], qo_indptr=[0, 3], q_dtype="bf16", kv_dtype="e4m3fn",
                   page_size=page_size, num_ctas=8)


@pytest.mark.parametrize("kv_len", [1 << 30, LONGEST])
def test_long_requests_keep_their_lengths(kv_len):
    m = _plan(kv_len).metadata()
    segs = m[int(m[13]):int(m[13]) + SEG * int(m[7])].reshape(-1, SEG)
    assert (segs[:, 7] == kv_len).all()
    assert segs[0, 2] == 0 and (segs[1:, 2] == segs[:-1, 3]).all() and segs[-1, 3] == -(-kv_len // 128)


@pytest.mark.parametrize("kv_len", [LONGEST + 1, (1 << 31) + 5, (1 << 32) + 77, 1 << 36])
def test_longer_ones_are_refused(kv_len):
    with pytest.raises(pa.Pafp8Error) as e:
        _plan(kv_len)
    assert e.value.status == 8 and f"kv_len {kv_len}" in str(e.value)
