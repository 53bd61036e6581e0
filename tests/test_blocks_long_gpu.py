"""Long appends and read-backs over block scales, whose warps and thread blocks take several rows in turn, against the
definition in numpy, number for number.  (A warp of the append looks through 1, 2, 4, 8 or 16 new tokens for its blocks, more
the longer the call; a thread block of the read-back takes 2, 4, 8 or 16 rows.)"""
import numpy as np
import pytest
import torch

import paged_attention_fp8_gb300 as pa
from blocks_ref import TORCH, raw
from test_blocks_append_gpu import Setup, ints, read_ref

pytestmark = pytest.mark.gpu


def lengths(kind, rows, gen):
    """(cached, new): positions with block borders anywhere."""
    if kind == "two":  # two prompts with a request of no tokens between them
        new = [rows // 3 + 1, 0, rows - rows // 3 - 1]
    elif kind == "ragged":  # prompts of 1 to 400 tokens
        new = []
        while sum(new) < rows:
            new.append(min(int(gen.integers(1, 401)), rows - sum(new)))
    else:  # requests of 16 to 40 tokens: two or three blocks each
        new = [int(x) for x in gen.integers(16, 41, rows // 28)]
    return [int(x) for x in gen.integers(0, 50, len(new))], new


# Rows times heads: from 2000 to 150000 pairs of K and V rows, so that every count of tokens a warp looks through comes up for
# rows of either size (fp32 rows: fewer warps an SM).
@pytest.mark.parametrize("kind,rows,heads,d,fmt,layout,page_size", [
    ("two", 501, 4, 128, "e4m3fn", "NHD", 16), ("two", 4003, 3, 64, "e5m2", "HND", 48), ("two", 9001, 8, 128, "e4m3fn", "NHD", 32),
    ("ragged", 1501, 5, 64, "e4m3fn", "NHD", 16), ("ragged", 5003, 4, 128, "e5m2", "HND", 32),
    ("ragged", 12001, 8, 128, "e4m3fn", "HND", 16), ("many", 2001, 4, 128, "e4m3fn", "NHD", 16),
    ("many", 9000, 7, 64, "e4m3fn", "NHD", 64), ("many", 9000, 8, 128, "e5m2", "NHD", 16)])
@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
def test_long_append(cuda_device, kind, rows, heads, d, fmt, layout, page_size, src):
    cached, new = lengths(kind, rows, np.random.default_rng(rows + heads))
    s = Setup([c + n for c, n in zip(cached, new)], heads=heads, d=d, fmt=fmt, layout=layout, page_size=page_size)
    qo = np.concatenate([[0], np.cumsum(new)])
    k, v = s.rows(int(qo[-1]) + 3, src, packed=kind == "two")
    k[qo[-1]:], v[qo[-1]:] = float("nan"), float("nan")  # padding behind the last request
    s.append(k, v, ints(qo), ints(cached))
    s.expect(k, v, qo, cached)
    s.check()


@pytest.mark.parametrize("rows", [1205, 2433, 4999, 9733, 20011])
@pytest.mark.parametrize("heads,d,fmt,layout,page_size,out", [
    (3, 128, "e4m3fn", "NHD", 16, "bf16"), (2, 64, "e5m2", "HND", 48, "f32"), (1, 64, "e4m3fn", "HND", 16, "f16")])
def test_long_read_back(cuda_device, rows, heads, d, fmt, layout, page_size, out):
    gen = np.random.default_rng(rows)
    for kind in ("two", "ragged", "many"):
        starts, counts = lengths(kind, rows, gen)
        s = Setup([a + n for a, n in zip(starts, counts)], heads=heads, d=d, fmt=fmt, layout=layout, page_size=page_size)
        n = sum(counts)
        ko, vo = (torch.full((n + 5, heads, d), 7.0, dtype=TORCH[out], device="cuda") for _ in range(2))
        pa.pafp8_read_kv(s.k, s.v, ints(np.concatenate([[0], np.cumsum(counts)])), ints(starts), s.ptr_d, s.ids_d, ko, vo,
                         k_scales=s.ks, v_scales=s.vs, kv_layout=layout, status=s.status)
        assert int(s.status) == 0
        for got, name in ((ko, "k"), (vo, "v")):
            assert torch.equal(raw(got[:n].cpu()), raw(read_ref(s, name, starts, counts).to(TORCH[out])))
            assert bool((got[n:] == 7).all())
