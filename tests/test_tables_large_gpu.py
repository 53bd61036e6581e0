"""pafp8_build_tables at the largest sizes it takes."""
import pytest
import torch

import paged_attention_fp8_gb300 as pa

pytestmark = pytest.mark.gpu


def test_nearly_2_31_new_tokens(cuda_device):
    """One request as long as the lengths allow: indexes run up to INT32_MAX and no further."""
    ps, tokens, most = 16, (1 << 31) - 1 - 16, (1 << 31) - 1
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    pages = -(-tokens // ps)
    i = dict(dtype=torch.int32, device="cuda")
    t = pa.StepTables(batch=1, max_pages=pages, max_tokens=most, page_size=ps, num_pages=pages + 1)
    free = torch.arange(pages, -1, -1, **i)  # page j is pages - j
    t.build(torch.zeros(1, **i), torch.tensor([tokens], **i), torch.zeros(1, pages, **i), free, torch.zeros(1, **i))
    assert int(t.status) == 0
    assert t.kv_indptr.tolist() == [0, pages] and t.qo_indptr.tolist() == [0, tokens] and t.free_used.tolist() == [pages]
    assert t.last_page_len.tolist() == [tokens - (pages - 1) * ps]
    assert torch.equal(t.kv_indices, free[:pages])
    chunk = 1 << 28
    for a in range(0, tokens, chunk):
        b = min(a + chunk, tokens)
        pos = torch.arange(a, b, **i)
        assert torch.equal(t.positions[a:b], pos) and not bool(t.batch_indices[a:b].any())
        assert torch.equal(t.slots[a:b], (pages - pos.div(ps, rounding_mode="floor")).long() * ps + pos % ps)
    assert bool((t.slots[tokens:] == -1).all()) and bool((t.batch_indices[tokens:] == -1).all())
    del t, free, pos
    torch.cuda.empty_cache()  # 36 GB that no other test needs
