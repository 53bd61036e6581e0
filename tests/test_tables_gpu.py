"""pafp8_build_tables against a plain restatement: every output is a whole
number and has to be equal."""
import numpy as np
import pytest
import torch

import paged_attention_fp8_gb300 as pa
from step_ref import tables as ref_tables

pytestmark = pytest.mark.gpu


def _case(seed, batch, top, new_top, page_size, *, spare=7, tree=True):
    r = np.random.default_rng(seed)
    cached = r.integers(0, top + 1, batch)
    new = r.integers(0, new_top + 1, batch)
    have, total = -(-cached // page_size), -(-(cached + new) // page_size)
    pool = int(total.sum()) + spare
    perm = r.permutation(pool)
    table = np.full((batch, int(total.max(initial=0)) + 2), -1, np.int32)
    at = 0
    for b in range(batch):
        table[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    parents = None
    if tree:
        parents = np.concatenate([[r.integers(-1, u) if u else -1 for u in range(n)] for n in new] + [[]]).astype(np.int32)
    return dict(cached=cached, new=new, table=table, free=np.concatenate([[3, 1, 2], perm[at:]]).astype(np.int32), used=3,
                pool=pool, pages=int(total.sum()), tokens=int(new.sum()), parents=parents)


def _run(c, page_size, words, *, max_pages=None, max_tokens=None, free=None, pad=0):
    dev = "cuda"
    max_pages = c["pages"] if max_pages is None else max_pages
    max_tokens = c["tokens"] + pad if max_tokens is None else max_tokens
    t = pa.StepTables(batch=len(c["cached"]), max_pages=max_pages, max_tokens=max_tokens, page_size=page_size,
                      num_pages=c["pool"], mask_words=words, device=dev)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)  # noqa: E731
    table = i32(c["table"])
    parents = None
    if c["parents"] is not None:
        parents = torch.full((max_tokens,), -1, dtype=torch.int32, device=dev)
        m = min(max_tokens, len(c["parents"]))
        parents[:m] = i32(c["parents"])[:m]
    args = (i32(c["cached"]), i32(c["new"]), table, i32(c["free"] if free is None else free), i32([c["used"]]))
    t.build(*args, parents=parents)
    return t, table, args, parents


def _check(t, table, want, words):
    got = dict(kv_indptr=t.kv_indptr, qo_indptr=t.qo_indptr, last_page_len=t.last_page_len, kv_indices=t.kv_indices,
               batch_indices=t.batch_indices, positions=t.positions, slots=t.slots, free_used=t.free_used, block_table=table)
    if words:
        got["rope_positions"] = t.rope_positions
        got["tree_mask"] = t.tree_mask
    for name, g in got.items():
        w = np.asarray(want[name]).astype(np.int64)
        g = g.cpu().numpy().astype(np.int64)
        if name == "tree_mask":
            g = g & 0xFFFFFFFF
        assert np.array_equal(g, w), f"{name}: {g.ravel()[:20]} != {w.ravel()[:20]}"


@pytest.mark.parametrize("batch,top,new_top,page_size,words,tree", [
    (1, 0, 1, 16, 1, True), (1, 1000, 1, 16, 0, False), (1, 5000, 3000, 16, 0, False), (3, 40, 0, 16, 1, True),
    (8, 64, 17, 16, 1, True), (9, 300, 33, 32, 2, True), (64, 4096, 16, 16, 1, True), (65, 700, 70, 48, 3, True),
    (257, 2000, 5, 64, 1, False), (1500, 90, 3, 16, 1, True), (2, 20, 400, 16, 13, True)])
def test_tables_equal_the_restatement(cuda_device, batch, top, new_top, page_size, words, tree):
    c = _case(17 * batch + top, batch, top, new_top, page_size, tree=tree)
    t, table, args, parents = _run(c, page_size, words, pad=70)
    want, bad = ref_tables(c["cached"], c["new"], c["table"], c["free"], c["used"], page_size=page_size,
                           num_pages=c["pool"], max_pages=c["pages"], max_tokens=c["tokens"] + 70, parents=c["parents"],
                           words=words)
    _check(t, table, want, words)
    assert not bad and int(t.status) == 0
    t.build(*args, parents=parents)  # the same step again writes the same
    _check(t, table, want, words)


def test_empty_batch(cuda_device):
    t = pa.StepTables(batch=0, max_pages=4, max_tokens=5, page_size=16, num_pages=4, mask_words=1)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    t.slots.fill_(9)
    t.build(none, none, none.view(0, 1)[:, :1], none, torch.tensor([0], dtype=torch.int32, device="cuda"))
    assert t.kv_indptr.tolist() == [0] and t.qo_indptr.tolist() == [0] and t.slots.tolist() == [-1] * 5


@pytest.mark.parametrize("what", ["free list", "pages", "tokens", "page id", "width"])
def test_what_has_no_room_is_reported_and_not_written(cuda_device, what):
    c = _case(5, 9, 200, 40, 16)
    max_pages, max_tokens, free = c["pages"], c["tokens"], c["free"]
    if what == "free list":
        free = c["free"][:c["used"] + 2]  # one page short
    elif what == "pages":
        max_pages -= 5
    elif what == "tokens":
        max_tokens -= 7
    elif what == "page id":
        c["table"][int(np.argmax(c["cached"])), 0] = c["pool"]
    else:
        c["table"] = c["table"][:, :c["table"].shape[1] - 4].copy()
    t, table, _, _ = _run(c, 16, 2, max_pages=max_pages, max_tokens=max_tokens, free=free)
    want, bad = ref_tables(c["cached"], c["new"], c["table"], free, c["used"], page_size=16, num_pages=c["pool"],
                           max_pages=max_pages, max_tokens=max_tokens, parents=c["parents"], words=2)
    assert bad and int(t.status) == 1
    _check(t, table, want, 2)


@pytest.mark.parametrize("parent", [4, 9, -2])
def test_parent_that_is_not_before_its_token_counts_as_a_root(cuda_device, parent):
    c = _case(3, 1, 30, 0, 16)
    c.update(new=np.array([6]), tokens=6, pages=c["pages"] + 2, parents=np.array([-1, 0, 1, 1, parent, 4], np.int32))
    t, table, _, _ = _run(c, 16, 1)
    want, bad = ref_tables(c["cached"], c["new"], c["table"], c["free"], c["used"], page_size=16, num_pages=c["pool"],
                           max_pages=c["pages"], max_tokens=6, parents=c["parents"], words=1)
    assert bad and int(t.status) == 1
    _check(t, table, want, 1)


def test_negative_length_counts_as_zero(cuda_device):
    c = _case(11, 4, 60, 5, 16)
    good = dict(c, cached=c["cached"].copy(), new=c["new"].copy())
    c["cached"][2] = -3
    good["cached"][2] = good["new"][2] = 0
    good["parents"] = None
    c["parents"] = None
    t, table, _, _ = _run(c, 16, 1)
    want, _ = ref_tables(good["cached"], good["new"], c["table"], c["free"], c["used"], page_size=16, num_pages=c["pool"],
                         max_pages=c["pages"], max_tokens=c["tokens"], words=1)
    assert int(t.status) == 1
    _check(t, table, want, 1)


def test_row_stride_and_graph_replay_with_new_lengths(cuda_device):
    """The block table as a column slice of a wider one, captured; a replay
    after the lengths changed in place gives the new step's tables."""
    c, d = _case(21, 12, 300, 9, 16), _case(22, 12, 300, 9, 16)
    width = max(c["table"].shape[1], d["table"].shape[1])
    dev = "cuda"
    wide = torch.full((12, width + 5), -7, dtype=torch.int32, device=dev)
    table = wide[:, :width]
    cached, new = torch.zeros(12, dtype=torch.int32, device=dev), torch.zeros(12, dtype=torch.int32, device=dev)
    free = torch.zeros(max(len(c["free"]), len(d["free"])), dtype=torch.int32, device=dev)
    used = torch.tensor([3], dtype=torch.int32, device=dev)
    pages, tokens = max(c["pages"], d["pages"]), max(c["tokens"], d["tokens"])
    t = pa.StepTables(batch=12, max_pages=pages, max_tokens=tokens, page_size=16, num_pages=max(c["pool"], d["pool"]))
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        t.build(cached, new, table, free, used)
    for x in (c, d):
        full = np.full((12, width), -1, np.int32)
        full[:, :x["table"].shape[1]] = x["table"]
        table.copy_(torch.tensor(full))
        cached.copy_(torch.tensor(x["cached"], dtype=torch.int32))
        new.copy_(torch.tensor(x["new"], dtype=torch.int32))
        free[:len(x["free"])] = torch.tensor(x["free"], device=dev)
        t.kv_indices.zero_()
        graph.replay()
        want, _ = ref_tables(x["cached"], x["new"], full, free.cpu().numpy(), 3, page_size=16, num_pages=t.num_pages,
                             max_pages=pages, max_tokens=tokens)
        _check(t, table, want, 0)
    assert bool((wide[:, width:] == -7).all())


def test_more_requests_than_made_for_are_refused():
    t = pa.StepTables(batch=2, max_pages=8, max_tokens=8, page_size=16, num_pages=8)
    i = dict(dtype=torch.int32, device="cuda")
    three = torch.ones(3, **i)
    with pytest.raises(ValueError, match="3 requests"):
        t.build(three, three, torch.zeros(3, 1, **i), torch.zeros(8, **i), torch.zeros(1, **i))
