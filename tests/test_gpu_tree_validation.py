"""KDA_VALIDATE=1 and trees: what the calls refuse, and what they take."""
import pytest
import torch

import hybrid_prefix_cache_amd as K
from test_gpu_tree_attn import Draft, ints
from test_gpu_tree_state import Conv, States
from tree_util import tree

pytestmark = pytest.mark.gpu


def refused(status, call):
    with pytest.raises(K.KdaError) as e:
        call()
    assert e.value.status == status, e.value


@pytest.fixture
def validate(monkeypatch):
    monkeypatch.setenv("KDA_VALIDATE", "1")


@pytest.mark.parametrize("row,pos", [([-2] * 8, 32), ([-1] + [-2] * 7, 28), ([-2] * 8, 30)])
def test_append_writes_the_slots_behind_the_last_node(validate, row, pos):
    """A request that drafted little or nothing, whose next page is another request's: refused before
    anything is enqueued; with no page there, or one of its own, it is taken."""
    x = Draft([40, pos], [tree("chain", 8), row], 1, 2, 64, 32, "int8", "bf16")
    call = lambda t: K.kda_kv_append_tree(x.f.kb.pool, None, x.k, x.v, None, x.parent, x.pos, t)
    table, before = x.f.table.clone(), x.f.kb.buf.clone()
    table[1, 1] = table[0, 1]
    refused(K.KDA_ERR_PAGE_ALIAS, lambda: call(table))
    torch.cuda.synchronize()
    assert torch.equal(before, x.f.kb.buf)
    table[1, 1] = -1
    call(table)
    call(table[:, :2].contiguous())
    call(x.f.table)


@pytest.mark.parametrize("path,count", [([2, 1, 0, 0, 0], 2), ([1, 1, 0, 0, 0], 2), ([0, 5, 0, 0, 0], 2), ([-1, 1, 0, 0, 0], 1),
                                        ([0, 1, 2, 3, 4], 6), ([0, 0, 0, 0, 0], -1)])
def test_commits_refuse_bad_paths(validate, path, count):
    """In every layer kind, the bad path a later request's."""
    trees = [tree("binary", 5)] * 2
    path, count = ints([[0, 1, 3, -9, -9], path]), ints([3, count])
    x, c = States(trees, 1, 64, "bf16"), Conv(trees, 64, 4, "bf16")
    before, a, pages = (x.pb.buf.clone(), c.buf.clone()), x.x, ints([0, 1])
    d = Draft([40, 60], trees, 1, 2, 64, 32, "int8", "bf16")
    calls = (lambda p, m: K.kda_decode_commit(x.pb.pool, a["k"], a["v"], a["g"], a["beta"], p, m, pages, pages),
             lambda p, m: K.kda_short_conv_commit(c.pool, c.x, p, m, pages, pages),
             lambda p, m: K.kda_kv_commit(d.f.kb.pool, p, m, d.pos, d.f.table))
    for call in calls:
        refused(K.KDA_ERR_SEQ, lambda: call(path, count))
    torch.cuda.synchronize()
    assert torch.equal(before[0], x.pb.buf) and torch.equal(before[1], c.buf)
    for call in calls:  # what is behind a path's end is not read
        call(ints([[0, 1, 3, -9, -9], [4, 2, 9, 9, 9]]), ints([3, 1]))


@pytest.mark.parametrize("cache", ["int8", "bf16"])
def test_commit_needs_the_pages_of_its_path_alone(validate, cache):
    """Slots 30, 70 of pages of 32 tokens: the page between is not touched, and need not be there; the other
    two are needed, and the one that receives the rows is no other request's."""
    row = [-1] + [-2] * 39 + [0]
    x = Draft([30, 10], [row] * 2, 2, 2, 64, 32, cache, "bf16")
    x.append()
    path, count = ints([[0, 40] + [-1] * 39, [0, 40] + [-1] * 39]), ints([2, 0])
    call = lambda t: K.kda_kv_commit(x.f.kb.pool, path, count, x.pos, t)
    table = x.f.table.clone()
    for j in (0, 2):
        table[0, j] = -1
        refused(K.KDA_ERR_PAGE_RANGE, lambda: call(table))
        table[0, j] = x.f.table[0, j]
    refused(K.KDA_ERR_PAGE_RANGE, lambda: call(table[:, :2].contiguous()))
    count[1] = 2
    table[1, 0] = table[0, 0]
    refused(K.KDA_ERR_PAGE_ALIAS, lambda: call(table))
    count[1] = 0
    start = x.f.kb.buf.clone()
    call(x.f.table)
    want = x.f.kb.buf.clone()
    assert not torch.equal(start, want)
    x.f.kb.buf.copy_(start)
    table[0, 1] = -1
    call(table)
    assert torch.equal(x.f.kb.buf, want)
