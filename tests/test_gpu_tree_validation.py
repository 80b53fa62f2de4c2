"""KDA_VALIDATE=1 and trees: what the calls refuse, and what they take."""
import pytest
import torch

import hybrid_prefix_cache_amd as K
from test_gpu_tree_attn import Draft, ints
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
