"""Packed steps without tokens (GPU)."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    import torch
    __graft_entry__.build()
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def _status():
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    torch.cuda.synchronize()
    return T.get_device_status(clear=True)


@pytest.mark.parametrize("which", ["slots", "positions", "both"])
def test_maps_without_room(dev, which):
    """Maps of no tokens are maps all the same: a step that has tokens does not fit them, one that gives pages back does."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    _status()
    cache = T.PagedCache(*(torch.zeros((8, 1, 16, 64), dtype=torch.bfloat16, device=dev) for _ in range(2)))
    tables = T.alloc_page_tables(cache, 2, 4)

    def ints(*x):
        return torch.tensor(x, dtype=torch.int32, device=dev)
    lens, starts, none = ints(0, 0), ints(0, 0, 0), ints()
    maps = {name: none for name in ("slots", "positions") if which in (name, "both")}
    T.paged_reserve(tables, ints(0, 0), ints(20, 3), lens, starts, **maps)
    assert _status() == T.DEVICE_BAD_KV_LEN
    assert int(tables.missing) == -1 and lens.tolist() == [0, 0] and starts.tolist() == [0, 0, 0]
    assert tables.held.tolist() == [0, 0] and int(tables.n_free) == 8
    T.paged_reserve(tables, ints(0, 0), ints(20, 3), lens, starts)             # no maps at all
    assert int(tables.missing) == 0 and lens.tolist() == [20, 3] and tables.held.tolist() == [2, 1]
    T.paged_reserve(tables, ints(0, 3), ints(0, 0), lens, starts, **maps)
    assert int(tables.missing) == 0 and lens.tolist() == [0, 3] and tables.held.tolist() == [0, 1]
    assert _status() == 0


@pytest.mark.parametrize("dim,dtype,batch,tokens,heads,group", [(128, "bf16", 3, 5, 2, 4), (64, "fp16", 40, 3, 1, 1),
                                                                (64, "bf16", 2, 20000, 8, 4)])
def test_attention_of_empty_sequences(dev, dim, dtype, batch, tokens, heads, group):
    """No sequence has a row: nothing is written.  With keys alone, dk and dv are 0."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step
    _status()
    step = Step(dev, dtype, dim, heads, group, [0] * batch, gap=tokens)
    out, lse = step.forward(T)
    assert (out == 7).all() and (lse == 7).all()
    assert all((g == 7).all() for g in step.backward(T, out, lse))
    step = Step(dev, dtype, dim, heads, group, [0] * batch, [tokens] + [0] * (batch - 1))
    out, lse = step.forward(T)
    assert (out == 7).all() and (lse == 7).all()
    dq, dk, dv = step.backward(T, out, lse)
    assert (dq == 7).all()
    for g in (dk, dv):
        assert (g[:tokens] == 0).all() and (g[tokens:] == 7).all()
    assert _status() == 0
