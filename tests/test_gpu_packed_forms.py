"""Packed attention in the forms that only large or lopsided calls take (GPU).

Which form a call takes goes by its sizes: how many CTAs share a unit's keys in
the forward pass, and a tile of keys' rows in the gradient.
"""

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


@pytest.fixture(autouse=True)
def _clean_status(dev):
    import trainable_block_sparse_infllm_gb300 as T
    T.get_device_status(clear=True)
    yield


def _both(step):
    """Output, log sum and gradients against the 64-bit forms."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from gradient_helpers import close, gradients
    from packed_helpers import check, plain
    out, lse = step.forward(T)
    want = plain(step, with_grads=False)
    check("out", out, want)
    check("lse", lse, want)
    wanted = gradients(step)
    for name, got in zip(("dq", "dk", "dv"), step.backward(T, out, lse)):
        close(name, got, wanted)
        assert (got[torch.isnan(wanted[name][0])] == 7.0).all()      # rows of no sequence
    torch.cuda.synchronize()
    assert T.get_device_status(clear=True) == 0


@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (64, "fp16")])
@pytest.mark.parametrize("heads,group,queries", [(1, 16, 9), (2, 4, 33), (5, 16, 7), (8, 32, 5), (9, 7, 3), (12, 1, 1),
                                                 (16, 16, 12), (30, 2, 2)])
def test_few_queries_after_many_keys(dev, dim, dtype, heads, group, queries):
    """One unit per head, its 71 tiles of keys over clusters of up to 16 CTAs."""
    from packed_helpers import Step
    _both(Step(dev, dtype, dim, heads, group, [queries], [9000]))


@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (128, "fp16"), (64, "bf16"), (64, "fp16")])
@pytest.mark.parametrize("group,lens", [(8, [1200]), (7, [1337]), (16, [1000, 200]), (32, [129])])
def test_rows_of_few_tiles_of_keys(dev, dim, dtype, group, lens):
    """dk and dv of a tile of keys by clusters of 8 (the first two) and of 4."""
    from packed_helpers import Step
    _both(Step(dev, dtype, dim, 1, group, lens))


@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (64, "fp16")])
@pytest.mark.parametrize("group", [16, 32])
def test_rows_of_few_tiles_of_many_sequences(dev, dim, dtype, group):
    """More than 32 sequences whose tiles of keys take clusters of 2 and 4."""
    from packed_helpers import Step
    lens = [128 + (37 * i) % 64 - 32 for i in range(40)]
    lens[17], lens[33] = 0, 1
    _both(Step(dev, dtype, dim, 1, group, lens))


@pytest.mark.parametrize("dim,dtype,heads,group,layout", [(128, "bf16", 1, 2, "fused"), (64, "fp16", 2, 3, "heads")])
def test_thousands_of_queries(dev, dim, dtype, heads, group, layout):
    from packed_helpers import Step
    _both(Step(dev, dtype, dim, heads, group, [5000, 777, 2048], layout=layout))


@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (64, "fp16")])
def test_a_chunk_after_many_keys(dev, dim, dtype):
    from packed_helpers import Step
    _both(Step(dev, dtype, dim, 2, 4, [500, 1, 90], [7000, 5000, 90]))
