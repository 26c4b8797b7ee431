"""The gradient of packed attention where its inputs are unlike each other (GPU).

tests/gradient_helpers.py derives how far off norms over many rows may be.
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


def _status():
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    torch.cuda.synchronize()
    return T.get_device_status(clear=True)


def _close(step, rows=slice(None)):
    """Forward and gradient of `step`, whose dq is looked at over `rows`, dk and dv over all."""
    import trainable_block_sparse_infllm_gb300 as T
    from gradient_helpers import close, gradients
    out, lse = step.forward(T)
    grads = step.backward(T, out, lse)
    want = gradients(step)
    for name, got in zip(("dq", "dk", "dv"), grads):
        close(name, got, want, rows if name == "dq" else slice(None))
    return grads, want


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3, 1e-4])
def test_small_upstream_gradients(dev, dim, dtype, size):
    """A mean over tokens makes every value of dout small."""
    from packed_helpers import Step
    step = Step(dev, dtype, dim, 1, 2, [3000, 40, 900])
    step.dout *= size
    _close(step)
    assert _status() == 0


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_large_upstream_gradients(dev, dim, dtype):
    """dS far beyond fp16's largest number; dq and dk stay below it."""
    import torch
    from packed_helpers import Step
    step = Step(dev, dtype, dim, 1, 2, [3000, 40, 900])
    step.dout *= 1000
    step.v *= 50
    step.q *= 0.05
    step.k *= 0.05
    grads, _ = _close(step)
    assert all(torch.isfinite(g[:3940]).all() for g in grads)
    assert _status() == 0


@pytest.mark.parametrize("dim,dtype", [(64, "fp16"), (128, "fp16"), (128, "bf16")])
def test_upstream_gradients_of_all_sizes(dev, dim, dtype):
    """Heads and tokens whose dout differ by 10^4: dq of the small ones is as good as of the large ones."""
    import torch
    from gradient_helpers import close
    from packed_helpers import Step
    step = Step(dev, dtype, dim, 1, 8, [1800, 600])
    size = 10.0 ** -torch.randint(0, 5, step.dout.shape[:2], generator=step.gen, device=dev)
    step.dout *= size[..., None].to(step.dtype)
    grads, want = _close(step)
    for decade in range(5):
        close("dq", grads[0], want, (size - 10.0 ** -decade).abs() < 10.0 ** -decade / 2)
    assert _status() == 0


@pytest.mark.parametrize("dim", [64, 128])
def test_values_that_cancel_in_out(dev, dim):
    """fp16 rows of many keys, whose |dS| is hundreds of times |dout| |out|.

    Keys 700 .. 999 and 1000 .. 1299 are alike in all that the queries look at and their values are opposite, so
    that they cancel in out and D, but not in dq.
    """
    import torch
    from packed_helpers import Step
    step = Step(dev, "fp16", dim, 1, 4, [2100, 300])
    step.q[:2100, :, 0] = 0.0
    step.v[700:1000] *= 10000.0
    step.v[1900:2100] *= 0.1
    step.v[1000:1300] = -step.v[700:1000]
    step.k[1000:1300] = step.k[700:1000]
    step.k[700:1000, :, 0], step.k[1000:1300, :, 0] = 5.0, -5.0
    step.dout *= 0.3
    grads, _ = _close(step, slice(1300, None))
    assert torch.isfinite(grads[0][:2400]).all()
    assert _status() == 0


@pytest.mark.parametrize("dim,dtype", [(64, "fp16"), (64, "bf16"), (128, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("keys,at", [(1000, 0), (1000, 500), (1000, 940), (2000, 0), (2000, 100), (2000, 1500),
                                     (2000, 1940), (2300, 128)])
@pytest.mark.parametrize("weight", [0.5, 0.9, 0.99])
def test_heavy_keys(dev, dim, dtype, keys, at, weight):
    """One key, in the first, a middle or the last tile, has most of the weight of every row behind it."""
    from gradient_helpers import close, heavy_key
    from packed_helpers import Step
    step = Step(dev, dtype, dim, 1, 2, [30, keys])
    heavy_key(step, at, weight, seq=1)
    grads, want = _close(step, slice(30 + at + 1, None))
    close("dq", grads[0], want)
    assert _status() == 0


@pytest.mark.parametrize("dim,dtype", [(64, "fp16"), (64, "bf16"), (128, "fp16"), (128, "bf16")])
def test_keys_and_values_with_means(dev, dim, dtype):
    """D is many times dout . v - D, and dq is what is left when the keys' mean has gone."""
    from packed_helpers import Step
    step = Step(dev, dtype, dim, 2, 3, [3000, 1100, 200], [3000, 2100, 200])
    step.k += 3
    step.v += 3
    _close(step)
    assert _status() == 0


def test_units_done_once_more_among_others(dev):
    """Some sequences have heavy keys: the others' bits stay as they are, and all are the same every time."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from gradient_helpers import heavy_key
    from packed_helpers import Step
    lens = [1500 + 37 * i for i in range(12)]
    step = Step(dev, "bf16", 64, 2, 4, lens)
    out, lse = step.forward(T)
    plain = step.backward(T, out, lse)
    for seq in (0, 5, 11):
        heavy_key(step, 700, 0.97, seq)
    out, lse = step.forward(T)
    grads = step.backward(T, out, lse)
    again = step.backward(T, out, lse)
    for a, b in zip(grads, again):
        assert torch.equal(a, b)
    for seq in range(12):
        rows = slice(step.q_starts[seq], step.q_starts[seq + 1])
        for a, b in zip(grads, plain):
            assert torch.equal(a[rows], b[rows]) == (seq not in (0, 5, 11))
    assert _status() == 0


def test_more_units_than_marks(dev):
    """A CTA marks 1024 units that it does once more; with more of them some share a mark, which changes no bit."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from gradient_helpers import heavy_key
    from packed_helpers import Step
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    tiles = 1100 * sms // 4095 + 1                  # of 4 tokens with group 32
    step = Step(dev, "bf16", 64, 1, 32, [1400, *[4 * tiles] * 4095])
    heavy_key(step, 300, 0.97)
    out, lse = step.forward(T)
    grads = step.backward(T, out, lse)

    def alone(first, last, lens):
        """dq of the same rows as a batch of their own (dk and dv may be summed in another order)."""
        rows = slice(first, last)
        part = Step(dev, "bf16", 64, 1, 32, lens, gap=0)
        for name in ("q", "k", "v", "dout"):
            setattr(part, name, getattr(step, name)[rows].contiguous())
        assert torch.equal(grads[0][rows], part.backward(T, out[rows].contiguous(), lse[rows].contiguous())[0])
    alone(0, 1400, [1400])                          # its own marks
    for first in range(1400, step.q_starts[-1], 500 * 4 * tiles):
        last = min(first + 500 * 4 * tiles, step.q_starts[-1])
        alone(first, last, [4 * tiles] * ((last - first) // (4 * tiles)))
    assert _status() == 0


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_heavy_key_beside_a_row_that_is_not_finite(dev, dtype, bad):
    """A row of dout with an infinity or NaN keeps no other row of its tile from being done once more."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from gradient_helpers import close, gradients, heavy_key
    from packed_helpers import Step
    step = Step(dev, dtype, 128, 1, 2, [2000])
    heavy_key(step, 1500, 0.97)
    step.dout[1501:2000:64, 1, 3] = bad            # one row of each tile
    out, lse = step.forward(T)
    dq, want = step.backward(T, out, lse)[0], gradients(step)
    rows = torch.ones(step.q.shape[:2], dtype=torch.bool, device=dev)
    rows[1501:2000:64, 1] = False
    rows[:1501] = False
    assert torch.isfinite(dq[rows]).all()
    close("dq", dq, want, rows)
    assert _status() == 0


@pytest.mark.parametrize("dim,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("queries,keys", [([3000, 5], [2000, 5]), ([40, 2500], [4000, 1100]), ([1], [3000])])
def test_heavy_keys_of_other_lengths(dev, dim, dtype, queries, keys):
    """Rows that attend no key before rows of many, and many keys before the first query."""
    from gradient_helpers import heavy_key
    from packed_helpers import Step
    step = Step(dev, dtype, dim, 2, 3, queries, keys)
    for seq, m in enumerate(keys):
        if m > 1024:
            heavy_key(step, m // 3, 0.97, seq)
    _close(step)
    assert _status() == 0


@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (128, "fp16")])
def test_heavy_keys_of_many_sequences(dev, dim, dtype):
    """More than 32 sequences, a few of them long, some of those with a heavy key."""
    from gradient_helpers import close, heavy_key
    from packed_helpers import Step
    lens = [1300 + i if i % 7 == 3 else (5 * i) % 40 for i in range(45)]
    step = Step(dev, dtype, dim, 1, 5, lens)
    for seq in (3, 17, 38):
        heavy_key(step, 600, 0.97, seq)
    grads, want = _close(step)
    for seq in (3, 17, 38):
        close("dq", grads[0], want, slice(step.q_starts[seq] + 601, step.q_starts[seq + 1]))
    assert _status() == 0
