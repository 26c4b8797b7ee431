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
def test_values_that_outgrow_the_first_tile(dev, dim):
    """fp16 rows that walk their keys from the last: neither the first tile nor D tells of the values before.

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
