"""Packed steps against plain 64-bit forms (GPU).

tests/packed_helpers.py derives the attention's tolerances.  Rows of no sequence
hold NaN in the inputs and a marker in the outputs.
"""

import math

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


# ---------------------------------------------------------------- attention

# head dim, type, KV heads, group, query lengths, key lengths (None: the same), layout
SHAPES = [
    (128, "bf16", 1, 1, [1], None, "own"),
    (128, "bf16", 2, 16, [1, 2, 0, 9], None, "fused"),
    (128, "fp16", 1, 1, [127, 128, 129], None, "own"),
    (64, "bf16", 2, 4, [255, 256, 257, 1], None, "heads"),
    (128, "bf16", 1, 16, [300, 5], None, "fused"),
    (64, "fp16", 3, 5, [77, 0, 26, 130], None, "fused"),          # 25 tokens of 5 heads: 125 rows of a tile
    (128, "fp16", 2, 7, [200, 19], None, "heads"),
    (64, "bf16", 1, 32, [3, 4, 5, 150], None, "own"),
    (128, "bf16", 1, 3, [43, 600], None, "own"),
    (128, "bf16", 2, 2, [1100], None, "own"),                      # dq from the rounded output in its later rows
    (64, "fp16", 1, 4, [1500, 40], None, "own"),
    (128, "bf16", 2, 8, [1, 12, 130], [700, 12, 1000], "own"),     # earlier keys
    (64, "fp16", 2, 1, [5, 300], [1300, 301], "heads"),
    (128, "bf16", 1, 4, [50, 300, 7], [20, 0, 300], "own"),        # fewer keys than queries: rows that attend none
    (64, "bf16", 1, 2, [300], [129], "own"),
    (128, "fp16", 2, 4, [0, 30, 0], [50, 40, 129], "own"),          # keys that no query attends
    # Few queries against many keys: divided over clusters.
    (128, "bf16", 2, 16, [12, 12], [4000, 1000], "own"),
    (64, "fp16", 1, 5, [1, 60, 0], [5000, 3001, 77], "heads"),
    (128, "fp16", 3, 4, [7], [2000], "own"),
    (64, "bf16", 1, 32, [2, 9], [6000, 20], "own"),
    (128, "bf16", 1, 1, [200], [3500], "own"),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "d%d-%s-%dx%d-%s-%s-%s" % (
    s[0], s[1], s[2], s[3], "_".join(map(str, s[4])), "_".join(map(str, s[5] or ["same"])), s[6]))
def test_attention_and_gradient(dev, shape):
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step, check, plain
    dim, dtype, heads, group, q_lens, k_lens, layout = shape
    step = Step(dev, dtype, dim, heads, group, q_lens, k_lens, layout)
    want = plain(step)
    out, lse = step.forward(T)
    assert _status() == 0
    check("out", out, want)
    check("lse", lse, want)
    for name, grad in zip(("dq", "dk", "dv"), step.backward(T, out, lse)):
        assert _status() == 0
        check(name, grad, want)


def test_attention_of_many_sequences(dev):
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step, check, plain
    lens = [(7 * i) % 23 for i in range(300)] + [140, 0, 290]
    step = Step(dev, "bf16", 64, 1, 4, lens, layout="fused")
    want = plain(step)
    out, lse = step.forward(T)
    check("out", out, want)
    check("lse", lse, want)
    for name, grad in zip(("dq", "dk", "dv"), step.backward(T, out, lse)):
        check(name, grad, want)
    assert _status() == 0


@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (128, "fp16")])
@pytest.mark.parametrize("count", [30, 64])
def test_units_one_after_another(dev, dim, dtype, count):
    """Far more tiles than SMs: short and long ones, whole and partly filled, follow each other on one SM."""
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step, check, plain
    lens = [1 + (i * 389) % 1000 for i in range(count)]
    step = Step(dev, dtype, dim, 4, 4, lens, layout="fused", seed=count)
    want = plain(step)
    out, lse = step.forward(T)
    assert _status() == 0
    check("out", out, want)
    check("lse", lse, want)
    for name, grad in zip(("dq", "dk", "dv"), step.backward(T, out, lse)):
        assert _status() == 0
        check(name, grad, want)


@pytest.mark.parametrize("dim,dtype,group,layout", [(64, "fp16", 5, "heads"), (128, "bf16", 7, "heads"),
                                                    (128, "fp16", 16, "own"), (64, "bf16", 32, "fused")])
def test_many_units_of_odd_groups(dev, dim, dtype, group, layout):
    """More than two tiles for every SM, so whole tiles are written at once: rows behind each, and of none, stay."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step, check, plain
    q_lens = [700, 1, 0, 640, 333, 411, 25, 128, 256]
    k_lens = [700, 1, 40, 500, 900, 411, 25, 129, 256]           # the fourth: rows that attend no key
    step = Step(dev, dtype, dim, 4, group, q_lens, None if layout == "fused" else k_lens, layout, seed=group)
    assert step.q_starts[-1] * 4 > 2 * (128 // group) * torch.cuda.get_device_properties(0).multi_processor_count
    want = plain(step)
    out, lse = step.forward(T)
    check("out", out, want)
    check("lse", lse, want)
    for name, grad in zip(("dq", "dk", "dv"), step.backward(T, out, lse)):
        check(name, grad, want)
    assert (out[step.q_starts[-1]:] == 7.0).all() and (lse[step.q_starts[-1]:] == 7.0).all()
    first = 300
    step.v[first, 2, 5] = math.inf                               # of the first sequence
    odd, _ = step.forward(T)
    hit = odd[first:700, 2 * group:3 * group, 5]
    assert (hit == math.inf).all()
    odd[first:700, 2 * group:3 * group] = out[first:700, 2 * group:3 * group]
    assert torch.equal(odd, out)                                 # the rest, bit for bit
    assert _status() == 0


def test_attention_of_4096_sequences_of_one_token(dev):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step
    step = Step(dev, "bf16", 64, 1, 1, [1] * 4096)
    out, lse = step.forward(T)
    n = 4096
    assert torch.equal(out[:n], step.v[:n])                     # one key: P = 1
    z = (step.q[:n].double() * step.k[:n].double()).sum(dim=2) * step.scale
    tol = 2 * 2.0 ** -24 * 67 * step.scale * (step.q[:n].double() * step.k[:n].double()).abs().sum(dim=2) + 2.0 ** -19
    assert ((lse[:n].double() - z).abs() <= tol + 2.0 ** -20 * z.abs()).all()
    assert _status() == 0


def test_gradient_of_4096_short_sequences(dev):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step
    step = Step(dev, "fp16", 64, 1, 2, [1, 2] * 2048)
    out, lse = step.forward(T)
    dq, dk, dv = step.backward(T, out, lse)
    n = 3 * 2048
    # Sequences of one token: P = 1 + d with |d| <= e_p (packed_helpers.py), so |dS| <= (e_p + 2^-23) |dout . v|, and
    # half the type's smallest step.
    one = torch.arange(0, n, 3, device=dev)
    q, k, v, g = (x[one].double() for x in (step.q, step.k, step.v, step.dout))
    e_p = 4 * 2.0 ** -24 * 67 * step.scale * (q * k).abs().sum(2, keepdim=True) + 2.0 ** -21 + 2.0 ** -23
    ds = 1.001 * e_p * (g * v).abs().sum(2, keepdim=True) + 2.0 ** -25
    assert (dq[one].double().abs() <= step.scale * ds * k.abs() + 2.0 ** -25).all()
    assert (dk[one].double().abs() <= (step.scale * ds * q.abs()).sum(1, keepdim=True) + 2.0 ** -25).all()
    want = step.dout[one].double().sum(dim=1, keepdim=True)
    # Two rounded probabilities of 1 (exact), an fp32 sum, and the rounding of the result.
    assert ((dv[one].double() - want).abs() <= 2.0 ** -11 * 1.001 * want.abs() + 2.0 ** -19 *
            step.dout[one].double().abs().sum(dim=1, keepdim=True) + 2.0 ** -25).all()
    last = one + 2                                              # the second token's key: only its own query attends it
    q, k = step.q[last].double(), step.k[:n].double()
    z = torch.stack([(q * k[last - 1]).sum(2), (q * k[last]).sum(2)]) * step.scale
    p = torch.softmax(z, dim=0)[1][..., None]
    want = (p * step.dout[last].double()).sum(dim=1, keepdim=True)
    size = (p * step.dout[last].double().abs()).sum(dim=1, keepdim=True)
    assert ((dv[last].double() - want).abs() <= (2.0 ** -11 + 2.0 ** -15) * size + 2.0 ** -11 * 1.001 * want.abs() +
            2.0 ** -24).all()
    assert _status() == 0


def test_lse_may_be_absent(dev):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step
    step = Step(dev, "bf16", 128, 2, 4, [33, 200])
    out, _ = step.forward(T)
    again = torch.full_like(out, 7.0)
    T.packed_attn(step.q, step.k, step.v, step.ints(step.q_starts), again, scale=step.scale)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_what_a_row_does_not_attend_does_not_reach_it(dev, dtype, bad):
    """A value, and a key, that only later rows attend: the earlier ones are as without it, bit for bit."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step
    for group, n, at, dim in ((1, 300, 200, 128), (16, 40, 21, 64), (5, 130, 128, 128), (4, 77, 0, 64)):
        step = Step(dev, dtype, dim, 2, group, [9, n], seed=at)
        clean, _ = step.forward(T)
        first = 9 + at
        step.v[first, 1, 5] = bad
        out, lse = step.forward(T)
        assert torch.equal(out[:first], clean[:first])
        assert torch.equal(out[first:9 + n, :group], clean[first:9 + n, :group])     # the other KV head
        column = out[first:9 + n, group:, 5]
        assert torch.isnan(column).all() if math.isnan(bad) else (column == bad).all()
        others = [c for c in range(dim) if c != 5]
        a, b = out[first:9 + n, group:][..., others].double(), clean[first:9 + n, group:][..., others].double()
        # The row with the infinity enters in 32 bits instead of as a 16-bit P.
        eps = torch.finfo(step.dtype).eps
        assert ((a - b).abs() <= eps * step.v[9:9 + n].nan_to_num(0, 0, 0).double().abs().max() * 2).all()
        assert torch.isfinite(lse[:9 + n]).all()
        step = Step(dev, dtype, dim, 2, group, [9, n], seed=at)
        step.k[first, 1, 5] = bad
        out, lse = step.forward(T)
        assert torch.equal(out[:first], clean[:first]) and torch.isfinite(lse[:first]).all()
    assert _status() == 0


def test_far_scores(dev):
    """Scores of some thousands, rising along the sequence: the running maximum moves in every tile."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step, check, plain
    for dtype in ("bf16", "fp16"):
        step = Step(dev, dtype, 64, 1, 2, [700])
        ramp = torch.linspace(0.0, 60.0, 700, device=dev)[:, None]
        step.k[:700, 0] = (step.k[:700, 0].float() * 0.1 + ramp).to(step.dtype)
        step.q[:700] = (step.q[:700].float() + 8).to(step.dtype)
        want = plain(step, with_grads=False)
        out, lse = step.forward(T)
        check("out", out, want)
        check("lse", lse, want)


def test_bad_starts_are_flagged_and_skipped(dev):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step
    step = Step(dev, "bf16", 128, 1, 4, [40, 50, 60])
    good, good_lse = step.forward(T)
    good_grads = step.backward(T, good, good_lse)
    assert _status() == 0
    for starts, ok in (([0, 40, 90, 10 ** 9], slice(0, 90)), ([0, 40, -5, 150], slice(0, 40)),
                       ([-1, 40, 90, 150], slice(40, 150)), ([0, 40, 90, 154], slice(0, 90))):
        step.q_starts = starts
        out, lse = step.forward(T)
        assert _status() == T.DEVICE_BAD_KV_LEN, starts
        assert torch.equal(out[ok], good[ok]) and torch.equal(lse[ok], good_lse[ok])
        grads = step.backward(T, good, good_lse)
        assert _status() == T.DEVICE_BAD_KV_LEN
        for a, b in zip(grads, good_grads):
            assert torch.equal(a[ok], b[ok])
        rest = [i for i in range(153) if not (ok.start <= i < ok.stop)]
        assert (out[rest] == 7.0).all() and all((g[rest] == 7.0).all() for g in grads)


def test_bad_starts_behind_many_good_ones_are_flagged(dev):
    """40 sequences of one query, each with more than a thousand keys: few units, divided over clusters."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step
    step = Step(dev, "bf16", 64, 1, 1, [1] * 40, [1100] * 40)
    good, good_lse = step.forward(T)
    assert _status() == 0
    step.q_starts = [*range(38), 38, 12, 40]       # sequence 38 descends; the last one has rows 12 .. 39
    out, lse = step.forward(T)
    assert _status() == T.DEVICE_BAD_KV_LEN
    assert torch.equal(out[:12], good[:12]) and torch.equal(lse[:12], good_lse[:12])


def test_same_bits_every_time(dev):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step
    step = Step(dev, "bf16", 128, 2, 4, [700, 33, 1300], [900, 33, 1300])
    out, lse = step.forward(T)
    grads = step.backward(T, out, lse)
    for _ in range(3):
        again, lse_again = step.forward(T)
        assert torch.equal(out, again) and torch.equal(lse, lse_again)
        for a, b in zip(grads, step.backward(T, out, lse)):
            assert torch.equal(a, b)


def test_gradient_against_differences(dev):
    """The forward formula's slope along random directions, by central differences in 64 bits."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step, plain
    step = Step(dev, "fp16", 64, 2, 3, [37, 150], [60, 150])
    out, lse = step.forward(T)
    grads = step.backward(T, out, lse)
    want = plain(step)
    total_q, total_k = step.q_starts[-1], step.k_starts[-1]
    g = step.dout[:total_q].double()

    def loss():
        return float((plain(step, with_grads=False)["out"][0][:total_q] * g).sum())
    for name, grad, rows in (("q", grads[0], total_q), ("k", grads[1], total_k), ("v", grads[2], total_k)):
        x = getattr(step, name).double()
        direction = torch.randn(x.shape, dtype=torch.float64, device=dev,
                                generator=torch.Generator(device=dev).manual_seed(3))
        step_size, values = 1e-4, []
        for sign in (1, -1):
            setattr(step, name, x + sign * step_size * direction)
            values.append(loss())
        setattr(step, name, x.to(step.dtype))
        slope = (values[0] - values[1]) / (2 * step_size)
        got = float((grad[:rows].double() * direction[:rows]).sum())
        tol = float((want["d" + name][1][:rows] * direction[:rows].abs()).sum())
        # Central differences: the third derivative's step^2 / 6, far below a millionth of the slope's parts.
        parts = float((grad[:rows].double() * direction[:rows]).abs().sum())
        assert abs(got - slope) <= tol + 1e-6 * parts, (name, got, slope)


def test_other_stream_and_graph(dev):
    """Forward and gradient on a side stream and captured, two graphs with workspaces of their own."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step, check, plain
    shapes = [dict(q_lens=[130, 70], layout="fused"), dict(q_lens=[9, 3], k_lens=[1200, 900])]   # (one over clusters)
    steps = [Step(dev, "bf16", 128, 2, 4, seed=i, **shapes[i]) for i in range(2)]
    captured = []
    for step in steps:
        out, lse = torch.full_like(step.q, 7.0), torch.full(step.q.shape[:2], 7.0, device=dev)
        grads = [torch.full_like(x, 7.0) for x in (step.q, step.k, step.v)]
        ws, starts = T.alloc_packed_workspace(step.q).fill_(0xff), step.ints(step.q_starts)
        k_starts = step.ints(step.k_starts) if step.own_keys else None

        def call():
            T.packed_attn(step.q, step.k, step.v, starts, out, lse, k_starts=k_starts, scale=step.scale)
            T.packed_attn_backward(step.q, step.k, step.v, starts, out, lse, step.dout, *grads, workspace=ws,
                                   k_starts=k_starts, scale=step.scale)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        captured.append((graph, step, out, lse, grads, ws, starts, k_starts))     # (a graph holds no tensors)
    for seed in (5, 6):                          # new contents, replayed in both orders
        for i, (graph, step, out, lse, grads, *_) in enumerate(captured):
            fresh = Step(dev, "bf16", 128, 2, 4, seed=10 * seed + i, **shapes[i])
            for name in ("q", "k", "v", "dout"):
                getattr(step, name).copy_(getattr(fresh, name))
            for t in (out, lse, *grads):
                t.fill_(7.0)
        for graph, *_ in captured if seed == 5 else captured[::-1]:
            graph.replay()
        for graph, step, out, lse, grads, *_ in captured:
            want = plain(step)
            for name, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
                check(name, got, want)
    assert _status() == 0


def test_two_calls_at_once(dev):
    """Forward and backward passes of two batches on two streams give what they give one after the other."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step
    steps = [Step(dev, "bf16", 128, 2, 4, [900, 31, 1700]), Step(dev, "fp16", 64, 4, 5, [64] * 40 + [700, 1100])]
    want = []
    for step in steps:
        out, lse = step.forward(T)
        want.append((out, lse, *step.backward(T, out, lse)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, step in enumerate(steps):
            with torch.cuda.stream(streams[i]):
                out, lse = step.forward(T)
                got[i].append((out, lse, *step.backward(T, out, lse)))
    torch.cuda.synchronize()
    for once, many in zip(want, got):
        for result in many:
            for a, b in zip(once, result):
                assert torch.equal(a.nan_to_num(9.0), b.nan_to_num(9.0))
    assert _status() == 0


def test_binding_refuses(dev):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from packed_helpers import Step
    step = Step(dev, "bf16", 64, 2, 4, [20, 30])
    starts, out = step.ints(step.q_starts), torch.empty_like(step.q)
    q, k, v = step.q, step.k, step.v

    def refused(*args, **kw):
        with pytest.raises(T.InfLLMv2Error):
            T.packed_attn(*args, **kw)
    refused(q.float(), k, v, starts, out)
    refused(q, k.half(), v, starts, out)
    refused(q, k, v[:, :1], starts, out)
    refused(q[:, :7], k, v, starts, out[:, :7])               # 7 heads over 2
    refused(q.cpu(), k, v, starts, out)
    refused(q, k, v, starts.long(), out)
    refused(q, k, v, starts.cpu(), out)
    refused(q, k, v, starts, out.float())
    refused(q, k, v, starts, out[:-1])
    refused(q[..., ::2], k[..., ::2], v[..., ::2], starts, out[..., ::2])
    refused(q, k, v, starts, out, lse=torch.empty((q.shape[0], 7), device=dev))
    refused(q, k, v, starts, out, k_starts=starts[:-1])
    refused(q, k.expand(-1, 2, -1)[:, :1].expand(-1, 2, -1), v, starts, out)   # one row for two heads
    refused(q, k, v, starts, out, scale=0.0)
    refused(q, k, v, starts, out, scale=float("nan"))
    refused(q, k, v, starts, out, scale=1e39)                 # past fp32
    refused(q[:10], k, v, starts, out[:10])                   # no k_starts, other counts of tokens
    lse = torch.empty(q.shape[:2], device=dev)
    grads = [torch.empty_like(x) for x in (q, k, v)]
    with pytest.raises(T.InfLLMv2Error):
        T.packed_attn_backward(q, k, v, starts, out, lse, out, *grads, workspace=T.alloc_packed_workspace(q)[:-8])
    with pytest.raises(T.InfLLMv2Error):
        T.packed_attn_backward(q, k, v, starts, out, lse, out, grads[0].float(), *grads[1:],
                               workspace=T.alloc_packed_workspace(q))


# ------------------------------------------------------------------- rotary

def _turn(x, positions, freq, scale, part, interleaved, transpose):
    """The formula in 64 bits, and what rounding may cost: (value, tolerance)."""
    import torch
    angle = positions.double()[:, None, None] * freq.to(x.device) * (-1 if transpose else 1)
    cos, sin = angle.cos() * scale, angle.sin() * scale
    y = x.double().clone()
    first, second = ((slice(0, part, 2), slice(1, part, 2)) if interleaved else
                     (slice(0, part // 2), slice(part // 2, part)))
    a, b = x[..., first].double(), x[..., second].double()
    y[..., first], y[..., second] = a * cos - b * sin, a * sin + b * cos
    # Angle: 2^-33 turn of rounding, 2^-24 of an eighth turn to fp32, and the 64-bit product of this formula
    # (2^-53 of it); sine and cosine: 2^-22; times scale, two products and a sum: 2^-22 of the magnitudes.
    far = float(positions.abs().max()) * float(freq.max())
    off = 2 * math.pi * (2.0 ** -33 + 2.0 ** -27) + 2.0 ** -51 * far + 2.0 ** -21
    size = torch.zeros_like(y)
    size[..., first] = size[..., second] = (a.abs() + b.abs()) * scale
    info = torch.finfo(x.dtype)
    return y, 1.001 * (off * size + info.eps / 2 * y.abs()) + info.tiny * info.eps / 2


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,part,heads,tokens", [(128, 128, 3, 5), (64, 32, 40, 700), (512, 512, 1, 3),
                                                   (80, 48, 2, 33), (128, 16, 17, 1), (16, 16, 1, 2000),
                                                   (256, 128, 9, 1300)])
def test_rotary(dev, dtype, interleaved, dim, part, heads, tokens):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    dtype = getattr(torch, dtype)
    gen = torch.Generator(device=dev).manual_seed(dim + tokens)
    whole = torch.randn((tokens, heads + 2, dim), device=dev, generator=gen).to(dtype)   # q and k of one projection
    q, k = whole[:, :heads], whole[:, heads:]
    positions = torch.randint(-100, 2 ** 31 - 1, (tokens,), device=dev, generator=gen,
                              dtype=torch.int64).to(torch.int32)
    positions[::2] %= 5000
    positions[-1] = 0
    plan = T.alloc_rotary_plan(part, base=50000.0, device=dev)
    freq = 50000.0 ** (-torch.arange(part // 2, dtype=torch.float64) * 2 / part)
    for transpose in (False, True):
        q_out, k_out = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty_like(k)
        T.rotary(q, k, positions, plan, q_out, k_out, interleaved=interleaved, transpose=transpose)
        for x, y in ((q, q_out), (k, k_out)):
            want, tol = _turn(x, positions, freq, 1.0, part, interleaved, transpose)
            assert ((y.double() - want).abs() <= tol).all()
            assert torch.equal(y[..., part:], x[..., part:])
        copy = whole.clone()
        assert T.rotary(copy[:, :heads], copy[:, heads:], positions, plan, interleaved=interleaved,
                        transpose=transpose)[0].data_ptr() == copy.data_ptr()
        assert torch.equal(copy[:, :heads], q_out) and torch.equal(copy[:, heads:], k_out)
        alone = torch.empty_like(q_out)
        T.rotary(q, None, positions, plan, alone, interleaved=interleaved, transpose=transpose)
        assert torch.equal(alone, q_out)
    assert _status() == 0


def test_rotary_scaled_and_back(dev):
    """Turned and turned back: scale^2 times the input; and the transposed turn is the gradient."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    plan = T.alloc_rotary_plan(64, scaling=T.ROTARY_PARTS, factor=16.0, original_len=4096, device=dev)
    gen = torch.Generator(device=dev).manual_seed(1)
    x, g = (torch.randn((300, 4, 64), device=dev, generator=gen) for _ in range(2))
    positions = torch.arange(300, device=dev, dtype=torch.int32) * 4001
    y, back = torch.empty_like(x), torch.empty_like(x)
    T.rotary(x, None, positions, plan, y)
    T.rotary(y, None, positions, plan, back, transpose=True)
    assert plan.scale == pytest.approx(0.1 * math.log(16.0) + 1, abs=1e-6)
    size = plan.scale ** 2 * (x.abs() + x.roll(32, dims=2).abs())
    assert ((back - plan.scale ** 2 * x).abs() <= 2.0 ** -19 * size).all()
    T.rotary(g, None, positions, plan, back, transpose=True)
    # <g, R x> = <R^T g, x>
    left, right = (g.double() * y.double()).sum(), (back.double() * x.double()).sum()
    parts = (g.double() * y.double()).abs().sum()
    assert abs(float(left - right)) <= 2.0 ** -19 * float(parts)


def test_rotary_binding_refuses(dev):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    plan = T.alloc_rotary_plan(64, device=dev)
    q, positions = torch.zeros((4, 2, 64), device=dev), torch.zeros(4, dtype=torch.int32, device=dev)

    def refused(*args, **kw):
        with pytest.raises(T.InfLLMv2Error):
            T.rotary(*args, **kw)
    refused(q.double(), None, positions, plan)
    refused(q.cpu(), None, positions, plan)
    refused(q, None, positions.long(), plan)
    refused(q, None, positions[:3], plan)
    refused(q[..., ::2], None, positions, plan)
    refused(q[..., :48].contiguous(), None, positions, plan)          # rotary_dim past the head
    refused(q, q.half(), positions, plan)
    refused(q, None, positions, plan, q.transpose(0, 1).contiguous().transpose(0, 1)[:, :1])
    refused(q, None, positions, plan, q[:1].expand(4, 2, 64))          # outputs that overlap


# ---------------------------------------------------------- pages and slots

class Book:
    """The page tables in plain Python: what paged_reserve leaves."""

    def __init__(self, tables):
        self.table, self.held = tables.page_table.tolist(), tables.held.tolist()
        self.free, self.n, self.page = tables.free_pages.tolist(), int(tables.n_free), tables.page_size

    def reserve(self, kv, new, seen, tokens):
        need = [-(-(a + b) // self.page) for a, b in zip(kv, new)]
        back = [p for row, h, m in zip(self.table, self.held, need) for p in row[m:h]]
        lacking = max(0, sum(max(0, m - h) for h, m in zip(self.held, need)) - self.n - len(back))
        if lacking:
            return dict(missing=lacking, new_lens=kv, starts=[0] * (len(kv) + 1), slots=[-1] * tokens,
                        positions=[0] * tokens)
        spare = list(back)
        for b, row in enumerate(self.table):
            for c in range(self.held[b], need[b]):
                if self.n:
                    self.n -= 1
                    row[c] = self.free[self.n]
                else:
                    row[c] = spare.pop(0)
        for p in spare:
            self.free[self.n] = p
            self.n += 1
        self.held = need
        starts, slots, positions = [0], [], []
        for b, row in enumerate(self.table):
            starts.append(starts[-1] + new[b])
            for t in range(new[b]):
                s = kv[b] + t
                slots.append(row[s // self.page] * self.page + s % self.page)
                positions.append(seen[b] + t)
        rest = tokens - len(slots)
        return dict(missing=0, new_lens=[a + b for a, b in zip(kv, new)], starts=starts, slots=slots + [-1] * rest,
                    positions=positions + [0] * rest)

    def check(self, tables):
        assert tables.page_table.tolist() == self.table and tables.held.tolist() == self.held
        assert int(tables.n_free) == self.n and tables.free_pages.tolist() == self.free


def _cache(dev, pages, page=16, heads=1, dim=64, metadata=False):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    k, v = (torch.zeros((pages, heads, page, dim), dtype=torch.bfloat16, device=dev) for _ in range(2))
    w = torch.full((pages, heads, page), 5.0, device=dev) if metadata else None
    p = torch.full((pages, heads, page), -5, dtype=torch.int32, device=dev) if metadata else None
    return T.PagedCache(k, v, w, p)


@pytest.mark.parametrize("batch,pages,page,most", [(1, 40, 16, 100), (5, 60, 16, 150), (70, 3000, 32, 500),
                                                   (1025, 9000, 16, 40), (4096, 9000, 16, 30), (3, 5000, 16, 30000)])
def test_reserve_through_the_life_of_a_batch(dev, batch, pages, page, most):
    """Prompts, decode steps, evictions, sequences that finish, and a pool that runs out."""
    import random
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    rng = random.Random(batch)
    cache = _cache(dev, pages, page)
    width = -(-2 * most // page)
    tables = T.alloc_page_tables(cache, batch, width)
    book = Book(tables)
    kv, seen, lacked = [0] * batch, [0] * batch, 0
    for turn in range(8):
        new = []
        for b in range(batch):
            if kv[b] and rng.random() < 0.2:
                kv[b] = seen[b] = 0                                   # finished
                new.append(0 if rng.random() < 0.5 else rng.randint(1, most))
            elif kv[b] and rng.random() < 0.2:
                kv[b] = max(1, kv[b] // 3)                            # evicted
                new.append(1)
            else:
                new.append(rng.randint(0, most) if kv[b] == 0 else min(1, 2 * most - kv[b]))
        tokens = sum(new) + rng.choice([0, 3, 500])
        ints = [torch.tensor(x, dtype=torch.int32, device=dev) for x in (kv, new, seen)]
        starts = torch.empty(batch + 1, dtype=torch.int32, device=dev)
        slots, positions = (torch.full((tokens + 5,), 77, dtype=torch.int32, device=dev) for _ in range(2))
        lens = ints[0] if turn % 2 else torch.empty_like(ints[0])      # in place every other time
        T.paged_reserve(tables, ints[0], ints[1], lens, starts, slots[:tokens], positions[:tokens], seq_lens=ints[2])
        assert _status() == 0
        want = book.reserve(kv, new, seen, tokens)
        book.check(tables)
        assert int(tables.missing) == want["missing"] and lens.tolist() == want["new_lens"]
        assert starts.tolist() == want["starts"]
        assert slots.tolist() == want["slots"] + [77] * 5 and positions.tolist() == want["positions"] + [77] * 5
        if want["missing"]:
            lacked += 1
        else:
            seen = [a + b for a, b in zip(seen, new)]
        kv = want["new_lens"]
    owned = [p for row, h in zip(book.table, book.held) for p in row[:h]]
    assert sorted(owned + book.free[:book.n]) == list(range(pages))   # every page once


def test_reserve_reuses_what_the_call_gives_back(dev):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    cache = _cache(dev, 4)
    tables = T.alloc_page_tables(cache, 2, 4)
    lens, starts = torch.zeros(2, dtype=torch.int32, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)

    def step(kv, new):
        kv, new = (torch.tensor(x, dtype=torch.int32, device=dev) for x in (kv, new))
        T.paged_reserve(tables, kv, new, lens, starts)
        return int(tables.missing), lens.tolist(), tables.held.tolist(), int(tables.n_free)
    assert step([0, 0], [64, 0]) == (0, [64, 0], [4, 0], 0)
    assert step([64, 0], [0, 17]) == (2, [64, 0], [4, 0], 0)           # none free: as it was
    assert step([0, 0], [0, 33]) == (0, [0, 33], [0, 3], 1)            # the first finishes: its pages serve
    assert tables.page_table[1].tolist()[:3] == [0, 1, 2] and tables.free_pages.tolist()[0] == 3
    assert step([0, 33], [60, 0]) == (3, [0, 33], [0, 3], 1) and step([0, 33], [64, 31]) == (4, [0, 33], [0, 3], 1)
    assert step([0, 0], [64, 64]) == (4, [0, 0], [0, 3], 1)            # more than the pool has
    assert _status() == 0
    assert step([0, 33], [0, -1])[0] == -1 and _status() == T.DEVICE_BAD_KV_LEN


def test_reserve_refuses_bad_lengths_whole(dev):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    cache = _cache(dev, 20)

    def ints(*x):
        return torch.tensor(x, dtype=torch.int32, device=dev)
    for kv, new, spoil in (((0, -1), (1, 1), None), ((0, 0), (1, -3), None), ((0, 60), (5, 5), None),
                           ((0, 2 ** 31 - 1), (1, 2 ** 31 - 1), None), ((0, 0), (20, 30), None),
                           ((0, 0), (1, 1), "held"), ((0, 0), (1, 1), "n_free")):
        tables = T.alloc_page_tables(cache, 2, 4)
        if spoil == "held":
            tables.held[1] = 5
        elif spoil == "n_free":
            tables.n_free[0] = 21
        before = [t.clone() for t in (tables.page_table, tables.held, tables.free_pages, tables.n_free)]
        lens, starts, slots = ints(7, 7), ints(7, 7, 7), ints(*[7] * 40)
        T.paged_reserve(tables, ints(*kv), ints(*new), lens, starts, slots)
        assert _status() == T.DEVICE_BAD_KV_LEN and int(tables.missing) == -1
        assert lens.tolist() == list(kv) and starts.tolist() == [0, 0, 0] and slots.tolist() == [-1] * 40
        for a, b in zip(before, (tables.page_table, tables.held, tables.free_pages, tables.n_free)):
            assert torch.equal(a, b)


def test_reserve_with_a_foreign_page_on_the_stack(dev):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    tables = T.alloc_page_tables(_cache(dev, 4), 1, 4)
    tables.free_pages[3] = 4                                           # no page of the pool, and on top
    kv, new, lens = (torch.tensor([n], dtype=torch.int32, device=dev) for n in (0, 18, 0))
    starts, slots = torch.zeros(2, dtype=torch.int32, device=dev), torch.zeros(18, dtype=torch.int32, device=dev)
    T.paged_reserve(tables, kv, new, lens, starts, slots)
    assert _status() == T.DEVICE_BAD_PAGE and slots.tolist() == [-1] * 16 + [16, 17]      # then page 1


def test_reserve_binding_refuses(dev):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    tables = T.alloc_page_tables(_cache(dev, 4), 2, 4)
    kv, starts = torch.zeros(2, dtype=torch.int32, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
    for args in ((kv.long(), kv, kv, starts), (kv, kv[:1], kv, starts), (kv, kv, kv.cpu(), starts), (kv, kv, kv, kv)):
        with pytest.raises(T.InfLLMv2Error):
            T.paged_reserve(tables, *args)
    with pytest.raises(T.InfLLMv2Error):
        T.paged_reserve(tables, kv, kv, kv, starts, slots=starts, positions=kv)
    with pytest.raises(T.InfLLMv2Error):
        T.paged_reserve(tables, kv, kv.clone(), kv.clone(), starts, seq_lens=starts)
    lens = kv.clone()
    with pytest.raises(T.InfLLMv2Error):
        T.paged_reserve(tables, kv, kv, lens, starts, seq_lens=lens)
    with pytest.raises(T.InfLLMv2Error):
        T.PageTables(tables.page_table, tables.held, tables.free_pages, kv, tables.missing, 16)


# ------------------------------------------------------------- packed append

@pytest.mark.parametrize("layout", ["hnd", "nhd", "pair"])
@pytest.mark.parametrize("dtype,heads,dim,page,tokens", [("bf16", 2, 128, 16, 1), ("fp16", 3, 64, 48, 133),
                                                         ("bf16", 1, 64, 256, 1000), ("fp16", 8, 128, 32, 70)])
def test_packed_append(dev, layout, dtype, heads, dim, page, tokens):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from paged_helpers import Pool
    pool = Pool(dev, dtype, layout, heads, dim, page, [tokens, 1], metadata=tokens != 70)
    slots = torch.randperm(pool.k.shape[0] * page, generator=pool.gen, device=dev)[:tokens].to(torch.int32)
    slots[tokens // 2::5] = -1
    slots[tokens // 3::7] = -(2 ** 31)
    whole = pool.normal(tokens, 2 * heads, dim)
    k_new, v_new = whole[:, :heads], whole[:, heads:]
    positions = torch.arange(tokens, dtype=torch.int32, device=dev) * 3
    want = [None if t is None else t.clone() for t in (pool.k, pool.v, pool.weights, pool.positions)]
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            want[0][s // page, :, s % page], want[1][s // page, :, s % page] = k_new[t], v_new[t]
            if want[2] is not None:
                want[2][s // page, :, s % page], want[3][s // page, :, s % page] = 0.0, 3 * t
    T.paged_append_packed(pool.cache, k_new, v_new, slots, positions)
    assert _status() == 0
    for got, w in zip((pool.k, pool.v, pool.weights, pool.positions), want):
        assert w is None or torch.equal(got.nan_to_num(9.0) if w.is_floating_point() else got,
                                        w.nan_to_num(9.0) if w.is_floating_point() else w)


def test_packed_append_from_pinned_memory_and_a_slot_past_the_pool(dev):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    cache = _cache(dev, 2, page=16, heads=2, dim=64, metadata=True)
    new = [torch.randn((3, 2, 64)).to(torch.bfloat16).pin_memory() for _ in range(2)]
    slots = torch.tensor([31, 32, 0], dtype=torch.int32, device=dev)
    T.paged_append_packed(cache, *new, slots, torch.tensor([4, 5, 6], dtype=torch.int32, device=dev))
    assert _status() == T.DEVICE_BAD_PAGE
    assert torch.equal(cache.k_pages[1, :, 15].cpu(), new[0][0])
    assert torch.equal(cache.v_pages[0, :, 0].cpu(), new[1][2])
    assert cache.positions[1, :, 15].tolist() == [4, 4] and cache.positions[0, :, 0].tolist() == [6, 6]
    assert int((cache.positions == -5).sum()) == 2 * 2 * 16 - 4 and int((cache.weights == 0).sum()) == 4
    for bad in ((new[0][:2], new[1], slots), (new[0], new[1], slots[:2]), (new[0].clone(), new[1], slots),
                (new[0].float(), new[1], slots), (new[0], new[1], slots.cpu())):
        with pytest.raises(T.InfLLMv2Error):
            T.paged_append_packed(cache, *bad, slots)
    with pytest.raises(T.InfLLMv2Error):
        T.paged_append_packed(cache, *new, slots)                      # a cache with positions needs them


# ------------------------------------------------------------ all of a step

@pytest.mark.parametrize("captured", [False, True])
def test_prompts_then_tokens_through_the_pages(dev, captured):
    """Tables, rotary positions, prompt attention, packed append, then decode steps (eager, or one graph replayed)."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    heads, group, dim, page, batch = 2, 4, 64, 16, 3
    gen = torch.Generator(device=dev).manual_seed(2)
    cache = _cache(dev, 60, page, heads, dim, metadata=True)
    tables = T.alloc_page_tables(cache, batch, 16)
    plan = T.alloc_rotary_plan(dim, device=dev)
    prompts, steps = [37, 1, 130], 20
    total = [n + steps for n in prompts]
    rows = [torch.randn((n, heads * (group + 2), dim), device=dev, generator=gen).to(torch.bfloat16) for n in total]

    def packed(parts):
        return torch.cat(parts).split([heads * group, heads, heads], dim=1)
    freq = 10000.0 ** (-torch.arange(dim // 2, dtype=torch.float64) * 2 / dim)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)
    lens, seen, n_new, starts = ints([0] * batch), ints([0] * batch), ints(prompts), ints([0] * (batch + 1))
    tokens = sum(prompts) + 7
    slots, positions = ints([0] * tokens), ints([0] * tokens)
    whole = torch.cat([r[:n] for r, n in zip(rows, prompts)] + [torch.full_like(rows[0][:7], float("nan"))])
    q, k, v = whole.split([heads * group, heads, heads], dim=1)
    T.paged_reserve(tables, lens, n_new, lens, starts, slots, positions, seq_lens=seen)
    T.rotary(q, k, positions, plan)
    out = torch.full_like(q, 7.0)
    T.packed_attn(q, k, v, starts, out)
    T.paged_append_packed(cache, k, v, slots, positions)
    seen += n_new

    # Decode steps: a step of three tokens, the same calls with the single-token attention.
    one, slots1, positions1 = ints([1] * batch), ints([0] * batch), ints([0] * batch)
    new = torch.empty((batch, heads * (group + 2), dim), dtype=torch.bfloat16, device=dev)
    nq, nk, nv = new.split([heads * group, heads, heads], dim=1)
    q1, k1 = torch.empty_like(nq, memory_format=torch.contiguous_format), torch.empty_like(nk)
    out1 = torch.empty((batch, 1, heads * group, dim), dtype=torch.bfloat16, device=dev)
    ws = T.alloc_paged_workspace(cache, tables.page_table, T.OP_PAGED_DECODE, group)

    def decode():
        T.paged_reserve(tables, lens, one, lens, starts, slots1, positions1, seq_lens=seen)
        T.rotary(nq, nk, positions1, plan, q1, k1)
        T.paged_append_packed(cache, k1, nv, slots1, positions1)
        T.paged_attn_decode(cache, q1.view(batch, 1, heads * group, dim), tables.page_table, lens, out1, workspace=ws)
        seen.add_(one)
    graph = None
    decoded = []
    for t in range(steps):
        new.copy_(torch.stack([r[n + t] for r, n in zip(rows, prompts)]))
        if not captured:
            decode()
        elif graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                decode()
        if graph is not None:
            graph.replay()
        decoded.append(out1.clone())
    assert _status() == 0 and int(tables.missing) == 0
    assert lens.tolist() == total and seen.tolist() == total

    # One causal pass over each whole sequence, from inputs turned in 64 bits and rounded as the kernel rounds.
    for b, n in enumerate(total):
        qkv = rows[b]
        at = torch.arange(n, device=dev)
        turned = torch.empty_like(qkv[:, :heads * (group + 1)], memory_format=torch.contiguous_format)
        T.rotary(qkv[:, :heads * (group + 1)], None, at.to(torch.int32), plan, turned)
        want, tol = _turn(qkv[:, :heads * (group + 1)], at, freq, 1.0, dim, False, False)
        assert ((turned.double() - want).abs() <= tol).all()
        q64 = turned[:, :heads * group].double().view(n, heads, group, dim)
        k64, v64 = turned[:, heads * group:].double(), qkv[:, heads * (group + 1):].double()
        z = torch.einsum("rhgd,khd->hgrk", q64, k64) * dim ** -0.5
        z.masked_fill_(at[None] > at[:, None], -math.inf)
        p = torch.softmax(z, dim=3)
        want = torch.einsum("hgrk,khd->rhgd", p, v64).reshape(n, heads * group, dim)
        # Scores to 2^-13 at most here (|z| < 16), P and the result rounded to bf16.
        size = torch.einsum("hgrk,khd->rhgd", p, v64.abs()).reshape(n, heads * group, dim)
        tol = (2.0 ** -8 + 2.0 ** -12) * size + 2.0 ** -8 * 1.001 * want.abs()
        first = sum(prompts[:b])
        got = torch.cat([out[first:first + prompts[b]]] + [d[b] for d in decoded])
        assert ((got.double() - want).abs() <= tol).all()
    assert (out[sum(prompts):] == 7.0).all()
    pages = [p for row, h in zip(tables.page_table.tolist(), tables.held.tolist()) for p in row[:h]]
    assert len(set(pages)) == len(pages) == sum(-(-n // page) for n in total)
