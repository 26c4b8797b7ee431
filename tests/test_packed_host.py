"""Refusals of the packed step's entry points, and the rotary frequencies (no GPU needed).

Every refused call fails validation before anything touches the device; the
fake pointers are never dereferenced.
"""

import ctypes
import math

import pytest

FAKE = 0x7F0000000000
ODD = FAKE + 8


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    from trainable_block_sparse_infllm_gb300 import _lib
    return _lib


def _ints64(*values):
    return (ctypes.c_int64 * len(values))(*values)


# ------------------------------------------------------------------- rotary

def _frequencies(L, **kw):
    d = kw.get("rotary_dim", 64)
    fields = dict(rotary_dim=d, scaling=L.ROTARY_PLAIN, base=10000.0, factor=4.0, original_len=4096, fast_turns=32.0,
                  slow_turns=1.0)
    factors = kw.pop("factors", None)
    fields.update(kw)
    if factors is not None:
        fields["factors"] = (ctypes.c_double * len(factors))(*factors)
    turns, scale = (ctypes.c_uint64 * 512)(), ctypes.c_float()
    rc = L.lib.infllmv2_rotary_frequencies(ctypes.byref(L.RotaryConfig(**fields)), turns, ctypes.byref(scale))
    return rc, [t / 2.0 ** 64 * 2 * math.pi for t in turns[:max(d, 0) // 2]], scale.value


# 2^64 turns are truncated to whole numbers: 2 pi 2^-64 < 2^-61 radians; the double arithmetic costs a few 2^-52.
UNIT = 2.0 ** -61


def _close(a, b):
    return all(abs(x - y) <= 1e-14 * y + UNIT for x, y in zip(a, b)) and len(a) == len(b)


def test_frequencies(L):
    for d in (2, 16, 64, 128, 512):
        rc, got, scale = _frequencies(L, rotary_dim=d)
        assert rc == L.OK and scale == 1.0
        assert _close(got, [10000.0 ** (-2 * i / d) for i in range(d // 2)])
        if d > 2:
            rc, got, scale = _frequencies(L, rotary_dim=d, scaling=L.ROTARY_BASE)
            base = 10000.0 * 4.0 ** (d / (d - 2))
            assert rc == L.OK and scale == 1.0 and _close(got, [base ** (-2 * i / d) for i in range(d // 2)])
            # The slowest pair is slowed by the factor.
            assert got[-1] == pytest.approx(10000.0 ** (-(d - 2) / d) / 4, rel=1e-12)
    rc, got, scale = _frequencies(L, scaling=L.ROTARY_LINEAR)
    assert rc == L.OK and scale == 1.0 and _close(got, [10000.0 ** (-i / 32) / 4 for i in range(32)])
    factors = [1.0 + i for i in range(32)]
    rc, got, scale = _frequencies(L, scaling=L.ROTARY_FACTORS, factors=factors)
    assert rc == L.OK and _close(got, [10000.0 ** (-i / 32) / f for i, f in enumerate(factors)])
    assert scale == pytest.approx(math.sqrt(1 + math.log(4) / math.log(4096)), rel=1e-7)


def test_frequencies_by_parts(L):
    rc, got, scale = _frequencies(L, rotary_dim=128, scaling=L.ROTARY_PARTS, factor=8.0)
    assert rc == L.OK and scale == pytest.approx(0.1 * math.log(8) + 1, rel=1e-7)
    plain = [10000.0 ** (-i / 64) for i in range(64)]
    turns = [4096 * f / (2 * math.pi) for f in plain]
    for i, (f, g) in enumerate(zip(plain, got)):
        if turns[i] > 32 and turns[min(i + 1, 63)] > 32:       # the ramp's ends are rounded outwards
            assert _close([g], [f])
        elif turns[i] < 1 and turns[i - 1] < 1:
            assert _close([g], [f / 8])
        else:
            assert f / 8 * (1 - 1e-14) - UNIT <= g <= f * (1 + 1e-14)
    ratio = [g / f for f, g in zip(plain, got)]
    assert all(a >= b - 2e-14 for a, b in zip(ratio, ratio[1:]))      # f >= 1e-4: UNIT is 4e-15 of it


def test_frequencies_refuse(L):
    for kw, code in ((dict(rotary_dim=0), L.INVALID_ARGUMENT), (dict(rotary_dim=7), L.INVALID_ARGUMENT),
                     (dict(rotary_dim=-2), L.INVALID_ARGUMENT), (dict(rotary_dim=514), L.UNSUPPORTED),
                     (dict(scaling=5), L.UNSUPPORTED), (dict(scaling=-1), L.UNSUPPORTED),
                     (dict(base=1.0), L.INVALID_ARGUMENT), (dict(base=math.nan), L.INVALID_ARGUMENT),
                     (dict(base=math.inf), L.INVALID_ARGUMENT),
                     (dict(scaling=L.ROTARY_LINEAR, factor=0.5), L.INVALID_ARGUMENT),
                     (dict(scaling=L.ROTARY_LINEAR, factor=math.nan), L.INVALID_ARGUMENT),
                     (dict(scaling=L.ROTARY_BASE, rotary_dim=2), L.INVALID_ARGUMENT),
                     (dict(scaling=L.ROTARY_PARTS, original_len=1), L.INVALID_ARGUMENT),
                     (dict(scaling=L.ROTARY_PARTS, fast_turns=1.0), L.INVALID_ARGUMENT),
                     (dict(scaling=L.ROTARY_PARTS, slow_turns=0.0), L.INVALID_ARGUMENT),
                     (dict(scaling=L.ROTARY_FACTORS), L.INVALID_ARGUMENT),
                     (dict(scaling=L.ROTARY_FACTORS, factors=[0.5] * 32), L.INVALID_ARGUMENT),
                     (dict(scaling=L.ROTARY_FACTORS, factors=[1.0] * 32, original_len=0), L.INVALID_ARGUMENT)):
        assert _frequencies(L, **kw)[0] == code, kw
    import trainable_block_sparse_infllm_gb300 as T
    with pytest.raises(T.InfLLMv2Error):
        T.rotary_frequencies(64, scaling=T.ROTARY_FACTORS, factors=[1.0] * 31, original_len=4096)


def _rotary(L, **kw):
    fields = dict(dtype=L.BF16, tokens=4, head_dim=64, rotary_dim=64, q_heads=2, k_heads=2, interleaved=0, transpose=0,
                  scale=1.0, positions=FAKE, turns=FAKE)
    for name in ("q", "q_out", "k", "k_out"):
        fields.update({name: FAKE, name + "_token": 128, name + "_head": 64})
    fields.update(kw)
    return L.lib.infllmv2_rotary(ctypes.byref(L.RotaryArgs(**fields)), None)


def test_rotary_refuses(L):
    bad, no = L.INVALID_ARGUMENT, L.UNSUPPORTED
    assert L.lib.infllmv2_rotary(None, None) == bad
    for kw, code in ((dict(dtype=3), no), (dict(tokens=0), bad), (dict(tokens=-1), bad),
                     (dict(head_dim=8, rotary_dim=8), no), (dict(head_dim=72), no), (dict(head_dim=528), no),
                     (dict(rotary_dim=0), no), (dict(rotary_dim=24), no), (dict(rotary_dim=80), no),
                     (dict(q_heads=0), bad), (dict(k_heads=-1), bad), (dict(positions=None), bad),
                     (dict(turns=None), bad), (dict(scale=0.0), bad), (dict(scale=math.inf), bad),
                     (dict(scale=math.nan), bad), (dict(interleaved=2), bad), (dict(transpose=-1), bad)):
        assert _rotary(L, **kw) == code, kw
    for x in ("q", "k"):
        other = {x + "_out": FAKE + 4096}
        for kw, code in (({x + "_heads": 5000}, no), ({x: None}, bad), ({x + "_out": None}, bad),
                         ({x: ODD, x + "_out": ODD}, no), ({x + "_token": -128}, bad), ({x + "_token": 130}, no),
                         ({x + "_token": 1 << 58}, no), (dict(other, **{x + "_out_token": 64}), bad),
                         (dict(other, **{x + "_out_head": 0}), bad), ({x + "_out_token": 256}, bad)):
            assert _rotary(L, **kw) == code, kw
    # fp32 rows of 4 elements are 16 bytes.
    assert _rotary(L, q_token=132) == no
    assert _rotary(L, q_token=130, dtype=L.FP32) == no
    # An output that the other tensor is read from or written to.
    assert _rotary(L) == bad
    for q_out, k, k_out in ((FAKE + 4096, FAKE + 8192, FAKE), (FAKE + 4096, FAKE + 4096, FAKE + 8192),
                            (FAKE + 4096, FAKE + 8192, FAKE + 4096)):
        assert _rotary(L, q_out=q_out, k=k, k_out=k_out) == bad, (q_out, k, k_out)


# ------------------------------------------------------------------ reserve

def _reserve(L, **kw):
    names = ("page_table", "held", "free_pages", "n_free", "kv_lens", "n_new", "new_lens", "starts", "slots",
             "positions", "missing")
    fields = dict({n: FAKE + 4096 * i for i, n in enumerate(names)}, page_size=16, num_pages=10, batch=2, max_pages=4,
                  max_tokens=8)
    fields.update(kw)
    return L.lib.infllmv2_paged_reserve(ctypes.byref(L.ReserveArgs(**fields)), None)


def test_reserve_refuses(L):
    bad, no = L.INVALID_ARGUMENT, L.UNSUPPORTED
    assert L.lib.infllmv2_paged_reserve(None, None) == bad
    for kw, code in ((dict(page_size=0), bad), (dict(num_pages=0), bad), (dict(batch=0), bad),
                     (dict(max_pages=0), bad), (dict(batch=4097), no), (dict(page_size=65537), no),
                     (dict(page_size=1 << 15, max_pages=1 << 16), no), (dict(page_size=1 << 15, num_pages=1 << 16), no),
                     (dict(max_tokens=-1), bad), (dict(max_tokens=(1 << 30) + 1), no)):
        assert _reserve(L, **kw) == code, kw
    for name in ("page_table", "held", "free_pages", "n_free", "kv_lens", "n_new", "new_lens", "starts", "missing"):
        assert _reserve(L, **{name: None}) == bad, name
    for a, b in (("new_lens", "seq_lens"), ("new_lens", "held"), ("starts", "kv_lens"), ("starts", "n_new"),
                 ("starts", "seq_lens"), ("starts", "new_lens"), ("starts", "held")):
        assert _reserve(L, **{a: FAKE, b: FAKE}) == bad, (a, b)


# ------------------------------------------------------------ packed append

def _cache(L, **kw):
    strides = (2 * 64 * 128, 64 * 128, 128)
    fields = dict(dtype=L.BF16, n_kv_heads=2, head_dim=128, page_size=64, num_pages=10, k_strides=_ints64(*strides),
                  v_strides=_ints64(*strides), k_pages=FAKE, v_pages=FAKE, weights=FAKE, positions=FAKE)
    fields.update(kw)
    return L.PagedCacheStruct(**fields)


def _append(L, cache=None, tokens=4, k=FAKE, v=FAKE, strides=None, slots=FAKE, positions=FAKE):
    cache = _cache(L) if cache is None else cache
    return L.lib.infllmv2_paged_append_packed(ctypes.byref(cache), tokens, k, v,
                                              None if strides is None else _ints64(*strides), slots, positions, None)


def test_packed_append_refuses(L):
    bad, no = L.INVALID_ARGUMENT, L.UNSUPPORTED
    for kw, code in ((dict(tokens=0), bad), (dict(k=None), bad), (dict(v=None), bad), (dict(slots=None), bad),
                     (dict(k=ODD), no), (dict(v=ODD), no), (dict(positions=None), bad),
                     (dict(strides=(-256, 128, 256, 128)), bad), (dict(strides=(256, 128, 256, 132)), no),
                     (dict(strides=(256, 128, 1 << 60, 128)), no), (dict(cache=_cache(L, head_dim=32)), no),
                     (dict(cache=_cache(L, k_pages=None)), bad)):
        assert _append(L, **kw) == code, kw


# ---------------------------------------------------------------- attention

def _args(L, **kw):
    fields = dict(dtype=L.BF16, batch=2, n_kv_heads=2, group_size=4, head_dim=128, q_tokens=10, k_tokens=10, scale=0.1,
                  q=FAKE, k=FAKE, v=FAKE, q_token=1024, q_head=128, k_token=256, k_head=128, v_token=256, v_head=128,
                  q_starts=FAKE, k_starts=FAKE)
    fields.update(kw)
    return L.PackedAttnArgs(**fields)


def _forward(L, args, out=FAKE + 65536, strides=(1024, 128), lse=FAKE):
    return L.lib.infllmv2_packed_attn(None if args is None else ctypes.byref(args), out,
                                      None if strides is None else _ints64(*strides), lse, None)


GRAD_STRIDES = (1024, 128) * 3 + (256, 128) * 2


def _backward(L, args, strides=GRAD_STRIDES, ws=FAKE, ws_bytes=640, **kw):
    a = {name: FAKE + 65536 * i for i, name in enumerate(("out", "lse", "dout", "dq", "dk", "dv"), 1)}
    a.update(kw)
    return L.lib.infllmv2_packed_attn_backward(None if args is None else ctypes.byref(args), a["out"], a["lse"],
                                               a["dout"], a["dq"], a["dk"], a["dv"],
                                               None if strides is None else _ints64(*strides), ws, ws_bytes, None)


def test_structs_match_the_header(L):
    assert ctypes.sizeof(L.PackedAttnArgs) == 8 * 4 + 3 * 8 + 6 * 8 + 2 * 8
    assert ctypes.sizeof(L.RotaryArgs) == 10 * 4 + 6 * 8 + 8 * 8
    assert ctypes.sizeof(L.ReserveArgs) == 6 * 4 + 12 * 8
    assert ctypes.sizeof(L.RotaryConfig) == 2 * 4 + 2 * 8 + 2 * 4 + 2 * 8 + 8


def test_attention_refuses(L):
    bad, no = L.INVALID_ARGUMENT, L.UNSUPPORTED
    for call in (_forward, _backward):
        assert call(L, None) == bad
        for kw, code in ((dict(dtype=L.FP32), no), (dict(dtype=-1), no), (dict(head_dim=96), no), (dict(batch=0), bad),
                         (dict(batch=4097), no), (dict(n_kv_heads=0), bad), (dict(n_kv_heads=1025), no),
                         (dict(group_size=0), bad), (dict(group_size=33), no), (dict(q_tokens=0), bad),
                         (dict(k_tokens=0), bad), (dict(q_tokens=1 << 29), no), (dict(k_tokens=1 << 29), no),
                         (dict(q=None), bad), (dict(k=None), bad), (dict(v=None), bad), (dict(q_starts=None), bad),
                         (dict(q=ODD), no), (dict(k=ODD), no), (dict(v=ODD), no), (dict(scale=0.0), bad),
                         (dict(scale=-1.0), bad), (dict(scale=math.nan), bad), (dict(scale=3e38), bad),
                         (dict(q_token=-1024), bad), (dict(q_token=1028), no), (dict(q_token=1000), bad),
                         (dict(k_head=0), bad), (dict(k_token=128), bad), (dict(v_token=1 << 40), no),
                         (dict(v_head=132), no), (dict(k_starts=None, k_tokens=11), bad)):
            assert call(L, _args(L, **kw)) == code, (call.__name__, kw)
    for kw, code in ((dict(out=None), bad), (dict(out=ODD), no), (dict(out=FAKE), bad), (dict(strides=None), bad),
                     (dict(strides=(1024, 0)), bad), (dict(strides=(1024, 132)), no), (dict(strides=(512, 128)), bad)):
        assert _forward(L, _args(L), **kw) == code, kw
    for name in ("out", "lse", "dout", "dq", "dk", "dv"):
        assert _backward(L, _args(L), **{name: None}) == bad, name
        if name != "lse":
            assert _backward(L, _args(L), **{name: ODD}) == no, name
    for name in ("dq", "dk", "dv"):
        for other in (FAKE, FAKE + 65536, FAKE + 2 * 65536, FAKE + 3 * 65536):
            assert _backward(L, _args(L), **{name: other}) == bad, name
    assert _backward(L, _args(L), dq=FAKE + 5 * 65536) == bad and _backward(L, _args(L), dv=FAKE + 4 * 65536) == bad
    assert _backward(L, _args(L), strides=None) == bad
    for i in range(5):
        strides = list(GRAD_STRIDES)
        strides[2 * i + 1] = 0
        assert _backward(L, _args(L), strides=strides) == bad, i
    assert _backward(L, _args(L), ws=None) == L.WORKSPACE_TOO_SMALL
    assert _backward(L, _args(L), ws_bytes=639) == L.WORKSPACE_TOO_SMALL
    assert _backward(L, _args(L), ws=ODD) == no


def test_workspace_size(L):
    assert L.lib.infllmv2_packed_workspace_size(ctypes.byref(_args(L))) == 8 * 10 * 8
    assert L.lib.infllmv2_packed_workspace_size(ctypes.byref(_args(L, head_dim=96))) == 0
    assert L.lib.infllmv2_packed_workspace_size(None) == 0
