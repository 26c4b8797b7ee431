"""Refusals of the paged cache's entry points (no GPU needed).

Every call fails validation before anything touches the device; the fake
pointers are never dereferenced.
"""

import ctypes

import pytest

FAKE = 0x7F0000000000
ODD = FAKE + 8


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    from trainable_block_sparse_infllm_gb300 import _lib
    return _lib


def _cache(L, **kw):
    heads, page, dim = kw.get("n_kv_heads", 2), kw.get("page_size", 64), kw.get("head_dim", 128)
    strides = (heads * page * dim, page * dim, dim)
    c = L.PagedCacheStruct(dtype=L.BF16, n_kv_heads=heads, head_dim=dim, page_size=page, num_pages=10,
                           k_strides=(ctypes.c_int64 * 3)(*strides), v_strides=(ctypes.c_int64 * 3)(*strides),
                           k_pages=FAKE, v_pages=FAKE, weights=FAKE, positions=FAKE)
    for k, v in kw.items():
        setattr(c, k, (ctypes.c_int64 * 3)(*v) if k.endswith("strides") else v)
    return c


def _append(L, c, batch=2, max_pages=4, n_q=1, k=FAKE, v=FAKE, strides=None, table=FAKE, lens=FAKE):
    st = None if strides is None else (ctypes.c_int64 * 6)(*strides)
    return L.lib.infllmv2_paged_append_kv(None if c is None else ctypes.byref(c), batch, max_pages, n_q, k, v, st,
                                          table, lens, None, None, None)


def _attn(L, c, batch=2, max_pages=4, group=16, q=FAKE, table=FAKE, lens=FAKE, scale=0.1, accumulate=0, out=FAKE,
          ws=FAKE, ws_bytes=1 << 40):
    return L.lib.infllmv2_paged_attn_decode(None if c is None else ctypes.byref(c), batch, max_pages, group, q, table,
                                            lens, scale, accumulate, out, None, ws, ws_bytes, None)


def _evict(L, c, batch=2, max_pages=4, table=FAKE, lens=FAKE, budget=10, n_init=0, n_local=0, seen=None, new=FAKE,
           ws=FAKE, ws_bytes=1 << 40):
    return L.lib.infllmv2_paged_evict(None if c is None else ctypes.byref(c), batch, max_pages, table, lens, budget,
                                      n_init, n_local, seen, new, ws, ws_bytes, None)


def test_struct_matches_the_header(L):
    assert ctypes.sizeof(L.PagedCacheStruct) == 24 + 48 + 32


def test_bad_caches(L):
    for call in (_append, _attn, _evict):
        assert call(L, None) == L.INVALID_ARGUMENT
        for field, value, code in (("dtype", 2, L.UNSUPPORTED), ("dtype", -1, L.UNSUPPORTED),
                                   ("n_kv_heads", 0, L.INVALID_ARGUMENT), ("n_kv_heads", 2000, L.UNSUPPORTED),
                                   ("num_pages", 0, L.INVALID_ARGUMENT), ("page_size", 0, L.INVALID_ARGUMENT),
                                   ("k_pages", None, L.INVALID_ARGUMENT), ("v_pages", None, L.INVALID_ARGUMENT),
                                   ("k_pages", ODD, L.UNSUPPORTED), ("v_pages", ODD, L.UNSUPPORTED),
                                   ("weights", ODD, L.UNSUPPORTED), ("positions", ODD, L.UNSUPPORTED)):
            c = _cache(L)
            setattr(c, field, value)
            assert call(L, c) == code, (call.__name__, field, value)
        for kw in (dict(head_dim=32), dict(head_dim=256), dict(page_size=8), dict(page_size=24),
                   dict(page_size=65536 + 16)):
            assert call(L, _cache(L, **kw)) == L.UNSUPPORTED, kw
        good = (2 * 64 * 128, 64 * 128, 128)
        for bad, code in (((0, 64 * 128, 128), L.INVALID_ARGUMENT), ((good[0], -1, 128), L.INVALID_ARGUMENT),
                          ((good[0], good[1], 132), L.UNSUPPORTED),          # not 16-byte rows
                          ((good[0], good[1], 64), L.INVALID_ARGUMENT),      # rows overlap
                          ((good[1], good[1], 128), L.INVALID_ARGUMENT),
                          ((1 << 40, good[1], 128), L.UNSUPPORTED)):
            for which in ("k_strides", "v_strides"):
                assert call(L, _cache(L, **{which: bad})) == code, bad
        assert call(L, _cache(L, num_pages=1 << 25)) == L.UNSUPPORTED             # 2^31 slots in the pool
        assert call(L, _cache(L), batch=0) == L.INVALID_ARGUMENT
        assert call(L, _cache(L), batch=4097) == L.UNSUPPORTED
        assert call(L, _cache(L, n_kv_heads=32), batch=4096) == L.UNSUPPORTED      # 131072 units
        assert call(L, _cache(L), max_pages=0) == L.INVALID_ARGUMENT
        assert call(L, _cache(L), max_pages=1 << 25) == L.UNSUPPORTED              # 2^31 slots
        assert call(L, _cache(L), table=None) == L.INVALID_ARGUMENT
        assert call(L, _cache(L), lens=None) == L.INVALID_ARGUMENT


def test_append_arguments(L):
    c = _cache(L)
    assert _append(L, c, n_q=0) == L.INVALID_ARGUMENT
    assert _append(L, c, n_q=4 * 64 + 1) == L.INVALID_ARGUMENT
    assert _append(L, c, k=None) == L.INVALID_ARGUMENT
    assert _append(L, c, v=ODD) == L.UNSUPPORTED
    assert _append(L, c, n_q=2, strides=(512, 256, 128, 512, 256, 130)) == L.UNSUPPORTED
    assert _append(L, c, n_q=2, strides=(512, 256, 128, 512, -256, 128)) == L.INVALID_ARGUMENT


def test_attention_arguments(L):
    c = _cache(L)
    assert _attn(L, c, group=0) == L.INVALID_ARGUMENT
    assert _attn(L, c, group=33) == L.UNSUPPORTED
    assert _attn(L, c, q=None) == L.INVALID_ARGUMENT
    assert _attn(L, c, out=ODD) == L.UNSUPPORTED
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _attn(L, c, scale=scale) == L.INVALID_ARGUMENT
    assert _attn(L, c, accumulate=2) == L.INVALID_ARGUMENT
    assert _attn(L, _cache(L, weights=None), accumulate=1) == L.INVALID_ARGUMENT
    need = L.lib.infllmv2_paged_workspace_size(ctypes.byref(c), 2, 4, 16, L.OP_PAGED_DECODE)
    assert need >= 2 * 2 * 16 * 4 * 64 * 4                 # a score per head and slot
    bare = _cache(L, weights=None, positions=None)
    assert 0 < L.lib.infllmv2_paged_workspace_size(ctypes.byref(bare), 2, 4, 16, L.OP_PAGED_DECODE) < need
    assert _attn(L, c, ws=None) == L.WORKSPACE_TOO_SMALL
    assert _attn(L, c, ws_bytes=need - 1) == L.WORKSPACE_TOO_SMALL
    assert _attn(L, c, ws=ODD) == L.UNSUPPORTED


def test_evict_arguments(L):
    c = _cache(L)
    assert _evict(L, _cache(L, weights=None)) == L.INVALID_ARGUMENT
    assert _evict(L, _cache(L, positions=None)) == L.INVALID_ARGUMENT
    assert _evict(L, c, budget=0) == L.INVALID_ARGUMENT
    assert _evict(L, c, n_init=-1) == L.INVALID_ARGUMENT
    assert _evict(L, c, n_local=-1) == L.INVALID_ARGUMENT
    assert _evict(L, c, budget=10, n_init=6, n_local=5) == L.INVALID_ARGUMENT
    assert _evict(L, c, budget=10, n_init=2 ** 31 - 1, n_local=2 ** 31 - 1) == L.INVALID_ARGUMENT
    assert _evict(L, c, new=None) == L.INVALID_ARGUMENT
    assert _evict(L, c, seen=FAKE + 64, new=FAKE + 64) == L.INVALID_ARGUMENT
    assert _evict(L, c, max_pages=8193) == L.UNSUPPORTED           # past 524288 slots
    need = L.lib.infllmv2_paged_workspace_size(ctypes.byref(c), 2, 4, 0, L.OP_PAGED_EVICT)
    assert need > 0
    assert _evict(L, c, ws_bytes=need - 1) == L.WORKSPACE_TOO_SMALL
    assert _evict(L, c, ws=None) == L.WORKSPACE_TOO_SMALL


def test_workspace_size_of_bad_arguments_is_zero(L):
    size = L.lib.infllmv2_paged_workspace_size
    c = _cache(L)
    assert size(None, 2, 4, 16, L.OP_PAGED_DECODE) == 0
    assert size(ctypes.byref(c), 0, 4, 16, L.OP_PAGED_DECODE) == 0
    assert size(ctypes.byref(c), 2, 4, 0, L.OP_PAGED_DECODE) == 0
    assert size(ctypes.byref(c), 2, 4, 16, 99) == 0
    assert size(ctypes.byref(c), 2, 8193, 16, L.OP_PAGED_EVICT) == 0


def test_python_binding_refuses(L):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    k = torch.zeros((4, 2, 64, 128), dtype=torch.bfloat16)
    with pytest.raises(T.InfLLMv2Error, match="CUDA"):
        T.PagedCache(k, k.clone())
    with pytest.raises(T.InfLLMv2Error, match="one shape"):
        T.PagedCache(k, k[:3])
    with pytest.raises(T.InfLLMv2Error, match="bf16"):
        T.PagedCache(k.float(), k.float())
    with pytest.raises(T.InfLLMv2Error, match="bf16"):
        T.PagedCache(k, k.half())


def _binding_on_cpu(monkeypatch, calls):
    """The binding with a cache of CPU tensors and a recorder in place of the C append: (token rows' address, strides)."""
    import torch
    from trainable_block_sparse_infllm_gb300 import paged

    class Cache(paged.PagedCache):
        def __init__(self):
            self.n_kv_heads, self.head_dim, self.dtype, self.index = 2, 64, torch.bfloat16, -1
            self.device, self._ref = torch.device("cpu"), None
            self._new_strides = (None, None)

    def append(ref, batch, max_pages, n_q, k, v, strides, *rest):
        calls.append((k, tuple(strides)))
        return 0
    monkeypatch.setattr(paged, "_append", append)
    monkeypatch.setattr(paged, "_stream", lambda cache, stream: 0)
    table, lens = torch.zeros((2, 4), dtype=torch.int32), torch.full((2,), 8, dtype=torch.int32)
    # A prompt thread's rows are token-major, a decode thread's head-major.
    token_major = torch.zeros((2, 8, 2, 64), dtype=torch.bfloat16).transpose(1, 2)
    head_major = torch.zeros((2, 2, 1, 64), dtype=torch.bfloat16)
    rows = (token_major, head_major)
    want = {r.data_ptr(): (*r.stride()[:3], *r.stride()[:3]) for r in rows}
    return Cache, (lambda cache, r: paged.paged_append_kv(cache, r, r, table, lens)), rows, want


def test_append_passes_its_own_strides_when_another_call_comes_between(L, monkeypatch):
    """Another thread's append may run between any two steps of this one: at every look at what the cache keeps."""
    calls = []
    Cache, append, (mine, other), want = _binding_on_cpu(monkeypatch, calls)

    class Interrupted(Cache):
        inside = False

        @property
        def _new_strides(self):
            if not self.inside:
                self.inside = True
                append(self, other)
                self.inside = False
            return self.kept

        @_new_strides.setter
        def _new_strides(self, pair):
            self.kept = pair
    cache = Interrupted()
    for _ in range(3):
        append(cache, mine)
    assert calls and all(strides == want[k] for k, strides in calls)


def test_append_from_two_threads(L, monkeypatch):
    import sys
    import threading
    calls = []
    Cache, append, rows, want = _binding_on_cpu(monkeypatch, calls)
    cache = Cache()
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=lambda r=r: [append(cache, r) for _ in range(20000)]) for r in rows]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    assert len(calls) == 40000 and all(strides == want[k] for k, strides in calls)


def _rules(tmp_path):
    """The attention kernel's rules for waits that gave up, compiled for the host."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src, lib = tmp_path / "rules.cc", tmp_path / "rules.so"
    src.write_text('#include "paged_rules.h"\nextern "C" int ok(int u, int s, int l, int p, int units, int most) '
                   "{ return infllmv2::cut_in_range(u, s, l, p, units, most); }\n"
                   'extern "C" unsigned first(unsigned issued, unsigned stages, int freed) '
                   "{ return infllmv2::first_in_flight(issued, stages, freed != 0); }\n")
    csrc = os.path.join(root, "trainable_block_sparse_infllm_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", csrc, str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


def test_join_follows_no_record_out_of_the_workspace(tmp_path):
    """Whatever an unwritten record holds: a unit that is none is not written, a place that is none not read."""
    import random
    ok = _rules(tmp_path).ok
    rng = random.Random(3)
    units, most = 7, 40
    edge = [-2 ** 31, -78, -2, -1, 0, 1, 2, 6, 7, 8, 38, 39, 40, 41, 79, 80, 81, 2 ** 30, 2 ** 31 - 1]
    taken = 0
    for _ in range(200000):
        u, s, l, p = (rng.choice(edge) if rng.random() < 0.7 else rng.randrange(-3, 90) for _ in range(4))
        if not ok(u, s, l, p, units, most):
            continue
        taken += 1
        places = [p] + [2 * k for k in range(s, l + 1)]      # what the join reads for the record
        assert 0 <= u < units and len(places) == l - s + 2 >= 2
        assert 0 <= min(places) and max(places) < 2 * most and len(set(places)) == len(places)
    assert taken > 0


def _split(lens, heads, tile, ctas, cost, counter):
    """The line of tiles cut into chunks, as csrc/paged_attn.cu words it: (chunks, {unit: [(place, first, last tile)]})."""
    width = [-(-n // tile) + cost if n else 0 for n in lens]
    W = sum(width) * heads
    n = min(ctas, W)
    borders = [k * W // n for k in range(n + 1)] if n else [0]
    if counter and n and W >= 32 * n:
        A = W - W // 5
        small = max(8, (W - A + 6 * n - 1) // (6 * n))
        borders = [k * A // n for k in range(n + 1)]
        borders += list(range(A + small, W, small)) + [W]
    pieces, at, k = {}, 0, 0
    for b, w in enumerate(width):
        for h in range(heads if w else 0):
            first = at + cost
            while k + 1 < len(borders) and borders[k + 1] <= first:
                k += 1
            t = 0
            while t < w - cost:
                end = min(w - cost, borders[k + 1] - first)
                pieces.setdefault(b * heads + h, []).append((2 * k + (first + t > borders[k]), t, end))
                t = end
                if first + t >= borders[k + 1]:
                    k += 1
            at += w
    return len(borders) - 1, pieces


@pytest.mark.parametrize("lens,heads,ctas,counter", [
    ([40001], 2, 304, False), ([100 + 37 * i for i in range(60)], 8, 304, False), ([9, 0, 70000, 0, 1], 1, 152, False),
    ([20000 + 300 * i for i in range(32)], 8, 304, True), ([600] * 400, 3, 304, True), ([1 + i % 97 for i in range(4096)], 15, 304, True),
    ([0, 0, 131072, 5], 4, 152, True)])
def test_join_follows_every_record_of_a_pass(tmp_path, lens, heads, ctas, counter):
    ok = _rules(tmp_path).ok
    chunks, pieces = _split(lens, heads, 64, ctas, 2, counter)
    most = 7 * ctas if counter else ctas
    assert chunks <= most
    seen = set()
    cut = 0
    for unit, parts in pieces.items():
        assert [p[1] for p in parts[1:]] == [p[2] for p in parts[:-1]] and parts[0][1] == 0
        if len(parts) == 1:
            continue
        cut += 1
        second, last = parts[1][0] // 2, parts[-1][0] // 2
        assert [p[0] for p in parts[1:]] == [2 * k for k in range(second, last + 1)]
        assert ok(unit, second, last, parts[0][0], len(lens) * heads, most)
        assert not seen & {p[0] for p in parts}              # no two pieces at one place
        seen |= {p[0] for p in parts}
    assert cut > 0


@pytest.mark.parametrize("stages", [3, 6])
def test_the_loading_warp_waits_for_every_copy_in_flight(tmp_path, stages):
    """Whoever gave up: each copy that may not have landed is waited for, and no wait is for a phase gone by."""
    first = _rules(tmp_path).first
    for issued in range(0, 5 * stages + 1):
        for freed in (0, 1):
            # Known to have landed: what was consumed before the last copy's stage was taken again, and
            # (freed: the end's stage) one more; the computing warps may have left with all others on their way.
            known = max(0, issued - stages + freed)
            waited = list(range(first(issued, stages, freed), issued))
            assert set(range(known, issued)) <= set(waited)
            for landed in range(known, issued + 1):          # copies land in order here
                # Phases that each stage's barrier has completed; the end arrives on the next one's.
                phases = [sum(1 for i in range(landed) if i % stages == s) for s in range(stages)]
                if freed:
                    phases[issued % stages] += 1
                for i in waited:
                    passes = phases[i % stages] % 2 != (i // stages) % 2
                    assert passes == (i < landed)


def test_a_scale_past_fp32_in_base_2_is_refused(L):
    """scale log2(e) has to be finite as well: beyond that every score would come out NaN."""
    c = _cache(L)
    for scale in (2.4e38, 3.4e38):
        assert _attn(L, c, scale=scale) == L.INVALID_ARGUMENT
    assert _attn(L, c, scale=2.3e38, ws_bytes=0) == L.WORKSPACE_TOO_SMALL      # past the check


def test_strides_that_pass_64_bits_are_refused(L):
    """Extents are computed in 64 bits: strides whose rows would wrap around must not look as if they did not overlap."""
    far = (1 << 39) - 8
    for which in ("k_strides", "v_strides"):
        c = _cache(L, num_pages=(1 << 27) - 1, page_size=16, **{which: (far, 16 * 128, 128)})     # 2^66 elements
        for call in (_append, _attn, _evict):
            assert call(L, c) == L.UNSUPPORTED
