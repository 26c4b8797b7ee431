"""The paged cache's operators against plain 64-bit forms (GPU).

tests/paged_helpers.py derives the tolerances.  Unused pages, unused rows and
unused table entries hold NaN or impossible page numbers in every test.
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


def _attn(pool, group, accumulate=True, scale=None, want_lse=True, q=None, lens=None, stream=None, ws=None):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    batch = pool.table.shape[0]
    q = pool.normal(batch, 1, pool.heads * group, pool.dim) if q is None else q
    out = torch.full_like(q, float("nan"))
    lse = torch.full((batch, 1, pool.heads * group), float("nan"), device=pool.dev) if want_lse else None
    ws = pool.workspace(T.OP_PAGED_DECODE, group) if ws is None else ws
    T.paged_attn_decode(pool.cache, q, pool.table, pool.lens if lens is None else lens, out, lse, scale=scale,
                        accumulate=accumulate, workspace=ws, stream=stream)
    return q, out, lse


EDGES = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 200, 0, 333]

ATTN = [
    # dtype, layout, heads, group, dim, page, lens
    ("bf16", "hnd", 2, 16, 128, 64, EDGES),
    ("bf16", "nhd", 3, 5, 128, 16, EDGES),
    ("fp16", "pair", 1, 8, 128, 32, EDGES),
    ("fp16", "hnd", 4, 1, 64, 48, EDGES),
    ("bf16", "nhd", 2, 32, 128, 64, EDGES),
    ("fp16", "nhd", 1, 17, 64, 128, EDGES),
    ("bf16", "pair", 2, 9, 64, 256, EDGES),
    ("bf16", "hnd", 1, 7, 128, 16, [1]),
    ("bf16", "hnd", 1, 16, 128, 64, [0, 0, 0]),
    ("bf16", "hnd", 2, 16, 128, 64, [40001]),            # every SM holds a piece of one unit
    ("fp16", "nhd", 2, 4, 128, 16, [20000, 3, 9999]),
    ("fp16", "hnd", 1, 32, 64, 80, [30011, 0, 1]),
    ("bf16", "pair", 8, 2, 64, 32, [100 + 37 * i for i in range(60)]),   # units cut and whole, several per CTA
]


@pytest.mark.parametrize("dtype,layout,heads,group,dim,page,lens", ATTN)
def test_attention(dev, dtype, layout, heads, group, dim, page, lens):
    from paged_helpers import Pool, check_attend
    pool = Pool(dev, dtype, layout, heads, dim, page, lens, seed=len(lens) + group)
    before = pool.weights.clone()
    k, v = pool.k.clone(), pool.v.clone()
    q, out, lse = _attn(pool, group)
    assert _status() == 0
    check_attend(pool, q, out, lse, before, dim ** -0.5)
    import torch
    for now, then in ((pool.k, k), (pool.v, v)):   # the pages are only read
        assert torch.equal(now.contiguous().view(torch.int16), then.contiguous().view(torch.int16))


@pytest.mark.parametrize("dtype,layout,heads,group,dim,page,lens,spare", [
    # A capacity at which the end of the line goes out in small chunks: by unit, and (more units than chunks) by chunk.
    ("bf16", "hnd", 4, 2, 128, 64, [16000, 0, 1, 9999] + [8000 + 77 * i for i in range(16)], 600),
    ("fp16", "nhd", 16, 1, 64, 32, [100 + 13 * (i % 97) for i in range(160)], 200),
    ("bf16", "pair", 2, 32, 128, 256, [20000 + 999 * i for i in range(9)], 600),
    # The same capacity, but too few slots in use for that.
    ("bf16", "hnd", 4, 2, 128, 64, [5, 640, 0, 64] * 5, 600),
    ("bf16", "hnd", 4, 2, 128, 64, [0] * 20, 600),
])
@pytest.mark.parametrize("accumulate", [False, True])
def test_long_lines(dev, dtype, layout, heads, group, dim, page, lens, spare, accumulate):
    from paged_helpers import Pool, check_attend
    pool = Pool(dev, dtype, layout, heads, dim, page, lens, spare_entries=spare, seed=21, metadata=accumulate)
    before = pool.weights.clone() if accumulate else None
    q, out, lse = _attn(pool, group, accumulate=accumulate)
    assert _status() == 0
    check_attend(pool, q, out, lse, before, dim ** -0.5)


@pytest.mark.parametrize("dtype,heads,group,dim,page,lens", [
    ("bf16", 2, 16, 128, 64, [1000]), ("fp16", 1, 8, 128, 16, [512, 1, 0, 300]), ("bf16", 4, 3, 64, 48, [2000, 129]),
    ("bf16", 2, 32, 128, 64, [1100, 5]), ("fp16", 8, 20, 64, 128, [640, 1]), ("bf16", 4, 16, 128, 32, [2500, 64, 65, 3000]),
])
@pytest.mark.parametrize("accumulate", [False, True])
def test_clusters(dev, dtype, heads, group, dim, page, lens, accumulate):
    """Few units of a few thousand slots: each by a cluster that joins its pieces itself; again with a bad page."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from paged_helpers import Pool, attend, check_attend
    pool = Pool(dev, dtype, "nhd", heads, dim, page, lens, seed=26, metadata=accumulate)
    before = pool.weights.clone() if accumulate else None
    q, out, lse = _attn(pool, group, accumulate=accumulate)
    assert _status() == 0
    check_attend(pool, q, out, lse, before, dim ** -0.5)
    last = (lens[0] - 1) // page
    pool.table[0, last] = pool.k.shape[0]            # the first sequence's last page is absent
    left = torch.tensor([last * page] + lens[1:])
    before = pool.weights.clone() if accumulate else None
    q, out, lse = _attn(pool, group, accumulate=accumulate)
    assert _status() == T.DEVICE_BAD_PAGE
    check_attend(pool, q, out, lse, before, dim ** -0.5, lens=left)


@pytest.mark.parametrize("heads,group,dim,lens", [(2, 16, 128, [256, 255, 1, 0, 129]), (8, 4, 64, [17 * i % 257 for i in range(90)]),
                                                  (1, 32, 128, [200, 256, 33])])
@pytest.mark.parametrize("accumulate", [False, True])
def test_short_caches_in_one_launch(dev, heads, group, dim, lens, accumulate):
    """A page table of at most 256 slots: no unit is cut."""
    from paged_helpers import Pool, check_attend
    pool = Pool(dev, "bf16", "hnd", heads, dim, 64, lens, spare_entries=0, seed=22, metadata=accumulate)
    assert pool.max_pages * 64 <= 256
    before = pool.weights.clone() if accumulate else None
    q, out, lse = _attn(pool, group, accumulate=accumulate)
    assert _status() == 0
    check_attend(pool, q, out, lse, before, dim ** -0.5)


def test_a_pool_past_32_bit_offsets(dev):
    """Pages whose rows lie beyond 2^32 elements of the pool, for all three operators."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from paged_helpers import Pool, check_attend, evict_plain
    small = Pool(dev, "bf16", "hnd", 8, 128, 64, [300, 64, 1], seed=23)
    P = 70000                                    # 70000 * 8 * 64 * 128 elements: 4.6e9
    shift = P - small.k.shape[0]
    k = torch.empty((P, 8, 64, 128), dtype=torch.bfloat16, device=dev)
    v = torch.empty_like(k)
    weights, positions = torch.zeros((P, 8, 64), device=dev), torch.zeros((P, 8, 64), dtype=torch.int32, device=dev)
    k[shift:], v[shift:], weights[shift:], positions[shift:] = small.k, small.v, small.weights, small.positions
    big = T.PagedCache(k, v, weights, positions)
    table = torch.where((small.table >= 0) & (small.table < P), small.table + shift, small.table)
    q = small.normal(3, 1, 32, 128)
    out, lse = torch.empty_like(q), torch.empty((3, 1, 32), device=dev)
    before = small.weights.clone()
    T.paged_attn_decode(big, q, table, small.lens, out, lse, accumulate=True,
                        workspace=T.alloc_paged_workspace(big, table, T.OP_PAGED_DECODE, 4))
    assert _status() == 0
    small.weights.copy_(weights[shift:])
    check_attend(small, q, out, lse, before, 128 ** -0.5)
    k_new = small.normal(3, 8, 1, 128)
    T.paged_append_kv(big, k_new, k_new, table, small.lens)
    for b, n in enumerate(small.lens.tolist()):
        at, row = small.places(b, n, n - 1)
        small.k[at, :, row] = k_new[b].transpose(0, 1)
        small.v[at, :, row] = k_new[b].transpose(0, 1)
        small.weights[at, :, row] = 0.0
        small.positions[at, :, row] = n - 1
    want = evict_plain(small, 100)
    new = torch.empty_like(small.lens)
    T.paged_evict(big, table, small.lens, new, 100, workspace=T.alloc_paged_workspace(big, table, T.OP_PAGED_EVICT))
    assert _status() == 0
    small.k, small.v, small.weights, small.positions = k[shift:], v[shift:], weights[shift:], positions[shift:]
    _check_evict(small, want, new)


def test_two_streams_at_once(dev):
    """Two calls that overlap, each with a workspace of its own."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from paged_helpers import Pool, check_attend
    pools = [Pool(dev, "bf16", "hnd", 2, 128, 64, [30000, 500], seed=24 + i) for i in range(2)]
    qs = [p.normal(2, 1, 32, 128) for p in pools]
    before = [p.weights.clone() for p in pools]
    outs = [(torch.empty_like(q), torch.empty((2, 1, 32), device=dev)) for q in qs]
    wss = [p.workspace(T.OP_PAGED_DECODE, 16) for p in pools]
    streams = [torch.cuda.Stream() for _ in pools]
    torch.cuda.synchronize()
    for p, q, (out, lse), ws, st in zip(pools, qs, outs, wss, streams):
        T.paged_attn_decode(p.cache, q, p.table, p.lens, out, lse, accumulate=True, workspace=ws, stream=st)
    assert _status() == 0
    for p, q, (out, lse), w in zip(pools, qs, outs, before):
        check_attend(p, q, out, lse, w, 128 ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group", [4, 12, 24])
def test_attention_without_weights_or_lse(dev, dtype, group):
    from paged_helpers import Pool, check_attend
    pool = Pool(dev, dtype, "hnd", 2, 128, 64, [70, 1000, 0, 5], seed=3, metadata=False)
    q, out, _ = _attn(pool, group, accumulate=False, want_lse=False, scale=0.3)
    assert _status() == 0
    check_attend(pool, q, out, None, None, 0.3)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_sharp_and_flat_softmax(dev, dtype):
    """One token holds nearly all the attention and a tail of 50,000 the rest: the tail is not lost."""
    import torch
    from paged_helpers import Pool, check_attend
    n = 50000
    pool = Pool(dev, dtype, "hnd", 1, 128, 64, [n, n], seed=5)
    q = torch.zeros((2, 1, 8, 128), dtype=pool.dtype, device=dev)
    q[..., 0] = 8.0
    at, row = pool.places(0, n)
    pool.k[at, :, row] = 0.0
    pool.k[at[100], 0, row[100], 0] = 24.0      # z = 17: the other tokens get e^-17 each
    pool.v[at, :, row] = 1.0
    pool.v[at[100], 0, row[100]] = 0.0          # out = the tail's share alone
    at, row = pool.places(1, n)
    pool.k[at, :, row] = 0.0                    # all equal
    before = pool.weights.clone()
    _, out, lse = _attn(pool, 8, q=q)
    assert _status() == 0
    check_attend(pool, q, out, lse, before, 128 ** -0.5)
    share = (n - 1) * math.exp(-8 * 24 / math.sqrt(128)) / (1 + (n - 1) * math.exp(-8 * 24 / math.sqrt(128)))
    assert abs(out[0].double().mean().item() / share - 1) < 2.0 ** -7


def test_large_scores(dev):
    """Scores beyond what exp can take without its maximum: +-4000."""
    from paged_helpers import Pool, check_attend
    pool = Pool(dev, "bf16", "hnd", 2, 128, 64, [500, 64, 1], seed=6)
    q = pool.normal(3, 1, 32, 128) * 1000
    before = pool.weights.clone()
    _, out, lse = _attn(pool, 16, q=q)
    assert _status() == 0
    check_attend(pool, q, out, lse, before, 128 ** -0.5)


def test_nan_and_inf_stay_in_their_sequence(dev):
    import torch
    from paged_helpers import Pool, check_attend
    pool = Pool(dev, "bf16", "hnd", 1, 128, 16, [100, 100, 100], seed=7)
    at, row = pool.places(1, 100)
    pool.k[at[50], 0, row[50], 3] = float("nan")
    before = pool.weights.clone()
    q, out, lse = _attn(pool, 16)
    assert _status() == 0
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    ok = [0, 2]
    pool.table, pool.lens = pool.table[ok].contiguous(), pool.lens[ok].contiguous()
    got = pool.weights
    at0, row0 = pool.places(0, 100)
    assert not torch.isnan(got[at0, :, row0]).any()
    check_attend(pool, q[ok], out[ok], lse[ok], None, 128 ** -0.5)
    assert before.shape == got.shape


def test_lengths_within_the_pages(dev):
    """kv_lens shorter than what the pages hold: a row past it takes no part."""
    import torch
    from paged_helpers import Pool, check_attend
    pool = Pool(dev, "bf16", "nhd", 2, 128, 64, [640, 640, 640, 640], seed=8)
    for lens in ([0, 1, 64, 65], [639, 640, 333, 16]):
        pool.lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        before = pool.weights.clone()
        q, out, lse = _attn(pool, 16)
        assert _status() == 0
        check_attend(pool, q, out, lse, before, 128 ** -0.5)


def test_shared_pages(dev):
    """A common prefix: three sequences over the same pages, each adding its weights."""
    import torch
    from paged_helpers import Pool, attend
    pool = Pool(dev, "bf16", "hnd", 2, 128, 64, [256, 256, 256], seed=9)
    pool.table[1] = pool.table[0]
    pool.table[2, :2] = pool.table[0, :2]
    before = pool.weights.clone()
    q, out, lse = _attn(pool, 16)
    assert _status() == 0
    (o, tol), _, added = attend(pool, q, 128 ** -0.5)
    assert ((out.double() - o).abs() <= tol).all()
    want, room = before.double(), torch.zeros_like(before, dtype=torch.float64)
    for b, (x, t) in enumerate(added):
        at, row = pool.places(b, 256)
        want[at, :, row] += x
        room[at, :, row] += t + 3 * 2.0 ** -24 * want[at, :, row].abs()
    used = ~torch.isnan(want)
    assert ((pool.weights.double() - want).abs() <= room)[used].all()


def test_bad_lengths_and_pages(dev):
    """A length or a page that cannot be is reported and read nowhere; other sequences are not disturbed."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from paged_helpers import Pool, attend, check_attend
    pool = Pool(dev, "bf16", "hnd", 2, 128, 64, [200, 200, 200], seed=10)
    good = pool.lens.clone()
    pool.lens = torch.tensor([200, -1, pool.max_pages * 64 + 1], dtype=torch.int32, device=dev)
    q, out, lse = _attn(pool, 16, accumulate=False)
    assert _status() == T.DEVICE_BAD_KV_LEN
    pool.lens = torch.tensor([200, 0, 0], dtype=torch.int32, device=dev)
    check_attend(pool, q, out, lse, None, 128 ** -0.5)
    pool.lens = good
    for wrong in (-1, -2, pool.k.shape[0], 2 ** 31 - 1):
        keep = pool.table.clone()
        pool.table[1, 1] = wrong                       # slots 64..127 are absent
        before = pool.weights.clone()
        q, out, lse = _attn(pool, 16)
        assert _status() == T.DEVICE_BAD_PAGE
        at, row = (torch.cat(x) for x in zip(pool.places(0, 200), pool.places(2, 200)))
        assert not torch.equal(pool.weights[at, :, row], before[at, :, row])
        # The plain form over the slots that are there.
        k = pool.table
        pool.table = keep.clone()
        pool.table[1, 1], pool.table[1, 2], pool.table[1, 3] = keep[1, 2], keep[1, 3], -1
        (o, tol), (z, ztol), _ = attend(pool, q, 128 ** -0.5, torch.tensor([200, 136, 200]))
        assert ((out.double() - o).abs() <= tol).all() and ((lse.double() - z).abs() <= ztol).all()
        at, row = pool.table[1].long()[:1].expand(64), torch.arange(64, device=dev)
        assert (pool.weights[at, :, row] > before[at, :, row]).all()
        gone = keep[1, 1].long().expand(64)
        assert torch.equal(pool.weights[gone, :, row], before[gone, :, row])
        assert k is not pool.table
        pool.table = keep


def test_stream_and_graph(dev):
    """Enqueued on a stream of its own and captured: replays read the inputs and lengths of their time."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from paged_helpers import Pool, check_attend
    pool = Pool(dev, "bf16", "hnd", 2, 128, 64, [700, 90, 2000], seed=11)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    before = pool.weights.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q, out, lse = _attn(pool, 16)
    side.synchronize()
    assert _status() == 0
    check_attend(pool, q, out, lse, before, 128 ** -0.5)
    ws = pool.workspace(T.OP_PAGED_DECODE, 16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        T.paged_attn_decode(pool.cache, q, pool.table, pool.lens, out, lse, accumulate=True, workspace=ws)
    for lens in ([700, 90, 2000], [1, 0, 1999]):
        pool.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(pool.normal(*q.shape))
        before = pool.weights.clone()
        graph.replay()
        assert _status() == 0
        check_attend(pool, q, out, lse, before, 128 ** -0.5)


def test_two_graphs_share_a_workspace(dev):
    """Captured with one workspace and replayed in turn on one stream: nothing is kept from one to the next."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from paged_helpers import Pool, check_attend
    pools = [Pool(dev, "bf16", "hnd", 2, 128, 64, lens, seed=30 + i)
             for i, lens in enumerate(([9000, 90, 2000], [1, 12000, 0]))]
    ws = max((p.workspace(T.OP_PAGED_DECODE, 16) for p in pools), key=lambda w: w.numel())
    qs = [p.normal(3, 1, 32, 128) for p in pools]
    outs = [(torch.empty_like(q), torch.empty((3, 1, 32), device=dev)) for q in qs]
    graphs = []
    for p, q, (out, lse) in zip(pools, qs, outs):
        T.paged_attn_decode(p.cache, q, p.table, p.lens, out, lse, accumulate=True, workspace=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            T.paged_attn_decode(p.cache, q, p.table, p.lens, out, lse, accumulate=True, workspace=ws)
    before = [p.weights.clone() for p in pools]
    for _ in range(3):
        for p, w in zip(pools, before):
            p.weights.copy_(w)
        for g in graphs:
            g.replay()
    assert _status() == 0
    for p, q, (out, lse), w in zip(pools, qs, outs, before):
        check_attend(p, q, out, lse, w, 128 ** -0.5)


@pytest.mark.parametrize("lens,budget", [([300, 64, 1, 777], 64), ([40000, 9000], 5000), ([4097, 4096], 4096)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_in_a_graph(dev, lens, budget, in_place):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from paged_helpers import Pool, evict_plain
    pool = Pool(dev, "bf16", "hnd", 2, 64, 64, lens, seed=32)
    start = [t.clone() for t in (pool.k, pool.v, pool.weights, pool.positions, pool.lens)]
    want = evict_plain(pool, budget, 2, 9)
    new = pool.lens if in_place else torch.empty_like(pool.lens)
    ws = pool.workspace(T.OP_PAGED_EVICT)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        T.paged_evict(pool.cache, pool.table, pool.lens, new, budget, 2, 9, workspace=ws)
    for _ in range(2):
        for t, was in zip((pool.k, pool.v, pool.weights, pool.positions, pool.lens), start):
            t.copy_(was)
        graph.replay()
        assert _status() == 0
        _check_evict(pool, want, new)


def test_same_result_every_time(dev):
    import torch
    from paged_helpers import Pool
    pool = Pool(dev, "bf16", "hnd", 2, 128, 16, [5000, 90, 2000, 1], seed=12)
    first = pool.weights.clone()
    q, out, lse = _attn(pool, 16)
    after = pool.weights.clone()
    for _ in range(3):
        pool.weights.copy_(first)
        _, o, z = _attn(pool, 16, q=q)
        assert torch.equal(o.view(torch.int16), out.view(torch.int16)) and torch.equal(z, lse)
        assert torch.equal(pool.weights.view(torch.int32), after.view(torch.int32))


# ------------------------------------------------------------------ append ------

@pytest.mark.parametrize("dtype,layout,heads,dim,page", [("bf16", "hnd", 2, 128, 64), ("fp16", "nhd", 3, 64, 48),
                                                         ("bf16", "pair", 1, 128, 16), ("bf16", "hnd", 8, 64, 128)])
@pytest.mark.parametrize("lens,new", [([1, 2, 64, 65], None), ([5, 300, 64, 17], [5, 300, 1, 0]),
                                      ([1000, 130, 1, 70], [999, 130, 0, 69])])
@pytest.mark.parametrize("strided", [False, True])
def test_append(dev, dtype, layout, heads, dim, page, lens, new, strided):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from paged_helpers import Pool
    pool = Pool(dev, dtype, layout, heads, dim, page, lens, seed=13)
    n_new = [1] * len(lens) if new is None else new
    most = max(n_new) if new is None else max(n_new) + 3       # rows behind the last new token are not read
    batch = len(lens)
    k_new, v_new = (pool.normal(batch, most, heads, dim).transpose(1, 2) for _ in range(2))
    if not strided:
        k_new, v_new = k_new.contiguous(), v_new.contiguous()
    seen = pool.lens + torch.arange(batch, device=dev, dtype=torch.int32) * 10 if new else None
    want = [t.clone() for t in (pool.k, pool.v, pool.weights, pool.positions)]
    for b, n in enumerate(lens):
        at, row = pool.places(b, n, n - n_new[b])
        want[0][at, :, row] = k_new[b, :, :n_new[b]].transpose(0, 1)
        want[1][at, :, row] = v_new[b, :, :n_new[b]].transpose(0, 1)
        want[2][at, :, row] = 0.0
        last = n if seen is None else int(seen[b])
        want[3][at, :, row] = torch.arange(last - n_new[b], last, dtype=torch.int32, device=dev)[:, None]
    T.paged_append_kv(pool.cache, k_new, v_new, pool.table, pool.lens,
                      None if new is None else torch.tensor(new, dtype=torch.int32, device=dev), seen)
    assert _status() == 0
    for got, w in zip((pool.k, pool.v, pool.weights, pool.positions), want):
        bits = torch.int16 if got.element_size() == 2 else torch.int32
        assert torch.equal(got.contiguous().view(bits), w.contiguous().view(bits))


def test_append_bad_inputs_touch_nothing(dev):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from paged_helpers import Pool
    pool = Pool(dev, "bf16", "hnd", 2, 128, 64, [100, 100, 100, 100], seed=14)
    was = [t.clone() for t in (pool.k, pool.v, pool.weights, pool.positions)]
    k = pool.normal(4, 2, 4, 128)
    cap = pool.max_pages * 64

    def same():
        return all(torch.equal(a.view(torch.int32), b.view(torch.int32))
                   for a, b in zip((pool.k, pool.v, pool.weights, pool.positions), was))
    lens = torch.tensor([3, -1, cap + 1, 0], dtype=torch.int32, device=dev)
    T.paged_append_kv(pool.cache, k, k, pool.table, lens)
    assert _status() == T.DEVICE_BAD_KV_LEN and same()
    n_new = torch.tensor([-1, 5, 6, 1000], dtype=torch.int32, device=dev)
    T.paged_append_kv(pool.cache, k, k, pool.table, pool.lens, n_new)
    assert _status() == T.DEVICE_BAD_KV_LEN and same()
    pool.table[:, 1] = torch.tensor([-1, pool.k.shape[0], 2 ** 31 - 1, -77], dtype=torch.int32)
    T.paged_append_kv(pool.cache, k, k, pool.table, pool.lens)
    assert _status() == T.DEVICE_BAD_PAGE and same()


def test_append_from_pinned_host(dev):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from paged_helpers import Pool
    pool = Pool(dev, "fp16", "hnd", 2, 128, 64, [10, 65], seed=15, metadata=False)
    k, v = (pool.normal(2, 2, 1, 128).cpu().pin_memory() for _ in range(2))
    T.paged_append_kv(pool.cache, k, v, pool.table, pool.lens)
    assert _status() == 0
    for b, n in enumerate([10, 65]):
        at, row = pool.places(b, n, n - 1)
        assert torch.equal(pool.k[at, :, row][0].cpu(), k[b, :, 0]) and torch.equal(pool.v[at, :, row][0].cpu(), v[b, :, 0])


# ---------------------------------------------------------------- eviction ------

def _evict(pool, budget, n_init=0, n_local=0, seq_lens=None, in_place=False):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    new = pool.lens if in_place else torch.full_like(pool.lens, -9)
    T.paged_evict(pool.cache, pool.table, pool.lens, new, budget, n_init, n_local, seq_lens,
                  pool.workspace(T.OP_PAGED_EVICT))
    return new


def _check_evict(pool, want, new):
    import torch
    assert new.tolist() == want[4]
    for got, w, name in zip((pool.k, pool.v, pool.weights, pool.positions), want[:4], "k v weights positions".split()):
        bits = torch.int16 if got.element_size() == 2 else torch.int32
        assert torch.equal(got.cpu().contiguous().view(bits), w.contiguous().view(bits)), name


EVICT = [
    # dtype, layout, heads, dim, page, lens, budget, n_init, n_local
    ("bf16", "hnd", 2, 128, 64, [65, 64, 63, 1, 0, 300], 64, 0, 0),
    ("bf16", "hnd", 2, 128, 64, [65, 200, 2048], 64, 4, 16),
    ("fp16", "nhd", 3, 64, 48, [1500, 47, 999], 333, 1, 100),
    ("bf16", "pair", 1, 128, 16, [4097, 4096, 2000], 1, 0, 0),
    ("bf16", "hnd", 2, 64, 32, [4097], 4096, 4, 256),
    ("fp16", "hnd", 1, 128, 256, [8000, 5000], 5000, 0, 5000),
    ("bf16", "nhd", 2, 64, 64, [20000, 12345], 8191, 64, 512),       # 4 CTAs per unit
    ("bf16", "hnd", 1, 64, 128, [140000], 70001, 100, 1000),          # 16 CTAs, 32 keys per thread
    ("bf16", "hnd", 1, 64, 64, [300000, 40], 1000, 0, 7),             # 16 CTAs, 64 keys per thread
]


@pytest.mark.parametrize("dtype,layout,heads,dim,page,lens,budget,n_init,n_local", EVICT)
@pytest.mark.parametrize("values", ["uniform", "ties", "crowded"])
def test_evict(dev, dtype, layout, heads, dim, page, lens, budget, n_init, n_local, values):
    import torch
    from paged_helpers import Pool, evict_plain
    pool = Pool(dev, dtype, layout, heads, dim, page, lens, seed=16)
    if values == "ties":
        pool.weights.mul_(4).floor_()
    elif values == "crowded":                       # nearly all in one exponent, the rest far below
        pool.weights.copy_(torch.where(pool.weights < 0.1, pool.weights * 1e-30, 1 + pool.weights * 1e-5))
    want = evict_plain(pool, budget, n_init, n_local)
    new = _evict(pool, budget, n_init, n_local, in_place=values == "ties")
    assert _status() == 0
    _check_evict(pool, want, new)


@pytest.mark.parametrize("most,budget", [(67, 40), (500, 100), (1000, 999), (2000, 700), (4000, 100)])
def test_evict_many_short(dev, most, budget):
    """More (sequence, KV head) units than the SMs hold CTAs of 512 threads."""
    from paged_helpers import Pool, evict_plain
    pool = Pool(dev, "bf16", "hnd", 8, 64, 16, [(most * (i + 1)) // 40 for i in range(40)], spare_entries=1, seed=25)
    want = evict_plain(pool, budget, 2, 7)
    new = _evict(pool, budget, 2, 7)
    assert _status() == 0
    _check_evict(pool, want, new)


def test_evict_strange_weights(dev):
    """NaN goes first, -0 ties with 0, infinities are ordinary values; positions need not be in order."""
    import torch
    from paged_helpers import Pool, evict_plain
    pool = Pool(dev, "bf16", "hnd", 2, 128, 64, [400, 130], seed=17)
    values = torch.tensor([float("nan"), 0.0, -0.0, float("inf"), -float("inf"), 1.0, -1.0, 1e-45, 3e38], device=dev)
    pick = torch.randint(0, 9, pool.weights.shape, generator=pool.gen, device=dev)
    pool.weights.copy_(values[pick])
    pool.positions.copy_(torch.randint(0, 900, pool.positions.shape, generator=pool.gen, device=dev, dtype=torch.int32))
    seen = torch.tensor([900, 880], dtype=torch.int32, device=dev)
    for budget, n_init, n_local in ((100, 20, 30), (7, 3, 4), (399, 0, 0)):
        want = evict_plain(pool, budget, n_init, n_local, seen)
        new = _evict(pool, budget, n_init, n_local, seen)
        assert _status() == 0
        _check_evict(pool, want, new)


def test_evict_leaves_a_sequence_with_a_bad_page(dev):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from paged_helpers import Pool, evict_plain
    for cap_lens in ([300, 300, 300], [20000, 20000, 20000]):      # one CTA per unit, and a cluster
        pool = Pool(dev, "bf16", "hnd", 2, 64, 64, cap_lens, seed=18)
        n = cap_lens[0]
        keep = pool.lens.clone()
        pool.lens = torch.tensor([n, 0, n], dtype=torch.int32, device=dev)
        want = list(evict_plain(pool, 100))
        want[4] = [100, n, 100]
        pool.lens = keep
        pool.table[1, n // 64] = pool.k.shape[0]
        new = _evict(pool, 100)
        assert _status() == T.DEVICE_BAD_PAGE
        _check_evict(pool, want, new)
        pool.lens = torch.tensor([-3, 50, pool.max_pages * 64 + 1], dtype=torch.int32, device=dev)
        new = _evict(pool, 100)
        assert _status() == T.DEVICE_BAD_KV_LEN
        want[4] = [0, 50, 0]
        _check_evict(pool, want, new)


# --------------------------------------------------------------- together ------

@pytest.mark.parametrize("dtype,layout,group", [("bf16", "hnd", 16), ("fp16", "nhd", 3)])
def test_decode_loop_under_a_budget(dev, dtype, layout, group):
    """Prompts in, then steps of append, attention and (every fourth) eviction, the step captured as a graph;
    against a plain cache of lists that evicts by the library's own weights."""
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from paged_helpers import Pool, check_attend, evict_plain
    heads, dim, page, budget = 2, 128, 16, 96
    prompts = [90, 200, 1, 0]
    pool = Pool(dev, dtype, layout, heads, dim, page, [budget + 140] * 4, seed=19)
    pool.weights.fill_(float("nan"))
    seen = torch.tensor(prompts, dtype=torch.int32, device=dev)
    pool.lens = seen.clone()
    k, v = pool.normal(4, heads, max(prompts), dim), pool.normal(4, heads, max(prompts), dim)
    T.paged_append_kv(pool.cache, k, v, pool.table, pool.lens, n_new=seen, seq_lens=seen)
    k_new, v_new = pool.normal(4, heads, 1, dim), pool.normal(4, heads, 1, dim)
    q = pool.normal(4, 1, heads * group, dim)
    out, lse = torch.empty_like(q), torch.empty((4, 1, heads * group), device=dev)
    ws = pool.workspace(T.OP_PAGED_DECODE, group)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.lens.add_(1)
        seen.add_(1)
        T.paged_append_kv(pool.cache, k_new, v_new, pool.table, pool.lens, seq_lens=seen)
        T.paged_attn_decode(pool.cache, q, pool.table, pool.lens, out, lse, accumulate=True, workspace=ws)
    for step in range(12):
        k_new.copy_(pool.normal(*k_new.shape))
        v_new.copy_(pool.normal(*v_new.shape))
        q.copy_(pool.normal(*q.shape))
        before = pool.weights.clone()
        for b, n in enumerate(pool.lens.tolist()):     # what the append will do to the weights
            at, row = pool.places(b, n + 1, n)
            before[at, :, row] = 0.0
        graph.replay()
        assert _status() == 0
        for b, n in enumerate(pool.lens.tolist()):
            at, row = pool.places(b, n, n - 1)
            assert torch.equal(pool.k[at, :, row][0], k_new[b, :, 0])
            assert (pool.positions[at, :, row] == int(seen[b]) - 1).all()
        check_attend(pool, q, out, lse, before, dim ** -0.5)
        if step % 4 == 3:
            want = evict_plain(pool, budget, 4, 16, seen)
            _evict(pool, budget, 4, 16, seen, in_place=True)
            assert _status() == 0
            _check_evict(pool, want, pool.lens)
            for b, n in enumerate(pool.lens.tolist()):  # what must stay has stayed
                at, row = pool.places(b, n)
                for h in range(heads):
                    have = set(pool.positions[at, h, row].tolist())
                    total = int(seen[b])
                    assert len(have) == n
                    assert set(range(min(4, total))) | set(range(max(0, total - 16), total)) <= have


# ------------------------------------------------------------ large scores ------

HUGE = {"fp16": (60000.0, [60000, 45024, 52000, 38016, 47008, 64992, 35008, 57984]),
        "bf16": (163840.0, [163840, 204800, 139264, 188416, 344064, 155648, 237568, 253952])}


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group", [(128, 8), (128, 16), (64, 24)])
@pytest.mark.parametrize("n,spare", [(200, 0), (300, 2), (5000, 2)])      # uncut, clusters, joined
def test_scores_of_any_finite_size(dev, dtype, dim, group, n, spare):
    """Scores of 10^8 and more, exact in fp32: equal ones share the attention, smaller ones get none.

    One dimension holds all of q and k, so a score is one exact product.  p is then 1 / (number of largest
    scores) or 0: what is left of the helper's tolerances is 2^-16 + 2^-19 of the magnitudes and the output's
    rounding; for lse three roundings of relative 2^-24 and the logarithm's, below 2^-20 |lse| + 2^-20.
    """
    import torch
    from paged_helpers import Pool
    q0, keys = HUGE[dtype]
    batch = len(keys)
    pool = Pool(dev, dtype, "hnd", 1, dim, 64, [n] * batch, spare_entries=spare, seed=40, metadata=False)
    q = torch.zeros((batch, 1, group, dim), dtype=pool.dtype, device=dev)
    q[..., 0] = q0
    scale = dim ** -0.5
    want = torch.empty((batch, dim), dtype=torch.float64, device=dev)
    mag = torch.empty_like(want)
    top = torch.arange(n, device=dev) % 3 != 1
    for b, key in enumerate(keys):
        at, row = pool.places(b, n)
        pool.k[at, :, row] = 0.0
        pool.k[at, 0, row, 0] = torch.where(top, float(key), key * 0.5).to(pool.dtype)
        v = pool.v[at, 0, row].double()[top]
        want[b], mag[b] = v.mean(dim=0), v.abs().mean(dim=0)
    _, out, lse = _attn(pool, group, accumulate=False, q=q)
    assert _status() == 0
    info = torch.finfo(pool.dtype)
    tol = (2.0 ** -16 + 2.0 ** -19) * mag + info.eps / 2 * 1.001 * want.abs() + info.tiny * info.eps / 2
    assert torch.isfinite(out).all()
    assert ((out[:, 0].double() - want[:, None]).abs() <= tol[:, None]).all()
    z = q0 * torch.tensor(keys, dtype=torch.float64, device=dev) * scale + math.log(int(top.sum()))
    assert ((lse[:, 0].double() - z[:, None]).abs() <= 2.0 ** -20 * z[:, None].abs() + 2.0 ** -20).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group", [(128, 4), (64, 16), (128, 20)])
@pytest.mark.parametrize("n,spare", [(200, 0), (1000, 2), (5000, 2)])     # uncut, clusters, joined
def test_weights_of_large_scores(dev, dtype, dim, group, n, spare):
    """Scores around 4000 to 6000 that are exact in fp32: a call's weights are the softmax's and sum to the heads.

    Two dimensions hold q and k: an offset of about 45,000 and a whole number in [-64, 64), so z - m is exact.
    Relative errors in units of 2^-24: the scale in base 2 and its product, 3 |x| ln 2 < 48 for |x| < 23.1, in a
    slot's term and again in the sum it is divided by; 4 for each exp2, merges included, 20 in all; fewer than 80
    additions in a row in the sum; 32 over the heads; the division and products, 4.  Together below 256, 2^-16.
    """
    import torch
    from paged_helpers import Pool
    heads, batch = 2, 2
    pool = Pool(dev, dtype, "nhd", heads, dim, 64, [n] * batch, spare_entries=spare, seed=41)
    q = torch.zeros((batch, 1, heads * group, dim), dtype=pool.dtype, device=dev)
    q[..., 0] = 200.0 + torch.arange(heads * group, device=dev) % 50      # each head an lse of its own
    q[..., 1] = 8.0
    scale = float(torch.tensor(dim ** -0.5, dtype=torch.float32))
    small = torch.randint(-64, 64, (batch, n, heads), generator=pool.gen, device=dev)
    want = torch.full_like(pool.weights, float("nan"), dtype=torch.float64)
    for b in range(batch):
        at, row = pool.places(b, n)
        pool.k[at, :, row] = 0.0
        pool.k[at, :, row, 0] = 214.0
        pool.k[at, :, row, 1] = (small[b] / 8).to(pool.dtype)
        pool.weights[at, :, row] = 0.0
        want[at, :, row] = group * torch.softmax(small[b].double() * scale, dim=0)
    _attn(pool, group, q=q, scale=scale)
    assert _status() == 0
    used = ~torch.isnan(want)
    got = pool.weights.double()
    off = ((got - want).abs() / want)[used].max().item()
    assert off <= 2.0 ** -16, f"weights off by {off} of their value"
    for b in range(batch):
        at, row = pool.places(b, n)
        assert ((got[at, :, row].sum(dim=0) / group - 1).abs() <= 2.0 ** -16).all()


# ----------------------------------------------------- infinities in attended rows ------

STRANGE = [("bf16", 128, 4), ("fp16", 128, 4), ("bf16", 64, 16), ("fp16", 64, 16), ("bf16", 128, 24), ("fp16", 64, 20)]


def _check_weights(pool, q, before, scale, skip=()):
    """The added weights of all sequences but those in `skip`, within the helper's tolerance."""
    from paged_helpers import attend
    _, _, added = attend(pool, q, scale)
    for b, (x, tol) in enumerate(added):
        if b in skip:
            continue
        at, row = pool.places(b, x.shape[0])
        want = before[at, :, row].double() + x
        room = tol + 2.0 ** -24 * want.abs()
        assert ((pool.weights[at, :, row].double() - want).abs() <= room).all()


@pytest.mark.parametrize("dtype,dim,group", STRANGE)
@pytest.mark.parametrize("n,spare", [(200, 0), (1000, 2), (9000, 2)])     # uncut, clusters, joined
def test_infinite_values(dev, dtype, dim, group, n, spare):
    """An infinity in an attended value row fills its column of out, two of both signs make NaN, and no more."""
    import torch
    from paged_helpers import Pool, attend
    pool = Pool(dev, dtype, "hnd", 2, dim, 64, [n, n, n], spare_entries=spare, seed=42)
    at, row = pool.places(1, n)
    inf = float("inf")
    put = [(3, 7, inf), (n // 2, 7, inf), (n - 1, 20, -inf), (5, 33, inf), (n - 2, 33, -inf), (n // 3, 50, float("nan"))]
    for slot, column, value in put:
        pool.v[at[slot], :, row[slot], column] = value
    before = pool.weights.clone()
    q, out, lse = _attn(pool, group)
    assert _status() == 0
    got = out[1, 0]
    assert (got[:, 7] == inf).all() and (got[:, 20] == -inf).all()
    assert torch.isnan(got[:, 33]).all() and torch.isnan(got[:, 50]).all()
    for slot, column, _ in put:                      # the rest is as with zeros there
        pool.v[at[slot], :, row[slot], column] = 0.0
    (o, tol), (z, z_tol), _ = attend(pool, q, dim ** -0.5)
    strange = torch.zeros(o.shape, dtype=torch.bool, device=dev)
    strange[1, 0, :, [7, 20, 33, 50]] = True
    assert (((out.double() - o).abs() <= tol) | strange).all()
    assert ((lse.double() - z).abs() <= z_tol).all()
    _check_weights(pool, q, before, dim ** -0.5)


@pytest.mark.parametrize("dtype,dim,group", STRANGE)
@pytest.mark.parametrize("n,spare", [(200, 0), (1000, 2), (9000, 2)])
def test_infinite_keys(dev, dtype, dim, group, n, spare):
    """A score of -inf takes no part; one of +inf makes its own sequence's heads NaN and no other's."""
    import torch
    from paged_helpers import Pool, attend
    pool = Pool(dev, dtype, "hnd", 2, dim, 64, [n, n, n], spare_entries=spare, seed=43)
    q = pool.normal(3, 1, 2 * group, dim)
    q[..., 11] = q[..., 11].abs() + 0.5
    (at, row), (at2, row2) = pool.places(0, n), pool.places(1, n)
    gone = torch.arange(n, device=dev) % 7 == 3
    pool.k[at[gone], :, row[gone], 11] = -float("inf")
    pool.k[at2[n // 2], :, row2[n // 2], 11] = float("inf")
    before = pool.weights.clone()
    _, out, lse = _attn(pool, group, q=q)
    assert _status() == 0
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert torch.equal(pool.weights[at[gone], :, row[gone]], before[at[gone], :, row[gone]])
    # Sequence 0 in the plain form: over the slots that are left, moved to the front of a table of their own.
    left = int((~gone).sum())
    kept = [t[at[~gone], :, row[~gone]].clone() for t in (pool.k, pool.v, before, pool.weights)]
    head, first = pool.places(0, left)
    for t, x in zip((pool.k, pool.v, before, pool.weights), kept):
        t[head, :, first] = x
    pool.k[at2[n // 2], :, row2[n // 2], 11] = 0.0
    pool.lens = torch.tensor([left, n, n], dtype=torch.int32, device=dev)
    (o, tol), (z, z_tol), _ = attend(pool, q, dim ** -0.5)
    for b in (0, 2):
        assert ((out[b].double() - o[b]).abs() <= tol[b]).all() and ((lse[b].double() - z[b]).abs() <= z_tol[b]).all()
    _check_weights(pool, q, before, dim ** -0.5, skip=(1,))


@pytest.mark.parametrize("dtype,dim,group", STRANGE)
def test_nan_leaves_other_sequences_weights(dev, dtype, dim, group):
    import torch
    from paged_helpers import Pool
    pool = Pool(dev, dtype, "nhd", 2, dim, 16, [100, 100, 100], seed=44)
    at, row = pool.places(1, 100)
    pool.k[at[50], 1, row[50], 3] = float("nan")     # one KV head of one sequence
    before = pool.weights.clone()
    q, out, lse = _attn(pool, group)
    assert _status() == 0
    assert torch.isnan(out[1, 0, group:]).all() and torch.isnan(lse[1, 0, group:]).all()
    assert torch.isfinite(out[:, :, :group]).all() and torch.isfinite(out[[0, 2]]).all()
    pool.k[at[50], 1, row[50], 3] = 0.0
    _check_weights(pool, q, before, dim ** -0.5, skip=(1,))


# -------------------------------------- more sequences than a CTA has threads ------

@pytest.mark.parametrize("batch,dtype,heads,group,dim,page,high,spare", [
    (161, "bf16", 2, 8, 64, 16, 300, 0),        # equal chunks; 160 threads
    (161, "fp16", 2, 4, 128, 64, 4000, 100),    # chunks from the counter
    (289, "bf16", 2, 20, 128, 16, 400, 0),      # equal chunks; 288 threads
    (289, "bf16", 1, 20, 64, 32, 4500, 150),    # chunks from the counter
    (4096, "bf16", 2, 4, 64, 16, 60, 40),       # chunks from the counter, more units than chunks
    (4096, "fp16", 1, 3, 128, 16, 100, 12),     # equal chunks, more units than chunks
    (4096, "bf16", 1, 24, 64, 16, 80, 12),
])
@pytest.mark.parametrize("accumulate", [False, True])
def test_many_sequences(dev, batch, dtype, heads, group, dim, page, high, spare, accumulate):
    """A thread of the split then has a run of sequences: empty ones at the runs' borders and whole runs of them."""
    import random
    from paged_helpers import Pool, check_attend
    rng = random.Random(batch + group)
    run = -(-batch // (288 if group > 16 else 160))
    lens = [rng.randrange(1, high + 1) for _ in range(batch)]
    for first in range(0, batch, run):
        kind = rng.randrange(6)
        for b in range(first, min(first + run, batch)):
            if kind == 0 or (kind == 1 and b == first) or (kind == 2 and b == first + run - 1):
                lens[b] = 0
    lens[0], lens[-1], lens[1] = 0, high, high
    pool = Pool(dev, dtype, "hnd", heads, dim, page, lens, spare_entries=spare, seed=45, metadata=accumulate)
    before = pool.weights.clone() if accumulate else None
    q, out, lse = _attn(pool, group, accumulate=accumulate)
    assert _status() == 0
    check_attend(pool, q, out, lse, before, dim ** -0.5)


# ----------------------------------------------------- eviction in one launch ------

def _one_launch(pool, budget, n_init=0, n_local=0):
    """An eviction of at most 64 slots of the capacity, new_lens apart from kv_lens: the selecting CTAs move the rows."""
    assert 0 < pool.max_pages * pool.page - budget <= 64
    return _evict(pool, budget, n_init, n_local)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype,cap,page,budget,n_init,n_local", [
    ("bf16", 320, 64, 256, 4, 16), ("fp16", 2048, 16, 1984, 0, 100), ("bf16", 4096, 64, 4033, 3, 0),
    ("fp16", 4160, 64, 4096, 4, 256),                                              # 512 threads, 4 to 16 keys
    ("bf16", 8208, 16, 8150, 64, 512), ("bf16", 33024, 256, 33000, 0, 1),        # clusters of 2 and 8
    ("bf16", 140032, 64, 139970, 100, 1000), ("fp16", 262208, 64, 262150, 0, 7),   # of 16, 32 and 64 keys
])
@pytest.mark.parametrize("values", ["uniform", "ties"])
def test_evict_in_one_launch(dev, dtype, cap, page, budget, n_init, n_local, values, dim):
    from paged_helpers import Pool, evict_plain
    lens = [cap, budget + 1, budget, 7, 0] if cap < 10000 else [cap, budget + 1]
    pool = Pool(dev, dtype, "nhd", 2, dim, page, lens, spare_entries=0, seed=46)
    if values == "ties":
        pool.weights.mul_(4).floor_()
    want = evict_plain(pool, budget, n_init, n_local)
    new = _one_launch(pool, budget, n_init, n_local)
    assert _status() == 0
    _check_evict(pool, want, new)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("cap,budget", [(512, 460), (1024, 961), (2048, 2000), (4096, 4032)])
def test_evict_many_short_in_one_launch(dev, cap, budget, dim):
    """More units than the SMs hold CTAs of 512 threads: CTAs of 128."""
    from paged_helpers import Pool, evict_plain
    lens = [cap - 3 * i for i in range(39)] + [cap]
    pool = Pool(dev, "bf16", "hnd", 8, dim, 16, lens, spare_entries=0, seed=47)
    pool.weights.mul_(50).floor_()
    want = evict_plain(pool, budget, 2, 7)
    new = _one_launch(pool, budget, 2, 7)
    assert _status() == 0
    _check_evict(pool, want, new)


@pytest.mark.parametrize("cap,page", [(320, 64), (16400, 16)])     # one CTA per unit, and a cluster
def test_evict_in_one_launch_leaves_a_bad_page(dev, cap, page):
    import torch
    import trainable_block_sparse_infllm_gb300 as T
    from paged_helpers import Pool, evict_plain
    budget = cap - 60
    pool = Pool(dev, "bf16", "hnd", 2, 128, page, [cap, cap, cap], spare_entries=0, seed=48)
    keep = pool.lens.clone()
    pool.lens = torch.tensor([cap, 0, cap], dtype=torch.int32, device=dev)
    want = list(evict_plain(pool, budget))
    want[4] = [budget, cap, budget]
    pool.lens = keep
    pool.table[1, cap // page - 1] = pool.k.shape[0]
    new = _one_launch(pool, budget)
    assert _status() == T.DEVICE_BAD_PAGE
    _check_evict(pool, want, new)
    pool.lens = torch.tensor([-3, 50, cap + 1], dtype=torch.int32, device=dev)
    new = _one_launch(pool, budget)
    assert _status() == T.DEVICE_BAD_KV_LEN
    want[4] = [0, 50, 0]
    _check_evict(pool, want, new)


@pytest.mark.parametrize("slack", [65, 127, 128, 129])
def test_evict_around_the_largest_one_launch(dev, slack):
    """The border between one launch and two, by the capacity past the budget: every slot of it to be moved."""
    from paged_helpers import Pool, evict_plain
    cap = 1024
    pool = Pool(dev, "bf16", "hnd", 2, 128, 64, [cap, cap - 1, cap - slack], spare_entries=0, seed=49)
    at, row = pool.places(0, cap, cap - slack)
    pool.weights[at, :, row] += 2.0
    want = evict_plain(pool, cap - slack, 1, 3)
    new = _evict(pool, cap - slack, 1, 3)
    assert _status() == 0
    _check_evict(pool, want, new)
