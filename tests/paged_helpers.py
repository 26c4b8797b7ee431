"""A paged cache for the tests, and its operators in plain 64-bit form.

Tolerances, from the arithmetic (D = head dim, u = 2^-24, all relative to the
64-bit value unless said otherwise):
  * a score is an fp32 sum of D exact products; tensor-core sums may truncate,
    so a step costs up to 2 u of the sum of magnitudes, and its product with
    the scale and log2(e) three more: dz = 2 u (D + 3) scale sum |q_i k_i|;
  * a probability exp2(z - m): z - m is rounded once (u |z|, below dz), and
    the exponential is good to 2^-21: e_p = 2 dz + 2^-21, and as much again
    through the sum it is divided by;
  * its two 16-bit parts keep 16 bits or more: 2^-16;
  * out: (2 e_p + 2^-16 + 2^-19) sum_s P |v| for those and the fp32 sums of
    the products, and half a step of the output's type, eps / 2 |out|, with a
    thousandth more for the second-order terms; and half of the type's smallest
    step where the value is below its normal numbers;
  * lse: e_p + 2^-20 |lse| + 2^-20;
  * weights: a slot's new weight is off by (2 e_p + 2^-20 + 2^-20 |lse|) of
    what was added, and the running sum is rounded once, u |sum|.
"""

import math

import torch

import trainable_block_sparse_infllm_gb300 as T

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -24


class Pool:
    """Pages of random rows under a shuffled table; everything that no slot uses holds NaN."""

    def __init__(self, dev, dtype, layout, heads, dim, page, lens, spare_pages=3, spare_entries=2, seed=0,
                 metadata=True):
        self.dev, self.heads, self.dim, self.page = dev, heads, dim, page
        self.dtype = DTYPES[dtype]
        self.gen = torch.Generator(device=dev).manual_seed(seed)
        each = [-(-n // page) for n in lens]
        self.max_pages = max(max(each), 1) + spare_entries
        used = sum(each)
        P = used + spare_pages
        shape = {"hnd": (P, heads, page, dim), "nhd": (P, page, heads, dim), "pair": (P, 2, heads, page, dim)}[layout]

        def full():
            return torch.full(shape, float("nan"), dtype=self.dtype, device=dev)
        if layout == "hnd":
            self.k, self.v = full(), full()
        elif layout == "nhd":
            self.k, self.v = full().transpose(1, 2), full().transpose(1, 2)
        else:
            both = full()
            self.k, self.v = both[:, 0], both[:, 1]
        order = torch.randperm(P, generator=self.gen, device=dev)[:used].tolist()
        # Entries past a sequence's pages are never read: they name no page.
        table = torch.full((len(lens), self.max_pages), -77, dtype=torch.int32)
        table[:, -1] = 2 ** 31 - 1
        at = 0
        for b, n in enumerate(each):
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.table = table.to(dev)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.weights = torch.full((P, heads, page), float("nan"), device=dev) if metadata else None
        self.positions = torch.full((P, heads, page), -5, dtype=torch.int32, device=dev) if metadata else None
        for b, n in enumerate(lens):
            if n:
                at, row = self.places(b, n)
                self.k[at, :, row] = self.normal(n, heads, dim)
                self.v[at, :, row] = self.normal(n, heads, dim)
                if metadata:
                    self.weights[at, :, row] = torch.rand((n, heads), generator=self.gen, device=dev)
                    self.positions[at, :, row] = torch.arange(n, dtype=torch.int32, device=dev)[:, None]
        self.cache = T.PagedCache(self.k, self.v, self.weights, self.positions)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.gen, device=self.dev, dtype=torch.float32).to(self.dtype)

    def places(self, b, n, first=0):
        slots = torch.arange(first, n, device=self.dev)
        return self.table[b].long()[slots // self.page], slots % self.page

    def workspace(self, op, group=1):
        ws = T.alloc_paged_workspace(self.cache, self.table, op, group)
        return ws.fill_(0xff)   # NaN everywhere: a call writes what it reads


def attend(pool, q, scale, lens=None):
    """out, lse, weights added per sequence ([n, heads]) in 64 bits, with their tolerances."""
    batch, _, all_heads, dim = q.shape
    heads, group = pool.heads, all_heads // pool.heads
    out = torch.zeros((batch, 1, all_heads, dim), dtype=torch.float64, device=pool.dev)
    out_tol = torch.zeros_like(out)
    lse = torch.full((batch, 1, all_heads), -math.inf, dtype=torch.float64, device=pool.dev)
    lse_tol = torch.zeros_like(lse)
    added = []
    for b, n in enumerate((pool.lens if lens is None else lens).tolist()):
        if n == 0:
            added.append(None)
            continue
        at, row = pool.places(b, n)
        k, v = pool.k[at, :, row].double(), pool.v[at, :, row].double()
        qb = q[b, 0].double().view(heads, group, dim)
        z = torch.einsum("hgd,nhd->hgn", qb, k) * scale
        dz = 2 * U * (dim + 3) * scale * torch.einsum("hgd,nhd->hgn", qb.abs(), k.abs()).amax(dim=2)
        norm = torch.logsumexp(z, dim=2)
        p = torch.exp(z - norm[..., None])
        e_p = 2 * dz + 2.0 ** -21
        o = torch.einsum("hgn,nhd->hgd", p, v)
        mag = torch.einsum("hgn,nhd->hgd", p, v.abs())
        info = torch.finfo(pool.dtype)
        tol = (2 * e_p[..., None] + 2.0 ** -16 + 2.0 ** -19) * mag + info.eps / 2 * 1.001 * o.abs() + \
            info.tiny * info.eps / 2
        out[b, 0], out_tol[b, 0] = o.reshape(-1, dim), tol.reshape(-1, dim)
        lse[b, 0] = norm.reshape(-1)
        lse_tol[b, 0] = (e_p + 2.0 ** -20 * norm.abs() + 2.0 ** -20).reshape(-1)
        rel = 2 * e_p + 2.0 ** -20 + 2.0 ** -20 * norm.abs()
        added.append((p.sum(dim=1).T, (p * rel[..., None]).sum(dim=1).T))
    return (out, out_tol), (lse, lse_tol), added


def check_attend(pool, q, out, lse, before, scale, lens=None):
    (o, o_tol), (z, z_tol), added = attend(pool, q, scale, lens)
    over = (out.double() - o).abs() - o_tol
    assert not torch.isnan(out).any() and over.max() <= 0, f"out off by {over.max()} more than allowed"
    if lse is not None:
        empty = torch.isinf(z)
        assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
        over = ((lse.double() - z).abs() - z_tol)[~empty]
        assert over.numel() == 0 or over.max() <= 0, f"lse off by {over.max()} more than allowed"
    if before is not None:
        want, tol = before.double().clone(), torch.zeros_like(before, dtype=torch.float64)
        for b, x in enumerate(added):
            if x is None:
                continue
            at, row = pool.places(b, x[0].shape[0])
            want[at, :, row] += x[0]
            tol[at, :, row] = x[1] + U * want[at, :, row].abs()
        got = pool.weights.double()
        untouched = torch.isnan(want)
        assert torch.equal(torch.isnan(got), untouched)
        over = ((got - want).abs() - tol)[~untouched]
        assert over.numel() == 0 or over.max() <= 0, f"weights off by {over.max()} more than allowed"


def evict_plain(pool, budget, n_init=0, n_local=0, seq_lens=None):
    """What paged_evict leaves: (k, v, weights, positions, new_lens), moved element by element on the CPU."""
    k, v, w, p = (t.cpu().clone() for t in (pool.k, pool.v, pool.weights, pool.positions))
    table, lens = pool.table.cpu(), pool.lens.tolist()
    seen = lens if seq_lens is None else seq_lens.tolist()
    for b, n in enumerate(lens):
        if n <= budget:
            continue
        slots = torch.arange(n)
        at, row = table[b].long()[slots // pool.page], slots % pool.page
        for h in range(pool.heads):
            pos, weight = p[at, h, row].tolist(), w[at, h, row].tolist()
            always = [x < n_init or x >= seen[b] - n_local for x in pos]
            gone = [not a and math.isnan(x) for a, x in zip(always, weight)]     # NaN: below -inf
            rank = sorted(range(n), key=lambda s: (not always[s], gone[s],
                                                   0.0 if always[s] or gone[s] else -weight[s], s))
            kept = set(rank[:budget])
            holes = [s for s in range(budget) if s not in kept]
            movers = [s for s in range(budget, n) if s in kept]
            assert len(holes) == len(movers)
            for t in (k, v, w, p):
                if holes:
                    t[at[holes], h, row[holes]] = t[at[movers], h, row[movers]]
    return k, v, w, p, [min(n, budget) for n in lens]
