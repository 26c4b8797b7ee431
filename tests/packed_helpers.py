"""Packed causal attention and its gradient in plain 64-bit form, with tolerances.

From the arithmetic (D = head dim, u = 2^-24, e = eps / 2 of the tensors' type,
the most that one rounding to it costs):
  * a score is off by dz = 2 u (D + 3) scale sum |q_i k_i| (an fp32 sum of D
    exact products whose steps may truncate, and three roundings of the scaled
    score), a probability by e_p = 2 dz + 2^-21 of itself, and as much again
    through the sum it is divided by;
  * out: (2 e_p + e + 2^-19) sum P |v|: P enters the product rounded to the type;
    then the result's own rounding, e |out|; a P below the type's normal numbers
    is off by half its smallest step, which sum |v| bounds;
  * lse: e_p + 2^-20 |lse| + 2^-20;
  * dout . v is off by d_in = 2 u (D + 1) sum |dout v|, D = sum P (dout . v) by
    d_D = sum P (e_p |dout . v| + d_in) + 2^-19 sum P |dout . v|, and where the row
    attends more than 1024 keys it may come from the rounded out instead, off by
    sum |dout| (the tolerance of out);
  * dS = P (dout . v - D) is off by P ((2 e_p + e) |dout . v - D| + d_in + d_D)
    and half the type's smallest step;
  * dq, dk: scale times the sum of that times |k| or |q|, 2^-19 of the sum of
    magnitudes for the fp32 sums, and the rounding of the result; dv likewise from
    P's (2 e_p + e) P.
A thousandth more on each covers the second-order terms.
"""

import math

import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -24


class Step:
    """Packed tensors of a batch; rows of no sequence (before, between and behind) hold NaN."""

    def __init__(self, dev, dtype, dim, heads, group, q_lens, k_lens=None, layout="own", seed=0, gap=3):
        self.dev, self.dtype, self.dim, self.heads, self.group = dev, DTYPES[dtype], dim, heads, group
        self.gen = torch.Generator(device=dev).manual_seed(seed)
        self.q_lens, self.k_lens = list(q_lens), list(q_lens if k_lens is None else k_lens)
        self.own_keys = k_lens is not None
        self.q_starts, self.k_starts = ([0], [0])
        for n, m in zip(self.q_lens, self.k_lens):
            self.q_starts.append(self.q_starts[-1] + n)
            self.k_starts.append(self.k_starts[-1] + m)
        tq, tk = self.q_starts[-1] + gap, self.k_starts[-1] + gap
        hq = heads * group
        if layout == "fused" and tq == tk:          # columns of one projection's output
            whole = self.full(tq, hq + 2 * heads, dim)
            self.q, self.k, self.v = whole.split([hq, heads, heads], dim=1)
        elif layout == "heads":                      # head-major storage
            self.q, self.k, self.v = (self.full(h, t, dim).transpose(0, 1)
                                      for h, t in ((hq, tq), (heads, tk), (heads, tk)))
        else:
            self.q, self.k, self.v = self.full(tq, hq, dim), self.full(tk, heads, dim), self.full(tk, heads, dim)
        self.q[:self.q_starts[-1]] = self.normal(self.q_starts[-1], hq, dim)
        self.k[:self.k_starts[-1]] = self.normal(self.k_starts[-1], heads, dim)
        self.v[:self.k_starts[-1]] = self.normal(self.k_starts[-1], heads, dim)
        self.dout = self.full(tq, hq, dim)
        self.dout[:self.q_starts[-1]] = self.normal(self.q_starts[-1], hq, dim)
        self.scale = dim ** -0.5

    def full(self, *shape):
        return torch.full(shape, float("nan"), dtype=self.dtype, device=self.dev)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.gen, device=self.dev).to(self.dtype)

    def ints(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.dev)

    def forward(self, T, stream=None, marker=7.0):
        out, lse = torch.full_like(self.q, marker), torch.full(self.q.shape[:2], marker, device=self.dev)
        T.packed_attn(self.q, self.k, self.v, self.ints(self.q_starts), out, lse,
                      k_starts=self.ints(self.k_starts) if self.own_keys else None, scale=self.scale, stream=stream)
        return out, lse

    def backward(self, T, out, lse, stream=None, marker=7.0, ws=None):
        grads = [torch.full_like(x, marker) for x in (self.q, self.k, self.v)]
        ws = T.alloc_packed_workspace(self.q).fill_(0xff) if ws is None else ws
        T.packed_attn_backward(self.q, self.k, self.v, self.ints(self.q_starts), out, lse, self.dout, *grads,
                               workspace=ws, k_starts=self.ints(self.k_starts) if self.own_keys else None,
                               scale=self.scale, stream=stream)
        return grads


def plain(step, with_grads=True):
    """{name: (value, tolerance)} in 64 bits; rows of no sequence are None's NaN (left as they were)."""
    info = torch.finfo(step.dtype)
    e, least, more = info.eps / 2, info.tiny * info.eps / 2, 1.001
    heads, group, scale = step.heads, step.group, step.scale

    def empty(x):
        return torch.full(x.shape, float("nan"), dtype=torch.float64, device=step.dev)
    names = dict(out=step.q, dq=step.q, dk=step.k, dv=step.v)
    result = {n: (empty(x), empty(x)) for n, x in names.items()}
    result["lse"] = tuple(torch.full(step.q.shape[:2], float("nan"), dtype=torch.float64, device=step.dev)
                          for _ in range(2))

    def put(name, at, heads_at, value, tol):
        result[name][0][at, heads_at], result[name][1][at, heads_at] = value, tol
    for b, (n, m) in enumerate(zip(step.q_lens, step.k_lens)):
        at = slice(step.q_starts[b], step.q_starts[b] + n)
        of = slice(step.k_starts[b], step.k_starts[b] + m)
        limit = m - n + torch.arange(n, device=step.dev)
        hidden = (torch.arange(m, device=step.dev)[None] > limit[:, None])[None]
        for h in range(heads):
            mine = slice(h * group, (h + 1) * group)
            q, k, v = step.q[at, mine].double(), step.k[of, h].double(), step.v[of, h].double()
            z = (torch.einsum("rgd,kd->grk", q, k) * scale).masked_fill(hidden, -math.inf)
            dz = 2 * U * (step.dim + 3) * scale * torch.einsum("rgd,kd->grk", q.abs(), k.abs())
            dz = dz.masked_fill(hidden, 0.0).amax(dim=2, keepdim=True) if m else torch.zeros((group, n, 1)).to(z)
            norm = torch.logsumexp(z, dim=2, keepdim=True) if m else torch.full((group, n, 1), -math.inf).to(z)
            p = torch.nan_to_num(torch.exp(z - norm), nan=0.0)           # rows that attend no key: 0
            e_p = 2 * dz + 2.0 ** -21
            seen = (~hidden).double().expand(group, -1, -1)
            out = torch.einsum("grk,kd->rgd", p, v)
            out_tol = torch.einsum("grk,kd->rgd", p * (2 * e_p + e + 2.0 ** -19) + least * seen, v.abs())
            out_tol = more * (out_tol + e * out.abs() + least)
            put("out", at, mine, out, out_tol)
            norm = norm[..., 0]
            put("lse", at, mine, norm.T, (e_p[..., 0] + 2.0 ** -20 * norm.abs() + 2.0 ** -20).T)
            if not with_grads:
                continue
            g = step.dout[at, mine].double()
            inner = torch.einsum("rgd,kd->grk", g, v) * seen
            d_in = 2 * U * (step.dim + 1) * torch.einsum("rgd,kd->grk", g.abs(), v.abs()) * seen
            D = (p * inner).sum(dim=2, keepdim=True)
            d_D = (p * ((e_p + 2.0 ** -19) * inner.abs() + d_in)).sum(dim=2, keepdim=True)
            if m > 1024:
                d_D = torch.maximum(d_D, (g.abs() * out_tol).sum(dim=2).T[..., None])
            ds = p * (inner - D)
            ds_tol = p * ((2 * e_p + e) * (inner - D).abs() + d_in + d_D) + least * seen
            ds_all = ds_tol + 2.0 ** -19 * ds.abs()
            for name, at_, heads_, value, tol in (
                    ("dq", at, mine, torch.einsum("grk,kd->rgd", ds, k), torch.einsum("grk,kd->rgd", ds_all, k.abs())),
                    ("dk", of, h, torch.einsum("grk,rgd->kd", ds, q), torch.einsum("grk,rgd->kd", ds_all, q.abs()))):
                value, tol = value * scale, tol * scale
                put(name, at_, heads_, value, more * (tol + e * value.abs() + least))
            value = torch.einsum("grk,rgd->kd", p, g)
            tol = torch.einsum("grk,rgd->kd", p * (2 * e_p + e + 2.0 ** -19) + least * seen, g.abs())
            put("dv", of, h, value, more * (tol + e * value.abs() + least))
    return result


def check(name, got, want, marker=7.0):
    """Within tolerance everywhere, and `marker` in every row of no sequence."""
    value, tol = want[name]
    rows = ~torch.isnan(value)
    got = got.double()
    assert torch.equal(got[~rows], torch.full_like(got[~rows], marker)), f"{name}: rows of no sequence were written"
    got, value, tol = got[rows], value[rows], tol[rows]
    fine = torch.isfinite(value)
    assert torch.equal(got[~fine], value[~fine]), f"{name}: infinities differ"
    over = (got[fine] - value[fine]).abs() - tol[fine]
    assert not torch.isnan(over).any(), f"{name} has NaN"
    assert over.numel() == 0 or over.max() <= 0, f"{name} off by {over.max()} more than allowed"
