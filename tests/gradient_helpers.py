"""The gradient of packed causal attention in 64 bits, with the size of its errors.

packed_helpers.py bounds every value by the sum of its parts' largest errors,
which for thousands of keys is far above what unrelated errors come to.  Here
errors that have nothing to do with each other add up as squares, and norms over
many rows are compared.  Each square is of the most that an error can be, at
least twice its mean square, which is the margin.  With u = 2^-24, D = head dim
and e = eps / 2 of the tensors' type:
  * of one score: dz = 2 u (D scale |q k| + 3 |z|) where |q k| is the norm of the D
    products, which their sums on the way are about (each of D steps may truncate),
    of one probability e_p = 2 dz + 2^-21 of itself; of dout . v likewise
    d_in = 2 u (D + 1) |dout v|;
  * dS = P (dout . v - D) enters dq and dk in 16 bits: e of itself and, where it is
    below the type's normal numbers, half a step, `step`; also 2 e_p of itself and
    P d_in.  All these are unrelated from key to key.  In fp16 dS is multiplied by
    powers of two: a row's for dq by one that takes 8 times |dout . v| + |D| (the norm
    over its keys) to 2^15, for rows of more than 1024 keys 4 times |dout| |out| to 2^10;
    and that of all rows that share a tile of keys, for dk, by one that takes 8 times the
    largest row's |dout . v| + |D|, or norm of dS, to 2^14.  step is 2^-25 over that.
  * of the whole row: D is off by d_D, the squares of P (e_p |dout . v| + d_in) and
    2^-19 of P (dout . v) and of D, which moves dq by scale d_D sum P k, and a key's dk
    by scale P d_D q; the row's lse moves dq by e_p + 2^-19 of itself.
  * a row that attends more than 1024 keys may have D from the rounded out for
    the keys from 128 on, as long as that moves the dq of a tile of rows, by the size
    of their keys, no more than e sqrt(sum dS^2): the square of that times the longest
    mean key of any row.
  * results are rounded: e of themselves and half the smallest step.
"""

import torch

U = 2.0 ** -24


def gradients(step):
    """{name: (value, squares of unrelated errors, errors of whole rows)}, NaN in rows of no sequence."""
    info = torch.finfo(step.dtype)
    e, least = info.eps / 2, info.tiny * info.eps / 2
    half = step.dtype is torch.float16
    scale, dim, group = step.scale, step.dim, step.group

    def empty(x):
        return tuple(torch.full(x.shape, float("nan"), dtype=torch.float64, device=step.dev) for _ in range(3))
    result = {n: empty(x) for n, x in dict(dq=step.q, dk=step.k, dv=step.v).items()}
    for b, (n, m) in enumerate(zip(step.q_lens, step.k_lens)):
        if m == 0:      # (rows that attend no key)
            for i in range(3):
                result["dq"][i][step.q_starts[b]:step.q_starts[b] + n] = 0.0
            continue
        at = slice(step.q_starts[b], step.q_starts[b] + n)
        of = slice(step.k_starts[b], step.k_starts[b] + m)
        limit = m - n + torch.arange(n, device=step.dev)
        hidden = torch.arange(m, device=step.dev)[None] > limit[:, None]
        seen = (~hidden).double()
        for h in range(step.heads):
            k, v = step.k[of, h].double(), step.v[of, h].double()
            sums, steps = {name: [0.0, 0.0] for name in ("dk", "dv")}, 0.0
            most, longest, rows = 0.0, 0.0, []
            for g in range(h * group, (h + 1) * group):      # (a head at a time: n x m values in 64 bits)
                q, d = step.q[at, g].double(), step.dout[at, g].double()
                z = (q @ k.T * scale).masked_fill(hidden, -float("inf"))
                dz = 2 * U * (dim * scale * (q ** 2 @ (k ** 2).T).sqrt() + 3 * (q @ k.T * scale).abs())
                e_p = 2 * torch.cat([dz * seen, 0 * dz[:, :1]], dim=1).amax(dim=1, keepdim=True) + 2.0 ** -21
                p = torch.nan_to_num(torch.exp(z - torch.logsumexp(z, dim=1, keepdim=True)), nan=0.0)
                inner, d_in = (d @ v.T) * seen, 2 * U * (dim + 1) * (d ** 2 @ (v ** 2).T).sqrt() * seen
                D = (p * inner).sum(dim=1, keepdim=True)
                ds = p * (inner - D)
                square = (e * ds) ** 2 + (2 * e_p * ds) ** 2 + (p * d_in) ** 2
                far = (limit >= 1024).double()[:, None]
                near_size = inner.norm(dim=1, keepdim=True) + D.abs()
                far_size = d.norm(dim=1, keepdim=True) * (p @ v).norm(dim=1, keepdim=True)
                step_q = torch.where(far > 0, 2.0 ** -33 * far_size, 2.0 ** -37 * near_size) if half else least
                d_D = ((p * (e_p * inner.abs() + d_in)) ** 2 + (2.0 ** -19 * p * inner) ** 2).sum(dim=1).sqrt() + \
                    2.0 ** -19 * D[:, 0].abs()
                dq, mean = scale * (ds @ k), p @ k
                rest = p[:, 128:] @ k[128:]
                weight = p[:, 128:].sum(dim=1).clamp(min=2.0 ** -20)
                longest = max([longest, *(rest.norm(dim=1) / weight)[limit >= 1024].tolist()])
                rows.append((g, dq, (square + step_q ** 2 * seen) @ k ** 2, far * (ds ** 2).sum(dim=1, keepdim=True),
                             (e_p + 2.0 ** -19) * dq.abs() + scale * d_D[:, None] * mean.abs()))
                most = max([most, *torch.where(far > 0, ds.norm(dim=1, keepdim=True), near_size)[:, 0].tolist()])
                p_square = (e * p) ** 2 + (2 * e_p * p) ** 2 + (least / 2 ** 8 if half else least) ** 2 * seen
                square = square + (p * d_D[:, None]) ** 2
                for name, x, y, z_ in (("dk", scale * ds, scale ** 2 * square, q), ("dv", p, p_square, d)):
                    for i, part in enumerate((x.T @ z_, y.T @ z_ ** 2)):
                        sums[name][i] = sums[name][i] + part
                steps = steps + seen.T @ q ** 2
            step_k = 2.0 ** -36 * most if half else least
            sums["dk"][1] = sums["dk"][1] + scale ** 2 * step_k ** 2 * steps
            for g, dq, square, square_far, lin in rows:
                square = scale ** 2 * (square + (e * longest) ** 2 * square_far / dim)
                for i, part in enumerate((dq, square + (e * dq) ** 2 + least ** 2, lin)):
                    result["dq"][i][at, g] = part
            for name in ("dk", "dv"):
                value, square = sums[name]
                for i, part in enumerate((value, square + (e * value) ** 2 + least ** 2, 2.0 ** -19 * value.abs())):
                    result[name][i][of, h] = part
    return result


def off(name, got, want, rows=slice(None)):
    """(norm of the error, what it may be, norm of the value) over `rows`."""
    value, square, lin = (x[rows] for x in want[name])
    inside = ~torch.isnan(value)
    got, value, square, lin = got[rows].double()[inside], value[inside], square[inside], lin[inside]
    return float((got - value).norm()), float(square.sum().sqrt() + lin.norm()), float(value.norm())


def close(name, got, want, rows=slice(None)):
    error, most, size = off(name, got, want, rows)
    assert error <= most, f"{name} off by {error / size:.3%} of its norm, {most / size:.3%} allowed"


def heavy_key(step, at, weight, seq=0):
    """Sequence `seq`'s key `at` takes about `weight` of every row behind it, by dimension 0 of q and k."""
    q0, k0, m = step.q_starts[seq], step.k_starts[seq], step.k_lens[seq]
    step.q[q0:q0 + step.q_lens[seq], :, 0] = 4.0
    step.k[k0:k0 + m, :, 0] = 0.0
    others = torch.log(torch.tensor(float(m))) + 0.5
    need = float(others + torch.log(torch.tensor(weight / (1 - weight))))
    step.k[k0 + at] *= 0.25
    step.k[k0 + at, :, 0] = need / step.scale / 4.0
