"""What a step of packed sequences needs around the paged cache, as measured workloads.

A step holds the new tokens of several sequences one after the other: starts
int32 [batch + 1] says where each begins.  The operators, in their order of use:
the page tables and slot maps of the step, the rotary positions of its queries
and keys, causal attention over packed sequences with its gradient, and the
write of the step's keys and values to their slots.  `run` with `own` false is
each operator in plain torch operations in 32 bits; with `own` true it calls the
library.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    attn = dict(op="attn", dtype="bf16", batch=1, heads=2, group=16, dim=128, low=1, high=64, before=0, fused=False,
                backward=False)
    rotary = dict(op="rotary", dtype="bf16", tokens=64, heads=2, group=16, dim=128, part=128, interleaved=False,
                  transpose=False, scaling="plain", fused=True, far=131072)
    append = dict(op="append", dtype="bf16", layout="hnd", tokens=64, pad=0, heads=8, dim=128, page=16, fused=True,
                  metadata=True)
    reserve = dict(op="reserve", batch=64, page=16, low=1, high=8191, new=1, pad=0, done=0.0, cut=0.0, spare=64)
    return [
        # One user's question: a short prompt, where latency is what there is.
        dict(attn, name="attention of one short prompt", low=301, high=301, fused=True),
        # One long document, the head layout of the block-sparse benchmark (2 KV heads of 16 query heads).
        dict(attn, name="attention of one 16K prompt", low=16384, high=16384),
        # A serving step: ragged prompts of a model with small heads, fp16.
        dict(attn, name="attention of 24 ragged prompts fp16", dtype="fp16", batch=24, heads=8, group=4, dim=64,
             low=1, high=2047, fused=True),
        # A few drafted tokens of each of 4 sequences against what they hold already.
        dict(attn, name="attention of 4 x 12 tokens after 32K", batch=4, low=12, high=12, before=32000),
        # Training on one long sequence.
        dict(attn, name="gradient of one 8K sequence", low=8192, high=8192, backward=True),
        # Training on packed documents of odd lengths, d 64, 5 query heads per KV head.
        dict(attn, name="gradient of 16 packed documents fp16", dtype="fp16", batch=16, heads=4, group=5, dim=64,
             low=17, high=2500, backward=True, fused=True),
        # A decode step of 64 sequences.
        dict(rotary, name="rotary positions of 64 tokens"),
        # The gradient of a training step's positions, a quarter of each head turned, pairs side by side.
        dict(rotary, name="rotary gradient of 16K tokens", tokens=16384, part=32, interleaved=True, transpose=True,
             scaling="parts", heads=8, group=4),
        # The same decode step's write.
        dict(append, name="packed append of 64 tokens"),
        # The write of a step of ragged prompts, padded to a captured graph's size.
        dict(append, name="packed append of 40000 tokens", tokens=40000, pad=960, heads=4, page=64, layout="nhd"),
        # A decode step's tables: a few sequences enter a new page.
        dict(reserve, name="pages and slots of a decode step"),
        # Prompts come in, finished sequences give their pages back, evicted ones their surplus.
        dict(reserve, name="pages and slots of 40 prompts", batch=48, page=64, low=1, high=8192, new=4096, pad=500,
             done=0.2, cut=0.1, spare=4000),
    ]


# A drawn case has at most so many score entries (padded), values or tokens, so
# that it costs no more than the largest listed case of its operator.
MOST_SCORES = {False: 32 * 16384 * 16384, True: 32 * 8192 * 8192}
MOST_VALUES = {"rotary": 16384 * 40 * 128, "append": 40000 * 8 * 128}
MOST_TOKENS = 48 * 4096


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "rotary", "append", "reserve"])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]), heads=rng.choice([1, 2, 3, 4, 8]),
                dim=rng.choice([64, 128, 128]), fused=rng.random() < 0.5)
    group = rng.choice([1, 2, 4, 5, 7, 8, 16, 16, 32])
    if op == "attn":
        case.update(group=group, backward=rng.random() < 0.5)
        rows = case["heads"] * group
        most = MOST_SCORES[case["backward"]] // rows
        high = _log_int(rng, 1, min(16384, math.isqrt(most)))
        case["before"] = rng.choice([0, 0, 0, _log_int(rng, 1, 32768)])
        case["before"] = max(0, min(case["before"], most // high - high))
        case["batch"] = _log_int(rng, 1, max(1, min(64, most // (high * (high + case["before"])), 65536 // high)))
        case["high"], case["low"] = high, rng.choice([0, 1, high // 2, high])
    elif op == "rotary":
        case.update(group=group, interleaved=rng.random() < 0.5, transpose=rng.random() < 0.5,
                    part=rng.choice([case["dim"], case["dim"], case["dim"] // 2, 32]),
                    scaling=rng.choice(["plain", "linear", "base", "parts", "factors"]),
                    far=_log_int(rng, 100, 2000000))
        case["tokens"] = _log_int(rng, 1, MOST_VALUES[op] // (case["heads"] * (group + 1) * case["dim"]))
    elif op == "append":
        case.update(layout=rng.choice(["hnd", "nhd", "pair"]), page=rng.choice([16, 32, 48, 64, 128, 256]),
                    metadata=rng.random() < 0.75)
        case["tokens"] = _log_int(rng, 1, MOST_VALUES[op] // (2 * case["heads"] * case["dim"]))
        case["pad"] = rng.choice([0, case["tokens"] // 8])
    else:
        case = dict(op=op, batch=_log_int(rng, 1, 512), page=rng.choice([16, 32, 48, 64, 128, 256]),
                    new=rng.choice([1, 1, 512, 8192]), pad=rng.choice([0, 77]), done=rng.choice([0.0, 0.1]),
                    cut=rng.choice([0.0, 0.2]), spare=rng.choice([50, 1000, 100000]))
        case["new"] = min(case["new"], MOST_TOKENS // case["batch"])
        case["high"] = _log_int(rng, 16, 32768)
        case["low"] = rng.choice([0, 1, case["high"] // 2])
    return case


def _spread(low, high, count):
    """`count` lengths spread evenly over [low, high], the longest among them."""
    spread = [low + int((high - low + 1) * (((i + 1) * 0.6180339887498949) % 1.0)) for i in range(count)]
    return [high] + spread[1:]


def _starts(lengths):
    starts = [0]
    for n in lengths:
        starts.append(starts[-1] + n)
    return starts


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _frequencies(case):
    """Radians per position of each pair, and the factor of the turned values, by scaling."""
    half, base, factor, length = case["part"] // 2, 10000.0, 8.0, 4096
    index = torch.arange(half, dtype=torch.float64) / half
    if case["scaling"] == "base":          # the base grows so that the slowest pair turns `factor` times slower
        base *= factor ** (half / (half - 1))
    freq = base ** -index
    if case["scaling"] == "linear":
        return freq / factor, 1.0
    if case["scaling"] == "parts":         # pairs that turn often keep their speed, the slowest are divided
        def pair(turns):
            return half * math.log(length / (turns * 2 * math.pi)) / math.log(base)
        low, high = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), case["part"] - 1)
        keep = 1 - ((torch.arange(half, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        return freq / factor * (1 - keep) + freq * keep, 0.1 * math.log(factor) + 1
    if case["scaling"] == "factors":       # a divisor for each pair
        return freq / _divisors(half), math.sqrt(1 + math.log(factor) / math.log(length))
    return freq, 1.0


def _divisors(half):
    return torch.tensor([1.0 + 7.0 * (i / half) ** 2 for i in range(half)], dtype=torch.float64)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"attn": _prepare_attn, "rotary": _prepare_rotary, "append": _prepare_append,
            "reserve": _prepare_reserve}[case["op"]](case, gen)


def _rows(case, gen, tokens, *heads):
    """Packed [tokens, heads, d] tensors: each of its own, or columns of one projection's output."""
    dtype, dim = DTYPES[case["dtype"]], case["dim"]
    if case["fused"]:
        whole = torch.randn((tokens, sum(heads), dim), device="cuda", dtype=dtype, generator=gen)
        return whole.split(list(heads), dim=1)
    return [torch.randn((tokens, h, dim), device="cuda", dtype=dtype, generator=gen) for h in heads]


def _prepare_attn(case, gen):
    heads, group, dim, before = case["heads"], case["group"], case["dim"], case["before"]
    n_q = _spread(case["low"], case["high"], case["batch"])
    q_starts = _starts(n_q)
    k_starts = _starts([n + before for n in n_q])
    if before:
        q, = _rows(case, gen, q_starts[-1], heads * group)
        k, v = _rows(case, gen, k_starts[-1], heads, heads)
    else:
        q, k, v = _rows(case, gen, q_starts[-1], heads * group, heads, heads)
    # The first token of a sequence draws much of the attention, as it does in trained models.
    sink = torch.randn((heads, dim), device="cuda", generator=gen)
    q += (0.5 * sink).to(q.dtype).repeat_interleave(group, dim=0)
    first = torch.tensor([k_starts[b] for b in range(case["batch"]) if n_q[b] + before], device="cuda")
    k[first] = (k[first].float() + sink).to(k.dtype)
    state = dict(op="attn", q=q, k=k, v=v, q_starts=_ints(q_starts), k_starts=_ints(k_starts), before=before,
                 most_q=max(n_q), most_k=max(n_q) + before, scale=dim ** -0.5, backward=case["backward"],
                 out=torch.empty(q.shape, dtype=q.dtype, device="cuda"),
                 lse=torch.empty(q.shape[:2], device="cuda"))
    if case["backward"]:
        # What the forward pass left: its output and the scores' log sum.
        out, lse = _plain_attn(state)[:2]
        state["out"].copy_(out)
        state["lse"].copy_(lse)
        state["dout"] = torch.randn(q.shape, device="cuda", dtype=q.dtype, generator=gen)
        for name in ("q", "k", "v"):
            state["d" + name] = torch.empty(state[name].shape, dtype=q.dtype, device="cuda")
    if own:
        import trainable_block_sparse_infllm_gb300 as T
        state["T"] = T
        if case["backward"]:
            state["workspace"] = T.alloc_packed_workspace(q)
    return state


def _prepare_rotary(case, gen):
    heads, tokens = case["heads"], case["tokens"]
    q, k = _rows(case, gen, tokens, heads * case["group"], heads)
    freq, scale = _frequencies(case)
    state = dict(op="rotary", q=q, k=k, part=case["part"], interleaved=case["interleaved"],
                 transpose=case["transpose"], freq=freq.cuda(), scale=scale,
                 positions=torch.randint(0, case["far"], (tokens,), device="cuda", generator=gen, dtype=torch.int32),
                 q_out=torch.empty(q.shape, dtype=q.dtype, device="cuda"),
                 k_out=torch.empty(k.shape, dtype=k.dtype, device="cuda"))
    if own:
        import trainable_block_sparse_infllm_gb300 as T
        kinds = {"plain": T.ROTARY_PLAIN, "linear": T.ROTARY_LINEAR, "base": T.ROTARY_BASE, "parts": T.ROTARY_PARTS,
                 "factors": T.ROTARY_FACTORS}
        state["T"] = T
        state["plan"] = T.alloc_rotary_plan(
            case["part"], base=10000.0, scaling=kinds[case["scaling"]], factor=8.0, original_len=4096,
            factors=_divisors(case["part"] // 2).tolist() if case["scaling"] == "factors" else None, device="cuda")
    return state


def _prepare_append(case, gen):
    dtype, dim, heads, page, tokens = (DTYPES[case["dtype"]], case["dim"], case["heads"], case["page"], case["tokens"])
    pages = -(-tokens // page) + 3

    def normal(*shape):
        return torch.randn(shape, device="cuda", dtype=dtype, generator=gen)

    if case["layout"] == "hnd":      # [page, head, token, d]
        k, v = normal(pages, heads, page, dim), normal(pages, heads, page, dim)
    elif case["layout"] == "nhd":    # [page, token, head, d]
        k, v = (normal(pages, page, heads, dim).transpose(1, 2) for _ in range(2))
    else:                            # keys and values of a page side by side
        both = normal(pages, 2, heads, page, dim)
        k, v = both[:, 0], both[:, 1]
    k_new, v_new = _rows(case, gen, tokens + case["pad"], heads, heads)
    # Prompts fill their pages in order; the pages lie anywhere.  Padding goes nowhere.
    where = torch.randperm(pages, device="cuda", generator=gen)
    at = torch.arange(tokens, device="cuda")
    slots = torch.full((tokens + case["pad"],), -1, dtype=torch.int32, device="cuda")
    slots[:tokens] = (where[at // page] * page + at % page).to(torch.int32)
    state = dict(op="append", k=k, v=v, k_new=k_new, v_new=v_new, slots=slots, used=tokens, weights=None,
                 positions=None, where=None)
    if case["metadata"]:
        state["weights"] = torch.rand((pages, heads, page), device="cuda", generator=gen)
        state["positions"] = torch.zeros((pages, heads, page), dtype=torch.int32, device="cuda")
        state["where"] = torch.randint(0, 100000, slots.shape, device="cuda", generator=gen, dtype=torch.int32)
    if own:
        import trainable_block_sparse_infllm_gb300 as T
        state["T"] = T
        state["cache"] = T.PagedCache(k, v, state["weights"], state["positions"])
    return state


def _requests(case):
    """Of each sequence: the pages it holds, the tokens its cache holds and its new ones, and whether some were evicted."""
    batch, page = case["batch"], case["page"]
    finished = int(case["done"] * batch)               # nothing cached any more, nothing new: all pages come back
    evicted = finished + int(case["cut"] * batch)
    prompts = _spread(1, case["new"], batch)
    requests = []
    for i, n in enumerate(_spread(case["low"], case["high"], batch)[::-1]):
        held = -(-n // page)
        if i < finished:
            requests.append((held, 0, 0, 0))
        elif i < evicted:
            requests.append((held, n // 3, 1, 1))
        elif case["new"] > 1:                          # a prompt: nothing cached yet
            requests.append((0, 0, prompts[i], 0))
        else:
            requests.append((held, n, 1, 0))
    return requests


def _prepare_reserve(case, gen):
    batch, page = case["batch"], case["page"]
    order = torch.randperm(batch, device="cuda", generator=gen)
    requests = _requests(case)
    held, kv, n_new, evicted = (_ints(x)[order] for x in zip(*requests))
    seen = kv + torch.randint(0, 100, (batch,), device="cuda", generator=gen, dtype=torch.int32) * evicted
    width = -(-(case["high"] + case["new"]) // page)
    owned = sum(r[0] for r in requests)
    pages = owned + case["spare"] + 1
    ids = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    columns = torch.arange(width, device="cuda")
    mine = columns[None] < held[:, None]
    place = (held.cumsum(0) - held)[:, None] + columns[None]
    # One buffer holds what a step changes, so that `run` starts from the same state each time.
    sizes = [batch * width, batch, pages, 1]
    before = torch.zeros(sum(sizes), dtype=torch.int32, device="cuda")
    table, own_pages, free, n_free = before.split(sizes)
    table.copy_(torch.where(mine, ids[place.clamp_max(pages - 1)], 0).view(-1))
    own_pages.copy_(held)
    free[:pages - owned] = ids[owned:]
    n_free.fill_(pages - owned)
    now = before.clone()
    table, own_pages, free, n_free = now.split(sizes)
    tokens = sum(r[2] for r in requests) + case["pad"]
    state = dict(op="reserve", before=before, now=now, table=table.view(batch, width), held=own_pages, free=free,
                 n_free=n_free, kv=kv, n_new=n_new, seen=seen, page=page,
                 new_lens=torch.empty_like(kv), starts=torch.empty(batch + 1, dtype=torch.int32, device="cuda"),
                 slots=torch.empty(max(tokens, 1), dtype=torch.int32, device="cuda"),
                 positions=torch.empty(max(tokens, 1), dtype=torch.int32, device="cuda"),
                 missing=torch.empty(1, dtype=torch.int32, device="cuda"))
    if own:
        import trainable_block_sparse_infllm_gb300 as T
        state["T"] = T
        state["tables"] = T.PageTables(state["table"], own_pages, free, n_free, state["missing"], page)
    return state


def run(state):
    return {"attn": _attn, "rotary": _rotary, "append": _append, "reserve": _reserve}[state["op"]](state)


def _attn(state):
    if state["backward"]:
        if own:
            state["T"].packed_attn_backward(state["q"], state["k"], state["v"], state["q_starts"], state["out"],
                                            state["lse"], state["dout"], state["dq"], state["dk"], state["dv"],
                                            k_starts=state["k_starts"] if state["before"] else None,
                                            scale=state["scale"], workspace=state["workspace"])
        else:
            dq, dk, dv = _plain_attn(state, state["dout"])
            state["dq"].copy_(dq)
            state["dk"].copy_(dk)
            state["dv"].copy_(dv)
        return {"dq": state["dq"], "dk": state["dk"], "dv": state["dv"]}
    if own:
        state["T"].packed_attn(state["q"], state["k"], state["v"], state["q_starts"], state["out"], state["lse"],
                               k_starts=state["k_starts"] if state["before"] else None, scale=state["scale"])
    else:
        out, lse = _plain_attn(state)
        state["out"].copy_(out)
        state["lse"].copy_(lse)
    return {"out": state["out"], "lse": state["lse"]}


def _padded(x, starts, most):
    """[batch, heads, most, d] of a packed tensor in 32 bits, rows past a sequence's end 0."""
    steps = torch.arange(most, device="cuda")
    rows = (starts[:-1, None] + steps).long().clamp_max(x.shape[0] - 1)
    here = steps[None] < (starts[1:] - starts[:-1])[:, None]
    return x[rows].float().mul_(here[:, :, None, None]).transpose(1, 2)


def _packed(x, starts, tokens):
    """The packed rows [tokens, heads, ...] of a padded [batch, heads, most, ...]."""
    at = torch.arange(tokens, device="cuda")
    batch = torch.searchsorted(starts[1:].long(), at, right=True)
    return x.transpose(1, 2)[batch, at - starts[batch]]


def _plain_attn(state, dout=None):
    """The output and the log sum; with an upstream gradient the three gradients, in 32 bits."""
    q_starts, k_starts, most_q, most_k = state["q_starts"], state["k_starts"], state["most_q"], state["most_k"]
    k = _padded(state["k"], k_starts, most_k)
    v = _padded(state["v"], k_starts, most_k)
    batch, heads, _, dim = k.shape

    def grouped(x):                    # the rows of a group's heads one after the other
        return _padded(x, q_starts, most_q).reshape(batch, heads, -1, dim)

    q = grouped(state["q"])
    last = (k_starts[1:] - k_starts[:-1] - q_starts[1:] + q_starts[:-1])[:, None] + torch.arange(most_q, device="cuda")
    hidden = torch.arange(most_k, device="cuda") > last[:, :, None]
    group = q.shape[2] // most_q
    z = torch.matmul(q, k.transpose(2, 3)).mul_(state["scale"]).view(batch, heads, group, most_q, most_k)
    z = z.masked_fill_(hidden[:, None, None], -math.inf)
    top = z.amax(dim=4, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    z = z.sub_(top).exp_()
    total = z.sum(dim=4, keepdim=True)
    lse = (top + total.log()).reshape(batch, heads * group, most_q)
    z = z.div_(total.clamp_min(torch.finfo(torch.float32).tiny)).view(batch, heads, -1, most_k)
    tokens = state["q"].shape[0]
    if dout is None:
        out = torch.matmul(z, v).view(batch, heads * group, most_q, dim)
        return _packed(out, q_starts, tokens), _packed(lse, q_starts, tokens)
    g = grouped(dout)
    dv = torch.matmul(z.transpose(2, 3), g)
    dz = torch.matmul(g, v.transpose(2, 3))
    dz = dz.sub_((dz * z).sum(dim=3, keepdim=True)).mul_(z).mul_(state["scale"])
    del z
    dq = torch.matmul(dz, k).view(batch, heads * group, most_q, dim)
    dk = torch.matmul(dz.transpose(2, 3), q)
    keys = state["k"].shape[0]
    return _packed(dq, q_starts, tokens), _packed(dk, k_starts, keys), _packed(dv, k_starts, keys)


def _rotary(state):
    if own:
        state["T"].rotary(state["q"], state["k"], state["positions"], state["plan"], state["q_out"], state["k_out"],
                          interleaved=state["interleaved"], transpose=state["transpose"])
    else:
        angle = state["positions"].double()[:, None] * state["freq"]
        cos, sin = (angle.cos() * state["scale"]).float()[:, None], (angle.sin() * state["scale"]).float()[:, None]
        sin = -sin if state["transpose"] else sin
        part = state["part"]
        if state["interleaved"]:
            first, second = slice(0, part, 2), slice(1, part, 2)
        else:
            first, second = slice(0, part // 2), slice(part // 2, part)
        x = torch.cat([state["q"], state["k"]], dim=1).float()
        a, b = x[:, :, first].clone(), x[:, :, second].clone()
        x[:, :, first] = a * cos - b * sin
        x[:, :, second] = a * sin + b * cos
        state["q_out"].copy_(x[:, :state["q"].shape[1]])
        state["k_out"].copy_(x[:, state["q"].shape[1]:])
    return {"q": state["q_out"], "k": state["k_out"]}


def _append(state):
    if own:
        state["T"].paged_append_packed(state["cache"], state["k_new"], state["v_new"], state["slots"], state["where"])
    else:
        used, page = state["used"], state["k"].shape[2]
        slot = state["slots"][:used].long()
        at, row = slot // page, slot % page
        state["k"][at, :, row] = state["k_new"][:used]
        state["v"][at, :, row] = state["v_new"][:used]
        if state["weights"] is not None:
            state["weights"][at, :, row] = 0.0
            state["positions"][at, :, row] = state["where"][:used, None].expand(-1, state["k"].shape[1])
    return {"k": state["k"], "v": state["v"], "weights": state["weights"], "positions": state["positions"]}


def _reserve(state):
    state["now"].copy_(state["before"])
    if own:
        state["T"].paged_reserve(state["tables"], state["kv"], state["n_new"], state["new_lens"], state["starts"],
                                 state["slots"], state["positions"], seq_lens=state["seen"])
    else:
        table, held, free, page = state["table"], state["held"], state["free"], state["page"]
        batch, width = table.shape
        pages = free.shape[0]
        need = (state["kv"] + state["n_new"] + page - 1) // page
        taken, given = (need - held).clamp_min(0), (held - need).clamp_min(0)
        take, give = taken.sum(), given.sum()
        n = state["n_free"][0]
        lacking = (take - n - give).clamp_min(0)
        enough = lacking == 0
        column = torch.arange(width, device="cuda")[None]
        # The pages given back, in order; entries that are none go behind the last.
        back = (column >= need[:, None]) & (column < held[:, None])
        rank = (given.cumsum(0) - given)[:, None] + column - need[:, None]
        returned = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
        returned.scatter_(0, torch.where(back, rank, pages).view(-1), table.view(-1))
        grown = (column >= held[:, None]) & (column < need[:, None]) & enough
        rank = (taken.cumsum(0) - taken)[:, None] + column - held[:, None]
        page_of = torch.where(rank < n, free[(n - 1 - rank).clamp(0, pages - 1)],
                              returned[(rank - n).clamp(0, pages)])
        table.copy_(torch.where(grown, page_of, table))
        # What is left of the returned pages lies on what is left of the stack.
        kept, used = n - torch.minimum(take, n), (take - n).clamp_min(0)
        at = torch.arange(pages, device="cuda")
        pushed = (at >= kept) & (at < kept + give - used) & enough
        free.copy_(torch.where(pushed, returned[(at - kept + used).clamp(0, pages)], free))
        state["n_free"].copy_(torch.where(enough, kept + give - used, n))
        held.copy_(torch.where(enough, need, held))
        state["missing"].copy_(lacking)
        n_new = torch.where(enough, state["n_new"], 0)
        torch.add(state["kv"], n_new, out=state["new_lens"])
        starts = state["starts"]
        starts[0] = 0
        starts[1:] = n_new.cumsum(0)
        token = torch.arange(state["slots"].shape[0], device="cuda")
        real = token < starts[-1]
        b = torch.searchsorted(starts[1:].long(), token, right=True).clamp_max(batch - 1)
        step = token - starts[b]
        slot = (state["kv"][b] + step).clamp(0, width * page - 1)
        state["slots"].copy_(torch.where(real, table[b, slot // page] * page + slot % page, -1))
        state["positions"].copy_(torch.where(real, state["seen"][b] + step, 0))
    return {name: state[name] for name in ("table", "held", "free", "n_free", "new_lens", "starts", "slots",
                                           "positions", "missing")}


def work(case):
    if case["op"] == "attn":
        n_q = _spread(case["low"], case["high"], case["batch"])
        heads, dim = case["heads"], case["dim"]
        q_heads = heads * case["group"]
        q_values = q_heads * dim * sum(n_q)
        k_values = heads * dim * sum(n + case["before"] for n in n_q)
        pairs = sum(n * case["before"] + n * (n + 1) // 2 for n in n_q)
        sums = 4 * q_heads * sum(n_q)
        if case["backward"]:           # reads q, k, v, out, dout, lse; writes dq, dk, dv
            return {"bytes": 2 * (4 * q_values + 4 * k_values) + sums, "flops": 10 * dim * q_heads * pairs}
        return {"bytes": 2 * (2 * q_values + 2 * k_values) + sums, "flops": 4 * dim * q_heads * pairs}
    if case["op"] == "rotary":
        rows = case["tokens"] * case["heads"] * (case["group"] + 1)
        return {"bytes": 4 * rows * case["dim"] + 4 * case["tokens"], "flops": 3 * rows * case["part"]}
    if case["op"] == "append":
        rows = case["tokens"] * case["heads"]
        extra = 8 * rows + 4 * case["tokens"] if case["metadata"] else 0
        return {"bytes": 8 * rows * case["dim"] + 4 * (case["tokens"] + case["pad"]) + extra, "flops": 0}
    requests = _requests(case)
    tokens = sum(r[2] for r in requests) + case["pad"]
    moved = sum(abs(-(-(kv + new) // case["page"]) - held) for held, kv, new, _ in requests)
    return {"bytes": 28 * case["batch"] + 8 * tokens + 8 * moved, "flops": 0}


def exact(case, seed):
    """The definitions in 64 bits (whole numbers: by hand), one sequence and head or one entry at a time."""
    state = prepare(case, seed)
    return {"attn": _exact_attn, "rotary": _exact_rotary, "append": _exact_append,
            "reserve": _exact_reserve}[case["op"]](case, state)


def _exact_attn(case, state):
    q, k, v, scale, group = state["q"], state["k"], state["v"], state["scale"], case["group"]
    q_starts, k_starts = state["q_starts"].tolist(), state["k_starts"].tolist()
    double = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.zeros(q.shape, **double), torch.full(q.shape[:2], -math.inf, **double)
    grads = [torch.zeros(x.shape, **double) for x in (q, k, v)]
    step = 1024
    for b in range(case["batch"]):
        n_q, n_k = q_starts[b + 1] - q_starts[b], k_starts[b + 1] - k_starts[b]
        for h in range(case["heads"]):
            for first in range(0, n_q, step):
                rows = min(step, n_q - first)
                seen = n_k - n_q + first + rows          # keys that some row of these attends
                at = slice(q_starts[b] + first, q_starts[b] + first + rows)
                of = slice(k_starts[b], k_starts[b] + seen)
                mine = slice(h * group, (h + 1) * group)
                x, keys, values = q[at, mine].double(), k[of, h].double(), v[of, h].double()
                z = torch.einsum("rgd,kd->grk", x, keys) * scale
                limit = n_k - n_q + first + torch.arange(rows, device="cuda")
                z.masked_fill_((torch.arange(seen, device="cuda")[None] > limit[:, None])[None], -math.inf)
                norm = torch.logsumexp(z, dim=2)
                p = torch.exp(z - norm[..., None])
                if not case["backward"]:
                    out[at, mine] = torch.einsum("grk,kd->rgd", p, values)
                    lse[at, mine] = norm.T
                    continue
                g = state["dout"][at, mine].double()
                inner = torch.einsum("rgd,kd->grk", g, values)
                ds = p * (inner - (p * inner).sum(dim=2, keepdim=True)) * scale
                grads[0][at, mine] = torch.einsum("grk,kd->rgd", ds, keys)
                grads[1][of, h] += torch.einsum("grk,rgd->kd", ds, x)
                grads[2][of, h] += torch.einsum("grk,rgd->kd", p, g)
    if case["backward"]:
        return {"dq": grads[0], "dk": grads[1], "dv": grads[2]}
    return {"out": out, "lse": lse}


def _exact_rotary(case, state):
    part, half = case["part"], case["part"] // 2
    scaling, factor, length = case["scaling"], 8.0, 4096
    base = 10000.0 * factor ** (part / (part - 2)) if scaling == "base" else 10000.0
    speeds, size = [], 1.0
    for i in range(half):
        speed = 1.0 / math.pow(base, 2 * i / part)
        if scaling == "linear":
            speed /= factor
        elif scaling == "factors":
            speed /= 1.0 + 7.0 * (i / half) ** 2
            size = math.sqrt(1.0 + math.log(factor, length))
        elif scaling == "parts":
            low = math.floor(part * math.log(length / (64 * math.pi)) / (2 * math.log(base)))
            high = math.ceil(part * math.log(length / (2 * math.pi)) / (2 * math.log(base)))
            low, high = max(low, 0), min(high, part - 1)
            slowed = min(1.0, max(0.0, (i - low) / (high - low if high > low else 0.001)))
            speed = speed * (1.0 - slowed) + speed / factor * slowed
            size = 1.0 + math.log(factor) / 10.0
        speeds.append(speed)
    turn = state["positions"].double()[:, None, None] * torch.tensor(speeds, dtype=torch.float64, device="cuda")
    if case["transpose"]:
        turn = -turn
    phase = torch.polar(torch.full_like(turn, size), turn)
    result = {}
    for name in ("q", "k"):
        x = state[name].double()
        head = x[..., :part]
        pairs = head.unflatten(2, (half, 2)) if case["interleaved"] else head.unflatten(2, (2, half)).transpose(2, 3)
        turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * phase)
        turned = turned if case["interleaved"] else turned.transpose(2, 3)
        result[name] = torch.cat([turned.flatten(2), x[..., part:]], dim=2)
    return result


def _exact_append(case, state):
    k, v = state["k"].double(), state["v"].double()
    weights = None if state["weights"] is None else state["weights"].double()
    positions = None if state["positions"] is None else state["positions"].clone()
    slots = state["slots"].tolist()
    source = torch.tensor([t for t, s in enumerate(slots) if s >= 0], device="cuda")
    page = torch.tensor([s // case["page"] for s in slots if s >= 0], device="cuda")
    row = torch.tensor([s % case["page"] for s in slots if s >= 0], device="cuda")
    for h in range(case["heads"]):
        k[page, h, row] = state["k_new"][source, h].double()
        v[page, h, row] = state["v_new"][source, h].double()
        if weights is not None:
            weights[page, h, row] = 0.0
            positions[page, h, row] = state["where"][source]
    return {"k": k, "v": v, "weights": weights, "positions": positions}


def _exact_reserve(case, state):
    table, held, free = state["table"].tolist(), state["held"].tolist(), state["free"].tolist()
    kv, n_new, seen, page = state["kv"].tolist(), state["n_new"].tolist(), state["seen"].tolist(), case["page"]
    n = int(state["n_free"])
    need = [-(-(a + b) // page) for a, b in zip(kv, n_new)]
    returned = [p for row, h, m in zip(table, held, need) for p in row[m:h]]
    lacking = max(0, sum(max(0, m - h) for h, m in zip(held, need)) - n - len(returned))
    starts, slots, positions, lens = [0] * (case["batch"] + 1), [], [], list(kv)
    if not lacking:
        spare = 0
        for b, row in enumerate(table):
            for column in range(held[b], need[b]):
                if n:
                    n -= 1
                    row[column] = free[n]
                else:
                    row[column] = returned[spare]
                    spare += 1
        for p in returned[spare:]:
            free[n] = p
            n += 1
        held = need
        lens = [a + b for a, b in zip(kv, n_new)]
        starts = _starts(n_new)
        for b, row in enumerate(table):
            for t in range(n_new[b]):
                slot = kv[b] + t
                slots.append(row[slot // page] * page + slot % page)
                positions.append(seen[b] + t)
    rest = state["slots"].numel() - len(slots)
    return {"table": _ints(table), "held": _ints(held), "free": _ints(free), "n_free": _ints([n]),
            "new_lens": _ints(lens), "starts": _ints(starts), "slots": _ints(slots + [-1] * rest),
            "positions": _ints(positions + [0] * rest), "missing": _ints([lacking])}
