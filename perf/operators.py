"""The paged key-value cache's operators as measured workloads.

Three operators share one cache of pages: the append of new tokens, the
attention of one new token over a sequence's pages (optionally adding each
cached token's attention weight to a running sum), and the eviction of the
tokens with the smallest sums.  `run` with `own` false is each operator in
plain torch operations in 32 bits; with `own` true it calls the library.

A cache: k_pages and v_pages [pages, kv heads, page size, d] (three storage
orders), weights fp32 and positions int32 [pages, kv heads, page size], a page
table int32 [batch, pages per sequence].  Slot s of a sequence is row
s % page size of page table[s // page size].
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    attn = dict(op="attn", dtype="bf16", layout="hnd", batch=1, heads=2, group=16, dim=128, page=64, low=1, high=64,
                accumulate=False)
    append = dict(op="append", dtype="bf16", layout="hnd", batch=1, heads=2, dim=128, page=64, low=1, high=64, new=1,
                  metadata=True)
    evict = dict(op="evict", dtype="bf16", layout="hnd", batch=1, heads=2, dim=128, page=64, low=1, high=64,
                 budget=32, initial=4, local=16)
    return [
        # One user's first turns: a short cache, where the latency of the call is all there is.
        dict(attn, name="attn one short sequence", low=517, high=517),
        # One long document, the head layout of the block-sparse decode benchmark (2 KV heads of 16 query
        # heads), with the running sums that a later eviction goes by.
        dict(attn, name="attn one 128K sequence", low=131072, high=131072, accumulate=True),
        # A serving batch in mid-flight: ragged lengths, small pages, token-major storage, fp16.
        dict(attn, name="attn 64 ragged fp16", dtype="fp16", layout="nhd", batch=64, heads=8, group=4, page=16, low=1,
             high=8191, accumulate=True),
        # Many short chats of a model without shared heads, d 64; some slots of the batch are empty.
        dict(attn, name="attn 96 short, unshared heads", batch=96, heads=16, group=1, dim=64, page=32, low=0,
             high=2047),
        # The largest: 32 long contexts at once.
        dict(attn, name="attn 32 long", batch=32, heads=8, group=8, low=16384, high=32768, accumulate=True),
        # One decode step's append for a serving batch.
        dict(append, name="append one token of 64", batch=64, heads=8, page=16, low=1, high=8191),
        # Prompts of ragged length written to their pages.
        dict(append, name="append 8 prompts", batch=8, heads=4, low=301, high=8192, new=8192),
        # A decode loop at its budget: each step brings one token and evicts one.
        dict(evict, name="evict one token of 4097", batch=16, low=4097, high=4097, budget=4096, initial=4, local=256),
        # A 128K prompt cut to a quarter before decoding starts.
        dict(evict, name="evict 128K to 32K", low=131072, high=131072, budget=32768, initial=64, local=2048),
        # A ragged serving batch cut to 4096 tokens each; the shortest stay whole.
        dict(evict, name="evict 32 ragged to 4096", batch=32, heads=8, page=16, low=2000, high=16384, budget=4096,
             initial=4, local=512),
        # Odd sizes: d 64, fp16, a page size that is no power of two, token-major storage.
        dict(evict, name="evict fp16 to 1001", dtype="fp16", layout="nhd", batch=8, heads=4, dim=64, page=48,
             low=1500, high=9999, budget=1001, initial=1, local=100),
    ]


# A drawn case holds at most so many (padded) cache elements, so that it costs
# no more than the largest listed case of its operator.
MOST = {"attn": 8 * 8 * 90000 * 128, "append": 8 * 4 * 4600 * 128, "evict": 16 * 8 * 16384 * 128}


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "evict"])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]), layout=rng.choice(["hnd", "nhd", "pair"]),
                heads=rng.choice([1, 2, 3, 4, 8, 16]), dim=rng.choice([64, 128, 128]),
                page=rng.choice([16, 32, 48, 64, 64, 128, 256]))
    per_slot = case["heads"] * case["dim"]
    high = _log_int(rng, 1 if op != "evict" else 64, 262144)
    high = min(high, MOST[op] // per_slot)
    case["batch"] = _log_int(rng, 1, max(1, min(256, MOST[op] // (per_slot * high))))
    case["high"] = high
    case["low"] = rng.choice([0, 1, high // 2, high]) if op == "attn" else max(1, rng.choice([1, high // 2, high]))
    if op == "attn":
        case["group"] = rng.choice([1, 2, 4, 5, 7, 8, 8, 16, 16, 32])
        case["accumulate"] = rng.random() < 0.5
    elif op == "append":
        case["new"] = rng.choice([1, 1, high])
        case["metadata"] = rng.random() < 0.75
    else:
        case["budget"] = max(16, int(high * rng.uniform(0.1, 0.95)))
        case["initial"] = rng.choice([0, 1, case["budget"] // 16])
        case["local"] = rng.choice([0, 1, case["budget"] // 4])
    return case


def _lengths(case):
    """The batch's cache lengths: spread evenly over [low, high], the longest among them."""
    low, high = case["low"], case["high"]
    spread = [low + int((high - low + 1) * (((i + 1) * 0.6180339887498949) % 1.0)) for i in range(case["batch"])]
    return [high] + spread[1:]


def _new(case):
    """How many tokens of each sequence an append writes: one, or (a prompt) all it has."""
    return [min(case["new"], n) for n in _lengths(case)]


def _pages_each(case):
    return -(-max(case["high"], 1) // case["page"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, dim, heads, batch, page = DTYPES[case["dtype"]], case["dim"], case["heads"], case["batch"], case["page"]
    each = _pages_each(case)
    pages = batch * each

    def normal(*shape):
        return torch.randn(shape, device="cuda", dtype=dtype, generator=gen)

    if case["layout"] == "hnd":      # [page, head, token, d]
        k, v = normal(pages, heads, page, dim), normal(pages, heads, page, dim)
    elif case["layout"] == "nhd":    # [page, token, head, d]
        k, v = (normal(pages, page, heads, dim).transpose(1, 2) for _ in range(2))
    else:                            # keys and values of a page side by side
        both = normal(pages, 2, heads, page, dim)
        k, v = both[:, 0], both[:, 1]
    table = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32).view(batch, each)
    order = torch.randperm(batch, device="cuda", generator=gen)
    lens = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")[order]
    state = dict(op=case["op"], k=k, v=v, table=table, lens=lens, weights=None, positions=None)

    def sums():                      # running sums of attention weights: few large, some exactly zero
        w = torch.randn((pages, heads, page), device="cuda", generator=gen).mul_(2).exp_().mul_(0.01)
        return w.masked_fill_(torch.rand((pages, heads, page), device="cuda", generator=gen) < 0.02, 0.0)

    if case["op"] == "attn":
        group = case["group"]
        q = normal(batch, 1, heads * group, dim)
        # The first token of a sequence draws much of the attention, as it does in trained models.
        sink = torch.randn((heads, dim), device="cuda", generator=gen)
        q += (0.5 * sink).to(dtype).repeat_interleave(group, dim=0)
        k[table[:, 0].long(), :, 0] = (k[table[:, 0].long(), :, 0].float() + sink).to(dtype)
        state.update(q=q, out=torch.empty_like(q), scale=dim ** -0.5,
                     lse=torch.empty((batch, 1, heads * group), device="cuda"))
        if case["accumulate"]:
            state["weights"] = sums()
    elif case["op"] == "append":
        new = torch.tensor(_new(case), dtype=torch.int32, device="cuda")[order]
        most = max(_new(case))
        # Projections leave tokens outside heads: [batch, token, head, d], read here as [batch, head, token, d].
        state.update(k_new=normal(batch, most, heads, dim).transpose(1, 2),
                     v_new=normal(batch, most, heads, dim).transpose(1, 2), n_new=new, most=most,
                     seen=lens + torch.randint(0, 100, (batch,), device="cuda", generator=gen, dtype=torch.int32))
        if case["metadata"]:
            state["weights"] = sums()
            state["positions"] = torch.zeros((pages, heads, page), dtype=torch.int32, device="cuda")
    else:
        # Earlier evictions left gaps in the positions; the newest token is the last one.
        gaps = torch.randint(1, 4, (batch, each * page), device="cuda", generator=gen, dtype=torch.int32)
        where = gaps.cumsum(1, dtype=torch.int32) - 1
        seen = where.gather(1, (lens.long() - 1)[:, None])[:, 0] + 1
        positions = torch.empty((pages, heads, page), dtype=torch.int32, device="cuda")
        positions[table.long()] = where.view(batch, each, 1, page).expand(-1, -1, heads, -1)
        # The sums and positions that the step before left; `run` starts from them each time.
        before = torch.stack([sums().view(torch.int32), positions])
        now = before.clone()
        state.update(before=before, now=now, weights=now[0].view(torch.float32), positions=now[1], seen=seen,
                     budget=case["budget"], initial=case["initial"], local=case["local"],
                     new_lens=torch.empty_like(lens))
    if own:
        import trainable_block_sparse_infllm_gb300 as T
        cache = T.PagedCache(k, v, state["weights"], state["positions"])
        state["cache"], state["T"] = cache, T
        if case["op"] == "attn":
            state["workspace"] = T.alloc_paged_workspace(cache, table, T.OP_PAGED_DECODE, case["group"])
        elif case["op"] == "evict":
            state["workspace"] = T.alloc_paged_workspace(cache, table, T.OP_PAGED_EVICT)
    return state


def run(state):
    return {"attn": _attn, "append": _append, "evict": _evict}[state["op"]](state)


def _slots(state):
    """The page and row of every slot, [batch, slots] each."""
    page = state["k"].shape[2]
    table = state["table"].long()
    rows = torch.arange(page, device=table.device)
    return table.repeat_interleave(page, dim=1), rows.repeat(table.shape[1])[None].expand(table.shape[0], -1)


def _attn(state):
    accumulate = state["weights"] is not None
    if own:
        state["T"].paged_attn_decode(state["cache"], state["q"], state["table"], state["lens"], state["out"],
                                     state["lse"], scale=state["scale"], accumulate=accumulate,
                                     workspace=state["workspace"])
    else:
        table = state["table"].long()
        batch, each = table.shape
        _, heads, page, dim = state["k"].shape
        q = state["q"].float().view(batch, heads, -1, dim)
        seen = torch.arange(each * page, device=table.device)[None] < state["lens"][:, None]
        seen = seen[:, None, None]
        k = state["k"][table].transpose(1, 2).reshape(batch, heads, each * page, dim).float()
        z = torch.matmul(q, k.transpose(2, 3)).mul_(state["scale"]).masked_fill_(~seen, -math.inf)
        del k
        top = z.amax(dim=3, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
        z = z.sub_(top).exp_()
        total = z.sum(dim=3, keepdim=True)
        v = state["v"][table].transpose(1, 2).reshape(batch, heads, each * page, dim).float()
        out = torch.matmul(z, v).div_(total.clamp_min(torch.finfo(torch.float32).tiny))
        del v
        state["out"].copy_(out.view(batch, 1, -1, dim))
        state["lse"].copy_((top + total.log()).view(batch, 1, -1))
        if accumulate:
            w = z.div_(total.clamp_min(torch.finfo(torch.float32).tiny)).sum(dim=2)
            w = w.view(batch, heads, each, page).transpose(1, 2).reshape(-1, heads, page)
            state["weights"].index_add_(0, table.reshape(-1), w)
    return {"out": state["out"], "lse": state["lse"], "weights": state["weights"]}


def _append(state):
    if own:
        state["T"].paged_append_kv(state["cache"], state["k_new"], state["v_new"], state["table"], state["lens"],
                                   n_new=state["n_new"], seq_lens=state["seen"])
    else:
        batch, most = state["lens"].shape[0], state["most"]
        page = state["k"].shape[2]
        steps = torch.arange(most, device="cuda")[None]
        n_new = state["n_new"].long()[:, None]
        # A sequence with fewer new tokens writes its last one again in place of those it lacks.
        token = torch.minimum(steps, n_new - 1)
        slot = state["lens"].long()[:, None] - n_new + token
        at, row = state["table"].long().gather(1, slot // page), slot % page
        which = torch.arange(batch, device="cuda")[:, None]
        state["k"][at, :, row] = state["k_new"][which, :, token]
        state["v"][at, :, row] = state["v_new"][which, :, token]
        if state["weights"] is not None:
            state["weights"][at, :, row] = 0.0
            where = state["seen"].long()[:, None] - n_new + token
            state["positions"][at, :, row] = where.to(torch.int32)[..., None].expand(-1, -1, state["k"].shape[1])
    return {"k": state["k"], "v": state["v"], "weights": state["weights"], "positions": state["positions"]}


def _evict(state):
    state["now"].copy_(state["before"])
    if own:
        state["T"].paged_evict(state["cache"], state["table"], state["lens"], state["new_lens"], state["budget"],
                               n_init=state["initial"], n_local=state["local"], seq_lens=state["seen"],
                               workspace=state["workspace"])
    else:
        budget, heads = state["budget"], state["k"].shape[1]
        at, row = _slots(state)
        batch, slots = at.shape
        lens = state["lens"].long()[:, None, None]
        index = torch.arange(slots, device="cuda").expand(batch, heads, -1)
        held = index < lens
        weight = state["weights"][at, :, row].transpose(1, 2)
        where = state["positions"][at, :, row].transpose(1, 2)
        always = (where < state["initial"]) | (where >= state["seen"][:, None, None] - state["local"])
        weight = weight.masked_fill(always, math.inf).masked_fill(~held, -math.inf)
        best = weight.sort(dim=2, descending=True, stable=True).indices
        kept = torch.zeros_like(held).scatter_(2, best[:, :, :budget], True) & held
        hole = ~kept & held & (index < budget)
        mover = kept & (index >= budget)
        movers = mover.to(torch.int8).sort(dim=2, descending=True, stable=True).indices
        first = min(budget, slots)
        rank = (hole.long().cumsum(2) - 1).clamp_min(0)
        source = torch.where(hole, movers.gather(2, rank), index)[:, :, :first]
        head = torch.arange(heads, device="cuda")[None, :, None]
        from_page = at[:, None].expand(-1, heads, -1).gather(2, source)
        from_row = row[:, None].expand(-1, heads, -1).gather(2, source)
        to_page, to_row = at[:, None, :first], row[:, None, :first]
        for t in (state["k"], state["v"], state["weights"], state["positions"]):
            t[to_page, head, to_row] = t[from_page, head, from_row]
        torch.minimum(state["lens"], torch.full_like(state["lens"], budget), out=state["new_lens"])
    return {"k": state["k"], "v": state["v"], "weights": state["weights"], "positions": state["positions"],
            "new_lens": state["new_lens"]}


def work(case):
    lengths, heads, dim, batch = _lengths(case), case["heads"], case["dim"], case["batch"]
    row = 4 * dim                                  # a key and a value of 16 bits
    table = 4 * sum(-(-n // case["page"]) for n in lengths) + 4 * batch
    if case["op"] == "attn":
        query = batch * heads * case["group"]
        sums = 8 * heads * sum(lengths) if case["accumulate"] else 0
        return {"bytes": heads * sum(lengths) * row + query * (4 * dim + 4) + sums + table,
                "flops": 4 * dim * heads * case["group"] * sum(lengths)}
    if case["op"] == "append":
        new = sum(_new(case))
        return {"bytes": new * heads * (2 * row + (8 if case["metadata"] else 0)) + 12 * batch, "flops": 0}
    # Weights that do not depend on the slot: of the slots below the budget, the share beyond it is replaced.
    budget = case["budget"]
    over = [n for n in lengths if n > budget]
    free = max(0, budget - case["initial"] - case["local"])
    moved = sum(max(1.0, free * (n - budget) / n + min(case["local"], n - budget) * budget / n) for n in over)
    return {"bytes": heads * (8 * sum(over) + moved * 2 * (row + 8)) + table + 8 * batch, "flops": 0}


def exact(case, seed):
    """The definitions in 64 bits, one sequence (and for the eviction one head) at a time."""
    state = prepare(case, seed)
    table, lens, page = state["table"].tolist(), state["lens"].tolist(), case["page"]
    heads, dim = case["heads"], case["dim"]

    def places(b, slots):
        slots = torch.as_tensor(slots, device="cuda", dtype=torch.int64)
        return torch.tensor(table[b], device="cuda")[slots // page], slots % page

    if case["op"] == "attn":
        group = case["group"]
        out = torch.zeros((case["batch"], 1, heads * group, dim), dtype=torch.float64, device="cuda")
        lse = torch.full((case["batch"], 1, heads * group), -math.inf, dtype=torch.float64, device="cuda")
        weights = state["weights"].double() if case["accumulate"] else None
        for b, n in enumerate(lens):
            if n == 0:
                continue
            at, row = places(b, range(n))
            k, v = state["k"][at, :, row].double(), state["v"][at, :, row].double()
            q = state["q"][b, 0].double().view(heads, group, dim)
            z = torch.einsum("hgd,nhd->hgn", q, k) * state["scale"]
            norm = torch.logsumexp(z, dim=2)
            p = torch.exp(z - norm[..., None])
            out[b, 0] = torch.einsum("hgn,nhd->hgd", p, v).reshape(-1, dim)
            lse[b, 0] = norm.reshape(-1)
            if weights is not None:
                weights[at, :, row] += p.sum(dim=1).T
        return {"out": out, "lse": lse, "weights": weights}

    k, v = state["k"].double(), state["v"].double()
    weights = state["weights"].double() if state["weights"] is not None else None
    positions = state["positions"].clone() if state["positions"] is not None else None
    if case["op"] == "append":
        for b, n in enumerate(lens):
            n_new = int(state["n_new"][b])
            at, row = places(b, range(n - n_new, n))
            k[at, :, row] = state["k_new"][b, :, :n_new].double().transpose(0, 1)
            v[at, :, row] = state["v_new"][b, :, :n_new].double().transpose(0, 1)
            if weights is not None:
                weights[at, :, row] = 0.0
                last = int(state["seen"][b])
                positions[at, :, row] = torch.arange(last - n_new, last, dtype=torch.int32, device="cuda")[:, None]
        return {"k": k, "v": v, "weights": weights, "positions": positions}

    budget = case["budget"]
    for b, n in enumerate(lens):
        if n <= budget:
            continue
        at, row = places(b, range(n))
        last = int(state["seen"][b])
        for h in range(heads):
            w, p = weights[at, h, row].cpu(), positions[at, h, row].cpu()
            free = ~((p < case["initial"]) | (p >= last - case["local"]))
            by_weight = torch.argsort(w, descending=True, stable=True)
            ranked = by_weight[torch.argsort(free[by_weight].int(), stable=True)]
            keep = torch.zeros(n, dtype=torch.bool)
            keep[ranked[:budget]] = True
            to = torch.nonzero(~keep[:budget])[:, 0].cuda()
            source = (torch.nonzero(keep[budget:])[:, 0] + budget).cuda()
            for t in (k, v, weights, positions):
                t[at[to], h, row[to]] = t[at[source], h, row[source]]
    return {"k": k, "v": v, "weights": weights, "positions": positions,
            "new_lens": torch.tensor([min(n, budget) for n in lens], dtype=torch.int32, device="cuda")}
