"""Cases of the key-value cache operators: attention of new tokens over a paged cache, attention
over the indexer's selected slots, and eviction by accumulated attention weight.

A case names its operator in "op":

- "decode": one query row (or a few) per sequence attends to a window of its sequence's pages
- "selected": every query row attends to its own list of cache slots (the indexer's output)
- "weights": every position's attention weight, summed over rows and heads, is added to a running sum
- "evict": the positions that a budget keeps are chosen by those sums and moved to other pages

With `own` false run() computes them in elementary torch operations in 32 bits; with `own` true it
calls the framework.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


# --- cases ------------------------------------------------------------------------------------------


def listed():
    return [
        # one user's short chat: the smallest call, all latency
        dict(name="decode one sequence", op="decode", seqs=1, rows=1, lo=1500, hi=1500, window=0, heads=32,
             kv_heads=8, dim=128, type="bf16", cache="bf16"),
        # an ordinary serving batch with grouped heads, lengths ragged by 8x
        dict(name="decode grouped batch", op="decode", seqs=32, rows=1, lo=2048, hi=16384, window=0, heads=32,
             kv_heads=8, dim=128, type="bf16", cache="bf16"),
        # the decode benchmark's batch (64 sequences of 32K-131K positions), 64 heads on one key head
        dict(name="decode shared head long", op="decode", seqs=64, rows=1, lo=32768, hi=131072, window=0,
             heads=64, kv_heads=1, dim=128, type="bf16", cache="bf16"),
        # an 8-bit cache, five query heads to a key head
        dict(name="decode 8-bit cache", op="decode", seqs=24, rows=1, lo=8192, hi=65536, window=0, heads=40,
             kv_heads=8, dim=128, type="bf16", cache="e4m3"),
        # sliding windows with two rows per sequence (one token drafted ahead), small heads
        dict(name="decode windows two rows", op="decode", seqs=17, rows=2, lo=700, hi=20011, window=4096, heads=24,
             kv_heads=6, dim=64, type="fp16", cache="fp16"),
        # what follows the indexer in a decode step
        dict(name="selected decode", op="selected", queries=16, pool=65536, k=512, short=0, heads=64, kv_heads=1,
             dim=128, type="bf16", cache="bf16"),
        # what follows the indexer in a prefill chunk
        dict(name="selected prefill", op="selected", queries=2048, pool=65536, k=1024, short=0, heads=64,
             kv_heads=1, dim=128, type="bf16", cache="bf16"),
        # the start of a prompt: an odd number of rows, the first ones shorter than K; wide grouped heads
        dict(name="selected prefill grouped", op="selected", queries=1001, pool=8192, k=512, short=400, heads=16,
             kv_heads=2, dim=256, type="fp16", cache="fp16"),
        # weights of one short sequence, after its decode step
        dict(name="weights one sequence", op="weights", seqs=1, lo=3001, hi=3001, heads=32, kv_heads=8, dim=128,
             type="bf16", cache="bf16"),
        # weights of a batch of long ones
        dict(name="weights batch", op="weights", seqs=32, lo=4096, hi=32768, heads=64, kv_heads=1, dim=128,
             type="bf16", cache="bf16"),
        # one sequence cut back to its budget
        dict(name="evict one sequence", op="evict", seqs=1, lo=9000, hi=9000, budget=2048, recent=256, kv_heads=1,
             dim=128, cache="bf16"),
        # a whole batch cut back at once
        dict(name="evict batch", op="evict", seqs=32, lo=16384, hi=32768, budget=8192, recent=1024, kv_heads=8,
             dim=128, cache="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = 3.0e9  # bytes; the largest listed case reads and writes about as many
    while True:
        op = rng.choice(["decode", "decode", "selected", "selected", "weights", "evict"])
        dim = rng.choice([64, 128, 128, 256])
        kv_heads = rng.choice([1, 1, 2, 3, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 16, 20, 32, 64] if kv_heads < 3 else [1, 2, 4, 5, 8])
        kind = rng.choice(["bf16", "fp16"])
        cache = rng.choice([kind, kind, "e4m3"])
        hi = _log(rng, 200, 131072)
        lo = rng.choice([hi, max(1, hi // rng.choice([2, 8]))])
        if op == "decode":
            case = dict(op=op, seqs=_log(rng, 1, 96), rows=rng.choice([1, 1, 2, 3]), lo=lo, hi=hi,
                        window=rng.choice([0, 0, _log(rng, 100, 8192)]), heads=heads, kv_heads=kv_heads, dim=dim,
                        type=kind, cache=cache)
            cost = 1.3 * case["seqs"] * case["rows"] * hi
        elif op == "selected":
            k = rng.choice([512, 1024])
            queries = _log(rng, 1, 3000)
            case = dict(op=op, queries=queries, pool=PAGE * _log(rng, k // PAGE, 4096), k=k,
                        short=rng.choice([0, queries // 2]), heads=heads, kv_heads=kv_heads, dim=dim, type=kind,
                        cache=cache)
            cost = 1.3 * queries * k
        elif op == "weights":
            case = dict(op=op, seqs=_log(rng, 1, 64), lo=lo, hi=hi, heads=heads, kv_heads=kv_heads, dim=dim,
                        type=kind, cache=cache)
            cost = 1.3 * case["seqs"] * hi
        else:
            budget = max(1, hi // rng.choice([2, 3, 5]))
            case = dict(op=op, seqs=_log(rng, 1, 48), lo=lo, hi=hi, budget=budget, recent=budget // rng.choice([2, 5]),
                        kv_heads=kv_heads, dim=dim, cache=kind)
            cost = 1.3 * case["seqs"] * hi
        if cost * kv_heads * dim * 4 <= most:
            return case


def _lengths(case):
    """The sequences' lengths: spread over [lo, hi] in a fixed order that is neither rising nor falling."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    return [lo + int((hi - lo) * ((i * 0.618033988749895 + 1.0) % 1.0)) if i else hi for i in range(n)]


def _windows(case):
    """(start, end) of every query row: causal rows at the end of each sequence, cut to the window."""
    got = []
    for n in _lengths(case):
        for j in range(case["rows"]):
            end = max(0, n - (case["rows"] - 1 - j))
            got.append((max(0, end - case["window"]) if case["window"] else 0, end))
    return got


def _counts(case):
    """Valid slots of every row of a "selected" case: the first `short` rows are the prompt's first ones."""
    q, k, short = case["queries"], case["k"], case["short"]
    return [min(k, 1 + (r * k) // short) if r < short else k for r in range(q)]


# --- inputs -----------------------------------------------------------------------------------------


def _normal(shape, gen, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def _tables(lengths, gen, spare):
    """Block table [n, pages] over one shuffled pool of pages; -1 past a sequence's pages."""
    pages = [(n + PAGE - 1) // PAGE for n in lengths]
    width, total = max(pages) + spare, sum(pages) + spare
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    own_pages = torch.arange(width, device="cuda")[None, :]
    count = torch.tensor(pages, device="cuda")[:, None]
    first = torch.cumsum(count, 0) - count
    table = torch.where(own_pages < count, perm[(first + own_pages).clamp(max=total - 1)], -1)
    return table.to(torch.int32).contiguous(), total


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dim, kv = case["op"], case["dim"], case["kv_heads"]
    state = {"case": case, "op": op}
    cache = TYPES[case["cache"]]
    # an 8-bit cache holds its values divided by one scale for the keys and one for the values
    state["k_scale"], state["v_scale"] = (0.25, 0.5) if case["cache"] == "e4m3" else (1.0, 1.0)
    if op == "selected":
        total = case["pool"] // PAGE
        table = None
    else:
        lengths = _lengths(case)
        table, total = _tables(lengths, gen, 2)
    shape = (total, PAGE, kv, dim)
    state["k"] = _normal(shape, gen, 1.0 / state["k_scale"], cache)
    if op != "weights":
        state["v"] = _normal(shape, gen, 1.0 / state["v_scale"], cache)
    if table is not None:
        state["table"] = table
    if op == "evict":
        n, width = table.shape
        state["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        # sums over many steps: a few heavy positions, many light ones, some that no row looked at
        acc = torch.exp(2.0 * torch.randn((n, width * PAGE), generator=gen, device="cuda"))
        state["acc"] = acc * (torch.rand(acc.shape, generator=gen, device="cuda") > 0.1)
        new = (case["budget"] + PAGE - 1) // PAGE
        state["new_table"] = torch.randperm(n * new, generator=gen, device="cuda").to(torch.int32).reshape(n, new)
        for name in ("k", "v"):
            state["new_" + name] = torch.zeros((n * new, PAGE, kv, dim), dtype=cache, device="cuda")
        state["keep"] = torch.empty((n, case["budget"]), dtype=torch.int32, device="cuda")
        state["kept"] = torch.empty((n,), dtype=torch.int32, device="cuda")
        state["kept_acc"] = torch.empty((n, case["budget"]), dtype=torch.float32, device="cuda")
        return state
    heads = case["heads"]
    state["scale"] = 1.0 / math.sqrt(dim)
    if op == "selected":
        rows = case["queries"]
        k, pool = case["k"], case["pool"]
        # ascending positions, one from each of k equal ranges; rows next to each other share most of them
        edge = torch.arange(k + 1, device="cuda") * pool // k
        width = edge[1:] - edge[:-1]
        block = torch.rand(((rows + 31) // 32, k), generator=gen, device="cuda").repeat_interleave(32, 0)[:rows]
        single = torch.rand((rows, k), generator=gen, device="cuda")
        shared = torch.rand((rows, k), generator=gen, device="cuda") < 0.75
        at = (edge[:-1] + (torch.where(shared, block, single) * width).long().clamp(max=width - 1)).long()
        pages = torch.randperm(total, generator=gen, device="cuda")
        count = torch.tensor(_counts(case), device="cuda")
        slots = pages[at // PAGE] * PAGE + at % PAGE
        valid = torch.arange(k, device="cuda")[None, :] < count[:, None]
        state["slots"] = torch.where(valid, slots, -1).to(torch.int32)
        state["count"] = count.to(torch.int32)
    elif op == "decode":
        rows = case["seqs"] * case["rows"]
        windows = _windows(case)
        state["start"] = torch.tensor([w[0] for w in windows], dtype=torch.int32, device="cuda")
        state["end"] = torch.tensor([w[1] for w in windows], dtype=torch.int32, device="cuda")
        state["seq"] = torch.arange(case["seqs"], dtype=torch.int32, device="cuda").repeat_interleave(case["rows"])
    else:
        rows = case["seqs"]
        state["start"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
        state["end"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        state["seq"] = torch.arange(rows, dtype=torch.int32, device="cuda")
    # scores with a spread of about two: most of the weight on a small part of the window
    state["q"] = _normal((rows, heads, dim), gen, 2.0, TYPES[case["type"]])
    if op == "weights":
        state["lse"] = torch.logsumexp(_scores(state)[0], dim=-1).reshape(rows, heads)
        state["acc"] = torch.rand((rows, state["table"].shape[1] * PAGE), generator=gen, device="cuda")
    else:
        state["out"] = torch.empty((rows, heads, dim), dtype=TYPES[case["type"]], device="cuda")
        state["lse"] = torch.empty((rows, heads), dtype=torch.float32, device="cuda")
    return state


# --- the plain form ---------------------------------------------------------------------------------


def _take(pages, index):
    """pages[index]; an 8-bit type is indexed through its bytes."""
    if pages.dtype == torch.float8_e4m3fn:
        return pages.view(torch.uint8)[index].view(torch.float8_e4m3fn)
    return pages[index]


def _rows_of(pages, table):
    """float32 rows [n, positions, kv_heads, dim] of every sequence's pages."""
    got = _take(pages, table.clamp(min=0).long()).float()
    return got.reshape(got.shape[0], got.shape[1] * PAGE, got.shape[3], got.shape[4])


def _products(q, keys, scale):
    """Scores [rows, kv_heads, group, positions] of q [rows, heads, dim] with keys [rows, positions, kv_heads, dim]."""
    rows, heads, dim = q.shape
    kv = keys.shape[2]
    grouped = q.float().reshape(rows, kv, heads // kv, dim)
    return torch.matmul(grouped, keys.permute(0, 2, 3, 1).contiguous()) * scale


def _scores(state):
    """Masked scores of a windowed case, and the mask."""
    keys = _rows_of(state["k"], state["table"])[state["seq"].long()]
    s = _products(state["q"], keys, state["scale"] * state["k_scale"])
    at = torch.arange(s.shape[-1], device=s.device)[None, :]
    inside = (at >= state["start"][:, None]) & (at < state["end"][:, None])
    return s.masked_fill(~inside[:, None, None, :], float("-inf")), inside


def _softmax_values(s, values, v_scale, dtype):
    """The weighted mean of the values under softmax(s), and the logarithm of the sum."""
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(dim=-1, keepdim=True)
    out = torch.matmul(p, values.permute(0, 2, 1, 3).contiguous()) * v_scale
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    rows, kv, group, dim = out.shape
    return {"out": out.reshape(rows, kv * group, dim).to(dtype), "lse": (m + torch.log(total)).reshape(rows, kv * group)}


def _plain_decode(state):
    s, _ = _scores(state)
    values = _rows_of(state["v"], state["table"])[state["seq"].long()]
    return _softmax_values(s, values, state["v_scale"], state["q"].dtype)


def _plain_selected(state):
    slots = state["slots"].clamp(min=0).long()
    kv, dim = state["k"].shape[2:]
    keys = _take(state["k"].reshape(-1, kv, dim), slots).float()
    s = _products(state["q"], keys, state["scale"] * state["k_scale"])
    inside = torch.arange(slots.shape[1], device=s.device)[None, :] < state["count"][:, None]
    s = s.masked_fill(~inside[:, None, None, :], float("-inf"))
    values = _take(state["v"].reshape(-1, kv, dim), slots).float()
    return _softmax_values(s, values, state["v_scale"], state["q"].dtype)


def _plain_weights(state):
    s, _ = _scores(state)
    rows, kv, group, _ = s.shape
    p = torch.exp(s - state["lse"].reshape(rows, kv, group, 1)).sum(dim=(1, 2))
    # one row per sequence here, in order
    state["acc"] += p
    return {"acc": state["acc"]}


def _plain_evict(state):
    acc, length = state["acc"], state["lengths"].long()[:, None]
    budget, recent = state["case"]["budget"], state["case"]["recent"]
    at = torch.arange(acc.shape[1], device=acc.device)[None, :]
    old = at < length - recent
    order = torch.sort(torch.where(old, acc, -1.0), dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, at.expand_as(order))
    kept = (old & ((rank < budget - recent) | (length <= budget))) | ((at >= length - recent) & (at < length))
    count = kept.sum(dim=1, keepdim=True)
    keep = torch.sort(torch.where(kept, at, acc.shape[1]), dim=1).values[:, :budget]
    if keep.shape[1] < budget:
        keep = torch.nn.functional.pad(keep, (0, budget - keep.shape[1]), value=acc.shape[1])
    to = torch.arange(budget, device=acc.device)[None, :].expand(acc.shape[0], -1)
    valid = to < count
    source = keep.clamp(max=acc.shape[1] - 1)
    src = state["table"].long().gather(1, source // PAGE).clamp(min=0) * PAGE + source % PAGE
    dst = state["new_table"].long().gather(1, to // PAGE) * PAGE + to % PAGE
    result = {"keep": torch.where(valid, keep, -1).to(torch.int32), "kept": count[:, 0].to(torch.int32),
              "kept_acc": torch.where(valid, acc.gather(1, source), 0.0)}
    _move(state["k"], src, state["new_k"], dst, valid)
    _move(state["v"], src, state["new_v"], dst, valid)
    return {**result, "k": state["new_k"], "v": state["new_v"]}


def _move(old, src, new, dst, valid):
    flat = new.view(-1, *new.shape[2:])
    rows = old.view(-1, *old.shape[2:])[src]
    flat[dst] = torch.where(valid[:, :, None, None], rows, flat[dst])


# --- the framework's calls --------------------------------------------------------------------------


def _own(state):
    import fp4_mqa_scoring_amd as mqa

    case, op = state["case"], state["op"]
    scales = {"scale": state.get("scale"), "k_scale": state["k_scale"]}
    if "workspace" not in state:  # a program keeps its workspace from call to call
        if op == "decode":
            size = mqa.mqa_kv_attention_decode_workspace_bytes(state["q"].shape[0], case["heads"], case["kv_heads"],
                                                               case["dim"])
        elif op == "selected":
            size = mqa.mqa_kv_attention_selected_workspace_bytes(state["q"].shape[0], case["k"], case["heads"],
                                                                 case["kv_heads"], case["dim"])
        elif op == "evict":
            size = mqa.mqa_kv_evict_workspace_bytes(state["acc"].shape[0], state["acc"].shape[1])
        else:
            size = 0
        state["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    if op == "decode":
        mqa.mqa_kv_attention_decode(state["q"], state["k"], state["v"], state["table"], state["seq"], state["start"],
                                    state["end"], state["out"], state["workspace"], lse=state["lse"],
                                    v_scale=state["v_scale"], **scales)
        return {"out": state["out"], "lse": state["lse"]}
    if op == "selected":
        mqa.mqa_kv_attention_selected(state["q"], state["k"], state["v"], state["slots"], state["count"],
                                      state["out"], state["workspace"], lse=state["lse"], v_scale=state["v_scale"],
                                      **scales)
        return {"out": state["out"], "lse": state["lse"]}
    if op == "weights":
        mqa.mqa_kv_weights_accumulate(state["q"], state["lse"], state["k"], state["table"], state["seq"],
                                      state["start"], state["end"], state["acc"], **scales)
        return {"acc": state["acc"]}
    mqa.mqa_kv_evict_select(state["acc"], state["lengths"], case["budget"], case["recent"], state["keep"],
                            state["kept"], state["workspace"], kept_acc=state["kept_acc"])
    mqa.mqa_kv_compact(state["keep"], state["kept"], state["table"], state["new_table"],
                       [(state["k"], state["new_k"]), (state["v"], state["new_v"])])
    return {"keep": state["keep"], "kept": state["kept"], "kept_acc": state["kept_acc"], "k": state["new_k"],
            "v": state["new_v"]}


def run(state):
    if own:
        return _own(state)
    return {"decode": _plain_decode, "selected": _plain_selected, "weights": _plain_weights,
            "evict": _plain_evict}[state["op"]](state)


# --- what a pass cannot do without ------------------------------------------------------------------


def work(case):
    op, dim, kv = case["op"], case["dim"], case["kv_heads"]
    row = dim * kv * (1 if case["cache"] == "e4m3" else 2)  # bytes of one position's keys (or values)
    if op == "evict":
        kept = sum(min(n, case["budget"]) for n in _lengths(case))
        return {"bytes": 4 * sum(_lengths(case)) + 8 * case["seqs"] * case["budget"] + 4 * kept + 2 * 2 * kept * row,
                "flops": sum(_lengths(case))}
    heads = case["heads"]
    if op == "weights":
        n = sum(_lengths(case))
        return {"bytes": n * (row + 8) + 2 * case["seqs"] * heads * dim + 4 * case["seqs"] * heads,
                "flops": n * heads * (2 * dim + 3)}
    if op == "decode":
        rows = case["seqs"] * case["rows"]
        windows = _windows(case)
        pairs = sum(e - s for s, e in windows)
        # rows of one sequence look at nearly the same window: its positions are read once
        firsts = windows[:: case["rows"]]
        lasts = windows[case["rows"] - 1 :: case["rows"]]
        positions = sum(last[1] - first[0] for first, last in zip(firsts, lasts))
    else:
        rows = case["queries"]
        pairs = sum(_counts(case))
        positions = min(pairs, case["pool"])
    return {"bytes": 2 * positions * row + 2 * 2 * rows * heads * dim + 4 * rows * heads + (4 * pairs if op == "selected" else 0),
            "flops": pairs * heads * (4 * dim + 4)}


# --- the definition in 64 bits ----------------------------------------------------------------------


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(case, state)
    q = state["q"].to(torch.float64)
    rows, heads, dim = q.shape
    kv = case["kv_heads"]
    group = heads // kv
    c = float(state["scale"]) * float(state["k_scale"])
    flat_k = state["k"].view(-1, kv, dim)
    flat_v = state["v"].view(-1, kv, dim) if "v" in state else None
    out = torch.zeros((rows, heads, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, heads), float("-inf"), dtype=torch.float64, device="cuda")
    acc = state["acc"].to(torch.float64) if case["op"] == "weights" else None
    if case["op"] == "selected":
        counts = _counts(case)
    else:
        starts, ends, seqs = (state[n].tolist() for n in ("start", "end", "seq"))
    for r in range(rows):
        if case["op"] == "selected":
            slots = state["slots"][r, : counts[r]].long()
        else:
            at = torch.arange(starts[r], ends[r], device="cuda")
            slots = state["table"][seqs[r]].long()[at // PAGE] * PAGE + at % PAGE
        if slots.numel() == 0:
            continue
        keys = _wide(flat_k, slots)
        for g in range(kv):
            mine = slice(g * group, (g + 1) * group)
            s = (q[r, mine] @ keys[:, g].t()) * c
            if acc is not None:
                acc[seqs[r], at] += torch.exp(s - state["lse"][r, mine, None].to(torch.float64)).sum(0)
                continue
            lse[r, mine] = torch.logsumexp(s, dim=1)
            p = torch.exp(s - lse[r, mine, None])
            out[r, mine] = (p @ _wide(flat_v, slots)[:, g]) * state["v_scale"]
    return {"acc": acc} if acc is not None else {"out": out, "lse": lse}


def _wide(pages, slots):
    """The slots' rows in 64 bits."""
    if pages.dtype == torch.float8_e4m3fn:
        return pages.view(torch.uint8)[slots].view(torch.float8_e4m3fn).to(torch.float64)
    return pages[slots].to(torch.float64)


def _exact_evict(case, state):
    acc, table, new_table = (state[n].cpu().numpy() for n in ("acc", "table", "new_table"))
    n, budget, recent = acc.shape[0], case["budget"], case["recent"]
    keep = np.full((n, budget), -1, np.int32)
    kept = np.zeros(n, np.int32)
    kept_acc = np.zeros((n, budget), np.float64)
    moved = {name: torch.zeros(state["new_" + name].shape, dtype=torch.float64, device="cuda") for name in ("k", "v")}
    for i, length in enumerate(_lengths(case)):
        if length <= budget:
            chosen = np.arange(length)
        else:
            old = length - recent
            best = np.lexsort((np.arange(old), -acc[i, :old].astype(np.float64)))[: budget - recent]
            chosen = np.sort(np.concatenate([best, np.arange(old, length)]))
        m = len(chosen)
        keep[i, :m], kept[i], kept_acc[i, :m] = chosen, m, acc[i, chosen]
        src = torch.from_numpy(table[i, chosen // PAGE].astype(np.int64) * PAGE + chosen % PAGE).cuda()
        to = np.arange(m)
        dst = torch.from_numpy(new_table[i, to // PAGE].astype(np.int64) * PAGE + to % PAGE).cuda()
        for name in ("k", "v"):
            rows = state[name].view(-1, *state[name].shape[2:])[src].to(torch.float64)
            moved[name].view(-1, *state[name].shape[2:])[dst] = rows
    return {"keep": keep, "kept": kept, "kept_acc": kept_acc, "k": moved["k"], "v": moved["v"]}
