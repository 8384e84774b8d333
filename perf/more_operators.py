"""Cases of what fills a paged key-value cache and of attention over one held in 4 bits.

A case names its operator in "op":

- "rotate": every head of new queries and keys is divided by its root mean square, weighted, and rotated by its
  position, in one pass
- "append": new keys and values go to their positions of a paged cache in 16, 8 or 4 bits, the keys normed and rotated
  on the way; with "heads" the same call norms and rotates the queries
- "decode": one query row (or a few) per sequence attends to a window of its sequence's pages, held in 4 bits
- "selected": every query row attends to its own list of slots (the indexer's output) of a cache held in 4 bits

A 4-bit cache holds E2M1 codes, two to a byte, and one UE8M0 scale for 32 dims of a head: the indexer's own format.

With `own` false run() computes them in elementary torch operations in 32 bits (angles in 64); with `own` true it calls
the framework.
"""
import math

import torch

own = False

PAGE = 64
BLOCK = 32  # dims that share a scale
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
EPS = 1e-6
LARGEST = 448.0  # of e4m3
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --- cases ------------------------------------------------------------------------------------------


def listed():
    return [
        # one user's next token: the smallest call, all latency
        dict(name="rotate one token", op="rotate", rows=1, heads=32, kv_heads=8, dim=128, type="bf16", norm=True,
             rotary=128, offset=0, interleaved=False, base=1e6, far=40000),
        # a decode batch of the indexer's model: 64 heads on one key head, the last 64 dims rotated in pairs, no norm
        dict(name="rotate shared head batch", op="rotate", rows=64, heads=64, kv_heads=1, dim=128, type="bf16",
             norm=False, rotary=64, offset=64, interleaved=True, base=1e4, far=500000),
        # a chunk of a prompt
        dict(name="rotate prompt chunk", op="rotate", rows=8192, heads=40, kv_heads=8, dim=128, type="bf16", norm=True,
             rotary=128, offset=0, interleaved=False, base=1e6, far=100000),
        # an odd number of rows, wide heads of which a quarter is rotated
        dict(name="rotate wide heads", op="rotate", rows=1001, heads=16, kv_heads=2, dim=256, type="fp16", norm=True,
             rotary=64, offset=0, interleaved=False, base=1e4, far=8000),
        # what a decode step writes, with its queries: one token of each sequence
        dict(name="append decode batch", op="append", seqs=32, lo=100, hi=1000, rows=1, heads=32, kv_heads=8, dim=128,
             type="bf16", cache="bf16", norm=True, rotary=128, offset=0, interleaved=False, base=1e6, far=0),
        # prompts of several users, into an 8-bit cache; their first positions are another request's
        dict(name="append prompts 8-bit", op="append", seqs=5, lo=700, hi=1500, rows=820, heads=0, kv_heads=8, dim=128,
             type="bf16", cache="e4m3", norm=False, rotary=128, offset=0, interleaved=False, base=1e4, far=0),
        # one long prompt's chunk, into a 4-bit cache, at positions that an eviction has moved
        dict(name="append prompt 4-bit", op="append", seqs=1, lo=5003, hi=5003, rows=4096, heads=0, kv_heads=8, dim=128,
             type="bf16", cache="fp4", norm=True, rotary=128, offset=0, interleaved=False, base=1e6, far=30000),
        # one user's short chat
        dict(name="decode one sequence", op="decode", seqs=1, rows=1, lo=1500, hi=1500, window=0, heads=32, kv_heads=8,
             dim=128, type="bf16"),
        # an ordinary serving batch with grouped heads, lengths ragged by 8x
        dict(name="decode grouped batch", op="decode", seqs=32, rows=1, lo=2048, hi=16384, window=0, heads=32,
             kv_heads=8, dim=128, type="bf16"),
        # the decode benchmark's batch (64 sequences of 32K-131K positions), 64 heads on one key head
        dict(name="decode shared head long", op="decode", seqs=64, rows=1, lo=32768, hi=131072, window=0, heads=64,
             kv_heads=1, dim=128, type="bf16"),
        # what follows the indexer in a decode step
        dict(name="selected decode", op="selected", queries=16, pool=65536, k=512, short=0, heads=64, kv_heads=1,
             dim=128, type="bf16"),
        # what follows the indexer in a prefill chunk, the first rows shorter than K
        dict(name="selected prefill", op="selected", queries=2048, pool=65536, k=1024, short=300, heads=64, kv_heads=1,
             dim=128, type="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = 7.0e8  # bytes; the largest listed case reads about 1.4e9
    while True:
        op = rng.choice(["rotate", "append", "append", "decode", "decode", "selected"])
        dim = rng.choice([64, 128, 128, 256])
        kind = rng.choice(["bf16", "fp16"])
        kv_heads = rng.choice([1, 1, 2, 3, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 16, 20, 32, 64] if kv_heads < 3 else [1, 2, 4, 5, 8])
        rotary = rng.choice([dim, dim, dim // 2, 32, 48, 0])
        turn = dict(norm=rng.choice([True, False]), rotary=rotary, offset=rng.choice([0, dim - rotary]) if rotary else 0,
                    interleaved=rng.choice([True, False]), base=rng.choice([1e4, 5e5, 1e6]),
                    far=rng.choice([0, _log(rng, 1000, 1000000)]))
        if op == "rotate":
            rows = _log(rng, 1, 16384)
            case = dict(op=op, rows=rows, heads=heads, kv_heads=rng.choice([0, kv_heads]), dim=dim, type=kind, **turn)
            cost = 4 * rows * (heads + kv_heads) * dim
        elif op == "append":
            cache = rng.choice([kind, "e4m3", "fp4"])
            seqs = _log(rng, 1, 64)
            hi = _log(rng, 64, 6000)
            lo = max(1, hi // rng.choice([1, 2, 8]))
            case = dict(op=op, seqs=seqs, lo=lo, hi=hi, rows=rng.choice([1, 1, 2, _log(rng, 1, hi)]),
                        heads=rng.choice([0, 0, heads]), kv_heads=kv_heads, dim=dim, type=kind, cache=cache, **turn)
            cost = 4 * seqs * hi * kv_heads * dim
        elif op == "decode":
            hi = _log(rng, 200, 131072)
            lo = rng.choice([hi, max(1, hi // rng.choice([2, 8]))])
            case = dict(op=op, seqs=_log(rng, 1, 96), rows=rng.choice([1, 1, 2, 3]), lo=lo, hi=hi,
                        window=rng.choice([0, 0, _log(rng, 100, 8192)]), heads=heads, kv_heads=kv_heads, dim=dim,
                        type=kind)
            cost = 1.1 * case["seqs"] * case["rows"] * hi * kv_heads * dim
        else:
            k = rng.choice([512, 1024])
            queries = _log(rng, 1, 3000)
            case = dict(op=op, queries=queries, pool=PAGE * _log(rng, k // PAGE, 4096), k=k,
                        short=rng.choice([0, queries // 2]), heads=heads, kv_heads=kv_heads, dim=dim, type=kind)
            cost = 1.1 * queries * k * kv_heads * dim
        if cost <= most:
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


def _new_rows(case):
    """(sequence, position) of every row that an "append" case writes: the last rows of each sequence."""
    return [(i, p) for i, n in enumerate(_lengths(case)) for p in range(max(0, n - case["rows"]), n)]


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


def _pack(values, scale_bytes):
    """(codes, scale bytes) of E2M1 values [..., dim] and their blocks' exponents: two codes to a byte, the even dim low."""
    table = torch.tensor(E2M1, device=values.device)
    code = torch.bucketize(values.abs(), table) + 8 * torch.signbit(values)
    code = code.to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale_bytes.to(torch.uint8)


def _fp4_pool(total, kv, dim, gen):
    """Codes and scales of normal keys (or values), a slice of the pool at a time."""
    codes = torch.empty((total, PAGE, kv, dim // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((total, PAGE, kv, dim // BLOCK), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (PAGE * kv * dim))
    for at in range(0, total, step):
        n = min(step, total - at)
        x = torch.randn((n, PAGE, kv, dim), generator=gen, device="cuda")
        codes[at : at + n], scales[at : at + n] = _pack(*_blocks(x))
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dim, kv, kind = case["op"], case["dim"], case["kv_heads"], TYPES[case["type"]]
    state = {"case": case, "op": op}
    if op in ("rotate", "append"):
        heads = case["heads"]
        if op == "append":
            table, total = _tables(_lengths(case), gen, 2)
            state["table"] = table
            rows = torch.tensor(_new_rows(case), dtype=torch.int32, device="cuda")
            state["seq"], state["at"] = rows[:, 0].contiguous(), rows[:, 1].contiguous()
            # rotated by the position in the cache, or (behind an eviction, or a shared prefix) by the token's own
            state["position"] = state["at"] + case["far"]
            n = rows.shape[0]
        else:
            n = case["rows"]
            first = int(torch.randint(0, max(1, case["far"]), (1,), generator=gen, device="cuda"))
            state["position"] = torch.arange(first, first + n, device="cuda").to(torch.int32)
        # one fused projection's output: queries, keys and values of a row beside each other
        wide = heads + kv * (2 if op == "append" else 1)
        fused = _normal((n, wide, dim), gen, 1.0, kind)
        state["q"], state["k"], state["v"] = fused[:, :heads], fused[:, heads : heads + kv], fused[:, heads + kv :]
        if case["rotary"]:
            i = torch.arange(0, case["rotary"], 2, device="cuda", dtype=torch.float64) / case["rotary"]
            state["freq"] = (case["base"] ** -i).float()
        if case["norm"]:
            state["q_weight"] = _normal((dim,), gen, 0.2, torch.float32).add(1.0).to(kind)
            state["k_weight"] = _normal((dim,), gen, 0.2, torch.float32).add(1.0).to(kind)
        state["q_out"] = torch.empty((n, heads, dim), dtype=kind, device="cuda")
        if op == "rotate":
            state["k_out"] = torch.empty((n, kv, dim), dtype=kind, device="cuda")
        elif case["cache"] == "fp4":
            state["k_pages"], state["k_blocks"] = _fp4_pool(total, kv, dim, gen)
            state["v_pages"], state["v_blocks"] = _fp4_pool(total, kv, dim, gen)
            # every byte's two values, and every scale, in a type that holds them
            pairs = torch.tensor([[E2M1[b & 7] * (-1 if b & 8 else 1) for b in (byte & 15, byte >> 4)] for byte in range(256)],
                                 device="cuda")
            state["pairs"] = pairs.to(torch.float8_e4m3fn).view(torch.int16).reshape(256)
            powers = torch.exp2(torch.arange(256, device="cuda", dtype=torch.float64) - 127.0)
            state["powers"] = powers.clamp(2.0**-9, 256.0).float().to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            state["k_scale"], state["v_scale"] = (0.03125, 0.0625) if case["cache"] == "e4m3" else (1.0, 1.0)
            for name, scale in (("k_pages", state["k_scale"]), ("v_pages", state["v_scale"])):
                state[name] = _normal((total, PAGE, kv, dim), gen, 1.0 / scale, TYPES[case["cache"]])
        return state
    heads = case["heads"]
    if op == "selected":
        total = case["pool"] // PAGE
    else:
        lengths = _lengths(case)
        state["table"], total = _tables(lengths, gen, 2)
    state["k_pages"], state["k_blocks"] = _fp4_pool(total, kv, dim, gen)
    state["v_pages"], state["v_blocks"] = _fp4_pool(total, kv, dim, gen)
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
    else:
        rows = case["seqs"] * case["rows"]
        windows = _windows(case)
        state["start"] = torch.tensor([w[0] for w in windows], dtype=torch.int32, device="cuda")
        state["end"] = torch.tensor([w[1] for w in windows], dtype=torch.int32, device="cuda")
        state["seq"] = torch.arange(case["seqs"], dtype=torch.int32, device="cuda").repeat_interleave(case["rows"])
    # scores with a spread of about two: most of the weight on a small part of the window
    state["q"] = _normal((rows, heads, dim), gen, 2.0, kind)
    state["out"] = torch.empty((rows, heads, dim), dtype=kind, device="cuda")
    state["lse"] = torch.empty((rows, heads), dtype=torch.float32, device="cuda")
    return state


# --- the plain form ---------------------------------------------------------------------------------


def _blocks(x):
    """E2M1 values [..., dim] of x / scale and the scales' bytes [..., dim / 32] (the OCP rule: the exponent of the
    block's largest magnitude less two; nearest value, ties to the even code, saturating at 6)."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    top = b.abs().amax(dim=-1, keepdim=True)
    byte = (torch.frexp(top).exponent - 1 - 2 + 127).clamp(0, 254)
    byte = torch.where(top > 0, byte, torch.zeros_like(byte))
    t = torch.ldexp(b, 127 - byte)
    a = t.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    near = (torch.round(a / step) * step).clamp(max=6.0)
    return torch.copysign(near, t).reshape(x.shape), byte[..., 0]


def _values_of(codes, blocks):
    """float32 values [..., dim] that codes and block scales stand for."""
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    both = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    scale = torch.ldexp(torch.ones((), device=codes.device), blocks.int() - 127)
    return table[both.int()] * scale.repeat_interleave(BLOCK, dim=-1)


def _turned(state, x, weight):
    """float32 rows x [n, heads, dim], normed by `weight` and rotated by the rows' positions."""
    case = state["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight.float()
    rotary, at = case["rotary"], case["offset"]
    if not rotary:
        return x
    angle = state["position"].double()[:, None] * state["freq"].double()[None, :]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    part = x[..., at : at + rotary]
    if case["interleaved"]:
        one, two = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([one * cos - two * sin, two * cos + one * sin], dim=-1).flatten(-2)
    else:
        one, two = part[..., : rotary // 2], part[..., rotary // 2 :]
        turned = torch.cat([one * cos - two * sin, two * cos + one * sin], dim=-1)
    return torch.cat([x[..., :at], turned, x[..., at + rotary :]], dim=-1)


def _plain_rotate(state):
    q = _turned(state, state["q"], state.get("q_weight")).to(state["q"].dtype)
    k = _turned(state, state["k"], state.get("k_weight")).to(state["k"].dtype)
    return {"q": q, "k": k}


def _plain_append(state):
    case = state["case"]
    page = state["table"].long()[state["seq"].long(), state["at"].long() // PAGE]
    where = (page, state["at"].long() % PAGE)
    k, v = _turned(state, state["k"], state.get("k_weight")), state["v"].float()
    for name, x in (("k", k), ("v", v)):
        pages = state[name + "_pages"]
        if case["cache"] == "fp4":
            pages[where], state[name + "_blocks"][where] = _pack(*_blocks(x))
        elif case["cache"] == "e4m3":
            # indexed through its bytes
            held = (x / state[name + "_scale"]).clamp(-LARGEST, LARGEST).to(pages.dtype)
            pages.view(torch.uint8)[where] = held.view(torch.uint8)
        else:
            pages[where] = x.to(pages.dtype)
    result = _written(state)
    if case["heads"]:
        result["q"] = _turned(state, state["q"], state.get("q_weight")).to(state["q"].dtype)
    return result


def _written(state):
    """The cache, as the values that it stands for."""
    if state["case"]["cache"] != "fp4":
        return {"k_pages": state["k_pages"], "v_pages": state["v_pages"]}
    result = {}
    for name in ("k", "v"):
        codes, blocks = state[name + "_pages"], state[name + "_blocks"]
        values = state["pairs"].index_select(0, codes.reshape(-1).int()).view(torch.float8_e4m3fn)
        scales = state["powers"].index_select(0, blocks.reshape(-1).int()).view(torch.float8_e4m3fn)
        result[name + "_values"] = values.reshape(*codes.shape[:-1], -1)
        result[name + "_scales"] = scales.reshape(blocks.shape)
    return result


def _products(q, keys, scale):
    """Scores [rows, kv_heads, group, positions] of q [rows, heads, dim] with keys [rows, positions, kv_heads, dim]."""
    rows, heads, dim = q.shape
    kv = keys.shape[2]
    grouped = q.float().reshape(rows, kv, heads // kv, dim)
    return torch.matmul(grouped, keys.permute(0, 2, 3, 1).contiguous()) * scale


def _softmax_values(s, values, dtype):
    """The weighted mean of the values under softmax(s), and the logarithm of the sum."""
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(dim=-1, keepdim=True)
    out = torch.matmul(p, values.permute(0, 2, 1, 3).contiguous())
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    rows, kv, group, dim = out.shape
    return {"out": out.reshape(rows, kv * group, dim).to(dtype), "lse": (m + torch.log(total)).reshape(rows, kv * group)}


def _rows_of(state, name):
    """float32 rows [rows, positions, kv_heads, dim] of every query row's sequence."""
    pages = state["table"].clamp(min=0).long()
    got = _values_of(state[name + "_pages"][pages], state[name + "_blocks"][pages])
    return got.reshape(got.shape[0], got.shape[1] * PAGE, *got.shape[3:])[state["seq"].long()]


def _plain_decode(state):
    s = _products(state["q"], _rows_of(state, "k"), state["scale"])
    at = torch.arange(s.shape[-1], device=s.device)[None, :]
    inside = (at >= state["start"][:, None]) & (at < state["end"][:, None])
    return _softmax_values(s.masked_fill(~inside[:, None, None, :], float("-inf")), _rows_of(state, "v"), state["q"].dtype)


def _plain_selected(state):
    slots = state["slots"].clamp(min=0).long()
    take = lambda name: _values_of(state[name + "_pages"].flatten(0, 1)[slots], state[name + "_blocks"].flatten(0, 1)[slots])  # noqa: E731
    s = _products(state["q"], take("k"), state["scale"])
    inside = torch.arange(slots.shape[1], device=s.device)[None, :] < state["count"][:, None]
    return _softmax_values(s.masked_fill(~inside[:, None, None, :], float("-inf")), take("v"), state["q"].dtype)


# --- the framework's calls --------------------------------------------------------------------------


def _own(state):
    import fp4_mqa_scoring_amd as mqa

    case, op = state["case"], state["op"]
    if op in ("rotate", "append"):
        turn = dict(inv_freq=state.get("freq"), q_weight=state.get("q_weight"), k_weight=state.get("k_weight"), eps=EPS,
                    rotary_offset=case["offset"], interleaved=case["interleaved"])
        if op == "rotate":
            if case["kv_heads"]:
                turn.update(k=state["k"], k_out=state["k_out"])
            else:
                turn.pop("k_weight")
            mqa.mqa_kv_norm_rotate(state["q"], state["q_out"], state["position"], **turn)
            return {"q": state["q_out"], "k": state["k_out"]}
        if case["heads"]:
            turn.update(q=state["q"], q_out=state["q_out"])
        else:
            turn.pop("q_weight")
        turn["rotary_position"] = state["position"]
        if case["cache"] == "fp4":
            mqa.mqa_kv_append_fp4(state["k"], state["v"], state["k_pages"], state["k_blocks"], state["v_pages"],
                                  state["v_blocks"], state["table"], state["seq"], state["at"], **turn)
        else:
            mqa.mqa_kv_append(state["k"], state["v"], state["k_pages"], state["v_pages"], state["table"], state["seq"],
                              state["at"], k_scale=state["k_scale"], v_scale=state["v_scale"], **turn)
        result = _written(state)
        if case["heads"]:
            result["q"] = state["q_out"]
        return result
    cache = (state["k_pages"], state["k_blocks"], state["v_pages"], state["v_blocks"])
    if "workspace" not in state:  # a program keeps its workspace from call to call
        sizes = (case["heads"], case["kv_heads"], case["dim"])
        if op == "decode":
            size = mqa.mqa_kv_attention_decode_workspace_bytes(state["q"].shape[0], *sizes)
        else:
            size = mqa.mqa_kv_attention_selected_workspace_bytes(state["q"].shape[0], case["k"], *sizes)
        state["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    if op == "decode":
        mqa.mqa_kv_attention_decode_fp4(state["q"], *cache, state["table"], state["seq"], state["start"], state["end"],
                                        state["out"], state["workspace"], lse=state["lse"], scale=state["scale"])
    else:
        mqa.mqa_kv_attention_selected_fp4(state["q"], *cache, state["slots"], state["count"], state["out"],
                                          state["workspace"], lse=state["lse"], scale=state["scale"])
    return {"out": state["out"], "lse": state["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"rotate": _plain_rotate, "append": _plain_append, "decode": _plain_decode,
            "selected": _plain_selected}[state["op"]](state)


# --- what a pass cannot do without ------------------------------------------------------------------


def work(case):
    op, dim, kv = case["op"], case["dim"], case["kv_heads"]
    if op in ("rotate", "append"):
        rows = case["rows"] if op == "rotate" else len(_new_rows(case))
        per = 2 * case["heads"] * 2 * dim  # queries read and written
        if op == "rotate":
            per += 2 * kv * 2 * dim + 4
        else:
            held = dim * 2 if case["cache"] == case["type"] else dim if case["cache"] == "e4m3" else dim // 2 + dim // BLOCK
            per += 2 * kv * (2 * dim + held) + 12 + 4
        turned = (case["heads"] + kv) * dim
        return {"bytes": rows * per, "flops": rows * turned * ((4 if case["norm"] else 0) + 3)}
    heads = case["heads"]
    row = kv * (dim // 2 + dim // BLOCK)  # bytes of one position's keys (or values)
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
    if case["op"] == "rotate":
        return {"q": _exact_turn(state, "q"), "k": _exact_turn(state, "k")}
    if case["op"] == "append":
        return _exact_append(case, state)
    q = state["q"].to(torch.float64)
    rows, heads, dim = q.shape
    kv = case["kv_heads"]
    group = heads // kv
    out = torch.zeros((rows, heads, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, heads), float("-inf"), dtype=torch.float64, device="cuda")
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
        keys, values = (_wide(state[n + "_pages"], state[n + "_blocks"], slots) for n in ("k", "v"))
        for g in range(kv):
            mine = slice(g * group, (g + 1) * group)
            s = (q[r, mine] @ keys[:, g].t()) * float(state["scale"])
            lse[r, mine] = torch.logsumexp(s, dim=1)
            out[r, mine] = torch.exp(s - lse[r, mine, None]) @ values[:, g]
    return {"out": out, "lse": lse}


def _wide(pages, blocks, slots):
    """The slots' rows [n, kv_heads, dim] in 64 bits: code s eem stands for (-1)^s m / 2 where ee is 0, else for
    (-1)^s (1 + m / 2) 2^(ee - 1)."""
    code = pages.reshape(-1, *pages.shape[2:])[slots].to(torch.int64)
    got = torch.zeros((*code.shape[:-1], 2 * code.shape[-1]), dtype=torch.float64, device=pages.device)
    for half in (0, 1):
        c = (code >> 4 * half) & 15
        e, m = ((c >> 1) & 3).double(), (c & 1).double()
        got[..., half::2] = torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2) * (1 - 2 * (c >> 3)).double()
    scale = torch.exp2(blocks.reshape(-1, *blocks.shape[2:])[slots].double() - 127)
    return got.unflatten(-1, (scale.shape[-1], BLOCK)).mul(scale[..., None]).flatten(-2)


def _exact_turn(state, name):
    """Rows normed and rotated in 64 bits: each pair of dims as one complex number."""
    case, x = state["case"], state[name].double()
    weight = state.get(name + "_weight")
    if weight is not None:
        x = x / torch.sqrt((x**2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    rotary, at = case["rotary"], case["offset"]
    if rotary:
        dims = torch.arange(rotary, device=x.device)
        first, second = (dims[0::2], dims[1::2]) if case["interleaved"] else dims.chunk(2)
        angle = state["position"].double()[:, None] * state["freq"].double()
        z = torch.complex(x[..., at + first], x[..., at + second]) * torch.polar(torch.ones_like(angle), angle)[:, None]
        x = x.clone()
        x[..., at + first], x[..., at + second] = z.real, z.imag
    return x


def _exact_append(case, state):
    page, within = torch.div(state["at"].long(), PAGE, rounding_mode="floor"), state["at"].long() % PAGE
    slot = state["table"].flatten().long()[state["seq"].long() * state["table"].shape[1] + page] * PAGE + within
    rows = {"k": _exact_turn(state, "k"), "v": state["v"].double()}
    result = {"q": _exact_turn(state, "q")} if case["heads"] else {}
    if case["cache"] != "fp4":
        for name, x in rows.items():
            pages = state[name + "_pages"].to(torch.float64)
            # what 8 bits hold is compared with the number before its rounding
            pages.view(-1, *pages.shape[2:])[slot] = x / float(state[name + "_scale"])
            result[name + "_pages"] = pages
        return result
    # next to a border between two codes, or two powers of two, the last bit of a rotated key decides: no such value
    result.update(k_values=None, k_scales=None)
    b = rows["v"].unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    power = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)))) - 2
    power = torch.where(top > 0, power, torch.full_like(power, -127.0))
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    a = (b / torch.exp2(power)).abs().clamp(max=6.0)
    # of two neighbours at the same distance the one with the even code
    far = (a[..., None] - grid).abs() + torch.arange(8, device="cuda") % 2 * 1e-12
    near = torch.copysign(grid[far.argmin(-1)], b).flatten(-2)
    whole = _decoded(state["v_pages"])
    whole.view(-1, *whole.shape[2:])[slot] = near
    scales = torch.exp2(state["v_blocks"].double() - 127).clamp(2.0**-9, 256.0)
    scales.view(-1, *scales.shape[2:])[slot] = torch.exp2(power[..., 0]).clamp(2.0**-9, 256.0)
    result.update(v_values=whole, v_scales=scales)
    return result


def _decoded(pages):
    """E2M1 values in 64 bits, unscaled."""
    ones = torch.full((*pages.shape[:-1], pages.shape[-1] * 2 // BLOCK), 127, dtype=torch.uint8, device=pages.device)
    slots = torch.arange(pages.shape[0] * PAGE, device=pages.device)
    got = _wide(pages, ones, slots)
    return got.reshape(*pages.shape[:3], -1)
