"""New heads into the cache and attention over it, together as a server uses them: what each call wrote is what the next
one reads, and every result is compared with the plain forms in 64 bits (tests/kv_ref.py, tests/kv_new_ref.py)."""
import os
import re

import numpy as np
import pytest
import torch

import fp4_mqa_scoring_amd as mqa
from kv_new_ref import assert_fp4, assert_rounded, fp4_numbers, fp4_of, fp4_values, turned
from kv_ref import Row, assert_row
from test_gpu_kv_append import Pool, freqs, fused, i32, raw, weights
from test_gpu_kv_fp4 import Case, check_decode, check_selected, lists, run_decode, run_selected

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


class Server:
    """A cache with its layer's weights; every step appends rows, attends, and checks both against 64 bits."""

    def __init__(self, cache, kind, H, Hkv, D, lengths, R, seed):
        self.cache, self.kind, self.kt, self.H, self.Hkv, self.D = cache, kind, TYPES[kind], H, Hkv, D
        self.pool = Pool(lengths, Hkv, D, cache, seed=seed, spare=3 * len(lengths))
        self.n = len(lengths)
        self.freq, (self.wq, self.wk) = freqs(R, 5e5), weights(D, self.kt, seed)
        self.rows = 0
        self.scales = dict(k_scale=0.05, v_scale=0.04) if cache == "e4m3" else {}

    def append(self, x, seq, at, position, stream=None):
        H, Hkv = self.H, self.Hkv
        q_out = torch.full((x.shape[0], H, self.D), 7.0, dtype=self.kt, device=DEV)
        self.call(x, seq, at, position, q_out, stream)
        return q_out

    def call(self, x, seq, at, position, q_out, stream=None):
        H, Hkv = self.H, self.Hkv
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:H + 2 * Hkv]
        if not hasattr(self, "dev"):
            self.dev = dict(inv_freq=self.freq.to(DEV), k_weight=self.wk.to(DEV), q_weight=self.wq.to(DEV), table=self.pool.table.to(DEV))
        d = self.dev
        call = mqa.mqa_kv_append_fp4 if self.cache == "fp4" else mqa.mqa_kv_append
        call(k, v, *self.pool.tensors(), d["table"], seq, at, rotary_position=position, inv_freq=d["inv_freq"], k_weight=d["k_weight"],
             q=q, q_out=q_out, q_weight=d["q_weight"], stream=stream, **self.scales)

    def attend(self, q, seq, start, end, out, lse, ws, table=None, stream=None):
        table = self.dev["table"] if table is None else table
        if self.cache == "fp4":
            mqa.mqa_kv_attention_decode_fp4(q, *self.pool.tensors(), table, seq, start, end, out, ws, lse=lse, stream=stream)
        else:
            mqa.mqa_kv_attention_decode(q, *self.pool.tensors(), table, seq, start, end, out, ws, lse=lse, stream=stream, **self.scales)

    def workspace(self, rows):
        return torch.empty(mqa.mqa_kv_attention_decode_workspace_bytes(rows, self.H, self.Hkv, self.D), dtype=torch.uint8, device=DEV)

    def numbers(self, slots):
        """Keys and values that the cache holds at these slots."""
        s = torch.as_tensor(np.asarray(slots, np.int64))
        at, out = (s // 64, s % 64), []
        for name in "kv":
            if self.cache == "fp4":
                out.append(fp4_numbers(self.pool.dev[name].cpu()[at], self.pool.dev[name + "_blocks"].cpu()[at]))
            else:
                kind = torch.float8_e4m3fn if self.cache == "e4m3" else self.kt
                out.append(self.pool.dev[name].cpu()[at].view(kind).float().double())
        return out

    def check(self, q, out, lse, seq, start, end, table=None):
        table = self.pool.table if table is None else table
        q, out, lse = q.cpu(), out.cpu(), lse.cpu()
        for r in range(q.shape[0]):
            pos = torch.arange(int(start[r]), int(end[r]))
            k, v = self.numbers(table[int(seq[r])].long()[pos // 64] * 64 + pos % 64)
            ks, vs = self.scales.get("k_scale", 1.0), self.scales.get("v_scale", 1.0)
            ks, vs = float(np.float32(ks)), float(np.float32(vs))
            row = Row(q[r], k, v, self.D ** -0.5 * ks, self.kt)
            # the values' factor is one rounding more, before the output's own
            err = (out[r].double() - row.out * vs).abs()
            assert (err <= row.out_tol * vs * (1 + 2.0 ** -22) + row.out.abs() * vs * 2.0 ** -22).all(), r
            ok = (lse[r].double() - row.lse).abs() <= row.lse_tol + 4 * 2.0 ** -24 * (row.lse.abs() + 1)
            assert (ok | (lse[r].double() == row.lse)).all(), r       # an empty window's is -inf


SERVED = [("fp4", "bf16", 16, 4, 128, 128), ("fp4", "fp16", 12, 2, 64, 32), ("fp4", "bf16", 8, 2, 256, 64),
          ("bf16", "bf16", 8, 2, 128, 128), ("fp16", "fp16", 6, 3, 64, 64), ("e4m3", "bf16", 16, 2, 128, 64)]


@pytest.mark.parametrize("cache,kind,H,Hkv,D,R", SERVED)
def test_prompts_steps_and_an_eviction(cache, kind, H, Hkv, D, R):
    """Ragged prompts in one padded batch, a captured step replayed with other tokens, and after an eviction a token whose
    place in the cache is no longer its position."""
    lens = [130, 1, 64, 77]
    s = Server(cache, kind, H, Hkv, D, [n + 8 for n in lens], R, seed=H + D)
    n = len(lens)
    # prompts, in rows of no order, with padding among them
    where = [(i, p) for i in range(n) for p in range(lens[i])] + [(0, -1)] * 9
    where = [where[i] for i in np.random.RandomState(1).permutation(len(where))]
    T = len(where)
    (host,), (x,) = fused(T, [H + 2 * Hkv], D, s.kt, 21, pitch=2)
    seq, at = (i32(c) for c in zip(*where))
    mqa.mqa_fp4_status()
    q = s.append(x, seq, at, at)
    position = at.cpu()
    turn = dict(position=position, freq=s.freq)
    assert_rounded(q.cpu(), *turned(host[:, :H], s.wq, **turn))
    s.pool.check([(r, *w) for r, w in enumerate(where) if w[1] >= 0], turned(host[:, H:H + Hkv], s.wk, **turn), host[:, H + Hkv:],
                 **{k: float(np.float32(v)) for k, v in s.scales.items()})
    # every token of the prompts attends to what came before it; padding to nothing
    start, end = i32(np.zeros(T)), i32([p + 1 for _, p in where])
    out, lse = torch.full_like(q, 7.0), torch.full((T, H), 7.0, device=DEV)
    s.attend(q, seq, start, end, out, lse, s.workspace(T))
    torch.cuda.synchronize()
    some = [r for r, w in enumerate(where) if w[1] in (0, 31, 63, 64, 76, 129)] + [r for r, w in enumerate(where) if w[1] < 0][:2]
    s.check(q[some], out[some], lse[some], seq[some], start[some], end[some])
    assert (out[[r for r, w in enumerate(where) if w[1] < 0]] == 0).all()
    # one token of each sequence, captured
    step = dict(x=torch.zeros(n, H + 2 * Hkv, D, dtype=s.kt, device=DEV), seq=i32(range(n)), at=i32(np.zeros(n)), end=i32(np.zeros(n)),
                start=i32(np.zeros(n)), q=torch.zeros(n, H, D, dtype=s.kt, device=DEV), out=torch.zeros(n, H, D, dtype=s.kt, device=DEV),
                lse=torch.zeros(n, H, device=DEV), ws=s.workspace(n))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.call(step["x"], step["seq"], step["at"], step["at"], step["q"])
        s.attend(step["q"], step["seq"], step["start"], step["end"], step["out"], step["lse"], step["ws"])
    for t in range(3):
        (host,), (x,) = fused(n, [H + 2 * Hkv], D, s.kt, 30 + t)
        step["x"].copy_(x)
        step["at"].copy_(i32([m + t for m in lens]))
        step["end"].copy_(i32([m + t + 1 for m in lens]))
        graph.replay()
        torch.cuda.synchronize()
        assert_rounded(step["q"].cpu(), *turned(host[:, :H], s.wq, position=step["at"].cpu(), freq=s.freq))
        s.check(step["q"], step["out"], step["lse"], range(n), [0] * n, [m + t + 1 for m in lens])
    # every third position stays, moved to spare pages; the next token goes behind them under its own position
    now = [m + 3 for m in lens]
    keep = [list(range(0, m, 3)) for m in now]
    budget = max(map(len, keep)) + 1
    pages = (budget + 63) // 64
    used = set(s.pool.table.flatten().tolist())
    spare = [p for p in range(s.pool.P) if p not in used][: n * pages]
    table = torch.tensor(spare, dtype=torch.int32).view(n, pages)
    kept = torch.zeros(n, budget, dtype=torch.int32)
    for i, k in enumerate(keep):
        kept[i, :len(k)] = torch.tensor(k)
    parts = [s.pool.dev[m].flatten(2) for m in s.pool.dev]      # a position's bytes as one row: whole words
    before = [s.numbers([int(s.pool.table[i, p // 64]) * 64 + p % 64 for p in k]) for i, k in enumerate(keep)]
    mqa.mqa_kv_compact(kept.to(DEV), i32([len(k) for k in keep]), s.dev["table"], table.to(DEV), [(p, p) for p in parts])
    torch.cuda.synchronize()
    for i, k in enumerate(keep):
        for got, want in zip(s.numbers([int(table[i, p // 64]) * 64 + p % 64 for p in range(len(k))]), before[i]):
            assert torch.equal(got, want)
    s.dev["table"] = table.to(DEV)
    (host,), (x,) = fused(n, [H + 2 * Hkv], D, s.kt, 40)
    position = i32(now)
    q = s.append(x, step["seq"], i32([len(k) for k in keep]), position)
    end = [len(k) + 1 for k in keep]
    s.attend(q, step["seq"], step["start"], i32(end), step["out"], step["lse"], step["ws"])
    torch.cuda.synchronize()
    assert_rounded(q.cpu(), *turned(host[:, :H], s.wq, position=position.cpu(), freq=s.freq))
    s.check(q, step["out"], step["lse"], range(n), [0] * n, end, table)
    assert mqa.mqa_fp4_status() == 0


def test_two_servers_on_two_streams_at_once():
    """Their own caches and workspaces, their calls in turn without a wait between them."""
    made = []
    for i in range(2):
        s = Server("fp4", "bf16", 32, 4, 128, [600 + 50 * i, 90], 128, seed=70 + i)
        T = 400
        (host,), (x,) = fused(T, [40], 128, s.kt, 80 + i)
        where = [(0, p) for p in range(T - 50)] + [(1, p) for p in range(50)]
        seq, at = (i32(c) for c in zip(*where))
        made.append(dict(s=s, host=host, x=x, seq=seq, at=at, end=at + 1, start=torch.zeros_like(at), stream=torch.cuda.Stream(),
                         q=torch.zeros(T, 32, 128, dtype=s.kt, device=DEV), out=torch.zeros(T, 32, 128, dtype=s.kt, device=DEV),
                         lse=torch.zeros(T, 32, device=DEV), ws=s.workspace(T)))
        s.dev = dict(inv_freq=s.freq.to(DEV), k_weight=s.wk.to(DEV), q_weight=s.wq.to(DEV), table=s.pool.table.to(DEV))
    torch.cuda.synchronize()
    for step in range(2):
        for m in made:
            m["s"].call(m["x"], m["seq"], m["at"], m["at"], m["q"], stream=m["stream"])
        for m in made:
            m["s"].attend(m["q"], m["seq"], m["start"], m["end"], m["out"], m["lse"], m["ws"], stream=m["stream"])
    torch.cuda.synchronize()
    for m in made:
        assert_rounded(m["q"].cpu(), *turned(m["host"][:, :32], m["s"].wq, position=m["at"].cpu(), freq=m["s"].freq))
        some = [0, 1, 33, 200, 349, 350, 399]
        m["s"].check(m["q"][some], m["out"][some], m["lse"][some], m["seq"][some], m["start"][some], m["end"][some])


@pytest.mark.parametrize("cache", ["bf16", "fp4"])
def test_a_position_named_twice_holds_one_of_the_rows(cache):
    p = Pool([64], 2, 128, cache, seed=90)
    (hk, hv), (k, v) = fused(300, [2, 2], 128, torch.bfloat16, 91)
    p.append(k, v, np.zeros(300), np.arange(300) % 64)
    torch.cuda.synchronize()
    for name, host in (("k", hk), ("v", hv)):
        got = p.dev[name].cpu()[int(p.table[0, 0])]
        if cache == "fp4":
            value, _ = fp4_of(host)
            held, want = fp4_values(got), value
        else:
            held, want = got.view(torch.int16), raw(host.contiguous())
        for at in range(64):
            rows = want[at::64]
            for h in range(2):      # each 16 bytes of numbers of one row
                for part in range(16):
                    cut = slice(8 * part, 8 * part + 8)
                    assert (rows[:, h, cut] == held[at, h, cut]).all(-1).any(), (name, at, h, part)


def test_heads_that_no_wave_is_filled_by_and_many_rows():
    """One, three and five heads of queries and keys over thousands of rows, several rows to a wave's heads."""
    for T, H, Hk, D in ((4099, 1, 1, 64), (3001, 3, 1, 256), (2500, 5, 3, 128), (5003, 1, 0, 256)):
        (hq, hk), (q, k) = fused(T, [H, Hk], D, torch.float16, T)
        wq, wk = weights(D, torch.float16, T)
        position = torch.from_numpy(np.random.RandomState(T).randint(0, 100_000, T).astype(np.int32))
        q_out, k_out = torch.empty(T, H, D, dtype=torch.float16, device=DEV), torch.empty(T, Hk, D, dtype=torch.float16, device=DEV)
        more = dict(k=k, k_out=k_out, k_weight=wk.to(DEV)) if Hk else {}
        mqa.mqa_kv_norm_rotate(q, q_out, position.to(DEV), inv_freq=freqs(64).to(DEV), q_weight=wq.to(DEV), **more)
        torch.cuda.synchronize()
        for x, got, w in ((hq, q_out, wq), (hk, k_out, wk)):
            if got.numel():
                assert_rounded(got.cpu(), *turned(x, w, position=position, freq=freqs(64)))


def test_rows_far_apart():
    """A row stride of 2 GiB: the third row lies beyond what 32 bits count."""
    T, D, pitch = 3, 64, 2 ** 30 + 8
    whole = torch.zeros((T - 1) * pitch + 2 * D, dtype=torch.bfloat16, device=DEV)
    x = whole.as_strided((T, 2, D), (pitch, D, 1))
    (host,), (src,) = fused(T, [2], D, torch.bfloat16, 95)
    x.copy_(src)
    position = torch.tensor([3, 70_000, 9], dtype=torch.int32)
    mqa.mqa_kv_norm_rotate(x, x, position.to(DEV), inv_freq=freqs(D).to(DEV))
    torch.cuda.synchronize()
    assert_rounded(x.cpu(), *turned(host, position=position, freq=freqs(D)))
    assert int((whole != 0).sum()) == int((x != 0).sum())


@pytest.mark.parametrize("scale", [3e-39, 1e-37, 1e-30, 0.7, 1.0, 1e30, 3e38])
def test_8_bit_scales_of_any_size(scale):
    """The quotient rounds as a division does, wherever the scale lies."""
    scale = float(np.float32(scale))
    g = torch.Generator().manual_seed(97)
    x = (torch.randn(64, 1, 64, generator=g) * 100).float() * scale
    x[0, 0, :8] = torch.tensor([0.0, -0.0, float("inf"), float("-inf"), float("nan"), 448.0 * scale, -464.0 * scale, 3e38])
    x = x.to(torch.bfloat16)
    p = Pool([64], 1, 64, "e4m3", seed=96)
    p.append(x.to(DEV), x.to(DEV), np.zeros(64), np.arange(64), k_scale=scale, v_scale=scale)
    torch.cuda.synchronize()
    quotient = x.double() / scale
    want = quotient.float().clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    nan = torch.isnan(want.float())
    for name in ("k", "v"):
        got = p.dev[name].cpu()[int(p.table[0, 0])].view(torch.float8_e4m3fn)
        assert torch.equal(torch.isnan(got.float()), nan)
        assert torch.equal(raw(got)[~nan], raw(want)[~nan])


def test_norms_of_tiny_rows_without_eps():
    """Sums of squares below the normal range: those have lost bits, but the result stays near the formula's."""
    x = torch.full((4, 1, 64), 2.0 ** -66, dtype=torch.bfloat16)       # squares of 2^-132, their mean too: exact
    x[1] = 2.0 ** -63
    x[2] = 2.0 ** -62.5
    x[3, 0, ::2] = -x[3, 0, ::2]
    w = torch.ones(64, dtype=torch.bfloat16)
    out = torch.empty_like(x, device=DEV)
    mqa.mqa_kv_norm_rotate(x.to(DEV), out, q_weight=w.to(DEV), eps=0.0)
    y, tol = turned(x, w, eps=0.0)
    assert_rounded(out.cpu()[[0, 1, 3]], y[[0, 1, 3]], tol[[0, 1, 3]])
    assert ((out.cpu().double() - y).abs() <= 2.0 ** -7).all()


# --- attention over 4 bits: two key heads at a time ----------------------------------


@pytest.mark.parametrize("H,Hkv,D,kind", [(24, 6, 128, "bf16"), (4, 4, 64, "fp16"), (40, 8, 128, "fp16"), (32, 2, 64, "bf16"), (24, 24, 128, "bf16")])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "pool"])
def test_even_numbers_of_key_heads(H, Hkv, D, kind, layout):
    lengths = [1, 0, 33, 64, 65, 1000, 2049]
    c = Case(lengths, H, Hkv, D, kind, seed=H + D, layout=layout, capacity=50)
    wins = [(s, 0, n) for s, n in enumerate(lengths)] + [(5, 1, 2), (5, 63, 65), (6, 31, 33), (6, 2048, 2049), (6, 95, 1537), (6, 7, 7), (5, 0, 999)]
    seq, start, end = zip(*wins)
    q = c.queries(len(wins))
    out, lse = run_decode(c, q, seq, start, end)
    check_decode(c, q, seq, start, end, out, lse)
    slots, count = lists(c, 6, 700, 3, [700, 0, 1, 33, 64, 699])
    out, lse = run_selected(c, q[:6], slots, count)
    check_selected(c, q[:6], slots, count, out, lse)


def test_more_key_heads_than_shares():
    c = Case([200, 77, 0, 64], 1100, 1100, 64, "bf16", seed=99)
    q = c.queries(4)
    args = (range(4), [0] * 4, c.lengths)
    out, lse = run_decode(c, q, *args)
    check_decode(c, q, *args, out, lse)


@pytest.mark.parametrize("Hkv", [100, 131, 600])
def test_many_key_heads_share_the_workgroups_unevenly(Hkv):
    """50 pairs of 256 workgroups, 131 heads of 512, and one share only."""
    c = Case([2500, 300, 65], Hkv, Hkv, 64, "bf16", seed=Hkv)
    q = c.queries(4)
    args = ([0, 1, 2, 0], [0, 3, 64, 1000], [2500, 300, 65, 2431])
    out, lse = run_decode(c, q, *args)
    check_decode(c, q, *args, out, lse)
    slots, count = lists(c, 4, 130, 5, [130, 1, 0, 77])
    out, lse = run_selected(c, q, slots, count)
    check_selected(c, q, slots, count, out, lse)


@pytest.mark.parametrize("rows", [1, 300])
def test_lists_longer_than_lds_holds(rows):
    """More slots than a workgroup has in LDS at once, 64 heads with queries in LDS and 16 with all in registers."""
    for H, Hkv in ((64, 1), (32, 2)):
        c = Case([4000], H, Hkv, 128, "bf16", seed=3 + H)
        slots, count = lists(c, rows, 2700, 9, [2700, 1025, 2048, 1])
        q = c.queries(rows)
        out, lse = run_selected(c, q, slots, count)
        some = list(range(min(rows, 6)))
        check_selected(c, q[some], slots[some], count[some], out[some], lse[some])


# --- the written example ---------------------------------------------------------------


def test_readme_example_of_a_cache_in_4_bits():
    code = re.findall(r"```python\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), re.S)[3]
    ns = {}
    exec(compile(code, "README.md", "exec"), ns)
    torch.cuda.synchronize()
    H, Hkv, D, K = ns["H"], ns["Hkv"], ns["D"], ns["K"]
    table, lens = ns["table"].cpu().long(), [int(n) for n in ns["lens"]]
    kc, ks, vc, vs = (ns[n].cpu() for n in ("k_codes", "k_scale", "v_codes", "v_scale"))
    x = ns["new"].cpu()
    position = torch.tensor(lens, dtype=torch.int32)
    turn = dict(position=position, freq=ns["inv_freq"].cpu())
    assert_rounded(ns["q"].cpu(), *turned(x[:, :H], ns["q_weight"].cpu(), **turn))
    y, tol = turned(x[:, H:H + Hkv], ns["k_weight"].cpu(), **turn)
    for r in range(ns["n_seq"]):
        pos = torch.arange(lens[r] + 1)
        at = (table[r][pos // 64], pos % 64)
        assert_fp4(kc[at][-1], ks[at][-1], y[r], tol[r], r)
        k, v = fp4_numbers(kc[at], ks[at]), fp4_numbers(vc[at], vs[at])
        q = ns["q"][r].cpu()
        assert_row(ns["out"][r].cpu(), None, Row(q, k, v, D ** -0.5, torch.bfloat16), r)
        chosen = ns["slot"][r].cpu().long()[: int(ns["count"][r])]
        assert len(chosen) == min(K, lens[r] + 1) and len(set(chosen.tolist())) == len(chosen)
        at = (chosen // 64, chosen % 64)
        k, v = fp4_numbers(kc[at], ks[at]), fp4_numbers(vc[at], vs[at])
        assert_row(ns["selected"][r].cpu(), None, Row(q, k, v, D ** -0.5, torch.bfloat16), r)
