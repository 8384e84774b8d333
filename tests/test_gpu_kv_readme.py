"""The README's key-value cache example runs as written and matches the plain form in 64 bits."""
import os
import re

import numpy as np
import pytest
import torch

from kv_ref import Row, evict_keep

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_key_value_cache_example():
    code = re.findall(r"```python\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), re.S)[2]
    before = code.split("mqa.mqa_kv_evict_select(")[0]
    ns = {}
    exec(compile(before, "README.md", "exec"), ns)
    torch.cuda.synchronize()
    first = {n: ns[n].clone() for n in ("out", "k", "v", "acc")}
    exec(compile(code[len(before):], "README.md", "exec"), ns)
    torch.cuda.synchronize()
    n, hkv, d = ns["n_seq"], ns["Hkv"], ns["D"]
    flat = {x: first[x].view(-1, hkv, d).cpu().double() for x in ("k", "v")}
    table, q = ns["table"].cpu().numpy(), ns["q"].cpu()

    def check(got, slots, r):
        s = torch.as_tensor(np.asarray(slots, np.int64))
        row = Row(q[r], flat["k"][s], flat["v"][s], d ** -0.5, torch.bfloat16)
        assert ((got[r].cpu().double() - row.out).abs() <= row.out_tol).all(), r

    for r in range(n):
        pos = np.arange(int(ns["lens"][r]))
        slots = table[r, pos // 64].astype(np.int64) * 64 + pos % 64
        check(first["out"], slots, r)
        check(ns["sel"], slots[:ns["K"]], r)
        want = evict_keep(first["acc"][r].cpu().numpy(), len(pos), ns["budget"], ns["recent"])
        m = int(ns["kept"][r])
        assert m == len(want) and np.array_equal(ns["keep"][r, :m].cpu().numpy(), want)
        check(ns["out"], slots[want], r)
