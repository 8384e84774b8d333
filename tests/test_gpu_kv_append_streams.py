"""Norm, rotation and appending run on the stream that they are given, or on the current one, in order with what it holds
already, on the GPU."""
import numpy as np
import pytest
import torch

import fp4_mqa_scoring_amd as mqa
from kv_new_ref import assert_rounded, turned
from test_gpu_kv_append import Pool, freqs, fused, i32, weights

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("cache", ["bf16", "e4m3", "fp4"])
def test_rows_that_the_stream_has_still_to_write(cache, given):
    """Two appends on streams of their own, each behind a product that takes a while and the copy that brings its rows."""
    T, H, Hkv, D = 300, 8, 2, 128
    scales = dict(k_scale=0.03, v_scale=0.0625) if cache == "e4m3" else {}
    wide = torch.randn(4096, 4096, device=DEV)
    made = []
    for i in range(2):
        p = Pool([T, 90], Hkv, D, cache, seed=100 + i)
        (host,), (x,) = fused(T, [H + 2 * Hkv], D, torch.bfloat16, 110 + i, pitch=0)
        wq, wk = weights(D, torch.bfloat16, 120 + i)
        at = np.random.RandomState(i).permutation(T)
        made.append(dict(p=p, host=host, src=x.clone(), x=torch.zeros_like(x), wq=wq, wk=wk, at=at, stream=torch.cuda.Stream(),
                         args=(*p.tensors(), p.table.to(DEV), i32(np.zeros(T)), i32(at)), q_out=torch.zeros(T, H, D, dtype=torch.bfloat16, device=DEV),
                         dev=dict(inv_freq=freqs(D).to(DEV), k_weight=wk.to(DEV), q_weight=wq.to(DEV)), ready=torch.empty_like(wide)))
    call = mqa.mqa_kv_append_fp4 if cache == "fp4" else mqa.mqa_kv_append
    torch.cuda.synchronize()
    for m in made:
        q, k, v = m["x"].split([H, Hkv, Hkv], dim=1)
        more = dict(m["dev"], q=q, q_out=m["q_out"], **scales)
        with torch.cuda.stream(m["stream"]):
            for _ in range(4):
                torch.matmul(wide, wide, out=m["ready"])
            m["x"].copy_(m["src"])
            if not given:
                call(k, v, *m["args"], **more)
        if given:
            call(k, v, *m["args"], stream=m["stream"], **more)
    torch.cuda.synchronize()
    for m in made:
        position = torch.from_numpy(m["at"].astype(np.int32))
        hq, hk, hv = m["host"].split([H, Hkv, Hkv], dim=1)
        assert_rounded(m["q_out"].cpu(), *turned(hq, m["wq"], position=position, freq=freqs(D)))
        m["p"].check([(r, 0, int(n)) for r, n in enumerate(m["at"])], turned(hk, m["wk"], position=position, freq=freqs(D)), hv, **scales)
