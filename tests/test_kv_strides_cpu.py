"""Strides of dimensions of one page, head or piece are never taken, and any value of them passes the
host's checks (a call then ends because its tensors are host memory)."""
import pytest
import torch

import fp4_mqa_scoring_amd as mqa

NO_DEVICE = (-5, -7)
BF16 = torch.bfloat16


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def code(call, *args, **kw):
    with pytest.raises(mqa.MQAError) as e:
        call(*args, stream=0, **kw)
    return e.value.code


def attention(k, v):
    q, out = torch.zeros(2, 4, k.shape[3], dtype=BF16), torch.zeros(2, 4, k.shape[3], dtype=BF16)
    ws = torch.zeros(1 << 27, dtype=torch.uint8)
    ws = ws[-ws.data_ptr() % 256:]
    kw = dict(seq_of_row=i32(2), row_start=i32(2), row_end=i32(2))
    table = i32(1, 3)
    return [code(mqa.mqa_kv_attention_decode, q, k, v, table, out=out, workspace=ws, **kw),
            code(mqa.mqa_kv_attention_selected, q, k, v, i32(2, 70), i32(2), out, ws),
            code(mqa.mqa_kv_weights_accumulate, q, torch.zeros(2, 4), k, table, acc=torch.zeros(1, 192), **kw)]


def test_one_key_head_or_page():
    one_head = torch.zeros(3, 64, 128, 1, dtype=BF16).transpose(2, 3)
    assert one_head.stride(2) == 1
    two = torch.zeros(2, 64 * 256 + 4, dtype=BF16)[:, :64 * 256].unflatten(1, (64, 2, 128))
    odd = two[:1]
    assert odd.stride(0) % 8
    for pages in (one_head, odd):
        assert set(attention(pages, pages)) <= set(NO_DEVICE)
    assert set(attention(torch.zeros(3, 64, 1, 128, dtype=BF16), one_head)) <= set(NO_DEVICE)
    # a stride that is taken has to be aligned
    assert attention(two, two) == [-3, -3, -3]


def test_arrays_of_one_page_or_piece():
    move = lambda *pair: code(mqa.mqa_kv_compact, i32(1, 5), i32(1), i32(1, 2), i32(1, 1), [pair])
    two = torch.zeros(2, 64 * 8 + 1, dtype=torch.uint8)[:, :512].unflatten(1, (64, 8))
    one_page = two[:1]
    assert one_page.stride(0) % 4
    assert move(one_page, one_page.clone()) in NO_DEVICE and move(one_page.clone(), one_page) in NO_DEVICE
    one_piece = torch.zeros(3, 64, 8, 1, dtype=torch.uint8).transpose(2, 3)
    assert move(one_piece, one_piece.clone()) in NO_DEVICE
    assert move(two, two.clone()) == -3 and move(two.clone(), two) == -3
