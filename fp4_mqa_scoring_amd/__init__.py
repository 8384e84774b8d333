"""MI355X-native FP4 paged-MQA prefill indexer fused with exact TopK.

Thin Python binding of the C ABI in ``include/mqa_fp4_topk.h``: every entry
point below marshals torch tensors (device memory, streams) into pointers and
sizes and calls the HIP library ``libmqa_fp4.so``; all arithmetic runs in the
library's kernels. The library is built in-tree by ``build.build()``; calling
an entry point without it raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

from . import synth  # noqa: F401  (seeded input generator)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmqa_fp4.so")

MQA_OK = 0
ERRORS = {
    -1: "MQA_ERR_UNSUPPORTED_K", -2: "MQA_ERR_NULL_POINTER", -3: "MQA_ERR_MISALIGNED",
    -4: "MQA_ERR_BAD_SIZE", -5: "MQA_ERR_DEVICE", -6: "MQA_ERR_CAPTURING", -7: "MQA_ERR_HIP",
    -8: "MQA_ERR_BAD_FLAGS", -9: "MQA_ERR_UNSUPPORTED", -10: "MQA_ERR_OVERLAP",
}
ROW_BAD_WINDOW, ROW_BAD_PAGE, ROW_UNDERFILL, ROW_SELECTOR = -1, -2, -3, -4
STATUS_BAD_WINDOW, STATUS_BAD_PAGE, STATUS_UNDERFILL, STATUS_SELECTOR = 1, 2, 4, 8
FLAG_SPLITS_MASK = 0xFF
FLAG_NO_PREFILTER = 0x100
FLAG_FORCE_UNDERFILL = 0x200
FLAG_NO_FALLBACK = 0x400
STATIC_SCRATCH_BYTES = 64 << 20          # MQA_STATIC_SCRATCH_BYTES
KV_MAX_ARRAYS = 8                        # MQA_KV_MAX_ARRAYS


class MQAError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__(f"{what}: {ERRORS.get(code, code)} ({_error_string(code)})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded HIP library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        try:  # share torch's HIP runtime (same SONAME) so torch streams and memory are valid here
            import torch  # noqa: F401
        except ImportError:
            pass
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"HIP library {LIB_PATH} is not built; run "
                               "`python -m fp4_mqa_scoring_amd.build` (or __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        P, i64, i32, u32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32
        prefill = [P, P, i64, P, P, i64, P, P, i64, P, P, i32, P, P, P]
        L.mqa_fp4_topk_prefill.argtypes = prefill + [P]
        L.mqa_fp4_topk_prefill_ex.argtypes = prefill + [P, u32, P]
        L.mqa_fp4_topk_prefill_static.argtypes = prefill + [P, u32, P]
        L.mqa_fp4_dense_topk_prefill.argtypes = [P, P, i64, P, P, i64, P, P, i64, P, P, i32, P, P, P, P, P, P]
        L.mqa_fp4_dense_logits.argtypes = [P, P, i64, P, P, i64, P, P, i64, P, P, P, P]
        L.mqa_fp4_logits_topk.argtypes = [P, i64, P, i64, i64, P, P, i32, P, P, P, P, P]
        L.mqa_fp4_supported_k.argtypes = [P, i32, P]
        L.mqa_fp4_topk_scratch_bytes.argtypes = [i64, i32, i32]
        L.mqa_fp4_topk_scratch_bytes.restype = i64
        L.mqa_fp4_status.argtypes = [P, P]
        L.mqa_fp4_error_string.argtypes = [i32]
        L.mqa_fp4_error_string.restype = ctypes.c_char_p
        L.mqa_fp4_abi_version.argtypes = []
        L.mqa_fp4_set_stage_events.argtypes = [P, i32]
        L.mqa_fp4_quantize.argtypes = [P, i64, P, P, P]
        L.mqa_fp4_tiled_topk_prefill.argtypes = prefill[:11] + [i32, i32, P, P, P, P, P]
        L.mqa_fp4_tiled_scratch_bytes.argtypes = [i64, i32, i32]
        L.mqa_fp4_tiled_scratch_bytes.restype = i64
        L.mqa_fp4_topk_decode.argtypes = [P, P, i64, P, P, i64, P, P, i64, i64, P, P, P, i32, P, P, P, P, P, i64,
                                          i32, u32, P]
        L.mqa_fp4_decode_workspace_bytes.argtypes = [i64, i32, i32, i32]
        L.mqa_fp4_decode_workspace_bytes.restype = i64
        L.mqa_fp4_cache_write.argtypes = [P, i64, P, P, i64, i64, P, P, P]
        L.mqa_kv_attention_decode.argtypes = [P, P, P, i64, i64, P, P, P, P, P, P, i64, P]
        L.mqa_kv_attention_decode_workspace_bytes.argtypes = [i64, i32, i32, i32]
        L.mqa_kv_attention_selected.argtypes = [P, P, P, P, i64, P, P, P, i64, P]
        L.mqa_kv_attention_selected_workspace_bytes.argtypes = [i64, i64, i32, i32, i32]
        L.mqa_kv_weights_accumulate.argtypes = [P, P, P, P, i64, i64, P, P, P, P, i64, P]
        L.mqa_kv_evict_select.argtypes = [P, i64, P, i64, i64, i64, i64, P, P, P, P, i64, P]
        L.mqa_kv_evict_workspace_bytes.argtypes = [i64, i64]
        L.mqa_kv_compact.argtypes = [P, P, i64, i64, P, i64, i64, P, i64, i64, P, i32, P]
        for name in ("mqa_kv_attention_decode_workspace_bytes", "mqa_kv_attention_selected_workspace_bytes",
                     "mqa_kv_evict_workspace_bytes"):
            getattr(L, name).restype = i64
        for name in ("mqa_kv_attention_decode", "mqa_kv_attention_selected", "mqa_kv_weights_accumulate",
                     "mqa_kv_evict_select", "mqa_kv_compact"):
            getattr(L, name).restype = i32
        for name in ("mqa_fp4_topk_prefill", "mqa_fp4_topk_prefill_ex", "mqa_fp4_topk_prefill_static",
                     "mqa_fp4_dense_topk_prefill",
                     "mqa_fp4_dense_logits", "mqa_fp4_logits_topk", "mqa_fp4_supported_k",
                     "mqa_fp4_status", "mqa_fp4_abi_version", "mqa_fp4_set_stage_events",
                     "mqa_fp4_quantize", "mqa_fp4_cache_write",
                     "mqa_fp4_tiled_topk_prefill", "mqa_fp4_topk_decode"):
            getattr(L, name).restype = i32
        _lib = L
    return _lib


def _error_string(code: int) -> str:
    try:
        return lib().mqa_fp4_error_string(int(code)).decode()
    except Exception:  # library missing
        return ""


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(t, name, dtype, ndim=None):
    import torch
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")


def _check_inputs(q, q_scale, k_pages, k_scale, weights, page_table, row_start, row_end):
    import torch
    _check(q, "q", torch.uint8, 3)
    _check(q_scale, "q_scale", torch.uint8, 3)
    _check(k_pages, "k_pages", torch.uint8, 3)
    _check(k_scale, "k_scale", torch.uint8, 3)
    _check(weights, "weights", torch.float32, 2)
    _check(page_table, "page_table", torch.int32, 1)
    _check(row_start, "row_start", torch.int32, 1)
    _check(row_end, "row_end", torch.int32, 1)
    Q = q.shape[0]
    if tuple(q.shape[1:]) != (64, 64) or tuple(q_scale.shape) != (Q, 64, 4):
        raise ValueError("q must be [Q,64,64] and q_scale [Q,64,4]")
    if tuple(k_pages.shape[1:]) != (64, 64) or tuple(k_scale.shape) != (k_pages.shape[0], 64, 4):
        raise ValueError("k_pages must be [P,64,64] and k_scale [P,64,4]")
    if tuple(weights.shape) != (Q, 64) or row_start.shape[0] != Q or row_end.shape[0] != Q:
        raise ValueError("weights must be [Q,64]; row_start/row_end [Q]")
    return Q, k_pages.shape[0], page_table.shape[0]


def _check_outputs(Q, K, out_raw, out_slot, out_count, out_score):
    import torch
    _check(out_raw, "out_raw", torch.int32, 2)
    _check(out_slot, "out_slot", torch.int32, 2)
    _check(out_count, "out_count", torch.int32, 1)
    _check(out_score, "out_score", torch.float32, 2)
    for t, n in ((out_raw, "out_raw"), (out_slot, "out_slot"), (out_score, "out_score")):
        if t is not None and tuple(t.shape) != (Q, K):
            raise ValueError(f"{n} must be [Q, K] = [{Q}, {K}]")
    if out_count.shape[0] != Q:
        raise ValueError("out_count must be [Q]")


def _rc(code, what):
    if code != MQA_OK:
        raise MQAError(code, what)


def alloc_outputs(Q: int, K: int, device, with_score: bool = False):
    """Output buffers (out_raw, out_slot, out_count[, out_score]) on ``device``."""
    import torch
    out = [torch.empty((Q, K), dtype=torch.int32, device=device),
           torch.empty((Q, K), dtype=torch.int32, device=device),
           torch.empty((Q,), dtype=torch.int32, device=device)]
    if with_score:
        out.append(torch.empty((Q, K), dtype=torch.float32, device=device))
    return tuple(out)


def mqa_fp4_topk_prefill(q, q_scale, k_pages, k_scale, weights, page_table, row_start, row_end, K,
                         out_raw, out_slot, out_count, stream=None):
    """Fused FP4 indexer scoring + exact TopK + page mapping (see the C header)."""
    return mqa_fp4_topk_prefill_ex(q, q_scale, k_pages, k_scale, weights, page_table, row_start,
                                   row_end, K, out_raw, out_slot, out_count, None, 0, stream)


def mqa_fp4_topk_prefill_ex(q, q_scale, k_pages, k_scale, weights, page_table, row_start, row_end, K,
                            out_raw, out_slot, out_count, out_score=None, flags=0, stream=None):
    Q, P_phys, P_log = _check_inputs(q, q_scale, k_pages, k_scale, weights, page_table, row_start, row_end)
    _check_outputs(Q, K, out_raw, out_slot, out_count, out_score)
    rc = lib().mqa_fp4_topk_prefill_ex(
        _ptr(q), _ptr(q_scale), Q, _ptr(k_pages), _ptr(k_scale), P_phys, _ptr(weights),
        _ptr(page_table), P_log, _ptr(row_start), _ptr(row_end), int(K), _ptr(out_raw), _ptr(out_slot),
        _ptr(out_count), _ptr(out_score), int(flags), _stream(stream, q.device))
    _rc(rc, "mqa_fp4_topk_prefill_ex")


def mqa_fp4_topk_prefill_static(q, q_scale, k_pages, k_scale, weights, page_table, row_start, row_end, K,
                                out_raw, out_slot, out_count, out_score=None, flags=0, stream=None):
    """Allocation-free form of mqa_fp4_topk_prefill_ex: scratch from the library's
    fixed per-device array (STATIC_SCRATCH_BYTES), so the batch is limited to
    1,636 rows at K = 1024 and 2,045 at K = 512; calls on one device must be
    ordered (they share the array). Accepts a capturing stream."""
    Q, P_phys, P_log = _check_inputs(q, q_scale, k_pages, k_scale, weights, page_table, row_start, row_end)
    _check_outputs(Q, K, out_raw, out_slot, out_count, out_score)
    rc = lib().mqa_fp4_topk_prefill_static(
        _ptr(q), _ptr(q_scale), Q, _ptr(k_pages), _ptr(k_scale), P_phys, _ptr(weights),
        _ptr(page_table), P_log, _ptr(row_start), _ptr(row_end), int(K), _ptr(out_raw), _ptr(out_slot),
        _ptr(out_count), _ptr(out_score), int(flags), _stream(stream, q.device))
    _rc(rc, "mqa_fp4_topk_prefill_static")


def mqa_fp4_dense_topk_prefill(q, q_scale, k_pages, k_scale, weights, page_table, row_start, row_end, K,
                               logits, out_raw, out_slot, out_count, out_score=None, stream=None):
    """Dense comparator: fp32 logits [Q, S] (caller-owned), then exact TopK."""
    import torch
    Q, P_phys, P_log = _check_inputs(q, q_scale, k_pages, k_scale, weights, page_table, row_start, row_end)
    _check_outputs(Q, K, out_raw, out_slot, out_count, out_score)
    _check(logits, "logits", torch.float32, 2)
    if tuple(logits.shape) != (Q, 64 * P_log):
        raise ValueError("logits must be [Q, 64 * P_log]")
    rc = lib().mqa_fp4_dense_topk_prefill(
        _ptr(q), _ptr(q_scale), Q, _ptr(k_pages), _ptr(k_scale), P_phys, _ptr(weights),
        _ptr(page_table), P_log, _ptr(row_start), _ptr(row_end), int(K), _ptr(logits), _ptr(out_raw),
        _ptr(out_slot), _ptr(out_count), _ptr(out_score), _stream(stream, q.device))
    _rc(rc, "mqa_fp4_dense_topk_prefill")


def mqa_fp4_tiled_topk_prefill(q, q_scale, k_pages, k_scale, weights, page_table, row_start, row_end, K,
                               out_raw, out_slot, out_count, out_score=None, tile_positions=0, stream=None):
    """Bounded context-tiled exact TopK (same contract and outputs as the fused path)."""
    Q, P_phys, P_log = _check_inputs(q, q_scale, k_pages, k_scale, weights, page_table, row_start, row_end)
    _check_outputs(Q, K, out_raw, out_slot, out_count, out_score)
    rc = lib().mqa_fp4_tiled_topk_prefill(
        _ptr(q), _ptr(q_scale), Q, _ptr(k_pages), _ptr(k_scale), P_phys, _ptr(weights),
        _ptr(page_table), P_log, _ptr(row_start), _ptr(row_end), int(K), int(tile_positions), _ptr(out_raw),
        _ptr(out_slot), _ptr(out_count), _ptr(out_score), _stream(stream, q.device))
    _rc(rc, "mqa_fp4_tiled_topk_prefill")


def mqa_fp4_tiled_scratch_bytes(num_rows: int, K: int, tile_positions: int = 0) -> int:
    r = int(lib().mqa_fp4_tiled_scratch_bytes(int(num_rows), int(K), int(tile_positions)))
    if r < 0:
        raise MQAError(r, "mqa_fp4_tiled_scratch_bytes")
    return r


def mqa_fp4_decode_workspace_bytes(num_rows: int, K: int, splits: int = 0, device: int = 0) -> int:
    r = int(lib().mqa_fp4_decode_workspace_bytes(int(num_rows), int(K), int(splits), int(device)))
    if r < 0:
        raise MQAError(r, "mqa_fp4_decode_workspace_bytes")
    return r


def mqa_fp4_topk_decode(q, q_scale, k_pages, k_scale, weights, block_table, seq_of_row, row_start, row_end, K,
                        out_raw, out_slot, out_count, workspace, out_score=None, splits=0, flags=0, stream=None):
    """Decode / multi-sequence form: block_table int32 [n_seq, max_pages], seq_of_row int32 [Q],
    workspace a uint8 device tensor of at least mqa_fp4_decode_workspace_bytes(Q, K, splits) bytes.
    Allocates nothing and does not synchronise (capturable)."""
    import torch
    _check(q, "q", torch.uint8, 3)
    _check(q_scale, "q_scale", torch.uint8, 3)
    _check(k_pages, "k_pages", torch.uint8, 3)
    _check(k_scale, "k_scale", torch.uint8, 3)
    _check(weights, "weights", torch.float32, 2)
    _check(block_table, "block_table", torch.int32, 2)
    for t, n in ((seq_of_row, "seq_of_row"), (row_start, "row_start"), (row_end, "row_end")):
        _check(t, n, torch.int32, 1)
    _check(workspace, "workspace", torch.uint8)
    Q = q.shape[0]
    _check_outputs(Q, K, out_raw, out_slot, out_count, out_score)
    rc = lib().mqa_fp4_topk_decode(
        _ptr(q), _ptr(q_scale), Q, _ptr(k_pages), _ptr(k_scale), k_pages.shape[0], _ptr(weights),
        _ptr(block_table), block_table.shape[0], block_table.shape[1], _ptr(seq_of_row), _ptr(row_start),
        _ptr(row_end), int(K), _ptr(out_raw), _ptr(out_slot), _ptr(out_count), _ptr(out_score), _ptr(workspace),
        workspace.numel(), int(splits), int(flags), _stream(stream, q.device))
    _rc(rc, "mqa_fp4_topk_decode")


def mqa_fp4_dense_logits(q, q_scale, k_pages, k_scale, weights, page_table, row_start, row_end, logits,
                         stream=None):
    import torch
    Q, P_phys, P_log = _check_inputs(q, q_scale, k_pages, k_scale, weights, page_table, row_start, row_end)
    _check(logits, "logits", torch.float32, 2)
    if tuple(logits.shape) != (Q, 64 * P_log):
        raise ValueError("logits must be [Q, 64 * P_log]")
    rc = lib().mqa_fp4_dense_logits(
        _ptr(q), _ptr(q_scale), Q, _ptr(k_pages), _ptr(k_scale), P_phys, _ptr(weights),
        _ptr(page_table), P_log, _ptr(row_start), _ptr(row_end), _ptr(logits), _stream(stream, q.device))
    _rc(rc, "mqa_fp4_dense_logits")


def mqa_fp4_logits_topk(logits, page_table, num_phys_pages, row_start, row_end, K, out_raw, out_slot,
                        out_count, out_score=None, stream=None):
    """Exact TopK over caller-provided fp32 logits [Q, 64 * P_log]."""
    import torch
    _check(logits, "logits", torch.float32, 2)
    _check(page_table, "page_table", torch.int32, 1)
    _check(row_start, "row_start", torch.int32, 1)
    _check(row_end, "row_end", torch.int32, 1)
    Q, P_log = logits.shape[0], page_table.shape[0]
    if logits.shape[1] != 64 * P_log:
        raise ValueError("logits must be [Q, 64 * P_log]")
    _check_outputs(Q, K, out_raw, out_slot, out_count, out_score)
    rc = lib().mqa_fp4_logits_topk(
        _ptr(logits), Q, _ptr(page_table), P_log, int(num_phys_pages), _ptr(row_start), _ptr(row_end),
        int(K), _ptr(out_raw), _ptr(out_slot), _ptr(out_count), _ptr(out_score),
        _stream(stream, logits.device))
    _rc(rc, "mqa_fp4_logits_topk")


def mqa_fp4_supported_k():
    buf = (ctypes.c_int32 * 8)()
    n = ctypes.c_int32(0)
    _rc(lib().mqa_fp4_supported_k(buf, 8, ctypes.byref(n)), "mqa_fp4_supported_k")
    return [int(buf[i]) for i in range(n.value)]


def mqa_fp4_topk_scratch_bytes(num_rows: int, K: int, device: int = 0) -> int:
    r = int(lib().mqa_fp4_topk_scratch_bytes(int(num_rows), int(K), int(device)))
    if r < 0:
        raise MQAError(r, "mqa_fp4_topk_scratch_bytes")
    return r


def mqa_fp4_status(stream=None, device=None) -> int:
    """Synchronises the stream, returns and clears the sticky status bits."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    st = ctypes.c_int32(0)
    _rc(lib().mqa_fp4_status(_stream(stream, dev), ctypes.byref(st)), "mqa_fp4_status")
    return int(st.value)


def mqa_fp4_abi_version() -> int:
    return int(lib().mqa_fp4_abi_version())


def mqa_fp4_quantize(x, codes=None, scales=None, stream=None):
    """MXFP4 quantisation (OCP MX conversion, E2M1 + UE8M0) of float32 x [..., 128]
    into codes uint8 [..., 64] and scales uint8 [..., 4] (allocated if None)."""
    import torch
    _check(x, "x", torch.float32)
    if x.shape[-1] != 128:
        raise ValueError("x must end in 128 elements")
    lead = tuple(x.shape[:-1])
    if codes is None:
        codes = torch.empty(lead + (64,), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(lead + (4,), dtype=torch.uint8, device=x.device)
    _check(codes, "codes", torch.uint8)
    _check(scales, "scales", torch.uint8)
    n = x.numel() // 128
    if codes.numel() != n * 64 or scales.numel() != n * 4:
        raise ValueError("codes / scales do not match x")
    _rc(lib().mqa_fp4_quantize(_ptr(x), n, _ptr(codes), _ptr(scales), _stream(stream, x.device)),
        "mqa_fp4_quantize")
    return codes, scales


def mqa_fp4_cache_write(k, positions, page_table, k_pages, k_scale, stream=None) -> None:
    """Quantise float32 keys k [n, 128] into the paged C4 cache at logical
    positions (int32 [n]) through page_table (int32 [P_log])."""
    import torch
    _check(k, "k", torch.float32)
    _check(positions, "positions", torch.int32)
    _check(page_table, "page_table", torch.int32)
    _check(k_pages, "k_pages", torch.uint8)
    _check(k_scale, "k_scale", torch.uint8)
    n = k.numel() // 128
    if positions.numel() != n:
        raise ValueError("positions must have one entry per key vector")
    _rc(lib().mqa_fp4_cache_write(_ptr(k), n, _ptr(positions), _ptr(page_table), page_table.numel(),
                                  k_pages.shape[0], _ptr(k_pages), _ptr(k_scale), _stream(stream, k.device)),
        "mqa_fp4_cache_write")


def mqa_fp4_set_stage_events(events) -> None:
    """Measurement hook: ``events`` is a ctypes array of 5 hipEvent_t handles
    (or None to turn the hook off); see the C header."""
    if events is None:
        _rc(lib().mqa_fp4_set_stage_events(None, 0), "mqa_fp4_set_stage_events")
    else:
        _rc(lib().mqa_fp4_set_stage_events(ctypes.cast(events, ctypes.c_void_p), len(events)),
            "mqa_fp4_set_stage_events")


# --- key-value cache operators (include/mqa_kv_cache.h) ------------------------------
#
# The decode step of a small batch takes the device about ten microseconds, so these
# calls are kept short on the host: the header's structures are packed as bytes (a
# ctypes structure of this size costs 4 us to fill) and the current stream is read as a handle.

_KV_CACHE = struct.Struct("@PP3q3qqiiiff4x")    # mqa_kv_cache
_KV_QUERY = struct.Struct("@Pqqiif4x")          # mqa_kv_query
_KV_ARRAY = struct.Struct("@PP3q3qqq")          # mqa_kv_array
_kv_const = None


def _kv():
    """(torch, its 16-bit and 8-bit types -> MQA_KV_*, the reader of a device's current stream handle)."""
    global _kv_const
    if _kv_const is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            raw = lambda index: torch.cuda.current_stream(index).cuda_stream  # noqa: E731
        _kv_const = (torch, {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}, raw)
    return _kv_const


def _kv_stream(stream, device):
    if stream is None and device.index is not None:
        return _kv()[2](device.index)
    return _stream(stream, device)


# Devices are checked by the library: every pointer must be memory of the stream's device.

def _kv_check(t, name, dtype, shape):
    """t is a contiguous tensor of this type and shape; its address."""
    try:
        if t.dtype == dtype and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _kv_table(t, name, rows):
    """t is a contiguous int32 table [rows (or any), X]; its address and sizes."""
    try:
        n, width = t.shape
    except (AttributeError, ValueError):
        raise (ValueError if hasattr(t, "shape") else TypeError)(f"{name} must be a tensor of two dimensions") from None
    return _kv_check(t, name, _kv()[0].int32, (n if rows is None else rows, width)), n, width


def _kv_workspace(t):
    """Address and bytes of a workspace (None: none)."""
    if t is None:
        return None, 0
    return _kv_check(t, "workspace", _kv()[0].uint8, getattr(t, "shape", None)), t.numel()


def _f32(x):
    """x as a 32-bit number; beyond their range an infinity, which the library refuses."""
    x = float(x)
    return x if -3.4e38 < x < 3.4e38 else ctypes.c_float(x).value


def _kv_query(q, scale):
    """mqa_kv_query of q, and q's shape."""
    torch, types, _ = _kv()
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    kind, shape = q.dtype, q.shape
    if kind != torch.bfloat16 and kind != torch.float16:
        raise TypeError(f"q must be bfloat16 or float16, got {kind}")
    if len(shape) != 3:
        raise ValueError(f"q must be [Q, H, D], got {list(shape)}")
    Q, H, D = shape
    row, head, element = q.stride()
    if Q > 0 and ((D > 1 and element != 1) or (H > 1 and head != D)):
        raise ValueError("the heads of one row of q must be contiguous")
    return _KV_QUERY.pack(q.data_ptr(), row if Q > 1 else H * D, Q, H, types[kind],
                          (D ** -0.5 if D else 0.0) if scale is None else _f32(scale)), shape


def _kv_cache(q, k_pages, v_pages, k_scale, v_scale):
    """mqa_kv_cache of the pages (v_pages None: keys only) for q."""
    torch, types, _ = _kv()
    if not isinstance(k_pages, torch.Tensor):
        raise TypeError("k_pages must be a torch.Tensor")
    kind, shape = k_pages.dtype, k_pages.shape
    _, H, D = q.shape
    if kind != q.dtype and kind != torch.float8_e4m3fn:
        raise TypeError(f"k_pages must be {q.dtype} or float8_e4m3fn, got {kind}")
    if len(shape) != 4 or shape[1] != 64 or shape[3] != D:
        raise ValueError(f"k_pages must be [P, 64, Hkv, {D}], got {list(shape)}")
    P, _, heads, _ = shape
    if heads < 1 or H % heads:
        raise ValueError(f"k_pages: {H} query heads over {heads} key heads")
    page, pos, head, element = k_pages.stride()
    if element != 1 and k_pages.numel():
        raise ValueError("k_pages: the elements of one head must be contiguous")
    v = (0, 0, 0)
    v_ptr = 0
    if v_pages is not None:
        if not isinstance(v_pages, torch.Tensor):
            raise TypeError("v_pages must be a torch.Tensor")
        if v_pages.dtype != kind or v_pages.shape != shape:
            raise ValueError("k_pages and v_pages must have one shape and type")
        *v, element = v_pages.stride()
        if element != 1 and v_pages.numel():
            raise ValueError("v_pages: the elements of one head must be contiguous")
        v_ptr = v_pages.data_ptr()
    return _KV_CACHE.pack(k_pages.data_ptr(), v_ptr, page, pos, head, *v, P, heads, D, types[kind], _f32(k_scale),
                          _f32(v_scale))


def _kv_windows(rows, block_table, seq_of_row, row_start, row_end):
    """Addresses of the table and the windows, with the table's sizes, in the order of the C calls."""
    i32 = _kv()[0].int32
    return (*_kv_table(block_table, "block_table", None), _kv_check(seq_of_row, "seq_of_row", i32, rows),
            _kv_check(row_start, "row_start", i32, rows), _kv_check(row_end, "row_end", i32, rows))


def _kv_outputs(q, shape, out, lse):
    """Addresses of out and lse (None: none)."""
    return (_kv_check(out, "out", q.dtype, shape),
            None if lse is None else _kv_check(lse, "lse", _kv()[0].float32, shape[:2]))


def mqa_kv_attention_decode(q, k_pages, v_pages, block_table, seq_of_row, row_start, row_end, out, workspace,
                            lse=None, scale=None, k_scale=1.0, v_scale=1.0, stream=None):
    """Attention of new tokens over a paged key-value cache: q [Q, H, D] (bfloat16 or float16; the row
    stride is free), k_pages and v_pages [P, 64, Hkv, D] of q's type or float8_e4m3fn (page, position and
    head strides are free), windows and block table as in mqa_fp4_topk_decode, out [Q, H, D] (a contiguous q
    itself, or apart from it), lse float32 [Q, H] or None, scale 1/sqrt(D) if None, workspace uint8 of at least
    mqa_kv_attention_decode_workspace_bytes(Q, H, Hkv, D) bytes. Allocates nothing on the device and does
    not synchronise (capturable)."""
    query, shape = _kv_query(q, scale)
    rc = lib().mqa_kv_attention_decode(
        query, _kv_cache(q, k_pages, v_pages, k_scale, v_scale),
        *_kv_windows(shape[:1], block_table, seq_of_row, row_start, row_end), *_kv_outputs(q, shape, out, lse),
        *_kv_workspace(workspace), _kv_stream(stream, q.device))
    _rc(rc, "mqa_kv_attention_decode")


def mqa_kv_attention_decode_workspace_bytes(num_rows: int, num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    r = int(lib().mqa_kv_attention_decode_workspace_bytes(int(num_rows), int(num_heads), int(num_kv_heads),
                                                          int(head_dim)))
    if r < 0:
        raise MQAError(r, "mqa_kv_attention_decode_workspace_bytes")
    return r


def mqa_kv_attention_selected(q, k_pages, v_pages, slots, count, out, workspace=None, lse=None, scale=None,
                              k_scale=1.0, v_scale=1.0, stream=None):
    """Attention over a list of cache slots per row (the indexer's out_slot and out_count): slots int32
    [Q, K], count int32 [Q]; the other arguments as in mqa_kv_attention_decode, workspace of at least
    mqa_kv_attention_selected_workspace_bytes(Q, K, H, Hkv, D) bytes (None where that is 0). Capturable."""
    query, shape = _kv_query(q, scale)
    cache = _kv_cache(q, k_pages, v_pages, k_scale, v_scale)
    lists, _, K = _kv_table(slots, "slots", shape[0])
    rc = lib().mqa_kv_attention_selected(
        query, cache, lists, _kv_check(count, "count", _kv()[0].int32, shape[:1]), K, *_kv_outputs(q, shape, out, lse),
        *_kv_workspace(workspace), _kv_stream(stream, q.device))
    _rc(rc, "mqa_kv_attention_selected")


def mqa_kv_attention_selected_workspace_bytes(num_rows: int, K: int, num_heads: int, num_kv_heads: int,
                                              head_dim: int) -> int:
    r = int(lib().mqa_kv_attention_selected_workspace_bytes(int(num_rows), int(K), int(num_heads),
                                                            int(num_kv_heads), int(head_dim)))
    if r < 0:
        raise MQAError(r, "mqa_kv_attention_selected_workspace_bytes")
    return r


def mqa_kv_weights_accumulate(q, lse, k_pages, block_table, seq_of_row, row_start, row_end, acc, scale=None,
                              k_scale=1.0, stream=None):
    """Adds every position's attention weight, summed over its sequence's rows and heads, to acc float32
    [n_seq, at least 64 * max_pages] (logical positions; the row stride is free); lse float32 [Q, H] as the
    attention returned it for the same rows. Capturable."""
    query, shape = _kv_query(q, scale)
    cache = _kv_cache(q, k_pages, None, k_scale, 1.0)
    windows = _kv_windows(shape[:1], block_table, seq_of_row, row_start, row_end)
    stride = _kv_sums(acc, "acc", windows[1], 64 * windows[2])
    rc = lib().mqa_kv_weights_accumulate(
        query, _kv_check(lse, "lse", _kv()[0].float32, shape[:2]), cache, *windows, acc.data_ptr(), stride,
        _kv_stream(stream, q.device))
    _rc(rc, "mqa_kv_weights_accumulate")


def _kv_sums(acc, name, n_seq, positions):
    """Checks accumulated weights [n_seq, >= positions] and returns their row stride."""
    torch = _kv()[0]
    if not isinstance(acc, torch.Tensor) or acc.dtype != torch.float32:
        raise TypeError(f"{name} must be a float32 tensor")
    if acc.dim() != 2 or acc.shape[0] != n_seq or acc.shape[1] < positions:
        raise ValueError(f"{name} must be [{n_seq}, at least {positions}], got {list(acc.shape)}")
    if acc.shape[1] > 1 and acc.stride(1) != 1:
        raise ValueError(f"the positions of one sequence must be contiguous in {name}")
    stride = acc.stride(0) if n_seq > 1 else acc.shape[1]
    if stride < acc.shape[1]:
        raise ValueError(f"the rows of {name} overlap")
    return stride


def mqa_kv_evict_select(acc, seq_len, budget, recent, keep, kept, workspace=None, kept_acc=None, stream=None):
    """Chooses what a budget keeps of every sequence: its last `recent` positions and the budget - recent
    earlier ones with the largest acc (float32 [n_seq, max_len]; seq_len int32 [n_seq]). Fills keep int32
    [n_seq, budget] (rising, padded with -1), kept int32 [n_seq] and, if given, kept_acc float32 [n_seq,
    budget], the sums to go on with: the first ones of the next acc. kept may be seq_len itself, nothing else
    may overlap. workspace: at least mqa_kv_evict_workspace_bytes(n_seq, max_len) bytes. Capturable."""
    torch = _kv()[0]
    if not isinstance(seq_len, torch.Tensor) or seq_len.dim() != 1:
        raise TypeError("seq_len must be a tensor of one dimension")
    n = seq_len.shape[0]
    stride = _kv_sums(acc, "acc", n, 0)
    shape = (n, int(budget))
    rc = lib().mqa_kv_evict_select(
        acc.data_ptr(), stride, _kv_check(seq_len, "seq_len", torch.int32, (n,)), n, acc.shape[1], shape[1], int(recent),
        _kv_check(keep, "keep", torch.int32, shape), _kv_check(kept, "kept", torch.int32, (n,)),
        None if kept_acc is None else _kv_check(kept_acc, "kept_acc", torch.float32, shape),
        *_kv_workspace(workspace), _kv_stream(stream, acc.device))
    _rc(rc, "mqa_kv_evict_select")


def mqa_kv_evict_workspace_bytes(num_seqs: int, max_len: int) -> int:
    r = int(lib().mqa_kv_evict_workspace_bytes(int(num_seqs), int(max_len)))
    if r < 0:
        raise MQAError(r, "mqa_kv_evict_workspace_bytes")
    return r


def _kv_array(src, dst, n):
    """mqa_kv_array of one pair of paged tensors."""
    torch = _kv()[0]
    if not isinstance(src, torch.Tensor) or not isinstance(dst, torch.Tensor):
        raise TypeError(f"array {n} must be a pair of tensors")
    shape, size = src.shape, src.element_size()
    if not 2 <= len(shape) <= 4 or shape[1] != 64:
        raise ValueError(f"array {n} must be [P, 64], [P, 64, X] or [P, 64, Y, X], got {list(shape)}")
    if src.dtype != dst.dtype or shape[1:] != dst.shape[1:]:
        raise ValueError(f"array {n}: source and destination differ in type or shape")
    rows, width = (shape[2], shape[3]) if len(shape) == 4 else (1, shape[2] if len(shape) == 3 else 1)
    if rows < 1 or width < 1:
        raise ValueError(f"array {n} has no elements per position")
    strides = []
    for t in (src, dst):
        stride = t.stride()
        if width > 1 and stride[-1] != 1 and t.numel():
            raise ValueError(f"array {n}: the last dimension must be contiguous")
        strides += [stride[0] * size, stride[1] * size, stride[2] * size if rows > 1 else width * size]
    return _KV_ARRAY.pack(src.data_ptr(), dst.data_ptr(), *strides, width * size, rows)


def mqa_kv_compact(keep, kept, src_table, dst_table, arrays, stream=None):
    """Moves the kept positions (keep int32 [n_seq, budget], kept int32 [n_seq]) of paged arrays from
    src_table's pages to the first positions of dst_table's. arrays: up to KV_MAX_ARRAYS pairs (source,
    destination) of tensors [P, 64], [P, 64, X] or [P, 64, Y, X] (keys, values, the indexer's codes and
    scales, ...), whole 4-byte words per position; source and destination may be one pool, with
    destination pages that the call does not read. One table serves all arrays, so a page counts as
    inside the pools where every array has it (STATUS_BAD_PAGE otherwise). Capturable."""
    i32 = _kv()[0].int32
    keep_at, n, budget = _kv_table(keep, "keep", None)
    arrays = list(arrays)
    if len(arrays) > KV_MAX_ARRAYS:
        raise ValueError(f"at most {KV_MAX_ARRAYS} arrays, got {len(arrays)}")
    made = b"".join([_kv_array(src, dst, i) for i, (src, dst) in enumerate(arrays)])
    src_at, _, src_pages = _kv_table(src_table, "src_table", n)
    dst_at, _, dst_pages = _kv_table(dst_table, "dst_table", n)
    rc = lib().mqa_kv_compact(
        keep_at, _kv_check(kept, "kept", i32, (n,)), n, budget, src_at, src_pages,
        min([src.shape[0] for src, _ in arrays], default=0), dst_at, dst_pages,
        min([dst.shape[0] for _, dst in arrays], default=0), made, len(arrays), _kv_stream(stream, keep.device))
    _rc(rc, "mqa_kv_compact")
