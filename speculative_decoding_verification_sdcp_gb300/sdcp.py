"""Thin Python binding of libsdcp (C ABI in include/sdcp.h): argument marshalling only.

Every step of the acceptance step runs in the library's CUDA kernels; this module turns
torch tensors into pointers, sizes and the current CUDA stream, and raises on a non-zero
return code.  There is no fallback: if libsdcp.so is missing, importing this module fails.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsdcp.so")

SDCP_F32, SDCP_BF16 = 0, 1
SDCP_RULE_GREEDY, SDCP_RULE_SPECULATIVE_SAMPLING = 1, 2
S_OK, S_BAD_PROPOSAL, S_LIMIT, S_BAD_PARAMS, S_Q_UNAVAILABLE, S_INTERNAL = 0, 1, 2, 3, 4, 5
ROW_INVALID, ROW_X_KEPT, ROW_SKIPPED, ROW_FALLBACK = 1, 2, 4, 8
MAX_M = 64
ROWS_TARGET, ROWS_DRAFT = 0, 1
ROTARY_HALF, ROTARY_INTERLEAVED = 0, 1

# sdcp_session_params (32 bytes) and sdcp_row_stat (32 bytes) as numpy records.
PARAMS_DTYPE = np.dtype([("rule_id", "<u4"), ("temperature_milli", "<u4"), ("top_k", "<u4"),
                         ("top_p_milli", "<u4"), ("seed", "<u8"), ("round", "<u4"),
                         ("session_tag", "<u4")])
ROW_STAT_DTYPE = np.dtype([("lmax", "<f4"), ("log_s", "<f4"), ("lp_x", "<f4"), ("argmax", "<i4"),
                           ("kept", "<i4"), ("thr_key", "<u4"), ("thr_n", "<i4"), ("flags", "<u4")])

# random generators of the acceptance step
RNG_PHILOX4X32_10, RNG_HMAC_SHA256 = 0, 1
# actions of a verdict, and the contract's "no self_load"
ACTION_NONE, ACTION_CONTINUE, ACTION_REDUCE, ACTION_SWITCH = -1, 0, 1, 2
ACTION_SELF_DECODE, ACTION_FINISH, ACTION_FAIL = 3, 4, 5
NO_SELF_LOAD = 0xFFFFFFFF
# sdcp_commit_params (48 bytes) and sdcp_session_state (64 bytes)
COMMIT_PARAMS_DTYPE = np.dtype([("max_new", "<u4"), ("stop_offset", "<u4"), ("stop_count", "<u4"),
                                ("m_max", "<u4"), ("low_rounds", "<u4"), ("low_ratio", "<u4"),
                                ("self_load", "<u4"), ("fallback_len", "<u4"), ("fallback", "u1", (8,)),
                                ("m_restore", "<u4"), ("reserved", "<u4")])
STATE_DTYPE = np.dtype([("digest", "u1", (32,)), ("committed", "<u4"), ("c", "<u4"), ("g", "<u4"),
                        ("j", "<u4"), ("m_cap", "<u4"), ("reserved", "<u4", (3,))])
# sdcp_logit_controls (32 bytes)
CONTROLS_DTYPE = np.dtype([("repetition", "<f4"), ("frequency", "<f4"), ("presence", "<f4"),
                           ("history_len", "<u4"), ("prompt_len", "<u4"), ("bias_offset", "<u4"),
                           ("bias_count", "<u4"), ("reserved", "<u4")])
assert COMMIT_PARAMS_DTYPE.itemsize == 48 and STATE_DTYPE.itemsize == 64


class VerifyOptions(ctypes.Structure):
    """sdcp_verify_options."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("rng_id", ctypes.c_uint32),
                ("session_ids", ctypes.c_void_p), ("q_rows", ctypes.c_void_p)]


class KvCacheDesc(ctypes.Structure):
    """sdcp_kv_cache."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("n_pages", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("page_table", ctypes.c_void_p), ("pages", ctypes.c_void_p)]


class RotaryDesc(ctypes.Structure):
    """sdcp_rotary."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("layout", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("n_positions", ctypes.c_int32), ("table", ctypes.c_void_p)]


class KvPoolDesc(ctypes.Structure):
    """sdcp_kv_pool."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("n_pages", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("n_slots", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("page_table", ctypes.c_void_p),
                ("held", ctypes.c_void_p), ("refs", ctypes.c_void_p)]


class SdcpError(RuntimeError):
    pass


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libsdcp.so is not built; run "
                          "`python -m speculative_decoding_verification_sdcp_gb300.build_ext` "
                          "(or __graft_entry__.build())")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    L.sdcp_workspace_bytes.argtypes = [i64, i32, i64]
    L.sdcp_workspace_bytes.restype = sz
    L.sdcp_verify_batch.argtypes = [vp, vp, ctypes.c_int, i64, i32, vp, i64, vp, vp, vp, vp, vp,
                                    vp, vp, sz, vp]
    L.sdcp_verify_batch.restype = ctypes.c_int
    L.sdcp_verify_rows.argtypes = [vp, vp, ctypes.c_int, i64, i32, vp, i64, vp, vp, vp, sz, vp]
    L.sdcp_verify_rows.restype = ctypes.c_int
    L.sdcp_verify_sessions.argtypes = [vp, vp, ctypes.c_int, i64, i32, vp, i64, vp, vp, vp, vp, vp,
                                       vp, vp, sz, vp]
    L.sdcp_verify_sessions.restype = ctypes.c_int
    L.sdcp_verify_batch_noalloc.argtypes = [vp, vp, ctypes.c_int, i64, i32, vp, i64, vp, vp, vp,
                                            vp, vp, vp, vp]
    L.sdcp_verify_batch_noalloc.restype = ctypes.c_int
    L.sdcp_row_stats.argtypes = [vp, vp, ctypes.c_int, i64, i32, vp, i64, vp, vp, vp, vp, sz, vp]
    L.sdcp_row_stats.restype = ctypes.c_int
    L.sdcp_verify_batch_ex.argtypes = [vp, vp, ctypes.c_int, i64, i32, vp, i64, vp, vp, vp, vp, vp,
                                       vp, vp, sz, ctypes.POINTER(VerifyOptions), vp]
    L.sdcp_verify_batch_ex.restype = ctypes.c_int
    L.sdcp_commit_batch.argtypes = [i32, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_uint32, vp, vp]
    L.sdcp_commit_batch.restype = ctypes.c_int
    L.sdcp_split_sessions.argtypes = [vp, vp, i32, i32, vp]
    L.sdcp_split_sessions.restype = ctypes.c_int
    L.sdcp_adjust_logits.argtypes = [vp, vp, ctypes.c_int, i64, i32, ctypes.c_int, vp, i64, vp, vp, vp, i64,
                                     vp, vp, i64, vp, i64, i64, vp, vp, vp]
    L.sdcp_adjust_logits.restype = ctypes.c_int
    L.sdcp_kv_page_bytes.argtypes = [i32, i32, i32]
    L.sdcp_kv_page_bytes.restype = sz
    L.sdcp_append_kv.argtypes = [vp, i32, vp, i64, vp, ctypes.c_int, vp, i64, vp, i64, vp, vp, i64, i32, vp, vp, vp]
    L.sdcp_append_kv.restype = ctypes.c_int
    L.sdcp_read_kv.argtypes = [vp, i32, vp, i64, vp, ctypes.c_int, vp, vp, vp, vp]
    L.sdcp_read_kv.restype = ctypes.c_int
    L.sdcp_fork_kv.argtypes = [vp, vp, vp, vp, vp]
    L.sdcp_fork_kv.restype = ctypes.c_int
    L.sdcp_pool_workspace_bytes.argtypes = [i32, i32]
    L.sdcp_pool_workspace_bytes.restype = sz
    L.sdcp_reserve_kv.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, sz, vp]
    L.sdcp_reserve_kv.restype = ctypes.c_int
    L.sdcp_copy_pages.argtypes = [vp, vp, i32, vp, vp, vp]
    L.sdcp_copy_pages.restype = ctypes.c_int
    L.sdcp_release_kv.argtypes = [vp, vp, vp, vp]
    L.sdcp_release_kv.restype = ctypes.c_int
    L.sdcp_compact_kv.argtypes = [vp, vp, i32, vp, vp, vp, sz, vp]
    L.sdcp_compact_kv.restype = ctypes.c_int
    L.sdcp_attend_workspace_bytes.argtypes = [i32, i64, i32, i32, i32]
    L.sdcp_attend_workspace_bytes.restype = sz
    L.sdcp_attend_kv.argtypes = [vp, i32, vp, i64, vp, vp, i64, i32, ctypes.c_float, i32, vp, vp, vp, sz, vp]
    L.sdcp_attend_kv.restype = ctypes.c_int
    L.sdcp_attend_shared_workspace_bytes.argtypes = [i32, i64, i32, i32, i32, i32]
    L.sdcp_attend_shared_workspace_bytes.restype = sz
    L.sdcp_attend_shared_kv.argtypes = [vp, i32, vp, i64, vp, i32, vp, vp, i64, i32, ctypes.c_float, vp, vp, vp, sz, vp]
    L.sdcp_attend_shared_kv.restype = ctypes.c_int
    L.sdcp_strerror.argtypes = [ctypes.c_int]
    L.sdcp_strerror.restype = ctypes.c_char_p
    L.sdcp_abi_version.argtypes = []
    L.sdcp_abi_version.restype = ctypes.c_int
    return L


lib = _load()


def sdcp_strerror(code: int) -> str:
    return lib.sdcp_strerror(code).decode()


def sdcp_abi_version() -> int:
    return lib.sdcp_abi_version()


def sdcp_workspace_bytes(V: int, B: int, total_drafts: int) -> int:
    return int(lib.sdcp_workspace_bytes(V, B, total_drafts))


def _check(rc: int, what: str):
    if rc != 0:
        raise SdcpError("%s failed: %s (code %d)" % (what, sdcp_strerror(rc), rc))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SDCP_BF16
    if t.dtype == torch.float32:
        return SDCP_F32
    raise TypeError("logits must be torch.float32 or torch.bfloat16, got %s" % t.dtype)


def params_tensor(params: np.ndarray, device) -> torch.Tensor:
    raw = np.ascontiguousarray(params, dtype=PARAMS_DTYPE).view(np.uint8)
    return torch.from_numpy(raw.copy()).to(device)


def alloc_workspace(V: int, B: int, total_drafts: int, device) -> torch.Tensor:
    n = sdcp_workspace_bytes(V, B, total_drafts)
    if n == 0:
        raise SdcpError("invalid sizes for the workspace (V=%d, B=%d, total=%d)" % (V, B, total_drafts))
    # torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(n, dtype=torch.uint8, device=device)


def _stream_handle(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _on(t: torch.Tensor):
    """The library launches on the current CUDA device: make the tensors' device current."""
    return torch.cuda.device(t.device)


def sdcp_verify_batch(target_logits, draft_logits, m_offsets, total_drafts, draft_tokens,
                      params_dev, accepted, n_out, out_tokens, status, workspace,
                      stream=None):
    """Device tensors in, device tensors out; enqueued on ``stream`` (default: current)."""
    V = target_logits.shape[1]
    B = accepted.shape[0]
    s = _stream_handle(target_logits.device) if stream is None else ctypes.c_void_p(stream)
    with _on(target_logits):
        rc = lib.sdcp_verify_batch(_ptr(target_logits), _ptr(draft_logits), dtype_code(target_logits),
                                   V, B, _ptr(m_offsets), int(total_drafts), _ptr(draft_tokens),
                                   _ptr(params_dev), _ptr(accepted), _ptr(n_out), _ptr(out_tokens),
                                   _ptr(status), _ptr(workspace), workspace.numel(), s)
    _check(rc, "sdcp_verify_batch")


def sdcp_verify_batch_ex(target_logits, draft_logits, m_offsets, total_drafts, draft_tokens,
                         params_dev, accepted, n_out, out_tokens, status, workspace,
                         rng_id=RNG_PHILOX4X32_10, session_ids=None, q_rows=None, stream=None):
    """sdcp_verify_batch with the random generator chosen by rng_id (session_ids: a device
    uint8 tensor [B, 16] of session identifiers, for the HMAC-SHA-256 generator), and q from
    the draft logits or from q_rows (a device float32 tensor [total_drafts, V] of the
    drafter's probabilities)."""
    V = target_logits.shape[1]
    B = accepted.shape[0]
    s = _stream_handle(target_logits.device) if stream is None else ctypes.c_void_p(stream)
    if q_rows is not None and q_rows.dtype != torch.float32:
        raise TypeError("q_rows must be torch.float32 probabilities")
    opts = VerifyOptions(ctypes.sizeof(VerifyOptions), int(rng_id),
                         None if session_ids is None else session_ids.data_ptr(),
                         None if q_rows is None else q_rows.data_ptr())
    with _on(target_logits):
        rc = lib.sdcp_verify_batch_ex(_ptr(target_logits), _ptr(draft_logits), dtype_code(target_logits),
                                      V, B, _ptr(m_offsets), int(total_drafts), _ptr(draft_tokens),
                                      _ptr(params_dev), _ptr(accepted), _ptr(n_out), _ptr(out_tokens),
                                      _ptr(status), _ptr(workspace), workspace.numel(),
                                      ctypes.byref(opts), s)
    _check(rc, "sdcp_verify_batch_ex")


def sdcp_commit_batch(m_offsets, accepted, n_out, out_tokens, status, cparams_dev, stop_tokens,
                      state_dev, load_percent, action, stream=None):
    """The commit step after acceptance (truncation, digest chain, control) on device tensors:
    cparams_dev / state_dev are uint8 tensors holding COMMIT_PARAMS_DTYPE / STATE_DTYPE
    records; n_out, out_tokens and state_dev are updated in place."""
    B = accepted.shape[0]
    s = _stream_handle(accepted.device) if stream is None else ctypes.c_void_p(stream)
    with _on(accepted):
        rc = lib.sdcp_commit_batch(B, _ptr(m_offsets), _ptr(accepted), _ptr(n_out), _ptr(out_tokens),
                                   _ptr(status), _ptr(cparams_dev), _ptr(stop_tokens), _ptr(state_dev),
                                   int(load_percent), _ptr(action), s)
    _check(rc, "sdcp_commit_batch")


NOALLOC_SCRATCH_BYTES = 2 << 20


def sdcp_verify_batch_noalloc(target_logits, draft_logits, m_offsets, total_drafts, draft_tokens,
                              params_dev, accepted, n_out, out_tokens, status, stream=None):
    """sdcp_verify_batch without a workspace argument: the library's own scratch array is
    used (for callers that cannot allocate device memory; calls must not overlap)."""
    V = target_logits.shape[1]
    B = accepted.shape[0]
    s = _stream_handle(target_logits.device) if stream is None else ctypes.c_void_p(stream)
    with _on(target_logits):
        rc = lib.sdcp_verify_batch_noalloc(_ptr(target_logits), _ptr(draft_logits),
                                           dtype_code(target_logits), V, B, _ptr(m_offsets),
                                           int(total_drafts), _ptr(draft_tokens), _ptr(params_dev),
                                           _ptr(accepted), _ptr(n_out), _ptr(out_tokens), _ptr(status), s)
    _check(rc, "sdcp_verify_batch_noalloc")


def sdcp_verify_rows(target_logits, draft_logits, m_offsets, total_drafts, draft_tokens,
                     params_dev, workspace, B, stream=None):
    V = target_logits.shape[1]
    s = _stream_handle(target_logits.device) if stream is None else ctypes.c_void_p(stream)
    with _on(target_logits):
        rc = lib.sdcp_verify_rows(_ptr(target_logits), _ptr(draft_logits), dtype_code(target_logits), V,
                                  B, _ptr(m_offsets), int(total_drafts), _ptr(draft_tokens),
                                  _ptr(params_dev), _ptr(workspace), workspace.numel(), s)
    _check(rc, "sdcp_verify_rows")


def sdcp_verify_sessions(target_logits, draft_logits, m_offsets, total_drafts, draft_tokens,
                         params_dev, accepted, n_out, out_tokens, status, workspace, stream=None):
    V = target_logits.shape[1]
    B = accepted.shape[0]
    s = _stream_handle(target_logits.device) if stream is None else ctypes.c_void_p(stream)
    with _on(target_logits):
        rc = lib.sdcp_verify_sessions(_ptr(target_logits), _ptr(draft_logits), dtype_code(target_logits),
                                      V, B, _ptr(m_offsets), int(total_drafts), _ptr(draft_tokens),
                                      _ptr(params_dev), _ptr(accepted), _ptr(n_out), _ptr(out_tokens),
                                      _ptr(status), _ptr(workspace), workspace.numel(), s)
    _check(rc, "sdcp_verify_sessions")


def sdcp_row_stats(target_logits, draft_logits, m_offsets, total_drafts, draft_tokens, params_dev,
                   stats_out, workspace, stream=None):
    V = target_logits.shape[1]
    B = m_offsets.shape[0] - 1
    s = _stream_handle(target_logits.device) if stream is None else ctypes.c_void_p(stream)
    with _on(target_logits):
        rc = lib.sdcp_row_stats(_ptr(target_logits), _ptr(draft_logits), dtype_code(target_logits), V, B,
                                _ptr(m_offsets), int(total_drafts), _ptr(draft_tokens), _ptr(params_dev),
                                _ptr(stats_out), _ptr(workspace), workspace.numel(), s)
    _check(rc, "sdcp_row_stats")


def controls_tensor(controls: np.ndarray, device) -> torch.Tensor:
    raw = np.ascontiguousarray(controls, dtype=CONTROLS_DTYPE).view(np.uint8)
    return torch.from_numpy(raw.copy()).to(device)


def _is(t, dtype, what):
    """The library reads raw memory: a tensor of another type or with gaps is refused here."""
    if t is not None and (t.dtype is not dtype or not t.is_contiguous()):
        raise TypeError("%s must be a contiguous %s tensor" % (what, dtype))
    return t


def _ints(what, a, b, c):
    """_is for the three index tensors of a call, together."""
    if not (a.dtype is b.dtype is c.dtype is torch.int32 and a.is_contiguous() and b.is_contiguous() and c.is_contiguous()):
        raise TypeError("%s must be contiguous torch.int32 tensors" % what)


def _addr(t):
    return None if t is None else t.data_ptr()


# the handle of a device's current stream, without the object around it
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, what, tensors, stream, *args):
    """One call of the library on the device that its tensors (None: not given) are all on: on the
    given stream handle, or the device's current stream.  (A serving step makes several calls of a few
    microseconds, so the device is only switched where it is not the current one.)"""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index or index < 0:  # -1: in host memory
            raise ValueError("%s: all tensors must be on one CUDA device" % what)
    here = torch.cuda.current_device()
    if stream is None:
        stream = _raw_stream(index)
    if index == here:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, stream)
    if rc != 0:
        _check(rc, what)


def sdcp_adjust_logits(logits, out, m_offsets, total_drafts, draft_tokens, controls_dev, history, status,
                       rows=ROWS_TARGET, bias_tokens=None, bias_values=None, masks=None, mask_rows=None,
                       stream=None):
    """Penalties, biases and grammar masks on target or draft rows: logits [rows, V] -> out (which
    may be logits).  controls_dev: CONTROLS_DTYPE records as a uint8 tensor; history: int32
    [B, stride] or None; bias_tokens / bias_values: int32 / float32 [n]; masks: int32 [n_masks,
    words], one bit a token; mask_rows: int32 [rows], -1 = none; status: int32 [B], written."""
    n_logits, V = logits.shape
    B, total = status.shape[0], int(total_drafts)
    code = dtype_code(logits)
    n_rows = total + (B if rows == ROWS_TARGET else 0)
    if out is not logits and (out.dtype is not logits.dtype or out.shape != logits.shape or not out.is_contiguous()) or not logits.is_contiguous():
        raise TypeError("logits and out must be contiguous tensors of one shape and type")
    _ints("m_offsets, status and mask_rows", m_offsets, status, status if mask_rows is None else mask_rows)
    if n_logits < n_rows or (mask_rows is not None and mask_rows.numel() < n_rows):
        raise ValueError("the batch has %d rows" % n_rows)
    if controls_dev.dtype is not torch.uint8 or not controls_dev.is_contiguous():
        raise TypeError("controls_dev must be a contiguous torch.uint8 tensor")
    if m_offsets.numel() < B + 1 or controls_dev.numel() < B * 32:
        raise ValueError("m_offsets and controls must cover the %d sessions" % B)
    if draft_tokens is not None and _is(draft_tokens, torch.int32, "draft_tokens").numel() < total:
        raise ValueError("draft_tokens must hold the %d drafts" % total)
    stride = n_bias = n_masks = words = 0
    if history is not None:
        if _is(history, torch.int32, "history").shape[0] < B:
            raise ValueError("history must have a row for each of the %d sessions" % B)
        stride = history.shape[1]
    if bias_tokens is not None:
        n_bias = _is(bias_tokens, torch.int32, "bias_tokens").numel()
        if bias_values is None or _is(bias_values, torch.float32, "bias_values").numel() != n_bias:
            raise ValueError("bias_tokens and bias_values must have the same length")
    if masks is not None:
        n_masks, words = _is(masks, torch.int32, "masks").shape
    _call(lib.sdcp_adjust_logits, "sdcp_adjust_logits",
          (logits, out, m_offsets, draft_tokens, controls_dev, history, status, bias_tokens, bias_values, masks, mask_rows), stream,
          logits.data_ptr(), out.data_ptr(), code, V, B, int(rows),
          m_offsets.data_ptr(), total, _addr(draft_tokens), controls_dev.data_ptr(), _addr(history), stride, _addr(bias_tokens),
          _addr(bias_values), n_bias, _addr(masks), words, n_masks, _addr(mask_rows), status.data_ptr())


_DESC_SIZE = ctypes.sizeof(KvCacheDesc)


class KvCache:
    """The pages of a 4-bit cache of keys and values (sdcp_kv_cache): a uint8 tensor [n_pages,
    kv_heads, 2, bytes], allocated here or given."""

    def __init__(self, n_pages: int, page_tokens: int, kv_heads: int, head_dim: int, device, pages=None):
        n = int(lib.sdcp_kv_page_bytes(page_tokens, kv_heads, head_dim))
        if n == 0 or n_pages < 1:
            raise SdcpError("unsupported cache geometry (%d pages of %d tokens, %d heads of %d)"
                            % (n_pages, page_tokens, kv_heads, head_dim))
        shape = (n_pages, kv_heads, 2, n // (2 * kv_heads))
        if pages is None:
            pages = torch.zeros(shape, dtype=torch.uint8, device=device)
        if tuple(pages.shape) != shape:
            raise ValueError("pages must have the shape %s" % (shape,))
        self.pages = _is(pages, torch.uint8, "pages")
        self.n_pages, self.page_tokens, self.kv_heads, self.head_dim = n_pages, page_tokens, kv_heads, head_dim

    def desc(self, page_table, B):
        """The description of the cache with a batch's page table (int32 [B, max_pages])."""
        n, most = _is(page_table, torch.int32, "page_table").shape
        if n < B:
            raise ValueError("page_table must have a row for each of the %d sessions" % B)
        return KvCacheDesc(_DESC_SIZE, self.n_pages, self.page_tokens, self.kv_heads, self.head_dim, most, page_table.data_ptr(), self.pages.data_ptr())


class Rotary:
    """A rotation table (sdcp_rotary): float32 [n_positions, rot_dim], rot_dim / 2 cosines and then
    as many sines of each position."""

    def __init__(self, table: torch.Tensor, layout: int = ROTARY_HALF):
        self.table = _is(table, torch.float32, "table")
        self.desc = RotaryDesc(ctypes.sizeof(RotaryDesc), int(layout), table.shape[1], table.shape[0], table.data_ptr())


def _heads(t, rows, heads, dim, what):
    """Row stride of a [rows, heads, dim] view whose rows may lie apart."""
    if t.dim() != 3 or t.shape[0] < rows or t.shape[1:] != (heads, dim) or t.stride(2) != 1 or (heads > 1 and t.stride(1) != dim):
        raise ValueError("%s must be [%d, %d, %d] with contiguous rows" % (what, rows, heads, dim))
    return t.stride(0) if t.shape[0] > 1 else heads * dim


def sdcp_append_kv(cache, page_table, m_offsets, total_drafts, kv_len, k, v, status, rotary=None, q=None,
                   q_out=None, stream=None):
    """Appends a round's keys and values, k and v [total_drafts + B, kv_heads, head_dim], at
    kv_len[b] .. of each session, turned by their positions; q [.., q_heads, head_dim] is turned
    into q_out.  The rows of k, v and q may be views of a fused projection's output."""
    B = status.shape[0]
    rows = int(total_drafts) + B
    code = dtype_code(k)
    if v.dtype != k.dtype or (q is not None and (q.dtype != k.dtype or q_out is None or q_out.dtype != k.dtype)):
        raise TypeError("q, k, v and q_out must have one type")
    ks, vs = _heads(k, rows, cache.kv_heads, cache.head_dim, "k"), _heads(v, rows, cache.kv_heads, cache.head_dim, "v")
    n_q = 0 if q is None else q.shape[1]
    qs = 0 if q is None else _heads(q, rows, n_q, cache.head_dim, "q")
    if q is not None and (not q_out.is_contiguous() or q_out.shape[0] < rows or q_out.shape[1:] != q.shape[1:]):
        raise ValueError("q_out must be contiguous and have q's shape")
    _ints("m_offsets, kv_len and status", m_offsets, kv_len, status)
    if m_offsets.numel() < B + 1 or kv_len.numel() < B:
        raise ValueError("m_offsets and kv_len must cover the %d sessions" % B)
    desc = cache.desc(page_table, B)
    _call(lib.sdcp_append_kv, "sdcp_append_kv",
          (k, v, q, q_out, page_table, cache.pages, m_offsets, kv_len, status, None if rotary is None else rotary.table), stream,
          ctypes.byref(desc), B, m_offsets.data_ptr(), int(total_drafts),
          kv_len.data_ptr(), code, k.data_ptr(), ks, v.data_ptr(), vs, None if rotary is None else ctypes.byref(rotary.desc),
          _addr(q), qs, n_q, _addr(q_out), status.data_ptr())


def sdcp_read_kv(cache, page_table, offsets, n_tokens, start, k_out, v_out, status, stream=None):
    """Cached tokens as values: tokens start[b] .. of session b into rows offsets[b] ..
    offsets[b+1] - 1 of k_out and v_out [n_tokens, kv_heads, head_dim] (either may be None)."""
    B = status.shape[0]
    some = k_out if k_out is not None else v_out
    if some is None:
        raise TypeError("k_out or v_out must be given")
    code, heads = dtype_code(some), (cache.kv_heads, cache.head_dim)
    for t in (k_out, v_out):
        if t is not None:
            if t.dtype is not some.dtype:
                raise TypeError("k_out and v_out must have one type")
            if not t.is_contiguous() or t.shape[0] < n_tokens or t.shape[1:] != heads:
                raise ValueError("outputs must be contiguous [n_tokens, kv_heads, head_dim] tensors")
    _ints("offsets, start and status", offsets, start, status)
    if offsets.numel() < B + 1 or start.numel() < B:
        raise ValueError("offsets and start must cover the %d sessions" % B)
    desc = cache.desc(page_table, B)
    _call(lib.sdcp_read_kv, "sdcp_read_kv", (status, page_table, cache.pages, offsets, start, k_out, v_out), stream,
          ctypes.byref(desc), B, offsets.data_ptr(), int(n_tokens),
          start.data_ptr(), code, _addr(k_out), _addr(v_out), status.data_ptr())


class KvPool:
    """Who holds which page of a cache (sdcp_kv_pool): page_table int32 [n_slots, max_pages], held int32
    [n_slots] and refs int32 [n_pages], allocated empty here or given.  One pool serves the caches of all
    layers; a batch's page table is made of rows of page_table."""

    def __init__(self, n_pages: int, page_tokens: int, n_slots=None, max_pages=None, device=None, page_table=None, held=None, refs=None):
        if page_table is None:
            page_table = torch.full((n_slots, max_pages), -1, dtype=torch.int32, device=device)
        if held is None:
            held = torch.zeros(page_table.shape[0], dtype=torch.int32, device=page_table.device)
        if refs is None:
            refs = torch.zeros(n_pages, dtype=torch.int32, device=page_table.device)
        for t, what in ((page_table, "page_table"), (held, "held"), (refs, "refs")):
            _is(t, torch.int32, what)
        if page_table.dim() != 2 or held.shape != page_table.shape[:1] or refs.shape != (n_pages,):
            raise ValueError("page_table must be [n_slots, max_pages], held [n_slots] and refs [n_pages]")
        if not page_table.get_device() == held.get_device() == refs.get_device():
            raise ValueError("page_table, held and refs must be on one device")
        self.page_table, self.held, self.refs = page_table, held, refs
        self.n_pages, self.page_tokens = n_pages, page_tokens
        self.n_slots, self.max_pages = page_table.shape
        self.desc = KvPoolDesc(ctypes.sizeof(KvPoolDesc), n_pages, page_tokens, self.n_slots, self.max_pages, page_table.data_ptr(),
                               held.data_ptr(), refs.data_ptr())
        self._at = ctypes.byref(self.desc)

    def _slots(self, what, *arrays):
        """The arrays of one entry a slot among a call's arguments."""
        for t in arrays:
            if t.dtype is not torch.int32 or not t.is_contiguous():
                raise TypeError("%s must be contiguous torch.int32 tensors" % what)
            if t.numel() != self.n_slots:
                raise ValueError("%s must have an entry for each of the %d slots" % (what, self.n_slots))


def _copy_list(copies, n_copies):
    if copies.dtype is not torch.int32 or n_copies.dtype is not torch.int32 or not copies.is_contiguous() or not n_copies.is_contiguous():
        raise TypeError("copies and n_copies must be contiguous torch.int32 tensors")
    if copies.dim() != 2 or copies.shape[1] != 4 or n_copies.numel() < 1:
        raise ValueError("copies must be [max_copies, 4] and n_copies [1]")
    return copies.shape[0]


def alloc_pool_workspace(pool) -> torch.Tensor:
    return torch.empty(int(lib.sdcp_pool_workspace_bytes(pool.n_pages, pool.n_slots)), dtype=torch.uint8, device=pool.refs.device)


def sdcp_fork_kv(pool, parent, length, status, stream=None):
    """Slot b with parent[b] >= 0 (-1: none) takes the pages of its parent's first length[b] tokens, shared
    with it; parent, length and status (written): int32 [n_slots]."""
    pool._slots("parent, length and status", parent, length, status)
    _call(lib.sdcp_fork_kv, "sdcp_fork_kv", (status, parent, length, pool.refs), stream,
          pool._at, parent.data_ptr(), length.data_ptr(), status.data_ptr())


def sdcp_reserve_kv(pool, kv_len, upto, copies, n_copies, status, workspace, stream=None):
    """Pages for positions kv_len[b] .. upto[b] - 1 of each slot, shared ones that lie there replaced.
    copies int32 [max_copies >= n_slots, 4] and n_copies int32 [1] receive the copies to make
    (sdcp_copy_pages); kv_len, upto and status (written): int32 [n_slots]."""
    pool._slots("kv_len, upto and status", kv_len, upto, status)
    most = _copy_list(copies, n_copies)
    _call(lib.sdcp_reserve_kv, "sdcp_reserve_kv",
          (status, kv_len, upto, copies, n_copies, workspace, pool.refs), stream,
          pool._at, kv_len.data_ptr(), upto.data_ptr(), copies.data_ptr(), most, n_copies.data_ptr(), status.data_ptr(),
          workspace.data_ptr(), workspace.numel())


def sdcp_copy_pages(cache, copies, n_copies, status, stream=None):
    """The first n_copies[0] records of copies int32 [max_copies, 4] (from, to, tokens, reserved), on one
    cache; status int32 [1], written."""
    most = _copy_list(copies, n_copies)
    if _is(status, torch.int32, "status").numel() < 1:
        raise ValueError("status must be [1]")
    desc = KvCacheDesc(_DESC_SIZE, cache.n_pages, cache.page_tokens, cache.kv_heads, cache.head_dim, 0, None, cache.pages.data_ptr())
    _call(lib.sdcp_copy_pages, "sdcp_copy_pages", (status, copies, n_copies, cache.pages), stream,
          ctypes.byref(desc), copies.data_ptr(), most, n_copies.data_ptr(), status.data_ptr())


def sdcp_release_kv(pool, keep, status, stream=None):
    """Each slot keeps the pages of its first keep[b] tokens (negative: all) and gives the others back;
    keep and status (written): int32 [n_slots]."""
    pool._slots("keep and status", keep, status)
    _call(lib.sdcp_release_kv, "sdcp_release_kv", (status, keep, pool.refs), stream,
          pool._at, keep.data_ptr(), status.data_ptr())


def sdcp_compact_kv(pool, copies, n_copies, n_live, workspace, stream=None):
    """Live pages to the front of the pool: rows and counts are changed, copies int32 [max_copies, 4] and
    n_copies int32 [1] receive the moves for sdcp_copy_pages, n_live int32 [1] the number of live pages."""
    most = _copy_list(copies, n_copies)
    if _is(n_live, torch.int32, "n_live").numel() < 1:
        raise ValueError("n_live must be [1]")
    _call(lib.sdcp_compact_kv, "sdcp_compact_kv", (n_live, copies, n_copies, workspace, pool.refs), stream,
          pool._at, copies.data_ptr(), most, n_copies.data_ptr(), n_live.data_ptr(), workspace.data_ptr(), workspace.numel())


def sdcp_attend_workspace_bytes(B: int, total_drafts: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib.sdcp_attend_workspace_bytes(B, total_drafts, q_heads, kv_heads, head_dim))


def alloc_attend_workspace(B: int, total_drafts: int, q_heads: int, kv_heads: int, head_dim: int, device) -> torch.Tensor:
    n = sdcp_attend_workspace_bytes(B, total_drafts, q_heads, kv_heads, head_dim)
    if n == 0:
        raise SdcpError("invalid sizes for the workspace (B=%d, total=%d, heads %d / %d of %d)"
                        % (B, total_drafts, q_heads, kv_heads, head_dim))
    return torch.empty(n, dtype=torch.uint8, device=device)


def sdcp_attend_kv(cache, page_table, m_offsets, total_drafts, kv_len, q, out, status, workspace, scale=None,
                   window=0, stream=None):
    """Attention of a round's rows, q [total_drafts + B, q_heads, head_dim] bfloat16 (rows may lie
    apart), over the cache: row i of session b sees positions up to kv_len[b] + i (the last
    `window` of them; 0: all).  scale defaults to 1 / sqrt(head_dim)."""
    B = status.shape[0]
    rows = int(total_drafts) + B
    if q.dtype != torch.bfloat16 or out.dtype != torch.bfloat16:
        raise TypeError("q and out must be torch.bfloat16")
    qs = _heads(q, rows, q.shape[1], cache.head_dim, "q")
    if not out.is_contiguous() or out.shape[0] < rows or out.shape[1:] != q.shape[1:]:
        raise ValueError("out must be contiguous and have q's shape")
    if window > 0x7FFFFFFF:
        raise ValueError("window must be below 2^31")
    _ints("m_offsets, kv_len and status", m_offsets, kv_len, status)
    if m_offsets.numel() < B + 1 or kv_len.numel() < B:
        raise ValueError("m_offsets and kv_len must cover the %d sessions" % B)
    desc = cache.desc(page_table, B)
    _call(lib.sdcp_attend_kv, "sdcp_attend_kv", (q, out, page_table, cache.pages, m_offsets, kv_len, status, workspace), stream,
          ctypes.byref(desc), B, m_offsets.data_ptr(), int(total_drafts),
          kv_len.data_ptr(), q.data_ptr(), qs, q.shape[1], float(cache.head_dim ** -0.5 if scale is None else scale), int(window),
          out.data_ptr(), status.data_ptr(), workspace.data_ptr(), workspace.numel())


def alloc_attend_shared_workspace(B: int, total_drafts: int, n_groups: int, q_heads: int, kv_heads: int, head_dim: int, device) -> torch.Tensor:
    n = int(lib.sdcp_attend_shared_workspace_bytes(B, total_drafts, n_groups, q_heads, kv_heads, head_dim))
    if n == 0:
        raise SdcpError("invalid sizes for the workspace (B=%d, total=%d, %d groups, heads %d / %d of %d)"
                        % (B, total_drafts, n_groups, q_heads, kv_heads, head_dim))
    return torch.empty(n, dtype=torch.uint8, device=device)


def sdcp_attend_shared_kv(cache, page_table, m_offsets, total_drafts, kv_len, group_offsets, q, out, status, workspace, scale=None,
                          stream=None):
    """sdcp_attend_kv (without a window) for sessions that have their first pages in common: sessions
    group_offsets[g] .. group_offsets[g+1] - 1 (int32 [groups + 1]; None: all) are a group, and the pages on
    which its rows of page_table agree are read once for it."""
    B = status.shape[0]
    rows = int(total_drafts) + B
    if q.dtype != torch.bfloat16 or out.dtype != torch.bfloat16:
        raise TypeError("q and out must be torch.bfloat16")
    qs = _heads(q, rows, q.shape[1], cache.head_dim, "q")
    if not out.is_contiguous() or out.shape[0] < rows or out.shape[1:] != q.shape[1:]:
        raise ValueError("out must be contiguous and have q's shape")
    _ints("m_offsets, kv_len and status", m_offsets, kv_len, status)
    if m_offsets.numel() < B + 1 or kv_len.numel() < B:
        raise ValueError("m_offsets and kv_len must cover the %d sessions" % B)
    groups = 0 if group_offsets is None else _is(group_offsets, torch.int32, "group_offsets").numel() - 1
    if groups < (group_offsets is not None):
        raise ValueError("group_offsets must be [groups + 1]")
    desc = cache.desc(page_table, B)
    _call(lib.sdcp_attend_shared_kv, "sdcp_attend_shared_kv",
          (q, out, page_table, cache.pages, m_offsets, kv_len, status, group_offsets, workspace), stream,
          ctypes.byref(desc), B, m_offsets.data_ptr(), int(total_drafts), kv_len.data_ptr(), groups, _addr(group_offsets), q.data_ptr(), qs,
          q.shape[1], float(cache.head_dim ** -0.5 if scale is None else scale), out.data_ptr(), status.data_ptr(), workspace.data_ptr(),
          workspace.numel())


def sdcp_split_sessions(m_offsets: np.ndarray, params: np.ndarray | None, n_parts: int) -> np.ndarray:
    """Contiguous session blocks for n_parts GPUs (host arrays in, [n_parts+1] bounds out)."""
    off = np.ascontiguousarray(m_offsets, dtype=np.int32)
    B = off.shape[0] - 1
    prm = None if params is None else np.ascontiguousarray(params, dtype=PARAMS_DTYPE)
    bounds = np.zeros(n_parts + 1, dtype=np.int32)
    rc = lib.sdcp_split_sessions(off.ctypes.data_as(ctypes.c_void_p),
                                 None if prm is None else prm.ctypes.data_as(ctypes.c_void_p),
                                 B, int(n_parts), bounds.ctypes.data_as(ctypes.c_void_p))
    _check(rc, "sdcp_split_sessions")
    return bounds


class Verifier:
    """Owns the output and workspace buffers of one batch shape on one device."""

    def __init__(self, V: int, B: int, total_drafts: int, device):
        self.V, self.B, self.total = V, B, int(total_drafts)
        self.device = torch.device(device)
        self.accepted = torch.empty(B, dtype=torch.int32, device=self.device)
        self.n_out = torch.empty(B, dtype=torch.int32, device=self.device)
        self.out_tokens = torch.empty(self.total + B, dtype=torch.int32, device=self.device)
        self.status = torch.empty(B, dtype=torch.int32, device=self.device)
        self.workspace = alloc_workspace(V, B, self.total, self.device)

    def __call__(self, target, draft, m_offsets, draft_tokens, params_dev, stream=None,
                 rng_id=RNG_PHILOX4X32_10, session_ids=None, q_rows=None):
        if rng_id == RNG_PHILOX4X32_10 and session_ids is None and q_rows is None:
            sdcp_verify_batch(target, draft, m_offsets, self.total, draft_tokens, params_dev,
                              self.accepted, self.n_out, self.out_tokens, self.status,
                              self.workspace, stream)
        else:
            sdcp_verify_batch_ex(target, draft, m_offsets, self.total, draft_tokens, params_dev,
                                 self.accepted, self.n_out, self.out_tokens, self.status,
                                 self.workspace, rng_id, session_ids, q_rows, stream)
        return self.accepted, self.n_out, self.out_tokens, self.status

    def phases(self, target, draft, m_offsets, draft_tokens, params_dev, ev_mid=None):
        """Phase 1 then phase 2 (identical to __call__), optionally recording ev_mid between."""
        sdcp_verify_rows(target, draft, m_offsets, self.total, draft_tokens, params_dev,
                         self.workspace, self.B)
        if ev_mid is not None:
            ev_mid.record()
        sdcp_verify_sessions(target, draft, m_offsets, self.total, draft_tokens, params_dev,
                             self.accepted, self.n_out, self.out_tokens, self.status,
                             self.workspace)
        return self.accepted, self.n_out, self.out_tokens, self.status

    def row_stats(self, target, draft, m_offsets, draft_tokens, params_dev):
        out = torch.empty((2 * self.total + self.B) * 32, dtype=torch.uint8, device=self.device)
        sdcp_row_stats(target, draft, m_offsets, self.total, draft_tokens, params_dev, out,
                       self.workspace)
        return out
