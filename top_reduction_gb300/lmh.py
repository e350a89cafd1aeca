"""Thin ctypes binding of liblmh (include/lmh.h).

Argument marshalling only: tensors are passed as device pointers and the
current torch CUDA stream as the launch stream; outputs and the workspace are
allocated with torch (the caching allocator), and every step of the path runs
in the library's CUDA kernels.  There is no fallback: if liblmh.so is missing
or no CUDA device is present, the calls raise.
"""
import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblmh.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE_TOO_SMALL, ERR_CUDA, ERR_TIMEOUT = range(6)
BF16, F16, F32 = 0, 1, 2
W_VH, W_HV = 0, 1
PATH_PROJECT, PATH_FROM_LOGITS, PATH_PROBE = 0, 1, 2
K_MAX = 128
K_FULL = -1  # k_max for the full-vocabulary output: topk_logprobs is [rows, V] in id order

DS_BAD_CU_SEQLENS = 0x1
DS_SEL_OUT_OF_RANGE = 0x2
DS_ROWS_OVERFLOW = 0x4
DS_ROW_IDX_OUT_OF_RANGE = 0x8
DS_TIMEOUT = 0x10
DS_NO_ALLOWED_TOKEN = 0x20
DS_ADAPTER_OUT_OF_RANGE = 0x40
BEAMS_MAX = 128  # beams of a group
ADAPTERS_MAX, ADAPTER_RANK_MAX = 4096, 128


class Sampling(ctypes.Structure):
    """struct lmh_sampling (include/lmh.h)."""
    _fields_ = [("temperature", ctypes.c_void_p), ("allowed_mask", ctypes.c_void_p), ("mask_words", ctypes.c_int32),
                ("seed", ctypes.c_uint64), ("offsets", ctypes.c_void_p), ("sampled_ids", ctypes.c_void_p),
                ("sampled_logprob", ctypes.c_void_p)]


class Filters(ctypes.Structure):
    """struct lmh_filters (include/lmh.h)."""
    _fields_ = [("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p), ("top_p", ctypes.c_void_p),
                ("min_p", ctypes.c_void_p), ("allowed_mask", ctypes.c_void_p), ("mask_words", ctypes.c_int32)]


class Q4TableArg(ctypes.Structure):
    """struct lmh_q4_table (include/lmh.h)."""
    _fields_ = [("packed", ctypes.c_void_p), ("packed_row_bytes", ctypes.c_int64), ("scales", ctypes.c_void_p),
                ("scale_dtype", ctypes.c_int), ("scale_row_stride", ctypes.c_int64), ("zeros", ctypes.c_void_p),
                ("zero_row_stride", ctypes.c_int64), ("V", ctypes.c_int32), ("H", ctypes.c_int32),
                ("group", ctypes.c_int32)]


class AdaptersArg(ctypes.Structure):
    """struct lmh_adapters (include/lmh.h)."""
    _fields_ = [("down", ctypes.c_void_p), ("down_adapter_stride", ctypes.c_int64), ("down_row_stride", ctypes.c_int64),
                ("up", ctypes.c_void_p), ("up_adapter_stride", ctypes.c_int64), ("up_row_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("scales", ctypes.c_void_p), ("ranks", ctypes.c_void_p),
                ("count", ctypes.c_int32), ("rank", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32)]


class BeamsArg(ctypes.Structure):
    """struct lmh_beams (include/lmh.h)."""
    _fields_ = [("groups", ctypes.c_int32), ("beams", ctypes.c_int32), ("k", ctypes.c_int32),
                ("keep_slots", ctypes.c_int32), ("scores", ctypes.c_void_p), ("finished", ctypes.c_void_p),
                ("pad_id", ctypes.c_int32), ("out_scores", ctypes.c_void_p), ("out_parents", ctypes.c_void_p),
                ("out_tokens", ctypes.c_void_p)]


class RowStateArg(ctypes.Structure):
    """struct lmh_row_state (include/lmh.h)."""
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("src_row_bytes", ctypes.c_int64),
                ("dst_row_bytes", ctypes.c_int64), ("src_outer_bytes", ctypes.c_int64 * 2),
                ("dst_outer_bytes", ctypes.c_int64 * 2), ("n0", ctypes.c_int32), ("n1", ctypes.c_int32),
                ("chunk_bytes", ctypes.c_int64), ("position_bytes", ctypes.c_int64)]


EXPORTS = ("lmh_select_rows", "lmh_count_selected_rows", "lmh_workspace_bytes",
           "lmh_project_logprobs", "lmh_project_logprobs_scaled", "lmh_project_logprobs_sample",
           "lmh_probe_selective",
           "lmh_logprobs_from_logits", "lmh_status_string",
           "lmh_version", "lmh_trace_enable", "lmh_trace_read", "lmh_trace_reset", "lmh_debug_set_wait_limit",
           "lmh_record_bytes", "lmh_project_partials", "lmh_merge_workspace_bytes", "lmh_merge_records",
           "lmh_sample_from_logits", "lmh_quantize_q4", "lmh_project_q4", "lmh_lookup_q4",
           "lmh_adapters_workspace_bytes", "lmh_add_adapters", "lmh_beam_workspace_bytes", "lmh_beam_select",
           "lmh_beam_select_lists", "lmh_reorder_rows")

_lib = None


class LMHError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s failed: %s" % (what, status_string(status)))


def load():
    """Load liblmh.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError("liblmh.so is not built (%s); run __graft_entry__.build() or "
                          "python top_reduction_gb300/_build.py" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.lmh_select_rows.argtypes = [P, i32, i32, P, i32, P, P, P, P]
    lib.lmh_select_rows.restype = ctypes.c_int
    lib.lmh_count_selected_rows.argtypes = [P, i32, i32, P]
    lib.lmh_count_selected_rows.restype = i32
    lib.lmh_workspace_bytes.argtypes = [i32, i32, i32, i32, ctypes.c_int]
    lib.lmh_workspace_bytes.restype = u64
    lib.lmh_project_logprobs.argtypes = [P, i64, i32, P, i32, i32, P, ctypes.c_int, i32, P, P, i32,
                                         P, P, P, P, P, P, u64, P, P]
    lib.lmh_project_logprobs.restype = ctypes.c_int
    lib.lmh_project_logprobs_scaled.argtypes = [P, i64, i32, P, i32, i32, P, ctypes.c_int, i32, P, P, i32,
                                                P, P, P, P, P, P, u64, P, ctypes.c_float, P]
    lib.lmh_project_logprobs_scaled.restype = ctypes.c_int
    lib.lmh_project_logprobs_sample.argtypes = [P, i64, i32, P, i32, i32, P, ctypes.c_int, i32, P, P, i32,
                                                P, P, P, P, P, P, u64, P, ctypes.c_float,
                                                ctypes.POINTER(Sampling), P]
    lib.lmh_project_logprobs_sample.restype = ctypes.c_int
    lib.lmh_probe_selective.argtypes = [P, i64, i32, P, i32, i32, P, i32, ctypes.c_float, P, ctypes.c_float, P,
                                        P, u64, P, P]
    lib.lmh_probe_selective.restype = ctypes.c_int
    lib.lmh_logprobs_from_logits.argtypes = [P, ctypes.c_int, i32, i32, i64, P, P, i32, P, P, P, P,
                                             P, u64, P, P]
    lib.lmh_logprobs_from_logits.restype = ctypes.c_int
    lib.lmh_status_string.argtypes = [ctypes.c_int]
    lib.lmh_status_string.restype = ctypes.c_char_p
    lib.lmh_version.restype = i32
    lib.lmh_trace_enable.argtypes = [i32]
    lib.lmh_trace_enable.restype = ctypes.c_int
    lib.lmh_trace_read.argtypes = [ctypes.c_char_p, ctypes.POINTER(i64), ctypes.POINTER(ctypes.c_double)]
    lib.lmh_trace_read.restype = ctypes.c_int
    lib.lmh_trace_reset.restype = None
    lib.lmh_debug_set_wait_limit.argtypes = [ctypes.c_uint64]
    lib.lmh_debug_set_wait_limit.restype = ctypes.c_int
    lib.lmh_record_bytes.argtypes = [i32]
    lib.lmh_record_bytes.restype = u64
    lib.lmh_project_partials.argtypes = [P, i64, i32, P, i32, i32, P, ctypes.c_int, i32, i32, i32, P, P, i32,
                                         P, P, u64, P, P]
    lib.lmh_project_partials.restype = ctypes.c_int
    lib.lmh_merge_workspace_bytes.argtypes = [i32, i32, i32]
    lib.lmh_merge_workspace_bytes.restype = u64
    lib.lmh_merge_records.argtypes = [P, i32, i32, i32, P, P, i32, P, P, P, P, P, u64, P, P]
    lib.lmh_merge_records.restype = ctypes.c_int
    lib.lmh_sample_from_logits.argtypes = [P, ctypes.c_int, i32, i32, i64, ctypes.POINTER(Filters), P, P, P, P, P]
    lib.lmh_sample_from_logits.restype = ctypes.c_int
    T = ctypes.POINTER(Q4TableArg)
    lib.lmh_quantize_q4.argtypes = [P, i64, T, P]
    lib.lmh_quantize_q4.restype = ctypes.c_int
    lib.lmh_project_q4.argtypes = [P, ctypes.c_int, i64, i32, P, i32, T, ctypes.c_float, P, ctypes.c_int, i64, P, P]
    lib.lmh_project_q4.restype = ctypes.c_int
    lib.lmh_lookup_q4.argtypes = [P, i32, T, ctypes.c_float, P, ctypes.c_int, i64, P, P]
    lib.lmh_lookup_q4.restype = ctypes.c_int
    A, B = ctypes.POINTER(AdaptersArg), ctypes.POINTER(BeamsArg)
    lib.lmh_adapters_workspace_bytes.argtypes = [i32, A]
    lib.lmh_adapters_workspace_bytes.restype = u64
    lib.lmh_add_adapters.argtypes = [P, i64, i32, P, i32, P, A, P, i64, P, ctypes.c_int, i64, P, u64, P, P]
    lib.lmh_add_adapters.restype = ctypes.c_int
    lib.lmh_beam_workspace_bytes.argtypes = [i32, i32, i32]
    lib.lmh_beam_workspace_bytes.restype = u64
    lib.lmh_beam_select.argtypes = [B, P, ctypes.c_int, i32, i64, P, i32, P, u64, P, P]
    lib.lmh_beam_select.restype = ctypes.c_int
    lib.lmh_beam_select_lists.argtypes = [B, P, P, i32, P, P]
    lib.lmh_beam_select_lists.restype = ctypes.c_int
    lib.lmh_reorder_rows.argtypes = [ctypes.POINTER(RowStateArg), i32, i32, i32, P, P, P, P]
    lib.lmh_reorder_rows.restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(status):
    return load().lmh_status_string(int(status)).decode()


def _check(status, what):
    if status != OK:
        raise LMHError(status, what)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dev_i32(t, device, n=None, name="array"):
    if t is None:
        return None
    t = torch.as_tensor(t, dtype=torch.int32, device=device).contiguous()
    if n is not None and t.numel() != n:
        raise ValueError("%s must have %d entries" % (name, n))
    return t


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def count_selected_rows(cu_seqlens_host, num_decode, all_rows_mask_host=None):
    """Rows lmh_select_rows will select, from host copies (no device sync)."""
    cu = torch.as_tensor(cu_seqlens_host, dtype=torch.int32).cpu().contiguous()
    mask = None
    if all_rows_mask_host is not None:
        mask = torch.as_tensor(all_rows_mask_host, dtype=torch.uint8).cpu().contiguous()
    n = load().lmh_count_selected_rows(ctypes.c_void_p(cu.data_ptr()), cu.numel() - 1, int(num_decode),
                                       None if mask is None else ctypes.c_void_p(mask.data_ptr()))
    if n < 0:
        raise ValueError("invalid packed batch (cu_seqlens / num_decode)")
    return int(n)


def select_rows(cu_seqlens, num_decode, all_rows_mask=None, max_out_rows=None, dev_status=None,
                stream=None):
    """Device row selection.  Returns (row_idx int32[max_out_rows], logits_cu_seqlens int32[S+1]).

    Pass max_out_rows (e.g. from count_selected_rows on a host copy) to avoid
    the device synchronisation needed to read cu_seqlens[-1].
    """
    cu = cu_seqlens
    assert cu.is_cuda and cu.dtype == torch.int32 and cu.is_contiguous()
    S = cu.numel() - 1
    if max_out_rows is None:
        max_out_rows = int(cu[-1].item()) if cu.numel() else 0
    row_idx = torch.empty(max(int(max_out_rows), 1), dtype=torch.int32, device=cu.device)
    lcu = torch.empty(S + 1, dtype=torch.int32, device=cu.device)
    mask = None
    if all_rows_mask is not None:
        mask = torch.as_tensor(all_rows_mask, dtype=torch.uint8, device=cu.device).contiguous()
    _check(load().lmh_select_rows(_p(cu), S, int(num_decode), _p(mask), int(max_out_rows), _p(row_idx),
                                  _p(lcu), _p(dev_status), _stream(stream)), "lmh_select_rows")
    return row_idx[:max_out_rows], lcu


def workspace_bytes(rows, hidden, vocab, k_max, path):
    n = load().lmh_workspace_bytes(int(rows), int(hidden), int(vocab), int(k_max), int(path))
    if n == 0:
        raise LMHError(ERR_INVALID_ARG, "lmh_workspace_bytes")
    return int(n)


def _outputs(rows, k_max, with_sel, device, V=None):
    out = {"lse": torch.empty(rows, dtype=torch.float32, device=device)}
    out["sel_logprob"] = torch.empty(rows, dtype=torch.float32, device=device) if with_sel else None
    if k_max == K_FULL:  # every id's logprob, in id order; no ids
        out["topk_ids"] = None
        out["topk_logprobs"] = torch.empty((rows, V), dtype=torch.float32, device=device)
        return out
    out["topk_ids"] = torch.empty((rows, k_max), dtype=torch.int32, device=device)
    out["topk_logprobs"] = torch.empty((rows, k_max), dtype=torch.float32, device=device)
    return out


def _workspace(workspace, nbytes, device):
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    assert workspace.numel() * workspace.element_size() >= nbytes
    return workspace


def project_logprobs(hidden, W, row_idx=None, rows=None, sel=None, row_k=None, k_max=0,
                     logits_out=None, workspace=None, dev_status=None, out=None, stream=None, logit_scale=1.0,
                     sampling=None, w_layout=W_VH):
    """Selective head projection + per-row lse / selected logprob / top-k.

    hidden: bf16 [T, H] (rows may be strided); W: bf16 [V, H] (lm_head.weight), or
    [H, V] with w_layout=W_HV (V a multiple of 8);
    row_idx: int32 [rows] device tensor or None (rows 0..rows-1).
    logit_scale: head transform, every logit is logit_scale * (A . W)
    (lmh_project_logprobs_scaled); 1.0 is the plain projection.
    sampling: dict with optional temperature (fp32 [rows]), mask (int32/uint32 [rows, words]
    allowed-token bits), seed (int), offsets (int64 [rows]): device-side Gumbel-max sampling
    (lmh_project_logprobs_sample); adds sampled_ids and sampled_logprob to the result.
    Returns a dict with lse, sel_logprob (or None), topk_ids, topk_logprobs.
    """
    assert hidden.is_cuda and hidden.dtype == torch.bfloat16 and hidden.dim() == 2
    assert hidden.stride(1) == 1
    assert W.is_cuda and W.dtype == torch.bfloat16 and W.dim() == 2 and W.is_contiguous()
    T, H = hidden.shape
    assert w_layout in (W_VH, W_HV)
    V = W.shape[0] if w_layout == W_VH else W.shape[1]
    assert W.shape[1 if w_layout == W_VH else 0] == H
    dev = hidden.device
    if row_idx is not None:
        rows = row_idx.numel() if rows is None else rows
        assert row_idx.dtype == torch.int32 and row_idx.is_cuda
    elif rows is None:
        rows = T
    sel_t = _dev_i32(sel, dev, rows, "sel")
    rk_t = _dev_i32(row_k, dev, rows, "row_k")
    o = out if out is not None else _outputs(rows, k_max, sel_t is not None, dev, V)
    ws = _workspace(workspace, workspace_bytes(rows, H, V, k_max, PATH_PROJECT), dev)
    args = (_p(hidden), hidden.stride(0) if T > 1 else H, T, _p(row_idx), int(rows), H, _p(W), int(w_layout), V,
            _p(sel_t), _p(rk_t), int(k_max), _p(o["lse"]), _p(o["sel_logprob"]), _p(o["topk_ids"]),
            _p(o["topk_logprobs"]), _p(logits_out), _p(ws), ws.numel() * ws.element_size(), _p(dev_status))
    if sampling is not None:
        def dev(t, dtype):
            return None if t is None else torch.as_tensor(t, dtype=dtype, device=dev_).contiguous()
        dev_ = hidden.device
        temp = dev(sampling.get("temperature"), torch.float32)
        mask = sampling.get("mask")
        if mask is not None:
            mask = torch.as_tensor(mask, device=dev_).contiguous()
            assert mask.dim() == 2 and mask.shape[0] == rows and mask.element_size() == 4
        offs = dev(sampling.get("offsets"), torch.int64)
        o["sampled_ids"] = torch.empty(rows, dtype=torch.int32, device=dev_)
        o["sampled_logprob"] = torch.empty(rows, dtype=torch.float32, device=dev_)
        def addr(t):
            return None if t is None else t.data_ptr()
        sp = Sampling(addr(temp), addr(mask), 0 if mask is None else mask.shape[1],
                      int(sampling.get("seed", 0)) & (2 ** 64 - 1), addr(offs), addr(o["sampled_ids"]),
                      addr(o["sampled_logprob"]))
        _check(load().lmh_project_logprobs_sample(*args, float(logit_scale), ctypes.byref(sp), _stream(stream)),
               "lmh_project_logprobs_sample")
    elif logit_scale == 1.0:
        _check(load().lmh_project_logprobs(*args, _stream(stream)), "lmh_project_logprobs")
    else:
        _check(load().lmh_project_logprobs_scaled(*args, float(logit_scale), _stream(stream)),
               "lmh_project_logprobs_scaled")
    return o


def probe_selective(hidden, W, ref_logits, row_idx=None, rows=None, logit_scale=1.0, tolerance=0.0,
                    workspace=None, dev_status=None, stream=None):
    """Mismatching elements between this library's head output for the given rows and the
    model's own logits `ref_logits` (f32 [rows, V]); returns a device uint32 tensor [1]."""
    assert hidden.is_cuda and hidden.dtype == torch.bfloat16 and hidden.dim() == 2 and hidden.stride(1) == 1
    assert W.is_cuda and W.dtype == torch.bfloat16 and W.is_contiguous()
    T, H = hidden.shape
    V = W.shape[0]
    if row_idx is not None:
        rows = row_idx.numel() if rows is None else rows
    elif rows is None:
        rows = T
    assert ref_logits.is_cuda and ref_logits.dtype == torch.float32 and ref_logits.is_contiguous()
    assert tuple(ref_logits.shape) == (rows, V)
    dev = hidden.device
    count = torch.empty(1, dtype=torch.int32, device=dev)
    ws = _workspace(workspace, workspace_bytes(rows, H, V, 0, PATH_PROBE), dev)
    st = load().lmh_probe_selective(
        _p(hidden), hidden.stride(0) if T > 1 else H, T, _p(row_idx), int(rows), H, _p(W), V, float(logit_scale),
        _p(ref_logits), float(tolerance), _p(count), _p(ws), ws.numel() * ws.element_size(), _p(dev_status),
        _stream(stream))
    _check(st, "lmh_probe_selective")
    return count


_DTYPES = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}


def logprobs_from_logits(logits, sel=None, row_k=None, k_max=0, workspace=None, dev_status=None,
                         out=None, stream=None):
    """Per-row lse / selected logprob / top-k of given logits [rows, V] (bf16, f16 or f32)."""
    assert logits.is_cuda and logits.dim() == 2 and logits.stride(1) == 1
    rows, V = logits.shape
    dev = logits.device
    sel_t = _dev_i32(sel, dev, rows, "sel")
    rk_t = _dev_i32(row_k, dev, rows, "row_k")
    o = out if out is not None else _outputs(rows, k_max, sel_t is not None, dev, V)
    ws = _workspace(workspace, workspace_bytes(rows, 0, V, k_max, PATH_FROM_LOGITS), dev)
    stride = logits.stride(0) if rows > 1 else V
    st = load().lmh_logprobs_from_logits(
        _p(logits), _DTYPES[logits.dtype], rows, V, stride, _p(sel_t), _p(rk_t), int(k_max),
        _p(o["lse"]), _p(o["sel_logprob"]), _p(o["topk_ids"]), _p(o["topk_logprobs"]), _p(ws),
        ws.numel() * ws.element_size(), _p(dev_status), _stream(stream))
    _check(st, "lmh_logprobs_from_logits")
    return o


# ---------------------------------------------------------------------------
# a decode step with a 4-bit head: lookup, projection, filtered draw
# ---------------------------------------------------------------------------

# These calls are made once or more per token of a stream, so the host's share is kept small:
# one look-up of the raw stream, no conversions of tensors that are already right.

def _raw_stream(device):
    """The current stream of `device`, as the C ABI takes it."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _other_device(device):
    """True where `device` is not the calling thread's current one: the library launches on that."""
    return device.index != torch._C._cuda_getDevice()


def _on_stream(stream, device):
    """Context of a call on `stream`, which has to be one of the tensors' device."""
    if stream.device != device:
        raise ValueError("stream is of %s, the tensors of %s" % (stream.device, device))
    return torch.cuda.stream(stream)


def _written(t, dtypes, n, device, name):
    """The address of a tensor that the kernels write `n` entries of (it may have more)."""
    if t is None:
        return None
    if t.device != device or t.dtype not in dtypes or not t.is_contiguous() or t.numel() < n:
        raise ValueError("%s must be a contiguous %s tensor on %s with %d entries"
                         % (name, " or ".join(str(d)[6:] for d in dtypes), device, n))
    return t.data_ptr()


_WORDS = (torch.int32, torch.uint32)
_FLOATS = (torch.float32,)


def _status_word(t, device):
    return None if t is None else _written(t, _WORDS, 1, device, "dev_status")


def _per_row(t, dtype, rows, device, name):
    """A per-row parameter as a contiguous device tensor (as it is when it already is one)."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == device and t.is_contiguous()):
        t = torch.as_tensor(t, dtype=dtype, device=device).contiguous()
    if t.numel() != rows:
        raise ValueError("%s must have %d entries" % (name, rows))
    return t


def sample_from_logits(logits, uniforms, temperature=None, top_k=None, top_p=None, min_p=None, mask=None,
                       dev_status=None, out=None, stream=None):
    """One token per row of logits [rows, V] (bf16, f16 or f32; rows may be strided), from one
    given uniform number per row (lmh_sample_from_logits).

    uniforms: fp32 [rows] in [0, 1).  temperature, top_p, min_p: fp32 [rows] or None; top_k: int32
    [rows] or None; mask: int32/uint32 [rows, words] allowed-token bits or None.  stream: the call
    is made on it, conversions and allocations included.
    Returns a dict with sampled_ids (int32 [rows], -1 where a row has no token) and sampled_logprob
    (fp32 [rows], in the distribution that was drawn from).  out: such a dict, filled (contiguous
    tensors on the logits' device; without sampled_logprob, or None there, none is written).
    """
    dev = logits.device
    if stream is not None:
        with _on_stream(stream, dev):
            return sample_from_logits(logits, uniforms, temperature, top_k, top_p, min_p, mask, dev_status, out)
    rows, V = logits.shape
    pitch, step = logits.stride()
    assert logits.is_cuda and (step == 1 or V == 1)
    if _other_device(dev):
        with torch.cuda.device(dev):
            return sample_from_logits(logits, uniforms, temperature, top_k, top_p, min_p, mask, dev_status, out)
    if uniforms is None:
        raise ValueError("uniforms is required")
    u = _per_row(uniforms, torch.float32, rows, dev, "uniforms")
    temp = _per_row(temperature, torch.float32, rows, dev, "temperature")
    k = _per_row(top_k, torch.int32, rows, dev, "top_k")
    p = _per_row(top_p, torch.float32, rows, dev, "top_p")
    m = _per_row(min_p, torch.float32, rows, dev, "min_p")
    words = 0
    if mask is not None:
        mask = torch.as_tensor(mask, device=dev).contiguous()
        if mask.dtype not in _WORDS or mask.dim() != 2 or mask.shape[0] != rows:
            raise ValueError("mask must be int32 or uint32 [%d, words]" % rows)
        words = mask.shape[1]
    if out is None:
        out = {"sampled_ids": torch.empty(rows, dtype=torch.int32, device=dev),
               "sampled_logprob": torch.empty(rows, dtype=torch.float32, device=dev)}
    f = Filters(_ptr(temp), _ptr(k), _ptr(p), _ptr(m), _ptr(mask), words)
    st = (_lib or load()).lmh_sample_from_logits(
        logits.data_ptr(), _DTYPES[logits.dtype], rows, V, pitch if rows > 1 else V, f, u.data_ptr(),
        _written(out["sampled_ids"], _WORDS, rows, dev, "sampled_ids"),
        _written(out.get("sampled_logprob"), _FLOATS, rows, dev, "sampled_logprob"), _status_word(dev_status, dev),
        _raw_stream(dev))
    if st != OK:
        raise LMHError(st, "lmh_sample_from_logits")
    return out


class Q4Table:
    """A [V, H] table in 4 bits with group scales (struct lmh_q4_table).

    packed: uint8 [V, H/2], the even entry of a pair in the low half; scales: bf16, f16 or f32
    [V, H/group]; zeros: uint8 [V, H/group] or None (8).  value = scale * (q - zero).  Rows may
    be strided; the object keeps the tensors alive.
    """

    def __init__(self, packed, scales, zeros=None, group=64):
        assert packed.is_cuda and packed.dtype == torch.uint8 and packed.dim() == 2 and packed.stride(1) == 1
        V, H = packed.shape[0], 2 * packed.shape[1]
        if H % group or tuple(scales.shape) != (V, H // group):
            raise ValueError("scales must be [V, H/group]")
        assert scales.device == packed.device and (scales.stride(1) == 1 or scales.shape[1] == 1)
        if zeros is not None:
            if tuple(zeros.shape) != (V, H // group):
                raise ValueError("zeros must be [V, H/group]")
            assert zeros.dtype == torch.uint8 and zeros.device == packed.device
            assert zeros.stride(1) == 1 or zeros.shape[1] == 1
        self.packed, self.scales, self.zeros, self.group = packed, scales, zeros, group
        self.V, self.H, self.device = V, H, packed.device

        def stride(t, n):
            return t.stride(0) if V > 1 else n
        self._arg = Q4TableArg(packed.data_ptr(), stride(packed, H // 2), scales.data_ptr(), _DTYPES[scales.dtype],
                               stride(scales, H // group), _ptr(zeros),
                               0 if zeros is None else stride(zeros, H // group), V, H, group)


def quantize_q4(W, group=64, zeros=False, scale_dtype=torch.bfloat16, stream=None):
    """Round a bf16 table [V, H] to 4 bits (lmh_quantize_q4): a Q4Table."""
    dev = W.device
    if stream is not None:
        with _on_stream(stream, dev):
            return quantize_q4(W, group, zeros, scale_dtype)
    assert W.is_cuda and W.dtype == torch.bfloat16 and W.dim() == 2 and W.stride(1) == 1
    if _other_device(dev):
        with torch.cuda.device(dev):
            return quantize_q4(W, group, zeros, scale_dtype)
    V, H = W.shape
    if H % group:
        raise ValueError("H must be a multiple of the group")
    packed = torch.empty((V, H // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((V, H // group), dtype=scale_dtype, device=dev)
    z = torch.empty((V, H // group), dtype=torch.uint8, device=dev) if zeros else None
    table = Q4Table(packed, scales, z, group)
    _check(load().lmh_quantize_q4(W.data_ptr(), W.stride(0) if V > 1 else H, table._arg, _raw_stream(dev)),
           "lmh_quantize_q4")
    return table


def project_q4(hidden, table, row_idx=None, rows=None, logit_scale=1.0, out_dtype=torch.float32, out=None,
               dev_status=None, stream=None):
    """Logits [rows, V] of hidden rows through a 4-bit head (lmh_project_q4).

    hidden: bf16 or f16 [T, H] (rows may be strided); row_idx: int32 [rows] device tensor or None;
    out_dtype: float32 or hidden's type, or give `out` (rows may be strided); stream: as
    sample_from_logits.
    """
    dev = hidden.device
    if stream is not None:
        with _on_stream(stream, dev):
            return project_q4(hidden, table, row_idx, rows, logit_scale, out_dtype, out, dev_status)
    T, H = hidden.shape
    V = table.V
    pitch, step = hidden.stride()
    assert step == 1 and dev == table.device
    if _other_device(dev):
        with torch.cuda.device(dev):
            return project_q4(hidden, table, row_idx, rows, logit_scale, out_dtype, out, dev_status)
    if H != table.H:
        raise ValueError("hidden has %d columns, the table %d" % (H, table.H))
    if row_idx is not None:
        assert row_idx.dtype == torch.int32 and row_idx.device == dev and row_idx.is_contiguous()
        rows = row_idx.numel() if rows is None else rows
        assert rows <= row_idx.numel()
    elif rows is None:
        rows = T
    if out is None:
        out = torch.empty((rows, V), dtype=out_dtype, device=dev)
        out_pitch = V
    else:
        assert out.device == dev and out.shape == (rows, V) and (out.stride(1) == 1 or V == 1)
        out_pitch = out.stride(0) if rows > 1 else V
    st = (_lib or load()).lmh_project_q4(
        hidden.data_ptr(), _DTYPES[hidden.dtype], pitch if T > 1 else H, T, _ptr(row_idx), rows, table._arg,
        logit_scale, out.data_ptr(), _DTYPES[out.dtype], out_pitch, _status_word(dev_status, dev), _raw_stream(dev))
    if st != OK:
        raise LMHError(st, "lmh_project_q4")
    return out


def lookup_q4(ids, table, scale=1.0, out_dtype=torch.bfloat16, out=None, dev_status=None, stream=None):
    """The rows [n, H] of int32 device ids from a 4-bit table, times scale (lmh_lookup_q4); an id of
    -1 (no token) gives zeros.  stream: as sample_from_logits."""
    dev = ids.device
    if stream is not None:
        with _on_stream(stream, dev):
            return lookup_q4(ids, table, scale, out_dtype, out, dev_status)
    n, = ids.shape
    H = table.H
    assert dev == table.device and ids.dtype == torch.int32 and ids.is_contiguous()
    if _other_device(dev):
        with torch.cuda.device(dev):
            return lookup_q4(ids, table, scale, out_dtype, out, dev_status)
    if out is None:
        out = torch.empty((n, H), dtype=out_dtype, device=dev)
        out_pitch = H
    else:
        assert out.device == dev and out.shape == (n, H) and out.stride(1) == 1
        out_pitch = out.stride(0) if n > 1 else H
    st = (_lib or load()).lmh_lookup_q4(ids.data_ptr(), n, table._arg, scale, out.data_ptr(), _DTYPES[out.dtype],
                                        out_pitch, _status_word(dev_status, dev), _raw_stream(dev))
    if st != OK:
        raise LMHError(st, "lmh_lookup_q4")
    return out


# ---------------------------------------------------------------------------
# beams and per-request adapters: adapters, selection, states that follow
# ---------------------------------------------------------------------------

class AdapterTable:
    """Low-rank adapters in one array each (struct lmh_adapters): adapter l adds
    scales[l] * up[l] @ (down[l] @ x) to a projection of x.

    down: bf16 or f16 [count, rank, H]; up: the same type [count, N, rank]; scales: fp32 [count] or None
    (1); ranks: int32 [count] or None (rank), the ranks in use: what stands behind them is not used.
    Adapters and rows may be strided; the object keeps the tensors alive.
    """

    def __init__(self, down, up, scales=None, ranks=None):
        assert down.is_cuda and down.device == up.device and down.dim() == 3 and up.dim() == 3
        if down.dtype != up.dtype or down.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("down and up must both be bfloat16 or float16")
        L, R, H = down.shape
        N = up.shape[1]
        if tuple(up.shape) != (L, N, R):
            raise ValueError("down must be [count, rank, H] and up [count, N, rank]")
        if (down.stride(2) != 1 and H > 1) or (up.stride(2) != 1 and R > 1):
            raise ValueError("the last dimension of down and up must be contiguous")
        dev = down.device
        self.scales = _per_row(scales, torch.float32, L, dev, "scales")
        self.ranks = _per_row(ranks, torch.int32, L, dev, "ranks")
        self.down, self.up, self.device, self.dtype = down, up, dev, down.dtype
        self.count, self.rank, self.H, self.N = L, R, H, N

        def strides(t):  # (a dimension of one entry may have any stride)
            row = t.stride(1) if t.shape[1] > 1 else t.shape[2]
            return (t.stride(0) if L > 1 else 0), row
        self._arg = AdaptersArg(down.data_ptr(), *strides(down), up.data_ptr(), *strides(up), _DTYPES[down.dtype],
                                _ptr(self.scales), _ptr(self.ranks), L, R, H, N)
        self._bytes = {}

    def workspace_bytes(self, rows):
        """Bytes of workspace that add_adapters needs for that many rows."""
        n = self._bytes.get(rows)
        if n is None:
            n = int(load().lmh_adapters_workspace_bytes(rows, self._arg))
            if n == 0:
                raise LMHError(ERR_UNSUPPORTED, "lmh_adapters_workspace_bytes")
            self._bytes[rows] = n
        return n


_SCRATCH = threading.local()
_SCRATCH_MOST = 64 << 20


def _scratch(nbytes, device, stream):
    """A workspace for a call on the raw `stream`, kept from call to call (an allocation costs a few microseconds): one
    for each host thread and stream.  A thread's calls on a stream follow one another; two threads' kernels may come
    in turn, one's second product behind the other's first.  While a stream is captured, and for large calls, one of
    its own: a graph may be replayed beside anything."""
    if nbytes > _SCRATCH_MOST or torch._C._cuda_isCurrentStreamCapturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    kept = _SCRATCH.__dict__
    key = device.index, stream
    t = kept.get(key)
    if t is None or t.numel() < nbytes:
        t = kept[key] = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
    return t


def _own_workspace(t, nbytes, device):
    """The address of a caller's workspace."""
    if t.device != device or not t.is_contiguous() or t.numel() * t.element_size() < nbytes:
        raise ValueError("workspace must be contiguous on %s with %d bytes" % (device, nbytes))
    return t.data_ptr()


def _pitch(t, rows, width):
    """The row stride of a [rows, width] tensor whose rows are contiguous."""
    pitch, step = t.stride()
    if step != 1 and width > 1:
        raise ValueError("rows must be contiguous")
    return pitch if rows > 1 else width


def add_adapters(x, table, adapter_idx, y, row_idx=None, out=None, workspace=None, dev_status=None, stream=None):
    """y [rows, N] and each row's adapter of x [T, H]: y[i] + scale * up @ (down @ x[row_idx[i]])
    (lmh_add_adapters).

    table: an AdapterTable; adapter_idx: int32 [rows], -1 for none; row_idx: int32 [rows] device tensor or
    None; y: fp32 or the table's type (rows of x and y may be strided); out: like y, or y itself (in
    place); workspace: table.workspace_bytes(rows) bytes, 256-byte aligned; stream: the call is made on
    it, conversions and allocations included.
    """
    dev = x.device
    if stream is not None:
        with _on_stream(stream, dev):
            return add_adapters(x, table, adapter_idx, y, row_idx, out, workspace, dev_status)
    if _other_device(dev):
        with torch.cuda.device(dev):
            return add_adapters(x, table, adapter_idx, y, row_idx, out, workspace, dev_status)
    rows, N = y.shape
    T, H = x.shape
    if dev != table.device or y.device != dev:
        raise ValueError("x, the table and y must be on one device")
    if H != table.H or N != table.N or x.dtype != table.dtype:
        raise ValueError("x must be %s [T, %d] and y [rows, %d]" % (str(table.dtype)[6:], table.H, table.N))
    idx = _per_row(adapter_idx, torch.int32, rows, dev, "adapter_idx")
    if row_idx is not None and not (row_idx.dtype == torch.int32 and row_idx.device == dev and
                                    row_idx.is_contiguous() and row_idx.numel() >= rows):
        raise ValueError("row_idx must be a contiguous int32 tensor on %s with %d entries" % (dev, rows))
    y_pitch = _pitch(y, rows, N)
    if out is None:
        out = torch.empty((rows, N), dtype=y.dtype, device=dev)
        out_pitch = N
    else:
        if out.device != dev or out.dtype != y.dtype or out.shape != y.shape:
            raise ValueError("out must be like y")
        out_pitch = _pitch(out, rows, N)
    if rows == 0:
        return out
    need = table.workspace_bytes(rows)
    raw = _raw_stream(dev)
    ws = _scratch(need, dev, raw).data_ptr() if workspace is None else _own_workspace(workspace, need, dev)
    st = _lib.lmh_add_adapters(
        x.data_ptr(), _pitch(x, T, H), T, _ptr(row_idx), rows, idx.data_ptr(), table._arg, y.data_ptr(), y_pitch,
        out.data_ptr(), _DTYPES[y.dtype], out_pitch, ws, need, _status_word(dev_status, dev), raw)
    if st != OK:
        raise LMHError(st, "lmh_add_adapters")
    return out


def _beams_arg(scores, beams, k, finished, pad_id, keep_slots, out, rows, dev):
    """(the argument of both selections, their results, tensors to keep until the call is made)"""
    if beams <= 0 or rows % beams:
        raise ValueError("the rows must be whole groups of %d beams" % beams)
    groups = rows // beams
    scores = _per_row(scores, torch.float32, rows, dev, "scores")
    if scores is None:
        raise ValueError("scores is required")
    if finished is not None:
        if isinstance(finished, torch.Tensor) and finished.dtype == torch.bool:
            finished = finished.view(torch.uint8)
        finished = _per_row(finished, torch.uint8, rows, dev, "finished")
    n = groups * k
    if out is None:  # (three allocations: views of one take longer)
        out = {"scores": torch.empty((groups, k), dtype=torch.float32, device=dev),
               "parents": torch.empty((groups, k), dtype=torch.int32, device=dev),
               "tokens": torch.empty((groups, k), dtype=torch.int32, device=dev)}
        to = out["scores"].data_ptr(), out["parents"].data_ptr(), out["tokens"].data_ptr()
    else:
        to = (_written(out["scores"], _FLOATS, n, dev, "scores"), _written(out["parents"], _WORDS, n, dev, "parents"),
              _written(out["tokens"], _WORDS, n, dev, "tokens"))
    arg = BeamsArg(groups, beams, k, 1 if keep_slots else 0, scores.data_ptr(), _ptr(finished), pad_id, *to)
    return arg, out, (scores, finished)


def beam_workspace_bytes(rows, beams, V):
    """Bytes of workspace that beam_select needs for logits [rows, V] of groups of `beams` rows."""
    n = int(load().lmh_beam_workspace_bytes(rows // beams, beams, V)) if beams > 0 else 0
    if n == 0:
        raise LMHError(ERR_UNSUPPORTED, "lmh_beam_workspace_bytes")
    return n


def beam_select(logits, scores, beams, k=None, finished=None, pad_id=0, mask=None, keep_slots=False, workspace=None,
                dev_status=None, out=None, stream=None):
    """The k best continuations (k: beams by default) of every group of `beams` rows, over the beams and
    the vocabulary of logits [rows, V] (bf16, f16 or f32; rows may be strided): scores[b] + log-softmax
    (lmh_beam_select).

    scores: fp32 [rows], the beams' sums of log-probabilities; finished: uint8 or bool [rows] or None,
    ended beams go on as they are with pad_id; mask: int32/uint32 [rows, words] allowed-token bits or
    None; keep_slots: survivors stay in their places (k == beams); workspace: beam_workspace_bytes
    bytes, 256-byte aligned; stream: the call is made on it, conversions and allocations included.
    Returns a dict with scores (fp32), parents (int32, rows of the batch) and tokens (int32), each
    [groups, k]; -inf, -1 and -1 where no continuation is left.  out: such a dict, filled.
    """
    dev = logits.device
    if stream is not None:
        with _on_stream(stream, dev):
            return beam_select(logits, scores, beams, k, finished, pad_id, mask, keep_slots, workspace, dev_status, out)
    if _other_device(dev):
        with torch.cuda.device(dev):
            return beam_select(logits, scores, beams, k, finished, pad_id, mask, keep_slots, workspace, dev_status, out)
    rows, V = logits.shape
    assert logits.is_cuda
    pitch = _pitch(logits, rows, V)
    words = 0
    if mask is not None:
        if not (isinstance(mask, torch.Tensor) and mask.device == dev and mask.is_contiguous()):
            mask = torch.as_tensor(mask, device=dev).contiguous()
        if mask.dtype not in _WORDS or mask.dim() != 2 or mask.shape[0] != rows:
            raise ValueError("mask must be int32 or uint32 [%d, words]" % rows)
        words = mask.shape[1]
    arg, out, kept = _beams_arg(scores, beams, beams if k is None else k, finished, pad_id, keep_slots, out, rows, dev)
    need = beam_workspace_bytes(rows, beams, V)
    raw = _raw_stream(dev)
    ws = _scratch(need, dev, raw).data_ptr() if workspace is None else _own_workspace(workspace, need, dev)
    st = _lib.lmh_beam_select(arg, logits.data_ptr(), _DTYPES[logits.dtype], V, pitch, _ptr(mask), words, ws, need,
                              _status_word(dev_status, dev), raw)
    if st != OK:
        raise LMHError(st, "lmh_beam_select")
    return out


def beam_select_lists(topk_ids, topk_logprobs, scores, beams, k=None, finished=None, pad_id=0, keep_slots=False,
                      dev_status=None, out=None, stream=None):
    """beam_select from each beam's own best tokens: topk_ids (int32) and topk_logprobs (fp32) [rows, n],
    as project_logprobs and logprobs_from_logits return them (lmh_beam_select_lists).  Lists of at least
    k entries hold every continuation that can be chosen."""
    dev = topk_ids.device
    if stream is not None:
        with _on_stream(stream, dev):
            return beam_select_lists(topk_ids, topk_logprobs, scores, beams, k, finished, pad_id, keep_slots,
                                     dev_status, out)
    if _other_device(dev):
        with torch.cuda.device(dev):
            return beam_select_lists(topk_ids, topk_logprobs, scores, beams, k, finished, pad_id, keep_slots,
                                     dev_status, out)
    rows, n = topk_ids.shape
    assert topk_ids.is_cuda
    if topk_ids.dtype != torch.int32 or topk_logprobs.dtype != torch.float32 or topk_logprobs.shape != (rows, n) or \
            topk_logprobs.device != dev or not topk_ids.is_contiguous() or not topk_logprobs.is_contiguous():
        raise ValueError("topk_ids must be contiguous int32, topk_logprobs contiguous float32 of the same shape")
    arg, out, kept = _beams_arg(scores, beams, beams if k is None else k, finished, pad_id, keep_slots, out, rows, dev)
    st = (_lib or load()).lmh_beam_select_lists(arg, topk_ids.data_ptr(), topk_logprobs.data_ptr(), n,
                                                _status_word(dev_status, dev), _raw_stream(dev))
    if st != OK:
        raise LMHError(st, "lmh_beam_select_lists")
    return out


def _row_state(src, dst, dim, length_dim):
    """(struct lmh_row_state, rows) of a tensor whose dimension `dim` is the rows of a batch."""
    nd = src.dim()
    if not -nd <= dim < nd:
        raise ValueError("no dimension %d in a tensor of %d" % (dim, nd))
    dim %= nd
    if dst.shape != src.shape or dst.dtype != src.dtype or dst.device != src.device:
        raise ValueError("a state's output must have its shape, type and device")
    if src.numel() == 0:
        return RowStateArg(), src.shape[dim]
    es, shape, a, b = src.element_size(), src.shape, src.stride(), dst.stride()
    # the chunk: the last dimensions, as far as both are contiguous (with positions: from them on)
    chunk, at = 1, nd
    first = dim + 1
    if length_dim is not None:
        length_dim %= nd
        if length_dim <= dim:
            raise ValueError("the positions' dimension must come after the rows'")
        first = length_dim
    while at > first and (shape[at - 1] == 1 or (a[at - 1] == chunk and b[at - 1] == chunk)):
        at -= 1
        chunk *= shape[at]
    position = 0
    if length_dim is not None:
        if at > length_dim:
            raise ValueError("a row's positions must be contiguous")
        position = chunk // max(shape[length_dim], 1) * es
    outer = []  # [size, stride, stride] of what is left, neighbours taken together where both strides allow it
    for d in range(at):
        if d == dim or shape[d] == 1:
            continue
        if outer and outer[-1][1] == a[d] * shape[d] and outer[-1][2] == b[d] * shape[d]:
            outer[-1] = [outer[-1][0] * shape[d], a[d], b[d]]
        else:
            outer.append([shape[d], a[d], b[d]])
    if len(outer) > 2:
        raise ValueError("a state may have two runs of strided dimensions beside its rows, not %d" % len(outer))
    outer = [[1, 0, 0]] * (2 - len(outer)) + outer
    if shape[dim] > 1 and b[dim] == 0 or any(n > 1 and t == 0 for n, _, t in outer):
        raise ValueError("a state's rows must not share memory")
    two = ctypes.c_int64 * 2
    return RowStateArg(src.data_ptr(), dst.data_ptr(), a[dim] * es, b[dim] * es, two(*(o[1] * es for o in outer)),
                       two(*(o[2] * es for o in outer)), outer[0][0], outer[1][0], chunk * es, position), shape[dim]


class RowStates:
    """States that follow the rows of a batch (struct lmh_row_state), made once and used every step.

    tensors: any types and shapes; dims: the dimension of each that is the rows (an int for all, or one
    each); length_dims: the dimension of each that holds positions, or None where it has none (after the
    rows' dimension, contiguous from there on); outs: tensors of the same shapes for the moved rows, or
    None (in place).  The object keeps the tensors alive.
    """

    def __init__(self, tensors, dims=0, length_dims=None, outs=None):
        tensors = list(tensors)
        n = len(tensors)
        if not n:
            raise ValueError("no states")
        dims = [dims] * n if isinstance(dims, int) else list(dims)
        length_dims = [length_dims] * n if length_dims is None or isinstance(length_dims, int) else list(length_dims)
        outs = tensors if outs is None else list(outs)
        if len(dims) != n or len(length_dims) != n or len(outs) != n:
            raise ValueError("dims, length_dims and outs must have one entry for each of the %d states" % n)
        dev = tensors[0].device
        self._arg = (RowStateArg * n)()
        self.rows = None
        for i, (src, dst, dim, along) in enumerate(zip(tensors, outs, dims, length_dims)):
            if src.device != dev:
                raise ValueError("the states must be on one device")
            self._arg[i], rows = _row_state(src, dst, dim, along)
            if self.rows not in (None, rows):
                raise ValueError("the states have %d and %d rows" % (self.rows, rows))
            self.rows = rows
        self._ranges = _check_apart(tensors, outs)
        self.tensors, self.outs, self.device, self._n = tensors, outs, dev, n


def _layout(t):
    """A tensor's bytes as ([(count, stride)], width): runs of `width` bytes at sums of multiples of the strides (none
    of them 0), the largest first."""
    es = t.element_size()
    dims = sorted(((s * es, n) for n, s in zip(t.shape, t.stride()) if n > 1 and s), reverse=True)
    width = es
    while dims and dims[-1][0] == width:
        width *= dims.pop()[1]
    return [(n, s) for s, n in dims], width


def _extent(dims, width):
    return width + sum((n - 1) * s for n, s in dims)


def _meet(a, b, shift, steps):
    """Whether two layouts, the second `shift` bytes behind the first, have a byte in common.  steps: [how many looks are
    left]; without one they count as meeting."""
    steps[0] -= 1
    if steps[0] < 0:
        return True
    if not -_extent(*b) < shift < _extent(*a):
        return False
    (da, wa), (db, wb) = a, b
    if not da and not db:
        return True
    S = max(d[0][1] for d in (da, db) if d)
    na, da = (da[0][0], da[1:]) if da and da[0][1] == S else (1, da)
    nb, db = (db[0][0], db[1:]) if db and db[0][1] == S else (1, db)
    a, b = (da, wa), (db, wb)
    # the second's place along S less the first's: those for which the rest can meet
    least, most = max(1 - na, -((_extent(*b) + shift - 1) // S)), min(nb - 1, (_extent(*a) - shift - 1) // S)
    return any(_meet(a, b, shift + d * S, steps) for d in range(least, most + 1))


_MEET_STEPS = 4096  # (nested strides take a few dozen)


def _meets_itself(t):
    """Whether two of a tensor's elements share memory."""
    if t.is_contiguous():
        return False
    if any(n > 1 and s == 0 for n, s in zip(t.shape, t.stride())):
        return True
    dims, width = _layout(t)
    steps = [_MEET_STEPS]
    for i, (n, S) in enumerate(dims):
        rest = dims[i + 1:], width
        if any(_meet(rest, rest, d * S, steps) for d in range(1, min(n - 1, (_extent(*rest) - 1) // S) + 1)):
            return True
    return False


def _check_apart(tensors, outs):
    """What is written is written once, and read by no state but one in place.  Returns the outputs' ranges."""
    spans, ranges = [], []
    for t, u in zip(tensors, outs):
        if not u.numel():
            continue
        if _meets_itself(u):
            raise ValueError("a state's rows must not share memory")
        lo, hi = _range(u)
        ranges.append((lo, hi))
        spans.append((lo, hi, u, True))
        if t is not u and (t.data_ptr() != lo or t.stride() != u.stride()):
            spans.append((*_range(t), t, False))
    spans.sort(key=lambda s: s[0])
    live, most = [], 0  # the spans so far that go on; where the last of them ends
    layouts = {}

    def layout(t):
        if id(t) not in layouts:
            layouts[id(t)] = _layout(t)
        return layouts[id(t)]
    for span in spans:
        lo, hi, t, written = span
        live = [s for s in live if s[1] > lo] if lo < most else []
        for first, _, u, too in live:
            if (written or too) and _meet(layout(u), layout(t), lo - first, [_MEET_STEPS]):
                raise ValueError("the same memory is written twice, or written and read by two states")
        live.append(span)
        most = max(most, hi)
    return ranges


def _range(t):
    """The first byte of a tensor's memory, and the one behind its last."""
    if t.is_contiguous():
        return t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def reorder_rows(states, parents, beams, lengths=None, dev_status=None, stream=None):
    """Every state's row r becomes what row parents[r] held, within groups of `beams` rows
    (lmh_reorder_rows).

    states: a RowStates (or a list of tensors [rows, ...], moved in place); parents: int32 [rows] or
    [groups, beams], as beam_select returns them with k == beams, -1 for the row itself; lengths: int32
    [rows] or None, the positions in use of every row as it is before: of states with positions a row's
    first lengths[parent] are moved.  stream: the call is made on it, conversions included.
    Returns the list of the states' outputs.
    """
    if not isinstance(states, RowStates):
        states = RowStates(states)
    dev, rows = states.device, states.rows
    if stream is not None:
        with _on_stream(stream, dev):
            return reorder_rows(states, parents, beams, lengths, dev_status)
    if _other_device(dev):
        with torch.cuda.device(dev):
            return reorder_rows(states, parents, beams, lengths, dev_status)
    if beams <= 0 or rows % beams:
        raise ValueError("the rows must be whole groups of %d beams" % beams)
    parents = _per_row(parents, torch.int32, rows, dev, "parents")
    lengths = _per_row(lengths, torch.int32, rows, dev, "lengths")
    for t in (parents, lengths):
        if t is not None:
            lo = t.data_ptr()
            if any(lo < e and b < lo + 4 * rows for b, e in states._ranges):
                raise ValueError("parents and lengths may not lie in a state that is written")
    st = (_lib or load()).lmh_reorder_rows(states._arg, states._n, rows // beams, beams, _ptr(parents), _ptr(lengths),
                                           _status_word(dev_status, dev), _raw_stream(dev))
    if st != OK:
        raise LMHError(st, "lmh_reorder_rows")
    return states.outs


# ---------------------------------------------------------------------------
# kernel trace
# ---------------------------------------------------------------------------

TRACE_KERNELS = ("select_rows", "gather_rows", "head_logprobs", "logits_reduce", "merge_partials",
                 "logits_select", "full_logprobs", "sample_logits", "project_q4", "lookup_q4", "quantize_q4",
                 "adapter_plan", "adapter_down", "adapter_up", "beam_stream", "beam_choose", "reorder_rows")


def trace_enable(on=True):
    _check(load().lmh_trace_enable(1 if on else 0), "lmh_trace_enable")


def trace_reset():
    load().lmh_trace_reset()


def trace_read(kernel):
    """(launches, total_ms) of a kernel since the last reset (waits for its events)."""
    n = ctypes.c_int64(0)
    ms = ctypes.c_double(0.0)
    _check(load().lmh_trace_read(kernel.encode(), ctypes.byref(n), ctypes.byref(ms)), "lmh_trace_read")
    return int(n.value), float(ms.value)


def debug_set_wait_limit(limit_ns):
    """Test hook: the kernels' bounded waits give up after limit_ns (0: the 2 s default)."""
    _check(load().lmh_debug_set_wait_limit(int(limit_ns)), "lmh_debug_set_wait_limit")


# ---------------------------------------------------------------------------
# vocabulary-parallel head (several GPUs, each holding a share of the vocabulary)
# ---------------------------------------------------------------------------

def vocab_share(V, rank, world):
    """(v_begin, v_count): rank's share of token ids [0, V), whole 64-id blocks spread as
    evenly as possible (the last share takes the ragged tail).  Pure host arithmetic."""
    assert 0 <= rank < world and V >= 1
    nblk = (V + 63) // 64
    lo = (nblk * rank) // world
    hi = (nblk * (rank + 1)) // world
    begin, end = 64 * lo, min(V, 64 * hi)
    return begin, max(0, end - begin)


def record_bytes(k_max):
    """Bytes of one row's record (include/lmh.h: lmh_record_bytes)."""
    n = int(load().lmh_record_bytes(int(k_max)))
    if n == 0:
        raise LMHError(ERR_INVALID_ARG, "lmh_record_bytes")
    return n


def project_partials(hidden, W_share, v_begin, V, row_idx=None, rows=None, sel=None, row_k=None, k_max=0,
                     records=None, workspace=None, dev_status=None, stream=None):
    """One share of a vocabulary-parallel head (lmh_project_partials).

    W_share: bf16 [v_count, H], rows v_begin.. of lm_head.weight; sel holds global ids.
    Returns the uint8 [rows, record_bytes(k_max)] record buffer.
    """
    assert hidden.is_cuda and hidden.dtype == torch.bfloat16 and hidden.dim() == 2 and hidden.stride(1) == 1
    assert W_share.is_cuda and W_share.dtype == torch.bfloat16 and W_share.is_contiguous()
    T, H = hidden.shape
    v_count = W_share.shape[0]
    assert W_share.shape[1] == H
    dev = hidden.device
    if row_idx is not None:
        rows = row_idx.numel() if rows is None else rows
        assert row_idx.dtype == torch.int32 and row_idx.is_cuda
    elif rows is None:
        rows = T
    sel_t = _dev_i32(sel, dev, rows, "sel")
    rk_t = _dev_i32(row_k, dev, rows, "row_k")
    rb = record_bytes(k_max)
    if records is None:
        records = torch.empty((rows, rb), dtype=torch.uint8, device=dev)
    assert records.is_cuda and records.is_contiguous() and records.numel() >= rows * rb
    ws = _workspace(workspace, workspace_bytes(rows, H, v_count, k_max, PATH_PROJECT), dev)
    _check(load().lmh_project_partials(
        _p(hidden), hidden.stride(0) if T > 1 else H, T, _p(row_idx), int(rows), H, _p(W_share), W_VH,
        int(v_begin), int(v_count), int(V), _p(sel_t), _p(rk_t), int(k_max), _p(records), _p(ws),
        ws.numel() * ws.element_size(), _p(dev_status), _stream(stream)), "lmh_project_partials")
    return records


def merge_records(records, num_parts, rows, V, sel=None, row_k=None, k_max=0, workspace=None, dev_status=None,
                  out=None, stream=None):
    """Final results from the gathered records [num_parts, rows, record_bytes] (lmh_merge_records)."""
    assert records.is_cuda and records.is_contiguous()
    dev = records.device
    sel_t = _dev_i32(sel, dev, rows, "sel")
    rk_t = _dev_i32(row_k, dev, rows, "row_k")
    o = out if out is not None else _outputs(rows, k_max, sel_t is not None, dev, V)
    need = int(load().lmh_merge_workspace_bytes(int(rows), int(num_parts), int(k_max)))
    if need == 0:
        raise LMHError(ERR_INVALID_ARG, "lmh_merge_workspace_bytes")
    ws = _workspace(workspace, need, dev)
    _check(load().lmh_merge_records(
        _p(records), int(num_parts), int(rows), int(V), _p(sel_t), _p(rk_t), int(k_max), _p(o["lse"]),
        _p(o["sel_logprob"]), _p(o["topk_ids"]), _p(o["topk_logprobs"]), _p(ws), ws.numel() * ws.element_size(),
        _p(dev_status), _stream(stream)), "lmh_merge_records")
    return o


def gather_records(records, group=None):
    """All-gather of every rank's record buffer, in rank order: [world, *records.shape].

    The one exchange step of the vocabulary-parallel head (a collective of the
    caller's torch.distributed group: NCCL into device memory on GPUs, gloo on the
    host).  Pure plumbing: the records are opaque bytes here.
    """
    import torch.distributed as dist
    world = dist.get_world_size(group)
    out = torch.empty((world,) + tuple(records.shape), dtype=records.dtype, device=records.device)
    if dist.get_backend(group) == "nccl":
        dist.all_gather_into_tensor(out, records.contiguous(), group=group)
    else:
        dist.all_gather(list(out.unbind(0)), records.contiguous(), group=group)
    return out


def vocab_parallel_logprobs(hidden, W_share, v_begin, V, row_idx=None, rows=None, sel=None, row_k=None, k_max=0,
                            group=None, dev_status=None, stream=None):
    """The rows' O(k+1) results with the head split over the ranks of `group` by vocabulary:
    this rank's share (project_partials), one all-gather of the records, the merge."""
    rec = project_partials(hidden, W_share, v_begin, V, row_idx=row_idx, rows=rows, sel=sel, row_k=row_k,
                           k_max=k_max, dev_status=dev_status, stream=stream)
    allrec = gather_records(rec, group)
    n = rec.shape[0]
    return merge_records(allrec, allrec.shape[0], n, V, sel=sel, row_k=row_k, k_max=k_max, dev_status=dev_status,
                         stream=stream)
