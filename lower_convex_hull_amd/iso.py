"""Thin ctypes binding of libiso.so (include/iso.h), argument marshalling only.

Every step of the fit runs in the library's gfx950 kernels; this module only
passes pointers, sizes and the current torch stream.  It raises if the built
library is missing: there is no fallback.

Functions with the C names take raw device pointers (ints); ``fit``, ``vjp``,
``calib_curve`` and the loss operators ``token_logp``, ``token_logp_vjp``,
``pref_loss``, ``policy_loss`` and ``policy_loss_logits`` and the decoding steps
``beam_select``, ``beam_reorder``, ``pages_fork`` and ``pages_compact`` are
convenience wrappers over torch CUDA tensors that allocate the outputs and the
workspace with torch.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libiso.so")

ISO_OK = 0
ISO_WARN_NONFINITE = 1
ISO_ERR_ARG = -1
ISO_ERR_WEIGHT = -2
ISO_ERR_NOMEM = -3
ISO_ERR_HIP = -4
ISO_ERR_WORKSPACE = -5
ISO_ERR_DATA = -6
ISO_ERR_INVARIANT = -7

ISO_F_NOCHECK = 1
ISO_F_DECREASING = 2
ISO_F_COPY_CONTROL = 4
ISO_F_DEBUG_INVARIANTS = 8
ISO_F_WAVE_MERGES = 0x400
ISO_F_THREE_CASE = 0x800
ISO_F_TREE_MERGES = 0x1000
ISO_F_WEIGHTED_HINT = 0x100
ISO_F_PHASE_STAMPS = 0x200

ISO_DT_F32 = 0
ISO_DT_F16 = 1
ISO_DT_BF16 = 2

ISO_PREF_MEAN = 1
ISO_PREF_SQUARED = 2
ISO_POLICY_SEQ_MEAN = 1
ISO_POLICY_ADV_TOKEN = 2

ISO_PHASE_NAMES = ("short_rows", "chunk_hulls", "merge", "expand", "copy_bridge", "copy_move",
                   "merge_top", "chunk_redo")

ISO_NOALLOC_BYTES = 64 << 20

EXPORTS = ("iso_fit", "iso_fit_ex", "iso_fit_noalloc", "iso_workspace_bytes", "iso_status_str",
           "iso_release", "iso_chunk_size", "iso_short_row_max", "iso_timing_enable",
           "iso_timing_read", "iso_vjp", "iso_vjp_f64", "iso_vjp_workspace_bytes", "iso_fit_ex_f64",
           "iso_fit_f64", "iso_calib_fit", "iso_calib_apply", "iso_calib_workspace_bytes",
           "iso_copy_probe", "iso_token_logp", "iso_token_logp_vjp", "iso_token_logp_workspace_bytes",
           "iso_pref_loss", "iso_pref_loss_workspace_bytes", "iso_policy_loss",
           "iso_policy_loss_workspace_bytes", "iso_policy_loss_logits",
           "iso_policy_loss_logits_workspace_bytes", "iso_beam_select", "iso_beam_select_workspace_bytes",
           "iso_beam_reorder", "iso_pages_fork", "iso_pages_fork_workspace_bytes", "iso_pages_compact",
           "iso_pages_compact_workspace_bytes")

ISO_MAX_BLOCKS = 512
LAUNCH_BLOCKS = 16  # arrays that one launch takes


class Blocks(ctypes.Structure):
    """iso_blocks: the blocks of an array that its rows (or pages) hold; strides in bytes."""

    _fields_ = [("base", ctypes.c_void_p), ("outer", ctypes.c_int64), ("outer_stride", ctypes.c_int64),
                ("row_stride", ctypes.c_int64), ("mid", ctypes.c_int64), ("mid_stride", ctypes.c_int64),
                ("inner", ctypes.c_int64)]


_lib = None


class IsoError(RuntimeError):
    def __init__(self, status: int):
        super().__init__(f"libiso status {status}: {iso_status_str(status)}")
        self.status = status


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run __graft_entry__.build() first")
        L = ctypes.CDLL(LIB_PATH)
        p, i64, u32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t
        L.iso_fit.argtypes = [p, p, i64, i64, p]
        L.iso_fit.restype = ctypes.c_int
        L.iso_fit_ex.argtypes = [p, p, i64, i64, p, p, p, sz, p, u32]
        L.iso_fit_ex.restype = ctypes.c_int
        L.iso_fit_ex_f64.argtypes = [p, p, i64, i64, p, p, p, sz, p, u32]
        L.iso_fit_ex_f64.restype = ctypes.c_int
        L.iso_fit_f64.argtypes = [p, p, i64, i64, p]
        L.iso_fit_f64.restype = ctypes.c_int
        L.iso_copy_probe.argtypes = [p, p, sz, p]
        L.iso_copy_probe.restype = ctypes.c_int
        L.iso_calib_fit.argtypes = [p, p, p, i64, p, p, p, p, sz, p]
        L.iso_calib_fit.restype = ctypes.c_int
        L.iso_calib_apply.argtypes = [p, p, i64, p, p, i64, p, p]
        L.iso_calib_apply.restype = ctypes.c_int
        L.iso_calib_workspace_bytes.argtypes = [i64]
        L.iso_calib_workspace_bytes.restype = sz
        L.iso_fit_noalloc.argtypes = [p, p, i64, i64, p, p, p, u32]
        L.iso_fit_noalloc.restype = ctypes.c_int
        L.iso_vjp.argtypes = [p, p, p, p, i64, i64, p, p, p, sz, p]
        L.iso_vjp.restype = ctypes.c_int
        L.iso_vjp_f64.argtypes = [p, p, p, p, i64, i64, p, p, p, sz, p]
        L.iso_vjp_f64.restype = ctypes.c_int
        L.iso_vjp_workspace_bytes.argtypes = [i64, i64]
        L.iso_vjp_workspace_bytes.restype = sz
        L.iso_workspace_bytes.argtypes = [i64, i64, u32]
        L.iso_workspace_bytes.restype = sz
        f64, i32 = ctypes.c_double, ctypes.c_int
        L.iso_token_logp.argtypes = [p, i32, i64, i64, i64, p, f64, p, p, p, p, sz, p]
        L.iso_token_logp.restype = ctypes.c_int
        L.iso_token_logp_workspace_bytes.argtypes = [i64, i64, i32]
        L.iso_token_logp_workspace_bytes.restype = sz
        L.iso_token_logp_vjp.argtypes = [p, i32, i64, i64, i64, p, f64, p, p, p, p, p, i64, p]
        L.iso_token_logp_vjp.restype = ctypes.c_int
        L.iso_pref_loss.argtypes = [p, p, p, p, i64, i64, f64, f64, p, p, p, p, f64, p, sz, p, u32]
        L.iso_pref_loss.restype = ctypes.c_int
        L.iso_pref_loss_workspace_bytes.argtypes = [i64, i64]
        L.iso_pref_loss_workspace_bytes.restype = sz
        L.iso_policy_loss.argtypes = [p, p, p, p, p, p, i64, i64, f64, f64, f64, f64, p, p, p, f64, p,
                                      sz, p, u32]
        L.iso_policy_loss.restype = ctypes.c_int
        L.iso_policy_loss_workspace_bytes.argtypes = [i64, i64]
        L.iso_policy_loss_workspace_bytes.restype = sz
        L.iso_policy_loss_logits.argtypes = [p, i32, i64, i64, i64, p, f64, p, p, p, p, i64, f64, f64,
                                             f64, f64, p, p, p, p, i64, f64, p, sz, p, u32]
        L.iso_policy_loss_logits.restype = ctypes.c_int
        L.iso_policy_loss_logits_workspace_bytes.argtypes = [i64, i64, i64, i32]
        L.iso_policy_loss_logits_workspace_bytes.restype = sz
        L.iso_beam_select.argtypes = [p, i32, i64, i64, i64, i64, p, p, p, ctypes.c_int32, f64, i64, p, p, p, p, p,
                                      sz, p]
        L.iso_beam_select.restype = ctypes.c_int
        L.iso_beam_select_workspace_bytes.argtypes = [i64, i64, i64, i64, i32]
        L.iso_beam_select_workspace_bytes.restype = sz
        L.iso_beam_reorder.argtypes = [p, i32, p, i64, i64, p]
        L.iso_beam_reorder.restype = ctypes.c_int
        L.iso_pages_fork.argtypes = [p, p, i64, i64, p, i64, i64, p, p, ctypes.c_int32, i64, p, i32, p, p, p, p, p, sz,
                                     p]
        L.iso_pages_fork.restype = ctypes.c_int
        L.iso_pages_fork_workspace_bytes.argtypes = [i64, i64, i64]
        L.iso_pages_fork_workspace_bytes.restype = sz
        L.iso_pages_compact.argtypes = [p, i64, p, i64, p, i32, p, p, p, p, p, sz, p]
        L.iso_pages_compact.restype = ctypes.c_int
        L.iso_pages_compact_workspace_bytes.argtypes = [i64]
        L.iso_pages_compact_workspace_bytes.restype = sz
        L.iso_status_str.argtypes = [ctypes.c_int]
        L.iso_status_str.restype = ctypes.c_char_p
        L.iso_release.argtypes = []
        L.iso_release.restype = None
        L.iso_chunk_size.argtypes = [i64]
        L.iso_chunk_size.restype = i64
        L.iso_short_row_max.argtypes = []
        L.iso_short_row_max.restype = i64
        L.iso_timing_enable.argtypes = [ctypes.c_int]
        L.iso_timing_enable.restype = ctypes.c_int
        L.iso_timing_read.argtypes = [p, p, ctypes.c_int]
        L.iso_timing_read.restype = ctypes.c_int
        _lib = L
    return _lib


def iso_fit(y_ptr, w_ptr, rows, n, out_ptr) -> int:
    return lib().iso_fit(y_ptr, w_ptr, rows, n, out_ptr)


def iso_fit_ex(y_ptr, w_ptr, rows, n, out_ptr, block_id_ptr, ws_ptr, ws_bytes, stream, flags) -> int:
    return lib().iso_fit_ex(y_ptr, w_ptr, rows, n, out_ptr, block_id_ptr, ws_ptr, ws_bytes,
                            stream, flags)


def iso_fit_ex_f64(y_ptr, w_ptr, rows, n, out_ptr, block_id_ptr, ws_ptr, ws_bytes, stream,
                   flags) -> int:
    return lib().iso_fit_ex_f64(y_ptr, w_ptr, rows, n, out_ptr, block_id_ptr, ws_ptr, ws_bytes,
                                stream, flags)


def iso_fit_f64(y_ptr, w_ptr, rows, n, out_ptr) -> int:
    return lib().iso_fit_f64(y_ptr, w_ptr, rows, n, out_ptr)


def iso_copy_probe(src_ptr, dst_ptr, nbytes, stream) -> int:
    return lib().iso_copy_probe(src_ptr, dst_ptr, nbytes, stream)


def iso_calib_fit(scores_ptr, outcomes_ptr, segment_ptr, n, xp_ptr, fp_ptr, k_out, ws_ptr, ws_bytes,
                  stream) -> int:
    """k_out: a ctypes.c_int64 receiving the number of distinct keys."""
    return lib().iso_calib_fit(scores_ptr, outcomes_ptr, segment_ptr, n, xp_ptr, fp_ptr,
                               ctypes.byref(k_out), ws_ptr, ws_bytes, stream)


def iso_calib_apply(xp_ptr, fp_ptr, k, scores_ptr, segment_ptr, m, out_ptr, stream) -> int:
    return lib().iso_calib_apply(xp_ptr, fp_ptr, k, scores_ptr, segment_ptr, m, out_ptr, stream)


def iso_calib_workspace_bytes(n) -> int:
    return lib().iso_calib_workspace_bytes(n)


def iso_fit_noalloc(y_ptr, w_ptr, rows, n, out_ptr, block_id_ptr, stream, flags) -> int:
    return lib().iso_fit_noalloc(y_ptr, w_ptr, rows, n, out_ptr, block_id_ptr, stream, flags)


def iso_vjp(g_ptr, y_ptr, w_ptr, block_id_ptr, rows, n, grad_y_ptr, grad_w_ptr, ws_ptr, ws_bytes,
            stream) -> int:
    return lib().iso_vjp(g_ptr, y_ptr, w_ptr, block_id_ptr, rows, n, grad_y_ptr, grad_w_ptr, ws_ptr,
                         ws_bytes, stream)


def iso_vjp_f64(g_ptr, y_ptr, w_ptr, block_id_ptr, rows, n, grad_y_ptr, grad_w_ptr, ws_ptr,
                ws_bytes, stream) -> int:
    return lib().iso_vjp_f64(g_ptr, y_ptr, w_ptr, block_id_ptr, rows, n, grad_y_ptr, grad_w_ptr,
                             ws_ptr, ws_bytes, stream)


def iso_vjp_workspace_bytes(rows, n) -> int:
    return lib().iso_vjp_workspace_bytes(rows, n)


def iso_token_logp(logits_ptr, dtype, rows, vocab, ld, target_ptr, temperature, logp_ptr, lse_ptr,
                   entropy_ptr, ws_ptr, ws_bytes, stream) -> int:
    return lib().iso_token_logp(logits_ptr, dtype, rows, vocab, ld, target_ptr, temperature, logp_ptr,
                                lse_ptr, entropy_ptr, ws_ptr, ws_bytes, stream)


def iso_token_logp_workspace_bytes(rows, vocab, dtype) -> int:
    return lib().iso_token_logp_workspace_bytes(rows, vocab, dtype)


def iso_token_logp_vjp(logits_ptr, dtype, rows, vocab, ld, target_ptr, temperature, lse_ptr,
                       entropy_ptr, g_logp_ptr, g_entropy_ptr, grad_ptr, ld_grad, stream) -> int:
    return lib().iso_token_logp_vjp(logits_ptr, dtype, rows, vocab, ld, target_ptr, temperature, lse_ptr,
                                    entropy_ptr, g_logp_ptr, g_entropy_ptr, grad_ptr, ld_grad, stream)


def iso_pref_loss(logp_ptr, ref_ptr, mask_ptr, off_ptr, pairs, tokens, beta, label_smoothing, loss_ptr,
                  pair_loss_ptr, reward_ptr, grad_ptr, grad_scale, ws_ptr, ws_bytes, stream, flags) -> int:
    return lib().iso_pref_loss(logp_ptr, ref_ptr, mask_ptr, off_ptr, pairs, tokens, beta, label_smoothing,
                               loss_ptr, pair_loss_ptr, reward_ptr, grad_ptr, grad_scale, ws_ptr, ws_bytes,
                               stream, flags)


def iso_pref_loss_workspace_bytes(tokens, pairs) -> int:
    return lib().iso_pref_loss_workspace_bytes(tokens, pairs)


def iso_policy_loss(logp_ptr, old_ptr, ref_ptr, adv_ptr, mask_ptr, off_ptr, seqs, tokens, clip_lo, clip_hi,
                    kl_coef, norm, loss_ptr, counts_ptr, grad_ptr, grad_scale, ws_ptr, ws_bytes, stream,
                    flags) -> int:
    return lib().iso_policy_loss(logp_ptr, old_ptr, ref_ptr, adv_ptr, mask_ptr, off_ptr, seqs, tokens,
                                 clip_lo, clip_hi, kl_coef, norm, loss_ptr, counts_ptr, grad_ptr, grad_scale,
                                 ws_ptr, ws_bytes, stream, flags)


def iso_policy_loss_workspace_bytes(tokens, seqs) -> int:
    return lib().iso_policy_loss_workspace_bytes(tokens, seqs)


def iso_policy_loss_logits(logits_ptr, dtype, rows, vocab, ld, target_ptr, temperature, old_ptr, ref_ptr,
                           adv_ptr, off_ptr, seqs, clip_lo, clip_hi, kl_coef, norm, loss_ptr, counts_ptr,
                           logp_ptr, grad_ptr, ld_grad, grad_scale, ws_ptr, ws_bytes, stream, flags) -> int:
    return lib().iso_policy_loss_logits(logits_ptr, dtype, rows, vocab, ld, target_ptr, temperature, old_ptr,
                                        ref_ptr, adv_ptr, off_ptr, seqs, clip_lo, clip_hi, kl_coef, norm,
                                        loss_ptr, counts_ptr, logp_ptr, grad_ptr, ld_grad, grad_scale, ws_ptr,
                                        ws_bytes, stream, flags)


def iso_policy_loss_logits_workspace_bytes(rows, vocab, seqs, dtype) -> int:
    return lib().iso_policy_loss_logits_workspace_bytes(rows, vocab, seqs, dtype)


def iso_beam_select(logits_ptr, dtype, batch, beams, vocab, ld, score_ptr, weight_ptr, ended_ptr, end_token,
                    temperature, take, out_score_ptr, out_logp_ptr, out_parent_ptr, out_token_ptr, ws_ptr, ws_bytes,
                    stream) -> int:
    return lib().iso_beam_select(logits_ptr, dtype, batch, beams, vocab, ld, score_ptr, weight_ptr, ended_ptr,
                                 end_token, temperature, take, out_score_ptr, out_logp_ptr, out_parent_ptr,
                                 out_token_ptr, ws_ptr, ws_bytes, stream)


def iso_beam_select_workspace_bytes(batch, beams, vocab, take, dtype) -> int:
    return lib().iso_beam_select_workspace_bytes(batch, beams, vocab, take, dtype)


def iso_beam_reorder(states, count, parent_ptr, batch, beams, stream) -> int:
    """states: a ctypes array of Blocks (here and below)."""
    return lib().iso_beam_reorder(states, count, parent_ptr, batch, beams, stream)


def iso_pages_fork(table_ptr, length_ptr, seqs, max_pages, refs_ptr, pages, page_size, parent_ptr, grow_ptr, grow_all,
                   children, pools, count, new_table_ptr, new_length_ptr, new_refs_ptr, status_ptr, ws_ptr, ws_bytes,
                   stream) -> int:
    return lib().iso_pages_fork(table_ptr, length_ptr, seqs, max_pages, refs_ptr, pages, page_size, parent_ptr,
                                grow_ptr, grow_all, children, pools, count, new_table_ptr, new_length_ptr,
                                new_refs_ptr, status_ptr, ws_ptr, ws_bytes, stream)


def iso_pages_fork_workspace_bytes(seqs, children, pages) -> int:
    return lib().iso_pages_fork_workspace_bytes(seqs, children, pages)


def iso_pages_compact(table_ptr, entries, refs_ptr, pages, pools, count, new_table_ptr, new_refs_ptr, moved_ptr,
                      status_ptr, ws_ptr, ws_bytes, stream) -> int:
    return lib().iso_pages_compact(table_ptr, entries, refs_ptr, pages, pools, count, new_table_ptr, new_refs_ptr,
                                   moved_ptr, status_ptr, ws_ptr, ws_bytes, stream)


def iso_pages_compact_workspace_bytes(pages) -> int:
    return lib().iso_pages_compact_workspace_bytes(pages)


def iso_workspace_bytes(rows, n, flags=0) -> int:
    return lib().iso_workspace_bytes(rows, n, flags)


def iso_status_str(status: int) -> str:
    return lib().iso_status_str(status).decode()


def iso_release() -> None:
    lib().iso_release()


def iso_chunk_size(n: int) -> int:
    return lib().iso_chunk_size(n)


def iso_short_row_max() -> int:
    return lib().iso_short_row_max()


def iso_timing_enable(on: bool) -> int:
    return lib().iso_timing_enable(1 if on else 0)


def iso_timing_read():
    """Per-phase (total ms, launches) of the launches recorded since the last read."""
    n = len(ISO_PHASE_NAMES)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    st = lib().iso_timing_read(ms, cnt, n)
    if st < 0:
        raise IsoError(st)
    return {ISO_PHASE_NAMES[i]: (ms[i], cnt[i]) for i in range(n)}


def _stream_handle(stream):
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def workspace(rows: int, n: int, weighted: bool, flags: int = 0, device=None):
    """A torch uint8 CUDA tensor large enough for iso_fit_ex (256-byte aligned by torch)."""
    import torch

    nbytes = iso_workspace_bytes(rows, n, flags | (ISO_F_WEIGHTED_HINT if weighted else 0))
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device or "cuda")


def fit(y, w=None, *, block_ids: bool = False, flags: int = 0, out=None, ws=None, stream=None,
        check: bool = True):
    """Weighted isotonic fit of each row of a 2-D (or 1-D) float32 or float64 CUDA tensor.

    Returns ``out`` (and ``block_id`` when ``block_ids``).  Raises IsoError on an
    error status; a NONFINITE warning is returned as NaN rows, not raised.
    """
    import torch

    if y.dtype not in (torch.float32, torch.float64) or not y.is_cuda:
        raise TypeError("y must be a float32 or float64 CUDA tensor")
    y2 = y.reshape(1, -1) if y.dim() == 1 else y
    if not y2.is_contiguous():
        raise ValueError("y must be contiguous")
    rows, n = y2.shape
    if w is not None:
        if w.dtype != y.dtype or not w.is_cuda or w.numel() != y2.numel() or not w.is_contiguous():
            raise ValueError("w must be a contiguous CUDA tensor of y's dtype, shaped like y")
    if out is None:
        out = torch.empty_like(y)
    bid = torch.empty(y.shape, dtype=torch.int32, device=y.device) if block_ids else None
    if ws is None:
        ws = workspace(rows, n, w is not None, flags, device=y.device)
    fn = iso_fit_ex if y.dtype == torch.float32 else iso_fit_ex_f64
    st = fn(y2.data_ptr(), None if w is None else w.data_ptr(), rows, n, out.data_ptr(),
                    None if bid is None else bid.data_ptr(), ws.data_ptr(),
                    ws.numel() * ws.element_size(), _stream_handle(stream),
                    flags | (0 if check else ISO_F_NOCHECK))
    if st < 0:
        raise IsoError(st)
    return (out, bid) if block_ids else out


def vjp(g, y, w, block_id, *, grad_w: bool = False, stream=None):
    """Backward pass over torch CUDA tensors (f32 or f64, like g): returns
    grad_y, or (grad_y, grad_w) when grad_w.  block_id is the forward call's."""
    import torch

    g2 = g.reshape(1, -1) if g.dim() == 1 else g
    rows, n = g2.shape
    gy = torch.empty_like(g)
    gw = torch.empty_like(g) if grad_w else None
    nb = iso_vjp_workspace_bytes(rows, n)
    ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=g.device)
    fn = iso_vjp if g.dtype == torch.float32 else iso_vjp_f64
    ptr = lambda t: None if t is None else t.data_ptr()
    st = fn(g.data_ptr(), ptr(y), ptr(w), block_id.data_ptr(), rows, n, gy.data_ptr(), ptr(gw),
            ws.data_ptr(), nb, _stream_handle(stream))
    if st < 0:
        raise IsoError(st)
    return (gy, gw) if grad_w else gy


def calib_curve(scores, outcomes, segment=None, stream=None):
    """Calibration curve over torch CUDA f64 tensors: returns (xp, fp), each of
    the number of distinct keys."""
    import torch

    n = scores.numel()
    xp = torch.empty(n, dtype=torch.float64, device=scores.device)
    fp = torch.empty_like(xp)
    nb = iso_calib_workspace_bytes(n)
    ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=scores.device)
    k = ctypes.c_int64(0)
    st = iso_calib_fit(scores.data_ptr(), outcomes.data_ptr(),
                       None if segment is None else segment.data_ptr(), n, xp.data_ptr(),
                       fp.data_ptr(), k, ws.data_ptr(), nb, _stream_handle(stream))
    if st < 0:
        raise IsoError(st)
    return xp[:k.value], fp[:k.value]


_codes = None


def _dtype_codes(torch):
    global _codes
    if _codes is None:
        _codes = {torch.float32: ISO_DT_F32, torch.float16: ISO_DT_F16, torch.bfloat16: ISO_DT_BF16}
    return _codes


class _Launch:
    """One call of a loss operator over torch tensors: their checks, the stream
    it runs on, and its outputs and workspace.  Outputs and workspace are
    allocated on that stream, and every tensor the call is given is recorded on
    it where it is not the current one, so that none is reused too early.

    A small call's time is the host's, most of it here: the current stream is
    asked for as a bare handle (0.1 us, a Stream object takes 1.9) and nothing
    is allocated that a call does not need (1.3 us a tensor)."""

    __slots__ = ("torch", "lib", "dev", "index", "other", "handle")

    def __init__(self, lead, stream):
        import torch

        if not lead.is_cuda:
            raise TypeError("the tensors must be CUDA tensors")
        self.torch, self.lib, self.dev, self.index = torch, lib(), lead.device, lead.get_device()
        if self.index != torch._C._cuda_getDevice():
            raise ValueError("the tensors must be on the current device")
        current = torch._C._cuda_getCurrentRawStream(self.index)
        self.handle = current if stream is None else stream.cuda_stream
        self.other = stream if self.handle != current else None

    def use(self, t, name, shape, dtypes):
        """The pointer of input t (None: NULL) after its checks."""
        if t is None:
            return None
        if t.get_device() != self.index or t.dtype not in dtypes:
            raise TypeError(f"{name} must be a tensor of {' or '.join(str(d) for d in dtypes)} on {self.dev}")
        if t.shape != shape:
            raise ValueError(f"{name} must have the shape {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if self.other is not None:
            t.record_stream(self.other)
        return t.data_ptr()

    def new(self, dtype, *shape):
        # sizes one by one: torch takes 0.4 us longer over a tuple
        if self.other is None:
            return self.torch.empty(*shape, dtype=dtype, device=self.dev)
        with self.torch.cuda.stream(self.other):
            return self.torch.empty(*shape, dtype=dtype, device=self.dev)

    def workspace(self, nbytes):
        """(tensor, pointer) of the workspace; none where a call needs none."""
        if not nbytes:
            return None, None
        ws = self.new(self.torch.uint8, nbytes)
        return ws, ws.data_ptr()

    def logits(self, t, name):
        """(pointer, dtype code, rows, vocab, ld) of a matrix of logits: 2-D, its rows contiguous."""
        code = _dtype_codes(self.torch).get(t.dtype)
        if code is None or t.get_device() != self.index:
            raise TypeError(f"{name} must be a float32, float16 or bfloat16 CUDA tensor")
        if t.dim() != 2 or t.shape[1] < 1:
            raise ValueError(f"{name} must have the shape (rows, vocab)")
        rows, vocab = t.shape
        ld = t.stride(0) if rows > 1 else vocab
        if (vocab > 1 and t.stride(1) != 1) or ld < vocab:
            raise ValueError(f"{name}'s rows must be contiguous and not overlap")
        if self.other is not None:
            t.record_stream(self.other)
        return t.data_ptr(), code, rows, vocab, ld

    def grad_of(self, logits, out):
        """The gradient's tensor (a new one, or `out`) with its pointer and ld."""
        if out is None:
            out = self.new(logits.dtype, *logits.shape)
            return out, out.data_ptr(), logits.shape[1]
        if out.shape != logits.shape or out.dtype != logits.dtype:
            raise ValueError("out must have the logits' shape and dtype")
        ptr, _, _, _, ld = self.logits(out, "out")
        return out, ptr, ld


def _sequences(launch, t, seq_off):
    """(sequences, tokens, pointer of the offsets) of a packed 1-D tensor with
    offsets, a padded 2-D (sequences, length) one, or one 1-D sequence."""
    if t.dim() == 2 and seq_off is None:
        return t.shape[0], t.numel(), None
    if t.dim() != 1:
        raise ValueError("tokens must be 1-D (packed) or, without seq_off, 2-D (sequences, length)")
    if seq_off is None:
        return 1, t.numel(), None
    if seq_off.dim() != 1 or seq_off.numel() < 1:
        raise ValueError("seq_off must have the shape (sequences + 1,)")
    off = launch.use(seq_off, "seq_off", seq_off.shape, (launch.torch.int32,))
    return seq_off.numel() - 1, t.numel(), off


def _done(st):
    if st < 0:
        raise IsoError(st)


def _int32(x, name):
    """x, where 32 bits hold it (ctypes would keep the low ones of any other)."""
    if not -0x80000000 <= x <= 0x7fffffff:
        raise ValueError(f"{name} must be a 32-bit number")
    return x


def token_logp(logits, target, *, temperature: float = 1.0, entropy: bool = False, stream=None):
    """Log-probabilities of the targets under softmax(logits / temperature), row
    by row: (logp, lse), or (logp, lse, entropies) when entropy.  logits: 2-D
    f32, f16 or bf16 CUDA tensor with contiguous rows; target: int32 (rows,),
    negative for ignored rows (outputs 0)."""
    c = _Launch(logits, stream)
    t = c.torch
    ptr, code, rows, vocab, ld = c.logits(logits, "logits")
    tgt = c.use(target, "target", (rows,), (t.int32,))
    logp, lse = c.new(t.float32, rows), c.new(t.float32, rows)
    ent = c.new(t.float32, rows) if entropy else None
    nb = c.lib.iso_token_logp_workspace_bytes(rows, vocab, code)
    ws, wptr = c.workspace(nb)
    _done(c.lib.iso_token_logp(ptr, code, rows, vocab, ld, tgt, temperature, logp.data_ptr(), lse.data_ptr(),
                               None if ent is None else ent.data_ptr(), wptr, nb, c.handle))
    return (logp, lse, ent) if entropy else (logp, lse)


def token_logp_vjp(g_logp, logits, target, lse, *, temperature: float = 1.0, entropy=None, g_entropy=None,
                   out=None, stream=None):
    """Backward pass of token_logp: the logits' gradient for g_logp (and, with
    the forward call's entropy, g_entropy).  out may be the logits themselves."""
    c = _Launch(logits, stream)
    f32 = (c.torch.float32,)
    ptr, code, rows, vocab, ld = c.logits(logits, "logits")
    if (entropy is None) != (g_entropy is None):
        raise ValueError("entropy and g_entropy go together")
    shape = (rows,)
    tgt, ls = c.use(target, "target", shape, (c.torch.int32,)), c.use(lse, "lse", shape, f32)
    ent, g = c.use(entropy, "entropy", shape, f32), c.use(g_logp, "g_logp", shape, f32)
    g_ent = c.use(g_entropy, "g_entropy", shape, f32)
    grad, gptr, gld = c.grad_of(logits, out)
    _done(c.lib.iso_token_logp_vjp(ptr, code, rows, vocab, ld, tgt, temperature, ls, ent, g, g_ent, gptr, gld,
                                   c.handle))
    return grad


def pref_loss(logp, ref_logp, seq_off=None, *, mask=None, beta: float = 0.1, label_smoothing: float = 0.0,
              squared: bool = False, mean: bool = False, grad: bool = True, grad_scale: float = 1.0,
              stream=None):
    """Paired preference loss over token log-probabilities: (loss, pair losses,
    rewards, gradient of logp or None).  Sequences alternate chosen, rejected:
    1-D packed by seq_off (int32), or 2-D (2 pairs, length).  ref_logp may be
    None; mask is a bool or uint8 tensor shaped like logp."""
    c = _Launch(logp, stream)
    t = c.torch
    seqs, tokens, off = _sequences(c, logp, seq_off)
    if seqs % 2:
        raise ValueError("sequences must come in pairs")
    lp = c.use(logp, "logp", logp.shape, (t.float32,))
    ref = c.use(ref_logp, "ref_logp", logp.shape, (t.float32,))
    mk = c.use(mask, "mask", logp.shape, (t.bool, t.uint8))
    pairs = seqs // 2
    loss, each, reward = c.new(t.float32, ()), c.new(t.float32, pairs), c.new(t.float32, seqs)
    g = c.new(t.float32, *logp.shape) if grad else None
    nb = c.lib.iso_pref_loss_workspace_bytes(tokens, pairs)
    ws, wptr = c.workspace(nb)
    _done(c.lib.iso_pref_loss(lp, ref, mk, off, pairs, tokens, beta, label_smoothing, loss.data_ptr(),
                              each.data_ptr(), reward.data_ptr(), None if g is None else g.data_ptr(), grad_scale,
                              wptr, nb, c.handle,
                              (ISO_PREF_SQUARED if squared else 0) | (ISO_PREF_MEAN if mean else 0)))
    return loss, each, reward, g


def _policy_flags(seq_mean, token_adv):
    return (ISO_POLICY_SEQ_MEAN if seq_mean else 0) | (ISO_POLICY_ADV_TOKEN if token_adv else 0)


def policy_loss(logp, old_logp, adv, *, ref_logp=None, mask=None, seq_off=None, clip_lo: float = 0.2,
                clip_hi: float = 0.2, kl_coef: float = 0.0, seq_mean: bool = False, token_adv: bool = False,
                norm: float = 0.0, grad: bool = True, grad_scale: float = 1.0, stream=None):
    """Clipped policy loss over token log-probabilities: (loss (3,) = [loss,
    policy part, KL], counts (2,) = [tokens, clipped tokens], gradient of logp
    or None).  Tokens: 1-D packed by seq_off (int32), 2-D (sequences, length),
    or one 1-D sequence.  adv: one value per sequence, or shaped like logp when
    token_adv."""
    c = _Launch(logp, stream)
    t = c.torch
    f32 = (t.float32,)
    seqs, tokens, off = _sequences(c, logp, seq_off)
    shape = logp.shape
    lp = c.use(logp, "logp", shape, f32)
    old, ref = c.use(old_logp, "old_logp", shape, f32), c.use(ref_logp, "ref_logp", shape, f32)
    mk = c.use(mask, "mask", shape, (t.bool, t.uint8))
    av = c.use(adv, "adv", shape if token_adv else (seqs,), f32)
    loss, counts = c.new(t.float32, 3), c.new(t.int32, 2)
    g = c.new(t.float32, *logp.shape) if grad else None
    nb = c.lib.iso_policy_loss_workspace_bytes(tokens, seqs)
    ws, wptr = c.workspace(nb)
    _done(c.lib.iso_policy_loss(lp, old, ref, av, mk, off, seqs, tokens, clip_lo, clip_hi, kl_coef, norm,
                                loss.data_ptr(), counts.data_ptr(), None if g is None else g.data_ptr(), grad_scale,
                                wptr, nb, c.handle, _policy_flags(seq_mean, token_adv)))
    return loss, counts, g


def policy_loss_logits(logits, target, old_logp, adv, *, ref_logp=None, seq_off=None, seqs: int = 1,
                       temperature: float = 1.0, clip_lo: float = 0.2, clip_hi: float = 0.2,
                       kl_coef: float = 0.0, seq_mean: bool = False, token_adv: bool = False,
                       norm: float = 0.0, grad: bool = True, grad_scale: float = 1.0, out=None, stream=None):
    """Clipped policy loss taken from the logits: (loss (3,), counts (2,), logp,
    gradient of the logits or None).  Rows of logits are tokens, packed by
    seq_off or `seqs` sequences of one length; rows whose target is negative
    take no part.  out may be the logits themselves."""
    c = _Launch(logits, stream)
    t = c.torch
    f32 = (t.float32,)
    ptr, code, rows, vocab, ld = c.logits(logits, "logits")
    off = None
    if seq_off is not None:
        if seq_off.dim() != 1 or seq_off.numel() < 1:
            raise ValueError("seq_off must have the shape (sequences + 1,)")
        off = c.use(seq_off, "seq_off", seq_off.shape, (t.int32,))
        seqs = seq_off.numel() - 1
    tgt = c.use(target, "target", (rows,), (t.int32,))
    old, ref = c.use(old_logp, "old_logp", (rows,), f32), c.use(ref_logp, "ref_logp", (rows,), f32)
    av = c.use(adv, "adv", (rows if token_adv else seqs,), f32)
    loss, counts, logp = c.new(t.float32, 3), c.new(t.int32, 2), c.new(t.float32, rows)
    g, gptr, gld = c.grad_of(logits, out) if grad else (None, None, vocab)
    nb = c.lib.iso_policy_loss_logits_workspace_bytes(rows, vocab, seqs, code)
    ws, wptr = c.workspace(nb)
    _done(c.lib.iso_policy_loss_logits(ptr, code, rows, vocab, ld, tgt, temperature, old, ref, av, off, seqs,
                                       clip_lo, clip_hi, kl_coef, norm, loss.data_ptr(), counts.data_ptr(),
                                       logp.data_ptr(), gptr, gld, grad_scale, wptr, nb, c.handle,
                                       _policy_flags(seq_mean, token_adv)))
    return loss, counts, logp, g


def beam_select(logits, score, *, take=None, weight=None, ended=None, end_token: int = -1,
                temperature: float = 1.0, stream=None):
    """The best continuations of each batch item's beams: (scores, log-probabilities,
    parents, tokens), each (batch, take) and in order; parents are rows of logits.
    logits: 2-D f32, f16 or bf16, row b * beams + k the beam k of item b; score:
    (batch, beams) f32; weight: its rank's factor, shaped like score; ended: bool
    or uint8, shaped like score; take: as many as beams, if not given."""
    c = _Launch(logits, stream)
    t = c.torch
    ptr, code, rows, vocab, ld = c.logits(logits, "logits")
    if score.dim() != 2 or score.shape[0] * score.shape[1] != rows:
        raise ValueError("score must have the shape (batch, beams), logits batch * beams rows")
    batch, beams = score.shape
    take = beams if take is None else take
    sc, wt = c.use(score, "score", score.shape, (t.float32,)), c.use(weight, "weight", score.shape, (t.float32,))
    en = c.use(ended, "ended", score.shape, (t.bool, t.uint8))
    if not 1 <= take <= 128:
        raise ValueError("take must be from 1 to 128")
    out, logp = c.new(t.float32, batch, take), c.new(t.float32, batch, take)
    parent, token = c.new(t.int32, batch, take), c.new(t.int32, batch, take)
    nb = c.lib.iso_beam_select_workspace_bytes(batch, beams, vocab, take, code)
    ws, wptr = c.workspace(nb)
    _done(c.lib.iso_beam_select(ptr, code, batch, beams, vocab, ld, sc, wt, en, _int32(end_token, "end_token"), temperature, take,
                                out.data_ptr(), logp.data_ptr(), parent.data_ptr(), token.data_ptr(), wptr, nb,
                                c.handle))
    return out, logp, parent, token


def _joined(shape, stride, begin, end):
    """(count, stride) of dimensions taken as one, None if they are not one; those of size 1 do not count."""
    n, step = 1, 0
    for i in range(begin, end):
        size = shape[i]
        if size != 1:
            if n != 1 and step != size * stride[i]:
                return None
            n, step = n * size, stride[i]
    return n, step


def _grad_mode():
    import torch

    return torch.is_grad_enabled()


def _written(launch, tensors):
    """Tells autograd that a call has written the tensors: a backward pass that saved one raises."""
    launch.torch._C._increment_version((tensors,) if hasattr(tensors, "data_ptr") else tensors)


_ONE = (1, 0)


def _block(launch, t, dim, rows, token_dim):
    """The fields of a Blocks: a tensor whose `rows` rows (or pages) are dimension
    `dim`.  What lies behind a row is blocks of adjacent elements at one stride: from
    `token_dim` on, or as long as they get.  The call writes the tensor and records
    nothing for autograd."""
    if t.get_device() != launch.index:
        raise TypeError(f"every tensor must be on {launch.dev}")
    if t.requires_grad and _grad_mode():
        raise ValueError("a tensor that is written in place may not require grad (but under torch.no_grad)")
    shape, stride = t.shape, t.stride()
    at = dims = len(shape)
    if not 0 <= dim < dims:
        raise ValueError(f"a tensor of shape {tuple(shape)} has no dimension {dim}")
    if shape[dim] != rows:
        raise ValueError(f"dimension {dim} of a tensor of shape {tuple(shape)} must have {rows} rows or pages")
    size = inner = t.element_size()
    last = dim + 1 if token_dim is None else token_dim
    if not dim < last <= dims or (token_dim is not None and last == dims):
        raise ValueError("token_dim must be behind page_dim")
    while at > last:
        if shape[at - 1] != 1 and stride[at - 1] * size != inner:
            if token_dim is None:
                break
            raise ValueError("a page's tokens must be adjacent from token_dim on")
        at -= 1
        inner *= shape[at]
    outer = _joined(shape, stride, 0, dim) if dim else _ONE
    mid = _joined(shape, stride, dim + 1, at) if at > dim + 1 else _ONE
    if outer is None or mid is None:
        raise ValueError("the dimensions before the rows, and those behind them, must have one stride")
    if launch.other is not None:
        t.record_stream(launch.other)
    return t.data_ptr(), outer[0], outer[1] * size, stride[dim] * size, mid[0], mid[1] * size, inner


def _blocks(launch, tensors, dims, rows, token_dim=None):
    """(array of Blocks, count) of tensors that hold `rows` rows each, of one launch."""
    if hasattr(tensors, "data_ptr"):
        tensors = (tensors,)
    count = len(tensors)
    if isinstance(dims, int):
        dims = (dims,) * count
    if len(dims) != count:
        raise ValueError("one dimension for each tensor")
    if count > LAUNCH_BLOCKS:
        raise ValueError(f"at most {LAUNCH_BLOCKS} tensors a launch")
    blocks = [_block(launch, t, dim, rows, token_dim) for t, dim in zip(tensors, dims)]
    return (Blocks * count)(*blocks) if count else None, count


def _arrays(launch, tensors, dims, rows, token_dim=None):
    """_blocks of the tensors of a call, which may be those of several launches."""
    count = 1 if hasattr(tensors, "data_ptr") else len(tensors)
    if count <= LAUNCH_BLOCKS:
        return _blocks(launch, tensors, dims, rows, token_dim)
    if count > ISO_MAX_BLOCKS:
        raise ValueError(f"at most {ISO_MAX_BLOCKS} tensors a call")
    if not isinstance(dims, int) and len(dims) != count:
        raise ValueError("one dimension for each tensor")
    out = (Blocks * count)()
    for i in range(0, count, LAUNCH_BLOCKS):
        part = dims if isinstance(dims, int) else dims[i:i + LAUNCH_BLOCKS]
        some, n = _blocks(launch, tensors[i:i + LAUNCH_BLOCKS], part, rows, token_dim)
        out[i:i + n] = some
    return out, count


def beam_reorder(states, parent, *, dim=0, stream=None):
    """States of beams in the order of their parents, in place: row r of each
    becomes what row parent[r] was.  states: a tensor or several, of any type,
    whose dimension `dim` (one for all, or one each) holds the rows; parent:
    (batch, beams) int32 as beam_select gives, rows of the same item (any other
    value: the row stays).  Returns states.  A state may not require grad (but
    under torch.no_grad); a backward pass that saved one raises."""
    c = _Launch(parent, stream)
    if parent.dim() != 2:
        raise ValueError("parent must have the shape (batch, beams)")
    pr = c.use(parent, "parent", parent.shape, (c.torch.int32,))
    batch, beams = parent.shape
    blocks, count = _arrays(c, states, dim, batch * beams)
    _done(c.lib.iso_beam_reorder(blocks, count, pr, batch, beams, c.handle))
    _written(c, states)
    return states


def pages_fork(table, length, refs, parent, *, page_size: int, grow=1, pools=(), page_dim: int = 0,
               token_dim: int = 1, stream=None):
    """One step of a paged cache: (table, length, refs, status), the cache after
    it.  Child i goes on from sequence parent[i] (none: -1) with room for grow
    more tokens (an int, or int32 shaped like parent); sequences without a child
    are freed.  table: (sequences, max_pages) int32; length, refs, parent: 1-D
    int32.  pools: the tensors of the pages' tokens, pages at dimension page_dim,
    a page's tokens at token_dim; as beam_reorder's states for autograd.  status (int32): pages lacking, children too
    long (nothing is done if either is not 0), pages copied, taken, left free."""
    c = _Launch(table, stream)
    t = c.torch
    i32 = (t.int32,)
    if table.dim() != 2 or refs.dim() != 1 or parent.dim() != 1:
        raise ValueError("table must be 2-D, refs and parent 1-D")
    seqs, most = table.shape
    tb, ln = c.use(table, "table", table.shape, i32), c.use(length, "length", (seqs,), i32)
    rf, pr = c.use(refs, "refs", refs.shape, i32), c.use(parent, "parent", parent.shape, i32)
    pages, children = refs.shape[0], parent.shape[0]
    each, gr = (_int32(grow, "grow"), None) if isinstance(grow, int) else (0, c.use(grow, "grow", parent.shape, i32))
    blocks, count = _arrays(c, pools, page_dim, pages, token_dim)
    for p in ((pools,) if hasattr(pools, "data_ptr") else pools):
        if p.shape[token_dim] != page_size:
            raise ValueError("each pool must have page_size tokens a page")
    new_table, new_length = c.new(t.int32, children, most), c.new(t.int32, children)
    new_refs, status = c.new(t.int32, pages), c.new(t.int32, 5)
    nb = c.lib.iso_pages_fork_workspace_bytes(seqs, children, pages)
    ws, wptr = c.workspace(nb)
    _done(c.lib.iso_pages_fork(tb, ln, seqs, most, rf, pages, page_size, pr, gr, each, children, blocks, count,
                               new_table.data_ptr(), new_length.data_ptr(), new_refs.data_ptr(), status.data_ptr(),
                               wptr, nb, c.handle))
    _written(c, pools)
    return new_table, new_length, new_refs, status


def pages_compact(table, refs, *, pools=(), page_dim: int = 0, stream=None):
    """The live pages (refs > 0) of a paged cache moved together, in place in
    the pools (as pages_fork's): (table, refs, moved, status), the cache after it; moved: where
    each page is now (-1: free); status (int32): live pages, pages moved."""
    c = _Launch(table, stream)
    t = c.torch
    if refs.dim() != 1:
        raise ValueError("refs must be 1-D")
    tb, rf = c.use(table, "table", table.shape, (t.int32,)), c.use(refs, "refs", refs.shape, (t.int32,))
    pages = refs.shape[0]
    blocks, count = _arrays(c, pools, page_dim, pages)
    new_table, new_refs = c.new(t.int32, *table.shape), c.new(t.int32, pages)
    moved, status = c.new(t.int32, pages), c.new(t.int32, 2)
    nb = c.lib.iso_pages_compact_workspace_bytes(pages)
    ws, wptr = c.workspace(nb)
    _done(c.lib.iso_pages_compact(tb, table.numel(), rf, pages, blocks, count, new_table.data_ptr(),
                                  new_refs.data_ptr(), moved.data_ptr(), status.data_ptr(), wptr, nb, c.handle))
    _written(c, pools)
    return new_table, new_refs, moved, status
