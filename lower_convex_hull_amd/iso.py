"""Thin ctypes binding of libiso.so (include/iso.h), argument marshalling only.

Every step of the fit runs in the library's gfx950 kernels; this module only
passes pointers, sizes and the current torch stream.  It raises if the built
library is missing: there is no fallback.

Functions with the C names take raw device pointers (ints); ``fit``, ``vjp``,
``calib_curve`` and the loss operators ``token_logp``, ``token_logp_vjp``,
``pref_loss``, ``policy_loss`` and ``policy_loss_logits`` are convenience
wrappers over torch CUDA tensors that allocate the outputs and the workspace
with torch.
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
           "iso_policy_loss_logits_workspace_bytes")

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
