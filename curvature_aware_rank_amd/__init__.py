"""Python binding of liblrc (argument marshalling only).

Every computation runs in the HIP kernels of liblrc.so; this module checks tensor
shapes, dtypes and devices, allocates device workspace with torch, passes raw device
pointers and torch's current HIP stream, and turns status codes into exceptions.  There
is no fallback: if liblrc.so is missing or no GPU is present the calls raise.

Like the library, the binding never waits for the GPU: failures the kernels find are
reported in the returned device `info` tensors, which the caller reads after its own
synchronisation.  Every tensor whose pointer is passed (contiguous copies included) is
held in a local variable until the C call has returned, so the caching allocator cannot
hand its memory to another tensor while the enqueued kernels may still read it.

Names match the C ABI in include/lrc.h.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "LRC_OK", "LRC_EINVAL", "LRC_EDTYPE", "LRC_EWORKSPACE", "LRC_EHIP", "LRC_ENOTPD",
    "LRC_ENOCONV", "LRC_ENONFINITE", "LRC_F32", "LRC_BF16", "LRC_COV_QUANT_INT8_TOKEN",
    "LRC_SCORE_FISHER", "LRC_SCORE_KFAC", "LRC_RANKSCORE_UNIRANK", "LRC_RANKSCORE_SWIFT", "LrcError", "lib",
    "library_path", "lrc_accumulate_cov", "lrc_whiten_decompose", "lrc_score_components", "lrc_allocate_ranks",
    "lrc_rank_scores", "lrc_rotate_quantize", "lrc_quantize_rows", "lrc_lowrank_ffn", "lrc_ffn_select_channels",
    "lrc_hybrid_ffn", "LRC_CKPT_BLOCK", "lrc_pack_activations", "lrc_unpack_activations", "lrc_layer_norm",
    "lrc_layer_norm_backward", "lrc_linear", "lrc_linear_backward",
    "lrc_status_string", "lrc_profile_start", "lrc_profile_stop", "lrc_profile_kernels",
]

LRC_OK, LRC_EINVAL, LRC_EDTYPE, LRC_EWORKSPACE, LRC_EHIP, LRC_ENOTPD, LRC_ENOCONV, LRC_ENONFINITE = range(8)
LRC_F32, LRC_BF16 = 0, 1
LRC_COV_QUANT_INT8_TOKEN = 0x1
LRC_SCORE_FISHER = 0x1
LRC_SCORE_KFAC = 0x2
LRC_RANKSCORE_UNIRANK = 0x1
LRC_RANKSCORE_SWIFT = 0x2
LRC_CKPT_BLOCK = 64                     # channels that share one checkpoint exponent
_ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "liblrc.so")

_i64, _u32, _sz, _vp, _i32 = ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int

_SIGS = {
    "lrc_accumulate_cov": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _i64, _u32, _vp, _vp, _sz, _vp]),
    "lrc_accumulate_cov_workspace": (_sz, [_i32, _i64, _i64, _u32]),
    "lrc_whiten_decompose": (_i32, [_vp, _i64, _i64, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64,
                                    _i64, ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "lrc_whiten_decompose_workspace": (_sz, [_i64, _i64, _i64, _i64, _i32, _i32]),
    "lrc_whiten_decompose_strided": (_i32, [_vp, _i64, _i64, _i64, _i64, _i64, _vp, _i64, _i64, _i64, _vp, _i64,
                                            _i64, _i64, _i64, ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "lrc_whiten_decompose_strided_workspace": (_sz, [_i64, _i64, _i64, _i64, _i64, _i64]),
    "lrc_score_components": (_i32, [_vp, _vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _u32, _i32, _i32,
                                    _i64, _vp, _vp, _vp, _sz, _vp]),
    "lrc_score_components_workspace": (_sz, [_i64, _i64, _i64, _i64, _u32]),
    "lrc_allocate_ranks": (_i32, [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "lrc_allocate_ranks_workspace": (_sz, [_i64, _i64]),
    "lrc_allocate_ranks_noalloc": (_i32, [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "lrc_allocate_ranks_noalloc_max_items": (_i64, []),
    "lrc_rank_scores": (_i32, [_vp, _vp, _i64, _i64, _vp, ctypes.c_float, _u32, _vp, _vp, _vp]),
    "lrc_rotate_quantize": (_i32, [_vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "lrc_rotate_quantize_workspace": (_sz, [_i64, _i64, _i64]),
    "lrc_quantize_rows": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _vp]),
    "lrc_lowrank_ffn": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _i64,
                               _vp, _vp, _vp, _vp, _i64, _vp, _vp, _sz, _vp]),
    "lrc_lowrank_ffn_workspace": (_sz, [_i64, _i64, _i64, _i64, _i64]),
    "lrc_ffn_select_channels": (_i32, [_vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _vp, _i64, _i64,
                                       ctypes.c_float, _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "lrc_ffn_select_channels_workspace": (_sz, [_i64, _i64]),
    "lrc_hybrid_ffn": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _vp, _vp,
                              _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "lrc_hybrid_ffn_workspace": (_sz, [_i64, _i64, _i64, _i64, _i64, _i64]),
    "lrc_pack_activations": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _vp]),
    "lrc_unpack_activations": (_i32, [_vp, _vp, _i64, _i64, _vp, _i32, _i64, _vp]),
    "lrc_layer_norm": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _vp, ctypes.c_float, _vp, _i64, _vp, _vp, _vp, _vp,
                              _vp, _vp]),
    "lrc_layer_norm_backward": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                       _vp, _vp, _vp, _sz, _vp]),
    "lrc_layer_norm_backward_workspace": (_sz, [_i64, _i64]),
    "lrc_linear": (_i32, [_vp, _i32, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _i32, _vp, _i64, _vp, _i64, _vp, _i64,
                          _vp, _vp, _vp, _vp, _sz, _vp]),
    "lrc_linear_workspace": (_sz, [_i32, _i64, _i64, _i64]),
    "lrc_linear_backward": (_i32, [_vp, _i32, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i32, _vp, _i64,
                                   _vp, _vp, _vp, _i64, _vp, _i64, _vp, _i32, _i64, _vp, _vp, _sz, _vp]),
    "lrc_linear_backward_workspace": (_sz, [_i32, _i64, _i64, _i64]),
    "lrc_status_string": (ctypes.c_char_p, [_i32]),
    "lrc_last_hip_error": (_i32, []),
    "lrc_profile_start": (_i32, []),
    "lrc_profile_stop": (_i32, []),
    "lrc_profile_kernels": (_i32, []),
    "lrc_profile_kernel": (_i32, [_i32, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(_i64),
                                  ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double),
                                  ctypes.POINTER(ctypes.c_double)]),
}


def _load():
    if not os.path.exists(library_path):
        raise ImportError(f"liblrc.so not built at {library_path}; run python curvature_aware_rank_amd/build.py")
    so = ctypes.CDLL(library_path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(so, name)
        fn.restype = res
        fn.argtypes = args
    return so


lib = _load()


class LrcError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = lib.lrc_status_string(status).decode()
        if status == LRC_EHIP:
            msg += f" (hipError {lib.lrc_last_hip_error()})"
        super().__init__(f"{where}: {msg}")
        self.status = status


def lrc_status_string(status: int) -> str:
    return lib.lrc_status_string(status).decode()


def _check(status: int, where: str):
    if status != LRC_OK:
        raise LrcError(status, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dev(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")


def _tensor(t, name, dtype, shape, device=None):
    """Check a GPU tensor's dtype, shape (None entries are free) and device; return it."""
    _dev(t, name)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if len(shape) != t.dim() or any(want is not None and want != got for want, got in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return t


def _info(info, device):
    """An optional caller-given int32 (1,) flag on `device`, or a fresh one set to 0."""
    if info is None:
        return torch.zeros(1, dtype=torch.int32, device=device)
    return _tensor(info, "info", torch.int32, (1,), device)


def _workspace(nbytes: int, device):
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return LRC_BF16
    if t.dtype == torch.float32:
        return LRC_F32
    raise ValueError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _rowmajor_ld(t, name):
    if t.dim() != 2 or t.stride(1) != 1 or t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} must be a row-major 2-D tensor")
    return t.stride(0)


def lrc_accumulate_cov(A: torch.Tensor, C: torch.Tensor, quant: bool = False, info=None):
    """C[lower] += sum_t a_t^T a_t over the rows of A (fake-quantised per token if quant).

    info: optional int32 (1,) device flag (sticky LRC_ENONFINITE); a fresh zeroed one is
    made otherwise.  Returns the flag (read it after synchronising)."""
    _dev(A, "A")
    if A.dim() != 2:
        raise ValueError("A must be (n_tokens, d)")
    n, d = A.shape
    _tensor(C, "C", torch.float32, (d, d), A.device)
    lda = _rowmajor_ld(A, "A")
    ldc = _rowmajor_ld(C, "C")
    dt = _dtype_code(A)
    info = _info(info, A.device)
    flags = LRC_COV_QUANT_INT8_TOKEN if quant else 0
    ws = _workspace(lib.lrc_accumulate_cov_workspace(dt, n, d, flags), A.device)
    _check(lib.lrc_accumulate_cov(_ptr(A), dt, n, d, lda, _ptr(C), ldc, flags, _ptr(info), _ptr(ws), ws.numel(),
                                  _stream()), "lrc_accumulate_cov")
    return info


def lrc_whiten_decompose(W: torch.Tensor, rank: int, Xsum=None, n_x: int = 0, Gsum=None, n_g: int = 0,
                         damping: float = 0.0):
    """Whitened truncated decomposition.  W: (d_out, d_in) or (batch, d_out, d_in) fp32;
    Xsum (d_in, d_in) and Gsum (d_out, d_out) fp32 sums shared by the batch, or
    (batch, d_in, d_in) / (batch, d_out, d_out) with one sum per slice (independent
    layers; the token counts n_x, n_g are common), or None for identity.

    Returns (sigma, left, right, info): sigma (batch, k), left (batch, d_out, r),
    right (batch, r, d_in), info (batch,) int32 -- batch dim dropped for 2-D W.  A
    covariance that is not positive definite or an eigensolver at its sweep cap is
    reported in info only (the call does not wait for the GPU)."""
    _dev(W, "W")
    if W.dtype != torch.float32:
        raise ValueError("W must be fp32")
    squeeze = W.dim() == 2
    W3 = W.unsqueeze(0) if squeeze else W
    if W3.dim() != 3 or W3.stride(2) != 1:
        raise ValueError("W must be (d_out, d_in) or (batch, d_out, d_in), row-major")
    batch, d_out, d_in = W3.shape
    ldw, sw = W3.stride(1), W3.stride(0)
    k = min(d_out, d_in)
    dev = W.device
    sigma = torch.empty(batch, k, dtype=torch.float32, device=dev)
    left = torch.empty(batch, d_out, rank, dtype=torch.float32, device=dev)
    right = torch.empty(batch, rank, d_in, dtype=torch.float32, device=dev)
    info = torch.empty(batch, dtype=torch.int32, device=dev)
    def cov_arg(S, name, dim):
        """(pointer tensor, leading dim, slice stride, slices) of a covariance argument"""
        if S is None:
            return None, 0, 0, 0
        if S.dim() == 3 and squeeze:
            raise ValueError(f"{name}: one sum per slice needs a batched W")
        if S.dim() == 3:
            _tensor(S, name, torch.float32, (batch, dim, dim), dev)
            if S.stride(2) != 1 or S.stride(1) < dim or S.stride(0) < dim * S.stride(1):
                raise ValueError(f"{name} must be row-major slices")
            return S, S.stride(1), S.stride(0), batch
        _tensor(S, name, torch.float32, (dim, dim), dev)
        return S, _rowmajor_ld(S, name), 0, 1

    Xs, ldx, sx, nxs = cov_arg(Xsum, "Xsum", d_in)
    Gs, ldg, sg, ngs = cov_arg(Gsum, "Gsum", d_out)
    nb = lib.lrc_whiten_decompose_strided_workspace(d_out, d_in, batch, rank, nxs, ngs)
    ws = _workspace(nb, dev)
    st = lib.lrc_whiten_decompose_strided(_ptr(W3), d_out, d_in, ldw, batch, sw, _ptr(Xs), ldx, sx, int(n_x),
                                          _ptr(Gs), ldg, sg, int(n_g), int(rank), float(damping), _ptr(sigma),
                                          _ptr(left), _ptr(right), _ptr(info), _ptr(ws), ws.numel(), _stream())
    _check(st, "lrc_whiten_decompose")
    if squeeze:
        return sigma[0], left[0], right[0], info
    return sigma, left, right, info


def lrc_score_components(left=None, right=None, sigma=None, A=None, B=None, mode: str = "fisher",
                         scores=None, accumulate: bool = False, finalize: bool = True, n_total=None, info=None):
    """Per-component scores; returns (scores (k,) fp32, info int32 (1,)).

    mode="fisher": needs left (d_out, k), right (k, d_in) fp32, A (n, d_in), B (n, d_out)
    (both bf16 or both fp32).  mode="kfac": needs sigma (k,) fp32 only.  info: optional
    int32 (1,) device flag that receives LRC_ENONFINITE when a score is NaN/Inf (sticky
    over a chunked stream); a fresh zeroed one is made otherwise."""
    if mode == "kfac":
        _dev(sigma, "sigma")
        if sigma.dtype != torch.float32 or sigma.dim() != 1:
            raise ValueError("sigma must be a 1-D fp32 tensor")
        sig = sigma.contiguous()
        k = sig.numel()
        dev = sig.device
        if scores is None:
            scores = torch.empty(k, dtype=torch.float32, device=dev)
        _tensor(scores, "scores", torch.float32, (k,), dev)
        info = _info(info, dev)
        _check(lib.lrc_score_components(None, None, LRC_F32, 0, 1, 1, None, None, _ptr(sig), k,
                                        LRC_SCORE_KFAC, 0, 1, 1, _ptr(scores), _ptr(info), None, 0, _stream()),
               "lrc_score_components")
        return scores, info
    if mode != "fisher":
        raise ValueError("mode is 'fisher' or 'kfac'")
    _dev(left, "left")
    if left.dim() != 2:
        raise ValueError("left must be (d_out, k)")
    d_out, k = left.shape
    dev = left.device
    _tensor(left, "left", torch.float32, (d_out, k), dev)
    _tensor(right, "right", torch.float32, (k, None), dev)
    d_in = right.shape[1]
    _dev(A, "A")
    _dev(B, "B")
    if A.dim() != 2:
        raise ValueError("A must be (n, d_in)")
    n = A.shape[0]
    _tensor(A, "A", A.dtype, (n, d_in), dev)
    _tensor(B, "B", A.dtype, (n, d_out), dev)
    dt = _dtype_code(A)
    if scores is None:
        scores = torch.empty(k, dtype=torch.float32, device=dev)
    _tensor(scores, "scores", torch.float32, (k,), dev)
    info = _info(info, dev)
    # contiguous copies (if any) stay referenced until the call has returned
    a, b, lf, rt = A.contiguous(), B.contiguous(), left.contiguous(), right.contiguous()
    ws = _workspace(lib.lrc_score_components_workspace(n, d_in, d_out, k, LRC_SCORE_FISHER), dev)
    _check(lib.lrc_score_components(_ptr(a), _ptr(b), dt, n, d_in, d_out, _ptr(lf), _ptr(rt), None, k,
                                    LRC_SCORE_FISHER, int(accumulate), int(finalize), int(n_total or n),
                                    _ptr(scores), _ptr(info), _ptr(ws), ws.numel(), _stream()), "lrc_score_components")
    return scores, info


def lrc_allocate_ranks(scores: torch.Tensor, offsets: torch.Tensor, cost: torch.Tensor, budget: int,
                       want_order: bool = True):
    """Global sort-and-truncate.  scores: (M,) fp32; offsets: (n_mat+1,) int64; cost: (n_mat,) int64.

    Returns (order int32 (M,), n_kept int64 (1,), ranks int32 (n_mat,), kept_mask uint8 (M,), info int32 (1,)).
    With want_order=False the library selects the cut without sorting (the same n_kept,
    ranks and mask) and order is None."""
    _dev(scores, "scores")
    dev = scores.device
    n_mat = cost.numel() if isinstance(cost, torch.Tensor) else 0
    _tensor(scores, "scores", torch.float32, (None,), dev)
    _tensor(offsets, "offsets", torch.int64, (n_mat + 1,), dev)
    _tensor(cost, "cost", torch.int64, (n_mat,), dev)
    M = scores.numel()
    sc, offs, cst = scores.contiguous(), offsets.contiguous(), cost.contiguous()
    order = torch.empty(M, dtype=torch.int32, device=dev) if want_order else None
    n_kept = torch.empty(1, dtype=torch.int64, device=dev)
    ranks = torch.empty(n_mat, dtype=torch.int32, device=dev)
    kept = torch.empty(M, dtype=torch.uint8, device=dev)
    info = torch.empty(1, dtype=torch.int32, device=dev)
    ws = _workspace(lib.lrc_allocate_ranks_workspace(n_mat, M), dev)
    _check(lib.lrc_allocate_ranks(_ptr(sc), _ptr(offs), _ptr(cst), n_mat, M, int(budget),
                                  _ptr(order) if want_order else None, _ptr(n_kept),
                                  _ptr(ranks), _ptr(kept), _ptr(info), _ptr(ws), ws.numel(), _stream()),
           "lrc_allocate_ranks")
    return order, n_kept, ranks, kept, info


def lrc_rank_scores(sigma: torch.Tensor, offsets: torch.Tensor, weight: torch.Tensor, mode: str = "unirank",
                    alpha: float = 0.5):
    """Alternative component scores from singular values.  sigma: (M,) fp32, matrices
    concatenated per offsets ((n_mat+1,) int64); weight: (n_mat,) fp32 -- the layer
    importance I_l (mode "unirank") or beta_l (mode "swift", with alpha).

    Returns (scores fp32 (M,), info int32 (1,))."""
    _dev(sigma, "sigma")
    dev = sigma.device
    n_mat = weight.numel() if isinstance(weight, torch.Tensor) else 0
    _tensor(sigma, "sigma", torch.float32, (None,), dev)
    _tensor(offsets, "offsets", torch.int64, (n_mat + 1,), dev)
    _tensor(weight, "weight", torch.float32, (n_mat,), dev)
    flag = {"unirank": LRC_RANKSCORE_UNIRANK, "swift": LRC_RANKSCORE_SWIFT}[mode]
    M = sigma.numel()
    sig, offs, wgt = sigma.contiguous(), offsets.contiguous(), weight.contiguous()
    scores = torch.empty(M, dtype=torch.float32, device=dev)
    info = torch.empty(1, dtype=torch.int32, device=dev)
    _check(lib.lrc_rank_scores(_ptr(sig), _ptr(offs), n_mat, M, _ptr(wgt), float(alpha), flag, _ptr(scores),
                               _ptr(info), _stream()), "lrc_rank_scores")
    return scores, info


def lrc_rotate_quantize(left: torch.Tensor, right: torch.Tensor, signs: torch.Tensor, keep_rotated: bool = False):
    """Rotate the factors by a sign-randomised Hadamard matrix and quantise each row to
    int8.  left: (d_out, r) fp32, right: (r, d_in) fp32, signs: (r,) fp32 of +-1.

    Returns (q_left int8, s_left fp32, q_right int8, s_right fp32) and, with
    keep_rotated, the rotated fp32 factors as two more entries."""
    _dev(left, "left")
    if left.dim() != 2:
        raise ValueError("left must be (d_out, r)")
    d_out, r = left.shape
    dev = left.device
    _tensor(left, "left", torch.float32, (d_out, r), dev)
    _tensor(right, "right", torch.float32, (r, None), dev)
    _tensor(signs, "signs", torch.float32, (r,), dev)
    d_in = right.shape[1]
    lf, rt, sg = left.contiguous(), right.contiguous(), signs.contiguous()
    ql = torch.empty(d_out, r, dtype=torch.int8, device=dev)
    sl = torch.empty(d_out, dtype=torch.float32, device=dev)
    qr = torch.empty(r, d_in, dtype=torch.int8, device=dev)
    sr = torch.empty(r, dtype=torch.float32, device=dev)
    lrot = torch.empty(d_out, r, dtype=torch.float32, device=dev) if keep_rotated else None
    rrot = torch.empty(r, d_in, dtype=torch.float32, device=dev) if keep_rotated else None
    ws = _workspace(lib.lrc_rotate_quantize_workspace(d_out, r, d_in), dev)
    _check(lib.lrc_rotate_quantize(_ptr(lf), _ptr(rt), d_out, r, d_in, _ptr(sg), _ptr(ql), _ptr(sl), _ptr(qr), _ptr(sr),
                                   _ptr(lrot) if keep_rotated else None, _ptr(rrot) if keep_rotated else None,
                                   _ptr(ws), ws.numel(), _stream()), "lrc_rotate_quantize")
    return (ql, sl, qr, sr, lrot, rrot) if keep_rotated else (ql, sl, qr, sr)


def lrc_quantize_rows(x: torch.Tensor):
    """Per-row int8 RTN of an fp32 matrix (rows, cols).  Returns (q int8, scale fp32 (rows,))."""
    _dev(x, "x")
    if x.dtype != torch.float32 or x.dim() != 2:
        raise ValueError("x must be a 2-D fp32 tensor")
    x = x.contiguous()
    rows, cols = x.shape
    q = torch.empty(rows, cols, dtype=torch.int8, device=x.device)
    s = torch.empty(rows, dtype=torch.float32, device=x.device)
    _check(lib.lrc_quantize_rows(_ptr(x), rows, cols, cols, _ptr(q), _ptr(s), _stream()), "lrc_quantize_rows")
    return q, s


def lrc_ffn_select_channels(w_gate: torch.Tensor, w_up: torch.Tensor, gate_factors, up_factors,
                            Xsum: torch.Tensor, n_x: int, n_lowrank: int, damping: float = 0.0):
    """Hidden-channel selection of an FFN's hybrid low-rank form.  w_gate, w_up: (d_ff, d)
    fp32; gate_factors, up_factors: (left (d_ff, r), right (r, d)) fp32 from
    lrc_whiten_decompose with the same Xsum (or None for r = 0); Xsum: (d, d) fp32 sum.

    Returns (err fp64 (d_ff,), order int32 (d_ff,), lowrank uint8 (d_ff,), info int32 (1,))."""
    _dev(w_gate, "w_gate")
    if w_gate.dim() != 2:
        raise ValueError("w_gate must be (d_ff, d)")
    d_ff, d = w_gate.shape
    dev = w_gate.device
    _tensor(w_gate, "w_gate", torch.float32, (d_ff, d), dev)
    _tensor(w_up, "w_up", torch.float32, (d_ff, d), dev)
    _tensor(Xsum, "Xsum", torch.float32, (d, d), dev)
    wg, wu = w_gate.contiguous(), w_up.contiguous()
    r = 0
    fac = []
    if gate_factors is not None or up_factors is not None:
        for pair, nm in ((gate_factors, "gate"), (up_factors, "up")):
            if pair is None:
                raise ValueError("give the factors of both gate and up, or of neither")
            left, right = pair
            _tensor(left, f"{nm} left", torch.float32, (d_ff, None), dev)
            _tensor(right, f"{nm} right", torch.float32, (None, d), dev)
            fac += [left.contiguous(), right.contiguous()]
        r = fac[0].shape[1]
        if any(tuple(f.shape) != shp for f, shp in zip(fac, [(d_ff, r), (r, d)] * 2)):
            raise ValueError("factors must be left (d_ff, r) and right (r, d) for both")
    err = torch.empty(d_ff, dtype=torch.float64, device=dev)
    order = torch.empty(d_ff, dtype=torch.int32, device=dev)
    lowrank = torch.empty(d_ff, dtype=torch.uint8, device=dev)
    info = torch.empty(1, dtype=torch.int32, device=dev)
    ws = _workspace(lib.lrc_ffn_select_channels_workspace(d_ff, d), dev)
    ptrs = [_ptr(f) for f in fac] if r > 0 else [None] * 4
    _check(lib.lrc_ffn_select_channels(_ptr(wg), _ptr(wu), d_ff, d, d, ptrs[0], ptrs[1], ptrs[2], ptrs[3], r,
                                       _ptr(Xsum), _rowmajor_ld(Xsum, "Xsum"), int(n_x), float(damping),
                                       int(n_lowrank), _ptr(err), _ptr(order), _ptr(lowrank), _ptr(info), _ptr(ws),
                                       ws.numel(), _stream()), "lrc_ffn_select_channels")
    return err, order, lowrank, info


def _lowrank_factors(gate, up, down, d, dev):
    """Check the int8 factor sets of a low-rank FFN (shapes, dtypes, device) and return
    contiguous copies plus (d_ff, rg, ru, rd)."""
    i8, f32 = torch.int8, torch.float32
    for t in [*gate, *up, *down]:
        _dev(t, "ffn factor")
    if len(gate) != 4 or len(up) != 4 or len(down) != 4:
        raise ValueError("gate, up and down are 4-tuples (q_R, s_R, q_L, s_L)")
    rg, ru = gate[0].shape[0], up[0].shape[0]
    d_ff = gate[2].shape[0]
    rd = down[0].shape[1]
    for (q_r, s_r, q_l, s_l), r, nm in ((gate, rg, "gate"), (up, ru, "up")):
        _tensor(q_r, f"{nm} q_R", i8, (r, d), dev)
        _tensor(s_r, f"{nm} s_R", f32, (r,), dev)
        _tensor(q_l, f"{nm} q_L", i8, (d_ff, r), dev)
        _tensor(s_l, f"{nm} s_L", f32, (d_ff,), dev)
    _tensor(down[0], "down q_Rt", i8, (d_ff, rd), dev)
    _tensor(down[1], "down s_R", f32, (rd,), dev)
    _tensor(down[2], "down q_L", i8, (d, rd), dev)
    _tensor(down[3], "down s_L", f32, (d,), dev)
    return ([t.contiguous() for t in gate], [t.contiguous() for t in up], [t.contiguous() for t in down],
            d_ff, rg, ru, rd)


def lrc_hybrid_ffn(x: torch.Tensor, gate=None, up=None, down=None, dense=None):
    """Hybrid FFN forward: hidden channels [0, n_lr) low-rank (gate, up, down as for
    lrc_lowrank_ffn, or all None when n_lr = 0), the next n_dense dense:
    dense = (q_gd (n_dense, d) int8, s_gd (n_dense,), q_ud, s_ud, q_dd (d, n_dense) int8 --
    W_down's dense columns as rows, s_dd (d,)), or None when n_dense = 0.
    Returns y (n_tok, d) fp32."""
    _dev(x, "x")
    if x.dtype != torch.float32 or x.dim() != 2:
        raise ValueError("x must be (n_tok, d) fp32")
    n_tok, d = x.shape
    dev = x.device
    xc = x.contiguous()
    lr = gate is not None
    if lr != (up is not None) or lr != (down is not None):
        raise ValueError("give gate, up and down together, or none of them")
    if lr:
        g, u, dn, n_lr, rg, ru, rd = _lowrank_factors(gate, up, down, d, dev)
    else:
        g = u = dn = [None] * 4
        rg = ru = rd = n_lr = 0
    if dense is not None:
        if len(dense) != 6:
            raise ValueError("dense is a 6-tuple (q_gd, s_gd, q_ud, s_ud, q_dd, s_dd)")
        _dev(dense[0], "q_gd")
        n_dense = dense[0].shape[0]
        for t, nm, dt, shp in zip(dense, ("q_gd", "s_gd", "q_ud", "s_ud", "q_dd", "s_dd"),
                                  (torch.int8, torch.float32) * 3,
                                  ((n_dense, d), (n_dense,), (n_dense, d), (n_dense,), (d, n_dense), (d,))):
            _tensor(t, nm, dt, shp, dev)
        dd = [t.contiguous() for t in dense]
    else:
        dd = [None] * 6
        n_dense = 0
    y = torch.empty(n_tok, d, dtype=torch.float32, device=dev)
    ws = _workspace(lib.lrc_hybrid_ffn_workspace(n_tok, n_lr, rg, ru, rd, n_dense), dev)
    p = lambda t: None if t is None else _ptr(t)
    _check(lib.lrc_hybrid_ffn(_ptr(xc), n_tok, d, n_lr, p(g[0]), p(g[1]), p(g[2]), p(g[3]), rg, p(u[0]), p(u[1]),
                              p(u[2]), p(u[3]), ru, p(dn[0]), p(dn[1]), p(dn[2]), p(dn[3]), rd, n_dense, p(dd[0]),
                              p(dd[1]), p(dd[2]), p(dd[3]), p(dd[4]), p(dd[5]), _ptr(y), _ptr(ws), ws.numel(),
                              _stream()), "lrc_hybrid_ffn")
    return y


def lrc_lowrank_ffn(x: torch.Tensor, gate, up, down):
    """Low-rank SwiGLU FFN forward with int8 factors.  x: (n_tok, d) fp32.
    gate, up: (q_R (r, d) int8, s_R (r,), q_L (d_ff, r) int8, s_L (d_ff,)).
    down: (q_Rt (d_ff, r_d) int8 -- R_down transposed, s_R (r_d,), q_L (d, r_d) int8, s_L (d,)).
    Returns y (n_tok, d) fp32."""
    _dev(x, "x")
    if x.dtype != torch.float32 or x.dim() != 2:
        raise ValueError("x must be (n_tok, d) fp32")
    n_tok, d = x.shape
    dev = x.device
    xc = x.contiguous()
    g, u, dn, d_ff, rg, ru, rd = _lowrank_factors(gate, up, down, d, dev)
    y = torch.empty(n_tok, d, dtype=torch.float32, device=dev)
    ws = _workspace(lib.lrc_lowrank_ffn_workspace(n_tok, d_ff, rg, ru, rd), dev)
    _check(lib.lrc_lowrank_ffn(_ptr(xc), n_tok, d, d_ff, _ptr(g[0]), _ptr(g[1]), _ptr(g[2]), _ptr(g[3]), rg,
                               _ptr(u[0]), _ptr(u[1]), _ptr(u[2]), _ptr(u[3]), ru, _ptr(dn[0]), _ptr(dn[1]),
                               _ptr(dn[2]), _ptr(dn[3]), rd, _ptr(y), _ptr(ws), ws.numel(), _stream()),
           "lrc_lowrank_ffn")
    return y


def _run(where, device, fn, *args):
    """Call fn(*args, stream) with `device` current, on its current stream (a launch needs its
    stream's device current), and turn a failure into an exception."""
    if device.index == torch.cuda.current_device():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    if st != LRC_OK:
        raise LrcError(st, where)


def _rows(t, name, n=None, d=None, dtype=None, device=None):
    """Check a 2-D GPU tensor (its dtype, its device and, where given, its n rows and d columns)
    and return (tensor, leading dim); rows that are not contiguous or overlap are copied."""
    _dev(t, name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {t.dim()}")
    rows, cols = t.shape
    if (n is not None and rows != n) or (d is not None and cols != d):
        raise ValueError(f"{name} must have shape {(n, d)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    s0, s1 = t.stride()
    if rows <= 1 or cols == 0:
        return t if s1 == 1 or cols <= 1 else t.contiguous(), max(cols, 1)
    if (cols > 1 and s1 != 1) or s0 < cols:
        return t.contiguous(), cols
    return t, s0


def _pieces(t, ld, work):
    """(tensor, leading dim) of an operand of a product of `work` multiplications, its rows whole
    aligned 16-byte pieces.  A bf16 operand whose rows could be such pieces but do not start on 16
    bytes keeps the product off the direct loads; from 2^30 multiplications on a copy costs less
    (2048 x 4096 x 4096 373 us against 74 with the copy, 65 x 4096 x 4096 35 against 22; below, 256
    x 1024 x 1024 17 against 22)."""
    if (t is None or t.dtype != torch.bfloat16 or work < 1 << 30 or t.shape[1] % 8
            or (t.data_ptr() % 16 == 0 and ld % 8 == 0)):
        return t, ld
    return t.clone(memory_format=torch.contiguous_format), t.shape[1]


def _vector(t, name, n, device):
    if t is None:
        return None
    _dev(t, name)
    if t.dtype != torch.float32 or t.dim() != 1 or t.shape[0] != n or t.device != device:
        raise ValueError(f"{name} must be fp32 of shape ({n},) on {device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.contiguous()


def _checkpoint(ck, name, n, d, device):
    """Check a (codes, exps) pair of n rows of d channels."""
    if len(ck) != 2:
        raise ValueError(f"{name} must be a tensor or a (codes, exps) pair")
    codes, ldc = _rows(ck[0], f"{name} codes", n, d, torch.int8, device)
    blocks = -(-d // LRC_CKPT_BLOCK)
    exps, lde = _rows(ck[1], f"{name} exps", n, blocks, torch.int8, device)
    return codes if ldc == max(d, 1) else codes.contiguous(), exps if lde == max(blocks, 1) else exps.contiguous()


def _kept(t, name, n, d, dtype, device):
    """(tensor, leading dim, codes, exps) of an activation given in full or as a checkpoint."""
    if t is None:
        return None, max(d, 1), None, None
    if isinstance(t, (tuple, list)):
        codes, exps = _checkpoint(t, name, n, d, device)
        return None, max(d, 1), codes, exps
    t, ld = _rows(t, name, n, d, dtype, device)
    return t, ld, None, None


def _new_checkpoint(n, d, device):
    return (torch.empty(n, d, dtype=torch.int8, device=device),
            torch.empty(n, -(-d // LRC_CKPT_BLOCK), dtype=torch.int8, device=device))


def lrc_pack_activations(x: torch.Tensor, info=None):
    """8-bit checkpoint of token rows.  x: (n_tokens, d) bf16 or fp32.

    Returns (codes int8 (n_tokens, d), exps int8 (n_tokens, ceil(d / 64)), info int32 (1,)):
    the values held are codes * 2^exps per 64 channels.  info (sticky, optional) receives
    LRC_ENONFINITE when an entry is NaN or Inf."""
    x, ldx = _rows(x, "x")
    dt, dev = _dtype_code(x), x.device
    n, d = x.shape
    codes, exps = _new_checkpoint(n, d, dev)
    info = _info(info, dev)
    _run("lrc_pack_activations", dev, lib.lrc_pack_activations, _ptr(x), dt, n, d, ldx, _ptr(codes), _ptr(exps),
         _ptr(info))
    return codes, exps, info


def lrc_unpack_activations(codes: torch.Tensor, exps: torch.Tensor, dtype=torch.bfloat16):
    """The values an 8-bit checkpoint holds, as bf16 or fp32 (both exact)."""
    _dev(codes, "codes")
    if codes.dim() != 2:
        raise ValueError("codes must be (n_tokens, d)")
    n, d = codes.shape
    dev = codes.device
    codes, exps = _checkpoint((codes, exps), "checkpoint", n, d, dev)
    x = torch.empty(n, d, dtype=dtype, device=dev)
    _run("lrc_unpack_activations", dev, lib.lrc_unpack_activations, _ptr(codes), _ptr(exps), n, d, _ptr(x),
         _dtype_code(x), max(d, 1))
    return x


def lrc_layer_norm(x: torch.Tensor, gamma=None, beta=None, eps: float = 1e-5, checkpoint: bool = False, info=None):
    """Layer norm of token rows.  x: (n_tokens, d) bf16 or fp32; gamma, beta: (d,) fp32 or None.

    Returns (y, mean, rstd, kept, info): y like x, mean and rstd fp32 (n_tokens,), kept the
    (codes, exps) checkpoint of x when `checkpoint` (else None, and info None unless given)."""
    x, ldx = _rows(x, "x")
    dt, dev = _dtype_code(x), x.device
    n, d = x.shape
    gamma, beta = _vector(gamma, "gamma", d, dev), _vector(beta, "beta", d, dev)
    y = torch.empty(n, d, dtype=x.dtype, device=dev)
    mean = torch.empty(n, dtype=torch.float32, device=dev)
    rstd = torch.empty(n, dtype=torch.float32, device=dev)
    kept = _new_checkpoint(n, d, dev) if checkpoint else None
    if checkpoint or info is not None:
        info = _info(info, dev)
    codes, exps = kept or (None, None)
    _run("lrc_layer_norm", dev, lib.lrc_layer_norm, _ptr(x), dt, n, d, ldx, _ptr(gamma), _ptr(beta), float(eps),
         _ptr(y), max(d, 1), _ptr(mean), _ptr(rstd), _ptr(codes), _ptr(exps), _ptr(info))
    return y, mean, rstd, kept, info


def lrc_layer_norm_backward(dy: torch.Tensor, x, mean: torch.Tensor, rstd: torch.Tensor, gamma=None,
                            need_dx: bool = True, need_dparams: bool = True):
    """Gradients of lrc_layer_norm.  dy: (n_tokens, d); x: the input like dy, or its
    (codes, exps) checkpoint; mean, rstd: (n_tokens,) fp32 as lrc_layer_norm returned them.

    Returns (dx like dy, dgamma fp32 (d,), dbeta fp32 (d,)), None where not needed."""
    dy, lddy = _rows(dy, "dy")
    dt, dev = _dtype_code(dy), dy.device
    n, d = dy.shape
    if x is None:
        raise ValueError("x must be a tensor or a (codes, exps) pair")
    xt, ldx, codes, exps = _kept(x, "x", n, d, dy.dtype, dev)
    mean, rstd = _vector(mean, "mean", n, dev), _vector(rstd, "rstd", n, dev)
    gamma = _vector(gamma, "gamma", d, dev)
    dx = torch.empty(n, d, dtype=dy.dtype, device=dev) if need_dx else None
    dgamma = torch.empty(d, dtype=torch.float32, device=dev) if need_dparams else None
    dbeta = torch.empty(d, dtype=torch.float32, device=dev) if need_dparams else None
    ws = _workspace(lib.lrc_layer_norm_backward_workspace(n, d), dev)
    _run("lrc_layer_norm_backward", dev, lib.lrc_layer_norm_backward, _ptr(dy), dt, n, d, lddy, _ptr(xt), ldx,
         _ptr(codes), _ptr(exps), _ptr(mean), _ptr(rstd), _ptr(gamma), _ptr(dx), max(d, 1), _ptr(dgamma), _ptr(dbeta),
         _ptr(ws), ws.numel())
    return dx, dgamma, dbeta


def _act_code(act):
    if act not in _ACTS:
        raise ValueError(f"act is one of {', '.join(_ACTS)}")
    return _ACTS[act]


def lrc_linear(x: torch.Tensor, W: torch.Tensor, bias=None, act: str = "none", residual=None, save: str = "none",
               info=None):
    """y = act(x W^T + bias) + residual.  x: (n_tokens, d_in), W: (d_out, d_in), residual:
    (n_tokens, d_out), all bf16 or all fp32; bias: (d_out,) fp32; act: none, relu, gelu
    (exact) or silu.  save keeps the pre-activation z = x W^T + bias for the backward pass:
    "z" in full, "checkpoint" in 8 bits, "none" not at all.

    Returns (y, saved, info): saved is z, (codes, exps) or None; info (int32 (1,), sticky
    LRC_ENONFINITE) is None unless given or save is "checkpoint"."""
    x, ldx = _rows(x, "x")
    dt, dev = _dtype_code(x), x.device
    n, d_in = x.shape
    W, ldw = _rows(W, "W", None, d_in, x.dtype, dev)
    d_out = W.shape[0]
    if n > 64:
        (x, ldx), (W, ldw) = _pieces(x, ldx, n * d_in * d_out), _pieces(W, ldw, n * d_in * d_out)
    code = _act_code(act)
    bias = _vector(bias, "bias", d_out, dev)
    ldr = d_out
    if residual is not None:
        residual, ldr = _rows(residual, "residual", n, d_out, x.dtype, dev)
    y = torch.empty(n, d_out, dtype=x.dtype, device=dev)
    z, codes, exps = None, None, None
    if save == "z":
        z = torch.empty(n, d_out, dtype=x.dtype, device=dev)
    elif save == "checkpoint":
        codes, exps = _new_checkpoint(n, d_out, dev)
    elif save != "none":
        raise ValueError("save is none, z or checkpoint")
    if codes is not None or info is not None:
        info = _info(info, dev)
    ws = _workspace(lib.lrc_linear_workspace(dt, n, d_in, d_out), dev)
    _run("lrc_linear", dev, lib.lrc_linear, _ptr(x), dt, n, d_in, d_out, ldx, _ptr(W), ldw, _ptr(bias), code,
         _ptr(residual), ldr, _ptr(y), max(d_out, 1), _ptr(z), max(d_out, 1), _ptr(codes), _ptr(exps), _ptr(info),
         _ptr(ws), ws.numel())
    return y, (codes, exps) if codes is not None else z, info


def lrc_linear_backward(dy: torch.Tensor, x, W: torch.Tensor, act: str = "none", z=None, need_dx: bool = True,
                        need_dw: bool = True, need_db: bool = True, dw_dtype=None):
    """Gradients of lrc_linear.  dy: (n_tokens, d_out); x: the input (n_tokens, d_in) like dy,
    or its (codes, exps) checkpoint (may be None without need_dw); W: (d_out, d_in); z: the
    pre-activation like dy or its (codes, exps) checkpoint (needed unless act is none).

    Returns (dz, dx, dW, db): dz = dy * act'(z), the layer's output-gradient stream (dy itself
    for act none), dx (n_tokens, d_in), dW (d_out, d_in) in dw_dtype (default dy's; torch.float32
    allowed), db fp32 (d_out,); None where not needed."""
    dy, lddy = _rows(dy, "dy")
    dt, dev = _dtype_code(dy), dy.device
    n, d_out = dy.shape
    W, ldw = _rows(W, "W", d_out, None, dy.dtype, dev)
    d_in = W.shape[1]
    code = _act_code(act)
    if need_dw and x is None:
        raise ValueError("dW needs x or its checkpoint")
    if code and z is None:
        raise ValueError("the gradient of an activation needs z or its checkpoint")
    xt, ldx, xcodes, xexps = _kept(x if need_dw else None, "x", n, d_in, dy.dtype, dev)
    zt, ldz, zcodes, zexps = _kept(z if code else None, "z", n, d_out, dy.dtype, dev)
    g = dy   # the output gradient as the kernels read it
    if n > 64:
        work = n * d_in * d_out
        (xt, ldx), (W, ldw) = _pieces(xt, ldx, work), _pieces(W, ldw, work if need_dx else 0)
        if not code:
            g, lddy = _pieces(dy, lddy, work)
    dw_dtype = dw_dtype or dy.dtype
    if dw_dtype not in (dy.dtype, torch.float32):
        raise ValueError("dw_dtype is dy's dtype or torch.float32")
    dz = torch.empty(n, d_out, dtype=dy.dtype, device=dev) if code else None
    dx = torch.empty(n, d_in, dtype=dy.dtype, device=dev) if need_dx else None
    dW = torch.empty(d_out, d_in, dtype=dw_dtype, device=dev) if need_dw else None
    db = torch.empty(d_out, dtype=torch.float32, device=dev) if need_db else None
    dw_dt = LRC_F32 if dw_dtype == torch.float32 else LRC_BF16
    ws = _workspace(lib.lrc_linear_backward_workspace(dt, n, d_in, d_out), dev)
    _run("lrc_linear_backward", dev, lib.lrc_linear_backward, _ptr(g), dt, n, d_in, d_out, lddy, _ptr(W), ldw,
         _ptr(xt), ldx, _ptr(xcodes), _ptr(xexps), code, _ptr(zt), ldz, _ptr(zcodes), _ptr(zexps), _ptr(dz),
         max(d_out, 1), _ptr(dx), max(d_in, 1), _ptr(dW), dw_dt, max(d_in, 1), _ptr(db), _ptr(ws), ws.numel())
    return dz if code else dy, dx, dW, db


def lrc_profile_start() -> None:
    """Start recording HIP events around every instrumented kernel launch (clears totals)."""
    _check(lib.lrc_profile_start(), "lrc_profile_start")


def lrc_profile_stop() -> None:
    """Stop recording; waits for the recorded events and folds their times into the totals."""
    _check(lib.lrc_profile_stop(), "lrc_profile_stop")


def lrc_profile_kernels() -> dict:
    """Totals per kernel name since the last start: launches, total_ms, flops, bytes."""
    out = {}
    for i in range(lib.lrc_profile_kernels()):
        name = ctypes.c_char_p()
        launches = _i64()
        ms, fl, by = ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
        _check(lib.lrc_profile_kernel(i, ctypes.byref(name), ctypes.byref(launches), ctypes.byref(ms),
                                      ctypes.byref(fl), ctypes.byref(by)), "lrc_profile_kernel")
        out[name.value.decode()] = {"launches": launches.value, "total_ms": ms.value, "flops": fl.value,
                                    "bytes": by.value}
    return out
