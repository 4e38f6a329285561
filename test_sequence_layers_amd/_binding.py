"""ctypes binding of libttt.so.

Argument marshalling only: every step of the forward pass runs in the library's HIP
kernels.  PyTorch supplies device memory and the current stream.  There is no CPU
fallback; if the library is missing every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libttt.so")

TTT_OK, TTT_E_INVALID, TTT_E_UNSUPPORTED, TTT_E_HIP, TTT_E_NONFINITE = 0, -1, -2, -3, -4
TTT_F32, TTT_BF16 = 0, 1

_lib = None
_lock = threading.Lock()

_vp = ctypes.c_void_p
_i = ctypes.c_int
_ll = ctypes.c_longlong
_f = ctypes.c_float

# name -> (restype, argtypes); mirrors include/ttt.h
SIGNATURES = {
    "ttt_linear_fwd": (_i, [_vp, _vp, _vp, _vp, _ll, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _i,
                            _i, _i, _vp]),
    "ttt_mlp_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _ll, _vp, _vp, _vp,
                         _i, _i, _i, _i, _i, _i, _i, _f, _vp, _i, _i, _i, _vp]),
    "ttt_linear_ln_fwd": (_i, [_vp, _vp, _vp, _vp, _ll, _vp, _vp, _f, _vp, _vp, _i, _i, _i, _i, _i,
                               _i, _f, _vp, _i, _i, _i, _vp]),
    "ttt_mlp_ln_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _ll, _vp, _vp, _f, _vp, _vp, _vp,
                            _i, _i, _i, _i, _i, _i, _i, _f, _vp, _i, _i, _i, _vp]),
    "ttt_mlp_fwd_workspace_size": (ctypes.c_size_t, [_i, _i, _i, _i, _i, _i, _i, _i]),
    "ttt_mlp_fwd_ws": (_i, [_vp, _vp, _vp, _vp, _vp, _ll, _vp, _vp, _vp,
                            _i, _i, _i, _i, _i, _i, _i, _f, _vp, _i, _i, _i,
                            _vp, ctypes.c_size_t, _vp]),
    "ttt_mlp_ln_fwd_ws": (_i, [_vp, _vp, _vp, _vp, _vp, _ll, _vp, _vp, _f, _vp, _vp, _vp,
                               _i, _i, _i, _i, _i, _i, _i, _f, _vp, _i, _i, _i,
                               _vp, ctypes.c_size_t, _vp]),
    "delta_rule_fwd": (_i, [_vp, _vp, _vp, _vp, _ll, _vp, _vp, _i, _i, _i, _i, _f, _vp, _i, _vp]),
    "ttt_linear_bwd": (_i, [_vp, _vp, _vp, _vp, _ll, _vp, _vp, _vp, _vp, _vp, _vp,
                            _i, _i, _i, _i, _i, _f, _vp, _vp, _i, _i, _vp]),
    "ttt_linear_bwd_noalloc": (_i, [_vp, _vp, _vp, _vp, _ll, _vp, _vp, _vp, _vp, _vp, _vp,
                                    _i, _i, _i, _i, _i, _f, _vp, _vp, _i, _i, _vp]),
    "ttt_mlp_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _ll, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                         _i, _i, _i, _i, _i, _i, _f, _vp, _vp, _i, _i, _vp]),
    "ttt_linear_ln_bwd": (_i, [_vp, _vp, _vp, _vp, _ll, _vp, _vp, _f, _vp, _vp, _vp, _vp, _vp, _vp,
                               _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp, _i, _i, _vp]),
    "ttt_mlp_ln_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _ll, _vp, _vp, _f, _vp, _vp, _vp, _vp, _vp, _vp,
                            _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _vp, _i, _i, _vp]),
    "ttt_linear_nc_bwd": (_i, [_vp, _vp, _vp, _vp, _ll, _vp, _vp, _vp, _vp, _vp, _vp,
                               _i, _i, _i, _i, _i, _i, _f, _vp, _vp, _i, _i, _vp]),
    "ttt_mlp_nc_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _ll, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                            _i, _i, _i, _i, _i, _i, _i, _f, _vp, _vp, _i, _i, _vp]),
    "gated_linear_fwd_workspace_size": (ctypes.c_size_t, [_i, _i, _i, _i, _i]),
    "gated_linear_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _ll, _vp, _vp, _vp, _i, _i, _i, _i, _f, _vp, _i,
                              _vp, ctypes.c_size_t, _vp]),
    "gated_linear_bwd_workspace_size": (ctypes.c_size_t, [_i, _i, _i, _i, _i, _i]),
    "gated_linear_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _ll, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                              _i, _i, _i, _i, _f, _vp, _vp, _i, _vp, ctypes.c_size_t, _vp]),
    "gated_linear_step": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _f, _vp, _i, _vp]),
    "token_norm_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp]),
    "token_norm_bwd_workspace_size": (ctypes.c_size_t, [_i, _i, _i, _i]),
    "token_norm_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                            _i, _i, _i, _i, _i, _i, _f, _i, _vp, ctypes.c_size_t, _vp]),
    "ttt_last_error": (ctypes.c_char_p, []),
    "ttt_abi_version": (_i, []),
    "ttt_set_check_finite": (_i, [_i]),
    "ttt_get_check_finite": (_i, []),
    "ttt_set_split_debug": (_i, [_i]),
}


class TTTError(RuntimeError):
    def __init__(self, code, message):
        super().__init__(f"libttt error {code}: {message}")
        self.code = code


def load_library(path: str = LIB_PATH):
    """Load libttt.so once (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m test_sequence_layers_amd.build`")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def last_error() -> str:
    return load_library().ttt_last_error().decode()


def set_check_finite(on: bool) -> bool:
    """Switch the library's finite check of every call's outputs on or off (debugging; calls
    then wait for their stream and fail with TTT_E_NONFINITE on a NaN or an infinity).
    Returns the previous setting."""
    return bool(load_library().ttt_set_check_finite(1 if on else 0))


def set_split_debug(flags: int) -> int:
    """Debug switches of the two-workgroup MLP kernel (TTT_SPLIT_FORMAL = 1,
    TTT_SPLIT_TEST_ABORT = 2); returns the previous flags."""
    return int(load_library().ttt_set_split_debug(int(flags)))


def get_check_finite() -> bool:
    return bool(load_library().ttt_get_check_finite())


def _check(rc):
    if rc != TTT_OK:
        raise TTTError(rc, last_error())


# --------------------------------------------------------------------------- torch wrappers

def _torch():
    import torch
    return torch


def _io_dtype(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return TTT_F32
    if t.dtype == torch.bfloat16:
        return TTT_BF16
    raise TypeError(f"token tensors must be float32 or bfloat16, got {t.dtype}")


def _tokens(q, k, v):
    torch = _torch()
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{name} must be a [B, H, T, d] tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be on a GPU")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if not (q.shape == k.shape == v.shape):
        raise ValueError("q, k and v must have the same shape")
    if not (q.dtype == k.dtype == v.dtype):
        raise ValueError("q, k and v must have the same dtype")
    if not (q.device == k.device == v.device):
        raise ValueError("q, k and v must be on the same device")
    return tuple(q.shape)


def _state(w, B, H, shape, name, device):
    """Return (tensor, batch_stride_in_floats) for an initial state [H,...] or [B,H,...]."""
    torch = _torch()
    if not isinstance(w, torch.Tensor) or w.dtype != torch.float32 or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor")
    if w.device != device:
        raise ValueError(f"{name} must be on {device}")
    per = 1
    for s in shape:
        per *= s
    if tuple(w.shape) == (H, *shape):
        return w, 0
    if tuple(w.shape) == (B, H, *shape):
        return w, H * per
    raise ValueError(f"{name} must have shape [H, {shape}] or [B, H, {shape}], got {tuple(w.shape)}")


def _rates(eta_tok, B, H, T, device):
    """Device pointer of optional per-token rate factors [B, H, T] float32 (None -> NULL)."""
    torch = _torch()
    if eta_tok is None:
        return None
    if (not isinstance(eta_tok, torch.Tensor) or eta_tok.dtype != torch.float32
            or not eta_tok.is_contiguous() or tuple(eta_tok.shape) != (B, H, T)
            or eta_tok.device != device):
        raise ValueError(f"eta_tok must be a contiguous float32 tensor of shape {(B, H, T)} on {device}")
    return eta_tok.data_ptr()


_LOSSES = {"mse": 0, "dot": 1}


def _loss(loss):
    if loss not in _LOSSES:
        raise ValueError(f"loss must be one of {sorted(_LOSSES)}, got {loss!r}")
    return _LOSSES[loss]


def _stream(device, stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _out(t, shape, dtype, device, name):
    torch = _torch()
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    return t


def _ln(ln_weight, ln_bias, ln_eps, H, d, device):
    """Pointers of the per-head layer-norm gain and bias ([H, d] float32 each)."""
    torch = _torch()
    for name, t in (("ln_weight", ln_weight), ("ln_bias", ln_bias)):
        if (not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or not t.is_contiguous()
                or tuple(t.shape) != (H, d) or t.device != device):
            raise ValueError(f"{name} must be a contiguous float32 tensor [H, d] = [{H}, {d}] on {device}")
    return ln_weight.data_ptr(), ln_bias.data_ptr(), float(ln_eps)


def _linear(q, k, v, w0, eta, chunk, causal, ln, eta_tok, loss, epochs, z, w_out, return_state,
            stream):
    torch = _torch()
    lib = load_library()
    B, H, T, d = _tokens(q, k, v)
    w0, stride = _state(w0, B, H, (d, d), "w0", q.device)
    z = _out(z, (B, H, T, d), q.dtype, q.device, "z")
    if return_state or w_out is not None:
        w_out = _out(w_out, (B, H, d, d), torch.float32, q.device, "w_out")
    tail = (z.data_ptr(), w_out.data_ptr() if w_out is not None else None,
            B, H, T, d, int(chunk), int(bool(causal)), float(eta),
            _rates(eta_tok, B, H, T, q.device), _loss(loss), int(epochs),
            _io_dtype(q), _stream(q.device, stream))
    with torch.cuda.device(q.device):
        if ln is None:
            rc = lib.ttt_linear_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), w0.data_ptr(), stride,
                                    *tail)
        else:
            rc = lib.ttt_linear_ln_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), w0.data_ptr(),
                                       stride, *_ln(*ln, H, d, q.device), *tail)
    _check(rc)
    return (z, w_out) if w_out is not None else z


def ttt_linear_fwd(q, k, v, w0, eta, chunk, causal=True, *, eta_tok=None, loss="mse", epochs=1,
                   z=None, w_out=None, return_state=False, stream=None):
    """TTT-Linear forward.  q, k, v [B,H,T,d] (float32 or bfloat16, same device);
    w0 float32 [H,d,d] (shared over the batch) or [B,H,d,d]; eta_tok optional float32
    [B,H,T] per-token rate factors (token t learns at eta * eta_tok[t]); loss "mse"
    (reconstruction) or "dot" (negative dot product); epochs: passes over the chunks
    before the queries are read (non-causal only).  Returns z (and the final state
    [B,H,d,d] when return_state or w_out is given)."""
    return _linear(q, k, v, w0, eta, chunk, causal, None, eta_tok, loss, epochs, z, w_out,
                   return_state, stream)


def ttt_linear_ln_fwd(q, k, v, w0, ln_weight, ln_bias, eta, chunk, causal=True, *, ln_eps=1e-6,
                      eta_tok=None, loss="mse", epochs=1, z=None, w_out=None,
                      return_state=False, stream=None):
    """The paper's TTT-Linear, f(x) = x + LN(W x) with per-head ln_weight, ln_bias float32
    [H, d]; every other argument as ttt_linear_fwd."""
    return _linear(q, k, v, w0, eta, chunk, causal, (ln_weight, ln_bias, ln_eps), eta_tok, loss,
                   epochs, z, w_out, return_state, stream)


def ttt_linear_bwd(q, k, v, w0, eta, chunk, dz, dw_out=None, *, eta_tok=None, loss="mse",
                   stream=None):
    """Gradients of the causal TTT-Linear layer (reconstruction loss) for the upstream
    gradients dz [B,H,T,d] (dtype of q) and dw_out [B,H,d,d] float32 (or None).  Returns
    (dq, dk, dv, dw0) with dw0 [B,H,d,d] per sequence (sum it over the batch when w0 is
    shared); with per-token rate factors eta_tok [B,H,T] float32 (as in ttt_linear_fwd) also
    their gradient, (dq, dk, dv, dw0, deta_tok).  loss: "mse" or "dot", as in the forward."""
    return _linear_bwd("ttt_linear_bwd", q, k, v, w0, eta, chunk, dz, dw_out, eta_tok, loss,
                       stream, None)


def ttt_linear_bwd_noalloc(q, k, v, w0, eta, chunk, dz, dw_out=None, *, eta_tok=None,
                           loss="mse", stream=None, out=None):
    """ttt_linear_bwd through the library's allocation-free entry point: the state history
    lives in the library's fixed 64 MiB scratch array (calls that need more raise).  out:
    optional preallocated (dq, dk, dv, dw0[, deta_tok]) to write into."""
    return _linear_bwd("ttt_linear_bwd_noalloc", q, k, v, w0, eta, chunk, dz, dw_out, eta_tok,
                       loss, stream, out)


def _linear_bwd(fn, q, k, v, w0, eta, chunk, dz, dw_out, eta_tok, loss, stream, out):
    torch = _torch()
    lib = load_library()
    B, H, T, d = _tokens(q, k, v)
    w0, stride = _state(w0, B, H, (d, d), "w0", q.device)
    if (not isinstance(dz, torch.Tensor) or tuple(dz.shape) != (B, H, T, d) or dz.dtype != q.dtype
            or dz.device != q.device or not dz.is_contiguous()):
        raise ValueError(f"dz must be a contiguous {q.dtype} tensor of shape {(B, H, T, d)}")
    if dw_out is not None:
        dw_out = _out(dw_out, (B, H, d, d), torch.float32, q.device, "dw_out")
    et = _rates(eta_tok, B, H, T, q.device)
    if out is not None:
        dq = _out(out[0], (B, H, T, d), q.dtype, q.device, "dq")
        dk = _out(out[1], (B, H, T, d), q.dtype, q.device, "dk")
        dv = _out(out[2], (B, H, T, d), q.dtype, q.device, "dv")
        dw0 = _out(out[3], (B, H, d, d), torch.float32, q.device, "dw0")
        deta = (_out(out[4], (B, H, T), torch.float32, q.device, "deta_tok")
                if et is not None else None)
    else:
        dq = torch.empty_like(q)
        dk = torch.empty_like(q)
        dv = torch.empty_like(q)
        dw0 = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device)
        deta = torch.empty((B, H, T), dtype=torch.float32, device=q.device) if et is not None else None
    with torch.cuda.device(q.device):
        rc = getattr(lib, fn)(q.data_ptr(), k.data_ptr(), v.data_ptr(), w0.data_ptr(), stride,
                              dz.data_ptr(), dw_out.data_ptr() if dw_out is not None else None,
                              dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dw0.data_ptr(),
                              B, H, T, d, int(chunk), float(eta), et,
                              deta.data_ptr() if deta is not None else None, _loss(loss),
                              _io_dtype(q), _stream(q.device, stream))
    _check(rc)
    return (dq, dk, dv, dw0) if deta is None else (dq, dk, dv, dw0, deta)


def ttt_mlp_bwd(q, k, v, w1, w2, eta, chunk, dz, dw1_out=None, dw2_out=None, *, eta_tok=None,
                loss="mse", stream=None):
    """Gradients of the causal TTT-MLP layer (SiLU; loss "mse" or "dot") for the upstream
    gradients dz [B,H,T,d] (dtype of q) and dw1_out [B,H,dh,d], dw2_out [B,H,d,dh] float32 (or
    None).  Returns (dq, dk, dv, dw1, dw2) with the state gradients per sequence (sum them over
    the batch when the states are shared); with per-token rate factors eta_tok [B,H,T] (as in
    ttt_mlp_fwd) also their gradient, (dq, dk, dv, dw1, dw2, deta_tok)."""
    torch = _torch()
    lib = load_library()
    B, H, T, d = _tokens(q, k, v)
    if w1.dim() < 2:
        raise ValueError("w1 must be [H, dh, d] or [B, H, dh, d]")
    dh = int(w1.shape[-2])
    w1, s1 = _state(w1, B, H, (dh, d), "w1", q.device)
    w2, s2 = _state(w2, B, H, (d, dh), "w2", q.device)
    if s1 != s2:
        raise ValueError("w1 and w2 must both be shared over the batch or both per batch")
    if (not isinstance(dz, torch.Tensor) or tuple(dz.shape) != (B, H, T, d) or dz.dtype != q.dtype
            or dz.device != q.device or not dz.is_contiguous()):
        raise ValueError(f"dz must be a contiguous {q.dtype} tensor of shape {(B, H, T, d)}")
    if (dw1_out is None) != (dw2_out is None):
        raise ValueError("give both dw1_out and dw2_out, or neither")
    if dw1_out is not None:
        dw1_out = _out(dw1_out, (B, H, dh, d), torch.float32, q.device, "dw1_out")
        dw2_out = _out(dw2_out, (B, H, d, dh), torch.float32, q.device, "dw2_out")
    et = _rates(eta_tok, B, H, T, q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    dw1 = torch.empty((B, H, dh, d), dtype=torch.float32, device=q.device)
    dw2 = torch.empty((B, H, d, dh), dtype=torch.float32, device=q.device)
    deta = torch.empty((B, H, T), dtype=torch.float32, device=q.device) if et is not None else None
    ptr = lambda t: t.data_ptr() if t is not None else None
    with torch.cuda.device(q.device):
        rc = lib.ttt_mlp_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), w1.data_ptr(), w2.data_ptr(),
                             s1, dz.data_ptr(), ptr(dw1_out), ptr(dw2_out), dq.data_ptr(),
                             dk.data_ptr(), dv.data_ptr(), dw1.data_ptr(), dw2.data_ptr(),
                             B, H, T, d, dh, int(chunk), float(eta), et, ptr(deta), _loss(loss),
                             _io_dtype(q), _stream(q.device, stream))
    _check(rc)
    return (dq, dk, dv, dw1, dw2) if deta is None else (dq, dk, dv, dw1, dw2, deta)


def _dz(dz, q, B, H, T, d):
    torch = _torch()
    if (not isinstance(dz, torch.Tensor) or tuple(dz.shape) != (B, H, T, d) or dz.dtype != q.dtype
            or dz.device != q.device or not dz.is_contiguous()):
        raise ValueError(f"dz must be a contiguous {q.dtype} tensor of shape {(B, H, T, d)}")
    return dz


def ttt_linear_ln_bwd(q, k, v, w0, ln_weight, ln_bias, eta, chunk, dz, dw_out=None, *,
                      ln_eps=1e-6, eta_tok=None, loss="mse", stream=None):
    """Gradients of the paper's causal TTT-Linear layer x + LN(W x) (ttt_linear_ln_fwd with
    the same arguments) for the upstream gradients dz and dw_out.  Returns (dq, dk, dv, dw0,
    dln_weight, dln_bias), plus deta_tok [B,H,T] with eta_tok; dw0 [B,H,d,d] and the layer-norm
    gradients [B,H,d] per sequence."""
    torch = _torch()
    lib = load_library()
    B, H, T, d = _tokens(q, k, v)
    w0, stride = _state(w0, B, H, (d, d), "w0", q.device)
    lw, lb, eps = _ln(ln_weight, ln_bias, ln_eps, H, d, q.device)
    dz = _dz(dz, q, B, H, T, d)
    if dw_out is not None:
        dw_out = _out(dw_out, (B, H, d, d), torch.float32, q.device, "dw_out")
    et = _rates(eta_tok, B, H, T, q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    dw0 = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device)
    dlw = torch.empty((B, H, d), dtype=torch.float32, device=q.device)
    dlb = torch.empty((B, H, d), dtype=torch.float32, device=q.device)
    deta = torch.empty((B, H, T), dtype=torch.float32, device=q.device) if et is not None else None
    ptr = lambda t: t.data_ptr() if t is not None else None
    with torch.cuda.device(q.device):
        rc = lib.ttt_linear_ln_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), w0.data_ptr(), stride,
                                   lw, lb, eps, dz.data_ptr(),
                                   ptr(dw_out), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                   dw0.data_ptr(), dlw.data_ptr(), dlb.data_ptr(), B, H, T, d,
                                   int(chunk), float(eta), et, ptr(deta), _loss(loss), _io_dtype(q),
                                   _stream(q.device, stream))
    _check(rc)
    res = (dq, dk, dv, dw0, dlw, dlb)
    return res if deta is None else res + (deta,)


def ttt_mlp_ln_bwd(q, k, v, w1, w2, ln_weight, ln_bias, eta, chunk, dz, dw1_out=None,
                   dw2_out=None, *, ln_eps=1e-6, eta_tok=None, loss="mse", stream=None):
    """Gradients of the paper's causal TTT-MLP layer x + LN(W2 GELU(W1 x)) (ttt_mlp_ln_fwd
    with the same arguments).  Returns (dq, dk, dv, dw1, dw2, dln_weight, dln_bias), plus
    deta_tok [B,H,T] with eta_tok; state and layer-norm gradients per sequence."""
    torch = _torch()
    lib = load_library()
    B, H, T, d = _tokens(q, k, v)
    if w1.dim() < 2:
        raise ValueError("w1 must be [H, dh, d] or [B, H, dh, d]")
    dh = int(w1.shape[-2])
    w1, s1 = _state(w1, B, H, (dh, d), "w1", q.device)
    w2, s2 = _state(w2, B, H, (d, dh), "w2", q.device)
    if s1 != s2:
        raise ValueError("w1 and w2 must both be shared over the batch or both per batch")
    lw, lb, eps = _ln(ln_weight, ln_bias, ln_eps, H, d, q.device)
    dz = _dz(dz, q, B, H, T, d)
    if (dw1_out is None) != (dw2_out is None):
        raise ValueError("give both dw1_out and dw2_out, or neither")
    if dw1_out is not None:
        dw1_out = _out(dw1_out, (B, H, dh, d), torch.float32, q.device, "dw1_out")
        dw2_out = _out(dw2_out, (B, H, d, dh), torch.float32, q.device, "dw2_out")
    et = _rates(eta_tok, B, H, T, q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    dw1 = torch.empty((B, H, dh, d), dtype=torch.float32, device=q.device)
    dw2 = torch.empty((B, H, d, dh), dtype=torch.float32, device=q.device)
    dlw = torch.empty((B, H, d), dtype=torch.float32, device=q.device)
    dlb = torch.empty((B, H, d), dtype=torch.float32, device=q.device)
    deta = torch.empty((B, H, T), dtype=torch.float32, device=q.device) if et is not None else None
    ptr = lambda t: t.data_ptr() if t is not None else None
    with torch.cuda.device(q.device):
        rc = lib.ttt_mlp_ln_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), w1.data_ptr(),
                                w2.data_ptr(), s1, lw, lb, eps, dz.data_ptr(), ptr(dw1_out),
                                ptr(dw2_out), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                dw1.data_ptr(), dw2.data_ptr(), dlw.data_ptr(), dlb.data_ptr(),
                                B, H, T, d, dh, int(chunk), float(eta), et, ptr(deta), _loss(loss),
                                _io_dtype(q), _stream(q.device, stream))
    _check(rc)
    res = (dq, dk, dv, dw1, dw2, dlw, dlb)
    return res if deta is None else res + (deta,)


def ttt_linear_nc_bwd(q, k, v, w0, eta, chunk, dz, dw_out=None, *, epochs=1, eta_tok=None,
                      loss="mse", stream=None):
    """Gradients of the non-causal TTT-Linear layer (ttt_linear_fwd with causal=False, the
    same chunk, epochs, eta_tok and loss) for the upstream gradients dz [B,H,T,d] (dtype of q)
    and dw_out [B,H,d,d] float32 (or None).  Returns (dq, dk, dv, dw0), plus deta_tok
    [B,H,T] with eta_tok; dw0 per sequence."""
    torch = _torch()
    lib = load_library()
    B, H, T, d = _tokens(q, k, v)
    w0, stride = _state(w0, B, H, (d, d), "w0", q.device)
    dz = _dz(dz, q, B, H, T, d)
    if dw_out is not None:
        dw_out = _out(dw_out, (B, H, d, d), torch.float32, q.device, "dw_out")
    et = _rates(eta_tok, B, H, T, q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    dw0 = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device)
    deta = torch.empty((B, H, T), dtype=torch.float32, device=q.device) if et is not None else None
    ptr = lambda t: t.data_ptr() if t is not None else None
    with torch.cuda.device(q.device):
        rc = lib.ttt_linear_nc_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), w0.data_ptr(), stride,
                                   dz.data_ptr(), ptr(dw_out), dq.data_ptr(), dk.data_ptr(),
                                   dv.data_ptr(), dw0.data_ptr(), B, H, T, d, int(chunk),
                                   int(epochs), float(eta), et, ptr(deta), _loss(loss),
                                   _io_dtype(q), _stream(q.device, stream))
    _check(rc)
    return (dq, dk, dv, dw0) if deta is None else (dq, dk, dv, dw0, deta)


def ttt_mlp_nc_bwd(q, k, v, w1, w2, eta, chunk, dz, dw1_out=None, dw2_out=None, *, epochs=1,
                   eta_tok=None, loss="mse", stream=None):
    """Gradients of the non-causal TTT-MLP layer (ttt_mlp_fwd with causal=False; SiLU) for
    the upstream gradients dz and dw1_out [B,H,dh,d], dw2_out [B,H,d,dh] (or None).  Returns
    (dq, dk, dv, dw1, dw2), plus deta_tok [B,H,T] with eta_tok; state gradients per
    sequence."""
    torch = _torch()
    lib = load_library()
    B, H, T, d = _tokens(q, k, v)
    if w1.dim() < 2:
        raise ValueError("w1 must be [H, dh, d] or [B, H, dh, d]")
    dh = int(w1.shape[-2])
    w1, s1 = _state(w1, B, H, (dh, d), "w1", q.device)
    w2, s2 = _state(w2, B, H, (d, dh), "w2", q.device)
    if s1 != s2:
        raise ValueError("w1 and w2 must both be shared over the batch or both per batch")
    dz = _dz(dz, q, B, H, T, d)
    if (dw1_out is None) != (dw2_out is None):
        raise ValueError("give both dw1_out and dw2_out, or neither")
    if dw1_out is not None:
        dw1_out = _out(dw1_out, (B, H, dh, d), torch.float32, q.device, "dw1_out")
        dw2_out = _out(dw2_out, (B, H, d, dh), torch.float32, q.device, "dw2_out")
    et = _rates(eta_tok, B, H, T, q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    dw1 = torch.empty((B, H, dh, d), dtype=torch.float32, device=q.device)
    dw2 = torch.empty((B, H, d, dh), dtype=torch.float32, device=q.device)
    deta = torch.empty((B, H, T), dtype=torch.float32, device=q.device) if et is not None else None
    ptr = lambda t: t.data_ptr() if t is not None else None
    with torch.cuda.device(q.device):
        rc = lib.ttt_mlp_nc_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), w1.data_ptr(),
                                w2.data_ptr(), s1, dz.data_ptr(), ptr(dw1_out), ptr(dw2_out),
                                dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dw1.data_ptr(),
                                dw2.data_ptr(), B, H, T, d, dh, int(chunk), int(epochs),
                                float(eta), et, ptr(deta), _loss(loss), _io_dtype(q),
                                _stream(q.device, stream))
    _check(rc)
    return (dq, dk, dv, dw1, dw2) if deta is None else (dq, dk, dv, dw1, dw2, deta)


def delta_rule_fwd(q, k, v, w0, eta, *, eta_tok=None, z=None, w_out=None, return_state=False,
                   stream=None):
    """Delta-rule forward (one token per update, causal).  Arguments as ttt_linear_fwd."""
    torch = _torch()
    lib = load_library()
    B, H, T, d = _tokens(q, k, v)
    w0, stride = _state(w0, B, H, (d, d), "w0", q.device)
    z = _out(z, (B, H, T, d), q.dtype, q.device, "z")
    if return_state or w_out is not None:
        w_out = _out(w_out, (B, H, d, d), torch.float32, q.device, "w_out")
    with torch.cuda.device(q.device):
        rc = lib.delta_rule_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), w0.data_ptr(), stride,
                                z.data_ptr(), w_out.data_ptr() if w_out is not None else None,
                                B, H, T, d, float(eta), _rates(eta_tok, B, H, T, q.device),
                                _io_dtype(q), _stream(q.device, stream))
    _check(rc)
    return (z, w_out) if w_out is not None else z


def _mlp(q, k, v, w1, w2, eta, chunk, causal, ln, eta_tok, loss, epochs, z, w1_out, w2_out,
         return_state, stream, workspace=False):
    torch = _torch()
    lib = load_library()
    B, H, T, d = _tokens(q, k, v)
    if w1.dim() < 2:
        raise ValueError("w1 must be [H, dh, d] or [B, H, dh, d]")
    dh = int(w1.shape[-2])
    w1, s1 = _state(w1, B, H, (dh, d), "w1", q.device)
    w2, s2 = _state(w2, B, H, (d, dh), "w2", q.device)
    if s1 != s2:
        raise ValueError("w1 and w2 must both be shared over the batch or both per batch")
    z = _out(z, (B, H, T, d), q.dtype, q.device, "z")
    want = return_state or w1_out is not None or w2_out is not None
    if want:
        w1_out = _out(w1_out, (B, H, dh, d), torch.float32, q.device, "w1_out")
        w2_out = _out(w2_out, (B, H, d, dh), torch.float32, q.device, "w2_out")
    tail = (z.data_ptr(), w1_out.data_ptr() if want else None, w2_out.data_ptr() if want else None,
            B, H, T, d, dh, int(chunk), int(bool(causal)), float(eta),
            _rates(eta_tok, B, H, T, q.device), _loss(loss), int(epochs),
            _io_dtype(q), _stream(q.device, stream))
    with torch.cuda.device(q.device):
        if workspace is not False:
            # the _ws entry points: tail without the stream, then workspace, size, stream
            need = lib.ttt_mlp_fwd_workspace_size(B, H, T, d, dh, int(chunk), int(bool(causal)),
                                                  _io_dtype(q))
            if workspace is None:
                workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
            if not (workspace.is_cuda and workspace.device == q.device and workspace.is_contiguous()):
                raise ValueError("workspace must be a contiguous tensor on the device of q")
            ws = (workspace.data_ptr(), workspace.numel() * workspace.element_size())
            if ln is None:
                rc = lib.ttt_mlp_fwd_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), w1.data_ptr(),
                                        w2.data_ptr(), s1, *tail[:-1], *ws, tail[-1])
            else:
                rc = lib.ttt_mlp_ln_fwd_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                           w1.data_ptr(), w2.data_ptr(), s1,
                                           *_ln(*ln, H, d, q.device), *tail[:-1], *ws, tail[-1])
        elif ln is None:
            rc = lib.ttt_mlp_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), w1.data_ptr(),
                                 w2.data_ptr(), s1, *tail)
        else:
            rc = lib.ttt_mlp_ln_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), w1.data_ptr(),
                                    w2.data_ptr(), s1, *_ln(*ln, H, d, q.device), *tail)
    _check(rc)
    return (z, w1_out, w2_out) if want else z


def ttt_mlp_fwd(q, k, v, w1, w2, eta, chunk, causal=True, *, eta_tok=None, loss="mse", epochs=1,
                z=None, w1_out=None, w2_out=None, return_state=False, stream=None):
    """TTT-MLP forward, f(k) = W2 SiLU(W1 k).  w1 float32 [H,dh,d] or [B,H,dh,d], w2 float32
    [H,d,dh] or [B,H,d,dh] (both shared or both per batch); eta_tok, loss and epochs as in
    ttt_linear_fwd.
    Returns z (and the final states when return_state or an output state is given)."""
    return _mlp(q, k, v, w1, w2, eta, chunk, causal, None, eta_tok, loss, epochs, z, w1_out,
                w2_out, return_state, stream)


def ttt_mlp_fwd_workspace_size(B, H, T, d, dh, chunk, causal=True, io_dtype="bf16"):
    """Bytes of workspace ttt_mlp_fwd_ws / ttt_mlp_ln_fwd_ws need for this shape (0: none,
    the call then runs as ttt_mlp_fwd / ttt_mlp_ln_fwd)."""
    lib = load_library()
    code = {"bf16": 1, "f32": 0, "float32": 0, "bfloat16": 1}[str(io_dtype).replace("torch.", "")]
    return int(lib.ttt_mlp_fwd_workspace_size(int(B), int(H), int(T), int(d), int(dh), int(chunk),
                                              int(bool(causal)), code))


def ttt_mlp_fwd_ws(q, k, v, w1, w2, eta, chunk, causal=True, *, workspace=None, eta_tok=None,
                   loss="mse", epochs=1, z=None, w1_out=None, w2_out=None, return_state=False,
                   stream=None):
    """ttt_mlp_fwd on the two-workgroup kernel, with a caller workspace: a contiguous device
    tensor of at least ttt_mlp_fwd_workspace_size(...) bytes (None: one is allocated with
    torch for this call)."""
    return _mlp(q, k, v, w1, w2, eta, chunk, causal, None, eta_tok, loss, epochs, z, w1_out,
                w2_out, return_state, stream, workspace)


def ttt_mlp_ln_fwd_ws(q, k, v, w1, w2, ln_weight, ln_bias, eta, chunk, causal=True, *,
                      workspace=None, ln_eps=1e-6, eta_tok=None, loss="mse", epochs=1, z=None,
                      w1_out=None, w2_out=None, return_state=False, stream=None):
    """ttt_mlp_ln_fwd on the two-workgroup kernel; workspace as in ttt_mlp_fwd_ws."""
    return _mlp(q, k, v, w1, w2, eta, chunk, causal, (ln_weight, ln_bias, ln_eps), eta_tok, loss,
                epochs, z, w1_out, w2_out, return_state, stream, workspace)


def ttt_mlp_ln_fwd(q, k, v, w1, w2, ln_weight, ln_bias, eta, chunk, causal=True, *, ln_eps=1e-6,
                   eta_tok=None, loss="mse", epochs=1, z=None, w1_out=None, w2_out=None,
                   return_state=False, stream=None):
    """The paper's TTT-MLP, f(x) = x + LN(W2 GELU(W1 x)) with per-head ln_weight, ln_bias
    float32 [H, d]; every other argument as ttt_mlp_fwd."""
    return _mlp(q, k, v, w1, w2, eta, chunk, causal, (ln_weight, ln_bias, ln_eps), eta_tok, loss,
                epochs, z, w1_out, w2_out, return_state, stream)


# ------------------------------------------------------- gated linear recurrence, token norm

_HERE = contextlib.nullcontext()


def _enter(device, stream):
    """(stream pointer, context) of a call: in the context torch allocates for the call's stream,
    so that outputs and workspaces are reused in that stream's order, and the call's device is
    the current one.  On the current stream of the current device there is nothing to enter."""
    torch = _torch()
    if stream is None:
        if device.index == torch.cuda.current_device():
            # the pointer alone: a Stream object takes 1.7 us more of a 12 us call
            return torch._C._cuda_getCurrentRawStream(device.index), _HERE
        stream = torch.cuda.current_stream(device)
    elif not hasattr(stream, "cuda_stream"):
        stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                  else torch.cuda.default_stream(device))
    return stream.cuda_stream, torch.cuda.stream(stream)


def _optional(t, shape, dtype, device, name):
    """Pointer of an optional contiguous tensor (None -> NULL)."""
    if t is None:
        return None
    if (not isinstance(t, _torch().Tensor) or t.shape != shape or t.dtype != dtype
            or t.device != device or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t.data_ptr()


def _pointer(t):
    return t.data_ptr() if t is not None else None


def _workspace(workspace, nbytes, device):
    """(tensor or None, bytes) of a caller workspace, or of one allocated for this call."""
    torch = _torch()
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    elif (not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous()
          or workspace.device != device):
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace, workspace.numel() * workspace.element_size() if workspace is not None else 0


def gated_linear_fwd(q, k, v, w0, eta, log_gate=None, *, eta_tok=None, lengths=None, z=None,
                     w_out=None, return_state=False, workspace=None, stream=None):
    """Gated linear recurrence W_t = exp(log_gate[t]) W_{t-1} + eta_t v_t k_t^T, z_t = W_t q_t.
    q, k, v [B,H,T,d] (float32 or bfloat16, d in 16, 32, 64); w0 float32 [H,d,d] (shared over the
    batch) or [B,H,d,d]; log_gate float32 [B,H,T] (None: no decay; -inf starts a new sequence);
    eta_tok optional float32 [B,H,T] rate factors; lengths optional int32 [B], tokens of each
    batch row (z is 0 past them).  workspace: a tensor of at least
    gated_linear_fwd_workspace_size(...) bytes (None: torch allocates one).  Returns z (and the
    final state [B,H,d,d] when return_state or w_out is given)."""
    torch = _torch()
    lib = load_library()
    B, H, T, d = _tokens(q, k, v)
    dev, io = q.device, _io_dtype(q)
    w0, stride = _state(w0, B, H, (d, d), "w0", dev)
    gate = _optional(log_gate, (B, H, T), torch.float32, dev, "log_gate")
    rate = _rates(eta_tok, B, H, T, dev)
    lens = _optional(lengths, (B,), torch.int32, dev, "lengths")
    on, here = _enter(dev, stream)
    with here:
        z = torch.empty_like(q) if z is None else _out(z, (B, H, T, d), q.dtype, dev, "z")
        if return_state or w_out is not None:
            w_out = _out(w_out, (B, H, d, d), torch.float32, dev, "w_out")
        ws, nbytes = _workspace(workspace, lib.gated_linear_fwd_workspace_size(B, H, T, d, io), dev)
        rc = lib.gated_linear_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), gate, w0.data_ptr(), stride,
                                  lens, z.data_ptr(), _pointer(w_out), B, H, T, d, float(eta), rate, io,
                                  _pointer(ws), nbytes, on)
    _check(rc)
    return (z, w_out) if w_out is not None else z


def gated_linear_bwd(q, k, v, w0, eta, log_gate, dz, dw_out=None, *, eta_tok=None, lengths=None,
                     workspace=None, stream=None):
    """Gradients of gated_linear_fwd for the upstream gradients dz [B,H,T,d] (dtype of q) and
    dw_out [B,H,d,d] float32 (or None).  Returns (dq, dk, dv, dw0) with dw0 [B,H,d,d] per
    sequence (sum it over the batch when w0 is shared), then dlog_gate [B,H,T] if log_gate is
    given and deta_tok [B,H,T] if eta_tok is.  It needs no output of the forward pass."""
    torch = _torch()
    lib = load_library()
    B, H, T, d = _tokens(q, k, v)
    dev, io = q.device, _io_dtype(q)
    w0, stride = _state(w0, B, H, (d, d), "w0", dev)
    _dz(dz, q, B, H, T, d)
    dw = _optional(dw_out, (B, H, d, d), torch.float32, dev, "dw_out")
    gate = _optional(log_gate, (B, H, T), torch.float32, dev, "log_gate")
    rate = _rates(eta_tok, B, H, T, dev)
    lens = _optional(lengths, (B,), torch.int32, dev, "lengths")
    on, here = _enter(dev, stream)
    with here:
        out = [torch.empty_like(q), torch.empty_like(q), torch.empty_like(q),
               w0.new_empty((B, H, d, d))]
        dgate, deta = (torch.empty_like(x) if x is not None else None for x in (log_gate, eta_tok))
        ws, nbytes = _workspace(workspace, lib.gated_linear_bwd_workspace_size(
            B, H, T, d, int(dgate is not None), io), dev)
        rc = lib.gated_linear_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), gate, w0.data_ptr(), stride,
                                  lens, dz.data_ptr(), dw, *(x.data_ptr() for x in out), _pointer(dgate),
                                  B, H, T, d, float(eta), rate, _pointer(deta), io, _pointer(ws), nbytes,
                                  on)
    _check(rc)
    return tuple(out + [x for x in (dgate, deta) if x is not None])


def gated_linear_step(q, k, v, w, eta, log_gate=None, *, eta_tok=None, z=None, stream=None):
    """One token of gated_linear_fwd for every sequence: q, k, v [B,H,d], log_gate and eta_tok
    [B,H] float32 (or None), and the states w [B,H,d,d] float32, updated in place.  Returns
    z [B,H,d]."""
    torch = _torch()
    lib = load_library()
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != 3 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [B, H, d] tensor on a GPU")
        if t.shape != q.shape or t.dtype != q.dtype or t.device != q.device:
            raise ValueError("q, k and v must have the same shape, dtype and device")
    B, H, d = q.shape
    dev, io = q.device, _io_dtype(q)
    state = _optional(w, (B, H, d, d), torch.float32, dev, "w")
    gate = _optional(log_gate, (B, H), torch.float32, dev, "log_gate")
    rate = _optional(eta_tok, (B, H), torch.float32, dev, "eta_tok")
    on, here = _enter(dev, stream)
    with here:
        z = torch.empty_like(q) if z is None else _out(z, (B, H, d), q.dtype, dev, "z")
        rc = lib.gated_linear_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), gate, state, z.data_ptr(),
                                   B, H, d, float(eta), rate, io, on)
    _check(rc)
    return z


def gated_linear_fwd_workspace_size(B, H, T, d, dtype) -> int:
    """Workspace bytes of gated_linear_fwd for token tensors [B,H,T,d] of a torch dtype."""
    io = TTT_BF16 if dtype == _torch().bfloat16 else TTT_F32
    return int(load_library().gated_linear_fwd_workspace_size(B, H, T, d, io))


def gated_linear_bwd_workspace_size(B, H, T, d, gated, dtype) -> int:
    """Workspace bytes of gated_linear_bwd; gated: whether log_gate's gradient is taken."""
    io = TTT_BF16 if dtype == _torch().bfloat16 else TTT_F32
    return int(load_library().gated_linear_bwd_workspace_size(B, H, T, d, int(bool(gated)), io))


_NORMS = {"layer": 0, "rms": 1, "l2": 2}
_ACTS = {"none": 0, "silu": 1, "gelu": 2, "sigmoid": 3}


def _norm_args(x, kind, act):
    torch = _torch()
    if not isinstance(x, torch.Tensor) or x.dim() != 4 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous [B, H, T, d] tensor on a GPU")
    if kind not in _NORMS:
        raise ValueError(f"kind must be one of {sorted(_NORMS)}, got {kind!r}")
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    return tuple(x.shape), x.device, _io_dtype(x)


def token_norm_fwd(x, kind, eps=1e-6, *, weight=None, bias=None, gate=None, act="silu", scale=None,
                   res=None, y=None, stream=None):
    """y = res + scale * act(gate) * (norm(x) * weight + bias) over the d features of every token.
    x, gate, res [B,H,T,d] (float32 or bfloat16); weight, bias, scale float32 [H,d]; each but x
    may be None.  kind: "layer", "rms" or "l2" (x / sqrt(sum x^2 + eps)); act: "silu", "gelu"
    (exact), "sigmoid" or "none" (the gate itself)."""
    torch = _torch()
    lib = load_library()
    (B, H, T, d), dev, io = _norm_args(x, kind, act)
    par = [_optional(t, (H, d), torch.float32, dev, n)
           for t, n in ((weight, "weight"), (bias, "bias"), (scale, "scale"))]
    gp, rp = (_optional(t, x.shape, x.dtype, dev, n) for t, n in ((gate, "gate"), (res, "res")))
    on, here = _enter(dev, stream)
    with here:
        y = torch.empty_like(x) if y is None else _out(y, x.shape, x.dtype, dev, "y")
        rc = lib.token_norm_fwd(x.data_ptr(), par[0], par[1], gp, par[2], rp, y.data_ptr(), B, H, T, d,
                                _NORMS[kind], _ACTS[act], float(eps), io, on)
    _check(rc)
    return y


def token_norm_bwd(x, dy, kind, eps=1e-6, *, weight=None, bias=None, gate=None, act="silu",
                   scale=None, workspace=None, stream=None):
    """Gradients of token_norm_fwd for the upstream gradient dy (dtype of x): returns
    (dx, dweight, dbias, dgate, dscale), None for each input that is None; that of res is dy
    itself.  dweight, dbias and dscale [H,d] float32 are sums over the batch and the tokens."""
    torch = _torch()
    lib = load_library()
    (B, H, T, d), dev, io = _norm_args(x, kind, act)
    dyp = _optional(dy, x.shape, x.dtype, dev, "dy")
    if dyp is None:
        raise ValueError("dy must be given")
    named = ((weight, "weight"), (bias, "bias"), (scale, "scale"))
    par = [_optional(t, (H, d), torch.float32, dev, n) for t, n in named]
    gp = _optional(gate, x.shape, x.dtype, dev, "gate")
    on, here = _enter(dev, stream)
    with here:
        dx = torch.empty_like(x)
        dpar = [torch.empty_like(t) if t is not None else None for t, _ in named]
        dg = torch.empty_like(x) if gate is not None else None
        need = lib.token_norm_bwd_workspace_size(B, H, T, d) if any(t is not None for t in dpar) else 0
        ws, nbytes = _workspace(workspace, need, dev)
        rc = lib.token_norm_bwd(x.data_ptr(), par[0], par[1], gp, par[2], dyp, dx.data_ptr(),
                                _pointer(dpar[0]), _pointer(dpar[1]), _pointer(dg), _pointer(dpar[2]),
                                B, H, T, d, _NORMS[kind], _ACTS[act], float(eps), io, _pointer(ws),
                                nbytes, on)
    _check(rc)
    return dx, dpar[0], dpar[1], dg, dpar[2]


def token_norm_bwd_workspace_size(B, H, T, d) -> int:
    """Workspace bytes of token_norm_bwd (when a parameter's gradient is taken)."""
    return int(load_library().token_norm_bwd_workspace_size(B, H, T, d))
