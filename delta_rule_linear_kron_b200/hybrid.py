"""Operators that stand beside the delta rules in a hybrid stack (binding over
the C ABI, like the package's own functions, which re-exports these):

  rotary_fwd, rotary_bwd, rotary_freqs      rotary positions of q and k
  swa_fwd, swa_bwd, swa_decode, swa_fill    attention over a sliding window
                                            with first tokens kept
  glr_fwd, glr_bwd, glr_decode              element-wise gated linear recurrence

Tensors of a call are on one CUDA device, which need not be the current one:
the call runs on the current stream of the tensors' device, or on `stream`.
"""
from __future__ import annotations

import functools
import math

from . import (KD_ERR_INVALID_ARG, KronDeltaError, _alloc_ws, _check, _dtype_code, _need, lib)

KD_SWA_WS_SAVE, KD_SWA_WS_BWD, KD_SWA_WS_DECODE = 0, 1, 2
KD_GLR_WS_SAVE, KD_GLR_WS_BWD = 0, 1
KD_SWA_MAX_SINKS = 128

__all__ = ["rotary_fwd", "rotary_bwd", "rotary_freqs", "swa_fwd", "swa_bwd", "swa_decode", "swa_fill",
           "swa_workspace_size", "glr_fwd", "glr_bwd", "glr_decode", "glr_workspace_size",
           "KD_SWA_WS_SAVE", "KD_SWA_WS_BWD", "KD_SWA_WS_DECODE", "KD_GLR_WS_SAVE", "KD_GLR_WS_BWD",
           "KD_SWA_MAX_SINKS"]


def _invalid(msg):
    return KronDeltaError(KD_ERR_INVALID_ARG, msg)


def _dims(t, name, n):
    if t.dim() != n:
        raise _invalid(f"{name} must have {n} dimensions (got shape {tuple(t.shape)})")
    return t.shape


def _device(t, name):
    """Ordinal of the CUDA device that the call's tensors share."""
    dev = t.get_device()
    if dev < 0:
        _need(t, name)
    return dev


def _arg(t, name, dev, dtype, shape):
    """The checked tensor's address (None for None).  One short test on the way
    of a good argument: these run on every decode step."""
    if t is None:
        return None
    if t.get_device() == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _need(t, name, dtype, shape)
    raise _invalid(f"{name} is on {t.device}, the call's first tensor on device {dev}")


def _out(out, like, dev):
    """The output tensor, made like `like` if none is given, and its address."""
    import torch
    if out is None:
        out = torch.empty_like(like)
        return out, out.data_ptr()
    return out, _arg(out, "out", dev, like.dtype, like.shape)


def _bytes_arg(t, name, dev):
    """Address and size of a workspace."""
    if t is None:
        return None, 0
    if t.get_device() != dev or not t.is_contiguous():
        _need(t, name)
        raise _invalid(f"{name} is on {t.device}, the call's first tensor on device {dev}")
    return t.data_ptr(), t.numel() * t.element_size()


def _streamed(fn):
    """The public form of a function: with `stream`, all of it runs under that
    stream, what it allocates too, so that the allocator hands none of that
    memory to another stream while the call's kernels use it."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        import torch
        first = next((a for a in (*args, *kw.values()) if isinstance(a, torch.Tensor)), None)
        if first is not None and first.device != stream.device:
            raise _invalid(f"stream belongs to {stream.device} but the call's tensors are on {first.device}")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _call(fn, dev, *args):
    """fn(*args, stream) on device `dev` and its current stream."""
    import torch
    s = torch._C._cuda_getCurrentRawStream(dev)
    if torch._C._cuda_getDevice() == dev:
        _check(fn(*args, s))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, s))


def _size(n):
    """A workspace size; 0 is either none needed (no error recorded) or an error."""
    if n == 0:
        msg = lib().kron_delta_last_error().decode()
        if msg:
            raise _invalid(msg)
    return n


def _int32(n, most=2 ** 31 - 1):
    """n as a C int: ctypes cuts off what is beyond 32 bits, and what is left
    may be in range."""
    return max(-2 ** 31, min(n, most))


def _window(window):
    """A window beyond the longest sequence is all of it."""
    return _int32(window, 2 ** 31 - 1 - KD_SWA_MAX_SINKS)


@functools.lru_cache(maxsize=1024)  # of its arguments alone; asked on every decode step
def swa_workspace_size(kind, B, T, H, Hk, d, window, sinks, dtype) -> int:
    window, sinks = _int32(window) if kind == KD_SWA_WS_DECODE else _window(window), _int32(sinks)
    return _size(lib().kron_delta_swa_workspace_size(kind, B, T, H, Hk, d, window, sinks, dtype))


@functools.lru_cache(maxsize=1024)
def glr_workspace_size(kind, B, T, D, dtype) -> int:
    return _size(lib().kron_delta_glr_workspace_size(kind, B, T, D, dtype))


# ---- rotary positions ---------------------------------------------------------


def rotary_freqs(rotary_dim, base=10000.0, *, scaling=None, factor=1.0, trained_len=None, low=1.0, high=32.0,
                 device="cuda"):
    """Angular frequencies [rotary_dim/2] (fp64, on `device`) and the factor on
    the rotated values, for rotary_fwd.  Pair j turns base^(-2j/rotary_dim)
    radians per position.  scaling, for contexts `factor` times the trained one:
      "linear"  every frequency divided by factor;
      "ntk"     base multiplied by factor^(rotary_dim/(rotary_dim-2)): the
                slowest pair slows by factor, the fastest keeps its pace;
      "yarn"    pairs that turn more than `high` times over trained_len
                positions keep their frequency, those below `low` turns are
                divided by factor, a linear ramp between; the rotated values
                are scaled by 0.1 ln(factor) + 1."""
    import torch
    if rotary_dim < 2 or rotary_dim % 2:
        raise _invalid(f"rotary_dim must be even and >= 2 (got {rotary_dim})")
    if not base > 1 or not factor >= 1 or not math.isfinite(base) or not math.isfinite(factor):
        raise _invalid(f"base must be > 1 and factor >= 1, both finite (got {base}, {factor})")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise _invalid(f"scaling must be None, 'linear', 'ntk' or 'yarn' (got {scaling!r})")
    if scaling == "ntk":
        if rotary_dim == 2:
            raise _invalid("'ntk' scaling needs rotary_dim > 2")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    w = base ** (torch.arange(0, rotary_dim, 2, dtype=torch.float64) / -rotary_dim)
    scale = 1.0
    if scaling == "linear":
        w = w / factor
    elif scaling == "yarn":
        if trained_len is None or trained_len < 1 or not low < high:
            raise _invalid(f"'yarn' scaling needs trained_len >= 1 and low < high (got {trained_len}, {low}, {high})")
        keep = ((trained_len * w / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        w = w * keep + w / factor * (1 - keep)
        scale = 0.1 * math.log(factor) + 1.0
    return w.to(device), scale


def _rotary(q, k, freqs, pos, interleaved, scale, inverse, out):
    import torch
    shape = q.shape
    if len(shape) == 4:
        B, T, H, d = shape
    else:  # one token per sequence: [B,H,d], pos [B]
        B, H, d = _dims(q, "q", 3)
        T = 1
    lead, dev, dtype = shape[:-2], _device(q, "q"), q.dtype
    dt = _dtype_code(q)
    Hk, k_shape = 0, None
    if k is not None:
        k_shape = _dims(k, "k", len(shape))
        Hk = k_shape[-2]
    half = _dims(freqs, "freqs", 1)[0]
    kk = (*lead, Hk, d)
    if out is None:
        oq, ok = torch.empty_like(q), None if k is None else torch.empty_like(k)
        pq, pk = oq.data_ptr(), None if k is None else ok.data_ptr()
    else:
        oq, ok = out
        if (ok is None) != (k is None):
            raise _invalid("out must be a pair like (q, k)")
        pq, pk = _arg(oq, "out[0]", dev, dtype, shape), _arg(ok, "out[1]", dev, dtype, kk)
    _call(lib().kron_delta_rotary, dev, _arg(q, "q", dev, dtype, shape), _arg(k, "k", dev, dtype, kk),
          _arg(freqs, "freqs", dev, torch.float64, (half,)), _arg(pos, "pos", dev, torch.int64, lead),
          pq, pk, B, T, H, Hk, d, 2 * half, 1 if interleaved else 0, inverse, scale, dt)
    return oq, ok


@_streamed
def rotary_fwd(q, k, freqs, pos=None, *, interleaved=False, scale=1.0, out=None, stream=None):
    """Rotary positions: pair j of the first 2*len(freqs) channels turns by
    pos*freqs[j] and is scaled by `scale`; the other channels are copied.
    q [B,T,H,d], k [B,T,Hk,d] or None (bf16 or fp32); freqs fp64; pos [B,T] int64
    or None for 0..T-1.  One token per sequence: q [B,H,d], k [B,Hk,d], pos [B].
    Pair j is channels (j, j + len(freqs)), or (2j, 2j+1) with interleaved.
    out=(q, k) works in place.  Returns (q, k) rotated."""
    return _rotary(q, k, freqs, pos, interleaved, scale, 0, out)


@_streamed
def rotary_bwd(dq, dk, freqs, pos=None, *, interleaved=False, scale=1.0, out=None, stream=None):
    """Backward of rotary_fwd: the gradients of q and k from those of its
    outputs (the rotation by -pos*freqs[j])."""
    return _rotary(dq, dk, freqs, pos, interleaved, scale, 1, out)


# ---- attention over a sliding window with first tokens kept -----------------


def _swa_inputs(q, k, v):
    """Sizes, dtype code, device and the three addresses."""
    shape = _dims(q, "q", 4)
    B, T, H, d = shape
    Hk = _dims(k, "k", 4)[2]
    dev, dtype, kv = _device(q, "q"), q.dtype, (B, T, Hk, d)
    return B, T, H, Hk, d, _dtype_code(q), dev, (_arg(q, "q", dev, dtype, shape), _arg(k, "k", dev, dtype, kv),
                                                 _arg(v, "v", dev, dtype, kv))


def _scale(scale, d):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


@_streamed
def swa_fwd(q, k, v, window, sinks=0, *, scale=None, out=None, save=False, workspace=None, stream=None):
    """Causal attention where query t sees key j when j <= t and (t - j < window
    or j < sinks); window >= T is plain causal attention.  q [B,T,H,d], k, v
    [B,T,Hk,d] (bf16 or fp32), H a multiple of Hk, finite in every row, padding
    included; scale defaults to 1/sqrt(d).  Returns (out [B,T,H,d], lse [B,T,H] fp32,
    workspace or None); pass all three (save=True) to swa_bwd."""
    import torch
    B, T, H, Hk, d, dt, dev, ptrs = _swa_inputs(q, k, v)
    window, sinks = _window(window), _int32(sinks)
    out, p_out = _out(out, q, dev)
    lse = q.new_empty((B, T, H), dtype=torch.float32)
    if save and workspace is None:
        n = swa_workspace_size(KD_SWA_WS_SAVE, B, T, H, Hk, d, window, sinks, dt)
        workspace = _alloc_ws(n, q.device) if n else None
    _call(lib().kron_delta_swa_fwd, dev, *ptrs, p_out, lse.data_ptr(), B, T, H, Hk, d, window, sinks, _scale(scale, d), dt, *_bytes_arg(workspace, "workspace", dev), 1 if save else 0)
    return out, lse, workspace


@_streamed
def swa_bwd(q, k, v, out, lse, dO, window, sinks=0, *, scale=None, fwd_workspace, workspace=None, stream=None):
    """Backward of swa_fwd for the loss <dO, out>, from its three results.
    Returns dict dq, dk, dv (summed in a fixed order: bitwise reproducible)."""
    import torch
    B, T, H, Hk, d, dt, dev, ptrs = _swa_inputs(q, k, v)
    window, sinks = _window(window), _int32(sinks)
    g = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v))
    if workspace is None:
        workspace = _alloc_ws(swa_workspace_size(KD_SWA_WS_BWD, B, T, H, Hk, d, window, sinks, dt), q.device)
    _call(lib().kron_delta_swa_bwd, dev, *ptrs, _arg(out, "out", dev, q.dtype, q.shape),
          _arg(lse, "lse", dev, torch.float32, (B, T, H)), _arg(dO, "dO", dev, q.dtype, q.shape), g["dq"].data_ptr(),
          g["dk"].data_ptr(), g["dv"].data_ptr(), B, T, H, Hk, d, window, sinks, _scale(scale, d), dt,
          *_bytes_arg(fwd_workspace, "fwd_workspace", dev), *_bytes_arg(workspace, "workspace", dev))
    return g


@_streamed
def swa_decode(q, k, v, k_cache, v_cache, pos, window, sinks=0, *, scale=None, out=None, workspace=None,
               stream=None):
    """One decode step of swa_fwd's attention.  q [B,H,d], k, v [B,Hk,d]: the new
    tokens, at positions pos [B] int64 (pos < 0: the sequence is idle, its cache
    stays and its out is zero); k_cache, v_cache [B,sinks+window,Hk,d], updated
    in place.  Position p lives in slot p (p < sinks) or
    sinks + (p - sinks) % window; see swa_fill for the start after a prefill.
    Returns out [B,H,d]."""
    import torch
    shape = _dims(q, "q", 3)
    B, H, d = shape
    Hk = _dims(k, "k", 3)[1]
    dev, dtype, dt = _device(q, "q"), q.dtype, _dtype_code(q)
    kv, cache = (B, Hk, d), (B, sinks + window, Hk, d)
    out, p_out = _out(out, q, dev)
    if workspace is None:
        n = swa_workspace_size(KD_SWA_WS_DECODE, B, 1, H, Hk, d, window, sinks, dt)
        workspace = _alloc_ws(n, q.device) if n else None
    _call(lib().kron_delta_swa_decode, dev, _arg(q, "q", dev, dtype, shape), _arg(k, "k", dev, dtype, kv),
          _arg(v, "v", dev, dtype, kv), _arg(k_cache, "k_cache", dev, dtype, cache),
          _arg(v_cache, "v_cache", dev, dtype, cache), _arg(pos, "pos", dev, torch.int64, (B,)),
          p_out, B, H, Hk, d, window, sinks, _scale(scale, d), dt,
          *_bytes_arg(workspace, "workspace", dev))
    return out


@_streamed
def swa_fill(k, v, lens, k_cache, v_cache, window, sinks=0, *, stream=None):
    """Fills swa_decode's caches from a prefill's k, v [B,T,Hk,d]: of sequence
    b's first lens[b] tokens (int64), the first `sinks` and the last `window` go
    to their slots; the other slots stay as they were."""
    import torch
    shape = _dims(k, "k", 4)
    B, T, Hk, d = shape
    dev, dtype, cache = _device(k, "k"), k.dtype, (B, sinks + window, Hk, d)
    dt = _dtype_code(k)
    _call(lib().kron_delta_swa_fill, dev, _arg(k, "k", dev, dtype, shape), _arg(v, "v", dev, dtype, shape),
          _arg(lens, "lens", dev, torch.int64, (B,)), _arg(k_cache, "k_cache", dev, dtype, cache),
          _arg(v_cache, "v_cache", dev, dtype, cache), B, T, Hk, d, window, sinks, dt)


# ---- gated linear recurrence --------------------------------------------------


def _glr_inputs(x, i_pre, f_pre, a_log, n):
    """Shape, dtype code, device and the four addresses."""
    import torch
    shape = _dims(x, "x", n)
    dev, dtype = _device(x, "x"), x.dtype
    return shape, _dtype_code(x), dev, (_arg(x, "x", dev, dtype, shape), _arg(i_pre, "i_pre", dev, dtype, shape),
                                        _arg(f_pre, "f_pre", dev, dtype, shape),
                                        _arg(a_log, "a_log", dev, torch.float32, shape[-1:]))


@_streamed
def glr_fwd(x, i_pre, f_pre, a_log, h0=None, *, out=None, want_state=True, save=False, workspace=None, stream=None):
    """Gated linear recurrence per channel: f = sigmoid(f_pre)^exp(a_log),
    h_t = f h_{t-1} + sqrt(1 - f^2) sigmoid(i_pre) x.  x, i_pre, f_pre [B,T,D]
    (bf16 or fp32, D a multiple of 8); a_log [D] fp32; h0 [B,D] fp32 or None.
    f_pre = -inf starts a new sequence at that token.  Returns (out [B,T,D] = h,
    hT [B,D] fp32 or None, workspace or None); pass the workspace (save=True) to
    glr_bwd."""
    import torch
    shape, dt, dev, ptrs = _glr_inputs(x, i_pre, f_pre, a_log, 3)
    B, T, D = shape
    out, p_out = _out(out, x, dev)
    hT = x.new_empty((B, D), dtype=torch.float32) if want_state else None
    if save and workspace is None:
        workspace = _alloc_ws(glr_workspace_size(KD_GLR_WS_SAVE, B, T, D, dt), x.device)
    _call(lib().kron_delta_glr_fwd, dev, *ptrs, _arg(h0, "h0", dev, torch.float32, (B, D)),
          p_out, hT.data_ptr() if want_state else None, B, T, D, dt,
          *_bytes_arg(workspace, "workspace", dev), 1 if save else 0)
    return out, hT, workspace


@_streamed
def glr_bwd(x, i_pre, f_pre, a_log, h0, dh, dhT=None, *, fwd_workspace, workspace=None, want_dh0=True, stream=None):
    """Backward of glr_fwd for the loss <dh, out> + <dhT, hT>, reading what
    glr_fwd(save=True) left in fwd_workspace (h0 included).  Returns dict dx,
    di_pre, df_pre (x's dtype), da_log [D] fp32 (fixed-order sum), dh0."""
    import torch
    shape, dt, dev, ptrs = _glr_inputs(x, i_pre, f_pre, a_log, 3)
    B, T, D = shape
    _arg(h0, "h0", dev, torch.float32, (B, D))
    g = dict(dx=torch.empty_like(x), di_pre=torch.empty_like(x), df_pre=torch.empty_like(x),
             da_log=torch.empty_like(a_log),
             dh0=torch.empty((B, D), dtype=torch.float32, device=x.device) if want_dh0 else None)
    if workspace is None:
        workspace = _alloc_ws(glr_workspace_size(KD_GLR_WS_BWD, B, T, D, dt), x.device)
    _call(lib().kron_delta_glr_bwd, dev, *ptrs, _arg(dh, "dh", dev, x.dtype, shape),
          _arg(dhT, "dhT", dev, torch.float32, (B, D)), g["dx"].data_ptr(), g["di_pre"].data_ptr(),
          g["df_pre"].data_ptr(), g["da_log"].data_ptr(), g["dh0"].data_ptr() if want_dh0 else None, B, T, D, dt,
          *_bytes_arg(fwd_workspace, "fwd_workspace", dev), *_bytes_arg(workspace, "workspace", dev))
    return g


@_streamed
def glr_decode(x, i_pre, f_pre, a_log, h, *, out=None, stream=None):
    """One decode step of the gated linear recurrence.  x, i_pre, f_pre [B,D];
    a_log [D] fp32; h [B,D] fp32 (updated in place).  Returns out [B,D]."""
    import torch
    shape, dt, dev, ptrs = _glr_inputs(x, i_pre, f_pre, a_log, 2)
    B, D = shape
    out, p_out = _out(out, x, dev)
    _call(lib().kron_delta_glr_decode, dev, *ptrs, _arg(h, "h", dev, torch.float32, shape),
          p_out, B, D, dt)
    return out


# ---- autograd ------------------------------------------------------------------


def make_rotary_function():
    import torch
    from torch.autograd.function import once_differentiable

    class RotaryFunction(torch.autograd.Function):
        """autograd wrapper of rotary_fwd / rotary_bwd.  apply(q, k, freqs, pos,
        interleaved, scale) -> (q, k); q and k are not changed, k may be None."""

        @staticmethod
        def forward(ctx, q, k, freqs, pos=None, interleaved=False, scale=1.0):
            ctx.save_for_backward(freqs, pos)
            ctx.how = dict(interleaved=interleaved, scale=scale)
            return rotary_fwd(q, k, freqs, pos, **ctx.how)

        @staticmethod
        @once_differentiable
        def backward(ctx, dq, dk):
            freqs, pos = ctx.saved_tensors
            dq, dk = rotary_bwd(dq.contiguous(), None if dk is None else dk.contiguous(), freqs, pos, **ctx.how)
            return dq, dk, None, None, None, None

    return RotaryFunction


def make_swa_function():
    import torch
    from torch.autograd.function import once_differentiable

    class SwaFunction(torch.autograd.Function):
        """autograd wrapper of swa_fwd / swa_bwd.  apply(q, k, v, window, sinks,
        scale) -> out."""

        @staticmethod
        def forward(ctx, q, k, v, window, sinks=0, scale=None):
            out, lse, ws = swa_fwd(q, k, v, window, sinks, scale=scale, save=True)
            ctx.save_for_backward(q, k, v, out, lse, ws)
            ctx.how = (window, sinks, scale)
            return out

        @staticmethod
        @once_differentiable
        def backward(ctx, dO):
            q, k, v, out, lse, ws = ctx.saved_tensors
            window, sinks, scale = ctx.how
            g = swa_bwd(q, k, v, out, lse, dO.contiguous(), window, sinks, scale=scale, fwd_workspace=ws)
            return g["dq"], g["dk"], g["dv"], None, None, None

    return SwaFunction


def make_glr_function():
    import torch
    from torch.autograd.function import once_differentiable

    class GlrFunction(torch.autograd.Function):
        """autograd wrapper of glr_fwd / glr_bwd.  apply(x, i_pre, f_pre, a_log,
        h0) -> (out, hT)."""

        @staticmethod
        def forward(ctx, x, i_pre, f_pre, a_log, h0=None):
            out, hT, ws = glr_fwd(x, i_pre, f_pre, a_log, h0, save=True)
            ctx.save_for_backward(x, i_pre, f_pre, a_log, h0, ws)
            return out, hT

        @staticmethod
        @once_differentiable
        def backward(ctx, dh, dhT):
            x, i_pre, f_pre, a_log, h0, ws = ctx.saved_tensors
            g = glr_bwd(x, i_pre, f_pre, a_log, h0, dh.contiguous(), dhT.contiguous(), fwd_workspace=ws,
                        want_dh0=h0 is not None)
            return g["dx"], g["di_pre"], g["df_pre"], g["da_log"], g["dh0"]

    return GlrFunction
