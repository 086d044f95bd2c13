"""Python front end of the operators that serve a Gated DeltaNet layer (the C ABI in include/gdn_layer.h).

``gdn_prep_fwd`` makes the delta rule's q, k, v, g and beta from a layer's projections,
``gdn_recurrent_fwd`` runs the rule token by token over a pool of states, ``add_rms_norm_fwd`` and
``gated_rms_norm_fwd`` are the norms in front of and behind it, and ``gdn_state_copy`` copies and clears
pool slots.  As in ``api.py``, the functions check shapes and dtypes, allocate what is not given and pass
pointers and the stream; every step of the computation runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _lib
from .api import _IO, _check, _stream_handle, device_status

_OUT = {torch.bfloat16: _lib.GDN_OUT_BF16, torch.float32: _lib.GDN_OUT_F32, torch.float8_e4m3fn: _lib.GDN_OUT_E4M3}


def _empty(shape, dtype, device, stream):
    """A new tensor that belongs to the stream the kernel runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _io(t, name):
    io = _IO.get(t.dtype)
    if io is None:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    return io


def _sequences(cu_seqlens, Bt):
    """(number of sequences, cu_seqlens pointer or None)."""
    if cu_seqlens is None:
        return Bt, None
    if Bt != 1:
        raise ValueError("with cu_seqlens the batch dimension must be 1")
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous 1-D int32 CUDA tensor")
    if cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must hold at least two offsets")
    return cu_seqlens.shape[0] - 1, cu_seqlens.data_ptr()


def _done(rc, what, check, stream):
    if rc != _lib.KKT_OK:
        raise _lib.KktError(rc, what)
    if check is None:
        check = os.environ.get("KKT_CHECK", "0") == "1"
    if check:
        st = device_status(stream)
        if st != _lib.KKT_OK:
            raise _lib.KktError(st, f"{what} (device)")


def gdn_recurrent_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor, state: torch.Tensor, *,
                      g: torch.Tensor | None = None, slots: torch.Tensor | None = None,
                      slots_out: torch.Tensor | None = None, cu_seqlens: torch.Tensor | None = None, scale=None,
                      o: torch.Tensor | None = None, stream=None, check: bool | None = None) -> torch.Tensor:
    """The gated delta rule token by token, over a pool of states that it updates in place: returns o.

    q, k [B, T, Hk, dk], v [B, T, Hv, dv] (bf16 or fp32, all one type; Hv a multiple of Hk, value head h
    uses key head h // (Hv // Hk)), ``beta`` and ``g`` [B, T, Hv] fp32 (``g``: log decays, or None).
    ``state`` [P, Hv, dk, dv] fp32 or bf16: sequence n's state is in slot ``slots[n]`` (int32 on the
    device; None: slot n) and goes back there, or to ``slots_out[n]``.  A negative slot reads as a zero
    state and is not written.  With ``cu_seqlens`` (int32 [N+1] on the device) the tensors are
    [1, T, ...] and hold N packed sequences.  dk and dv are 64 or 128; ``scale`` defaults to dk ** -0.5.
    The result is that of ``chunk_gated_delta_rule`` on the same inputs, in fp32 arithmetic; it takes
    time in proportion to a sequence's length, so prompts go through the chunked form.
    """
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4 or state.dim() != 4:
        raise ValueError("expected q, k [B,T,Hk,dk], v [B,T,Hv,dv], state [P,Hv,dk,dv]")
    Bt, T, Hk, dk = k.shape
    Hv, dv = v.shape[2], v.shape[3]
    io = _io(q, "q")
    _check(q, "q", q.dtype, (Bt, T, Hk, dk))
    _check(k, "k", q.dtype, (Bt, T, Hk, dk))
    _check(v, "v", q.dtype, (Bt, T, Hv, dv))
    _check(beta, "beta", torch.float32, (Bt, T, Hv))
    if g is not None:
        _check(g, "g", torch.float32, (Bt, T, Hv))
    P = state.shape[0]
    st_io = _io(state, "state")
    _check(state, "state", state.dtype, (P, Hv, dk, dv))
    N, cu_ptr = _sequences(cu_seqlens, Bt)
    if slots is not None:
        _check(slots, "slots", torch.int32, (N,))
    if slots_out is not None:
        _check(slots_out, "slots_out", torch.int32, (N,))
    if o is None:
        o = _empty(v.shape, v.dtype, v.device, stream)
    else:
        _check(o, "o", v.dtype, v.shape)
    if scale is None:
        scale = dk ** -0.5
    rc = _lib.lib().gdn_recurrent_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), beta.data_ptr(), _ptr(g), cu_ptr, N, T,
                                      Hk, Hv, dk, dv, float(scale), io, state.data_ptr(), st_io, P, _ptr(slots),
                                      _ptr(slots_out), o.data_ptr(), _stream_handle(stream))
    _done(rc, "gdn_recurrent_fwd", check, stream)
    return o


def gdn_prep_fwd(x: torch.Tensor, weight: torch.Tensor, a: torch.Tensor, b: torch.Tensor, A_log: torch.Tensor,
                 dt_bias: torch.Tensor, conv_state: torch.Tensor, *, Hk: int, Hv: int, dk: int, dv: int,
                 bias: torch.Tensor | None = None, slots: torch.Tensor | None = None,
                 cu_seqlens: torch.Tensor | None = None, expand: bool = False, eps: float = 1e-6, stream=None,
                 check: bool | None = None):
    """From a layer's projections to the delta rule's inputs: returns (q, k, v, g, beta).

    ``x`` [B, T, D] holds each token's channels packed as [q | k | v], D = 2 Hk dk + Hv dv.  The short
    causal convolution ``weight`` [D, taps] (2 to 4 taps, the last one on the token itself) with
    ``bias`` [D] or None runs along each sequence, then SiLU, then the L2 norm (with ``eps``) of each
    head of q and k.  beta = sigmoid(b) and g = -exp(A_log) softplus(a + dt_bias), with ``a``, ``b``
    [B, T, Hv] of x's type and ``A_log``, ``dt_bias`` [Hv] fp32.  ``conv_state`` [P, taps - 1, D] of x's
    type holds the inputs before each sequence's first token, oldest first, in slot ``slots[n]`` (None:
    slot n; negative: zeros, not written), and is updated in place to the sequence's last ones.
    q, k are [B, T, Hk, dk], or with ``expand`` [B, T, Hv, dk], each key head repeated for the value
    heads that use it, as ``chunk_gated_delta_rule`` takes them.  v [B, T, Hv, dv]; g, beta fp32
    [B, T, Hv].  dk = dv = 64 or 128.  ``cu_seqlens`` as in ``gdn_recurrent_fwd``.
    """
    if x.dim() != 3 or weight.dim() != 2 or conv_state.dim() != 3:
        raise ValueError("expected x [B,T,D], weight [D,taps], conv_state [P,taps-1,D]")
    Bt, T, D = x.shape
    if Hk < 1 or Hv < 1 or D != 2 * Hk * dk + Hv * dv:
        raise ValueError(f"x must have 2 Hk dk + Hv dv = {2 * Hk * dk + Hv * dv} channels, got {D}")
    taps = weight.shape[1]
    io = _io(x, "x")
    _check(x, "x", x.dtype, (Bt, T, D))
    _check(weight, "weight", x.dtype, (D, taps))
    if bias is not None:
        _check(bias, "bias", x.dtype, (D,))
    _check(a, "a", x.dtype, (Bt, T, Hv))
    _check(b, "b", x.dtype, (Bt, T, Hv))
    _check(A_log, "A_log", torch.float32, (Hv,))
    _check(dt_bias, "dt_bias", torch.float32, (Hv,))
    P = conv_state.shape[0]
    _check(conv_state, "conv_state", x.dtype, (P, taps - 1, D))
    N, cu_ptr = _sequences(cu_seqlens, Bt)
    if slots is not None:
        _check(slots, "slots", torch.int32, (N,))
    Hq = Hv if expand else Hk
    q = _empty((Bt, T, Hq, dk), x.dtype, x.device, stream)
    k = _empty((Bt, T, Hq, dk), x.dtype, x.device, stream)
    v = _empty((Bt, T, Hv, dv), x.dtype, x.device, stream)
    g = _empty((Bt, T, Hv), torch.float32, x.device, stream)
    beta = _empty((Bt, T, Hv), torch.float32, x.device, stream)
    rc = _lib.lib().gdn_prep_fwd(x.data_ptr(), weight.data_ptr(), _ptr(bias), a.data_ptr(), b.data_ptr(),
                                 A_log.data_ptr(), dt_bias.data_ptr(), cu_ptr, N, T, Hk, Hv, dk, dv, taps, float(eps),
                                 int(expand), io, conv_state.data_ptr(), P, _ptr(slots), q.data_ptr(), k.data_ptr(),
                                 v.data_ptr(), g.data_ptr(), beta.data_ptr(), _stream_handle(stream))
    _done(rc, "gdn_prep_fwd", check, stream)
    return q, k, v, g, beta


def _out_type(out_dtype, like):
    out = like if out_dtype is None else out_dtype
    code = _OUT.get(out)
    if code is None:
        raise ValueError(f"out_dtype must be torch.bfloat16, torch.float32 or torch.float8_e4m3fn, got {out}")
    return out, code


def add_rms_norm_fwd(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, *, eps: float = 1e-6,
                     out_dtype=None, group: int | None = 128, residual_out: torch.Tensor | None = None, stream=None,
                     check: bool | None = None):
    """Root-mean-square norm of x + residual over the last dimension: returns (y, scales, residual_out).

    x and ``residual`` [..., dim], ``weight`` [dim], bf16 or fp32, all one type.  The sum is normalised
    as it is in fp32 and returned rounded to x's type as ``residual_out`` (pass ``residual`` itself to
    update it in place; None without a residual).  ``out_dtype``: x's type by default, torch.bfloat16,
    torch.float32, or torch.float8_e4m3fn with ``scales`` fp32 [..., ceil(dim / 128)], one for each
    ``group`` of 128 values (``group=None``: one a row, [...]): y * scale is the norm's result.
    """
    if x.dim() < 1:
        raise ValueError("expected x [..., dim]")
    dim = x.shape[-1]
    io = _io(x, "x")
    _check(x, "x", x.dtype, x.shape)
    _check(weight, "weight", x.dtype, (dim,))
    if residual is not None:
        _check(residual, "residual", x.dtype, x.shape)
        if residual_out is None:
            residual_out = _empty(x.shape, x.dtype, x.device, stream)
    elif residual_out is not None:
        raise ValueError("residual_out given without a residual")
    if residual_out is not None:
        _check(residual_out, "residual_out", x.dtype, x.shape)
    out, code = _out_type(out_dtype, x.dtype)
    if group not in (None, 128):
        raise ValueError(f"group must be 128 or None, got {group}")
    rows = x.numel() // dim if dim else 0
    y = _empty(x.shape, out, x.device, stream)
    scales = None
    if code == _lib.GDN_OUT_E4M3:
        scales = _empty(x.shape[:-1] if group is None else (*x.shape[:-1], -(-dim // 128)), torch.float32, x.device,
                        stream)
    rc = _lib.lib().add_rms_norm_fwd(x.data_ptr(), _ptr(residual), weight.data_ptr(), rows, dim, float(eps), io, code,
                                     group or 0, y.data_ptr(), _ptr(scales), _ptr(residual_out),
                                     _stream_handle(stream))
    _done(rc, "add_rms_norm_fwd", check, stream)
    return y, scales, residual_out


def gated_rms_norm_fwd(x: torch.Tensor, z: torch.Tensor, weight: torch.Tensor, *, eps: float = 1e-6, out_dtype=None,
                       stream=None, check: bool | None = None):
    """Root-mean-square norm of each head's output times silu(z): returns (y, scales).

    x (the delta rule's o) and ``z`` [..., d], ``weight`` [d], bf16 or fp32, all one type; d is 64 or
    128.  ``out_dtype`` as in ``add_rms_norm_fwd``; in 8 bits ``scales`` [...] fp32 holds one for each
    head of each token.
    """
    if x.dim() < 1:
        raise ValueError("expected x [..., d]")
    dim = x.shape[-1]
    io = _io(x, "x")
    _check(x, "x", x.dtype, x.shape)
    _check(z, "z", x.dtype, x.shape)
    _check(weight, "weight", x.dtype, (dim,))
    out, code = _out_type(out_dtype, x.dtype)
    y = _empty(x.shape, out, x.device, stream)
    scales = _empty(x.shape[:-1], torch.float32, x.device, stream) if code == _lib.GDN_OUT_E4M3 else None
    rc = _lib.lib().gated_rms_norm_fwd(x.data_ptr(), z.data_ptr(), weight.data_ptr(), x.numel() // dim if dim else 0,
                                       dim, float(eps), io, code, y.data_ptr(), _ptr(scales), _stream_handle(stream))
    _done(rc, "gated_rms_norm_fwd", check, stream)
    return y, scales


def _copy_side(tensors, name):
    """Tensors [P, ...] of one slot count whose slots are contiguous: (pointers, slot bytes, strides, P)."""
    P = tensors[0].shape[0] if tensors[0].dim() else 0
    ptrs, size, stride = [], [], []
    for t in tensors:
        if not t.is_cuda or t.dim() < 2 or t.shape[0] != P:
            raise ValueError(f"{name} must be CUDA tensors [P, ...] with one slot count P")
        e = t.element_size()
        n = t.numel() // P if P else 0
        if P and (n == 0 or not t[0].is_contiguous() or (P > 1 and t.stride(0) < n)):
            raise ValueError(f"{name} must have contiguous, non-empty slots that do not overlap")
        ptrs.append(t.data_ptr())
        size.append(n * e)
        stride.append(max(t.stride(0), n) * e)
    return ptrs, size, stride, P


def gdn_state_copy(dst, dst_slots: torch.Tensor, src=None, src_slots: torch.Tensor | None = None, *, stream=None,
                   check: bool | None = None) -> None:
    """Copies slots of pools: for every tensor of the list and every m, dst[dst_slots[m]] = src[src_slots[m]].

    ``dst`` and ``src``: a tensor [P, ...] or a list of up to 64 of them (``src`` may be the same list),
    paired in order, of equal slot shapes and types; slots may be strided (a layer's part of a larger
    tensor) but are contiguous in themselves.  ``dst_slots`` and ``src_slots`` are int32 on the device.
    A negative source, or ``src`` None, clears the slot to zeros; a negative destination is skipped.
    Naming a source twice forks it.  No two moves may share a destination, and none may write a slot
    that another one of the call reads.
    """
    dst = [dst] if isinstance(dst, torch.Tensor) else list(dst)
    if not 1 <= len(dst) <= _lib.GDN_COPY_MAX_TENSORS:
        raise ValueError(f"1 to {_lib.GDN_COPY_MAX_TENSORS} tensors, got {len(dst)}")
    dp, size, ds, P = _copy_side(dst, "dst")
    _check(dst_slots, "dst_slots", torch.int32, (dst_slots.numel(),))
    n = len(dst)
    src_ptr = src_stride_ptr = src_slots_ptr = None
    Ps = 0
    if src is not None:
        src = [src] if isinstance(src, torch.Tensor) else list(src)
        if src_slots is None:
            raise ValueError("src given without src_slots")
        _check(src_slots, "src_slots", torch.int32, tuple(dst_slots.shape))
        if len(src) != n:
            raise ValueError(f"{n} destination tensors and {len(src)} sources")
        for d, s in zip(dst, src):
            if d.dtype != s.dtype or d.shape[1:] != s.shape[1:]:
                raise ValueError("a source's slots must have the shape and type of its destination's")
        sp, _, ss, Ps = _copy_side(src, "src")
        src_arr, ss_arr = (ctypes.c_void_p * n)(*sp), (ctypes.c_size_t * n)(*ss)
        src_ptr, src_stride_ptr = ctypes.addressof(src_arr), ctypes.addressof(ss_arr)
        src_slots_ptr = src_slots.data_ptr()
    elif src_slots is not None:
        raise ValueError("src_slots given without src")
    if P == 0 or dst_slots.numel() == 0:
        return
    dst_arr, size_arr, ds_arr = (ctypes.c_void_p * n)(*dp), (ctypes.c_size_t * n)(*size), (ctypes.c_size_t * n)(*ds)
    rc = _lib.lib().gdn_state_copy(ctypes.addressof(dst_arr), src_ptr, ctypes.addressof(size_arr),
                                   ctypes.addressof(ds_arr), src_stride_ptr, n, dst_slots.data_ptr(), src_slots_ptr,
                                   dst_slots.numel(), P, Ps, _stream_handle(stream))
    _done(rc, "gdn_state_copy", check, stream)
