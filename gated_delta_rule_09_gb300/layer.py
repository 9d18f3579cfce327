"""The operators around the recurrence: short causal convolution, selective
state space scan (prompts and single tokens) and group norm.

Marshalling only, as in the package's main module: the compute is in libgdn.so
(``include/gdn.h`` has the contract of each call).  Activations may be slices
of wider rows (unit stride along the channels, one stride between rows);
parameters are contiguous fp32.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib

_DTYPES = {torch.float32: _lib.GDN_F32, torch.bfloat16: _lib.GDN_BF16}
_ACTS = {"none": _lib.GDN_ACT_NONE, "silu": _lib.GDN_ACT_SILU}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _cuda(name, t):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)


def _on(name, t, dtype, device):
    _cuda(name, t)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, x on %s" % (name, t.device, device))


def _param(name, t, dtype, device, shape):
    """A contiguous parameter or state of the given shape (None allowed)."""
    if t is None:
        return
    _on(name, t, dtype, device)
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _rows(name, t, dtype, device, shape, inner=1):
    """Row stride in elements of a matrix argument whose last ``inner``
    dimensions are a row and whose others count rows one stride apart."""
    _on(name, t, dtype, device)
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    size, stride = t.shape, t.stride()
    width = 1
    for k in range(len(size) - 1, len(size) - 1 - inner, -1):
        if size[k] > 1 and stride[k] != width:
            raise ValueError("%s: the channels of a row must be contiguous" % name)
        width *= size[k]
    ld, rows = width, 1
    for k in range(len(size) - 1 - inner, -1, -1):
        if size[k] == 0:
            return width
        if size[k] > 1:
            if rows == 1:
                ld = stride[k]
            elif stride[k] != rows * ld:
                raise ValueError("%s: rows must be one stride apart" % name)
            rows *= size[k]
    if rows > 1 and ld < width:
        raise ValueError("%s: rows overlap" % name)
    return ld


def _stream(stream, device):
    """(raw handle, context in which to allocate for it): what a call allocates
    belongs to the stream that its kernels run on."""
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream, contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return stream.cuda_stream, torch.cuda.stream(stream)


def _device(device):
    if torch.cuda.current_device() == device.index:
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _act(act):
    if act not in _ACTS:
        raise ValueError("act must be one of %s, got %r" % (sorted(_ACTS), act))
    return _ACTS[act]


def _first(x, dims, layout):
    """Checks of the argument that fixes type, device and sizes."""
    _cuda("x", x)
    if x.dtype not in _DTYPES:
        raise TypeError("x must be float32 or bfloat16, got %s" % x.dtype)
    if x.dim() != dims:
        raise ValueError("x must be %s" % layout)


def _sequences(x, cu_seqlens):
    """Number of sequences of a prompt call and tokens per sequence (or of the pack)."""
    B, T = x.shape[:2]
    if cu_seqlens is None:
        return B, T
    _on("cu_seqlens", cu_seqlens, torch.int32, x.device)
    if B != 1:
        raise ValueError("packed (cu_seqlens) inputs must have B == 1")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous 1-D int32 tensor of N + 1 >= 2 offsets")
    return cu_seqlens.numel() - 1, T


def _states(state_in, state_out, slots, N, entry, dtype, device, want, alloc):
    """Checked pools and the number of their entries; ``state_out`` is filled
    in: the pool itself in place when slots address it, else a new tensor."""
    pool = N
    if slots is not None:
        _param("slots", slots, torch.int32, device, (N,))
        given = state_in if state_in is not None else state_out
        if given is None:
            if want:
                raise ValueError("slots need a pool of states (state_in or state_out)")
            return None, 0
        if not isinstance(given, torch.Tensor) or given.dim() != 1 + len(entry):
            raise ValueError("a pool of states must be [pool, %s]" % ", ".join(map(str, entry)))
        pool = given.shape[0]
    shape = (pool,) + entry
    _param("state_in", state_in, dtype, device, shape)
    _param("state_out", state_out, dtype, device, shape)
    if state_out is None and want:
        if slots is not None:
            state_out = state_in
        else:
            with alloc:
                state_out = torch.empty(shape, dtype=dtype, device=device)
    return state_out, pool


def _out(name, y, x, alloc):
    if y is None:
        with alloc:
            return torch.empty(x.shape, dtype=x.dtype, device=x.device)
    return y


def gdn_conv_fwd(x, weight, bias=None, state_in=None, y=None, state_out=None, slots=None,
                 cu_seqlens=None, act="silu", stream=None, want_final_state=True):
    """Short causal depthwise convolution over prompts; returns ``(y, state_out)``.

    x [B,T,C] (fp32 or bf16); weight [C,W] and bias [C] fp32, 1 <= W <= 8;
    y[t] = act(bias + sum_j weight[:, j] x[t - (W - 1) + j]).  The inputs ahead
    of a sequence come from ``state_in`` [N,W-1,C] (x's dtype, oldest first),
    zeros if None; ``state_out`` receives the last W - 1 inputs and may be
    ``state_in``.  With ``slots`` (int32 [N]) the states are pools
    [pool,W-1,C] and sequence n uses entry slots[n] (negative: no state),
    updated in place unless ``state_out`` is another pool.  ``cu_seqlens``
    (int32 [N+1]) packs N sequences into B == 1.  ``act`` is "silu" or "none".
    """
    _first(x, 3, "[B,T,C]")
    C, dev = x.shape[2], x.device
    N, T = _sequences(x, cu_seqlens)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [C,W]")
    W = weight.shape[1]
    _param("weight", weight, torch.float32, dev, (C, W))
    _param("bias", bias, torch.float32, dev, (C,))
    code = _act(act)
    handle, alloc = _stream(stream, dev)
    ld_x = _rows("x", x, x.dtype, dev, x.shape)
    lib = _lib.load()
    with _device(dev):
        state_out, pool = _states(state_in, state_out, slots, N, (W - 1, C), x.dtype, dev,
                                  want_final_state, alloc)
        y = _out("y", y, x, alloc)
        ld_y = _rows("y", y, x.dtype, dev, x.shape)
        _lib.check(lib.gdn_conv_fwd(
            _ptr(x), _ptr(weight), _ptr(bias), _ptr(state_in), _ptr(slots), _ptr(y),
            _ptr(state_out), N, T, C, W, ld_x, ld_y, pool, _ptr(cu_seqlens), code,
            _DTYPES[x.dtype], handle))
    return y, state_out


def gdn_conv_step(x, weight, bias=None, state_in=None, y=None, state_out=None, slots=None,
                  act="silu", stream=None):
    """``gdn_conv_fwd`` for one new token per sequence: x, y [N,C]; returns
    ``(y, state_out)``.  States as there; ``state_out`` may be ``state_in``."""
    _first(x, 2, "[N,C]")
    (N, C), dev = x.shape, x.device
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [C,W]")
    W = weight.shape[1]
    _param("weight", weight, torch.float32, dev, (C, W))
    _param("bias", bias, torch.float32, dev, (C,))
    code = _act(act)
    handle, alloc = _stream(stream, dev)
    ld_x = _rows("x", x, x.dtype, dev, x.shape)
    lib = _lib.load()
    with _device(dev):
        state_out, pool = _states(state_in, state_out, slots, N, (W - 1, C), x.dtype, dev, True, alloc)
        y = _out("y", y, x, alloc)
        ld_y = _rows("y", y, x.dtype, dev, x.shape)
        _lib.check(lib.gdn_conv_step(
            _ptr(x), _ptr(weight), _ptr(bias), _ptr(state_in), _ptr(slots), _ptr(y),
            _ptr(state_out), N, C, W, ld_x, ld_y, pool, code, _DTYPES[x.dtype], handle))
    return y, state_out


def _ssm_params(x, delta, A, B, C, D, z, delta_bias):
    """Checks shared by scan and step; returns (d_state, groups, row strides)."""
    ch, dt, dev = x.shape[-1], x.dtype, x.device
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be [C,d_state]")
    if not isinstance(B, torch.Tensor) or B.dim() != x.dim() + 1:
        raise ValueError("B and C must be [..., groups, d_state]")
    S, G = A.shape[1], B.shape[-2]
    _param("A", A, torch.float32, dev, (ch, S))
    _param("D", D, torch.float32, dev, (ch,))
    _param("delta_bias", delta_bias, torch.float32, dev, (ch,))
    bc = tuple(x.shape[:-1]) + (G, S)
    lds = [_rows("x", x, dt, dev, x.shape), _rows("delta", delta, dt, dev, x.shape),
           _rows("B", B, dt, dev, bc, 2), _rows("C", C, dt, dev, bc, 2),
           0 if z is None else _rows("z", z, dt, dev, x.shape)]
    return S, G, lds


def gdn_ssm_fwd(x, delta, A, B, C, D=None, z=None, delta_bias=None, state_in=None, y=None,
                state_out=None, slots=None, cu_seqlens=None, delta_softplus=False, segment=0,
                workspace=None, stream=None, want_final_state=True):
    """Selective state space scan over prompts; returns ``(y, state_out)``.

    x, delta, z, y [b,T,ch] and B, C [b,T,groups,S] (fp32 or bf16, one dtype);
    A [ch,S], D and delta_bias [ch] fp32.  With d = delta + delta_bias
    (softplus of it if ``delta_softplus``), per channel and token
    h = exp(d A) h + d B x, y = (C h + D x) silu(z).  States are fp32
    [N,ch,S], or pools addressed by ``slots``, as in ``gdn_conv_fwd``.
    ``segment`` is the length in tokens of the pieces that long sequences are
    cut into (0: chosen by the library); ``workspace`` a uint8 CUDA tensor of
    ``gdn_ssm_fwd_workspace_size(...)`` bytes, allocated here if None.
    """
    _first(x, 3, "[b,T,ch]")
    ch, dev = x.shape[2], x.device
    N, T = _sequences(x, cu_seqlens)
    S, G, lds = _ssm_params(x, delta, A, B, C, D, z, delta_bias)
    handle, alloc = _stream(stream, dev)
    lib = _lib.load()
    with _device(dev):
        state_out, pool = _states(state_in, state_out, slots, N, (ch, S), torch.float32, dev,
                                  want_final_state, alloc)
        y = _out("y", y, x, alloc)
        lds.append(_rows("y", y, x.dtype, dev, x.shape))
        need = lib.gdn_ssm_fwd_workspace_size(N, T, ch, S, _ptr(cu_seqlens), int(segment))
        if workspace is None and need:
            with alloc:
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        if workspace is not None:
            _on("workspace", workspace, torch.uint8, dev)
        _lib.check(lib.gdn_ssm_fwd(
            _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
            _ptr(state_in), _ptr(slots), _ptr(y), _ptr(state_out), N, T, ch, S, G, *lds, pool,
            _ptr(cu_seqlens), bool(delta_softplus), _DTYPES[x.dtype], int(segment),
            _ptr(workspace), 0 if workspace is None else workspace.numel(), handle))
    return y, state_out


def gdn_ssm_fwd_workspace_size(N, T, channels, d_state, packed=False, segment=0):
    """Bytes of device workspace ``gdn_ssm_fwd`` needs for N sequences of T
    tokens (``packed``: T rows in all); 0 when it needs none."""
    marker = 1 if packed else None  # only NULL-ness reaches the library
    return int(_lib.load().gdn_ssm_fwd_workspace_size(N, T, channels, d_state, marker, int(segment)))


def gdn_ssm_step(x, delta, A, B, C, D=None, z=None, delta_bias=None, state_in=None, y=None,
                 state_out=None, slots=None, delta_softplus=False, stream=None):
    """``gdn_ssm_fwd`` for one new token per sequence: x, delta, z, y [N,ch],
    B, C [N,groups,S]; returns ``(y, state_out)``; ``state_out`` may be
    ``state_in``."""
    _first(x, 2, "[N,ch]")
    (N, ch), dev = x.shape, x.device
    S, G, lds = _ssm_params(x, delta, A, B, C, D, z, delta_bias)
    handle, alloc = _stream(stream, dev)
    lib = _lib.load()
    with _device(dev):
        state_out, pool = _states(state_in, state_out, slots, N, (ch, S), torch.float32, dev, True, alloc)
        y = _out("y", y, x, alloc)
        lds.append(_rows("y", y, x.dtype, dev, x.shape))
        _lib.check(lib.gdn_ssm_step(
            _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
            _ptr(state_in), _ptr(slots), _ptr(y), _ptr(state_out), N, ch, S, G, *lds, pool,
            bool(delta_softplus), _DTYPES[x.dtype], handle))
    return y, state_out


def gdn_group_norm(x, groups, weight=None, bias=None, gate=None, y=None, eps=1e-5, rms=False,
                   act="none", stream=None):
    """Group norm of token rows, channels last; returns ``y``.

    x, gate, y [..., C] (fp32 or bf16); the C channels of a row are cut into
    ``groups`` runs (a head's outputs), each normalised by its own mean and
    variance (``rms``: by its root mean square):
    y = act(u weight + bias) silu(gate).  weight, bias [C] fp32.  ``y`` may be
    ``x`` or ``gate``.
    """
    _cuda("x", x)
    if x.dtype not in _DTYPES:
        raise TypeError("x must be float32 or bfloat16, got %s" % x.dtype)
    if x.dim() < 1:
        raise ValueError("x must be [..., C]")
    C, dev = x.shape[-1], x.device
    rows = x.numel() // C if C else 0
    _param("weight", weight, torch.float32, dev, (C,))
    _param("bias", bias, torch.float32, dev, (C,))
    code = _act(act)
    handle, alloc = _stream(stream, dev)
    ld_x = _rows("x", x, x.dtype, dev, x.shape)
    ld_g = 0 if gate is None else _rows("gate", gate, x.dtype, dev, x.shape)
    lib = _lib.load()
    with _device(dev):
        y = _out("y", y, x, alloc)
        ld_y = _rows("y", y, x.dtype, dev, x.shape)
        _lib.check(lib.gdn_group_norm(
            _ptr(x), _ptr(gate), _ptr(weight), _ptr(bias), _ptr(y), rows, C, int(groups), ld_x,
            ld_g, ld_y, float(eps), bool(rms), code, _DTYPES[x.dtype], handle))
    return y
