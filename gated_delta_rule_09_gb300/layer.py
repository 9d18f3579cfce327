"""The operators around the recurrence: short causal convolution, selective
state space scan (prompts and single tokens) and group norm.

Marshalling only, as in the package's main module: the compute is in libgdn.so
(``include/gdn.h`` has the contract of each call).  Activations may be slices
of wider rows (unit stride along the channels, one stride between rows);
parameters are contiguous fp32.
"""
from __future__ import annotations

import torch

from . import _lib

_DTYPES = {torch.float32: _lib.GDN_F32, torch.bfloat16: _lib.GDN_BF16}
_ACTS = {"none": _lib.GDN_ACT_NONE, "silu": _lib.GDN_ACT_SILU}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _cuda(name, t):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)


def _on(name, t, dtype, index):
    """Type and device (by number) of an argument; x's are those of the call."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != index:
        raise ValueError("%s is on %s, x on device %d" % (name, t.device, index))


def _param(name, t, dtype, index, shape):
    """A contiguous parameter or state of the given shape."""
    _on(name, t, dtype, index)
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _rows(name, t, dtype, index, shape, inner=1):
    """Row stride in elements of a matrix argument whose last ``inner``
    dimensions are a row and whose others count rows one stride apart."""
    _on(name, t, dtype, index)
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    if t.is_contiguous():
        return shape[-1] if inner == 1 else shape[-1] * shape[-2]
    size, stride = shape, t.stride()
    width = 1
    for k in range(len(size) - 1, len(size) - 1 - inner, -1):
        if size[k] > 1 and stride[k] != width:
            raise ValueError("%s: the channels of a row must be contiguous" % name)
        width *= size[k]
    ld, rows = width, 1
    for k in range(len(size) - 1 - inner, -1, -1):
        if size[k] > 1:
            if rows == 1:
                ld = stride[k]
            elif stride[k] != rows * ld:
                raise ValueError("%s: rows must be one stride apart" % name)
            rows *= size[k]
    if rows > 1 and ld < width:
        raise ValueError("%s: rows overlap" % name)
    return ld


def _empty(stream, like, shape=None, dtype=None):
    """A new tensor that belongs to the stream the call runs on."""
    if stream is None:
        if shape is None:
            return torch.empty_like(like, memory_format=torch.contiguous_format)
        return like.new_empty(shape, dtype=dtype)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    with torch.cuda.stream(stream):
        return _empty(None, like, shape, dtype)


def _handle(stream, index):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return getattr(stream, "cuda_stream", stream)


def _call(fn, index, *args):
    """One library call on the device of its tensors."""
    if torch._C._cuda_getDevice() == index:
        status = fn(*args)
    else:
        with torch.cuda.device(index):
            status = fn(*args)
    if status:
        _lib.check(status)


def _act(act):
    if act not in _ACTS:
        raise ValueError("act must be one of %s, got %r" % (sorted(_ACTS), act))
    return _ACTS[act]


def _first(x, dims, layout):
    """The argument that fixes sizes, type and device: (shape, dtype, device number)."""
    _cuda("x", x)
    dtype = x.dtype
    if dtype not in _DTYPES:
        raise TypeError("x must be float32 or bfloat16, got %s" % dtype)
    if x.dim() != dims:
        raise ValueError("x must be %s" % layout)
    return x.shape, dtype, x.get_device()


def _sequences(shape, cu_seqlens, index):
    """Number of sequences of a prompt call and tokens per sequence (or of the pack)."""
    B, T = shape[:2]
    if cu_seqlens is None:
        return B, T
    _on("cu_seqlens", cu_seqlens, torch.int32, index)
    if B != 1:
        raise ValueError("packed (cu_seqlens) inputs must have B == 1")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous 1-D int32 tensor of N + 1 >= 2 offsets")
    return cu_seqlens.numel() - 1, T


def _states(state_in, state_out, slots, N, entry, dtype, index, want, x, stream):
    """Checked pools and the number of their entries; ``state_out`` is filled
    in: the pool itself in place when slots address it, else a new tensor."""
    pool = N
    if slots is not None:
        _param("slots", slots, torch.int32, index, (N,))
        given = state_in if state_in is not None else state_out
        if given is None:
            if want:
                raise ValueError("slots need a pool of states (state_in or state_out)")
            return None, 0
        if not isinstance(given, torch.Tensor) or given.dim() != 1 + len(entry):
            raise ValueError("a pool of states must be [pool, %s]" % ", ".join(map(str, entry)))
        pool = given.shape[0]
    shape = (pool,) + entry
    if state_in is not None:
        _param("state_in", state_in, dtype, index, shape)
    if state_out is not None:
        _param("state_out", state_out, dtype, index, shape)
    elif want:
        state_out = state_in if slots is not None else _empty(stream, x, shape, dtype)
    return state_out, pool


def _taps(weight, bias, C, index):
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [C,W]")
    W = weight.shape[1]
    _param("weight", weight, torch.float32, index, (C, W))
    if bias is not None:
        _param("bias", bias, torch.float32, index, (C,))
    return W


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
    shape, dtype, index = _first(x, 3, "[B,T,C]")
    C = shape[2]
    N, T = _sequences(shape, cu_seqlens, index)
    W = _taps(weight, bias, C, index)
    ld_x = _rows("x", x, dtype, index, shape)
    code = _act(act)
    fn = _lib.load().gdn_conv_fwd
    state_out, pool = _states(state_in, state_out, slots, N, (W - 1, C), dtype, index,
                              want_final_state, x, stream)
    if y is None:
        y, ld_y = _empty(stream, x), C
    else:
        ld_y = _rows("y", y, dtype, index, shape)
    _call(fn, index, _ptr(x), _ptr(weight), _ptr(bias), _ptr(state_in), _ptr(slots), _ptr(y),
          _ptr(state_out), N, T, C, W, ld_x, ld_y, pool, _ptr(cu_seqlens), code, _DTYPES[dtype],
          _handle(stream, index))
    return y, state_out


def gdn_conv_step(x, weight, bias=None, state_in=None, y=None, state_out=None, slots=None,
                  act="silu", stream=None):
    """``gdn_conv_fwd`` for one new token per sequence: x, y [N,C]; returns
    ``(y, state_out)``.  States as there; ``state_out`` may be ``state_in``."""
    shape, dtype, index = _first(x, 2, "[N,C]")
    N, C = shape
    W = _taps(weight, bias, C, index)
    ld_x = _rows("x", x, dtype, index, shape)
    code = _act(act)
    fn = _lib.load().gdn_conv_step
    state_out, pool = _states(state_in, state_out, slots, N, (W - 1, C), dtype, index, True, x, stream)
    if y is None:
        y, ld_y = _empty(stream, x), C
    else:
        ld_y = _rows("y", y, dtype, index, shape)
    _call(fn, index, _ptr(x), _ptr(weight), _ptr(bias), _ptr(state_in), _ptr(slots), _ptr(y),
          _ptr(state_out), N, C, W, ld_x, ld_y, pool, code, _DTYPES[dtype], _handle(stream, index))
    return y, state_out


def _ssm_params(x, shape, dtype, index, delta, A, B, C, D, z, delta_bias):
    """Checks shared by scan and step: (d_state, groups, row strides of x, delta, B, C, z)."""
    ch = shape[-1]
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be [C,d_state]")
    if not isinstance(B, torch.Tensor) or B.dim() != len(shape) + 1:
        raise ValueError("B and C must be [..., groups, d_state]")
    S, G = A.shape[1], B.shape[-2]
    _param("A", A, torch.float32, index, (ch, S))
    if D is not None:
        _param("D", D, torch.float32, index, (ch,))
    if delta_bias is not None:
        _param("delta_bias", delta_bias, torch.float32, index, (ch,))
    bc = shape[:-1] + (G, S)
    return (S, G, _rows("x", x, dtype, index, shape), _rows("delta", delta, dtype, index, shape),
            _rows("B", B, dtype, index, bc, 2), _rows("C", C, dtype, index, bc, 2),
            0 if z is None else _rows("z", z, dtype, index, shape))


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
    shape, dtype, index = _first(x, 3, "[b,T,ch]")
    ch = shape[2]
    N, T = _sequences(shape, cu_seqlens, index)
    S, G, ld_x, ld_d, ld_b, ld_c, ld_z = _ssm_params(x, shape, dtype, index, delta, A, B, C, D, z, delta_bias)
    lib = _lib.load()
    state_out, pool = _states(state_in, state_out, slots, N, (ch, S), torch.float32, index,
                              want_final_state, x, stream)
    if y is None:
        y, ld_y = _empty(stream, x), ch
    else:
        ld_y = _rows("y", y, dtype, index, shape)
    segment = int(segment)
    if workspace is None:
        need = lib.gdn_ssm_fwd_workspace_size(N, T, ch, S, _ptr(cu_seqlens), segment)
        if need:
            workspace = _empty(stream, x, (need,), torch.uint8)
    else:
        _on("workspace", workspace, torch.uint8, index)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    _call(lib.gdn_ssm_fwd, index, _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
          _ptr(delta_bias), _ptr(state_in), _ptr(slots), _ptr(y), _ptr(state_out), N, T, ch, S, G,
          ld_x, ld_d, ld_b, ld_c, ld_z, ld_y, pool, _ptr(cu_seqlens), bool(delta_softplus),
          _DTYPES[dtype], segment, _ptr(workspace), 0 if workspace is None else workspace.numel(),
          _handle(stream, index))
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
    shape, dtype, index = _first(x, 2, "[N,ch]")
    N, ch = shape
    S, G, ld_x, ld_d, ld_b, ld_c, ld_z = _ssm_params(x, shape, dtype, index, delta, A, B, C, D, z, delta_bias)
    fn = _lib.load().gdn_ssm_step
    state_out, pool = _states(state_in, state_out, slots, N, (ch, S), torch.float32, index, True, x, stream)
    if y is None:
        y, ld_y = _empty(stream, x), ch
    else:
        ld_y = _rows("y", y, dtype, index, shape)
    _call(fn, index, _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
          _ptr(delta_bias), _ptr(state_in), _ptr(slots), _ptr(y), _ptr(state_out), N, ch, S, G, ld_x,
          ld_d, ld_b, ld_c, ld_z, ld_y, pool, bool(delta_softplus), _DTYPES[dtype],
          _handle(stream, index))
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
    shape, dtype, index = x.shape, x.dtype, x.get_device()
    if dtype not in _DTYPES:
        raise TypeError("x must be float32 or bfloat16, got %s" % dtype)
    if len(shape) < 1:
        raise ValueError("x must be [..., C]")
    C = shape[-1]
    if weight is not None:
        _param("weight", weight, torch.float32, index, (C,))
    if bias is not None:
        _param("bias", bias, torch.float32, index, (C,))
    code = _act(act)
    ld_x = _rows("x", x, dtype, index, shape)
    ld_g = 0 if gate is None else _rows("gate", gate, dtype, index, shape)
    fn = _lib.load().gdn_group_norm
    if y is None:
        y, ld_y = _empty(stream, x), C
    else:
        ld_y = _rows("y", y, dtype, index, shape)
    _call(fn, index, _ptr(x), _ptr(gate), _ptr(weight), _ptr(bias), _ptr(y), x.numel() // C if C else 0,
          C, int(groups), ld_x, ld_g, ld_y, float(eps), bool(rms), code, _DTYPES[dtype],
          _handle(stream, index))
    return y
