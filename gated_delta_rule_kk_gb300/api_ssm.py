"""Python entry points of the short causal convolution and the state space scan.

As in ``api.py``: torch tensors in, library call, tensors out; argument
marshalling only.  Token tensors may be column ranges of wider buffers (their
last dimensions dense, rows any stride apart), so nothing has to be copied
between an input projection, the convolution and the scan.  Outputs belong to
``stream`` (the current one by default), as tensors made under it do.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib
from ._lib import ShortConvArgs, ShortConvBwdArgs, ShortConvDecodeArgs, SsmChunkArgs, SsmDecodeArgs

_F32, _BF16 = torch.float32, torch.bfloat16
_CODE = {_F32: 0, _BF16: 1}
_ACTIVATIONS = {None: 0, "silu": 1}

# A call for one token is a few microseconds on the GPU, so the checks below
# read each tensor property once, and the stream's handle comes without a
# Stream object around it where PyTorch offers that (0.1 us instead of 3), as
# does the current device.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream_handle(stream, device):
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream must be one of {device}, where the tensors are, got one of "
                             f"{stream.device}")
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _empty(size, dtype, device, stream):
    """An output or workspace, from the pool of the stream that writes it."""
    if stream is None:
        return torch.empty(size, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(size, dtype=dtype, device=device)


def _misfit(t, name, dtype, device, shape, dense="dense rows"):
    return ValueError(f"{name} must be a {dtype} tensor of shape {list(shape)} with {dense} on "
                      f"{device}, got {t.dtype} {list(t.shape)} with strides {list(t.stride())} "
                      f"on {t.device}")


def _first(x, name, dims):
    """Dtype code and device of a call's first tensor, which the others follow."""
    code = _CODE.get(x.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16, got {x.dtype}")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, got one on {x.device}")
    if x.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {list(x.shape)}")
    return code, x.device


def _rows(t, name, dtype, device, shape):
    """Token and batch stride of a tensor [B, T, D] whose rows are dense."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        raise _misfit(t, name, dtype, device, shape)
    sb, st, sd = t.stride()
    if sd != 1 and shape[2] != 1:
        raise _misfit(t, name, dtype, device, shape)
    # the stride over a single token is never used
    return st if shape[1] > 1 or st > shape[2] else shape[2], sb


def _heads(t, name, dtype, device, shape):
    """Token and batch stride of a tensor [B, T, H, V] whose [H, V] rows are dense."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        raise _misfit(t, name, dtype, device, shape)
    sb, st, sh, sv = t.stride()
    if (sv != 1 and shape[3] != 1) or (sh != shape[3] and shape[2] != 1):
        raise _misfit(t, name, dtype, device, shape)
    row = shape[2] * shape[3]
    return st if shape[1] > 1 or st > row else row, sb


def _flat(t, name, dtype, device, shape):
    """A contiguous tensor's address, None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.device != device or t.shape != shape or not t.is_contiguous():
        raise _misfit(t, name, dtype, device, shape, "no gaps")
    return t.data_ptr()


def _offsets(cu_seqlens, B, device):
    """cu_seqlens' address and the number of sequences."""
    if cu_seqlens is None:
        return None, B
    n = cu_seqlens.numel()
    if n < 2:
        raise ValueError("cu_seqlens must be [N + 1]")
    return _flat(cu_seqlens, "cu_seqlens", torch.int32, device, (n,)), n - 1


def _conv_weights(weight, bias, dt, dev, D):
    wt = weight.dtype
    if wt is not dt and wt is not _F32:
        raise ValueError(f"weight must be {dt} or float32, got {wt}")
    shape = weight.shape
    if len(shape) != 2 or shape[0] != D:
        raise ValueError(f"weight must be [{D}, W], got {list(shape)}")
    return (shape[1], _CODE[wt], _flat(weight, "weight", wt, dev, shape),
            None if bias is None else _flat(bias, "bias", wt, dev, (D,)))


def _activation(activation):
    code = _ACTIVATIONS.get(activation)
    if code is None:
        raise ValueError(f"activation must be one of {list(_ACTIVATIONS)}")
    return code


def _call(name, args, stream, device):
    """Call the library with the tensors' device current: it launches, counts SMs and
    records errors there."""
    fn, handle = getattr(_lib._lib or _lib.load(), name), _stream_handle(stream, device)
    if _current_device() == device.index:
        st = fn(ctypes.byref(args), handle)
    else:
        with torch.cuda.device(device):
            st = fn(ctypes.byref(args), handle)
    if st:
        _lib.check(st, name)


def short_conv_fwd(x, weight, bias=None, initial_state=None, cu_seqlens=None, activation="silu",
                   output_final_state=True, out=None, final_state=None, stream=None):
    """Short causal depthwise convolution over prompts.  Returns ``(y, ht)``
    (``ht`` None if not requested).

    x [B,T,D] (float32 or bfloat16, rows any stride apart); weight [D,W] with
    W = 2..4 and bias [D], both in x's dtype or both float32; activation "silu"
    or None; initial_state [N,W-1,D] in x's dtype: the rows before each
    sequence, oldest first (zeros if None); cu_seqlens [N+1] int32 (then
    B == 1).  ``ht`` [N,W-1,D] holds the last W-1 rows of each sequence.
    """
    code, dev = _first(x, "x", 3)
    dt, size = x.dtype, x.shape
    B, T, D = size
    xs, xb = _rows(x, "x", dt, dev, size)
    W, wcode, wp, bp = _conv_weights(weight, bias, dt, dev, D)
    cu, N = _offsets(cu_seqlens, B, dev)
    shape = (N, W - 1, D)
    if out is None:
        out = _empty(size, dt, dev, stream)
    ys, yb = _rows(out, "out", dt, dev, size)
    if final_state is None and output_final_state:
        final_state = _empty(shape, dt, dev, stream)
    a = ShortConvArgs(code, wcode, x.data_ptr(), wp, bp,
                      _flat(initial_state, "initial_state", dt, dev, shape),
                      _flat(final_state, "final_state", dt, dev, shape), out.data_ptr(), cu,
                      xs, xb, ys, yb, B, T, D, W, N, _activation(activation))
    _call("short_conv_fwd", a, stream, dev)
    return out, final_state


def short_conv_bwd(dy, x, weight, bias=None, initial_state=None, dfinal_state=None,
                   cu_seqlens=None, activation="silu", output_dweight=True, workspace=None,
                   stream=None):
    """Gradient of :func:`short_conv_fwd`.  Returns ``(dx, dweight, dbias,
    dinitial_state)``.

    dy [B,T,D] and x, weight, bias, initial_state, cu_seqlens as in the forward
    call; dfinal_state [N,W-1,D] the gradient of its final state (zeros if
    None).  dx has x's dtype, dweight [D,W] and dbias [D] are float32 (dbias
    None without a bias, both None with ``output_dweight=False``),
    dinitial_state is None without an initial_state.
    """
    code, dev = _first(x, "x", 3)
    dt, size = x.dtype, x.shape
    B, T, D = size
    xs, xb = _rows(x, "x", dt, dev, size)
    gs, gb = _rows(dy, "dy", dt, dev, size)
    W, wcode, wp, bp = _conv_weights(weight, bias, dt, dev, D)
    cu, N = _offsets(cu_seqlens, B, dev)
    shape = (N, W - 1, D)
    dx = _empty(size, dt, dev, stream)
    dw = db = dh0 = None
    if output_dweight:
        dw = _empty((D, W), _F32, dev, stream)
        if bias is not None:
            db = _empty((D,), _F32, dev, stream)
    if initial_state is not None:
        dh0 = _empty(shape, dt, dev, stream)
    a = ShortConvBwdArgs(code, wcode, dy.data_ptr(), x.data_ptr(), wp, bp,
                         _flat(initial_state, "initial_state", dt, dev, shape),
                         _flat(dfinal_state, "dfinal_state", dt, dev, shape), dx.data_ptr(),
                         None if dw is None else dw.data_ptr(),
                         None if db is None else db.data_ptr(),
                         None if dh0 is None else dh0.data_ptr(), cu,
                         gs, gb, xs, xb, D, T * D, B, T, D, W, N, _activation(activation))
    if dw is not None:
        workspace = _workspace(a, "short_conv_bwd_workspace_size", workspace, dev, stream)
    _call("short_conv_bwd", a, stream, dev)
    return dx, dw, db, dh0


def _workspace(args, size_fn, workspace, device, stream):
    """Hand ``args`` a buffer of the size the library asks for (from PyTorch's
    caching allocator, which keeps it valid for the work enqueued on its stream,
    unless the caller passes one)."""
    n = ctypes.c_size_t(0)
    here = _current_device() == device.index
    with contextlib.nullcontext() if here else torch.cuda.device(device):
        st = getattr(_lib._lib or _lib.load(), size_fn)(ctypes.byref(args), ctypes.byref(n))
    if st:
        _lib.check(st, size_fn)
    if n.value == 0:
        return None
    if workspace is None:
        workspace = _empty(n.value, torch.uint8, device, stream)
    elif (workspace.device != device or not workspace.is_contiguous()
          or workspace.numel() * workspace.element_size() < n.value):
        raise ValueError(f"workspace needs {n.value} bytes on {device}")
    args.workspace = workspace.data_ptr()
    args.workspace_bytes = workspace.numel() * workspace.element_size()
    return workspace


def short_conv_decode(x, weight, state, bias=None, slot_indices=None, activation="silu", out=None,
                      stream=None):
    """The convolution for T = 1..4 new tokens of each request.  Returns y.

    x [B,T,D]; weight and bias as :func:`short_conv_fwd`; ``state``
    [pool,W-1,D] in x's dtype holds every request's last W-1 rows and is
    updated in place; slot_indices [B] int32 names each entry's slot (distinct;
    None = entry b uses slot b).
    """
    code, dev = _first(x, "x", 3)
    dt, size = x.dtype, x.shape
    B, T, D = size
    xs, xb = _rows(x, "x", dt, dev, size)
    W, wcode, wp, bp = _conv_weights(weight, bias, dt, dev, D)
    if out is None:
        out = _empty(size, dt, dev, stream)
    ys, yb = _rows(out, "out", dt, dev, size)
    pool = state.shape[0]
    a = ShortConvDecodeArgs(code, wcode, x.data_ptr(), wp, bp,
                            _flat(state, "state", dt, dev, (pool, W - 1, D)),
                            _flat(slot_indices, "slot_indices", torch.int32, dev, (B,)),
                            out.data_ptr(), xs, xb, ys, yb, B, T, D, W, pool,
                            _activation(activation))
    _call("short_conv_decode", a, stream, dev)
    return out


def _ssm_common(x, dt, A_log, Bm, Cm, D, z, dt_bias, out, out_dtype, stream):
    """Checks shared by the scan's two forms: sizes, types, addresses, strides."""
    code, dev = _first(x, "x", 4)
    xt, size = x.dtype, x.shape
    B, T, H, V = size
    group = Bm.shape
    if len(group) != 4:
        raise ValueError(f"Bm must be [B, T, Hg, K], got {list(group)}")
    Hg, K = group[2], group[3]
    group = (B, T, Hg, K)
    dtt = dt.dtype
    if dtt is not xt and dtt is not _F32:
        raise ValueError(f"dt must be {xt} or float32, got {dtt}")
    if out_dtype is None:
        out_dtype = xt
    elif out_dtype is not xt and out_dtype is not _F32:
        raise ValueError(f"out_dtype must be None, {xt} or torch.float32")
    if out is None:
        out = _empty(size, out_dtype, dev, stream)
    strides = (*_heads(x, "x", xt, dev, size),
               *((0, 0) if z is None else _heads(z, "z", xt, dev, size)),
               *_heads(Bm, "Bm", xt, dev, group), *_heads(Cm, "Cm", xt, dev, group),
               *_rows(dt, "dt", dtt, dev, (B, T, H)), *_heads(out, "out", out_dtype, dev, size))
    heads = (H,)
    tokens = (x.data_ptr(), None if z is None else z.data_ptr(), Bm.data_ptr(), Cm.data_ptr(),
              dt.data_ptr(), _flat(A_log, "A_log", _F32, dev, heads),
              _flat(D, "D", _F32, dev, heads), _flat(dt_bias, "dt_bias", _F32, dev, heads))
    return (code, dev, _CODE[dtt], (B, T, H, Hg, K, V), tokens, strides, out,
            int(out_dtype is _F32))


def ssm_chunk_fwd(x, dt, A_log, Bm, Cm, D=None, z=None, dt_bias=None, dt_softplus=True,
                  initial_state=None, cu_seqlens=None, output_final_state=True, out=None,
                  final_state=None, workspace=None, stream=None, out_dtype=None, segment_tokens=0):
    """Selective state space scan over prompts.  Returns ``(y, ht)`` (``ht``
    None if not requested).

    Per head, with the state h [V,K]: s = softplus(dt + dt_bias),
    h = exp(-exp(A_log) s) h + s x Bm^T, y = (h Cm + D x) silu(z).
    x, z [B,T,H,V]; Bm, Cm [B,T,Hg,K] (H % Hg == 0); dt [B,T,H] in x's dtype or
    float32; A_log, D, dt_bias [H] float32; initial_state and ht [N,H,V,K]
    float32; cu_seqlens [N+1] int32 (then B == 1).  ``dt_softplus=False`` takes
    dt + dt_bias as it is; ``out_dtype=torch.float32`` writes y in float32;
    ``segment_tokens`` (a multiple of 128, 0 = the library's choice) is the
    longest run of tokens that is taken in sequence.
    """
    code, dev, dcode, (B, T, H, Hg, K, V), tokens, strides, out, y32 = _ssm_common(
        x, dt, A_log, Bm, Cm, D, z, dt_bias, out, out_dtype, stream)
    cu, N = _offsets(cu_seqlens, B, dev)
    shape = (N, H, V, K)
    if final_state is None and output_final_state:
        final_state = _empty(shape, _F32, dev, stream)
    a = SsmChunkArgs(code, dcode, *tokens, _flat(initial_state, "initial_state", _F32, dev, shape),
                     _flat(final_state, "final_state", _F32, dev, shape), out.data_ptr(), cu,
                     *strides, B, T, H, Hg, K, V, N, int(bool(dt_softplus)), y32,
                     int(segment_tokens))
    workspace = _workspace(a, "ssm_chunk_workspace_size", workspace, dev, stream)
    _call("ssm_chunk_fwd", a, stream, dev)
    return out, final_state


def ssm_decode(x, dt, A_log, Bm, Cm, state, D=None, z=None, dt_bias=None, dt_softplus=True,
               slot_indices=None, out=None, stream=None, out_dtype=None):
    """The scan for T = 1..4 new tokens of each request.  Returns y.

    Arguments as :func:`ssm_chunk_fwd`; ``state`` [pool,H,V,K] (bfloat16 or
    float32) is updated in place; slot_indices [B] int32 names each entry's
    slot (distinct; None = entry b uses slot b).
    """
    code, dev, dcode, (B, T, H, Hg, K, V), tokens, strides, out, y32 = _ssm_common(
        x, dt, A_log, Bm, Cm, D, z, dt_bias, out, out_dtype, stream)
    st = state.dtype
    if st not in _CODE:
        raise ValueError(f"state must be float32 or bfloat16, got {st}")
    pool = state.shape[0]
    a = SsmDecodeArgs(code, dcode, _CODE[st], *tokens,
                      _flat(state, "state", st, dev, (pool, H, V, K)),
                      _flat(slot_indices, "slot_indices", torch.int32, dev, (B,)), out.data_ptr(),
                      *strides, B, T, H, Hg, K, V, pool, int(bool(dt_softplus)), y32)
    _call("ssm_decode", a, stream, dev)
    return out
