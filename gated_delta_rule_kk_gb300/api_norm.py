"""Python entry points of the norm over groups of channels, forward and backward.

As in ``api_ssm.py``: token tensors may be column ranges of wider buffers, and
outputs belong to ``stream`` (the current one by default).
"""
from __future__ import annotations

from ._lib import GroupNormArgs, GroupNormBwdArgs
from .api_ssm import _CODE, _F32, _call, _empty, _first, _flat, _rows, _workspace

_ACT = {None: 0, "silu": 1, "sigmoid": 2}


def _norm_common(x, groups, weight, bias, z, center, activation, gate_first, eps):
    code, dev = _first(x, "x", 3)
    dt, size = x.dtype, x.shape
    D = size[2]
    if groups < 1 or D % groups:
        raise ValueError(f"x's {D} channels must be a multiple of groups ({groups})")
    wt, shared, addresses = dt, 0, [None, None]
    for i, (w, name) in enumerate(((weight, "weight"), (bias, "bias"))):
        if w is None:
            continue
        if i == 0 or weight is None:
            wt, shared = w.dtype, int(w.numel() != D)
            if wt is not dt and wt is not _F32:
                raise ValueError(f"{name} must be {dt} or float32, got {wt}")
        addresses[i] = _flat(w, name, wt, dev, (D // groups if shared else D,))
    act = _ACT.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {list(_ACT)}")
    return (code, dev, dt, size, _CODE[wt], shared, addresses, _rows(x, "x", dt, dev, size),
            (0, 0) if z is None else _rows(z, "z", dt, dev, size),
            (*size, groups, shared, int(bool(center)), int(bool(gate_first)), act, float(eps)))


def group_norm_fwd(x, groups, weight=None, bias=None, z=None, eps=1e-5, center=True,
                   activation=None, gate_first=False, out=None, stream=None):
    """Norm over ``groups`` groups of every token's channels, with an activation or a gate.
    Returns y.

    x, z [B,T,D] (float32 or bfloat16, rows any stride apart); weight and bias [D], or
    [D // groups] for all groups, in x's dtype or float32 (ones and zeros if None).  A group
    is brought to mean 0 and variance 1 (``center=False``: to a mean square of 1), then
    multiplied by weight and bias added.  ``activation`` (None, "silu" or "sigmoid") is taken
    of z, which the result is multiplied by, or without z of the result itself;
    ``gate_first`` multiplies x instead, before the norm.
    """
    code, dev, dt, size, wcode, _, (wp, bp), xs, zs, sizes = _norm_common(
        x, groups, weight, bias, z, center, activation, gate_first, eps)
    if out is None:
        out = _empty(size, dt, dev, stream)
    a = GroupNormArgs(code, wcode, x.data_ptr(), None if z is None else z.data_ptr(), wp, bp,
                      out.data_ptr(), *xs, *zs, *_rows(out, "out", dt, dev, size), *sizes)
    _call("group_norm_fwd", a, stream, dev)
    return out


def group_norm_bwd(dy, x, groups, weight=None, bias=None, z=None, eps=1e-5, center=True,
                   activation=None, gate_first=False, output_dweight=True, workspace=None,
                   stream=None):
    """Gradient of :func:`group_norm_fwd`.  Returns ``(dx, dweight, dbias, dz)``.

    dy [B,T,D] and the rest as in the forward call.  dx and dz have x's dtype (dz None
    without z); dweight and dbias are float32 and shaped as weight and bias (None without
    one, both None with ``output_dweight=False``).
    """
    code, dev, dt, size, wcode, shared, (wp, bp), xs, zs, sizes = _norm_common(
        x, groups, weight, bias, z, center, activation, gate_first, eps)
    gs = _rows(dy, "dy", dt, dev, size)
    dx = _empty(size, dt, dev, stream)
    dz = None if z is None else _empty(size, dt, dev, stream)
    shape = (size[2] // groups if shared else size[2],)
    dw = db = None
    if output_dweight:
        dw = None if weight is None else _empty(shape, _F32, dev, stream)
        db = None if bias is None else _empty(shape, _F32, dev, stream)
    dense = (size[2], size[1] * size[2])
    a = GroupNormBwdArgs(code, wcode, dy.data_ptr(), x.data_ptr(),
                         None if z is None else z.data_ptr(), wp, bp, dx.data_ptr(),
                         *(None if t is None else t.data_ptr() for t in (dz, dw, db)),
                         *gs, *xs, *zs, *dense, *((0, 0) if z is None else dense), *sizes)
    if dw is not None or db is not None:
        workspace = _workspace(a, "group_norm_bwd_workspace_size", workspace, dev, stream)
    _call("group_norm_bwd", a, stream, dev)
    return dx, dw, db, dz
