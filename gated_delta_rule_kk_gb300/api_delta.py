"""Python entry point of KDA for single tokens.

As in ``api_ssm.py``: token tensors may be column ranges of wider buffers, so that q, k
and v may be columns of the short convolution's output.
"""
from __future__ import annotations

import torch

from ._lib import KdaDecodeArgs
from .api_ssm import _CODE, _F32, _call, _empty, _first, _flat, _heads, _rows


def kda_decode(q, k, v, a, b, A_log, dt_bias, state, scale=None, slot_indices=None,
               use_qk_l2norm=True, eps=1e-6, out=None, out_dtype=None, stream=None):
    """KDA for T = 1..4 new tokens of each request.  Returns o [B,T,HV,V].

    q, k [B,T,H,K]; v [B,T,HV,V]; a [B,T,HV,K] and b [B,T,HV], all float32 or bfloat16;
    A_log [HV] and dt_bias [HV,K] (or None) float32.  Per key channel the log-gate is
    -exp(A_log) softplus(a + dt_bias), and beta is sigmoid(b).  ``state`` [pool,HV,V,K]
    (bfloat16 or float32) is updated in place; slot_indices [B] int32 names each entry's
    slot (distinct; None = entry b uses slot b).  ``use_qk_l2norm`` divides q and k by
    sqrt(sum x^2 + eps); scale defaults to 1/sqrt(K).
    """
    code, dev = _first(v, "v", 4)
    dt, size = v.dtype, v.shape
    B, T, HV, V = size
    heads = q.shape
    if len(heads) != 4:
        raise ValueError(f"q must be [B, T, H, K], got {list(heads)}")
    H, K = heads[2], heads[3]
    heads = (B, T, H, K)
    st = state.dtype
    if st not in _CODE:
        raise ValueError(f"state must be float32 or bfloat16, got {st}")
    if scale is not None and not scale > 0:
        raise ValueError(f"scale must be positive, got {scale}")
    if not eps >= 0:
        raise ValueError(f"eps must not be negative, got {eps}")
    if out_dtype is None:
        out_dtype = dt
    elif out_dtype is not dt and out_dtype is not _F32:
        raise ValueError(f"out_dtype must be None, {dt} or torch.float32")
    if out is None:
        out = _empty(size, out_dtype, dev, stream)
    strides = (*_heads(q, "q", dt, dev, heads), *_heads(k, "k", dt, dev, heads),
               *_heads(v, "v", dt, dev, size), *_heads(a, "a", dt, dev, (B, T, HV, K)),
               *_rows(b, "b", dt, dev, (B, T, HV)), *_heads(out, "out", out_dtype, dev, size))
    pool = state.shape[0]
    args = KdaDecodeArgs(code, _CODE[st], q.data_ptr(), k.data_ptr(), v.data_ptr(), a.data_ptr(),
                         b.data_ptr(), _flat(A_log, "A_log", _F32, dev, (HV,)),
                         _flat(dt_bias, "dt_bias", _F32, dev, (HV, K)),
                         _flat(state, "state", st, dev, (pool, HV, V, K)),
                         _flat(slot_indices, "slot_indices", torch.int32, dev, (B,)),
                         out.data_ptr(), *strides, B, T, H, HV, K, V, pool,
                         int(bool(use_qk_l2norm)), int(out_dtype is _F32),
                         0.0 if scale is None else float(scale), float(eps))
    _call("kda_decode", args, stream, dev)
    return out
