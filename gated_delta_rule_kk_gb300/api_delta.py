"""Python entry points of the chunked gated delta rule's gradient and of KDA for single
tokens.

As in ``api_ssm.py``: outputs belong to ``stream`` (the current one by default), and the
token tensors of ``kda_decode`` may be column ranges of wider buffers, so that q, k and v
may be columns of the short convolution's output.
"""
from __future__ import annotations

import torch

from ._lib import GdnChunkBwdArgs, KdaDecodeArgs
from .api_ssm import _CODE, _F32, _call, _empty, _first, _flat, _heads, _offsets, _rows, _workspace


def gdn_chunk_bwd(do, q, k, v, g, beta, scale=None, initial_state=None, dfinal_state=None,
                  cu_seqlens=None, g_is_cumsum=False, state_v_first=False,
                  output_dinitial_state=None, workspace=None, stream=None):
    """Gradient of :func:`gdn_chunk_fwd`.  Returns ``(dq, dk, dv, dg, dbeta,
    dinitial_state)``.

    do [B,T,H,V] (v's dtype) is the gradient of o and dfinal_state (as ht, zeros if None)
    that of the final state; the rest as in the forward call.  dq, dk and dv have q's dtype,
    dg (of g as given) and dbeta are float32, dinitial_state is float32 and shaped as
    initial_state: returned when one was given, or as ``output_dinitial_state`` says.
    """
    code, dev = _first(q, "q", 4)
    dt, heads = q.dtype, q.shape
    B, T, Hg, K = heads
    size = v.shape
    if len(size) != 4 or size[:2] != heads[:2]:
        raise ValueError(f"v must be [{B}, {T}, H, V], got {list(size)}")
    H, V = size[2], size[3]
    if scale is not None and not scale > 0:
        raise ValueError(f"scale must be positive, got {scale}")
    cu, N = _offsets(cu_seqlens, B, dev)
    states = (N, H, V, K) if state_v_first else (N, H, K, V)
    if output_dinitial_state is None:
        output_dinitial_state = initial_state is not None
    inputs = [_flat(t, name, dt, dev, shape) for t, name, shape in
              ((q, "q", heads), (k, "k", heads), (v, "v", size))]
    inputs += [_flat(t, name, _F32, dev, size[:3]) for t, name in ((g, "g"), (beta, "beta"))]
    inputs += [_flat(initial_state, "initial_state", _F32, dev, states),
               _flat(do, "do", dt, dev, size),
               _flat(dfinal_state, "dfinal_state", _F32, dev, states)]
    dq, dk, dv = (_empty(s, dt, dev, stream) for s in (heads, heads, size))
    dg, dbeta = (_empty(size[:3], _F32, dev, stream) for _ in range(2))
    dh0 = _empty(states, _F32, dev, stream) if output_dinitial_state else None
    a = GdnChunkBwdArgs(code, *inputs, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dg.data_ptr(),
                        dbeta.data_ptr(), None if dh0 is None else dh0.data_ptr(), cu,
                        B, T, H, Hg, K, V, N, 64, int(bool(g_is_cumsum)), int(bool(state_v_first)),
                        0.0 if scale is None else float(scale), None, 0)
    workspace = _workspace(a, "gdn_chunk_bwd_workspace_size", workspace, dev, stream)
    _call("gdn_chunk_bwd", a, stream, dev)
    return dq, dk, dv, dg, dbeta, dh0


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
