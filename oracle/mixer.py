"""The short causal convolution, its gradient and the state space scan, written
out in fp64 numpy from their definitions (token by token)."""
import numpy as np


def _np(x):
    if x is None:
        return None
    if hasattr(x, "detach"):
        x = x.detach().cpu().double().numpy()
    return np.asarray(x, dtype=np.float64)


def bounds(B, T, cu_seqlens):
    """(batch row, first token, last + 1) of every sequence."""
    if cu_seqlens is None:
        return [(b, 0, T) for b in range(B)]
    cu = [int(v) for v in cu_seqlens]
    return [(0, a, b) for a, b in zip(cu, cu[1:])]


def sigmoid(p):
    return 1.0 / (1.0 + np.exp(-p))


def softplus(v):
    v = np.asarray(v, dtype=np.float64)
    return np.where(v > 20, v, np.log1p(np.exp(np.minimum(v, 20))))


def short_conv(x, weight, bias=None, h0=None, cu_seqlens=None, silu=True):
    """y [B,T,D] and the last W - 1 rows of every sequence [N,W-1,D]."""
    x, weight, bias, h0 = _np(x), _np(weight), _np(bias), _np(h0)
    B, T, D = x.shape
    W = weight.shape[1]
    seqs = bounds(B, T, cu_seqlens)
    y, ht = np.zeros_like(x), np.zeros((len(seqs), W - 1, D))
    for n, (b, lo, hi) in enumerate(seqs):
        window = list(h0[n]) if h0 is not None else [np.zeros(D)] * (W - 1)
        for t in range(lo, hi):
            window.append(x[b, t])
            p = sum(weight[:, i] * window[i] for i in range(W))
            if bias is not None:
                p = p + bias
            y[b, t] = p * sigmoid(p) if silu else p
            window.pop(0)
        ht[n] = np.array(window).reshape(W - 1, D)
    return y, ht


def short_conv_grad(dy, x, weight, bias=None, h0=None, dht=None, cu_seqlens=None, silu=True):
    """dx, dweight, dbias, dh0 of <dy, y> + <dht, ht>."""
    dy, x, weight, bias, h0, dht = (_np(v) for v in (dy, x, weight, bias, h0, dht))
    B, T, D = x.shape
    W = weight.shape[1]
    seqs = bounds(B, T, cu_seqlens)
    dx, dw, db = np.zeros_like(x), np.zeros((D, W)), np.zeros(D)
    dh0 = np.zeros((len(seqs), W - 1, D))
    for n, (b, lo, hi) in enumerate(seqs):
        before = h0[n] if h0 is not None else np.zeros((W - 1, D))
        rows = np.concatenate([before, x[b, lo:hi]])
        drows = np.zeros_like(rows)
        for t in range(hi - lo):
            p = sum(weight[:, i] * rows[t + i] for i in range(W)) + (0 if bias is None else bias)
            s = sigmoid(p)
            dp = dy[b, lo + t] * (s * (1 + p * (1 - s)) if silu else 1.0)
            db += dp
            for i in range(W):
                dw[:, i] += dp * rows[t + i]
                drows[t + i] += dp * weight[:, i]
        if dht is not None:
            drows[len(rows) - (W - 1):] += dht[n]
        dh0[n], dx[b, lo:hi] = drows[:W - 1], drows[W - 1:]
    return dx, dw, db, dh0


def ssm_scan(x, dt, A_log, Bm, Cm, D=None, z=None, dt_bias=None, dt_softplus=True, h0=None,
             cu_seqlens=None):
    """y [B,T,H,V] and the final states [N,H,V,K]."""
    x, dt, A_log, Bm, Cm, D, z, dt_bias, h0 = (
        _np(v) for v in (x, dt, A_log, Bm, Cm, D, z, dt_bias, h0))
    B, T, H, V = x.shape
    Hg, K = Bm.shape[2:]
    seqs = bounds(B, T, cu_seqlens)
    head = np.arange(H) // (H // Hg)
    step = dt if dt_bias is None else dt + dt_bias
    if dt_softplus:
        step = softplus(step)
    y, ht = np.zeros_like(x), np.zeros((len(seqs), H, V, K))
    for n, (b, lo, hi) in enumerate(seqs):
        h = h0[n].copy() if h0 is not None else np.zeros((H, V, K))
        for t in range(lo, hi):
            h *= np.exp(-np.exp(A_log) * step[b, t])[:, None, None]
            h += (step[b, t][:, None] * x[b, t])[:, :, None] * Bm[b, t][head][:, None, :]
            y[b, t] = np.einsum("hvk,hk->hv", h, Cm[b, t][head])
        ht[n] = h
    if D is not None:
        y += D[:, None] * x
    if z is not None:
        y *= z * sigmoid(z)
    return y, ht
