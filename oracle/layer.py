"""The gated delta rule's gradient, KDA for single tokens and the norm over groups of
channels, written out in fp64 numpy from their definitions (the recurrences token by
token)."""
import numpy as np

from .mixer import _np, bounds, sigmoid, softplus
from .recurrence import raw_gate_from_chunk_cumsum


def gdn_grad(do, q, k, v, g, beta, scale, h0=None, dht=None, cu_seqlens=None, g_is_cumsum=False):
    """dq, dk, dv, dg, dbeta, dh0 of <do, o> + <dht, ht>, with h' = e^g h,
    d = beta (v - k h'), h = h' + k d, o = scale q h.  dg is the gradient of g as given."""
    do, q, k, v, g, beta, h0, dht = (_np(x) for x in (do, q, k, v, g, beta, h0, dht))
    B, T, Hg, K = q.shape
    H, V = v.shape[2:]
    head = np.arange(H) // (H // Hg)
    seqs = bounds(B, T, cu_seqlens)
    dq, dk, dv, dg, db = (np.zeros_like(x) for x in (q, k, v, g, beta))
    dh0 = np.zeros((len(seqs), H, K, V))
    for n, (b, lo, hi) in enumerate(seqs):
        h = np.zeros((H, K, V)) if h0 is None else h0[n].copy()
        raw = g[b].copy()
        if g_is_cumsum:
            for i in range(H):
                raw[lo:hi, i] = np.asarray(raw_gate_from_chunk_cumsum(g[b, :, i], lo, hi))[lo:hi]
        kept = []
        for t in range(lo, hi):
            before = np.exp(raw[t])[:, None, None] * h
            kt = k[b, t, head]
            miss = v[b, t] - np.einsum("hk,hkv->hv", kt, before)
            h = before + kt[:, :, None] * (beta[b, t][:, None] * miss)[:, None]
            kept.append((before, miss, h))
        G = np.zeros((H, K, V)) if dht is None else dht[n].copy()
        for t in range(hi - 1, lo - 1, -1):
            before, miss, h = kept[t - lo]
            kt, qt, bt = k[b, t, head], q[b, t, head], beta[b, t][:, None]
            np.add.at(dq[b, t], head, scale * np.einsum("hkv,hv->hk", h, do[b, t]))
            G = G + scale * qt[:, :, None] * do[b, t][:, None]
            dd = np.einsum("hk,hkv->hv", kt, G)       # of beta miss
            np.add.at(dk[b, t], head, bt * (np.einsum("hkv,hv->hk", G, miss)
                                            - np.einsum("hkv,hv->hk", before, dd)))
            dv[b, t] = bt * dd
            db[b, t] = (dd * miss).sum(1)
            G = G - kt[:, :, None] * (bt * dd)[:, None]
            dg[b, t] = (G * before).sum((1, 2))
            G = np.exp(raw[t])[:, None, None] * G
        dh0[n] = G
        if g_is_cumsum:  # g_t = c_t - c_{t-1}, and c_t itself at a chunk's first token
            for t in range(lo, hi - 1):
                if (t + 1 - lo) % 64:
                    dg[b, t] -= dg[b, t + 1]
    return dq, dk, dv, dg, db, dh0


def kda_decode(q, k, v, a, b, A_log, dt_bias, state, slots=None, scale=None, l2norm=True, eps=1e-6):
    """o [B,T,HV,V] and the states [B,HV,V,K] after the tokens."""
    q, k, v, a, b, A_log, dt_bias, state = (_np(x) for x in (q, k, v, a, b, A_log, dt_bias, state))
    B, T, H, K = q.shape
    HV = v.shape[2]
    head = np.arange(HV) // (HV // H)
    if l2norm:
        q = q / np.sqrt((q * q).sum(-1, keepdims=True) + eps)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + eps)
    scale = K ** -0.5 if scale is None else scale
    S = state[np.arange(B) if slots is None else _np(slots).astype(int)].copy()
    o = np.zeros_like(v)
    for t in range(T):
        g = -np.exp(A_log)[:, None] * softplus(a[:, t] + (0 if dt_bias is None else dt_bias))
        S = S * np.exp(g)[:, :, None]
        kt, qt = k[:, t][:, head], q[:, t][:, head]
        d = sigmoid(b[:, t])[..., None] * (v[:, t] - np.einsum("bhvk,bhk->bhv", S, kt))
        S = S + d[..., None] * kt[:, :, None]
        o[:, t] = scale * np.einsum("bhvk,bhk->bhv", S, qt)
    return o, S


def _act(name, z):
    return z if name is None else z * sigmoid(z) if name == "silu" else sigmoid(z)


def _slope(name, z):
    s = sigmoid(z)
    return np.ones_like(z) if name is None else s * (1 + z * (1 - s)) if name == "silu" else s * (1 - s)


def _norm(x, groups, weight, bias, z, eps, center, activation, gate_first):
    x, weight, bias, z = (_np(v) for v in (x, weight, bias, z))
    shape = (*x.shape[:2], groups, x.shape[2] // groups)
    z = None if z is None else z.reshape(shape)
    u = x.reshape(shape)
    if gate_first:
        u = u * _act(activation, z)
    c = u - u.mean(-1, keepdims=True) if center else u
    r = 1 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    w, b = (d if v is None else v.reshape(-1, shape[3]) for v, d in ((weight, 1.0), (bias, 0.0)))
    return x.reshape(shape), z, c * r, r, w, b


def group_norm(x, groups, weight=None, bias=None, z=None, eps=1e-5, center=True, activation=None,
               gate_first=False):
    """y [B,T,D]: every token's groups of channels to their normal form, weighted, gated."""
    x, z, n, _, w, b = _norm(x, groups, weight, bias, z, eps, center, activation, gate_first)
    m = n * w + b
    if not gate_first:
        m = _act(activation, m) if z is None else m * _act(activation, z)
    return m.reshape(*m.shape[:2], -1)


def group_norm_grad(dy, x, groups, weight=None, bias=None, z=None, eps=1e-5, center=True,
                    activation=None, gate_first=False):
    """dx, dweight, dbias, dz of <dy, y> (dweight and dbias per group and channel [G, W])."""
    x, z, n, r, w, b = _norm(x, groups, weight, bias, z, eps, center, activation, gate_first)
    dy = _np(dy).reshape(n.shape)
    m, dm, dz = n * w + b, dy, None
    if z is not None and not gate_first:
        dm, dz = dy * _act(activation, z), dy * m * _slope(activation, z)
    elif z is None:
        dm = dy * _slope(activation, m)
    dw, db = (dm * n).sum((0, 1)), dm.sum((0, 1))
    dn = dm * w
    du = dn - n * (dn * n).mean(-1, keepdims=True)
    if center:
        du = du - dn.mean(-1, keepdims=True)
    dx = du = du * r
    if gate_first:
        dx, dz = du * _act(activation, z), du * x * _slope(activation, z)
    flat = (*n.shape[:2], -1)
    return dx.reshape(flat), dw, db, None if dz is None else dz.reshape(flat)
