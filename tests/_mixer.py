"""Inputs and bounds shared by the tests of the short convolution and the scan."""
import numpy as np
import torch

from oracle import mixer

from _util import RECORDS, CURRENT_TEST, _np


def assert_each_close(got, ref, what, atol_rms):
    """|got - ref| <= u |ref| + atol_rms RMS(ref) for every element, u the unit
    round-off of got's type (2^-8 in bfloat16, nothing in float32, whose own
    rounding is far inside the second term)."""
    g, r = _np(got), np.asarray(ref, dtype=np.float64)
    assert g.shape == r.shape, (what, g.shape, r.shape)
    if not g.size:
        return
    rms = float(np.sqrt(np.mean(r * r))) or 1.0
    unit = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    room = unit * np.abs(r) + atol_rms * rms
    worst = float(np.max(np.abs(g - r) / room))
    RECORDS.append((CURRENT_TEST[0], what, worst * atol_rms, worst * atol_rms, atol_rms))
    assert np.isfinite(worst) and worst <= 1.0, f"{what}: {worst:.2f} times the allowed error"


def conv_inputs(seed, B, T, D, W, dtype, bias=True, lens=None, state=True, gap=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(dtype)

    N = B if lens is None else len(lens)
    rows = normal(B, T, D + gap)
    off = gap // 16 * 8
    d = dict(x=rows[:, :, off:off + D], weight=normal(D, W, std=0.5),
             bias=normal(D, std=0.2) if bias else None,
             h0=normal(N, W - 1, D) if state else None, dy=normal(B, T, D),
             dht=normal(N, W - 1, D) if state else None, cu=None)
    if lens is not None:
        d["cu"] = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32)
    return d


def ssm_inputs(seed, B, T, H, Hg, V, K, dtype, lens=None, h0=True, z=True, skip=True, fast=False):
    """x, Bm, Cm as column ranges of one buffer and z, dt of another, as a layer
    has them; ``fast`` draws decays of up to e^-100 a token."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g) * std

    N = B if lens is None else len(lens)
    C = H * V + 2 * Hg * K
    conv = torch.nn.functional.silu(normal(B, T, C)).to(dtype)
    proj = normal(B, T, (H * V + H + 7) // 8 * 8).to(dtype)
    step = torch.exp(torch.rand(H, generator=g) * 4.6 - 6.9)
    d = dict(x=conv[:, :, :H * V].unflatten(2, (H, V)),
             Bm=conv[:, :, H * V:H * V + Hg * K].unflatten(2, (Hg, K)),
             Cm=conv[:, :, H * V + Hg * K:].unflatten(2, (Hg, K)),
             z=proj[:, :, :H * V].unflatten(2, (H, V)) if z else None,
             dt=proj[:, :, H * V:H * V + H],
             A_log=torch.log(torch.rand(H, generator=g) * 15 + 1),
             dt_bias=step + torch.log(-torch.expm1(-step)) + (4.0 if fast else 0.0),
             D=1 + normal(H, std=0.2) if skip else None,
             h0=normal(N, H, V, K, std=0.5) if h0 else None, cu=None)
    if lens is not None:
        d["cu"] = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32)
    return d


def cuda(d):
    """Copies on the GPU that keep their strides (ranges of one buffer too)."""
    out = {}
    for k, v in d.items():
        if isinstance(v, torch.Tensor) and not v.is_contiguous():
            base = torch.zeros(v.untyped_storage().nbytes() // v.element_size(), dtype=v.dtype,
                               device="cuda")
            out[k] = base.as_strided(v.shape, v.stride(), v.storage_offset()).copy_(v)
        else:
            out[k] = v.cuda() if isinstance(v, torch.Tensor) else v
    return out


def scan_rooms(i, pieces=2):
    """What y may be off by where the scan runs on the tensor cores, element for element.

    A 128-token chunk from state h is y = e^G (C h) + M x with M and h in two bfloat16 pieces,
    each to 2^-8 of what it is taken from: at most 2^-16 of |M| |x| + e^G |C| |h| (2^-8 with one).
    M's own sums over K, the products' (16 terms at a time, some 20 partial sums of float32) and
    the decays' exponentials: 2^-18 of the same with the magnitudes taken inside M and h."""
    x, Bm, Cm, dt = (_np(i[k]) for k in ("x", "Bm", "Cm", "dt"))
    H, V = x.shape[2:]
    head = np.arange(H) // (H // Bm.shape[2])
    a, bias = -np.exp(_np(i["A_log"])), _np(i["dt_bias"])
    step = mixer.softplus(dt + bias)
    skip = np.zeros(H) if i["D"] is None else _np(i["D"])
    room = np.zeros_like(x)
    for n, (b, lo, hi) in enumerate(mixer.bounds(x.shape[0], x.shape[1], i["cu"])):
        h = np.zeros((H, V, Bm.shape[3])) if i["h0"] is None else _np(i["h0"])[n]
        most = np.abs(h)  # h's magnitudes, summed without cancelling
        for t in range(lo, hi, 128):
            e = min(t + 128, hi)
            s, xc = step[b, t:e].T, x[b, t:e].transpose(1, 0, 2)  # heads first
            G = np.cumsum(a[:, None] * s, 1)
            low = np.tril(np.ones((e - t, e - t), bool))
            L = np.exp(np.where(low, G[:, :, None] - G[:, None, :], -np.inf)) * s[:, None, :]
            B, C = (v[b, t:e].transpose(1, 0, 2)[head] for v in (Bm, Cm))
            eye = skip[:, None, None] * np.eye(e - t)
            M, most_M = C @ B.transpose(0, 2, 1) * L + eye, \
                np.abs(C) @ np.abs(B).transpose(0, 2, 1) * L + np.abs(eye)
            eG = np.exp(G)[:, :, None]
            near = np.abs(M) @ np.abs(xc) + eG * (np.abs(C) @ np.abs(h).transpose(0, 2, 1))
            sums = most_M @ np.abs(xc) + eG * (np.abs(C) @ most.transpose(0, 2, 1))
            room[b, t:e] = (2.0 ** (-8 * pieces) * near + 2.0 ** -18 * sums).transpose(1, 0, 2)
            W = (s * np.exp(G[:, -1:] - G))[:, :, None] * xc
            end = np.exp(G[:, -1])[:, None, None]
            h = end * h + W.transpose(0, 2, 1) @ B
            most = end * most + np.abs(W).transpose(0, 2, 1) @ np.abs(B)
    if i["z"] is not None:
        z = _np(i["z"])
        room *= np.abs(z * mixer.sigmoid(z))
    return room


def assert_inside(got, ref, room, what):
    """|got - ref| <= room for every element."""
    worst = float(np.max(np.abs(_np(got) - ref) / np.maximum(room, 1e-300)))
    RECORDS.append((CURRENT_TEST[0], what, worst, worst, 1.0))
    assert np.isfinite(worst) and worst <= 1.0, f"{what}: {worst:.2f} times the allowed error"
