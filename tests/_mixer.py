"""Inputs and bounds shared by the tests of the short convolution and the scan."""
import numpy as np
import torch

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
