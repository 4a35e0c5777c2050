"""Inputs shared by the tests of the delta rule's gradient, KDA's tokens and the norm."""
import numpy as np
import torch


def delta_inputs(seed, B, T, H, Hg, K, V, dtype, lens=None, states=True, cumsum=False, reset=False,
                 zero_beta=False, v_first=False):
    """``reset``: every fifth token's gate is e^-30; ``zero_beta``: every third beta is 0."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g) * std

    def unit(*shape):
        x = normal(*shape)
        return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)).to(dtype)

    N = B if lens is None else len(lens)
    gate = torch.nn.functional.logsigmoid(normal(B, T, H) + 3)
    beta = torch.sigmoid(normal(B, T, H))
    if reset:
        gate[:, ::5] = -30.0
    if zero_beta:
        beta[:, ::3] = 0.0
    cu = None if lens is None else torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32)
    if cumsum:
        starts = [0] if lens is None else cu[:-1].tolist()
        ends = [T] if lens is None else cu[1:].tolist()
        for lo, hi in zip(starts, ends):
            for c in range(lo, hi, 64):
                gate[:, c:min(c + 64, hi)] = gate[:, c:min(c + 64, hi)].cumsum(1)
    i = dict(do=normal(B, T, H, V).to(dtype), q=unit(B, T, Hg, K), k=unit(B, T, Hg, K),
             v=normal(B, T, H, V).to(dtype), g=gate, beta=beta, scale=K ** -0.5, cu=cu,
             h0=normal(N, H, K, V, std=0.3) if states else None,
             dht=normal(N, H, K, V, std=0.3) if states else None)
    if v_first and states:
        i["h0"], i["dht"] = (i[s].transpose(2, 3).contiguous() for s in ("h0", "dht"))
    return i


def kda_inputs(seed, B, T, H, HV, K, V, dtype, state_dtype, gap=0):
    """q, k and v as column ranges of one buffer, ``gap`` columns wider than they are."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g) * std

    rows = normal(B, T, 2 * H * K + HV * V + gap).to(dtype)
    at = gap // 2
    i = dict(q=rows[..., at:at + H * K].unflatten(2, (H, K)),
             k=rows[..., at + H * K:at + 2 * H * K].unflatten(2, (H, K)),
             v=rows[..., at + 2 * H * K:at + 2 * H * K + HV * V].unflatten(2, (HV, V)),
             a=normal(B, T, HV, K).to(dtype), b=normal(B, T, HV).to(dtype),
             A_log=torch.log(torch.rand(HV, generator=g) * 15 + 1),
             dt_bias=normal(HV, K) - 3)
    pool = B + B // 2 + 1
    i["state"] = normal(pool, HV, V, K, std=0.3).to(state_dtype)
    i["slots"] = torch.randperm(pool, generator=g)[:B].to(torch.int32)
    return i


def norm_inputs(seed, B, T, groups, width, dtype, shared=False, weight=True, bias=True, z=True,
                gap=0, weight_dtype=None):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=g) * std + mean

    D, wide = groups * width, width if shared else groups * width
    wt = weight_dtype or dtype

    def rows():
        return normal(B, T, D + gap).to(dtype)[..., gap // 2:gap // 2 + D]

    return dict(dy=normal(B, T, D).to(dtype), x=rows(), z=rows() if z else None,
                weight=normal(wide, std=0.2, mean=1).to(wt) if weight else None,
                bias=normal(wide, std=0.3).to(wt) if bias else None)
