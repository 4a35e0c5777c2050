"""Cases of the short causal convolution and of the selective state space scan.

Each case is one call of one operator: the convolution over prompts, its
gradient and its form for single tokens; the scan over prompts and its form
for single tokens.  ``run`` computes the plain form in 32 bits, or calls the
library's operator when ``own`` is set; ``exact`` computes the definition in
64 bits, token by token for the scan.

Inputs are laid out as a model's layer has them: the input projection of a
state space layer is one buffer [z | x B C | dt], the convolution reads its
[x B C] columns in place, and the scan reads x, B and C as column ranges of the
convolution's output.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # q, k and v channels of 16 heads of 128, two prompts of 4096 tokens
        dict(name="conv-prompt", op="conv_fwd", dtype="bf16", seqs=2, T=8192, cut=0, D=6144, W=4,
             silu=True, bias=False, h0=False, gap=0),
        # eight packed prompts continuing from their states; x B C of 64 heads
        # of 64 and one group of 128 states inside the projection's rows
        dict(name="conv-packed", op="conv_fwd", dtype="bf16", seqs=8, T=32068, cut=3, D=4352, W=4,
             silu=True, bias=True, h0=True, gap=4160),
        # odd channels and lengths, three taps, no activation, float32
        dict(name="conv-odd-f32", op="conv_fwd", dtype="f32", seqs=3, T=1527, cut=0, D=771, W=3,
             silu=False, bias=True, h0=True, gap=0),
        # gradient of the first case
        dict(name="conv-bwd-prompt", op="conv_bwd", dtype="bf16", seqs=2, T=8192, cut=0, D=6144,
             W=4, silu=True, bias=False, h0=False, gap=0),
        # gradient over packed documents of odd lengths, float32
        dict(name="conv-bwd-packed-f32", op="conv_bwd", dtype="f32", seqs=5, T=3001, cut=7, D=1160,
             W=4, silu=True, bias=True, h0=True, gap=0),
        # one new token of 256 requests: q, k (16 heads each) and v (32 heads)
        dict(name="conv-token-256", op="conv_decode", dtype="bf16", B=256, T=1, D=8192, W=4,
             silu=True, bias=False),
        # one new token of one request: the smallest call, where latency counts
        dict(name="conv-token-1", op="conv_decode", dtype="bf16", B=1, T=1, D=4352, W=4,
             silu=True, bias=True),
        # two prompts of 4096 tokens, 64 heads on one group, gated output
        dict(name="scan-prompt", op="scan", dtype="bf16", seqs=2, T=8192, cut=0, H=64, Hg=1, V=64,
             K=128, z=True, h0=False),
        # eight packed prompts continuing from their states, grouped B and C
        dict(name="scan-packed", op="scan", dtype="bf16", seqs=8, T=32068, cut=3, H=32, Hg=8, V=64,
             K=128, z=False, h0=True),
        # odd head and state sizes, float32: the exact path
        dict(name="scan-odd-f32", op="scan", dtype="f32", seqs=1, T=773, cut=0, H=12, Hg=2, V=40,
             K=48, z=True, h0=True),
        # one new token of 256 requests, bfloat16 states
        dict(name="scan-token-256", op="scan_decode", dtype="bf16", state="bf16", B=256, T=1, H=64,
             Hg=1, V=64, K=128, z=True),
        # four drafted tokens of three requests, float32 states
        dict(name="scan-token-few", op="scan_decode", dtype="bf16", state="f32", B=3, T=4, H=48,
             Hg=8, V=64, K=128, z=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_decode", "scan", "scan_decode"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    wide = 4 if dtype == "f32" else 2
    if op in ("conv_fwd", "conv_bwd"):
        seqs = rng.randint(1, 12)
        D = _log(rng, 64, 8192)
        if rng.random() < 0.75:
            D = max(8, D // 8 * 8)
        top = 100_000_000 if op == "conv_bwd" else 250_000_000
        T = min(_log(rng, 1, 32768), max(1, top // (D * wide)))
        return dict(op=op, dtype=dtype, seqs=seqs, T=T if T % seqs else T // seqs * seqs,
                    cut=rng.randint(1, 1 << 20) if T % seqs or rng.random() < 0.5 else 0, D=D,
                    W=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.75, bias=rng.random() < 0.5,
                    h0=rng.random() < 0.5, gap=rng.choice([0, 0, 64, 4160]))
    if op == "conv_decode":
        D = _log(rng, 64, 8192)
        if rng.random() < 0.75:
            D = max(8, D // 8 * 8)
        return dict(op=op, dtype=dtype, B=_log(rng, 1, 512), T=rng.randint(1, 4), D=D,
                    W=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.75, bias=rng.random() < 0.5)
    Hg = rng.choice([1, 1, 2, 4, 8])
    if op == "scan":
        V, K = rng.choice([(64, 128), (64, 128), (64, 64), (128, 128), (40, 48)])
        H = Hg * max(1, _log(rng, 4, 64) // Hg)
        seqs = rng.randint(1, 12)
        top = 60_000_000 if dtype == "bf16" and K != 48 else 4_000_000
        T = min(_log(rng, 1, 32768), max(1, top // (H * V)))
        return dict(op=op, dtype=dtype, seqs=seqs, T=T if T % seqs else T // seqs * seqs,
                    cut=rng.randint(1, 1 << 20) if T % seqs or rng.random() < 0.5 else 0, H=H,
                    Hg=Hg, V=V, K=K, z=rng.random() < 0.5, h0=rng.random() < 0.5)
    V, K = rng.choice([(64, 128), (64, 128), (64, 64), (128, 128), (40, 48)])
    H = Hg * max(1, _log(rng, 4, 64) // Hg)
    state = rng.choice(["bf16", "f32"])
    B = min(_log(rng, 1, 256), max(1, (60 if state == "f32" else 120) * 10 ** 6 // (H * V * K)))
    return dict(op=op, dtype=dtype, state=state, B=B, T=rng.randint(1, 4), H=H, Hg=Hg, V=V, K=K,
                z=rng.random() < 0.5)


def _lengths(case):
    """Tokens of each sequence: equal ones, or cut at random places (then some may be empty)."""
    n, T = case["seqs"], case["T"]
    if not case["cut"]:
        return [T // n] * n
    r = random.Random(case["cut"])
    at = sorted(r.randint(0, T) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + at, at + [T])]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo

    s = {"case": case}
    packed = case.get("cut", 0) != 0
    if packed:
        lens = torch.tensor([0] + _lengths(case))
        s["cu"] = lens.cumsum(0).to(torch.int32).cuda()
    if "seqs" in case:
        B, T = (1, case["T"]) if packed else (case["seqs"], case["T"] // case["seqs"])
    else:
        B, T = case["B"], case["T"]
    if case["op"].startswith("conv"):
        D, W, gap = case["D"], case["W"], case.get("gap", 0)
        rows = normal(B, T, gap + D)
        s["x"] = rows[:, :, gap // 16 * 8:gap // 16 * 8 + D]
        s["weight"] = normal(D, W, std=0.5)
        s["bias"] = normal(D, std=0.1) if case["bias"] else None
        s["act"] = "silu" if case["silu"] else None
        if case["op"] == "conv_decode":
            s["state"] = normal(B + B // 2 + 1, W - 1, D)
            s["slots"] = torch.randperm(B + B // 2 + 1, generator=g, device="cuda")[:B].to(torch.int32)
        elif case["h0"]:
            s["h0"] = normal(case["seqs"], W - 1, D)
        if case["op"] == "conv_bwd":
            s["dy"] = normal(B, T, D)
            if case["h0"]:
                s["dht"] = normal(case["seqs"], W - 1, D)
        return s
    H, Hg, V, K = (case[k] for k in ("H", "Hg", "V", "K"))
    # the input projection's rows [z | x B C | dt] and the convolution's output
    C = H * V + 2 * Hg * K
    proj = normal(B, T, (H * V + C + H + 7) // 8 * 8)
    conv = torch.nn.functional.silu(normal(B, T, C))
    s["x"] = conv[:, :, :H * V].unflatten(2, (H, V))
    s["Bm"] = conv[:, :, H * V:H * V + Hg * K].unflatten(2, (Hg, K))
    s["Cm"] = conv[:, :, H * V + Hg * K:].unflatten(2, (Hg, K))
    s["z"] = proj[:, :, :H * V].unflatten(2, (H, V)) if case["z"] else None
    s["dt"] = proj[:, :, H * V + C:H * V + C + H]
    s["A_log"] = uniform(H, lo=1.0, hi=16.0).log()
    step = torch.exp(uniform(H, lo=math.log(1e-3), hi=math.log(0.1)))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus of it is `step`
    s["D"] = normal(H, std=0.2, mean=1.0, dtype=torch.float32)
    if case["op"] == "scan_decode":
        pool = B + B // 2 + 1
        s["state"] = normal(pool, H, V, K, std=0.5, dtype=_DTYPES[case["state"]])
        s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:B].to(torch.int32)
    elif case["h0"]:
        s["h0"] = normal(case["seqs"], H, V, K, std=0.5, dtype=torch.float32)
    return s


# ---------------------------------------------------------------- plain forms

def _bounds(s, B, T):
    """First and last + 1 token of every sequence, of all B * T tokens."""
    if "cu" in s:
        cu = s["cu"].long()
    else:
        cu = torch.arange(B + 1, device="cuda") * T
    return cu[:-1], cu[1:]


def _conv_rows(s):
    """Rows of the inputs and of the states before them, in 32 bits, and for
    every token the rows its W taps read."""
    x, W = s["x"].float(), s["case"]["W"]
    B, T, D = x.shape
    bos, eos = _bounds(s, B, T)
    n, tokens = bos.numel(), B * T
    h0 = s["h0"].float() if "h0" in s else x.new_zeros(n, W - 1, D)
    rows = torch.cat([x.reshape(tokens, D), h0.reshape(n * (W - 1), D)])
    t = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(eos, t, right=True)
    pos = (t - bos[seq])[:, None] - (W - 1) + torch.arange(W, device="cuda")
    first = (tokens + seq * (W - 1))[:, None]
    taps = torch.where(pos >= 0, bos[seq][:, None] + pos, first + (W - 1) + pos)
    back = (eos - bos)[:, None] - (W - 1) + torch.arange(W - 1, device="cuda")
    last = torch.where(back >= 0, bos[:, None] + back,
                       (tokens + torch.arange(n, device="cuda") * (W - 1))[:, None] + (W - 1) + back)
    return rows, taps, last, bos, eos


def _conv_pre(s, rows, taps):
    p = (rows[taps] * s["weight"].float().t()).sum(1)
    return p if s["bias"] is None else p + s["bias"].float()


def _plain_conv_fwd(s):
    x = s["x"]
    rows, taps, last, _, _ = _conv_rows(s)
    p = _conv_pre(s, rows, taps)
    y = p * torch.sigmoid(p) if s["act"] else p
    return {"y": y.reshape(x.shape).to(x.dtype), "ht": rows[last].to(x.dtype)}


def _plain_conv_bwd(s):
    x, W = s["x"], s["case"]["W"]
    B, T, D = x.shape
    rows, taps, _, bos, eos = _conv_rows(s)
    dp = s["dy"].float().reshape(B * T, D)
    if s["act"]:
        p = _conv_pre(s, rows, taps)
        e = torch.sigmoid(p)
        dp = dp * (e * (1 + p * (1 - e)))
    dw = (dp[:, None, :] * rows[taps]).sum(0).t()
    # a row's gradient: w[i] times dp of the token that reads it with tap i
    n, tokens = bos.numel(), B * T
    r = torch.arange(rows.shape[0], device="cuda")
    seq = torch.where(r < tokens, torch.searchsorted(eos, r, right=True).clamp(max=n - 1),
                      (r - tokens) // max(1, W - 1))
    pos = torch.where(r < tokens, r - bos[seq], (r - tokens) % max(1, W - 1) - (W - 1))
    at = pos[:, None] + (W - 1) - torch.arange(W, device="cuda")
    there = (at >= 0) & (at < (eos - bos)[seq][:, None])
    dpz = torch.cat([dp, dp.new_zeros(1, D)])
    dr = (dpz[torch.where(there, bos[seq][:, None] + at, tokens)] * s["weight"].float().t()).sum(1)
    if "dht" in s:
        j = pos - (eos - bos)[seq] + (W - 1)
        dhz = torch.cat([s["dht"].float().reshape(n * (W - 1), D), dp.new_zeros(1, D)])
        dr = dr + dhz[torch.where(j >= 0, seq * (W - 1) + j, n * (W - 1))]
    out = {"dx": dr[:tokens].reshape(x.shape).to(x.dtype), "dw": dw.contiguous()}
    if s["bias"] is not None:
        out["db"] = dp.sum(0)
    if "h0" in s:
        out["dh0"] = dr[tokens:].reshape(n, W - 1, D).to(x.dtype)
    return out


def _plain_conv_decode(s):
    x, W, slots = s["x"], s["case"]["W"], s["slots"].long()
    T = x.shape[1]
    rows = torch.cat([s["state"][slots].float(), x.float()], 1)
    at = torch.arange(T, device="cuda")[:, None] + torch.arange(W, device="cuda")
    p = (rows[:, at] * s["weight"].float().t()).sum(2)
    if s["bias"] is not None:
        p = p + s["bias"].float()
    y = p * torch.sigmoid(p) if s["act"] else p
    s["state"][slots] = rows[:, T:].to(x.dtype)
    return {"y": y.to(x.dtype), "state": s["state"]}


def _softplus(x):
    return torch.where(x > 20, x, torch.log1p(torch.exp(x.clamp(max=20))))


def _scan_inputs(s):
    """Step sizes, log-decays and B, C repeated for every head, in 32 bits."""
    rep = s["case"]["H"] // s["case"]["Hg"]
    step = _softplus(s["dt"].float() + s["dt_bias"])
    g = -torch.exp(s["A_log"]) * step
    return (s["x"].float(), step, g, s["Bm"].float().repeat_interleave(rep, 2),
            s["Cm"].float().repeat_interleave(rep, 2))


def _scan_gate(s, y):
    y = y + s["D"][:, None] * s["x"].float()
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    return y


def _plain_scan(s, Q=64):
    case = s["case"]
    H, V, K = case["H"], case["V"], case["K"]
    x, step, g, Bm, Cm = _scan_inputs(s)
    shape = x.shape
    bos, eos = _bounds(s, shape[0], shape[1])
    n = bos.numel()
    lens = eos - bos
    C = max(1, -(-max(_lengths(case)) // Q))
    # every sequence on its own row of C chunks; a step past its end is zero
    pos = torch.arange(C * Q, device="cuda")
    there = pos < lens[:, None]
    at = torch.where(there, bos[:, None] + pos, 0)

    def rows(v):
        v = v.reshape(shape[0] * shape[1], *v.shape[2:])[at]
        return torch.where(there.reshape(n, C * Q, *[1] * (v.dim() - 2)), v, 0).unflatten(1, (C, Q))

    xs = rows(x * step[..., None])              # n C Q H V
    Bs, Cs = rows(Bm), rows(Cm)                 # n C Q H K
    G = rows(g).cumsum(2).permute(0, 3, 1, 2)   # n H C Q
    low = torch.ones(Q, Q, device="cuda", dtype=torch.bool).tril()
    L = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -torch.inf))
    Bs, Cs, xs = (v.permute(0, 3, 1, 2, 4) for v in (Bs, Cs, xs))
    y = ((Cs @ Bs.transpose(3, 4)) * L) @ xs    # within a chunk
    # state of every chunk alone, then of every chunk's start
    ends = (xs * torch.exp(G[..., -1:] - G)[..., None]).transpose(3, 4) @ Bs  # n H C V K
    h0 = s["h0"] if "h0" in s else x.new_zeros(n, H, V, K)
    total = torch.nn.functional.pad(G[..., -1], (1, 0)).cumsum(2)             # n H C+1
    low = torch.ones(C + 1, C + 1, device="cuda", dtype=torch.bool).tril()
    carry = torch.exp(torch.where(low, total[..., :, None] - total[..., None, :], -torch.inf))
    h = carry @ torch.cat([h0[:, :, None], ends], 2).flatten(3)
    h = h.unflatten(3, (V, K))
    y = y + torch.exp(G)[..., None] * (Cs @ h[:, :, :-1].transpose(3, 4))
    y = y.permute(0, 2, 3, 1, 4).reshape(n * C * Q, H, V)[there.reshape(-1)].reshape(shape)
    return {"y": _scan_gate(s, y).to(s["x"].dtype), "ht": h[:, :, -1].contiguous()}


def _plain_scan_decode(s):
    # T tokens as one small chunk on the state
    slots = s["slots"].long()
    x, step, g, Bm, Cm = _scan_inputs(s)
    T = x.shape[1]
    G = g.cumsum(1).transpose(1, 2)                                            # B H T
    low = torch.ones(T, T, device="cuda", dtype=torch.bool).tril()
    L = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -torch.inf))
    xs, Bs, Cs = ((v.transpose(1, 2)) for v in (x * step[..., None], Bm, Cm))  # B H T .
    h = s["state"][slots].float()
    y = ((Cs @ Bs.transpose(2, 3)) * L) @ xs + torch.exp(G)[..., None] * (Cs @ h.transpose(2, 3))
    h = torch.exp(G[..., -1])[..., None, None] * h + \
        (xs * torch.exp(G[..., -1:] - G)[..., None]).transpose(2, 3) @ Bs
    s["state"][slots] = h.to(s["state"].dtype)
    return {"y": _scan_gate(s, y.transpose(1, 2)).to(s["x"].dtype), "state": s["state"]}


# ---------------------------------------------------------------- one pass

def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd,
                "conv_decode": _plain_conv_decode, "scan": _plain_scan,
                "scan_decode": _plain_scan_decode}[op](s)
    import gated_delta_rule_kk_gb300 as gdn
    if op == "conv_fwd":
        y, ht = gdn.short_conv_fwd(s["x"], s["weight"], bias=s["bias"], initial_state=s.get("h0"),
                                   cu_seqlens=s.get("cu"), activation=s["act"])
        return {"y": y, "ht": ht}
    if op == "conv_bwd":
        dx, dw, db, dh0 = gdn.short_conv_bwd(s["dy"], s["x"], s["weight"], bias=s["bias"],
                                             initial_state=s.get("h0"), dfinal_state=s.get("dht"),
                                             cu_seqlens=s.get("cu"), activation=s["act"])
        return {k: v for k, v in (("dx", dx), ("dw", dw), ("db", db), ("dh0", dh0)) if v is not None}
    if op == "conv_decode":
        y = gdn.short_conv_decode(s["x"], s["weight"], s["state"], bias=s["bias"],
                                  slot_indices=s["slots"], activation=s["act"])
        return {"y": y, "state": s["state"]}
    if op == "scan":
        y, ht = gdn.ssm_chunk_fwd(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], D=s["D"], z=s["z"],
                                  dt_bias=s["dt_bias"], initial_state=s.get("h0"),
                                  cu_seqlens=s.get("cu"))
        return {"y": y, "ht": ht}
    y = gdn.ssm_decode(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], s["state"], D=s["D"], z=s["z"],
                       dt_bias=s["dt_bias"], slot_indices=s["slots"])
    return {"y": y, "state": s["state"]}


def work(case):
    """Bytes with every input read and output written once; operations of the recurrence."""
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("conv"):
        D, W = case["D"], case["W"]
        if case["op"] == "conv_decode":
            tokens, states = case["B"] * case["T"], 2 * case["B"]
        else:
            tokens, states = case["T"], case["seqs"] * (2 if case["h0"] else 1)
        flops = tokens * D * 2 * W
        if case["op"] == "conv_bwd":
            states = case["seqs"] * (3 if case["h0"] else 0)
            return {"bytes": e * D * (3 * tokens + states * (W - 1) + W) + 4 * D * W, "flops": 3 * flops}
        return {"bytes": e * D * (2 * tokens + states * (W - 1) + W), "flops": flops}
    H, Hg, V, K = (case[k] for k in ("H", "Hg", "V", "K"))
    tokens = case["T"] * case.get("B", 1)
    row = e * (H * V * (3 if case["z"] else 2) + 2 * Hg * K + H)
    if case["op"] == "scan":
        states = 4 * case["seqs"] * (2 if case["h0"] else 1)
    else:
        states = (4 if case["state"] == "f32" else 2) * 2 * case["B"]
    return {"bytes": tokens * row + states * H * V * K, "flops": tokens * H * 4 * V * K}


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f64 = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    return {"conv_fwd": _exact_conv_fwd, "conv_bwd": _exact_conv_bwd,
            "conv_decode": _exact_conv_decode, "scan": _exact_scan,
            "scan_decode": _exact_scan_decode}[case["op"]](s, f64)


def _each(s):
    """(n, row, first, last + 1) of every sequence: its index, its batch row and its tokens there."""
    x = s["x"]
    if "cu" in s:
        cu = s["cu"].tolist()
        return [(n, 0, a, b) for n, (a, b) in enumerate(zip(cu, cu[1:]))]
    return [(n, n, 0, x.shape[1]) for n in range(x.shape[0])]


def _one_conv(x, before, w, bias):
    """Pre-activation of one sequence [T, D] after the rows `before`, and all its rows."""
    rows = torch.cat([before, x])
    W = w.shape[1]
    p = x.new_zeros(x.shape)
    for i in range(W):
        p += rows[i:i + x.shape[0]] * w[:, i]
    return (p if bias is None else p + bias), rows


def _exact_conv_fwd(s, f):
    W, D = s["case"]["W"], s["case"]["D"]
    y, ht = torch.zeros_like(f["x"]), f["x"].new_zeros(s["case"]["seqs"], W - 1, D)
    for n, b, lo, hi in _each(s):
        before = f["h0"][n] if "h0" in f else f["x"].new_zeros(W - 1, D)
        p, rows = _one_conv(f["x"][b, lo:hi], before, f["weight"], f.get("bias"))
        y[b, lo:hi] = p / (1 + torch.exp(-p)) if s["act"] else p
        ht[n] = rows[rows.shape[0] - (W - 1):]
    return {"y": y, "ht": ht}


def _exact_conv_bwd(s, f):
    W, D = s["case"]["W"], s["case"]["D"]
    dx = torch.zeros_like(f["x"])
    dw, db = f["x"].new_zeros(D, W), f["x"].new_zeros(D)
    dh0 = f["x"].new_zeros(s["case"]["seqs"], W - 1, D)
    for n, b, lo, hi in _each(s):
        before = f["h0"][n] if "h0" in f else f["x"].new_zeros(W - 1, D)
        p, rows = _one_conv(f["x"][b, lo:hi], before, f["weight"], f.get("bias"))
        dp, T = f["dy"][b, lo:hi], hi - lo
        if s["act"]:
            e = 1 / (1 + torch.exp(-p))
            dp = dp * e * (1 + p * (1 - e))
        dr = torch.zeros_like(rows)
        for i in range(W):
            dr[i:i + T] += dp * f["weight"][:, i]
            dw[:, i] += (dp * rows[i:i + T]).sum(0)
        if "dht" in f:
            dr[rows.shape[0] - (W - 1):] += f["dht"][n]
        db += dp.sum(0)
        dx[b, lo:hi], dh0[n] = dr[W - 1:], dr[:W - 1]
    out = {"dx": dx, "dw": dw}
    if s["bias"] is not None:
        out["db"] = db
    if "h0" in f:
        out["dh0"] = dh0
    return out


def _exact_conv_decode(s, f):
    y, state, T = torch.zeros_like(f["x"]), f["state"].clone(), f["x"].shape[1]
    for b, slot in enumerate(s["slots"].tolist()):
        p, rows = _one_conv(f["x"][b], f["state"][slot], f["weight"], f.get("bias"))
        y[b] = p / (1 + torch.exp(-p)) if s["act"] else p
        state[slot] = rows[T:]
    return {"y": y, "state": state}


def _recurrence(s, f, h, x, dt, Bm, Cm):
    """Token by token over [n, T, ...]: outputs before the gate, and the last
    state.  A step of exactly zero (padding) leaves the state as it is."""
    rep = s["case"]["H"] // s["case"]["Hg"]
    a = -torch.exp(f["A_log"])
    ys = torch.zeros_like(x)
    for t in range(x.shape[1]):
        h = torch.exp(a * dt[:, t])[:, :, None, None] * h
        h += (dt[:, t, :, None] * x[:, t])[..., None] * Bm[:, t].repeat_interleave(rep, 1)[:, :, None]
        ys[:, t] = (h @ Cm[:, t].repeat_interleave(rep, 1)[..., None])[..., 0]
    return ys, h


def _steps(f):
    v = f["dt"] + f["dt_bias"]
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _gated(s, f, y):
    y = y + f["D"][:, None] * f["x"]
    if s["z"] is not None:
        y = y * f["z"] / (1 + torch.exp(-f["z"]))
    return y


def _exact_scan(s, f):
    H, V, K, n = (s["case"][k] for k in ("H", "V", "K", "seqs"))
    h = f["h0"] if "h0" in f else f["x"].new_zeros(n, H, V, K)
    each, step = _each(s), _steps(f)
    most = max(hi - lo for _, _, lo, hi in each)

    def side_by_side(v):
        out = v.new_zeros(n, most, *v.shape[2:])
        for i, b, lo, hi in each:
            out[i, :hi - lo] = v[b, lo:hi]
        return out

    ys, h = _recurrence(s, f, h, *(side_by_side(v) for v in (f["x"], step, f["Bm"], f["Cm"])))
    y = torch.zeros_like(f["x"])
    for i, b, lo, hi in each:
        y[b, lo:hi] = ys[i, :hi - lo]
    return {"y": _gated(s, f, y), "ht": h}


def _exact_scan_decode(s, f):
    slots = s["slots"].long()
    ys, h = _recurrence(s, f, f["state"][slots], f["x"], _steps(f), f["Bm"], f["Cm"])
    state = f["state"].clone()
    state[slots] = h
    return {"y": _gated(s, f, ys), "state": state}
