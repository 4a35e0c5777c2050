"""Cases of the chunked gated delta rule's gradient, of the per-channel gated
delta rule for single tokens, and of the group norm that follows a recurrence.

Each case is one call of one operator: the gradient of the chunked forward over
prompts; T = 1..4 tokens against a pool of states, with one log-gate per key
channel; the norm over groups of channels of every token with its activation or
gate, forward and backward.  ``run`` computes the plain form in 32 bits, or calls
the library's operator when ``own`` is set; ``exact`` computes the definition in
64 bits, token by token for the recurrences.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a training step's layer: two rows of 4096 tokens, 16 heads of 128 x 128
        dict(name="delta-bwd-prompt", op="delta_bwd", dtype="bf16", seqs=2, T=8192, cut=0, H=16,
             Hg=16, K=128, V=128, h0=False),
        # eight packed documents carried on from states, four value heads a key head
        dict(name="delta-bwd-packed", op="delta_bwd", dtype="bf16", seqs=8, T=32068, cut=3, H=16,
             Hg=4, K=128, V=128, h0=True),
        # odd head sizes and lengths, float32: the exact path
        dict(name="delta-bwd-odd-f32", op="delta_bwd", dtype="f32", seqs=3, T=1001, cut=5, H=12,
             Hg=4, K=48, V=40, h0=True),
        # one short row of a small model: the smallest training call
        dict(name="delta-bwd-short", op="delta_bwd", dtype="bf16", seqs=1, T=130, cut=0, H=8, Hg=8,
             K=64, V=64, h0=False),
        # one new token of 256 requests, bfloat16 states
        dict(name="kda-token-256", op="kda_decode", dtype="bf16", state="bf16", B=256, T=1, H=32,
             HV=32, K=128, V=128),
        # four drafted tokens of three requests, float32 states, grouped key heads
        dict(name="kda-token-few", op="kda_decode", dtype="bf16", state="f32", B=3, T=4, H=8,
             HV=32, K=128, V=128),
        # one new token of one request: where latency counts
        dict(name="kda-token-1", op="kda_decode", dtype="bf16", state="bf16", B=1, T=1, H=16,
             HV=16, K=128, V=128),
        # the output norm of 16 heads of 128 with its SiLU gate, 2 x 4096 tokens
        dict(name="norm-prompt", op="norm_fwd", dtype="bf16", T=8192, groups=16, width=128,
             shared=True, center=False, bias=False, z="after", act="silu", gap=0),
        # eight groups of 512 channels, mean taken off, SiLU on the result; columns of wider rows
        dict(name="norm-wide-groups", op="norm_fwd", dtype="bf16", T=32068, groups=8, width=512,
             shared=False, center=True, bias=True, z="none", act="silu", gap=4160),
        # a few tokens of odd channels, gate before the norm, float32: the smallest norm
        dict(name="norm-odd-f32", op="norm_fwd", dtype="f32", T=61, groups=3, width=257,
             shared=False, center=False, bias=True, z="before", act="silu", gap=0),
        # gradient of the output norm
        dict(name="norm-bwd-prompt", op="norm_bwd", dtype="bf16", T=8192, groups=16, width=128,
             shared=True, center=False, bias=False, z="after", act="silu", gap=0),
        # gradient over odd groups, float32, mean taken off, sigmoid gate
        dict(name="norm-bwd-odd-f32", op="norm_bwd", dtype="f32", T=3001, groups=8, width=145,
             shared=False, center=True, bias=True, z="after", act="sigmoid", gap=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta_bwd", "kda_decode", "norm_fwd", "norm_bwd"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    if op == "delta_bwd":
        K, V = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64), (48, 40), (96, 80)])
        Hg = rng.choice([1, 2, 4, 8, 16])
        H = Hg * rng.choice([1, 1, 1, 2, 4])
        top = 3_000_000 if dtype == "f32" else 60_000_000
        T = min(_log(rng, 1, 32768), max(1, top // (H * V)))
        seqs = rng.randint(1, 8)
        return dict(op=op, dtype=dtype, seqs=seqs, T=T if T % seqs else T // seqs * seqs,
                    cut=rng.randint(1, 1 << 20) if T % seqs or rng.random() < 0.5 else 0, H=H,
                    Hg=Hg, K=K, V=V, h0=rng.random() < 0.5)
    if op == "kda_decode":
        K, V = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64), (48, 40)])
        H = rng.choice([1, 2, 4, 8, 16, 32])
        HV = H * rng.choice([1, 1, 2, 4])
        state = rng.choice(["bf16", "f32"])
        B = min(_log(rng, 1, 256), max(1, (65 if state == "f32" else 130) * 10 ** 6 // (HV * K * V)))
        return dict(op=op, dtype=dtype, state=state, B=B, T=rng.randint(1, 4), H=H, HV=HV, K=K, V=V)
    width = _log(rng, 16, 4096)
    if rng.random() < 0.75:
        width = max(8, width // 8 * 8)
    groups = _log(rng, 1, max(1, 8192 // width))
    top = (30 if op == "norm_bwd" else 130) * 10 ** 6 // (2 if dtype == "f32" else 1)
    T = min(_log(rng, 1, 32768), max(1, top // (groups * width)))
    return dict(op=op, dtype=dtype, T=T, groups=groups, width=width, shared=rng.random() < 0.3,
                center=rng.random() < 0.5, bias=rng.random() < 0.5,
                z=rng.choice(["none", "after", "after", "before"]),
                act=rng.choice(["silu", "silu", "sigmoid"]), gap=rng.choice([0, 0, 64, 4160]))


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

    def unit(*shape):
        x = torch.randn(*shape, generator=g, device="cuda")
        return (x / (x * x).sum(-1, keepdim=True).sqrt()).to(dt)

    s = {"case": case}
    if case["op"].startswith("norm"):
        T, G, W, gap = (case[k] for k in ("T", "groups", "width", "gap"))
        D, lead = G * W, gap // 16 * 8

        def rows():
            return normal(1, T, gap + D)[:, :, lead:lead + D]

        s["x"] = rows()
        s["z"] = None if case["z"] == "none" else rows()
        wide = W if case["shared"] else D
        s["weight"] = normal(wide, std=0.2, mean=1.0)
        s["bias"] = normal(wide, std=0.2) if case["bias"] else None
        s["eps"] = 1e-5
        if case["op"] == "norm_bwd":
            s["dy"] = normal(1, T, D)
        return s
    K, V = case["K"], case["V"]
    if case["op"] == "delta_bwd":
        H, Hg, n = case["H"], case["Hg"], case["seqs"]
        if case["cut"]:
            s["cu"] = torch.tensor([0] + _lengths(case)).cumsum(0).to(torch.int32).cuda()
        B, T = (1, case["T"]) if case["cut"] else (n, case["T"] // n)
        s["q"], s["k"] = unit(B, T, Hg, K), unit(B, T, Hg, K)
        s["v"], s["do"] = normal(B, T, H, V), normal(B, T, H, V)
        s["g"] = -torch.log1p(torch.exp(-normal(B, T, H, mean=3.0, dtype=torch.float32)))
        s["beta"] = torch.sigmoid(normal(B, T, H, dtype=torch.float32))
        s["scale"] = K ** -0.5
        if case["h0"]:
            s["h0"] = normal(n, H, K, V, std=0.1, dtype=torch.float32)
            s["dht"] = normal(n, H, K, V, std=0.1, dtype=torch.float32)
        return s
    B, T, H, HV = (case[k] for k in ("B", "T", "H", "HV"))
    # q, k and v as columns of the short convolution's output
    conv = normal(B, T, 2 * H * K + HV * V)
    s["q"] = conv[:, :, :H * K].unflatten(2, (H, K))
    s["k"] = conv[:, :, H * K:2 * H * K].unflatten(2, (H, K))
    s["v"] = conv[:, :, 2 * H * K:].unflatten(2, (HV, V))
    s["a"], s["b"] = normal(B, T, HV, K), normal(B, T, HV)
    s["A_log"] = torch.log(torch.rand(HV, generator=g, device="cuda") * 15 + 1)
    step = torch.exp(torch.rand(HV, K, generator=g, device="cuda") * math.log(100) + math.log(1e-3))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus of it is `step`
    pool = B + B // 2 + 1
    s["state"] = normal(pool, HV, V, K, std=0.1, dtype=_DTYPES[case["state"]])
    s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:B].to(torch.int32)
    s["scale"] = K ** -0.5
    return s


# ---------------------------------------------------------------- plain forms

def _act(case, z):
    e = torch.sigmoid(z)
    return z * e if case["act"] == "silu" else e


def _dact(case, z):
    e = torch.sigmoid(z)
    return e * (1 + z * (1 - e)) if case["act"] == "silu" else e * (1 - e)


def _norm_parts(s):
    """What is normalised, its normal form and 1 / root, over [T, groups, width] in 32 bits."""
    case = s["case"]
    shape = (case["T"], case["groups"], case["width"])
    u = s["x"][0].float().reshape(shape)
    z = None if s["z"] is None else s["z"][0].float().reshape(shape)
    if case["z"] == "before":
        u = u * _act(case, z)
    c = u - u.mean(2, keepdim=True) if case["center"] else u
    r = 1 / torch.sqrt((c * c).mean(2, keepdim=True) + s["eps"])
    w, b = (None if v is None else v.float().reshape(1, -1, case["width"])
            for v in (s["weight"], s["bias"]))
    return u, z, c * r, r, w, b


def _plain_norm_fwd(s):
    case = s["case"]
    _, z, n, _, w, b = _norm_parts(s)
    m = n * w if b is None else n * w + b
    y = m * _act(case, z) if case["z"] == "after" else m if case["z"] == "before" else _act(case, m)
    return {"y": y.reshape(s["x"].shape).to(s["x"].dtype)}


def _plain_norm_bwd(s):
    case, x = s["case"], s["x"]
    _, z, n, r, w, b = _norm_parts(s)
    dy = s["dy"][0].float().reshape(n.shape)
    m = n * w if b is None else n * w + b
    dm, dz = dy, None
    if case["z"] == "after":
        dm, dz = dy * _act(case, z), dy * m * _dact(case, z)
    elif case["z"] == "none":
        dm = dy * _dact(case, m)
    dw, db = (dm * n).sum(0), dm.sum(0)
    if case["shared"]:
        dw, db = dw.sum(0), db.sum(0)
    dn = dm * w
    du = dn - n * (dn * n).mean(2, keepdim=True)
    if case["center"]:
        du = du - dn.mean(2, keepdim=True)
    dx = du = du * r
    if case["z"] == "before":
        dx, dz = du * _act(case, z), du * x[0].float().reshape(n.shape) * _dact(case, z)
    out = {"dx": dx.reshape(x.shape).to(x.dtype), "dw": dw.reshape(-1)}
    if b is not None:
        out["db"] = db.reshape(-1)
    if dz is not None:
        out["dz"] = dz.reshape(x.shape).to(x.dtype)
    return out


def _plain_kda_decode(s):
    # token by token: every token's state is the next one's
    slots = s["slots"].long()
    H, HV = s["case"]["H"], s["case"]["HV"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6) * s["scale"]
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    q, k = q.repeat_interleave(HV // H, 2), k.repeat_interleave(HV // H, 2)
    x = s["a"].float() + s["dt_bias"]
    step = torch.where(x > 20, x, torch.log1p(torch.exp(x.clamp(max=20))))
    decay = torch.exp(-torch.exp(s["A_log"])[:, None] * step)
    beta = torch.sigmoid(s["b"].float())
    h = s["state"][slots].float()
    os = []
    for t in range(v.shape[1]):
        h = h * decay[:, t, :, None, :]
        d = beta[:, t, :, None] * (v[:, t] - (h * k[:, t, :, None, :]).sum(-1))
        h = h + d[..., None] * k[:, t, :, None, :]
        os.append((h * q[:, t, :, None, :]).sum(-1))
    s["state"][slots] = h.to(s["state"].dtype)
    return {"o": torch.stack(os, 1).to(s["v"].dtype), "state": s["state"]}


def _plain_delta_bwd(s, Q=64):
    """Chunks of Q tokens: with the lower triangles A_ij = beta_i k_i.k_j e^{G_i - G_j} (i > j)
    and P_ij = q_i.k_j e^{G_i - G_j} (i >= j), the chunk's corrected values are
    n = (I + A)^-1 beta (v - e^G k h).  Forward and backward walk the chunks in turn; all that
    does not hang on the carried state is computed for every chunk at once."""
    case = s["case"]
    H, K, V, rep = case["H"], case["K"], case["V"], case["H"] // case["Hg"]
    shape = s["v"].shape
    lens = _lengths(case)
    n, C = len(lens), max(1, -(-max(lens) // Q))
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0)
    bos, lens = cu[:-1], cu[1:] - cu[:-1]
    # every sequence on its own row of C chunks; tokens past its end are zero
    pos = torch.arange(C * Q, device="cuda")
    there = pos < lens[:, None]
    at = torch.where(there, bos[:, None] + pos, 0)

    def rows(x, rep=1):
        x = x.float().reshape(-1, *x.shape[2:])[at]
        x = torch.where(there.reshape(n, C * Q, *[1] * (x.dim() - 2)), x, 0)
        return x.repeat_interleave(rep, 2).unflatten(1, (C, Q)).transpose(2, 3)  # n C H Q ...

    q, k, v, do = rows(s["q"], rep) * s["scale"], rows(s["k"], rep), rows(s["v"]), rows(s["do"])
    beta, G = rows(s["beta"])[..., None], rows(s["g"]).cumsum(3)[..., None]      # n C H Q 1
    last = torch.exp(G[..., -1:, :])                                             # n C H 1 1
    eG, eL = torch.exp(G), torch.exp(G[..., -1:, :] - G)
    low = torch.ones(Q, Q, device="cuda", dtype=torch.bool).tril()
    L = torch.exp(torch.where(low, G - G.transpose(3, 4), -torch.inf))
    P = (q @ k.transpose(3, 4)) * L
    A = (k @ k.transpose(3, 4)) * L * beta * low.tril(-1)
    inv = torch.eye(Q, device="cuda") - A
    A2 = A @ A
    for _ in range(5):  # (I - A)(I + A^2)(I + A^4)... = (I + A)^-1, as A^64 = 0
        inv, A2 = inv + inv @ A2, A2 @ A2
    w, new = inv @ (beta * eG * k), inv @ (beta * v)
    h = s["h0"] if "h0" in s else v.new_zeros(n, H, K, V)
    hs = v.new_empty(n, C, H, K, V)
    for c in range(C):
        hs[:, c] = h
        new[:, c] -= w[:, c] @ h
        h = last[:, c] * h + (k[:, c] * eL[:, c]).transpose(2, 3) @ new[:, c]
    dnew = P.transpose(3, 4) @ do
    d = s["dht"] if "dht" in s else v.new_zeros(n, H, K, V)
    ds = v.new_empty(n, C, H, K, V)
    for c in range(C - 1, -1, -1):
        ds[:, c] = d
        dnew[:, c] += (k[:, c] * eL[:, c]) @ d
        d = last[:, c] * d + (q[:, c] * eG[:, c]).transpose(2, 3) @ do[:, c] \
            - w[:, c].transpose(2, 3) @ dnew[:, c]
    dr = inv.transpose(3, 4) @ dnew                     # of beta (v - e^G k h)
    dA = -(dr @ new.transpose(3, 4)) * low.tril(-1)
    dP = (do @ new.transpose(3, 4)) * low
    dqh = eG * (do @ hs.transpose(3, 4))                # of q, through the state
    dkh = -eG * beta * (dr @ hs.transpose(3, 4))        # of k, in front of the state
    dks = eL * (new @ ds.transpose(3, 4))               # of k, into the state
    dPL, dAL = dP * L, dA * L * beta
    dq = dqh + dPL @ k
    dk = dkh + dks + dPL.transpose(3, 4) @ q + (dAL + dAL.transpose(3, 4)) @ k
    MA, MP = dA * A, dP * P
    M = MA + MP
    dks_k = (dks * k).sum(4, keepdim=True)
    dG = M.sum(4, keepdim=True) - M.sum(3)[..., None] + (dqh * q).sum(4, keepdim=True) \
        + (dkh * k).sum(4, keepdim=True) - dks_k
    dG[..., -1, :] += (last * hs * ds).sum((3, 4))[..., None] + dks_k.sum(3)
    dg = dG.flip(3).cumsum(3).flip(3)
    safe = (dr * v).sum(4, keepdim=True)
    dbeta = safe + (MA.sum(4, keepdim=True) + (dkh * k).sum(4, keepdim=True)) / torch.where(beta == 0, 1, beta)

    def back(x, like):
        x = x.transpose(2, 3).reshape(n * C * Q, H, -1)[there.reshape(-1)]
        if like.shape[2] != H:
            x = x.unflatten(1, (like.shape[2], -1)).sum(2)
        return x.reshape(like.shape).to(like.dtype)

    out = {"dq": back(dq * s["scale"], s["q"]), "dk": back(dk, s["k"]), "dv": back(beta * dr, s["v"]),
           "dg": back(dg, s["g"]), "dbeta": back(dbeta, s["beta"])}
    assert out["dv"].shape == shape
    if "h0" in s:
        out["dh0"] = d
    return out


# ---------------------------------------------------------------- one pass

def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"delta_bwd": _plain_delta_bwd, "kda_decode": _plain_kda_decode,
                "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}[op](s)
    import gated_delta_rule_kk_gb300 as gdn
    case = s["case"]
    if op == "delta_bwd":
        dq, dk, dv, dg, dbeta, dh0 = gdn.gdn_chunk_bwd(
            s["do"], s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"],
            initial_state=s.get("h0"), dfinal_state=s.get("dht"), cu_seqlens=s.get("cu"))
        out = {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta}
        return out if dh0 is None else out | {"dh0": dh0}
    if op == "kda_decode":
        o = gdn.kda_decode(s["q"], s["k"], s["v"], s["a"], s["b"], s["A_log"], s["dt_bias"],
                           s["state"], scale=s["scale"], slot_indices=s["slots"])
        return {"o": o, "state": s["state"]}
    how = dict(weight=s["weight"], bias=s["bias"], z=s["z"], eps=s["eps"], center=case["center"],
               activation=case["act"], gate_first=case["z"] == "before")
    if op == "norm_fwd":
        return {"y": gdn.group_norm_fwd(s["x"], case["groups"], **how)}
    dx, dw, db, dz = gdn.group_norm_bwd(s["dy"], s["x"], case["groups"], **how)
    return {k: v for k, v in (("dx", dx), ("dw", dw), ("db", db), ("dz", dz)) if v is not None}


def work(case):
    """Bytes with every input read and output written once; operations of the recurrence (a
    token's state is decayed, read, corrected and read again: 6 K V, and for its gradient the
    states once more and their gradients twice that)."""
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("norm"):
        n, D = case["T"] * case["groups"] * case["width"], case["groups"] * case["width"]
        wide = case["width"] if case["shared"] else D
        gate, par = case["z"] != "none", 2 if case["bias"] else 1
        if case["op"] == "norm_fwd":
            return {"bytes": e * (n * (3 if gate else 2) + par * wide), "flops": 10 * n}
        return {"bytes": e * (n * (5 if gate else 3) + par * wide) + 4 * par * wide, "flops": 25 * n}
    K, V = case["K"], case["V"]
    if case["op"] == "kda_decode":
        H, HV, tokens = case["H"], case["HV"], case["B"] * case["T"]
        states = (4 if case["state"] == "f32" else 2) * 2 * case["B"] * HV * K * V
        return {"bytes": states + tokens * e * (2 * H * K + 2 * HV * V + HV * K + HV) + 4 * HV * (K + 1),
                "flops": tokens * HV * 7 * K * V}
    H, Hg, tokens = case["H"], case["Hg"], case["T"]
    states = 4 * case["seqs"] * H * K * V * (3 if case["h0"] else 0)
    return {"bytes": tokens * (e * (4 * Hg * K + 3 * H * V) + 16 * H) + states,
            "flops": tokens * H * 18 * K * V}


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f64 = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    return {"delta_bwd": _exact_delta_bwd, "kda_decode": _exact_kda_decode,
            "norm_fwd": _exact_norm, "norm_bwd": _exact_norm}[case["op"]](s, f64)


def _exact_norm(s, f):
    """The definition as one expression; its gradient by differentiating that."""
    case = s["case"]
    f = {k: v.clone().requires_grad_(k != "dy") for k, v in f.items()}
    act = {"silu": lambda z: z / (1 + torch.exp(-z)), "sigmoid": lambda z: 1 / (1 + torch.exp(-z))}[case["act"]]
    u = f["x"] * act(f["z"]) if case["z"] == "before" else f["x"]
    u = u.unflatten(2, (case["groups"], case["width"]))
    if case["center"]:
        u = u - u.sum(3, keepdim=True) / case["width"]
    n = u * ((u * u).sum(3, keepdim=True) / case["width"] + s["eps"]) ** -0.5
    w, b = f["weight"].reshape(-1, case["width"]), f.get("bias")
    m = n * w if b is None else n * w + b.reshape(-1, case["width"])
    m = m.flatten(2)
    y = m * act(f["z"]) if case["z"] == "after" else m if case["z"] == "before" else act(m)
    if case["op"] == "norm_fwd":
        return {"y": y.detach()}
    names = [(o, i) for o, i in (("dx", "x"), ("dw", "weight"), ("db", "bias"), ("dz", "z")) if i in f]
    grads = torch.autograd.grad(y, [f[i] for _, i in names], f["dy"])
    return {o: d for (o, _), d in zip(names, grads)}


def _exact_kda_decode(s, f):
    H, HV = s["case"]["H"], s["case"]["HV"]
    slots = s["slots"].long()
    state, o = f["state"].clone(), torch.zeros_like(f["v"])
    h = state[slots]                                                   # B HV V K
    for t in range(o.shape[1]):
        x = f["a"][:, t] + f["dt_bias"]
        g = -torch.exp(f["A_log"])[:, None] * (torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs())))
        q, k = ((v / (v.square().sum(-1, keepdim=True) + 1e-6).sqrt()).repeat_interleave(HV // H, 1)
                for v in (f["q"][:, t], f["k"][:, t]))
        h = torch.exp(g)[:, :, None] * h
        d = (f["v"][:, t] - (h @ k[..., None])[..., 0]) / (1 + torch.exp(-f["b"][:, t, :, None]))
        h = h + d[..., None] * k[:, :, None]
        o[:, t] = s["scale"] * (h @ q[..., None])[..., 0]
    state[slots] = h
    return {"o": o, "state": state}


def _exact_delta_bwd(s, f):
    """Token by token: h' = e^g h, d = beta (v - k h'), h = h' + k d, o = scale q h, and back."""
    case = s["case"]
    H, K, V, rep = case["H"], case["K"], case["V"], case["H"] // case["Hg"]
    out = {"dq": torch.zeros_like(f["q"]), "dk": torch.zeros_like(f["k"]), "dv": torch.zeros_like(f["v"]),
           "dg": torch.zeros_like(f["g"]), "dbeta": torch.zeros_like(f["beta"])}
    if case["cut"]:
        cu = s["cu"].tolist()
        each = [[0, a, b, [i]] for i, (a, b) in enumerate(zip(cu, cu[1:]))]
    else:  # equal sequences side by side
        each = [[slice(None), 0, f["q"].shape[1], list(range(case["seqs"]))]]
    dh0 = f["v"].new_zeros(case["seqs"], H, K, V)
    for rows, lo, hi, which in each:
        pick = [rows] if rows == 0 else rows
        q, k = (f[i][pick, lo:hi].repeat_interleave(rep, 2) for i in ("q", "k"))
        v, do, g, beta = (f[i][pick, lo:hi] for i in ("v", "do", "g", "beta"))
        h = f["h0"][which] if "h0" in f else v.new_zeros(len(which), H, K, V)
        kept = []
        for t in range(hi - lo):
            kept.append(h)
            h = torch.exp(g[:, t])[..., None, None] * h
            d = beta[:, t, :, None] * (v[:, t] - (k[:, t, :, None] @ h)[:, :, 0])
            h = h + k[:, t, :, :, None] * d[:, :, None]
        G = f["dht"][which] if "dht" in f else torch.zeros_like(h)
        dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, beta))
        for t in range(hi - lo - 1, -1, -1):
            decay = torch.exp(g[:, t])[..., None, None]
            before = decay * kept.pop()
            kt, qt, dot = k[:, t, :, :, None], q[:, t, :, :, None], do[:, t, :, None]
            miss = v[:, t, :, None] - kt.transpose(2, 3) @ before        # 1 x V
            bt = beta[:, t, :, None, None]
            dq[:, t] = s["scale"] * (h @ dot.transpose(2, 3))[..., 0]
            G = G + s["scale"] * qt * dot
            dd = kt.transpose(2, 3) @ G
            dk[:, t] = (bt * (G @ miss.transpose(2, 3)) - bt * (before @ dd.transpose(2, 3)))[..., 0]
            dv[:, t] = bt[..., 0] * dd[:, :, 0]
            db[:, t] = (dd * miss).sum((2, 3))
            G = G - bt * kt * dd
            dg[:, t] = (before * G).sum((2, 3))
            G = decay * G
            h = before / decay
        dh0[which] = G
        for name, x, by in (("dq", dq, rep), ("dk", dk, rep), ("dv", dv, 1), ("dg", dg, 1), ("dbeta", db, 1)):
            out[name][pick, lo:hi] = x.unflatten(2, (-1, by)).sum(3) if by > 1 else x
    return out | {"dh0": dh0} if "h0" in s else out
