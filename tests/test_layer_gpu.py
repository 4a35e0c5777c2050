"""The gated delta rule's gradient, KDA's tokens and the norm over groups of channels on the
GPU against their definitions in fp64.

Bounds.  float32 paths: the library's 1e-4 RMS for the recurrences, whose longest sums have
some 200 terms over a few chunks; 1e-5 RMS for the norm and KDA's tokens (sums of up to 8192
products of order one in a tree, and hardware exponentials and reciprocals to a few 2^-23).
The gradient on the tensor cores: pairs of bfloat16 pieces are off by 2^-17 of a value and
their product by 2^-16 with the dropped term; at most six such products follow one another (T,
n, h, dn, dr, D), each a sum of up to 256 terms whose magnitudes add up to at most 32 RMS:
6 x 2^-16 x 32 = 3e-3 RMS element for element, besides a bfloat16 output's own half step.  In
norm the pieces' errors are independent: 2^-19 of a value each, some 20 of them that matter in
quadrature, 1e-5.
"""
import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

import gated_delta_rule_kk_gb300 as gdn
from gated_delta_rule_kk_gb300 import GdnError, Status, _lib, build_lib
from gated_delta_rule_kk_gb300._lib import GdnChunkBwdArgs
from oracle import layer as L

from _layer import delta_inputs, kda_inputs, norm_inputs
from _mixer import assert_each_close, cuda
from _util import TOL_F32, _np

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
PIECES, NORM = 3e-3, 1e-5


def ok():
    assert gdn.gdn_check_device_error() == Status.OK


def run_delta(d, **kw):
    return gdn.gdn_chunk_bwd(d["do"], d["q"], d["k"], d["v"], d["g"], d["beta"], scale=d["scale"],
                             initial_state=d["h0"], dfinal_state=d["dht"], cu_seqlens=d["cu"], **kw)


def check_delta(got, i, cumsum=False, v_first=False, pieces=True, norm=True):
    h0, dht = (None if i[s] is None else i[s].transpose(2, 3) if v_first else i[s]
               for s in ("h0", "dht"))
    ref = L.gdn_grad(i["do"], i["q"], i["k"], i["v"], i["g"], i["beta"], i["scale"], h0, dht,
                     i["cu"], cumsum)
    if v_first:
        ref = (*ref[:5], ref[5].transpose(0, 1, 3, 2))
    for name, x, r in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got, ref):
        if x is None:
            continue
        assert_each_close(x, r, name, PIECES if pieces else TOL_F32)
        if norm and pieces and x.dtype is F32 and x.numel():
            off = ((_np(x) - r) ** 2).sum() ** 0.5 / max((r ** 2).sum() ** 0.5, 1e-30)
            assert off <= 1e-5, f"{name}: {off:.2e} of its norm"


# (B, T, H, Hg, K, V, lens): one token; ends before, at and behind a chunk's; grouped heads;
# packed with empty and one-token sequences; heads that do not fill a tile
DELTA = [
    (1, 1, 1, 1, 128, 128, None),
    (2, 63, 2, 2, 128, 128, None),
    (1, 64, 2, 1, 64, 64, None),
    (1, 65, 4, 1, 128, 64, None),
    (1, 200, 3, 3, 8, 8, None),
    (2, 129, 4, 2, 96, 40, None),
    (1, 70, 2, 2, 120, 104, None),
    (1, 300, 4, 4, 64, 128, [0, 1, 64, 0, 65, 170, 0]),
    (1, 260, 6, 2, 128, 128, [130, 2, 128]),
]


@pytest.mark.parametrize("B,T,H,Hg,K,V,lens", DELTA)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("states,cumsum,v_first", [(True, False, False), (False, True, False),
                                                   (True, True, True)])
def test_delta_gradient(B, T, H, Hg, K, V, lens, dtype, states, cumsum, v_first):
    i = delta_inputs(T + K, B, T, H, Hg, K, V, dtype, lens, states, cumsum, v_first=v_first)
    got = run_delta(cuda(i), g_is_cumsum=cumsum, state_v_first=v_first,
                    output_dinitial_state=True)
    ok()
    # (the norm's bound counts on many independent errors)
    check_delta(got, i, cumsum, v_first, pieces=dtype is BF16, norm=T * H >= 200)


@pytest.mark.parametrize("K,V", [(20, 12), (33, 7), (128, 136), (1, 1), (100, 200)])
def test_delta_gradient_of_odd_heads_in_bfloat16(K, V):
    i = delta_inputs(K, 1, 131, 2, 1, K, V, BF16, [66, 65])
    got = run_delta(cuda(i))
    ok()
    check_delta(got, i, pieces=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_delta_gradient_of_resets_and_of_beta_zero(dtype):
    """Gates of e^-30 (what came before is gone) and tokens that write nothing."""
    i = delta_inputs(9, 1, 150, 4, 2, 64, 64, dtype, [81, 69], reset=True, zero_beta=True)
    got = run_delta(cuda(i))
    ok()
    check_delta(got, i, pieces=dtype is BF16)
    # A reset token's gate has next to no effect, so its dg is what rounding leaves: dg is a
    # running sum whose value at every step is that token's dg, each of the up to 64 steps
    # rounds by 2^-24 of it, and the terms that cancel (a row's and a column's sum) by as much
    # again.  So at most 128 x 2^-24 of the largest dg; a difference of long sums, or a rounding
    # to bfloat16, would be 2^-17 of terms of order one from each of 64 tokens.
    assert got[3][:, ::5].abs().max() <= 2.0 ** -17 * got[3].abs().max()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gate", [-float("inf"), -3.4e38, -1e4, -150.0])
def test_delta_gradient_of_gates_that_forget_all(dtype, gate):
    i = delta_inputs(19, 1, 150, 2, 2, 64, 64, dtype, [90, 60])
    i["g"][:, [0, 40, 41, 100]] = gate
    got = run_delta(cuda(i))
    ok()
    check_delta(got, i, pieces=dtype is BF16, norm=False)


@pytest.mark.parametrize("dtype,K", [(BF16, 16), (F32, 12)])
def test_delta_gradient_of_more_sequences_than_threads(dtype, K):
    """1100 sequences of nothing to a few tokens, some of several chunks: the order in which
    they are taken is by their lengths."""
    lens = [n % 3 for n in range(1100)]
    lens[5], lens[700], lens[1099] = 200, 65, 130
    i = delta_inputs(17, 1, sum(lens), 1, 1, K, K, dtype, lens)
    got = run_delta(cuda(i))
    ok()
    check_delta(got, i, pieces=dtype is BF16, norm=False)


def test_delta_gradient_of_beta_next_to_zero():
    """Products of a tiny beta and a tiny gradient are not lost."""
    i = delta_inputs(20, 1, 130, 2, 2, 64, 64, BF16)
    i["beta"][:, ::3] *= 1e-25
    i["do"], i["dht"] = i["do"] * 2.0 ** -50, i["dht"] * 2.0 ** -50
    dbeta = run_delta(cuda(i))[4]
    ok()
    ref = L.gdn_grad(i["do"], i["q"], i["k"], i["v"], i["g"], i["beta"], i["scale"], i["h0"],
                     i["dht"], i["cu"])[4]
    assert_each_close(dbeta, ref, "dbeta", PIECES)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", ["v", "do"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_delta_gradient_keeps_what_is_not_finite_in_its_sequence_and_head(dtype, name, value):
    i = cuda(delta_inputs(21, 1, 400, 4, 2, 64, 64, dtype, [90, 210, 0, 100]))
    clean = run_delta(i)
    i[name] = i[name].clone()
    i[name][0, 200, 1, 7] = value  # of the second sequence, the first key head's second head
    got = run_delta(i)
    ok()
    for what, a, b in zip(("dq", "dk", "dv", "dg", "dbeta"), clean, got):
        # (o is linear in v: its gradient is without v)
        assert torch.equal(a, b) if (name, what) == ("v", "dv") else not b.isfinite().all(), what
        heads = slice(1, None) if what in ("dq", "dk") else [0, 2, 3]
        assert torch.equal(a[:, :, heads], b[:, :, heads]), what
        assert torch.equal(a[:, :90], b[:, :90]) and torch.equal(a[:, 300:], b[:, 300:]), what
    assert torch.equal(clean[5][[0, 2, 3]], got[5][[0, 2, 3]])
    assert torch.equal(clean[5][:, [0, 2, 3]], got[5][:, [0, 2, 3]])


def test_delta_gradient_of_growing_states():
    """Gates above zero: the running sums grow to +20 within a chunk."""
    i = delta_inputs(10, 1, 130, 2, 2, 64, 64, BF16)
    i["g"] = i["g"].abs() * 2
    i["beta"] *= 0.1
    got = run_delta(cuda(i))
    ok()
    check_delta(got, i, norm=False)


def test_delta_gradient_joins_the_forward():
    """Differences of the library's own forward, in float32 along a random direction."""
    i = delta_inputs(11, 2, 100, 2, 2, 32, 32, F32)
    d = cuda(i)
    grads = run_delta(d)
    ok()

    def loss(x):
        o, ht = gdn.gdn_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], scale=i["scale"],
                                  initial_state=x["h0"])
        return (o.double() * d["do"]).sum() + (ht.double() * d["dht"]).sum()

    g = torch.Generator().manual_seed(0)
    for name, grad in zip(("q", "k", "v", "g", "beta", "h0"), grads):
        way = torch.randn(grad.shape, generator=g).cuda()
        e = 1e-2
        diff = (loss({**d, name: d[name] + e * way}) - loss({**d, name: d[name] - e * way})) / (2 * e)
        # e^2 / 6 of the third derivative along the way (|way|^3 over the gradient's size), and
        # float32 outputs' rounding, 2^-24 sqrt(12800) over e
        size = float(grad.double().norm() * way.double().norm())
        assert abs(float(diff - (grad.double() * way).sum())) <= 2e-2 * size


def test_delta_gradient_repeats_and_replays():
    i = delta_inputs(12, 1, 400, 4, 2, 128, 128, BF16, [150, 250])
    d = cuda(i)
    first = run_delta(d)
    again = run_delta(d)
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run_delta(d)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run_delta(d)
    other = cuda(delta_inputs(13, 1, 400, 4, 2, 128, 128, BF16, [150, 250]))
    for name in ("do", "q", "k", "v", "g", "beta", "h0", "dht"):
        d[name].copy_(other[name])
    graph.replay()
    for a, b in zip(held, run_delta(other)):
        assert torch.equal(a, b)
    with torch.cuda.stream(s):
        there = run_delta(d, stream=s)
    s.synchronize()
    for a, b in zip(held, there):
        assert torch.equal(a, b)
    ok()


@pytest.mark.parametrize("dtype,K", [(BF16, 64), (F32, 20)])
@pytest.mark.parametrize("cu", [[0, 40, 30, 70], [0, 40, 71], [1, 70], [0, 69]])
def test_delta_gradient_with_bad_offsets_writes_nothing(dtype, K, cu):
    N = len(cu) - 1
    i = delta_inputs(14, 1, 70, 2, 2, K, K, dtype, [70] + [0] * (N - 1))
    d = cuda(i)
    d["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    outs = {n: torch.full_like(d[t], 7.0) for n, t in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"),
                                                       ("dbeta", "beta"), ("dh0", "h0"))}
    a = GdnChunkBwdArgs(dtype=int(dtype is BF16), B=1, T=70, H=2, Hg=2, K=K, V=K, N=N, chunk_size=64,
                        **{n: d[n].data_ptr() for n in ("q", "k", "v", "g", "beta", "h0", "dht")},
                        do_=d["do"].data_ptr(), cu_seqlens=d["cu"].data_ptr(),
                        **{n: t.data_ptr() for n, t in outs.items()})
    n = ctypes.c_size_t(0)
    lib = _lib.load()
    assert lib.gdn_chunk_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n)) == Status.OK
    room = torch.empty(n.value, dtype=torch.uint8, device="cuda")
    a.workspace, a.workspace_bytes = room.data_ptr(), n.value
    assert lib.gdn_chunk_bwd(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == Status.OK
    assert gdn.gdn_check_device_error() == Status.BAD_SEQLENS
    for x in outs.values():
        assert torch.equal(x, torch.full_like(x, 7.0))


def test_delta_gradient_without_tokens():
    i = delta_inputs(15, 2, 0, 2, 2, 64, 64, BF16)
    d = cuda(i)
    *grads, dh0 = run_delta(d)
    assert all(g.numel() == 0 for g in grads) and torch.equal(dh0, d["dht"])
    d["dht"] = None
    assert not run_delta(d)[5].any()
    ok()


def test_delta_gradient_past_2_31_elements():
    """q and k of 2^31 + elements: the last rows are those of a call of their own."""
    B, T, K, V = 4097, 4096, 128, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k = (torch.empty(B, T, 1, K, device="cuda", dtype=BF16).normal_(std=0.09, generator=g)
            for _ in range(2))
    assert q.numel() > 1 << 31
    v, do = (torch.empty(B, T, 1, V, device="cuda", dtype=BF16).normal_(generator=g) for _ in range(2))
    gate = torch.full((B, T, 1), -0.1, device="cuda")
    beta = torch.full((B, T, 1), 0.5, device="cuda")
    got = gdn.gdn_chunk_bwd(do, q, k, v, gate, beta)
    one = gdn.gdn_chunk_bwd(*(x[-1:].contiguous() for x in (do, q, k, v, gate, beta)))
    for a, b in zip(got[:5], one[:5]):
        assert torch.equal(a[-1:], b)
    ok()


def test_delta_gradient_refusals_in_python():
    d = cuda(delta_inputs(16, 1, 10, 2, 2, 16, 16, BF16))
    for change in (dict(q=d["q"].float()), dict(do=d["do"].float()), dict(g=d["g"].double()),
                   dict(v=d["v"][:, :5]), dict(k=d["k"].transpose(1, 2)), dict(scale=-1.0),
                   dict(h0=d["h0"][:, :1]), dict(cu=torch.tensor([0, 10], device="cuda"))):
        with pytest.raises(ValueError):
            run_delta({**d, **change})
    with pytest.raises(ValueError):
        run_delta(d, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(GdnError):
        run_delta(cuda(delta_inputs(16, 1, 10, 2, 2, 136, 16, BF16)))


# ---------------------------------------------------------------- KDA, single tokens

# (B, T, H, HV, K, V, gap): the smallest; odd V; grouped; every width of a row; more states
# than blocks, so that they stream; rows wider than q, k and v that begin anywhere
KDA = [
    (1, 1, 1, 1, 8, 1, 0), (2, 4, 2, 4, 48, 40, 0), (3, 2, 1, 3, 64, 33, 6), (2, 3, 2, 2, 128, 128, 2),
    (1, 4, 1, 2, 256, 100, 0), (5, 1, 4, 8, 200, 17, 16), (64, 1, 4, 8, 128, 128, 0),
    (90, 4, 2, 4, 128, 64, 2), (40, 2, 8, 16, 64, 128, 0), (60, 3, 4, 8, 256, 64, 0),
]


@pytest.mark.parametrize("B,T,H,HV,K,V,gap", KDA)
@pytest.mark.parametrize("dtype,state", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_kda_tokens(B, T, H, HV, K, V, gap, dtype, state):
    i = kda_inputs(B + K, B, T, H, HV, K, V, dtype, state, gap)
    d = cuda(i)
    before = d["state"].clone()
    o = gdn.kda_decode(d["q"], d["k"], d["v"], d["a"], d["b"], d["A_log"], d["dt_bias"], d["state"],
                       slot_indices=d["slots"])
    ok()
    ro, rS = L.kda_decode(**i)
    assert_each_close(o, ro, "o", 1e-5)
    slots = d["slots"].long()
    assert_each_close(d["state"][slots], rS, "state", 1e-5)
    others = torch.ones(len(before), dtype=torch.bool, device="cuda")
    others[slots] = False
    assert torch.equal(d["state"][others], before[others])


def test_kda_tokens_without_norm_bias_and_slots():
    i = kda_inputs(3, 2, 3, 2, 4, 32, 24, F32, F32)
    i["q"], i["k"] = i["q"] * 0.2, i["k"] * 0.2
    d = cuda(i)
    state = d["state"].clone()
    o = gdn.kda_decode(d["q"], d["k"], d["v"], d["a"], d["b"], d["A_log"], None, state, scale=0.7,
                       use_qk_l2norm=False, out_dtype=F32)
    ok()
    i["dt_bias"], i["slots"] = None, None
    ro, rS = L.kda_decode(**i, scale=0.7, l2norm=False)
    assert_each_close(o, ro, "o", 1e-5)
    assert_each_close(state[:2], rS, "state", 1e-5)


def test_kda_tokens_continue_a_prompt():
    """Tokens after kda_chunk_fwd are the same call's on all of them."""
    i = kda_inputs(4, 2, 4, 2, 2, 64, 32, F32, F32)
    g = torch.Generator().manual_seed(2)
    N, T, H, K, V = 2, 100, 2, 64, 32
    q, k = (torch.nn.functional.normalize(torch.randn(N, T, H, K, generator=g), dim=-1) for _ in range(2))
    v, b = torch.randn(N, T, H, V, generator=g), torch.randn(N, T, H, generator=g)
    a = torch.randn(N, T, H, K, generator=g)
    gate = -torch.exp(i["A_log"])[:, None] * torch.nn.functional.softplus(a + i["dt_bias"])
    c = [x.cuda() for x in (q, k, v, gate, torch.sigmoid(b))]
    whole, _ = gdn.kda_chunk_fwd(*c, g_is_cumsum=False)
    _, ht = gdn.kda_chunk_fwd(*(x[:, :96].contiguous() for x in c), g_is_cumsum=False,
                              state_v_first=True)
    o = gdn.kda_decode(*(x[:, 96:].cuda() for x in (q, k, v, a, b)), i["A_log"].cuda(),
                       i["dt_bias"].cuda(), ht, eps=0.0)
    ok()
    assert_each_close(o, _np(whole[:, 96:]), "o", TOL_F32)


@pytest.mark.parametrize("B", [3, 300])
def test_kda_tokens_of_a_bad_slot(B):
    i = kda_inputs(5, B, 2, 2, 4, 64, 64, BF16, BF16)
    i["slots"][1], i["slots"][2] = -1, len(i["state"])
    d = cuda(i)
    before = d["state"].clone()
    o = gdn.kda_decode(d["q"], d["k"], d["v"], d["a"], d["b"], d["A_log"], d["dt_bias"], d["state"],
                       slot_indices=d["slots"])
    assert gdn.gdn_check_device_error() == Status.BAD_SLOT
    assert not o[1:3].any() and o[0].any()
    held = set(i["slots"].tolist())
    for s in range(len(before)):
        if s not in held:
            assert torch.equal(d["state"][s], before[s])


@pytest.mark.parametrize("B", [2, 300])
def test_kda_tokens_of_gates_that_are_no_numbers(B):
    """A NaN reaches its own head's channel and no other; infinities mean keep and forget."""
    i = kda_inputs(7, B, 2, 2, 2, 64, 64, F32, F32)
    bad = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in i.items()}
    i["a"][0, 0, 1, 3], i["a"][1, 1, 0, 5] = -float("inf"), float("inf")
    bad["a"][0, 0, 1, 3], bad["a"][0, 1, 0, 5] = float("nan"), -float("inf")
    for x in (i, bad):
        d = cuda(x)
        o = gdn.kda_decode(d["q"], d["k"], d["v"], d["a"], d["b"], d["A_log"], d["dt_bias"],
                           d["state"], slot_indices=d["slots"])
        if x is i:
            assert_each_close(o, L.kda_decode(**i)[0], "o", 1e-5)
    assert o[0, :, 1].isnan().all() and d["state"][d["slots"][0], 1, :, 3].isnan().all()
    o[0, :, 1] = 0
    assert o.isfinite().all()
    ok()


def test_kda_tokens_replay():
    i = kda_inputs(6, 40, 1, 4, 8, 128, 128, BF16, BF16)
    d = cuda(i)
    start = d["state"].clone()

    def call():
        return gdn.kda_decode(d["q"], d["k"], d["v"], d["a"], d["b"], d["A_log"], d["dt_bias"],
                              d["state"], slot_indices=d["slots"])

    first = call().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(graph):
        o = call()
    for _ in range(2):
        d["state"].copy_(start)
        graph.replay()
        assert torch.equal(o, first)
    ok()


def test_kda_tokens_in_a_pool_past_2_31_elements():
    pool, HV, K, V = 16400, 8, 128, 128
    state = torch.zeros(pool, HV, V, K, dtype=BF16, device="cuda")
    assert state.numel() > 1 << 31
    i = kda_inputs(7, 2, 1, 8, 8, K, V, BF16, BF16)
    d = cuda(i)
    slots = torch.tensor([0, pool - 1], dtype=torch.int32, device="cuda")
    state[slots.long()] = d["state"][:2]
    o = gdn.kda_decode(d["q"], d["k"], d["v"], d["a"], d["b"], d["A_log"], d["dt_bias"], state,
                       slot_indices=slots)
    small = d["state"][:2].clone()
    ref = gdn.kda_decode(d["q"], d["k"], d["v"], d["a"], d["b"], d["A_log"], d["dt_bias"], small)
    ok()
    assert torch.equal(o, ref) and torch.equal(state[slots.long()], small)


def test_kda_token_refusals_in_python():
    d = cuda(kda_inputs(8, 2, 1, 2, 4, 16, 16, BF16, BF16))
    d["dt_bias"] = d["dt_bias"].contiguous()

    def call(**kw):
        x = {**d, **kw}
        return gdn.kda_decode(x["q"], x["k"], x["v"], x["a"], x["b"], x["A_log"], x["dt_bias"],
                              x["state"], slot_indices=x["slots"], scale=x.get("scale"))

    for change in (dict(q=d["q"].float()), dict(k=d["k"][:1]), dict(a=d["a"][..., :8]),
                   dict(state=d["state"].half()), dict(A_log=d["A_log"].double()),
                   dict(slots=d["slots"].long()), dict(scale=0.0), dict(b=d["b"].float())):
        with pytest.raises(ValueError):
            call(**change)


# ---------------------------------------------------------------- the norm

# (B, T, groups, width, dtype, gap): widths of one channel to the most, whole pieces and odd
# ones, within a warp and over several; rows wider than D that begin anywhere; many tokens
NORMS = [
    (1, 1, 1, 1, F32, 0), (2, 3, 3, 5, BF16, 0), (1, 7, 40, 8, BF16, 0), (3, 50, 16, 128, BF16, 0),
    (2, 33, 3, 257, F32, 0), (1, 20, 5, 136, BF16, 2), (1, 9, 2, 1000, BF16, 64), (1, 5, 1, 4096, BF16, 0),
    (1, 4, 2, 5001, F32, 0), (1, 3, 1, 8192, F32, 0), (1, 3, 2, 8192, BF16, 0), (1, 3, 1, 8191, BF16, 0),
    (2, 30, 300, 4, F32, 0), (1, 2, 2, 6, BF16, 3), (1, 6000, 2, 24, F32, 8), (2, 1100, 4, 512, BF16, 0),
    (1, 9, 1500, 3, BF16, 0),
]


@pytest.mark.parametrize("B,T,groups,width,dtype,gap", NORMS)
@pytest.mark.parametrize("z,first,act,center,shared", [
    (True, False, "silu", False, True), (False, False, "silu", True, False),
    (True, True, "silu", False, False), (True, False, "sigmoid", True, False),
    (False, False, None, True, True)])
def test_norm(B, T, groups, width, dtype, gap, z, first, act, center, shared):
    i = norm_inputs(T + width, B, T, groups, width, dtype, shared, z=z, gap=gap)
    d = cuda(i)
    how = dict(eps=1e-5, center=center, activation=act, gate_first=first)
    y = gdn.group_norm_fwd(d["x"], groups, d["weight"], d["bias"], d["z"], **how)
    assert_each_close(y, L.group_norm(i["x"], groups, i["weight"], i["bias"], i["z"], **how), "y", NORM)
    got = gdn.group_norm_bwd(d["dy"], d["x"], groups, d["weight"], d["bias"], d["z"], **how)
    ok()
    dx, dw, db, dz = L.group_norm_grad(i["dy"], i["x"], groups, i["weight"], i["bias"], i["z"], **how)
    if shared:
        dw, db = dw.sum(0), db.sum(0)
    # (a group of one or two channels with its mean off has slopes of up to 1 / root(eps): the
    # terms of dx then cancel to what is left of 300 times their size)
    few = width <= 2 or not center and width == 1
    assert_each_close(got[0], dx, "dx", 1e-2 if few else 3 * NORM)
    assert_each_close(got[1], dw.reshape(-1), "dw", NORM)
    assert_each_close(got[2], db.reshape(-1), "db", NORM)
    if z:
        assert_each_close(got[3], dz, "dz", 1e-2 if few else 3 * NORM)


@pytest.mark.parametrize("width", [32, 64, 96, 128, 192, 256, 384, 512, 1024, 2048])
@pytest.mark.parametrize("groups", [1, 4, 12])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_of_even_groups(width, groups, dtype):
    """Groups that teams and pieces divide, with as many groups as blocks have teams and other
    numbers of them; then batch rows that lie further apart."""
    i = norm_inputs(width + groups, 2, 70, groups, width, dtype, True)
    d = cuda(i)
    apart = {k: torch.zeros(3, 80, *d[k].shape[2:], dtype=dtype, device="cuda") for k in ("x", "z", "dy")}
    for k, t in apart.items():
        t[1:, 5:75] = d[k]
        apart[k] = t[1:, 5:75]
    for z, how in ((True, dict(center=False, activation="silu")),
                   (True, dict(activation="sigmoid", gate_first=True)), (False, dict(activation="silu"))):
        ref = L.group_norm(i["x"], groups, i["weight"], i["bias"], i["z"] if z else None, **how)
        grads = L.group_norm_grad(i["dy"], i["x"], groups, i["weight"], i["bias"],
                                  i["z"] if z else None, **how)
        for t in (d, apart):
            gate = t["z"] if z else None
            y = gdn.group_norm_fwd(t["x"], groups, d["weight"], d["bias"], gate, **how)
            got = gdn.group_norm_bwd(t["dy"], t["x"], groups, d["weight"], d["bias"], gate, **how)
            ok()
            assert_each_close(y, ref, "y", NORM)
            assert_each_close(got[0], grads[0], "dx", 3 * NORM)
            assert_each_close(got[1], grads[1].sum(0), "dw", NORM)
            assert_each_close(got[2], grads[2].sum(0), "db", NORM)
            if z:
                assert_each_close(got[3], grads[3], "dz", 3 * NORM)


def test_norm_without_weights_and_with_float32_ones():
    i = norm_inputs(1, 2, 5, 4, 32, BF16, weight=False, bias=False, z=False)
    d = cuda(i)
    y = gdn.group_norm_fwd(d["x"], 4)
    assert_each_close(y, L.group_norm(i["x"], 4), "y", NORM)
    dx, dw, db, dz = gdn.group_norm_bwd(d["dy"], d["x"], 4)
    assert dw is None and db is None and dz is None
    assert_each_close(dx, L.group_norm_grad(i["dy"], i["x"], 4)[0], "dx", NORM)
    i = norm_inputs(2, 2, 5, 4, 32, BF16, weight_dtype=F32)
    d = cuda(i)
    how = dict(center=False, activation="silu")
    y = gdn.group_norm_fwd(d["x"], 4, d["weight"], d["bias"], d["z"], **how)
    assert_each_close(y, L.group_norm(i["x"], 4, i["weight"], i["bias"], i["z"], **how), "y", NORM)
    got = gdn.group_norm_bwd(d["dy"], d["x"], 4, d["weight"], d["bias"], d["z"], output_dweight=False, **how)
    assert got[1] is None and got[2] is None
    ref = L.group_norm_grad(i["dy"], i["x"], 4, i["weight"], i["bias"], i["z"], **how)
    assert_each_close(got[0], ref[0], "dx", 3 * NORM)
    ok()


def test_norm_of_no_tokens():
    x = torch.zeros(2, 0, 24, dtype=BF16, device="cuda")
    w = torch.ones(24, dtype=BF16, device="cuda")
    assert gdn.group_norm_fwd(x, 3, w).shape == x.shape
    dx, dw, db, dz = gdn.group_norm_bwd(x, x, 3, w, w)
    assert dx.shape == x.shape and not dw.any() and not db.any()
    ok()


def test_norm_keeps_what_is_not_finite_in_its_group():
    i = norm_inputs(5, 1, 40, 8, 64, BF16)
    d = cuda(i)
    y = gdn.group_norm_fwd(d["x"], 8, d["weight"], d["bias"], d["z"], activation="silu")
    x = d["x"].clone()
    x[0, 7, 70], x[0, 9, 5] = float("nan"), float("inf")
    dx = gdn.group_norm_bwd(d["dy"], d["x"], 8, d["weight"], d["bias"], d["z"], activation="silu")[0]
    y2 = gdn.group_norm_fwd(x, 8, d["weight"], d["bias"], d["z"], activation="silu")
    dx2 = gdn.group_norm_bwd(d["dy"], x, 8, d["weight"], d["bias"], d["z"], activation="silu")[0]
    same = torch.ones(1, 40, 512, dtype=torch.bool, device="cuda")
    same[0, 7, 64:128] = same[0, 9, :64] = False
    assert torch.equal(y[same], y2[same]) and torch.equal(dx[same], dx2[same])
    assert not y2[0, 7, 64:128].isfinite().any()
    ok()


def test_norm_of_large_and_of_equal_values():
    """A mean of 2^12 root variances, and groups without any variance."""
    x = torch.randn(1, 30, 256, generator=torch.Generator().manual_seed(1)) + 4096
    x[0, 3] = 7.0
    y = gdn.group_norm_fwd(x.cuda(), 2)
    # x itself is rounded to 2^-12 of its spread; the kernel adds the mean's rounding, 2^-12
    assert_each_close(y, L.group_norm(x, 2), "y", 2.0 ** -10)
    assert not y[0, 3].any()


def test_norm_repeats_replays_and_takes_streams():
    d = cuda(norm_inputs(6, 2, 3000, 8, 96, BF16))

    def call(**kw):
        y = gdn.group_norm_fwd(d["x"], 8, d["weight"], d["bias"], d["z"], activation="silu", **kw)
        return [y, *gdn.group_norm_bwd(d["dy"], d["x"], 8, d["weight"], d["bias"], d["z"],
                                       activation="silu", **kw)]

    first = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    there = call(stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    graph.replay()
    for a, b, c in zip(first, there, held):
        assert torch.equal(a, b) and torch.equal(a, c)
    ok()


def test_norm_past_2_31_elements():
    T, D = 262200, 8192
    x = torch.empty(1, T, D, dtype=BF16, device="cuda").normal_()
    assert x.numel() > 1 << 31
    w = torch.rand(64, device="cuda") + 0.5
    y = gdn.group_norm_fwd(x, 128, w, center=False)
    assert torch.equal(y[:, -70:], gdn.group_norm_fwd(x[:, -70:], 128, w, center=False))
    dx = gdn.group_norm_bwd(y, x, 128, w, center=False)[0]
    assert torch.equal(dx[:, -70:], gdn.group_norm_bwd(y[:, -70:], x[:, -70:], 128, w, center=False)[0])
    ok()


def test_norm_refusals_in_python():
    d = cuda(norm_inputs(7, 1, 4, 4, 8, BF16))
    x = d["x"]
    for args, kw in (((x, 5), {}), ((x, 4, d["weight"][:5]), {}), ((x, 4, d["weight"].double()), {}),
                     ((x, 4, d["weight"], d["bias"].float()), {}), ((x, 4), dict(activation="relu")),
                     ((x, 4), dict(z=x.float())), ((x.half(), 4), {}), ((x.transpose(1, 2), 4), {})):
        with pytest.raises(ValueError):
            gdn.group_norm_fwd(*args, **kw)
    with pytest.raises(GdnError):
        gdn.group_norm_fwd(x, 4, gate_first=True)


# ---------------------------------------------------------------- together

def test_a_layer_trains_and_decodes():
    """Convolution, delta rule and gated norm with their gradients chained, against the same
    layer's gradient in fp64; then the KDA layer's token behind its prompt."""
    B, T, H, K, V = 2, 90, 2, 32, 32
    g = torch.Generator().manual_seed(3)
    D = H * (2 * K + V)
    x = torch.randn(B, T, D, generator=g)
    cw, nw = torch.randn(D, 4, generator=g) * 0.5, torch.rand(V, generator=g) + 0.5
    z, dy = torch.randn(B, T, H * V, generator=g), torch.randn(B, T, H * V, generator=g)
    gate, beta = torch.nn.functional.logsigmoid(torch.randn(B, T, H, generator=g) + 3), \
        torch.sigmoid(torch.randn(B, T, H, generator=g))
    c = dict(x=x.cuda(), cw=cw.cuda(), nw=nw.cuda(), z=z.cuda(), dy=dy.cuda(), gate=gate.cuda(),
             beta=beta.cuda())
    u, _ = gdn.short_conv_fwd(c["x"], c["cw"])
    q, k, v = (t.contiguous() for t in u.split([H * K, H * K, H * V], 2))
    q, k, v = (q * 0.1).view(B, T, H, K), (k * 0.1).view(B, T, H, K), v.view(B, T, H, V)
    o, _ = gdn.gdn_chunk_fwd(q, k, v, c["gate"], c["beta"])
    how = dict(center=False, activation="silu")
    do, dnw, _, dz = gdn.group_norm_bwd(c["dy"], o.view(B, T, -1), H, c["nw"], z=c["z"], **how)
    dq, dk, dv, dg, db, _ = gdn.gdn_chunk_bwd(do.view(B, T, H, V), q, k, v, c["gate"], c["beta"])
    du = torch.cat([dq.flatten(2) * 0.1, dk.flatten(2) * 0.1, dv.flatten(2)], 2)
    dx, dcw, _, _ = gdn.short_conv_bwd(du, c["x"], c["cw"])
    ok()

    p = {n: t.double().requires_grad_() for n, t in dict(x=x, cw=cw, nw=nw, z=z, gate=gate, beta=beta).items()}
    r = torch.nn.functional.silu(torch.nn.functional.conv1d(
        torch.nn.functional.pad(p["x"].transpose(1, 2), (3, 0)), p["cw"][:, None], groups=D)).transpose(1, 2)
    rq, rk, rv = r.split([H * K, H * K, H * V], 2)
    rq, rk, rv = (rq * 0.1).view(B, T, H, K), (rk * 0.1).view(B, T, H, K), rv.view(B, T, H, V)
    h, ro = torch.zeros(B, H, K, V, dtype=torch.float64), []
    for t in range(T):
        h = torch.exp(p["gate"][:, t])[..., None, None] * h
        d = p["beta"][:, t, :, None] * (rv[:, t] - torch.einsum("bhk,bhkv->bhv", rk[:, t], h))
        h = h + rk[:, t, :, :, None] * d[:, :, None]
        ro.append(K ** -0.5 * torch.einsum("bhk,bhkv->bhv", rq[:, t], h))
    ro = torch.stack(ro, 1)
    n = ro * (ro.square().mean(-1, keepdim=True) + 1e-5) ** -0.5 * p["nw"]
    y = n.flatten(2) * torch.nn.functional.silu(p["z"])
    ref = torch.autograd.grad(y, list(p.values()), dy.double())
    # (the norm divides by outputs of 0.1 and less: its slopes multiply what came before by
    # up to 30, so 30 times the float32 bound of the recurrence's 1e-5 typical error)
    for name, got, want in zip(p, (dx, dcw, dnw, dz, dg, db), ref):
        assert_each_close(got, want.numpy(), name, 3e-4)


# ---------------------------------------------------------------- calls at once, the checked build

def everything(seed, K, heads):
    """One call of each operator as a function of the stream; the states are new every time."""
    i = cuda(delta_inputs(seed, 1, 300, heads, 1, K, K, BF16, [170, 130]))
    t = cuda(kda_inputs(seed, 40, 2, heads, 2 * heads, K, 64, BF16, BF16))
    n = cuda(norm_inputs(seed, 1, 400, heads, K, BF16))
    start = t["state"].clone()

    def run(stream=None):
        state = t["state"] if stream is None else torch.empty_like(start)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            state.copy_(start)
        o = gdn.kda_decode(t["q"], t["k"], t["v"], t["a"], t["b"], t["A_log"], t["dt_bias"], state,
                           slot_indices=t["slots"], stream=stream)
        y = gdn.group_norm_fwd(n["x"], heads, n["weight"], n["bias"], n["z"], activation="silu",
                               stream=stream)
        g = gdn.group_norm_bwd(n["dy"], n["x"], heads, n["weight"], n["bias"], n["z"],
                               activation="silu", stream=stream)
        return [o, state, y, *g, *run_delta(i, stream=stream)]

    return run


def test_calls_from_several_threads():
    """Each on a stream of its own, of other sizes, all at once."""
    calls = [everything(30 + k, (128, 64, 40)[k % 3], 2 + k) for k in range(6)]
    begin, results = threading.Barrier(6), [None] * 6
    torch.cuda.synchronize()

    def work(k):
        stream = torch.cuda.Stream()
        begin.wait()
        for _ in range(5):
            out = calls[k](stream)
        stream.synchronize()
        results[k] = out

    threads = [threading.Thread(target=work, args=(k,)) for k in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    ok()
    for out, call in zip(results, calls):
        for a, b in zip(out, call()):
            assert torch.equal(a, b)


def test_graphs_that_share_a_workspace():
    ins = [cuda(delta_inputs(40 + k, 1, 260, 4, 2, 128, 64, BF16, [100, 160])) for k in range(2)]
    n = cuda(norm_inputs(41, 1, 500, 8, 64, BF16))
    want = [run_delta(i) for i in ins]
    norm = gdn.group_norm_bwd(n["dy"], n["x"], 8, n["weight"], n["bias"])
    room = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    graphs, held = [], []
    for i in ins:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append((run_delta(i, workspace=room),
                         gdn.group_norm_bwd(n["dy"], n["x"], 8, n["weight"], n["bias"], workspace=room)))
    for k in (0, 1, 1, 0):
        room.fill_(255)
        for x in (*held[k][0], *held[k][1][:3]):
            x.fill_(7)
        graphs[k].replay()
        for a, b in zip((*held[k][0], *held[k][1][:3]), (*want[k], *norm[:3])):
            assert torch.equal(a, b)
    ok()


@pytest.mark.parametrize("dtype,K", [(BF16, 128), (BF16, 40), (F32, 40), (F32, 128)])
def test_a_workspace_may_hold_anything(dtype, K):
    i = cuda(delta_inputs(45, 1, 330, 4, 2, K, 72, dtype, [100, 1, 0, 229]))
    want = run_delta(i)
    for byte in (0, 255):  # (all bits set: every float a NaN)
        room = torch.full((64 << 20,), byte, dtype=torch.uint8, device="cuda")
        for a, b in zip(want, run_delta(i, workspace=room)):
            assert torch.equal(a, b)
    ok()


CHECKED = r"""
import sys
sys.path[:0] = [sys.argv[1], sys.argv[2]]
import torch
from gated_delta_rule_kk_gb300 import _lib
import gated_delta_rule_kk_gb300 as gdn
from _layer import delta_inputs, kda_inputs, norm_inputs
from _mixer import cuda

checked, release = _lib.load(), _lib.load(sys.argv[3])
BF16, F32 = torch.bfloat16, torch.float32


def delta(T, H, Hg, K, V, dtype, lens=None):
    d = cuda(delta_inputs(1, 1, T, H, Hg, K, V, dtype, lens))
    return gdn.gdn_chunk_bwd(d["do"], d["q"], d["k"], d["v"], d["g"], d["beta"], scale=d["scale"],
                             initial_state=d["h0"], dfinal_state=d["dht"], cu_seqlens=d["cu"])


def tokens(B, T, K, V, state):
    d = cuda(kda_inputs(2, B, T, 4, 8, K, V, BF16, state))
    o = gdn.kda_decode(d["q"], d["k"], d["v"], d["a"], d["b"], d["A_log"], d["dt_bias"], d["state"],
                       slot_indices=d["slots"])
    return o, d["state"]


def norm(T, groups, width, dtype):
    d = cuda(norm_inputs(3, 1, T, groups, width, dtype))
    how = dict(activation="silu")
    y = gdn.group_norm_fwd(d["x"], groups, d["weight"], d["bias"], d["z"], **how)
    return y, *gdn.group_norm_bwd(d["dy"], d["x"], groups, d["weight"], d["bias"], d["z"], **how)


cases = []
for dt in (BF16, F32):
    cases += [lambda dt=dt: delta(1, 2, 2, 128, 128, dt), lambda dt=dt: delta(200, 4, 2, 64, 40, dt),
              lambda dt=dt: delta(300, 2, 1, 120, 128, dt, [129, 0, 1, 170]),
              lambda dt=dt: delta(70, 2, 1, 20, 136, dt), lambda dt=dt: tokens(1, 1, 128, 33, dt),
              lambda dt=dt: tokens(100, 3, 256, 128, dt), lambda dt=dt: norm(37, 5, 24, dt),
              lambda dt=dt: norm(3000, 3, 8191, dt), lambda dt=dt: norm(1, 300, 1, dt)]
for i, case in enumerate(cases):
    results = []
    for lib in (checked, release):
        _lib._lib = lib
        results.append(case())
        status = gdn.gdn_check_device_error()
        assert status == 0, (i, status)
    for a, b in zip(*results):
        assert torch.equal(a, b), i
"""


def test_checked_build():
    """The bounds-checked build records nothing on valid calls and computes the same."""
    tests = os.path.dirname(os.path.abspath(__file__))
    build_lib.build(checked=True)
    r = subprocess.run([sys.executable, "-c", CHECKED, os.path.dirname(tests), tests,
                        build_lib.build()], env=dict(os.environ, GDN_CHECKED="1"),
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout + r.stderr
