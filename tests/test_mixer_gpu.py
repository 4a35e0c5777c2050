"""The short convolution and the state space scan on the GPU against their
definitions in fp64.

Bounds.  Convolution: at most 8 products summed in float32 and one SiLU, a few
2^-23 of the sum of magnitudes (below 10 RMS): 1e-5 RMS, plus a bfloat16
output's own rounding.  Its weight gradients sum up to 2000 products, in
float32 partial sums: 1e-5 RMS as well.  Scan: the library's bounds, 1e-4 RMS
in float32 and for float32 states, 2e-2 RMS for bfloat16 inputs.
"""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

import gated_delta_rule_kk_gb300 as gdn
from gated_delta_rule_kk_gb300 import GdnError, Status, build_lib
from oracle import mixer as M

from _mixer import assert_each_close, conv_inputs, cuda, ssm_inputs
from _util import TOL_BF16, TOL_F32, assert_close

pytestmark = pytest.mark.gpu

CONV_TOL = 1e-5
F32, BF16 = torch.float32, torch.bfloat16


def ok():
    assert gdn.gdn_check_device_error() == Status.OK


# (B, T, D, W, dtype, lens, gap): one token; odd channels; runs that end inside
# a batch of rows; packed with empty and one-token sequences; rows wider than D
CONV_CASES = [
    (1, 1, 8, 4, BF16, None, 0),
    (2, 3, 40, 4, BF16, None, 0),
    (1, 2, 5, 3, BF16, None, 0),
    (3, 37, 771, 3, F32, None, 0),
    (2, 129, 264, 2, F32, None, 64),
    (1, 300, 72, 4, BF16, [0, 1, 2, 0, 3, 150, 144, 0], 0),
    (1, 70, 33, 2, BF16, [1, 1, 68], 0),
    (1, 515, 1032, 4, BF16, [512, 3], 80),
    (1, 97, 12, 4, F32, [5, 0, 92], 16),
    (1, 2050, 16, 4, BF16, None, 0),
]


@pytest.mark.parametrize("B,T,D,W,dtype,lens,gap", CONV_CASES)
@pytest.mark.parametrize("silu,bias,state", [(True, True, True), (False, False, False)])
def test_conv(B, T, D, W, dtype, lens, gap, silu, bias, state):
    i = conv_inputs(T + D, B, T, D, W, dtype, bias, lens, state, gap)
    d = cuda(i)
    act = "silu" if silu else None
    y, ht = gdn.short_conv_fwd(d["x"], d["weight"], bias=d["bias"], initial_state=d["h0"],
                               cu_seqlens=d["cu"], activation=act)
    ok()
    ry, rht = M.short_conv(i["x"], i["weight"], i["bias"], i["h0"], i["cu"], silu)
    assert_each_close(y, ry, "y", CONV_TOL)
    assert_each_close(ht, rht, "ht", CONV_TOL)
    if not state:
        d["dht"] = i["dht"] = None
    dx, dw, db, dh0 = gdn.short_conv_bwd(d["dy"], d["x"], d["weight"], bias=d["bias"],
                                         initial_state=d["h0"], dfinal_state=d["dht"],
                                         cu_seqlens=d["cu"], activation=act)
    ok()
    rx, rw, rb, rh = M.short_conv_grad(i["dy"], i["x"], i["weight"], i["bias"], i["h0"], i["dht"],
                                       i["cu"], silu)
    assert_each_close(dx, rx, "dx", CONV_TOL)
    assert_each_close(dw, rw, "dw", CONV_TOL)
    if bias:
        assert_each_close(db, rb, "db", CONV_TOL)
    if state:
        assert_each_close(dh0, rh, "dh0", CONV_TOL)


# long enough for the ring of tiles: runs that end inside a sequence and at its
# end, sequences shorter than the taps, channels that end inside a box
@pytest.mark.parametrize("B,T,D,W,dtype,lens,gap,silu", [
    (1, 3001, 4100, 4, BF16, [1000, 0, 1, 2, 3, 1995], 36, True),
    (2, 1601, 4104, 3, BF16, None, 0, False),
    (1, 5003, 1156, 4, F32, [7, 4000, 2, 994], 0, True),
    (1, 14000, 520, 2, BF16, None, 8, True),
    # the last token(s) on a run of their own, or just before a run's end
    (1, 3000, 1160, 4, F32, [500, 2500], 0, True),
    (1, 3001, 1160, 4, F32, [500, 2501], 0, True),
    (1, 3002, 1160, 4, F32, [500, 2502], 0, True),
    (1, 3003, 1160, 3, F32, [500, 2503], 0, True),
    (1, 3001, 1160, 2, F32, [2999, 2], 0, False),
])
def test_conv_of_long_prompts(B, T, D, W, dtype, lens, gap, silu):
    i = conv_inputs(T, B, T, D, W, dtype, True, lens, True, gap)
    d = cuda(i)
    act = "silu" if silu else None
    y, ht = gdn.short_conv_fwd(d["x"], d["weight"], bias=d["bias"], initial_state=d["h0"],
                               cu_seqlens=d["cu"], activation=act)
    ok()
    ry, rht = M.short_conv(i["x"], i["weight"], i["bias"], i["h0"], i["cu"], silu)
    assert_each_close(y, ry, "y", CONV_TOL)
    assert_each_close(ht, rht, "ht", CONV_TOL)
    out = gdn.short_conv_bwd(d["dy"], d["x"], d["weight"], bias=d["bias"], initial_state=d["h0"],
                             dfinal_state=d["dht"], cu_seqlens=d["cu"], activation=act)
    ok()
    ref = M.short_conv_grad(i["dy"], i["x"], i["weight"], i["bias"], i["h0"], i["dht"], i["cu"], silu)
    for got, want, name in zip(out, ref, ("dx", "dw", "db", "dh0")):
        assert_each_close(got, want, name, CONV_TOL)
    again = gdn.short_conv_bwd(d["dy"], d["x"], d["weight"], bias=d["bias"],
                               initial_state=d["h0"], dfinal_state=d["dht"], cu_seqlens=d["cu"],
                               activation=act)
    assert all(torch.equal(a, b) for a, b in zip(out, again))


def test_conv_float32_weights_beside_bfloat16_rows():
    i = conv_inputs(5, 2, 50, 24, 4, BF16)
    i["weight"], i["bias"] = i["weight"].float() * 1.001, i["bias"].float() * 1.001
    d = cuda(i)
    y, _ = gdn.short_conv_fwd(d["x"], d["weight"], bias=d["bias"], initial_state=d["h0"])
    ry, _ = M.short_conv(i["x"], i["weight"], i["bias"], i["h0"])
    assert_each_close(y, ry, "y", CONV_TOL)


def test_conv_without_tokens():
    d = cuda(conv_inputs(6, 2, 0, 16, 4, BF16))
    _, ht = gdn.short_conv_fwd(d["x"], d["weight"], initial_state=d["h0"])
    assert torch.equal(ht, d["h0"])
    _, dw, _, dh0 = gdn.short_conv_bwd(d["dy"], d["x"], d["weight"], initial_state=d["h0"],
                                       dfinal_state=d["dht"])
    assert torch.equal(dh0, d["dht"]) and not dw.any()
    ok()


def test_conv_into_a_wider_buffer():
    """Outputs strided as the inputs may be; the columns beside them stay."""
    i = conv_inputs(7, 2, 40, 32, 4, BF16)
    d = cuda(i)
    wide = torch.full((2, 40, 64), 7.0, dtype=BF16, device="cuda")
    gdn.short_conv_fwd(d["x"], d["weight"], initial_state=d["h0"], out=wide[:, :, 16:48])
    ry, _ = M.short_conv(i["x"], i["weight"], None, i["h0"])
    assert_each_close(wide[:, :, 16:48], ry, "y", CONV_TOL)
    assert (wide[:, :, :16] == 7).all() and (wide[:, :, 48:] == 7).all()


def test_conv_gradient_is_the_same_every_time():
    d = cuda(conv_inputs(8, 1, 3000, 136, 4, BF16, lens=[1000, 0, 2000]))
    one, two = (gdn.short_conv_bwd(d["dy"], d["x"], d["weight"], bias=d["bias"],
                                   initial_state=d["h0"], cu_seqlens=d["cu"]) for _ in range(2))
    assert all(torch.equal(a, b) for a, b in zip(one, two))


@pytest.mark.parametrize("T", [1, 2, 3, 4])
@pytest.mark.parametrize("D,W,dtype", [(64, 4, BF16), (33, 3, BF16), (20, 2, F32), (1032, 4, F32)])
def test_conv_tokens(T, D, W, dtype):
    i = conv_inputs(T, 3, T, D, W, dtype)
    d = cuda(i)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32)
    pool = torch.randn(5, W - 1, D).to(dtype)
    pool[slots.long()] = i["h0"]
    state = pool.cuda()
    y = gdn.short_conv_decode(d["x"], d["weight"], state, bias=d["bias"], slot_indices=slots.cuda())
    ok()
    ry, rht = M.short_conv(i["x"], i["weight"], i["bias"], i["h0"])
    assert_each_close(y, ry, "y", CONV_TOL)
    assert_each_close(state[slots.long().cuda()], rht, "state", CONV_TOL)
    others = torch.tensor([1, 3])
    assert torch.equal(state[others.cuda()].cpu(), pool[others])


def test_bad_slots_write_zeros_and_are_recorded():
    d = cuda(conv_inputs(9, 2, 1, 16, 4, BF16))
    state = d["h0"].clone()
    slots = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    y = gdn.short_conv_decode(d["x"], d["weight"], state, slot_indices=slots)
    assert gdn.gdn_check_device_error() == Status.BAD_SLOT
    assert not y[1].any() and y[0].any() and torch.equal(state[0], d["h0"][0])
    s = cuda(ssm_inputs(9, 2, 1, 4, 2, 16, 16, BF16))
    state = s["h0"].clone()
    slots = torch.tensor([-1, 0], dtype=torch.int32, device="cuda")
    y = gdn.ssm_decode(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], state, slot_indices=slots)
    assert gdn.gdn_check_device_error() == Status.BAD_SLOT
    assert not y[0].any() and y[1].any() and torch.equal(state[1], s["h0"][1])


@pytest.mark.parametrize("cu", [[0, 5, 3, 10], [1, 5, 8, 10], [0, 5, 8, 11]])
def test_bad_offsets_write_nothing_and_are_recorded(cu):
    d = cuda(conv_inputs(10, 1, 10, 16, 4, BF16, lens=[3, 3, 4]))
    d["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    y = torch.full_like(d["dy"], 7.0)
    gdn.short_conv_fwd(d["x"], d["weight"], initial_state=d["h0"], cu_seqlens=d["cu"], out=y)
    assert gdn.gdn_check_device_error() == Status.BAD_SEQLENS and (y == 7).all()
    s = cuda(ssm_inputs(10, 1, 10, 2, 1, 16, 16, BF16, lens=[3, 3, 4]))
    y = torch.full((1, 10, 2, 16), 7.0, dtype=BF16, device="cuda")
    gdn.ssm_chunk_fwd(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], cu_seqlens=d["cu"], out=y)
    assert gdn.gdn_check_device_error() == Status.BAD_SEQLENS and (y == 7).all()


# ---------------------------------------------------------------- scan

def run_scan(i, **kw):
    d = cuda(i)
    y, ht = gdn.ssm_chunk_fwd(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], D=d["D"], z=d["z"],
                              dt_bias=d["dt_bias"], initial_state=d["h0"], cu_seqlens=d["cu"],
                              out_dtype=F32, **kw)
    ok()
    if i["x"].dtype == BF16:
        y16, _ = gdn.ssm_chunk_fwd(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], D=d["D"],
                                   z=d["z"], dt_bias=d["dt_bias"], initial_state=d["h0"],
                                   cu_seqlens=d["cu"], **kw)
        assert torch.equal(y16, y.to(BF16)), "bf16 y is not the RNE of the fp32 y"
    return y, ht


def check_scan(i, **kw):
    y, ht = run_scan(i, **kw)
    ry, rht = M.ssm_scan(i["x"], i["dt"], i["A_log"], i["Bm"], i["Cm"], i["D"], i["z"],
                         i["dt_bias"], h0=i["h0"], cu_seqlens=i["cu"])
    assert_close(y, ry, TOL_F32 if i["x"].dtype == F32 else TOL_BF16, "y")
    assert_close(ht, rht, TOL_F32, "ht")


# (B, T, H, Hg, V, K, lens): one token; odd sizes; chunk edges; packed with
# empty and one-token sequences; every head its own group; wide heads and states
SCAN_CASES = [
    (1, 1, 2, 1, 64, 128, None),
    (2, 63, 4, 2, 64, 128, None),
    (1, 128, 2, 2, 64, 64, None),
    (1, 129, 3, 1, 64, 128, None),
    (2, 257, 2, 1, 128, 128, None),
    (1, 300, 4, 2, 64, 128, [0, 1, 130, 0, 41, 128, 0]),
    (1, 200, 3, 3, 40, 48, [77, 123]),
    (1, 150, 2, 1, 33, 20, None),
    (1, 140, 2, 1, 16, 200, None),
    (1, 600, 2, 1, 64, 64, [256, 344]),
    (1, 90, 2, 1, 72, 1, None),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,H,Hg,V,K,lens", SCAN_CASES)
def test_scan(B, T, H, Hg, V, K, lens, dtype):
    check_scan(ssm_inputs(T + K, B, T, H, Hg, V, K, dtype, lens))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_bare(dtype):
    """No skip, gate or initial state."""
    check_scan(ssm_inputs(3, 2, 200, 2, 1, 64, 128, dtype, h0=False, z=False, skip=False))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_with_strong_decays(dtype):
    """Decays of up to e^-100 a token: sums of log-decays in the thousands."""
    check_scan(ssm_inputs(4, 1, 300, 4, 1, 64, 128, dtype, fast=True))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens", [None, [700, 0, 1, 128, 171]])
def test_scan_in_segments(dtype, lens):
    i = ssm_inputs(5, 1, 1000, 2, 1, 64, 128, dtype, lens)
    check_scan(i, segment_tokens=128)
    check_scan(i, segment_tokens=384)
    check_scan(i, segment_tokens=1024)


def test_scan_step_sizes_as_given_and_in_float32():
    i = ssm_inputs(6, 1, 100, 2, 1, 64, 64, BF16)
    i["dt"] = i["dt"].float().abs() * 0.1
    d = cuda(i)
    y, ht = gdn.ssm_chunk_fwd(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], dt_softplus=False,
                              out_dtype=F32)
    ry, rht = M.ssm_scan(i["x"], i["dt"], i["A_log"], i["Bm"], i["Cm"], dt_softplus=False)
    assert_close(y, ry, TOL_BF16, "y")
    assert_close(ht, rht, TOL_F32, "ht")


def test_scan_without_tokens():
    d = cuda(ssm_inputs(7, 2, 0, 2, 1, 64, 128, BF16))
    y, ht = gdn.ssm_chunk_fwd(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], initial_state=d["h0"])
    ok()
    assert torch.equal(ht, d["h0"]) and y.numel() == 0


def test_scan_keeps_sequences_apart():
    """NaN in one sequence reaches no other."""
    i = ssm_inputs(8, 1, 300, 2, 1, 64, 128, BF16, lens=[100, 50, 150])
    d = cuda(i)
    call = dict(dt_bias=d["dt_bias"], initial_state=d["h0"], cu_seqlens=d["cu"])
    y, ht = gdn.ssm_chunk_fwd(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], **call)
    for name in ("x", "Bm", "Cm", "dt"):
        bad = {k: v.clone() if k == name else v for k, v in d.items()}
        bad[name][:, 100:150] = float("nan")
        y2, ht2 = gdn.ssm_chunk_fwd(bad["x"], bad["dt"], d["A_log"], bad["Bm"], bad["Cm"], **call)
        assert torch.equal(y2[:, :100], y[:, :100]) and torch.equal(y2[:, 150:], y[:, 150:]), name
        assert torch.equal(ht2[0], ht[0]) and torch.equal(ht2[2], ht[2]), name
        assert y2[:, 100:150].isnan().any()


@pytest.mark.parametrize("T", [1, 2, 3, 4])
@pytest.mark.parametrize("dtype,sdtype,H,Hg,V,K", [
    (BF16, BF16, 4, 2, 64, 128), (BF16, F32, 4, 1, 64, 128), (F32, F32, 2, 1, 33, 40),
    (F32, BF16, 2, 2, 100, 64), (BF16, F32, 2, 1, 16, 256), (BF16, BF16, 2, 1, 20, 8)])
def test_scan_tokens(T, dtype, sdtype, H, Hg, V, K):
    i = ssm_inputs(T + K, 3, T, H, Hg, V, K, dtype)
    slots = torch.tensor([3, 0, 4], dtype=torch.int32)
    pool = torch.randn(5, H, V, K).to(sdtype)
    i["h0"] = pool[slots.long()]
    d = cuda(i)
    state = pool.cuda()
    y = gdn.ssm_decode(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], state, D=d["D"], z=d["z"],
                       dt_bias=d["dt_bias"], slot_indices=slots.cuda(), out_dtype=F32)
    ok()
    ry, rht = M.ssm_scan(i["x"], i["dt"], i["A_log"], i["Bm"], i["Cm"], i["D"], i["z"],
                         i["dt_bias"], h0=i["h0"])
    # float32 arithmetic throughout: the state's type only rounds what is stored
    assert_close(y, ry, TOL_F32, "y")
    assert_each_close(state[slots.long().cuda()], rht, "state", 1e-5)
    others = torch.tensor([1, 2])
    assert torch.equal(state[others.cuda()].cpu(), pool[others])


@pytest.mark.parametrize("T,dtype,sdtype,B,H,V,K", [
    (1, BF16, BF16, 70, 32, 64, 128), (3, BF16, F32, 70, 16, 100, 64), (2, F32, F32, 40, 13, 80, 136),
    (4, BF16, BF16, 100, 31, 33, 248)])
def test_scan_tokens_of_many_requests(T, dtype, sdtype, B, H, V, K):
    """Enough states to stream through the ring: checked on some requests, two
    of them with bad slots."""
    i = ssm_inputs(T + K, B, T, H, 1, V, K, dtype, h0=False)
    slots = torch.randperm(B + 20)[:B].to(torch.int32)
    slots[3], slots[B - 1] = -1, B + 20
    d = cuda(i)
    state = torch.randn(B + 20, H, V, K, device="cuda").to(sdtype)
    before = state.clone()
    y = gdn.ssm_decode(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], state, D=d["D"], z=d["z"],
                       dt_bias=d["dt_bias"], slot_indices=slots.cuda(), out_dtype=F32)
    assert gdn.gdn_check_device_error() == Status.BAD_SLOT
    assert not y[3].any() and not y[B - 1].any()
    some = [0, 1, 2, 4, B // 2, B - 3, B - 2]
    at = slots[some].long()
    sub = {k: v[some] if k in ("x", "dt", "Bm", "Cm", "z") else v for k, v in i.items()}
    ry, rht = M.ssm_scan(sub["x"], sub["dt"], sub["A_log"], sub["Bm"], sub["Cm"], sub["D"], sub["z"],
                         sub["dt_bias"], h0=before[at.cuda()])
    assert_close(y[some], ry, TOL_F32, "y")
    assert_each_close(state[at.cuda()], rht, "state", 1e-5)
    rest = torch.ones(B + 20, dtype=torch.bool)
    rest[slots[(slots >= 0) & (slots < B + 20)].long()] = False
    assert torch.equal(state[rest.cuda()], before[rest.cuda()])


def test_tokens_continue_prompts():
    """Convolution and scan over a prompt, then token by token, as the whole
    prompt at once: the layer of examples/ssm_block.py."""
    H, V, K, T = 4, 64, 128, 150
    i = ssm_inputs(11, 2, T, H, 1, V, K, BF16, h0=False)
    w = conv_inputs(12, 2, T, H * V + 2 * K, 4, BF16)
    d, c = cuda(i), cuda(w)

    def split(v):
        x, Bm, Cm = v.split([H * V, K, K], 2)
        return x.unflatten(2, (H, V)), Bm.unflatten(2, (1, K)), Cm.unflatten(2, (1, K))

    kw = dict(D=d["D"], dt_bias=d["dt_bias"], out_dtype=F32)
    v, _ = gdn.short_conv_fwd(c["x"], c["weight"], bias=c["bias"])
    x, Bm, Cm = split(v)
    whole, _ = gdn.ssm_chunk_fwd(x, d["dt"], d["A_log"], Bm, Cm, z=d["z"], **kw)
    n = 143
    v, rows = gdn.short_conv_fwd(c["x"][:, :n], c["weight"], bias=c["bias"])
    x, Bm, Cm = split(v)
    y, h = gdn.ssm_chunk_fwd(x, d["dt"][:, :n], d["A_log"], Bm, Cm, z=d["z"][:, :n], **kw)
    got = [y]
    for lo, hi in ((n, n + 1), (n + 1, n + 3), (n + 3, n + 7)):
        v = gdn.short_conv_decode(c["x"][:, lo:hi], c["weight"], rows, bias=c["bias"])
        x, Bm, Cm = split(v)
        got.append(gdn.ssm_decode(x, d["dt"][:, lo:hi], d["A_log"], Bm, Cm, h,
                                  z=d["z"][:, lo:hi], **kw))
    ok()
    assert_close(torch.cat(got, 1), whole.cpu().double().numpy(), TOL_BF16, "y")


def test_offsets_past_32_bits():
    """The last rows of buffers of more than 2^31 elements."""
    T, D = 263000, 8192
    x = torch.zeros((1, T, D), dtype=BF16, device="cuda")
    i = conv_inputs(21, 1, 300, D, 4, BF16, state=False)
    c = cuda(i)
    x[:, -300:] = c["x"]
    y, ht = gdn.short_conv_fwd(x, c["weight"], c["bias"])
    y_ref, _ = M.short_conv(i["x"], i["weight"], i["bias"])
    assert_each_close(y[:, -300:], y_ref, "y", CONV_TOL)
    assert torch.equal(ht, c["x"][:, -3:])
    dx = gdn.short_conv_bwd(x, x, c["weight"], c["bias"])[0]
    dx_ref = M.short_conv_grad(i["x"], i["x"], i["weight"], i["bias"])[0]
    assert_each_close(dx[:, -300:], dx_ref, "dx", CONV_TOL)
    ok()
    del x, y, dx

    H, V, K, slots = 64, 64, 128, 4200
    d = cuda(ssm_inputs(22, 2, 1, H, 1, V, K, BF16))
    pool = torch.zeros((slots, H, V, K), dtype=BF16, device="cuda")
    at = torch.tensor([slots - 1, 3], dtype=torch.int32, device="cuda")
    pool[at.long()] = d["h0"].to(BF16)
    state = d["h0"].to(BF16)
    args = (d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"])
    y = gdn.ssm_decode(*args, pool, slot_indices=at)
    want = gdn.ssm_decode(*args, state)
    assert torch.equal(y, want) and torch.equal(pool[at.long()], state)
    ok()


@pytest.mark.parametrize("dtype,H,V,T", [(BF16, 512, 64, 66000), (F32, 16, 64, 2400)])
def test_scan_over_wide_buffers(dtype, H, V, T):
    """x, z and y of more than 2^31 elements (or of more than 2^31 bytes between two
    rows of a batch): the last tokens as a prompt of their own from the state before."""
    d = cuda(ssm_inputs(23, 1, 300, H, 1, V, 128, dtype))
    if dtype is F32:
        base = torch.zeros((2, 2 ** 29 + 64), dtype=dtype, device="cuda")
        x = base.as_strided((2, T, H, V), (base.stride(0), H * V, V, 1))
        rep = 2
    else:
        x, rep = torch.zeros((1, T, H, V), dtype=dtype, device="cuda"), 1
    x[:, -300:] = d["x"]

    def grown(t):
        out = torch.zeros((rep, T, *t.shape[2:]), dtype=dtype, device="cuda")
        out[:, -300:] = t
        return out

    kw = dict(A_log=d["A_log"], D=d["D"], dt_bias=d["dt_bias"], out_dtype=F32)
    y, ht = gdn.ssm_chunk_fwd(x, grown(d["dt"]), Bm=grown(d["Bm"]), Cm=grown(d["Cm"]), z=x, **kw)
    want, h = gdn.ssm_chunk_fwd(d["x"], d["dt"], Bm=d["Bm"], Cm=d["Cm"], z=d["x"], **kw)
    ok()
    tol = TOL_F32 if dtype is F32 else TOL_BF16
    for b in range(rep):
        assert_close(y[b:b + 1, -300:], want.double().cpu().numpy(), tol, "y")
        assert_close(ht[b:b + 1], h.double().cpu().numpy(), TOL_F32, "ht")


def test_example():
    """Both sides round to bfloat16 in four places (the two projections, the
    convolution, the scan), of values summed in different orders: four units of
    2^-8 of a value of up to six RMS."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("ssm_block",
                                                  os.path.join(root, "examples", "ssm_block.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(steps=5) < 4 * 6 * 2 ** -8


CHECKED = """
import sys
sys.path[:0] = sys.argv[1:3]
import torch
from gated_delta_rule_kk_gb300 import _lib
import gated_delta_rule_kk_gb300 as gdn
from _mixer import conv_inputs, cuda, ssm_inputs

checked, release = _lib.load(), _lib.load(sys.argv[3])


def conv(T, dtype, lens=None):
    d = cuda(conv_inputs(1, 1, T, 520, 4, dtype, lens=lens))
    y = gdn.short_conv_fwd(d["x"], d["weight"], d["bias"], d["h0"], d["cu"])
    g = gdn.short_conv_bwd(d["dy"], d["x"], d["weight"], d["bias"], d["h0"], d["dht"], d["cu"])
    return *y, *g


def conv_token():
    d = cuda(conv_inputs(2, 3, 2, 520, 4, torch.bfloat16))
    return gdn.short_conv_decode(d["x"], d["weight"], d["h0"], d["bias"]), d["h0"]


def scan(T, dtype, lens=None, segment=0):
    d = cuda(ssm_inputs(3, 1, T, 4, 2, 72, 128, dtype, lens=lens))
    return gdn.ssm_chunk_fwd(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], D=d["D"], z=d["z"],
                             dt_bias=d["dt_bias"], initial_state=d["h0"], cu_seqlens=d["cu"],
                             segment_tokens=segment)


def token(B, T, state):
    d = cuda(ssm_inputs(4, B, T, 16, 2, 72, 128, torch.bfloat16))
    h = d["h0"].to(state)
    return gdn.ssm_decode(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], h, D=d["D"], z=d["z"],
                          dt_bias=d["dt_bias"]), h


cases = [lambda: conv_token()]
for dt in (torch.bfloat16, torch.float32):
    cases += [lambda dt=dt: conv(1, dt), lambda dt=dt: conv(37, dt, [0, 1, 36]),
              lambda dt=dt: conv(3001, dt, [1500, 0, 1501]), lambda dt=dt: scan(1, dt),
              lambda dt=dt: scan(300, dt, [129, 0, 1, 170]), lambda dt=dt: scan(300, dt, None, 128),
              lambda dt=dt: token(1, 1, dt), lambda dt=dt: token(100, 3, dt)]
for i, case in enumerate(cases):
    results = []
    for lib in (checked, release):
        _lib._lib = lib
        results.append(case())
        status = gdn.gdn_check_device_error()
        assert status == 0, (i, status)
    for a, b in zip(*results):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b)), i
"""


def test_checked_build():
    """The bounds-checked build records nothing on valid calls and computes the same."""
    tests = os.path.dirname(os.path.abspath(__file__))
    build_lib.build(checked=True)
    r = subprocess.run([sys.executable, "-c", CHECKED, os.path.dirname(tests), tests,
                        build_lib.build()], env=dict(os.environ, GDN_CHECKED="1"),
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout + r.stderr


def test_calls_on_another_stream():
    d = cuda(ssm_inputs(13, 1, 400, 2, 1, 64, 128, BF16))
    args = (d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"])
    y, ht = gdn.ssm_chunk_fwd(*args, dt_bias=d["dt_bias"], segment_tokens=128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2, ht2 = gdn.ssm_chunk_fwd(*args, dt_bias=d["dt_bias"], segment_tokens=128, stream=s)
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(ht, ht2)


def test_graph_capture():
    d = cuda(ssm_inputs(14, 2, 1, 4, 1, 64, 128, BF16))
    state = d["h0"].clone()
    want = gdn.ssm_decode(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], state.clone())
    graph = torch.cuda.CUDAGraph()
    start = state.clone()
    out = torch.empty_like(want)
    with torch.cuda.graph(graph):
        gdn.ssm_decode(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], state, out=out)
    state.copy_(start)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_refusals():
    d = cuda(conv_inputs(15, 2, 8, 16, 4, BF16))
    x, w = d["x"], d["weight"]
    for bad in (dict(x=x.half()), dict(x=x[0]), dict(x=x.cpu()), dict(x=x.transpose(1, 2)),
                dict(weight=w[:5]), dict(weight=w.half()), dict(bias=w[:, 0]),
                dict(activation="gelu"), dict(initial_state=d["h0"][:1]),
                dict(cu_seqlens=torch.zeros(1, dtype=torch.int32, device="cuda")),
                dict(out=torch.empty(2, 8, 17, dtype=BF16, device="cuda"))):
        with pytest.raises(ValueError):
            gdn.short_conv_fwd(**{**dict(x=x, weight=w), **bad})
    with pytest.raises(GdnError) as e:
        gdn.short_conv_fwd(x, torch.ones(16, 5, dtype=BF16, device="cuda"))
    assert e.value.status == Status.UNSUPPORTED
    with pytest.raises(GdnError) as e:
        gdn.short_conv_decode(torch.zeros(2, 5, 16, dtype=BF16, device="cuda"), w, d["h0"])
    assert e.value.status == Status.UNSUPPORTED
    s = cuda(ssm_inputs(16, 2, 8, 4, 2, 16, 16, BF16))
    args = dict(x=s["x"], dt=s["dt"], A_log=s["A_log"], Bm=s["Bm"], Cm=s["Cm"])
    for bad in (dict(dt=s["dt"].half()), dict(A_log=s["A_log"].bfloat16()), dict(D=s["D"][:2]),
                dict(z=s["z"].float()), dict(Cm=s["Cm"][:, :4]), dict(out_dtype=torch.float16),
                dict(x=s["x"].transpose(2, 3)), dict(initial_state=s["h0"].bfloat16())):
        with pytest.raises(ValueError):
            gdn.ssm_chunk_fwd(**{**args, **bad})
    with pytest.raises(GdnError) as e:
        gdn.ssm_chunk_fwd(**args, segment_tokens=100)
    assert e.value.status == Status.INVALID_ARG
    ok()
