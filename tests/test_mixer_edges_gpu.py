"""Edges of the short convolution and the state space scan on the GPU."""
import threading

import numpy as np
import pytest
import torch

import gated_delta_rule_kk_gb300 as gdn
from gated_delta_rule_kk_gb300 import Status
from oracle import mixer as M

from _mixer import assert_each_close, assert_inside, conv_inputs, cuda, scan_rooms, ssm_inputs
from _util import TOL_F32, assert_close

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def ok():
    assert gdn.gdn_check_device_error() == Status.OK


def scan(d, **kw):
    return gdn.ssm_chunk_fwd(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], D=d["D"], z=d["z"],
                             dt_bias=d["dt_bias"], initial_state=d["h0"], cu_seqlens=d["cu"], **kw)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype,T,V,K,lens,segment,at", [
    (BF16, 300, 64, 128, None, 0, [(5, 1, 3)]),
    (BF16, 300, 64, 128, None, 0, [(127, 0, 63), (128, 0, 0), (299, 1, 33)]),
    (BF16, 300, 64, 64, None, 128, [(200, 1, 17), (140, 1, 17), (256, 0, 5)]),
    (BF16, 300, 72, 128, [100, 0, 200], 0, [(50, 0, 71), (120, 1, 64), (299, 0, 2)]),
    (F32, 100, 40, 48, None, 0, [(5, 1, 3), (70, 0, 39)]),
])
@pytest.mark.parametrize("out", [BF16, F32])
def test_scan_keeps_the_tokens_before_a_value_that_is_not_finite(value, dtype, T, V, K, lens,
                                                                 segment, at, out):
    """x of one token and state row reaches that row's outputs from the token on, and no other.
    The others are the same arithmetic: the same bits."""
    if dtype == F32 and out == BF16:
        out = None
    d = cuda(ssm_inputs(31, 1, T, 2, 1, V, K, dtype, lens))
    kw = dict(segment_tokens=segment, out_dtype=out)
    y, ht = scan(d, **kw)
    bad = {**d, "x": d["x"].clone()}
    clean = torch.ones((1, T, 2, V), dtype=torch.bool, device="cuda")
    kept = torch.ones(ht.shape, dtype=torch.bool, device="cuda")
    ends = [0, T] if lens is None else [0, lens[0], lens[0] + lens[1], T]
    for t, h, v in at:
        bad["x"][0, t, h, v] = value
        n = next(n for n in range(len(ends) - 1) if ends[n] <= t < ends[n + 1])
        clean[0, t:ends[n + 1], h, v] = False
        kept[n, h, v] = False
    y2, ht2 = scan(bad, **kw)
    ok()
    assert torch.equal(y2[clean], y[clean])
    assert not y2[~clean].isfinite().any()
    assert torch.equal(ht2[kept], ht[kept])
    assert not ht2[~kept].isfinite().any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", ["Bm", "Cm", "z"])
def test_scan_keeps_the_tokens_before_nan_in_the_other_inputs(dtype, name):
    d = cuda(ssm_inputs(32, 1, 300, 2, 1, 64, 128, dtype))
    y, _ = scan(d)
    for t in (0, 77, 130, 299):
        bad = {**d, name: d[name].clone()}
        bad[name][:, t] = float("nan")
        y2, _ = scan(bad)
        ok()
        assert torch.equal(y2[:, :t], y[:, :t]), t
        if name != "Bm":  # B lives on in the state, C and z only in their own token
            assert torch.equal(y2[:, t + 1:], y[:, t + 1:]), t
        assert y2[:, t].isnan().all(), t


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("segment", [0, 128])
def test_scan_states_keep_an_infinite_value(dtype, segment):
    """An infinite x leaves infinities of B's signs in its row of the state, two of opposite
    signs NaN, as the recurrence does (few enough tokens after it that no decay is zero)."""
    i = ssm_inputs(33, 1, 300, 2, 1, 64, 128, dtype)
    i["x"] = i["x"].clone()
    i["x"][0, 290, 0, 7] = i["x"][0, 280, 1, 63] = i["x"][0, 299, 1, 0] = float("inf")
    i["x"][0, 288, 1, 20] = float("-inf")
    i["x"][0, 285, 0, 50], i["x"][0, 295, 0, 50] = float("inf"), float("-inf")
    _, ht = scan(cuda(i), segment_tokens=segment)
    ok()
    with np.errstate(invalid="ignore"):
        _, ref = M.ssm_scan(i["x"], i["dt"], i["A_log"], i["Bm"], i["Cm"], i["D"], i["z"],
                            i["dt_bias"], h0=i["h0"])
    ref = torch.from_numpy(ref)
    there = ~ref.isfinite()
    assert there.sum() >= 4 * 128 and ref[there].isinf().any() and ref[there].isnan().any()
    got = ht.cpu().double()
    assert torch.equal(got.isfinite(), ~there)
    assert torch.equal(got[there].nan_to_num(0.5, 1, -1), ref[there].nan_to_num(0.5, 1, -1))


def check_inside(i, **kw):
    """y of the tensor cores within what their roundings allow, element for element, and the
    states within the float32 bound."""
    y, ht = scan(cuda(i), out_dtype=F32, **kw)
    ok()
    ref, rht = M.ssm_scan(i["x"], i["dt"], i["A_log"], i["Bm"], i["Cm"], i["D"], i["z"],
                          i["dt_bias"], h0=i["h0"], cu_seqlens=i["cu"])
    assert_inside(y, ref, scan_rooms(i), "y")
    assert_close(ht, rht, TOL_F32, "ht")


@pytest.mark.parametrize("B,T,H,Hg,V,K,lens,segment", [
    (1, 1, 2, 1, 64, 128, None, 0),
    (2, 63, 4, 2, 64, 128, None, 0),
    (1, 128, 2, 2, 64, 64, None, 0),
    (1, 129, 3, 1, 64, 128, None, 0),
    (2, 257, 2, 1, 128, 128, None, 0),
    (1, 300, 4, 2, 64, 128, [0, 1, 130, 0, 41, 128, 0], 0),
    (1, 200, 3, 3, 40, 48, [77, 123], 0),
    (1, 1000, 2, 1, 64, 128, None, 128),
    (1, 1000, 2, 1, 64, 128, [700, 0, 1, 128, 171], 384),
])
def test_scan_within_its_roundings(B, T, H, Hg, V, K, lens, segment):
    check_inside(ssm_inputs(T + K + 1, B, T, H, Hg, V, K, BF16, lens), segment_tokens=segment)


@pytest.mark.parametrize("fast", [False, True])
def test_scan_within_its_roundings_bare_and_with_strong_decays(fast):
    check_inside(ssm_inputs(42, 1, 400, 4, 1, 64, 128, BF16, fast=fast))
    check_inside(ssm_inputs(43, 2, 200, 2, 1, 64, 128, BF16, h0=False, z=False, skip=False,
                            fast=fast))


@pytest.mark.parametrize("resets", [[40], [0, 31, 32], [100, 101, 110, 250]])
def test_scan_after_a_token_that_resets_the_state(resets):
    """A step size of 6e4 (log-decays of down to -1e6) in one token: the tokens after it in its
    block differ by decays near one, which no difference of such sums gives."""
    i = ssm_inputs(44, 1, 300, 4, 2, 64, 128, BF16)
    i["dt"] = i["dt"].clone()
    i["dt"][:, resets] = 6e4
    check_inside(i)


@pytest.mark.parametrize("T,resets", [(2, [0]), (3, [1]), (4, [0, 2]), (4, [3])])
@pytest.mark.parametrize("B,H", [(2, 4), (60, 32)])  # straight from memory, and through the ring
def test_scan_tokens_after_one_that_resets_the_state(T, resets, B, H):
    """As above, among the tokens of one call."""
    i = ssm_inputs(45, B, T, H, 1, 64, 128, BF16)
    i["dt"] = i["dt"].clone()
    i["dt"][:, resets] = 6e4
    d = cuda(i)
    state = d["h0"].clone()
    y = gdn.ssm_decode(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], state, D=d["D"], z=d["z"],
                       dt_bias=d["dt_bias"], out_dtype=F32)
    ok()
    ref, rht = M.ssm_scan(i["x"], i["dt"], i["A_log"], i["Bm"], i["Cm"], i["D"], i["z"],
                          i["dt_bias"], h0=i["h0"])
    assert_close(y, ref, TOL_F32, "y")
    assert_close(state, rht, TOL_F32, "state")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_of_single_tokens_with_any_stride_between_them(dtype):
    """The stride over one token, or one batch row, is never used: 2^41 elements here."""
    d = cuda(ssm_inputs(46, 2, 1, 4, 1, 64, 128, dtype))
    y, ht = scan(d)

    def wide(t):
        s = list(t.stride())
        s[1] = 2 ** 41 + 8
        return t.as_strided(t.shape, s)

    y2, ht2 = scan({**d, **{k: wide(d[k]) for k in ("x", "Bm", "Cm", "z", "dt")}}, out=wide(
        torch.empty_like(y)))
    ok()
    assert torch.equal(y2, y) and torch.equal(ht2, ht)
    one = {k: v[:1] if k in ("x", "Bm", "Cm", "z", "dt", "h0") else v for k, v in d.items()}
    far = {k: v.as_strided(v.shape, (2 ** 42, *v.stride()[1:]))
           if k in ("x", "Bm", "Cm", "z", "dt") else v for k, v in one.items()}
    y3, ht3 = scan(far)
    ok()
    assert torch.equal(y3, y[:1]) and torch.equal(ht3, ht[:1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_inputs_shared_by_a_batch(dtype):
    """Rows of a batch that are one row expanded (a batch stride of zero)."""
    d = cuda(ssm_inputs(47, 1, 300, 2, 1, 64, 128, dtype))
    both = {k: v.expand(3, *v.shape[1:]) if k in ("x", "Bm", "Cm", "z", "dt") else v
            for k, v in d.items()}
    y, ht = scan(d)
    y2, ht2 = scan({**both, "h0": d["h0"].repeat(3, 1, 1, 1)})
    ok()
    assert all(torch.equal(y2[b], y[0]) and torch.equal(ht2[b], ht[0]) for b in range(3))
    for T, D in ((40, 72), (4000, 2056)):  # from memory, and through the ring
        c = cuda(conv_inputs(48, 1, T, D, 4, dtype))
        y, ht = gdn.short_conv_fwd(c["x"], c["weight"], c["bias"], c["h0"])
        y2, ht2 = gdn.short_conv_fwd(c["x"].expand(3, T, D), c["weight"], c["bias"],
                                     c["h0"].repeat(3, 1, 1))
        ok()
        assert all(torch.equal(y2[b], y[0]) and torch.equal(ht2[b], ht[0]) for b in range(3))
        g = gdn.short_conv_bwd(c["dy"], c["x"], c["weight"], c["bias"], c["h0"])
        g2 = gdn.short_conv_bwd(c["dy"].expand(3, T, D), c["x"].expand(3, T, D), c["weight"],
                                c["bias"], c["h0"].repeat(3, 1, 1))
        ok()
        assert all(torch.equal(g2[0][b], g[0][0]) and torch.equal(g2[3][b], g[3][0])
                   for b in range(3))


def test_calls_from_several_threads():
    """Each on a stream of its own, all at once, the first calls among them."""
    c, d = cuda(conv_inputs(49, 1, 4000, 2056, 4, BF16)), cuda(ssm_inputs(49, 1, 400, 2, 1, 64, 128,
                                                                          BF16))
    start, results = threading.Barrier(6), [None] * 6
    torch.cuda.synchronize()

    def work(k):
        stream = torch.cuda.Stream()
        start.wait()
        out = [*gdn.short_conv_fwd(c["x"], c["weight"], c["bias"], c["h0"], stream=stream),
               *scan(d, segment_tokens=128, stream=stream)]
        stream.synchronize()
        results[k] = out

    threads = [threading.Thread(target=work, args=(k,)) for k in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    ok()
    want = [*gdn.short_conv_fwd(c["x"], c["weight"], c["bias"], c["h0"]),
            *scan(d, segment_tokens=128)]
    for out in results:
        assert out is not None and all(torch.equal(a, b) for a, b in zip(out, want))


def test_convolution_of_the_longest_row():
    """One channel of 2^31 - 256 tokens: the last run ends where 31 bits do."""
    T, n = 0x7fffff00, 600
    i = conv_inputs(50, 1, n, 1, 4, BF16, state=False)
    c = cuda(i)
    x = torch.zeros((1, T, 1), dtype=BF16, device="cuda")
    x[:, -n:] = c["x"]
    y, ht = gdn.short_conv_fwd(x, c["weight"], c["bias"])
    ok()
    ry, rht = M.short_conv(i["x"], i["weight"], i["bias"])
    assert_each_close(y[:, -n:], ry, "y", 1e-5)
    assert_each_close(ht, rht, "ht", 1e-5)
    del y
    dx, dw, _, _ = gdn.short_conv_bwd(x, x, c["weight"], c["bias"])
    ok()
    rx, rw, _, _ = M.short_conv_grad(i["x"], i["x"], i["weight"], i["bias"])
    assert_each_close(dx[:, -n:], rx, "dx", 1e-5)
    assert not dx[:, :-n - 3].any()
    assert_each_close(dw, rw, "dw", 1e-5)


def replayed(call, *changed):
    """The outputs of `call` captured in a graph and replayed on the same inputs, with the
    buffers it changes in place put back before and returned behind."""
    before = [t.clone() for t in changed]
    call()  # attributes and look-ups of a first call
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [t for t in call() if t is not None]
    for t in out:
        t.fill_(7)
    for t, b in zip(changed, before):
        t.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    ok()
    return [t.clone() for t in (*out, *changed)]


@pytest.mark.parametrize("B,T,H", [(2, 1, 4), (3, 4, 4), (100, 1, 16)])  # the last by the ring
def test_graphs_of_tokens(B, T, H):
    d = cuda(ssm_inputs(51, B, T, H, 1, 64, 128, BF16))
    c = cuda(conv_inputs(51, B, T, 264, 4, BF16))

    def token(state):
        return gdn.ssm_decode(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], state, D=d["D"],
                              z=d["z"], dt_bias=d["dt_bias"]),

    def conv(state):
        return gdn.short_conv_decode(c["x"], c["weight"], state, c["bias"]),

    for call, start in ((token, d["h0"]), (conv, c["h0"])):
        state = start.clone()
        want = [*call(state), state]
        assert not torch.equal(state, start)
        held = start.clone()
        assert all(map(torch.equal, replayed(lambda: call(held), held), want))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,D", [(300, 72), (4000, 2056)])  # from memory, and through the ring
def test_graphs_of_prompts(dtype, T, D):
    lens = [T // 3, 0, T - T // 3]
    c = cuda(conv_inputs(52, 1, T, D, 4, dtype, lens=lens))
    d = cuda(ssm_inputs(52, 1, T, 2, 1, 64, 128, dtype, lens=lens))
    calls = (lambda: gdn.short_conv_fwd(c["x"], c["weight"], c["bias"], c["h0"], c["cu"]),
             lambda: gdn.short_conv_bwd(c["dy"], c["x"], c["weight"], c["bias"], c["h0"], c["dht"],
                                        c["cu"]),
             lambda: scan(d), lambda: scan(d, segment_tokens=128))
    for call in calls:
        want = [t for t in call() if t is not None]
        assert all(map(torch.equal, replayed(call), want))


@pytest.mark.parametrize("B,H,K", [(3, 24, 128), (64, 28, 128), (116, 28, 48)])
def test_scan_token_states_are_rounded_step_by_step(B, H, K):
    """A bfloat16 state is its update with every float32 product and sum rounded by itself and
    one rounding at the end, bit for bit: kept over many calls, it does not drift from that."""
    d = cuda(ssm_inputs(53, B, 1, H, 1, 64, K, F32))
    state = (torch.randn((B, H, 64, K), device="cuda") / 2).to(BF16)
    s = d["dt"][:, 0] + d["dt_bias"]
    s = torch.where(s > 20, s, torch.log1p(torch.exp(s)))
    keep = torch.exp(-torch.exp(d["A_log"]) * s)[..., None, None]
    new = (d["x"][:, 0] * s[..., None])[..., None] * d["Bm"][:, 0, :, None, :]
    old = keep * state.float()
    want = (old + new).to(BF16)
    gdn.ssm_decode(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], state, dt_bias=d["dt_bias"])
    ok()
    assert torch.equal(state, want)
