"""Calls of the delta rule layers' operators that their other tests do not make.

Bounds.  In norm, float32 results of the tensor cores as tests/test_layer_gpu.py derives
(1e-5).  Of float32 inputs: a product's sum of up to 64 terms rounds by 2^-24 a step, sqrt(64)
of them in quadrature, and six products follow one another: 7e-6 at most if all rounded the same
way, sqrt(6) x 8 x 2^-24 = 1.2e-6 as they do; e^x is off by 2^-24 |x|, where |x| e^x is below
one.  1e-5 as well.  Element for element as there: 3e-3 RMS with pieces, 1e-4 without.

Pieces end at bfloat16's smallest step, 2^-133, half of which an operand is off by besides.
Each token that reaches dh0 adds two products to it, of do with q and of dr with k, whose rows
of q and k have length 1: in norm sqrt(V) 2^-134 each.  (Counts where e^G is 1e-35.)
"""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import gated_delta_rule_kk_gb300 as gdn
from gated_delta_rule_kk_gb300 import Status, _lib, build_lib
from gated_delta_rule_kk_gb300._lib import GdnChunkBwdArgs
from oracle import layer as L
from oracle import mixer as M

from _layer import delta_inputs, kda_inputs
from _mixer import assert_each_close, cuda
from _util import TOL_F32, _np
from test_layer_gpu import PIECES, run_delta

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def ok():
    assert gdn.gdn_check_device_error() == Status.OK


def check_norms(got, i, reach=64, **kw):
    """Every result element for element, the float32 ones within 1e-5 of their norm; ``reach``
    tokens of a sequence reach its initial state.  The norm's bound for pieces is that of many
    independent errors (2^-19 of a value each, in quadrature): below 200 values of dg it says
    nothing, as what is left of a sum whose terms cancel may be all there is (dg of two tokens and
    heads is four such sums, of terms up to four times as large), and 3e-3 element for element,
    which counts every term with its largest error, is the bound."""
    ref = L.gdn_grad(i["do"], i["q"], i["k"], i["v"], i["g"], i["beta"], i["scale"], i["h0"],
                     i["dht"], i["cu"], **kw)
    K, V = i["q"].shape[3], i["v"].shape[3]
    pieces = i["q"].dtype is BF16 and K % 8 == 0 and V % 8 == 0 and V <= 128
    step = reach * 2 * 2.0 ** -134 * np.sqrt(ref[5].size / ref[5].shape[2]) if pieces else 0.0
    off = {}
    for name, x, r in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got, ref):
        if name != "dh0" or not pieces or np.abs(r).max() > 2.0 ** -100:
            assert_each_close(x, r, name, PIECES if pieces else TOL_F32)
        if x.dtype is F32 and (not pieces or ref[3].size >= 200):
            room = 1e-5 * np.linalg.norm(r) + (step if name == "dh0" else 0.0)
            off[name] = np.linalg.norm(_np(x) - r) / max(room, 1e-300)
    assert max(off.values(), default=0) <= 1.0, {k: f"{v:.2f} times the allowed error" for k, v in off.items()}


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("every", [2, 3, 4, 8, 21])
@pytest.mark.parametrize("gate", [-float("inf"), -1e4, -80.0, -30.0])
def test_delta_gradient_of_many_gates_that_forget(dtype, every, gate):
    """The running sums reach some -3300 in a chunk; the tokens between two such gates are
    coupled by differences of them."""
    i = delta_inputs(every, 1, 150, 2, 2, 64, 64, dtype, [90, 60])
    i["g"][:, ::every] = gate
    got = run_delta(cuda(i))
    ok()
    check_norms(got, i, reach=every)


@pytest.mark.parametrize("dtype,K,V", [(BF16, 64, 64), (F32, 64, 64), (BF16, 20, 30)])
@pytest.mark.parametrize("T", [1, 2, 63, 130])
@pytest.mark.parametrize("gate", [-30.0, -15.0])
def test_delta_gradient_where_every_gate_forgets(dtype, K, V, T, gate):
    """dg is as small as e^g, and right to its own size: nothing of order one cancels in it."""
    i = delta_inputs(T, 1, T, 2, 1, K, V, dtype)
    i["g"][:] = gate
    got = run_delta(cuda(i))
    ok()
    check_norms(got, i)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_delta_gradient_of_many_gates_that_forget_and_shared_heads(dtype):
    i = delta_inputs(3, 2, 200, 4, 2, 96, 40, dtype)
    i["g"][:, 1::3] = -60.0
    i["g"][:, :, 1] = -5.0
    got = run_delta(cuda(i))
    ok()
    check_norms(got, i)


def test_delta_gradient_without_tokens_checks_its_offsets():
    i = delta_inputs(15, 1, 0, 2, 2, 64, 64, BF16, [0, 0])
    d = cuda(i)
    assert torch.equal(run_delta(d)[5], d["dht"])
    ok()
    for cu in ([0, 5, 0], [0, 0, 3], [1, 1, 1]):
        d["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        run_delta(d)
        assert gdn.gdn_check_device_error() == Status.BAD_SEQLENS, cu


@pytest.mark.parametrize("dht", [False, True])
def test_delta_gradient_of_bad_offsets_without_tokens_writes_nothing(dht):
    """Also through the C entry, with and without a gradient of the last states."""
    states = torch.ones(2, 2, 8, 8, device="cuda")
    dh0 = torch.full_like(states, 7.0)
    a = GdnChunkBwdArgs(dtype=1, B=1, T=0, H=2, Hg=2, K=8, V=8, N=2, chunk_size=64,
                        dht=states.data_ptr() if dht else None, dh0=dh0.data_ptr())
    for cu, status in (([0, 5, 0], Status.BAD_SEQLENS), ([0, 0, 1], Status.BAD_SEQLENS),
                       ([0, 0, 0], Status.OK)):
        at = torch.tensor(cu, dtype=torch.int32, device="cuda")
        a.cu_seqlens = at.data_ptr()
        st = _lib.load().gdn_chunk_bwd(ctypes.byref(a), torch.cuda.current_stream().cuda_stream)
        assert st == Status.OK and gdn.gdn_check_device_error() == status
        want = 7.0 if status else float(dht)
        assert torch.equal(dh0, torch.full_like(dh0, want))
    a.cu_seqlens, a.B = None, 2
    dh0.fill_(7)
    assert _lib.load().gdn_chunk_bwd(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == Status.OK
    assert torch.equal(dh0, torch.full_like(dh0, float(dht)))
    ok()


@pytest.mark.parametrize("dtype,K,V", [(BF16, 128, 64), (BF16, 64, 32), (F32, 64, 64)])
def test_delta_gradient_along_a_long_chain(dtype, K, V):
    """64 chunks whose gates hardly forget."""
    i = delta_inputs(22, 1, 4096, 1, 1, K, V, dtype)
    i["g"] = i["g"] * 0.02
    got = run_delta(cuda(i))
    ok()
    check_norms(got, i)


def test_delta_gradient_is_the_forward_s():
    """Differences of the library's own forward in float32 along the gradient and as much of a
    random direction (each of length 1), where a wrong sign or size shows as itself.  The
    differences' own error, from the definition in 64 bits: 6e-4 of the gradient's length (g;
    the others below 1e-5).  The forward's rounding: 12800 values of o of 0.2 off by 1e-6
    of that, random against do, over 2 x 0.05: 3e-4, 6e-5 of the smallest gradient's 4.8."""
    i = delta_inputs(11, 2, 100, 2, 2, 32, 32, F32)
    d = cuda(i)
    grads = run_delta(d)
    ok()

    def loss(x):
        o, ht = gdn.gdn_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], scale=i["scale"],
                                  initial_state=x["h0"])
        return float((o.double() * d["do"]).sum() + (ht.double() * d["dht"]).sum())

    rng, e = torch.Generator().manual_seed(0), 0.05
    for name, grad in zip(("q", "k", "v", "g", "beta", "h0"), grads):
        noise = torch.randn(grad.shape, generator=rng).cuda()
        # (as the kernel sees it: both sides' inputs rounded to float32)
        up = (d[name].double() + e * (grad / grad.norm() + noise / noise.norm()).double()).float()
        down = (2 * d[name].double() - up.double()).float()
        diff = loss({**d, name: up}) - loss({**d, name: down})
        along = float(((up.double() - down.double()) * grad).sum())
        size = 2 * e * float(grad.double().norm())
        assert abs(along) >= 0.5 * size, name
        assert abs(diff - along) <= 2e-3 * size, (name, diff, along)


# ---------------------------------------------------------------- waits that run out

@pytest.fixture(scope="module")
def waiting_out(tmp_path_factory):
    """By role, the library whose warps of that role find every wait run out."""
    build_lib.build()
    jobs, links, libs = [], [], {}
    for role in range(4):
        folder, objs = str(tmp_path_factory.mktemp(f"role{role}")), []
        for src in build_lib._sources():
            name = os.path.basename(src)[:-3] + ".o"
            if "role_polls" in open(src).read():
                objs.append(os.path.join(folder, name))
                jobs.append([build_lib._nvcc(), *build_lib.NVCC_FLAGS, f"-DGDN_WAITS_OUT={role}", "-c",
                             src, "-o", objs[-1]])
            else:
                objs.append(os.path.join(build_lib.BUILD_DIR, name))
        libs[role] = os.path.join(folder, f"libgdn_waits_out_{role}.so")
        links.append([build_lib._nvcc(), *build_lib.ARCH, "-shared", "-cudart", "shared", "-o", libs[role],
                      *objs])
    for commands in (jobs, links):
        for p in [subprocess.Popen(c) for c in commands]:
            assert p.wait() == 0
    return libs


def run_waiting_out(script, role, libs):
    tests = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", PRELUDE + script, os.path.dirname(tests), tests,
                        build_lib.build(), libs[role], str(role)],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr


PRELUDE = r"""
import sys
sys.path[:0] = [sys.argv[1], sys.argv[2]]
import torch
from gated_delta_rule_kk_gb300 import _lib, Status
import gated_delta_rule_kk_gb300 as gdn
from _layer import delta_inputs, kda_inputs
from _mixer import cuda

release, other, role = _lib.load(sys.argv[3]), _lib.load(sys.argv[4]), int(sys.argv[5])
BF16, F32 = torch.bfloat16, torch.float32


def call(lib, f, status):
    _lib._lib = lib
    out = f()
    got = gdn.gdn_check_device_error()
    assert got == status, (got, status)
    return out
"""

KDA_WAITS = r"""
d = cuda(kda_inputs(5, 400, 1 + role % 2, 2, 4, 128, 128, BF16, F32 if role % 2 else BF16))
before = d["state"].clone()


def tokens(state):
    gdn.kda_decode(d["q"], d["k"], d["v"], d["a"], d["b"], d["A_log"], d["dt_bias"], state,
                   slot_indices=d["slots"])
    return state


after = call(release, lambda: tokens(before.clone()), Status.OK)
mid = call(other, lambda: tokens(before.clone()), Status.TIMEOUT)
same, done = ((mid == x).all(-1) for x in (before, after))
assert (same | done).all(), int((~(same | done)).sum())
if role in (0, 3):  # nothing is taken, or nothing stored
    assert same.all()
assert torch.equal(call(release, lambda: tokens(before.clone()), Status.OK), after)
"""


@pytest.mark.parametrize("role", [0, 1, 2, 3])
def test_kda_tokens_whose_waits_run_out_leave_states_whole(role, waiting_out):
    """Warps that take tiles, prepare, load or store: every row is the call's, or as it was."""
    run_waiting_out(KDA_WAITS, role, waiting_out)


SSM_WAITS = r"""
from _mixer import ssm_inputs
d = cuda(ssm_inputs(5, 400, 2, 16, 2, 64, 128, BF16, h0=False))
g = torch.Generator(device="cuda").manual_seed(1)
before = torch.randn(400, 16, 64, 128, device="cuda", generator=g).bfloat16()


def tokens(state):
    gdn.ssm_decode(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], state, dt_bias=d["dt_bias"])
    return state


after = call(release, lambda: tokens(before.clone()), Status.OK)
mid = call(other, lambda: tokens(before.clone()), Status.TIMEOUT)
same, done = ((mid == x).all(-1) for x in (before, after))
assert (same | done).all(), int((~(same | done)).sum())
if role in (0, 3):
    assert same.all()
assert torch.equal(call(release, lambda: tokens(before.clone()), Status.OK), after)
"""


@pytest.mark.parametrize("role", [0, 1, 2, 3])
def test_state_space_tokens_whose_waits_run_out_leave_states_whole(role, waiting_out):
    run_waiting_out(SSM_WAITS, role, waiting_out)


CONV_WAITS = r"""
from _mixer import conv_inputs
d = cuda(conv_inputs(5, 2, 4096, 6144, 4, BF16))


def rows():
    y, _ = gdn.short_conv_fwd(d["x"], d["weight"], d["bias"])
    return y, *gdn.short_conv_bwd(d["dy"], d["x"], d["weight"], d["bias"])[:3]


want = call(release, rows, Status.OK)
call(other, rows, Status.TIMEOUT)
for a, b in zip(want, call(release, rows, Status.OK)):
    assert torch.equal(a, b)
"""


@pytest.mark.parametrize("role", [0, 2])
def test_convolution_whose_waits_run_out_ends(role, waiting_out):
    run_waiting_out(CONV_WAITS, role, waiting_out)


DELTA_WAITS = r"""
import ctypes
from gated_delta_rule_kk_gb300._lib import GdnChunkBwdArgs
H, Hg, K = 4, 2, 128
d = cuda(delta_inputs(6, 1, 2000, H, Hg, K, K, BF16, [900, 1100]))


def gradient():  # its outputs between guards of 7
    outs = {}
    for n, t in dict(dq="q", dk="k", dv="v", dg="g", dbeta="beta", dh0="h0").items():
        room = torch.full((d[t].numel() + (2 << 16),), 7.0, dtype=d[t].dtype, device="cuda")
        outs[n] = room, room[1 << 16:-(1 << 16)]
    a = GdnChunkBwdArgs(dtype=1, B=1, T=2000, H=H, Hg=Hg, K=K, V=K, N=2, chunk_size=64,
                        **{n: d[n].data_ptr() for n in ("q", "k", "v", "g", "beta", "h0", "dht")},
                        do_=d["do"].data_ptr(), cu_seqlens=d["cu"].data_ptr(),
                        **{n: t.data_ptr() for n, (_, t) in outs.items()})
    n = ctypes.c_size_t(0)
    assert _lib._lib.gdn_chunk_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n)) == Status.OK
    room = torch.zeros(n.value + (1 << 20), dtype=torch.uint8, device="cuda")
    a.workspace, a.workspace_bytes = room.data_ptr(), n.value
    assert _lib._lib.gdn_chunk_bwd(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == Status.OK
    torch.cuda.synchronize()
    assert not room[n.value:].any()
    for r, _ in outs.values():
        assert (r[:1 << 16] == 7).all() and (r[-(1 << 16):] == 7).all()
    return [t for _, t in outs.values()]


want = call(release, gradient, Status.OK)
call(other, gradient, Status.TIMEOUT)
for a, b in zip(want, call(release, gradient, Status.OK)):
    assert torch.equal(a, b)
"""


@pytest.mark.parametrize("role", [0, 1, 2, 3])
def test_delta_gradient_whose_waits_run_out_ends(role, waiting_out):
    """Warps that carry (finish), hand on (multiply), load or store (count): the call ends with
    an error, nothing is written elsewhere and the next call is right."""
    run_waiting_out(DELTA_WAITS, role, waiting_out)


# ---------------------------------------------------------------- KDA's tokens, both kernels

@pytest.mark.parametrize("T,state", [(1, BF16), (1, F32), (2, BF16), (2, F32), (3, F32), (4, BF16)])
@pytest.mark.parametrize("K,V", [(128, 128), (256, 72), (40, 24)])
def test_kda_tokens_of_many_requests_are_those_of_few(T, state, K, V):
    """A call whose states stream and calls of a few requests each: the same to the bit (the
    kernels share the arithmetic of a tile), other slots untouched."""
    B = 600
    d = cuda(kda_inputs(9, B, T, 2, 4, K, V, BF16, state))
    before, few = d["state"].clone(), d["state"].clone()

    def tokens(pool, lo, hi):
        return gdn.kda_decode(*(d[n][lo:hi] for n in ("q", "k", "v", "a", "b")), d["A_log"],
                              d["dt_bias"], pool, slot_indices=d["slots"][lo:hi].contiguous())

    o = tokens(d["state"], 0, B)
    parts = torch.cat([tokens(few, lo, lo + 40) for lo in range(0, B, 40)])
    ok()
    assert torch.equal(o, parts) and torch.equal(d["state"], few)
    others = torch.ones(len(before), dtype=torch.bool, device="cuda")
    others[d["slots"].long()] = False
    assert torch.equal(d["state"][others], before[others])


# ---------------------------------------------------------------- a layer that serves

def test_a_layer_serves():
    """A KDA layer: two prompts through convolution, recurrence and gated norm into pooled
    states, then 1, 2, 4 and 1 tokens of each through the same three, against the whole in 64
    bits.  (Tokens and prompts are within 1e-5 of o's RMS; the norm divides by a head's own
    size, and where that is a thirtieth of the RMS an error is thirty times as large.)"""
    B, T, H, K, V, W = 2, 70, 2, 64, 32, 4
    g = torch.Generator().manual_seed(8)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g) * std

    D, whole = H * (2 * K + V), T + 8
    x, z, a = normal(B, whole, D), normal(B, whole, H * V), normal(B, whole, H, K)
    b, cw, nw = normal(B, whole, H), normal(D, W, std=0.5), torch.rand(V, generator=g) + 0.5
    A_log, dt_bias = torch.log(torch.rand(H, generator=g) * 15 + 1), normal(H, K) - 3
    how = dict(center=False, activation="silu")

    def heads(u):
        return (t.unflatten(2, (H, -1)) for t in u.split([H * K, H * K, H * V], 2))

    u = torch.from_numpy(M.short_conv(x, cw, None)[0])
    o, _ = L.kda_decode(*heads(u), a, b, A_log, dt_bias, torch.zeros(B, H, V, K))
    want = L.group_norm(o.reshape(B, whole, -1), H, nw, z=z, **how)

    c = [t.cuda() for t in (x, z, a, b, cw, nw, A_log, dt_bias)]
    x, z, a, b, cw, nw, A_log, dt_bias = c
    slots = torch.tensor([3, 0], dtype=torch.int32, device="cuda")
    rows, states = torch.zeros(4, W - 1, D, device="cuda"), torch.zeros(4, H, V, K, device="cuda")
    u, last = gdn.short_conv_fwd(x[:, :T], cw)
    q, k, v = (t.contiguous() for t in heads(u))
    q, k = (t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt() for t in (q, k))
    gate = -torch.exp(A_log)[:, None] * torch.nn.functional.softplus(a[:, :T] + dt_bias)
    o, ht = gdn.kda_chunk_fwd(q, k, v, gate.contiguous(), torch.sigmoid(b[:, :T]).contiguous(),
                              g_is_cumsum=False, state_v_first=True)
    rows[slots.long()], states[slots.long()] = last, ht
    got = [gdn.group_norm_fwd(o.flatten(2), H, nw, z=z[:, :T], **how)]
    at = T
    for n in (1, 2, 4, 1):
        here = slice(at, at + n)
        u = gdn.short_conv_decode(x[:, here], cw, rows, slot_indices=slots)
        o = gdn.kda_decode(*heads(u), a[:, here], b[:, here], A_log, dt_bias, states, slot_indices=slots)
        got.append(gdn.group_norm_fwd(o.flatten(2), H, nw, z=z[:, here], **how))
        at += n
    ok()
    assert_each_close(torch.cat(got, 1), want, "y", 3e-4)
    assert not states[1:3].any() and not rows[1:3].any()
