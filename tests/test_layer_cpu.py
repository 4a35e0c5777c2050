"""The oracle of the delta rule's gradient, of KDA's tokens and of the norm against
differences and the recurrences it shares no code with; the C structures and the refusals of
the entry points, before any CUDA call."""
import ctypes
import os
import shutil
import subprocess
import tempfile

import numpy as np
import pytest
import torch

import gated_delta_rule_kk_gb300 as gdn
from gated_delta_rule_kk_gb300 import _lib, build_lib
from gated_delta_rule_kk_gb300._lib import (GdnChunkBwdArgs, GroupNormArgs, GroupNormBwdArgs,
                                            KdaDecodeArgs, Status)
from oracle import layer as L
from oracle import recurrence as R

from _layer import delta_inputs, kda_inputs, norm_inputs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return _lib.load()


# ---------------------------------------------------------------- the oracle

@pytest.mark.parametrize("cumsum", [False, True])
@pytest.mark.parametrize("lens", [None, [3, 0, 66]])
def test_delta_gradient_is_the_difference(cumsum, lens):
    i = delta_inputs(1, 1, 69, 4, 2, 5, 3, torch.float64, lens=lens, cumsum=cumsum)
    i = {k: v.double() if torch.is_tensor(v) and k != "cu" else v for k, v in i.items()}
    grads = L.gdn_grad(i["do"], i["q"], i["k"], i["v"], i["g"], i["beta"], i["scale"], i["h0"],
                       i["dht"], i["cu"], cumsum)

    def loss(x):
        o, ht = R.gdn_recurrent(x["q"], x["k"], x["v"], x["g"], x["beta"], i["scale"], x["h0"],
                                i["cu"], cumsum)
        return (o * i["do"].numpy()).sum() + (ht * i["dht"].numpy()).sum()

    r = np.random.default_rng(0)
    for name, grad in zip(("q", "k", "v", "g", "beta", "h0"), grads):
        d = r.standard_normal(grad.shape)
        e = 1e-6
        x = {n: i[n].numpy() for n in ("q", "k", "v", "g", "beta", "h0")}
        up, down = ({**x, name: x[name] + s * e * d} for s in (1, -1))
        # (second differences: e^2 of the third derivative, and rounding of the loss over e)
        np.testing.assert_allclose((loss(up) - loss(down)) / (2 * e), (grad * d).sum(), rtol=1e-6,
                                   atol=1e-6)


def test_kda_tokens_are_the_recurrence():
    i = kda_inputs(2, 3, 4, 2, 4, 6, 5, torch.float64, torch.float64)
    o, S = L.kda_decode(**{k: v for k, v in i.items()})
    gate = -np.exp(i["A_log"].double().numpy())[:, None] * R.softplus((i["a"] + i["dt_bias"]).numpy())
    ref, ht = R.kda_recurrent(R.l2_normalize(i["q"].numpy()), R.l2_normalize(i["k"].numpy()),
                              i["v"], gate, torch.sigmoid(i["b"]), None,
                              i["state"][i["slots"].long()].transpose(2, 3), g_is_cumsum=False)
    np.testing.assert_allclose(o, ref, atol=1e-12)
    np.testing.assert_allclose(S, ht.transpose(0, 1, 3, 2), atol=1e-12)


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("z,first", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("act", [None, "silu", "sigmoid"])
def test_norm_gradient_is_the_difference(center, z, first, act):
    i = norm_inputs(3, 2, 3, 3, 5, torch.float64, z=z)
    how = dict(eps=1e-3, center=center, activation=act, gate_first=first)
    dx, dw, db, dz = L.group_norm_grad(i["dy"], i["x"], 3, i["weight"], i["bias"], i["z"], **how)
    r = np.random.default_rng(1)
    for name, grad in (("x", dx), ("weight", dw), ("bias", db), ("z", dz)):
        if grad is None:
            continue
        d = torch.from_numpy(r.standard_normal(tuple(i[name].shape)))
        e = 1e-6
        y = [L.group_norm(**{k: v + s * e * d if k == name else v for k, v in i.items() if k != "dy"},
                          groups=3, **how) for s in (1, -1)]
        np.testing.assert_allclose(((y[0] - y[1]) * i["dy"].numpy()).sum() / (2 * e),
                                   (grad.reshape(d.shape) * d.numpy()).sum(), rtol=1e-6, atol=1e-7)


def test_norm_is_torch_group_norm():
    i = norm_inputs(4, 2, 3, 4, 6, torch.float64, z=False)
    y = L.group_norm(i["x"], 4, i["weight"], i["bias"], activation="silu")
    ref = torch.nn.functional.silu(torch.nn.functional.group_norm(
        i["x"].reshape(6, 24), 4, i["weight"], i["bias"])).reshape(2, 3, 24)
    np.testing.assert_allclose(y, ref.numpy(), atol=1e-12)


# ---------------------------------------------------------------- the C interface

STRUCTS = (("gdn_chunk_bwd_args", GdnChunkBwdArgs), ("kda_decode_args", KdaDecodeArgs),
           ("group_norm_args", GroupNormArgs), ("group_norm_bwd_args", GroupNormBwdArgs))


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_structures_match_the_header():
    lines = [f'printf("{s} size %zu\\n", sizeof({s}));' for s, _ in STRUCTS]
    lines += [f'printf("{s} {f} %zu\\n", offsetof({s}, {f}));' for s, c in STRUCTS
              for f, _ in c._fields_]
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"gdn.h\"\nint main(void) {\n" + \
        "\n".join(lines) + "\nreturn 0; }\n"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "p.c"), os.path.join(d, "p")
        open(c, "w").write(src)
        subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), c, "-o", exe])
        got = {tuple(ln.split()[:2]): int(ln.split()[2])
               for ln in subprocess.check_output([exe], text=True).splitlines()}
    for s, c in STRUCTS:
        assert got[(s, "size")] == ctypes.sizeof(c), s
        for f, _ in c._fields_:
            assert got[(s, f)] == getattr(c, f).offset, (s, f)


def delta_args(**kw):
    a = dict(dtype=1, **{n: FAKE for n in ("q", "k", "v", "g", "beta", "do_", "dq", "dk", "dv", "dg",
                                           "dbeta")},
             B=2, T=128, H=4, Hg=2, K=128, V=128, N=2, chunk_size=64)
    return GdnChunkBwdArgs(**{**a, **kw})


@pytest.mark.parametrize("change,expect", [
    (dict(q=None), Status.INVALID_ARG), (dict(do_=None), Status.INVALID_ARG),
    (dict(dbeta=None), Status.INVALID_ARG), (dict(dq=FAKE + 2), Status.MISALIGNED),
    (dict(h0=FAKE + 4), Status.MISALIGNED), (dict(dht=FAKE + 8), Status.MISALIGNED),
    (dict(dtype=2), Status.INVALID_ARG), (dict(T=-1), Status.INVALID_ARG),
    (dict(H=3), Status.UNSUPPORTED), (dict(K=129), Status.UNSUPPORTED),
    (dict(V=(1 << 20) + 1), Status.UNSUPPORTED), (dict(H=65536), Status.UNSUPPORTED),
    (dict(N=65536), Status.UNSUPPORTED), (dict(chunk_size=32), Status.UNSUPPORTED),
    (dict(N=1), Status.INVALID_ARG), (dict(cu_seqlens=FAKE), Status.INVALID_ARG),
    (dict(g_is_cumsum=2), Status.INVALID_ARG), (dict(state_v_first=-1), Status.INVALID_ARG),
    (dict(scale=float("nan")), Status.INVALID_ARG), (dict(T=0x7fffffff), Status.UNSUPPORTED),
    (dict(B=65535, N=65535, T=0x7fffff00), Status.UNSUPPORTED),
    (dict(), Status.WORKSPACE), (dict(dtype=0), Status.WORKSPACE),
    (dict(workspace=FAKE, workspace_bytes=1 << 20), Status.WORKSPACE),
    (dict(workspace=FAKE + 16, workspace_bytes=1 << 40), Status.MISALIGNED),
])
def test_delta_gradient_refusals(lib, change, expect):
    a = delta_args(**change)
    assert lib.gdn_chunk_bwd(ctypes.byref(a), None) == expect
    assert lib.gdn_last_error_message()
    assert lib.gdn_chunk_bwd(None, None) == Status.INVALID_ARG


def test_delta_gradient_workspace(lib):
    n = ctypes.c_size_t(9)

    def need(**kw):
        a = delta_args(**{"Hg": 4, **kw})
        assert lib.gdn_chunk_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n)) == Status.OK
        return n.value

    square, rows, state = 4 * 64 * 64, 4 * 64 * 128, 4 * 128 * 128
    block = 1024 + 3 * square + 2 * (rows + state)
    assert need() == 2 * 2 * 4 * block
    assert need(T=0) == 0
    assert need(T=1) == 2 * 4 * block
    # packed: at most one more chunk than the whole chunks of the tokens, a sequence
    assert need(B=1, N=5, T=128, cu_seqlens=FAKE) == 256 + (5 + 2) * 4 * block
    # in float32 once, not as pieces and images: gates, T, P, n, dr, h, D
    assert need(dtype=0) == 2 * 2 * 4 * 4 * (2 * 64 + 2 * 64 * 64 + 2 * 64 * 128 + 2 * 128 * 128)
    # heads that share a key head: sums of dq and dk for every block of the last kernel
    assert need(Hg=2) == 2 * 2 * 4 * block + 2 * 2 * 2 * 2 * 64 * 128 * 4
    big = need(B=1, N=1, T=1 << 24)
    assert big == (1 << 18) * 4 * block  # beyond 32 bits
    a = delta_args(H=3)
    assert lib.gdn_chunk_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n)) == Status.UNSUPPORTED


def kda_args(**kw):
    a = dict(dtype=1, state_dtype=1, q=FAKE, k=FAKE, v=FAKE, a=FAKE, b=FAKE, A_log=FAKE,
             dt_bias=FAKE, state=FAKE, o=FAKE, B=2, T=2, H=2, HV=4, K=128, V=64, pool=4)
    for t, row in (("q", 256), ("k", 256), ("v", 256), ("a", 512), ("b", 4), ("o", 256)):
        a[t + "_stride"], a[t + "_batch_stride"] = row, 2 * row
    return KdaDecodeArgs(**{**a, **kw})


@pytest.mark.parametrize("change,expect", [
    (dict(q=None), Status.INVALID_ARG), (dict(a=FAKE + 1), Status.MISALIGNED),
    (dict(state=FAKE + 8), Status.MISALIGNED), (dict(dt_bias=FAKE + 4), Status.MISALIGNED),
    (dict(A_log=None), Status.INVALID_ARG), (dict(dtype=5), Status.INVALID_ARG),
    (dict(state_dtype=2), Status.INVALID_ARG), (dict(T=0), Status.UNSUPPORTED),
    (dict(T=5), Status.UNSUPPORTED), (dict(HV=3), Status.UNSUPPORTED), (dict(K=100), Status.UNSUPPORTED),
    (dict(K=264), Status.UNSUPPORTED), (dict(pool=0), Status.INVALID_ARG),
    (dict(pool=1), Status.INVALID_ARG), (dict(q_stride=255), Status.INVALID_ARG),
    (dict(a_stride=511), Status.INVALID_ARG), (dict(use_qk_l2norm=2), Status.INVALID_ARG),
    (dict(scale=float("inf")), Status.INVALID_ARG), (dict(V=0x7fffffff), Status.UNSUPPORTED),
    (dict(B=1 << 30, pool=1 << 30), Status.UNSUPPORTED), (dict(slot_indices=FAKE + 4), Status.MISALIGNED),
])
def test_kda_token_refusals(lib, change, expect):
    a = kda_args(**change)
    assert lib.kda_decode(ctypes.byref(a), None) == expect
    assert lib.gdn_last_error_message()
    assert lib.kda_decode(None, None) == Status.INVALID_ARG


NORM = dict(dtype=1, weight_dtype=1, x=FAKE, weight=FAKE, bias=FAKE, B=2, T=4, D=64, groups=4,
            eps=1e-5, activation=1)
NORM_CHANGES = [
    (dict(x=None), Status.INVALID_ARG), (dict(x=FAKE + 1), Status.MISALIGNED),
    (dict(dtype=2), Status.INVALID_ARG), (dict(dtype=0), Status.INVALID_ARG),
    (dict(groups=0), Status.INVALID_ARG), (dict(groups=5), Status.INVALID_ARG),
    (dict(D=8193, groups=1, x_stride=8193), Status.UNSUPPORTED),
    (dict(D=1 << 29, groups=1 << 20, x_stride=1 << 29), Status.UNSUPPORTED),
    (dict(B=1 << 15, T=1 << 16), Status.UNSUPPORTED), (dict(x_stride=63), Status.INVALID_ARG),
    (dict(center=2), Status.INVALID_ARG), (dict(shared_weight=3), Status.INVALID_ARG),
    (dict(activation=3), Status.INVALID_ARG), (dict(activation=-1), Status.INVALID_ARG),
    (dict(eps=-1.0), Status.INVALID_ARG), (dict(eps=float("nan")), Status.INVALID_ARG),
    (dict(gate_first=1), Status.INVALID_ARG),
]


@pytest.mark.parametrize("change,expect", NORM_CHANGES + [
    (dict(y=None), Status.INVALID_ARG), (dict(y_stride=1), Status.INVALID_ARG)])
def test_norm_refusals(lib, change, expect):
    a = GroupNormArgs(**{**NORM, "y": FAKE, "x_stride": 64, "y_stride": 64, "x_batch_stride": 256,
                         "y_batch_stride": 256, **change})
    assert lib.group_norm_fwd(ctypes.byref(a), None) == expect
    assert lib.gdn_last_error_message()
    assert lib.group_norm_fwd(None, None) == Status.INVALID_ARG


@pytest.mark.parametrize("change,expect", NORM_CHANGES + [
    (dict(dy=None), Status.INVALID_ARG), (dict(dx=None), Status.INVALID_ARG),
    (dict(dz=FAKE), Status.INVALID_ARG), (dict(z=FAKE, z_stride=64, dz_stride=64), Status.INVALID_ARG),
    (dict(weight=None), Status.INVALID_ARG), (dict(bias=None), Status.INVALID_ARG),
    (dict(dy_stride=3), Status.INVALID_ARG), (dict(), Status.WORKSPACE)])
def test_norm_gradient_refusals(lib, change, expect):
    a = {**NORM, "dy": FAKE, "dx": FAKE, "dweight": FAKE, "dbias": FAKE}
    for t in ("dy", "x", "dx"):
        a[t + "_stride"], a[t + "_batch_stride"] = 64, 256
    a = GroupNormBwdArgs(**{**a, **change})
    assert lib.group_norm_bwd(ctypes.byref(a), None) == expect
    assert lib.gdn_last_error_message()
    assert lib.group_norm_bwd(None, None) == Status.INVALID_ARG


def test_norm_gradient_workspace(lib):
    n = ctypes.c_size_t(9)
    a = GroupNormBwdArgs(**{**NORM, "dy": FAKE, "dx": FAKE, "dweight": FAKE, "x_stride": 64,
                            "dy_stride": 64, "dx_stride": 64})
    assert lib.group_norm_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n)) == Status.OK
    assert n.value >= 2 * 64 * 4
    a.dweight = None
    assert lib.group_norm_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n)) == Status.OK
    assert n.value == 0
    assert lib.group_norm_bwd_workspace_size(None, ctypes.byref(n)) == Status.INVALID_ARG


def test_python_refuses_what_is_not_on_the_gpu():
    x = torch.zeros(1, 2, 8)
    q = torch.zeros(1, 2, 1, 8)
    with pytest.raises(ValueError):
        gdn.group_norm_fwd(x, 2)
    with pytest.raises(ValueError):
        gdn.group_norm_bwd(x, x, 2)
    with pytest.raises(ValueError):
        gdn.gdn_chunk_bwd(q, q, q, q, q[..., 0], q[..., 0])
    with pytest.raises(ValueError):
        gdn.kda_decode(q, q, q, q, q[..., 0], x[0, 0], None, q)
