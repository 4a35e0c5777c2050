"""The short convolution and the state space scan without a GPU: the oracle
against closed forms and differences, the C structures and the refusals that
are found on the host."""
import ctypes
import os
import shutil
import subprocess
import tempfile

import numpy as np
import pytest

from gated_delta_rule_kk_gb300 import _lib, build_lib
from gated_delta_rule_kk_gb300._lib import (ShortConvArgs, ShortConvBwdArgs, ShortConvDecodeArgs,
                                            SsmChunkArgs, SsmDecodeArgs, Status)
from oracle import mixer as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return _lib.load()


# ---------------------------------------------------------------- the oracle

def conv_case(seed=0, lens=(4, 0, 1, 6), D=3, W=4):
    r = np.random.default_rng(seed)
    T, N = sum(lens), len(lens)
    return dict(x=r.normal(size=(1, T, D)), weight=r.normal(size=(D, W)), bias=r.normal(size=D),
                h0=r.normal(size=(N, W - 1, D)), cu_seqlens=[0, *np.cumsum(lens)])


def test_convolution_is_a_convolution():
    c = conv_case()
    y, ht = M.short_conv(**c, silu=False)
    for n, (lo, hi) in enumerate(zip(c["cu_seqlens"], c["cu_seqlens"][1:])):
        rows = np.concatenate([c["h0"][n], c["x"][0, lo:hi]])
        for d in range(3):
            if hi > lo:
                full = np.convolve(rows[:, d], c["weight"][d][::-1], "valid") + c["bias"][d]
                np.testing.assert_allclose(y[0, lo:hi, d], full, atol=1e-12)
        np.testing.assert_array_equal(ht[n], rows[-3:])


@pytest.mark.parametrize("silu", [True, False])
def test_convolution_gradient_against_differences(silu):
    c = conv_case(1)
    r = np.random.default_rng(2)
    dy, dht = r.normal(size=c["x"].shape), r.normal(size=c["h0"].shape)

    def loss(**change):
        y, ht = M.short_conv(**{**c, **change}, silu=silu)
        return np.sum(y * dy) + np.sum(ht * dht)

    grads = dict(zip(("x", "weight", "bias", "h0"),
                     M.short_conv_grad(dy, c["x"], c["weight"], c["bias"], c["h0"], dht,
                                       c["cu_seqlens"], silu)))
    for name, g in grads.items():
        way = r.normal(size=c[name].shape)
        diff = (loss(**{name: c[name] + 1e-5 * way}) - loss(**{name: c[name] - 1e-5 * way})) / 2e-5
        assert abs(diff - np.sum(g * way)) < 1e-7 * max(1, abs(diff)), name


def scan_case(seed=0, T=7, H=4, Hg=2, V=3, K=5):
    r = np.random.default_rng(seed)
    return dict(x=r.normal(size=(1, T, H, V)), dt=r.normal(size=(1, T, H)), A_log=r.normal(size=H),
                Bm=r.normal(size=(1, T, Hg, K)), Cm=r.normal(size=(1, T, Hg, K)),
                D=r.normal(size=H), z=r.normal(size=(1, T, H, V)), dt_bias=r.normal(size=H),
                h0=r.normal(size=(1, H, V, K)))


def test_scan_is_the_sum_over_earlier_tokens():
    c = scan_case()
    y, ht = M.ssm_scan(**c)
    s = np.log1p(np.exp(c["dt"] + c["dt_bias"]))[0]
    G = np.cumsum(-np.exp(c["A_log"]) * s, 0)
    for h in range(4):
        B, C = c["Bm"][0, :, h // 2], c["Cm"][0, :, h // 2]
        for t in range(7):
            want = np.exp(G[t, h]) * c["h0"][0, h] @ C[t] + c["D"][h] * c["x"][0, t, h]
            for r in range(t + 1):
                want = want + np.exp(G[t, h] - G[r, h]) * (B[r] @ C[t]) * s[r, h] * c["x"][0, r, h]
            z = c["z"][0, t, h]
            np.testing.assert_allclose(y[0, t, h], want * z / (1 + np.exp(-z)), atol=1e-12)


def test_scan_resumes_and_packs():
    c = scan_case(3)
    y, ht = M.ssm_scan(**c)
    cut = {k: (v[:, :4], v[:, 4:]) if k in ("x", "dt", "Bm", "Cm", "z") else (v, v)
           for k, v in c.items()}
    ya, ha = M.ssm_scan(**{k: v[0] for k, v in cut.items()})
    yb, hb = M.ssm_scan(**{**{k: v[1] for k, v in cut.items()}, "h0": ha})
    np.testing.assert_allclose(np.concatenate([ya, yb], 1), y, atol=1e-12)
    np.testing.assert_allclose(hb, ht, atol=1e-12)
    packed = {**c, "h0": np.concatenate([c["h0"], 0 * c["h0"], ha])}
    yp, hp = M.ssm_scan(**packed, cu_seqlens=[0, 4, 4, 7])
    np.testing.assert_allclose(yp, y, atol=1e-12)
    np.testing.assert_allclose(hp[2], ht[0], atol=1e-12)
    assert not hp[1].any()


# ---------------------------------------------------------------- the C interface

STRUCTS = (("short_conv_args", ShortConvArgs), ("short_conv_bwd_args", ShortConvBwdArgs),
           ("short_conv_decode_args", ShortConvDecodeArgs), ("ssm_chunk_args", SsmChunkArgs),
           ("ssm_decode_args", SsmDecodeArgs))


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


def conv_args(**kw):
    a = dict(dtype=1, weight_dtype=1, x=FAKE, weight=FAKE, y=FAKE, x_stride=64, x_batch_stride=512,
             y_stride=64, y_batch_stride=512, B=2, T=8, D=64, W=4, N=2, silu=1)
    return ShortConvArgs(**{**a, **kw})


@pytest.mark.parametrize("change,expect", [
    (dict(x=None), Status.INVALID_ARG), (dict(y=FAKE + 1), Status.MISALIGNED),
    (dict(weight=FAKE + 2), Status.MISALIGNED),
    (dict(W=1), Status.UNSUPPORTED), (dict(W=5), Status.UNSUPPORTED),
    (dict(dtype=3), Status.INVALID_ARG), (dict(dtype=0), Status.INVALID_ARG),
    (dict(x_stride=63), Status.INVALID_ARG), (dict(N=3), Status.INVALID_ARG),
    (dict(cu_seqlens=FAKE), Status.INVALID_ARG), (dict(silu=2), Status.INVALID_ARG),
    (dict(D=0), Status.INVALID_ARG), (dict(weight=None), Status.INVALID_ARG),
])
def test_convolution_refusals(lib, change, expect):
    a = conv_args(**change)
    assert lib.short_conv_fwd(ctypes.byref(a), None) == expect
    assert lib.gdn_last_error_message()
    assert lib.short_conv_fwd(None, None) == Status.INVALID_ARG


def test_gradient_needs_its_workspace(lib):
    a = ShortConvBwdArgs(dtype=1, weight_dtype=1, dy=FAKE, x=FAKE, weight=FAKE, dx=FAKE,
                         dweight=FAKE, dy_stride=64, x_stride=64, dx_stride=64, dy_batch_stride=512,
                         x_batch_stride=512, dx_batch_stride=512, B=2, T=8, D=64, W=4, N=2)
    n = ctypes.c_size_t(0)
    assert lib.short_conv_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n)) == Status.OK
    assert n.value >= 5 * 64 * 4
    assert lib.short_conv_bwd(ctypes.byref(a), None) == Status.WORKSPACE
    a.dweight = None
    assert lib.short_conv_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n)) == Status.OK
    assert n.value == 0
    a.W = 9
    assert lib.short_conv_bwd(ctypes.byref(a), None) == Status.UNSUPPORTED


@pytest.mark.parametrize("change,expect", [
    (dict(T=0), Status.UNSUPPORTED), (dict(T=5), Status.UNSUPPORTED),
    (dict(pool=1), Status.INVALID_ARG), (dict(state=None), Status.INVALID_ARG),
])
def test_token_convolution_refusals(lib, change, expect):
    a = dict(dtype=1, weight_dtype=1, x=FAKE, weight=FAKE, state=FAKE, y=FAKE, x_stride=64,
             x_batch_stride=64, y_stride=64, y_batch_stride=64, B=2, T=1, D=64, W=4, pool=4)
    a = ShortConvDecodeArgs(**{**a, **change})
    assert lib.short_conv_decode(ctypes.byref(a), None) == expect


def scan_args(cls, **kw):
    a = dict(dtype=1, dt_dtype=1, x=FAKE, Bm=FAKE, Cm=FAKE, dt=FAKE, A_log=FAKE, y=FAKE, B=2, T=3,
             H=4, Hg=2, K=128, V=64)
    for t, row in (("x", 256), ("z", 256), ("Bm", 256), ("Cm", 256), ("dt", 8), ("y", 256)):
        a[t + "_stride"], a[t + "_batch_stride"] = row, 3 * row
    a.update(dict(N=2) if cls is SsmChunkArgs else dict(state_dtype=1, state=FAKE, pool=4))
    return cls(**{**a, **kw})


@pytest.mark.parametrize("change,expect", [
    (dict(x=None), Status.INVALID_ARG), (dict(Bm=FAKE + 1), Status.MISALIGNED),
    (dict(dt=FAKE + 1), Status.MISALIGNED), (dict(H=3), Status.UNSUPPORTED),
    (dict(K=257), Status.UNSUPPORTED), (dict(x_stride=255), Status.INVALID_ARG),
    (dict(dt_softplus=2), Status.INVALID_ARG), (dict(N=1), Status.INVALID_ARG),
    (dict(segment_tokens=64), Status.INVALID_ARG), (dict(A_log=None), Status.INVALID_ARG),
    (dict(T=300, segment_tokens=128), Status.WORKSPACE),
])
def test_scan_refusals(lib, change, expect):
    a = scan_args(SsmChunkArgs, **change)
    assert lib.ssm_chunk_fwd(ctypes.byref(a), None) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(K=100), Status.UNSUPPORTED), (dict(T=5), Status.UNSUPPORTED),
    (dict(state_dtype=4), Status.INVALID_ARG), (dict(pool=0), Status.INVALID_ARG),
    (dict(slot_indices=FAKE + 4), Status.MISALIGNED),
])
def test_token_scan_refusals(lib, change, expect):
    a = scan_args(SsmDecodeArgs, **change)
    assert lib.ssm_decode(ctypes.byref(a), None) == expect


def test_scan_workspace_holds_the_segments(lib):
    n = ctypes.c_size_t(9)
    a = scan_args(SsmChunkArgs, T=128, segment_tokens=128)
    assert lib.ssm_chunk_workspace_size(ctypes.byref(a), ctypes.byref(n)) == Status.OK
    assert n.value == 0
    a = scan_args(SsmChunkArgs, T=300, segment_tokens=128)  # 3 segments of 2 sequences
    assert lib.ssm_chunk_workspace_size(ctypes.byref(a), ctypes.byref(n)) == Status.OK
    assert n.value == 6 * 4 * (64 * 128 + 1) * 4
    # packed: at most one more than the whole segments of the tokens, a sequence
    a = scan_args(SsmChunkArgs, B=1, N=5, T=300, segment_tokens=128, cu_seqlens=FAKE)
    assert lib.ssm_chunk_workspace_size(ctypes.byref(a), ctypes.byref(n)) == Status.OK
    assert n.value == (5 + 2) * 4 * (64 * 128 + 1) * 4
