"""Edges of the short convolution and the state space scan that the host decides, without a GPU."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from gated_delta_rule_kk_gb300 import _lib, api_ssm, build_lib
from gated_delta_rule_kk_gb300._lib import ShortConvBwdArgs, SsmChunkArgs, SsmDecodeArgs, Status
from oracle import mixer as M

from _mixer import scan_rooms, ssm_inputs
from test_mixer_cpu import FAKE, conv_args, scan_args

TESTS = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return _lib.load()


def in_a_process(body):
    """Runs `body` with the library loaded, apart from this process: a fault of the host's
    arithmetic would end it."""
    head = f"import sys\nsys.path[:0] = [{os.path.dirname(TESTS)!r}, {TESTS!r}]\n" \
        "import ctypes\nfrom gated_delta_rule_kk_gb300 import _lib\n" \
        "from gated_delta_rule_kk_gb300._lib import *\n" \
        "from test_mixer_cpu import FAKE, conv_args, scan_args\nlib = _lib.load()\n"
    r = subprocess.run([sys.executable, "-c", head + body], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout + r.stderr)


# no tokens; packed prompts of which most are empty (the mean length rounds to zero)
@pytest.mark.parametrize("T,N,packed", [(0, 2, False), (0, 1, True), (0, 9, True), (1, 2, True),
                                        (1, 4, True), (3, 10, True), (16, 25, True)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_scan_of_fewer_tokens_than_sequences(lib, T, N, packed, dtype):
    """Nothing is cut into segments: no workspace, and no division by a length of zero."""
    in_a_process(f"""
a = scan_args(SsmChunkArgs, dtype={dtype}, dt_dtype={dtype}, T={T}, N={N},
              B={1 if packed else N}, cu_seqlens={FAKE if packed else None})
n = ctypes.c_size_t(9)
assert lib.ssm_chunk_workspace_size(ctypes.byref(a), ctypes.byref(n)) == Status.OK
assert n.value == 0
""")


@pytest.mark.parametrize("dtype", [0, 1])
def test_convolution_without_tokens(lib, dtype):
    """Without a state to return there is nothing to launch; with one, the launch's shape
    (formed before the device is asked for) has no length of zero to divide by."""
    in_a_process(f"""
a = conv_args(dtype={dtype}, weight_dtype={dtype}, T=0, x=None, y=None)
assert lib.short_conv_fwd(ctypes.byref(a), None) == Status.OK
a = conv_args(dtype={dtype}, weight_dtype={dtype}, T=0, B=1, N=3, cu_seqlens=FAKE)
assert lib.short_conv_fwd(ctypes.byref(a), None) == Status.OK
import torch
if not torch.cuda.is_available():
    a = conv_args(dtype={dtype}, weight_dtype={dtype}, T=0, ht=FAKE)
    assert lib.short_conv_fwd(ctypes.byref(a), None) == Status.CUDA
""")


def pieces(v, n):
    """The sum of v's first n bfloat16 pieces, each the nearest to what is left."""
    v = torch.from_numpy(np.asarray(v))
    total = torch.zeros_like(v)
    for _ in range(n):
        total = total + (v - total).to(torch.bfloat16).double()
    return total.numpy()


def chunked_scan(i, of_m, of_h):
    """y in 128-token chunks with M and h in so many bfloat16 pieces, all else exact."""
    x, Bm, Cm, dt, A_log, bias, D, z, h0 = (
        None if i[k] is None else i[k].double().numpy()
        for k in ("x", "Bm", "Cm", "dt", "A_log", "dt_bias", "D", "z", "h0"))
    H = x.shape[2]
    head = np.arange(H) // (H // Bm.shape[2])
    s = M.softplus(dt + bias)
    y = np.zeros_like(x)
    for n, (b, lo, hi) in enumerate(M.bounds(x.shape[0], x.shape[1], i["cu"])):
        h = h0[n].copy()
        for t in range(lo, hi, 128):
            e = min(t + 128, hi)
            for k in range(H):
                G = np.cumsum(-np.exp(A_log[k]) * s[b, t:e, k])
                L = np.tril(np.exp(np.minimum(G[:, None] - G[None], 0)))
                B, C, X = Bm[b, t:e, head[k]], Cm[b, t:e, head[k]], x[b, t:e, k]
                m = C @ B.T * L * s[b, t:e, k] + D[k] * np.eye(e - t)
                y[b, t:e, k] = np.exp(G)[:, None] * (C @ pieces(h[k], of_h).T) + pieces(m, of_m) @ X
                w = (s[b, t:e, k] * np.exp(G[-1] - G))[:, None] * X
                h[k] = np.exp(G[-1]) * h[k] + w.T @ B
    return y * z * M.sigmoid(z)


@pytest.mark.parametrize("T,lens", [(1, None), (129, None), (300, [0, 1, 130, 0, 41, 128, 0])])
def test_the_scan_bound_sees_a_lost_piece(T, lens):
    """What y may be off by on the tensor cores (test_mixer_edges_gpu.py) holds for two pieces of
    M and h, and for neither of them with one."""
    i = ssm_inputs(41, 1, T, 2, 1, 64, 128, torch.bfloat16, lens)
    ref, _ = M.ssm_scan(i["x"], i["dt"], i["A_log"], i["Bm"], i["Cm"], i["D"], i["z"], i["dt_bias"],
                        h0=i["h0"], cu_seqlens=i["cu"])
    room = scan_rooms(i)
    worst = {k: np.max(np.abs(chunked_scan(i, *k) - ref) / room) for k in ((2, 2), (1, 2), (2, 1))}
    assert worst[2, 2] < 1 < min(worst[1, 2], worst[2, 1]), worst


class Devices:
    """Two GPUs of which the first is current, and a library that notes where it was called."""

    def __init__(self, monkeypatch):
        self.current, self.calls = 0, []
        devices = self

        class Device:
            def __init__(self, device):
                self.to = torch.device(device).index

            def __enter__(self):
                self.back, devices.current = devices.current, self.to

            def __exit__(self, *exc):
                devices.current = self.back

        class Library:
            def __getattr__(self, name):
                return lambda *args: devices.calls.append((name, devices.current, args)) or 0

        monkeypatch.setattr(api_ssm, "_current_device", lambda: self.current, raising=False)
        monkeypatch.setattr(torch.cuda, "device", Device)
        monkeypatch.setattr(api_ssm, "_raw_stream", lambda index: 0x1000 + index)
        monkeypatch.setattr(_lib, "_lib", Library())


@pytest.mark.parametrize("index", [0, 1])
def test_calls_run_on_the_device_of_their_tensors(monkeypatch, index):
    """The library launches, counts SMs and records errors on the current device: it has to be
    the tensors', whichever was current before."""
    devices = Devices(monkeypatch)
    device, args = torch.device("cuda", index), ShortConvBwdArgs()
    api_ssm._call("short_conv_bwd", args, None, device)
    assert api_ssm._workspace(args, "short_conv_bwd_workspace_size", None, device, None) is None
    assert [c[:2] for c in devices.calls] == [("short_conv_bwd", index),
                                              ("short_conv_bwd_workspace_size", index)]
    assert devices.calls[0][2][1] == 0x1000 + index  # that device's stream
    assert devices.current == 0


def test_a_stream_of_another_device_is_refused(monkeypatch):
    devices = Devices(monkeypatch)

    class Stream:
        device, cuda_stream = torch.device("cuda:0"), 7

    api_ssm._call("ssm_decode", SsmDecodeArgs(), Stream(), torch.device("cuda:0"))
    with pytest.raises(ValueError, match="stream"):
        api_ssm._call("ssm_decode", SsmDecodeArgs(), Stream(), torch.device("cuda:1"))
    assert len(devices.calls) == 1


MOST = 0x7fffff00  # tokens of a batch row


def bwd_args(**kw):
    a = dict(dtype=1, weight_dtype=1, dy=FAKE, x=FAKE, weight=FAKE, dx=FAKE, dweight=FAKE,
             dy_stride=1, x_stride=1, dx_stride=1, B=1, T=8, D=1, W=4, N=1)
    return ShortConvBwdArgs(**{**a, **kw})


def workspace(lib, name, args):
    n = ctypes.c_size_t(0)
    status = getattr(lib, name + "_workspace_size")(ctypes.byref(args), ctypes.byref(n))
    return status, n.value


@pytest.mark.parametrize("T", [2 ** 31 - 2 ** 20, MOST])
def test_shapes_of_the_longest_calls(lib, T):
    """The sums behind runs and segments do not pass 31 bits."""
    status, n = workspace(lib, "short_conv_bwd", bwd_args(T=T))
    assert status == Status.OK
    # a block's partial sums cover eight runs; runs are as long as 152 SMs of 256 threads want
    run = -(-T // (152 * 256))
    run += -run % 4
    assert n == -(-T // (8 * run)) * 5 * 4
    a = dict(T=T, H=1, Hg=1, V=8, K=8, B=1, N=1)
    status, n = workspace(lib, "ssm_chunk", scan_args(SsmChunkArgs, **a, segment_tokens=128))
    assert (status, n) == (Status.OK, -(-T // 128) * (8 * 8 + 1) * 4)
    status, n = workspace(lib, "ssm_chunk", scan_args(SsmChunkArgs, **a))
    assert status == Status.OK and n >= 2 * (8 * 8 + 1) * 4  # few heads: cut into segments


def test_longer_calls_are_refused(lib):
    assert workspace(lib, "short_conv_bwd", bwd_args(T=MOST + 1))[0] == Status.UNSUPPORTED
    a = bwd_args(T=MOST + 1)
    assert lib.short_conv_bwd(ctypes.byref(a), None) == Status.UNSUPPORTED
    a = conv_args(B=1, N=1, T=MOST + 1)
    assert lib.short_conv_fwd(ctypes.byref(a), None) == Status.UNSUPPORTED
    a = scan_args(SsmChunkArgs, B=1, N=1, T=MOST + 1)
    assert workspace(lib, "ssm_chunk", a)[0] == Status.UNSUPPORTED
    assert lib.ssm_chunk_fwd(ctypes.byref(a), None) == Status.UNSUPPORTED
    # more segments than one launch counts
    a = scan_args(SsmChunkArgs, B=65535, N=65535, T=MOST, segment_tokens=128)
    assert workspace(lib, "ssm_chunk", a)[0] == Status.UNSUPPORTED
    assert lib.ssm_chunk_fwd(ctypes.byref(a), None) == Status.UNSUPPORTED


@pytest.mark.parametrize("cls,name", [(SsmChunkArgs, "ssm_chunk_fwd"), (SsmDecodeArgs, "ssm_decode")])
def test_heads_of_more_rows_than_a_launch_counts_are_refused(lib, cls, name):
    a = scan_args(cls, V=2 ** 31 - 1, H=1, Hg=1, T=1,
                  **{t + "_stride": 2 ** 31 for t in ("x", "z", "y")})
    assert getattr(lib, name)(ctypes.byref(a), None) == Status.UNSUPPORTED
