"""Edges of the short convolution and the state space scan that the host decides, without a GPU."""
import ctypes
import os
import subprocess
import sys

import pytest

from gated_delta_rule_kk_gb300 import _lib, build_lib

from test_mixer_cpu import FAKE

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
