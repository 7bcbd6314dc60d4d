"""The C ABI before and after cudaDeviceReset, which ends the process's context and begins another: in a process of its own,
without torch's use of the GPU."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

CHILD = r"""
import numpy as np
from cuda.bindings import runtime as cu
import exact_io_aware_75_b200 as fa


def ok(r):
    assert r[0] == cu.cudaError_t.cudaSuccess, r
    return r[1] if len(r) > 1 else None


def put(a):
    p = ok(cu.cudaMalloc(max(a.nbytes, 256)))
    ok(cu.cudaMemcpy(p, a.ctypes.data, a.nbytes, cu.cudaMemcpyKind.cudaMemcpyHostToDevice))
    return p


def calls(d):
    # one token whose value is 1: O = 1
    lib, one = fa.library(), np.full((1, 16, 1, d), 0x3f80, dtype=np.uint16)
    q, kv, o = put(one[0, :1]), put(one), put(np.zeros(d, np.uint16))
    table, lens = put(np.zeros(1, np.int32)), put(np.ones(1, np.int32))
    need = max(fa.decode_shared_workspace_bytes(1, 1, 1, d), fa.decode_cross_workspace_bytes(1, 1, 1, 1, d))
    ws = ok(cu.cudaMalloc(need))
    for call in (lambda: lib.fa_decode_shared(q, kv, kv, table, lens, None, None, o, None, None, 1, 0, 1, 1, 1, d, 16, 1, 0.1, ws,
                                              need, None),
                 lambda: lib.fa_decode_cross(q, kv, kv, lens, o, None, 1, 1, 1, 1, 16, d, 0.1, ws, need, None)):
        ok(cu.cudaMemset(o, 0, 2 * d))
        assert call() == 0
        assert fa.check_device_error_without_torch() == 0
        got = np.zeros(d, np.uint16)
        ok(cu.cudaMemcpy(got.ctypes.data, o, 2 * d, cu.cudaMemcpyKind.cudaMemcpyDeviceToHost))
        assert (got == 0x3f80).all(), got


fa.check_device_error_without_torch = lambda: fa.library().fa_check_device_error(None)
for turn in range(3):
    calls(64)
    calls(128)
    ok(cu.cudaDeviceReset())
print("three contexts")
"""


def test_decode_in_a_new_context():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", CHILD], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "three contexts" in run.stdout, run.stdout + run.stderr
