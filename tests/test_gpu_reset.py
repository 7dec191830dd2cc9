"""A plan made after cudaDeviceReset works like the first one.

The reset ends the process's own context, and with it what was set for the kernels there (their
shared memory limits).  It runs in a process of its own, which allocates with the runtime alone.
"""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
import ctypes, glob, os
import numpy as np
import torch   # (for the place of its runtime library: no CUDA call goes through it)
import mha_mla_latent_b200._lib as L

here = os.path.join(os.path.dirname(torch.__file__), "..", "nvidia", "cuda_runtime", "lib", "libcudart.so*")
rt = ctypes.CDLL(sorted(glob.glob(here))[0])
rt.cudaMalloc.argtypes = [ctypes.c_void_p, ctypes.c_size_t]
rt.cudaMemset.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t]


def dev(n):
    p = ctypes.c_void_p()
    assert rt.cudaMalloc(ctypes.byref(p), n) == 0 and rt.cudaMemset(p, 0, n) == 0
    return p.value


def calls():
    cfg = L.make_config(64, 32, 32, 128, 4, 256)
    zeros = lambda *s: np.zeros(s, dtype=np.uint16)
    pairs = np.tile(np.arange(4, dtype=np.int32), (32, 1))
    plan = L.mla_plan_create(cfg, zeros(64, 256), zeros(64, 32 * 128), pairs, zeros(32, 256, 120), zeros(32, 256, 128))
    B, T, Q = 2, 2048, 3
    cache = L.MlaCache(dev(B * T * 256 * 2), None, dev(B * T * 256 * 2), B, T)
    q, out, lens, n = dev(B * Q * 32 * 128 * 2), dev(B * Q * 32 * 128 * 2), dev(256), L.mla_decode_chunk_workspace_bytes(plan, B, Q)
    n = max(n, L.mla_decode_workspace_bytes(plan, B))
    ws, c = dev(n), ctypes.byref(cache)
    f, h = L._lib, plan.handle
    got = [f.mla_decode(h, c, lens, q, B, out, ws, n, None), f.mla_decode_window(h, c, lens, q, B, 4, 2000, out, ws, n, None),
           f.mla_decode_window(h, c, lens, q, B, 4, 8, out, ws, n, None), f.mla_decode_chunk(h, c, lens, q, B, Q, out, ws, n, None),
           f.mla_decode_chunk_window(h, c, lens, q, B, Q, 4, 100, out, ws, n, None)]
    got.append(rt.cudaDeviceSynchronize())
    plan.close()
    return got


first = calls()
assert rt.cudaDeviceReset() == 0
print("first", first, "then", calls())
"""


def test_plan_after_a_reset():
    env = dict(os.environ, PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, timeout=300, cwd=ROOT, env=env)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.strip().endswith(f"first {[0] * 6} then {[0] * 6}"), r.stdout
