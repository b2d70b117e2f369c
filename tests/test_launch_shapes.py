"""Launch shapes the library's host side chooses, seen through a stand-in for the CUDA runtime
(fake_cudart.c, preloaded into a process of its own): no GPU, nothing runs."""
from __future__ import annotations

import json
import os
import subprocess
import sys
import textwrap

import pytest

from fp8_quant_row_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))

PRELUDE = """
import ctypes, json, sys
L, F = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(sys.argv[2])
class Launch(ctypes.Structure):
    _fields_ = [("fn", ctypes.c_void_p), ("grid", ctypes.c_uint), ("block", ctypes.c_uint),
                ("cluster", ctypes.c_uint), ("smem", ctypes.c_ulong)]
F.fake_launch_at.restype = Launch
P, I64 = ctypes.c_void_p, ctypes.c_int64
G = [P((1 + i) << 40) for i in range(8)]  # addresses that nothing reads
def rms(rows, cols, residual=False, e4m3=0):
    return L.fp8q_rms_norm_quant(G[0] if residual else None, G[1], G[2], G[3],
                                 G[4] if residual else None, G[5], e4m3, I64(rows), I64(cols),
                                 ctypes.c_float(1e-6), None)
def silu(rows, cols, e4m3=0):
    return L.fp8q_silu_mul_quant(G[0], G[1], G[2], G[3], I64(cols), e4m3, I64(rows), I64(cols), None)
def last():
    l = F.fake_launch_at(F.fake_launches() - 1)
    return [l.grid, l.block, l.cluster, l.smem]
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("fake") / "fake_cudart.so")
    subprocess.run([os.environ.get("CC", "gcc"), "-O1", "-fPIC", "-shared", "-Wall", "-Werror",
                    f"-I{_build.CUDA_HOME}/include", os.path.join(HERE, "fake_cudart.c"), "-o", so],
                   check=True)
    lib = _build.build()

    def run(code):
        out = subprocess.run([sys.executable, "-c", PRELUDE + textwrap.dedent(code), lib, so],
                             env={**os.environ, "LD_PRELOAD": so}, capture_output=True, text=True,
                             timeout=120)
        assert out.returncode == 0, out.stderr[-2000:]
        return json.loads(out.stdout)

    return run


@pytest.mark.parametrize("op", ["rms", "silu"])
def test_a_grid_does_not_depend_on_earlier_widths(fake, op):
    """Widths that share a register kernel but not its threads per CTA: each grid is the one of the
    CTAs that are resident at that width, whichever came first."""
    code = f"""
    got = {{}}
    for cols in %s:
        assert {op}(4608, cols) == 0
        got[cols] = last()
    print(json.dumps(got))
    """
    widths = [768, 1536, 6144, 1024, 2048, 4096, 8192] if op == "rms" else [768, 1536, 6144, 512, 4096]
    up, down = fake(code % widths), fake(code % widths[::-1])
    assert up == down
    for cols, (grid, block, _, smem) in up.items():
        if smem:
            continue  # (rows kept in shared memory)
        rows_cta = 4 if block == 128 and int(cols) <= (1024 if op == "rms" else 768) else 1
        resident = min(2048 // block, 65536 // (128 * block), 32)
        assert grid == min(-(-4608 // rows_cta), 152 * resident), (cols, grid, block)


def test_launch_cache_holds_many_widths(fake):
    """Wide rows have an entry for each width. However many a process has seen, calls that it has
    made before ask the runtime nothing."""
    got = fake("""
    widths = [8200 + 8 * i for i in range(600)]
    def calls():
        for cols in widths:
            assert rms(400, cols) == 0 and silu(400, cols + 8192) == 0
        before = F.fake_queries()
        for _ in range(50):
            assert rms(4608, 2048) == 0 and silu(4608, 12288) == 0
        return before
    calls()
    first = F.fake_queries()
    again = calls()
    print(json.dumps([first, again - first, F.fake_queries() - again]))
    """)
    assert got == [1202, 0, 0]


def test_shared_memory_limits_of_many_devices(fake):
    """A function's limit only ever grows, on each of the 64 devices that the library knows: a small
    launch after a large one must not lower it, since another thread may be launching the large one."""
    got = fake("""
    F.fake_limit_falls.restype = ctypes.c_int
    wide = [12296, 24584, 16392]
    for sweep in (wide, wide[::-1]):
        for dev in range(64):
            F.fake_device(dev)
            for cols in sweep:
                for e4m3 in (0, 1):
                    for residual in (False, True):
                        assert rms(400, cols, residual, e4m3) == 0
                    assert silu(400, cols, e4m3) == 0
    print(json.dumps([F.fake_refused(), F.fake_limit_falls()]))
    """)
    assert got == [0, 0]
