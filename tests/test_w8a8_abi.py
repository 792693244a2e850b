"""CPU checks of the 8-bit layer's C ABI (include/w8a8.h): declarations and
exports agree, size queries and argument checks behave as documented.  Every
call returns before any HIP work is enqueued."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import pytest

import bit_weight_only_03_amd as lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GOOD = 1 << 20    # an aligned address that no refused call touches


def declared(header):
    text = open(os.path.join(ROOT, "include", header)).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return set(re.findall(r"^\s*int\s+(\w+)\s*\(", text, re.M))


def status(call, *a, **k):
    with pytest.raises(lib.W4A16Error) as e:
        call(*a, **k)
    return e.value.status


def test_header_and_exports_agree():
    so = ctypes.CDLL(lib.LIB_PATH)
    names = declared("w8a8.h")
    assert names == {"w8a8_rmsnorm_quant", "w8a8_silu_mul_quant", "w8a8_workspace_bytes", "w8a8_gemm"}
    for n in names:
        assert hasattr(so, n) and n in lib.EXPORTED_W8A8


def test_header_compiles_as_c_and_cpp(tmp_path):
    for cc, lang in (("gcc", "c"), ("g++", "c++")):
        if not shutil.which(cc):
            continue
        src = tmp_path / ("u.c" if lang == "c" else "u.cpp")
        src.write_text('#include "w8a8.h"\nint main(void) { return (int)sizeof(w4a16_status) - (int)sizeof(int); }\n')
        r = subprocess.run([cc, "-fsyntax-only", "-Wall", "-Wextra", "-Werror", "-x", lang,
                            "-I" + os.path.join(ROOT, "include"), str(src)], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr


def norm(x=GOOD, xd="bf16", ldx=256, res=GOOD, rd="bf16", h=GOOD, w=GOOD, wd="bf16", eps=1e-6, y=GOOD, yd="bf16",
         q=GOOD, s=GOOD, M=2, K=256):
    return status(lib.w8a8_rmsnorm_quant, x, xd, ldx, res, rd, h, w, wd, eps, y, yd, q, s, M, K, stream=0)


def test_norm_refusals():
    assert norm(x=0) == -1 and norm(w=0) == -1 and norm(y=0, q=0, s=0) == -1
    assert norm(q=0) == -1 and norm(s=0) == -1                      # codes and scales come together
    assert norm(res=0) == -1                                        # h_out without a residual
    assert norm(xd=3) == -4 and norm(rd=9) == -4 and norm(wd=-1) == -4 and norm(yd=5) == -4
    assert norm(M=0) == -2 and norm(K=0, ldx=0) == -2 and norm(K=248) == -2 and norm(ldx=248) == -2 and norm(ldx=260) == -2
    assert norm(eps=-1.0) == -2 and norm(eps=float("nan")) == -2 and norm(eps=float("inf")) == -2
    for p in ("x", "res", "h", "w", "y", "q", "s"):
        assert norm(**{p: GOOD + 8}) == -3
    assert norm(K=32784, ldx=32784) == -6


def gated(x=GOOD, xd="f16", ldx=512, y=GOOD, yd="f16", q=GOOD, s=GOOD, M=2, K=256):
    return status(lib.w8a8_silu_mul_quant, x, xd, ldx, y, yd, q, s, M, K, stream=0)


def test_gated_refusals():
    assert gated(x=0) == -1 and gated(y=0, q=0, s=0) == -1 and gated(s=0) == -1 and gated(q=0) == -1
    assert gated(xd=7) == -4 and gated(yd=7) == -4
    assert gated(M=0) == -2 and gated(K=250) == -2 and gated(K=0) == -2 and gated(ldx=504) == -2 and gated(ldx=516) == -2
    assert gated(M=(1 << 31) - 1, K=4096, ldx=8192) == -2           # more workgroups than a grid holds
    for p in ("x", "y", "q", "s"):
        assert gated(**{p: GOOD + 4}) == -3


def gemm(x=GOOD, xs=GOOD, w=GOOD, ws=GOOD, y=GOOD, yd="bf16", M=1, N=64, K=256, buf=None, n=0):
    return status(lib.w8a8_gemm, x, xs, w, ws, y, yd, M, N, K, buf, n, stream=0)


def test_gemm_refusals_and_sizes():
    for p in ("x", "xs", "w", "ws", "y"):
        assert gemm(**{p: 0}) == -1
        assert gemm(**{p: GOOD + 8}) == -3
    assert gemm(yd=4) == -4
    for M, N, K in ((0, 64, 256), (1, 0, 256), (1, 12, 256), (1, 64, 0), (1, 64, 200), (1, 64, (1 << 20) + 16), ((1 << 26) + 1, 64, 256)):
        assert gemm(M=M, N=N, K=K) == -2
        assert status(lib.w8a8_workspace_bytes, M, N, K) == -2
    # A long sum over few columns is split: the size query says so, and less is refused.
    need = lib.w8a8_workspace_bytes(8, 640, 17408)
    assert need > lib.W4A16_WORKSPACE_HEAD_BYTES
    assert gemm(M=8, N=640, K=17408) == -1
    assert gemm(M=8, N=640, K=17408, buf=GOOD, n=need - 1) == -5
    assert gemm(M=8, N=640, K=17408, buf=GOOD + 4, n=need) == -3
    # Enough tiles need no workspace, and no shape needs more than 64 MiB and the head.
    assert lib.w8a8_workspace_bytes(4096, 34816, 5120) == 0
    for M in (1, 7, 8, 9, 16, 17, 64, 65, 100, 128, 300, 512, 1000, 5000):
        for N in (8, 512, 5120, 34816):
            for K in (16, 128, 5136, 17408, 1 << 20):
                assert lib.w8a8_workspace_bytes(M, N, K) <= lib.W4A16_WORKSPACE_HEAD_BYTES + (64 << 20)


def test_gemm_refuses_overridden_slices_that_leave_no_plan():
    # 8 slices of 4096 x 34816 in 256 x 256 tiles need more than the largest workspace: no kernel may be launched.
    code = ("import ctypes, bit_weight_only_03_amd as L\n"
            "lib = ctypes.CDLL(L.LIB_PATH)\n"
            "p = ctypes.c_void_p(4096)\n"
            "print(lib.w8a8_gemm(p, p, p, p, p, 1, 4096, 34816, 5120, p, ctypes.c_size_t(1 << 40), None))\n")
    env = dict(os.environ, W8A8_VARIANT="7", W8A8_SPLIT="8")
    out = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert out.returncode == 0, out.stderr[-500:]
    assert int(out.stdout.split()[-1]) == -6   # W4A16_ERR_UNSUPPORTED


def gemm_statuses_without_a_device(*shapes):
    """(size query's status, call's status) of each M, N, K in a process that sees no GPU: a call that passes the
    checks reports its failed launch (W4A16_ERR_HIP), nothing runs."""
    code = ("import ctypes, sys, bit_weight_only_03_amd as L\n"
            "lib = ctypes.CDLL(L.LIB_PATH)\n"
            "p, b = ctypes.c_void_p(4096), ctypes.c_size_t()\n"
            "for s in sys.argv[1:]:\n"
            "    M, N, K = (int(v) for v in s.split('x'))\n"
            "    q = lib.w8a8_workspace_bytes(M, N, K, ctypes.byref(b))\n"
            "    print(q, lib.w8a8_gemm(p, p, p, p, p, 1, M, N, K, p, ctypes.c_size_t(1 << 40), None))\n")
    env = {k: v for k, v in os.environ.items() if not k.startswith("W8A8_")}
    out = subprocess.run([sys.executable, "-c", code, *("%dx%dx%d" % s for s in shapes)], env=dict(env, HIP_VISIBLE_DEVICES="-1"),
                         capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert out.returncode == 0, out.stderr[-500:]
    return [tuple(int(v) for v in line.split()) for line in out.stdout.split("\n")[-len(shapes) - 1:-1]]


def test_gemm_counts_the_tiles_of_the_largest_n():
    # N + 255 passes 32 bits: more workgroups than a launch takes, whatever the kernel, and so refused.
    for (_, rc), M in zip(gemm_statuses_without_a_device((1, 2**31 - 8, 16), (8, 2**31 - 8, 16), (16, 2**31 - 8, 16), (600, 2**31 - 8, 16)),
                          (1, 8, 16, 600)):
        assert rc == -6, M   # W4A16_ERR_UNSUPPORTED


def test_gemm_long_sums_over_many_columns_have_a_plan():
    # Up to 16 rows, K past what the table of scales holds, and so many columns that the slices pass their limits: by the
    # counters (the first two) and by the partial sums' size (the others).
    shapes = [(9, 524296, 16400), (1, 524296, 32784), (16, 152064, 131072), (1, 34816, 1 << 20), (1, 65536, 1 << 20), (1, 1 << 30, 16)]
    for got, s in zip(gemm_statuses_without_a_device(*shapes), shapes):
        assert got == (0, -7), (s, got)   # as far as the launch: W4A16_ERR_HIP


def test_gemm_size_query_refuses_what_the_call_refuses():
    for got in gemm_statuses_without_a_device((1, 2**31 - 8, 16), (1 << 26, 1 << 14, 16)):
        assert got == (-6, -6), got


def test_row_operators_refuse_launches_past_their_size():
    assert norm(M=1 << 26, K=16, ldx=16) == -6 and norm(M=1 << 22, K=8192, ldx=8192) == -6
    assert gated(M=1 << 28, K=16, ldx=32) == -6 and gated(M=1 << 24, K=2048, ldx=4096) == -6
    assert gated(K=(1 << 30) + 16, ldx=1 << 32) == -2
