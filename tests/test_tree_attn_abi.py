"""CPU checks of the draft-tree attention's C ABI (include/tree_attn.h): every
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
GOOD = 1 << 20


def status(call, *a, **k):
    with pytest.raises(lib.W4A16Error) as e:
        call(*a, **k)
    return e.value.status


def test_header_and_exports_agree(tmp_path):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "tree_attn.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*int\s+(\w+)\s*\(", text, re.M))
    assert names == set(lib.EXPORTED_TREE) == {"tree_attn", "tree_attn_workspace_bytes"}
    so = ctypes.CDLL(lib.LIB_PATH)
    assert all(hasattr(so, n) for n in names)
    for cc, lang in (("gcc", "c"), ("g++", "c++")):
        if not shutil.which(cc):
            continue
        src = tmp_path / ("u.c" if lang == "c" else "u.cpp")
        src.write_text('#include "tree_attn.h"\n#include "w8a8.h"\nint main(void) { return 0; }\n')
        r = subprocess.run([cc, "-fsyntax-only", "-Wall", "-Wextra", "-Werror", "-x", lang,
                            "-I" + os.path.join(ROOT, "include"), str(src)], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr


def call(**over):
    a = dict(q=GOOD, qs=1280, k=GOOD, v=GOOD, dtype="bf16", pages=100, page=16, ps=16 * 256, ts=256, hs=128, table=GOOD,
             stride=20, lens=GOOD, max_len=300, mask=GOOD, scale=0.1, out=GOOD, lse=GOOD, B=1, T=4, Hq=10, Hkv=2, D=128,
             work=GOOD, n=1 << 30)
    a.update(over)
    return status(lib.tree_attn, a["q"], a["qs"], a["k"], a["v"], a["dtype"], a["pages"], a["page"], a["ps"], a["ts"], a["hs"],
                  a["table"], a["stride"], a["lens"], a["max_len"], a["mask"], a["scale"], a["out"], a["lse"], a["B"], a["T"],
                  a["Hq"], a["Hkv"], a["D"], a["work"], a["n"], stream=0)


def test_refusals():
    for p in ("q", "k", "v", "table", "lens", "mask", "out"):
        assert call(**{p: 0}) == -1
    for p in ("q", "k", "v", "out", "work"):
        assert call(**{p: GOOD + 8}) == -3
    for p in ("table", "lens", "lse"):
        assert call(**{p: GOOD + 2}) == -3
    assert call(mask=GOOD + 4) == -3
    assert call(dtype="f32") == -4 and call(dtype=9) == -4
    for over in (dict(B=0), dict(T=0), dict(T=65), dict(Hq=9), dict(Hkv=0), dict(Hq=0), dict(max_len=-1), dict(page=24),
                 dict(page=0), dict(pages=0), dict(stride=0), dict(stride=18), dict(qs=1272), dict(qs=1284), dict(ps=-8),
                 dict(ts=260), dict(hs=4), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**over) == -2, over
    assert call(D=96) == -6


def test_workspace_query():
    assert lib.tree_attn_workspace_bytes(1, 1, 1, 1, 64, 0) == 0
    # many requests fill the GPU without a split of the keys
    assert lib.tree_attn_workspace_bytes(64, 1, 40, 8, 128, 4096) == 0
    need = lib.tree_attn_workspace_bytes(1, 1, 40, 8, 128, 150000)
    assert need > lib.W4A16_WORKSPACE_HEAD_BYTES
    assert call(T=1, Hq=40, Hkv=8, qs=5120, max_len=150000, stride=10000, work=None, n=0) == -1
    assert call(T=1, Hq=40, Hkv=8, qs=5120, max_len=150000, stride=10000, n=need - 1) == -5
    assert status(lib.tree_attn_workspace_bytes, 1, 65, 1, 1, 64, 10) == -2
    for B in (1, 2, 7, 16, 100):
        for T in (1, 8, 64):
            for Hq, Hkv in ((1, 1), (40, 8), (64, 1), (128, 128)):
                for D in (64, 128, 256):
                    for n in (0, 1000, 1 << 20, 1 << 30):
                        assert lib.tree_attn_workspace_bytes(B, T, Hq, Hkv, D, n) <= lib.W4A16_WORKSPACE_HEAD_BYTES + (64 << 20)


def test_size_limits_are_the_same_for_the_query_and_the_call():
    assert call(Hq=65538, qs=65538 * 128) == -2 and status(lib.tree_attn_workspace_bytes, 1, 1, 65538, 2, 128, 10) == -2
    assert call(B=1 << 20, T=1, Hq=32, Hkv=8, qs=4096) == -2
    assert status(lib.tree_attn_workspace_bytes, 1 << 20, 1, 32, 8, 128, 10) == -2
    # A launch of 2^32 work-items, whatever the kernel (calls in a process that sees no GPU: -7 is a launch that failed there).
    code = ("import ctypes, bit_weight_only_03_amd as L\n"
            "lib, b, p = L._lib_get(), ctypes.c_size_t(), 4096\n"
            "for B, T, Hq, Hkv, D in ((1 << 24, 1, 1, 1, 64), (1 << 20, 64, 16, 1, 256), (1 << 22, 64, 1, 1, 64), (1 << 24, 1, 1, 1, 256)):\n"
            "    print(lib.tree_attn_workspace_bytes(B, T, Hq, Hkv, D, 10, ctypes.byref(b)), lib.tree_attn(p, Hq * D, p, p, 1, 1, 16, 0, D, 0,\n"
            "          p, 1000, p, 10, p, 0.1, p, None, B, T, Hq, Hkv, D, p, 1 << 40, None))\n")
    out = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, HIP_VISIBLE_DEVICES="-1"), capture_output=True, text=True,
                         timeout=300, cwd=ROOT)
    assert out.returncode == 0, out.stderr[-500:]
    got = [tuple(int(v) for v in line.split()) for line in out.stdout.strip().split("\n")[-4:]]
    assert got == [(-6, -6), (-6, -6), (0, -7), (0, -7)]
