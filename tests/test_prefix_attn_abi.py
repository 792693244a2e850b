"""CPU checks of the C ABI of the attention behind a shared prefix
(include/prefix_attn.h): every call returns before any HIP work is enqueued."""
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
MOST = lib.W4A16_WORKSPACE_HEAD_BYTES + (128 << 20)


def status(call, *a, **k):
    with pytest.raises(lib.W4A16Error) as e:
        call(*a, **k)
    return e.value.status


def test_header_and_exports_agree(tmp_path):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "prefix_attn.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*int\s+(\w+)\s*\(", text, re.M))
    assert names == set(lib.EXPORTED_PREFIX) == {"prefix_attn", "prefix_attn_workspace_bytes"}
    so = ctypes.CDLL(lib.LIB_PATH)
    assert all(hasattr(so, n) for n in names)
    for cc, lang in (("gcc", "c"), ("g++", "c++")):
        if not shutil.which(cc):
            continue
        src = tmp_path / ("u.c" if lang == "c" else "u.cpp")
        src.write_text('#include "prefix_attn.h"\n#include "tree_attn.h"\n#include "lora.h"\nint main(void) { return 0; }\n')
        r = subprocess.run([cc, "-fsyntax-only", "-Wall", "-Wextra", "-Werror", "-x", lang,
                            "-I" + os.path.join(ROOT, "include"), str(src)], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr


def call(**over):
    a = dict(q=GOOD, qs=1280, k=GOOD, v=GOOD, dtype="bf16", pages=100, page=16, ps=16 * 256, ts=256, hs=128, ptable=GOOD, plen=GOOD,
             max_prefix=500, table=GOOD, stride=20, lens=GOOD, max_len=300, mask=GOOD, scale=0.1, out=GOOD, lse=GOOD, B=2, T=4, Hq=10,
             Hkv=2, D=128, work=GOOD, n=1 << 30)
    a.update(over)
    return status(lib.prefix_attn, a["q"], a["qs"], a["k"], a["v"], a["dtype"], a["pages"], a["page"], a["ps"], a["ts"], a["hs"],
                  a["ptable"], a["plen"], a["max_prefix"], a["table"], a["stride"], a["lens"], a["max_len"], a["mask"], a["scale"],
                  a["out"], a["lse"], a["B"], a["T"], a["Hq"], a["Hkv"], a["D"], a["work"], a["n"], stream=0)


def test_refusals():
    for p in ("q", "k", "v", "ptable", "plen", "table", "lens", "mask", "out"):
        assert call(**{p: 0}) == -1, p
    for p in ("q", "k", "v", "out", "work"):
        assert call(**{p: GOOD + 8}) == -3, p
    for p in ("ptable", "plen", "table", "lens", "lse"):
        assert call(**{p: GOOD + 2}) == -3, p
    assert call(mask=GOOD + 4) == -3
    assert call(dtype="f32") == -4 and call(dtype=9) == -4
    for over in (dict(B=0), dict(T=0), dict(T=65), dict(Hq=9), dict(Hkv=0), dict(Hq=0), dict(max_len=-1), dict(max_prefix=-1),
                 dict(max_prefix=(1 << 30) + 1), dict(max_len=(1 << 30) + 1), dict(page=24), dict(page=0), dict(pages=0), dict(stride=0),
                 dict(stride=18), dict(qs=1272), dict(qs=1284), dict(ps=-8), dict(ts=260), dict(hs=4), dict(ts=1 << 26),
                 dict(scale=float("nan")), dict(scale=float("inf")), dict(Hq=65538, qs=65538 * 128), dict(B=1 << 20, Hq=32, qs=4096)):
        assert call(**over) == -2, over
    assert call(D=96) == -6 and call(page=8, stride=40) == -6 and call(page=1, stride=400) == -6


def test_workspace_query():
    q = lib.prefix_attn_workspace_bytes
    # without a prefix, or with a short one, requests that fill the GPU need no parts
    assert q(512, 1, 40, 8, 128, 0, 100) == 0 and q(512, 1, 40, 8, 128, 20, 100) == 0
    need = q(8, 1, 40, 8, 128, 131000, 1000)
    assert need > lib.W4A16_WORKSPACE_HEAD_BYTES
    a = dict(B=8, T=1, Hq=40, Hkv=8, qs=5120, max_prefix=131000, max_len=1000, stride=100)
    assert call(**a, work=None, n=0) == -1 and call(**a, n=need - 1) == -5
    for over in ((0, 1, 1, 1, 64, 10, 10), (1, 65, 1, 1, 64, 10, 10), (1, 1, 3, 2, 64, 10, 10), (1, 1, 1, 1, 64, -1, 10)):
        assert status(q, *over) == -2, over
    assert status(q, 1, 1, 1, 1, 80, 10, 10) == -6
    assert lib._lib_get().prefix_attn_workspace_bytes(1, 1, 1, 1, 64, 10, 10, None) == -1
    for B in (1, 7, 100, 3000):
        for T in (1, 8, 64):
            for Hq, Hkv in ((1, 1), (40, 8), (64, 1), (128, 128)):
                for D in (64, 128, 256):
                    for n in (0, 1000, 1 << 20, 1 << 30):
                        for m in (0, 300, 1 << 30):
                            assert q(B, T, Hq, Hkv, D, n, m) <= MOST


def test_size_limits_are_the_same_for_the_query_and_the_call():
    # Launches of 2^32 work-items (calls in a process that sees no GPU: -7 is a launch that failed there).
    code = ("import ctypes, bit_weight_only_03_amd as L\n"
            "lib, b, p = L._lib_get(), ctypes.c_size_t(), 4096\n"
            "for B, T, Hq, Hkv, D, P in ((1 << 24, 1, 1, 1, 64, 0), (1 << 20, 64, 16, 1, 256, 100), (1 << 23, 1, 1, 1, 128, 64), (1, 1, 1, 1, 64, 10)):\n"
            "    print(lib.prefix_attn_workspace_bytes(B, T, Hq, Hkv, D, P, 10, ctypes.byref(b)), lib.prefix_attn(p, Hq * D, p, p, 1, 1, 16, 0, D, 0,\n"
            "          p, p, P, p, 1000, p, 10, p, 0.1, p, None, B, T, Hq, Hkv, D, p, 1 << 40, None))\n")
    out = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, HIP_VISIBLE_DEVICES="-1"), capture_output=True, text=True,
                         timeout=300, cwd=ROOT)
    assert out.returncode == 0, out.stderr[-500:]
    got = [tuple(int(v) for v in line.split()) for line in out.stdout.strip().split("\n")[-4:]]
    assert got[0] == (-6, -6) and got[3] == (0, -7), got
    for query, run in got:
        assert (query == -6) == (run == -6) and query in (0, -6) and run in (-6, -7), got
