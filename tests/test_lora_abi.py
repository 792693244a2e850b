"""CPU checks of the C ABI of the low-rank adapters (include/lora.h): every call
returns before any HIP work is enqueued."""
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
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "lora.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*int\s+(\w+)\s*\(", text, re.M))
    assert names == set(lib.EXPORTED_LORA) == {"lora_add", "lora_workspace_bytes"}
    so = ctypes.CDLL(lib.LIB_PATH)
    assert all(hasattr(so, n) for n in names)
    for cc, lang in (("gcc", "c"), ("g++", "c++")):
        if not shutil.which(cc):
            continue
        src = tmp_path / ("u.c" if lang == "c" else "u.cpp")
        src.write_text('#include "lora.h"\n#include "w8a8.h"\nint main(void) { return 0; }\n')
        r = subprocess.run([cc, "-fsyntax-only", "-Wall", "-Wextra", "-Werror", "-x", lang,
                            "-I" + os.path.join(ROOT, "include"), str(src)], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr


def call(**over):
    a = dict(x=GOOD, dtype="bf16", ldx=512, a=GOOD, b=GOOD, ranks=GOOD, scales=GOOD, n=4, adapter=GOOD, base=GOOD, y=GOOD, ydt="bf16", ldy=320,
             cols=[128, 64, 128], M=3, N=320, K=512, R=16, work=GOOD, bytes=1 << 40)
    a.update(over)
    return status(lib.lora_add, a["x"], a["dtype"], a["ldx"], a["a"], a["b"], a["ranks"], a["scales"], a["n"], a["adapter"], a["base"], a["y"],
                  a["ydt"], a["ldy"], a["cols"], a["M"], a["N"], a["K"], a["R"], a["work"], a["bytes"], stream=0)


def test_refusals():
    for p in ("x", "a", "b", "adapter", "y"):
        assert call(**{p: 0}) == -1, p
    for p in ("x", "a", "b", "base", "y", "work"):
        assert call(**{p: GOOD + 8}) == -3, p
    for p in ("ranks", "scales", "adapter"):
        assert call(**{p: GOOD + 2}) == -3, p
    assert call(dtype="f32") == -4 and call(dtype=9) == -4 and call(ydt=5) == -4
    for over in (dict(M=0), dict(M=(1 << 26) + 1), dict(N=0), dict(N=324), dict(N=(1 << 24) + 8), dict(K=0), dict(K=12), dict(K=(1 << 20) + 8),
                 dict(R=0), dict(R=12), dict(R=264), dict(n=0), dict(ldx=504), dict(ldx=516), dict(ldx=(1 << 24) + 8), dict(ldy=(1 << 25) + 8), dict(ldy=312), dict(ldy=324),
                 dict(cols=[128, 128]), dict(cols=[128, 64, 136]), dict(cols=[120, 72, 128]), dict(cols=[320, 0]), dict(cols=[64, -64, 320]),
                 dict(cols=[312]), dict(cols=[64, 64, 64, 64, 64]), dict(cols=[256, 64, 4, -4])):
        assert call(**over) == -2, over
    # the parts' widths are needed where there are several
    lib_get = lib._lib_get()
    p = GOOD
    assert lib_get.lora_add(p, 1, 512, p, p, p, p, 4, p, p, p, 1, 320, None, 2, 3, 320, 512, 16, p, 1 << 40, None) == -1


def test_workspace():
    assert lib.lora_workspace_bytes(1, 7168, 5120, 16, 3) == 0
    need = lib.lora_workspace_bytes(8, 5120, 17408, 64, 1)
    assert need > lib.W4A16_WORKSPACE_HEAD_BYTES
    a = dict(M=8, N=5120, K=17408, R=64, ldx=17408, ldy=5120, cols=None)
    assert call(**a, bytes=need - 1) == -5 and call(**a, work=None, bytes=0) == -1
    for over in ((0, 64, 64, 16, 1), (1, 60, 64, 16, 1), (1, 64, 4, 16, 1), (1, 64, 64, 20, 1), (1, 64, 64, 16, 0), (1, 64, 64, 16, 5)):
        assert status(lib.lora_workspace_bytes, *over) == -2, over
    assert lib._lib_get().lora_workspace_bytes(1, 64, 64, 16, 1, None) == -1


def test_size_limits_are_the_same_for_the_query_and_the_call():
    # Launches of 2^32 work-items (calls in a process that sees no GPU: -7 is a launch that failed there).
    code = ("import ctypes, bit_weight_only_03_amd as L\n"
            "lib, b, p = L._lib_get(), ctypes.c_size_t(), 4096\n"
            "for M, parts, K, R in ((1 << 26, 4, 64, 128), (1 << 26, 1, 1 << 20, 256), (1 << 26, 2, 64, 8), (1, 1, 64, 8)):\n"
            "    N, cols = 256 * parts, (ctypes.c_int * parts)(*([256] * parts))\n"
            "    print(lib.lora_workspace_bytes(M, N, K, R, parts, ctypes.byref(b)),\n"
            "          lib.lora_add(p, 1, K, p, p, None, None, 1, p, None, p, 1, N, cols, parts, M, N, K, R, p, 1 << 60, None))\n")
    out = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, HIP_VISIBLE_DEVICES="-1"), capture_output=True, text=True,
                         timeout=300, cwd=ROOT)
    assert out.returncode == 0, out.stderr[-500:]
    got = [tuple(int(v) for v in line.split()) for line in out.stdout.strip().split("\n")[-4:]]
    assert got[0] == (-6, -6) and got[3] == (0, -7), got
    for query, run in got:
        assert (query == -6) == (run == -6) and query in (0, -6) and run in (-6, -7), got
