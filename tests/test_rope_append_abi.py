"""CPU checks of the C ABI of rotary positions and the append to the paged cache
(include/rope_append.h): every call returns before any HIP work is enqueued."""
import ctypes
import math
import os
import re
import shutil
import struct
import subprocess

import pytest

import bit_weight_only_03_amd as lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GOOD = 1 << 20


def status(call, *a, **k):
    with pytest.raises(lib.W4A16Error) as e:
        call(*a, **k)
    return e.value.status


def test_header_and_exports_agree(tmp_path):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "rope_append.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*int\s+(\w+)\s*\(", text, re.M))
    assert names == set(lib.EXPORTED_ROPE) == {"rope_append", "rope_frequencies"}
    so = ctypes.CDLL(lib.LIB_PATH)
    assert all(hasattr(so, n) for n in names)
    for cc, lang in (("gcc", "c"), ("g++", "c++")):
        if not shutil.which(cc):
            continue
        src = tmp_path / ("u.c" if lang == "c" else "u.cpp")
        src.write_text('#include "rope_append.h"\n#include "tree_attn.h"\nint main(void) { return 0; }\n')
        r = subprocess.run([cc, "-fsyntax-only", "-Wall", "-Wextra", "-Werror", "-x", lang,
                            "-I" + os.path.join(ROOT, "include"), str(src)], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr


def call(**over):
    a = dict(q=GOOD, qs=1280, k=GOOD, ks=256, v=GOOD, vs=256, dtype="bf16", pos=GOOD, freq=GOOD, rot=128, inter=0, gain=1.0, qo=GOOD + 64,
             qos=1280, kc=GOOD, vc=GOOD, pages=10, page=16, ps=4096, ts=256, hs=128, slots=GOOD, M=3, Hq=10, Hkv=2, D=128)
    a.update(over)
    return status(lib.rope_append, a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["dtype"], a["pos"], a["freq"], a["rot"], a["inter"],
                  a["gain"], a["qo"], a["qos"], a["kc"], a["vc"], a["pages"], a["page"], a["ps"], a["ts"], a["hs"], a["slots"], a["M"],
                  a["Hq"], a["Hkv"], a["D"], stream=0)


def test_refusals():
    for p in ("q", "qo", "k", "v", "kc", "vc", "slots", "pos", "freq"):
        assert call(**{p: 0}) == -1, p
    nothing = dict(k=0, v=0, kc=0, vc=0, slots=0)
    assert call(q=0, qo=0, **nothing) == -1
    for p in ("q", "qo", "k", "v", "kc", "vc"):
        assert call(**{p: GOOD + 8}) == -3, p
    assert call(pos=GOOD + 2) == -3 and call(freq=GOOD + 2) == -3 and call(slots=GOOD + 4) == -3
    assert call(dtype="f32") == -4 and call(dtype=7) == -4
    for over in (dict(M=0), dict(M=-1), dict(D=0), dict(D=120), dict(D=528), dict(rot=-16), dict(rot=144), dict(rot=24), dict(inter=2),
                 dict(gain=math.nan), dict(gain=math.inf), dict(Hq=0), dict(Hq=1 << 17), dict(Hkv=0), dict(qs=1272), dict(qs=1284), dict(qos=1272),
                 dict(ks=248), dict(vs=260), dict(pages=0), dict(page=0), dict(page=24), dict(ps=-8), dict(ts=4), dict(hs=-128),
                 dict(qo=GOOD, qos=1288)):
        assert call(**over) == -2, over
    # more work-items than a launch takes
    assert call(M=(1 << 31) - 1) == -6
    # the parts that are left out are not looked at
    assert call(**nothing, M=(1 << 31) - 1, Hkv=-5, page=3, ks=1, ps=-1) == -6
    assert call(q=0, qo=0, M=(1 << 31) - 1, Hq=-5, qs=1) == -6


def bits(x):
    return struct.unpack("<I", struct.pack("<f", x))[0]


def test_frequencies():
    f = lib.rope_frequencies(128, 10000.0)
    assert len(f) == 64 and f[0] == 1.0
    for i, x in enumerate(f):
        assert abs(bits(x) - bits(10000.0 ** (-2 * i / 128))) <= 1
    assert all(abs(a * 4 - b) <= 2.0 ** -23 * b for a, b in zip(lib.rope_frequencies(128, 10000.0, 4.0), f))
    parts = lib.rope_frequencies(128, 10000.0, 8.0, 4096, 1.0, 32.0)
    for x, y in zip(f, parts):
        turns = 4096 * x / (2 * math.pi)
        w = min(1.0, max(0.0, (turns - 1.0) / 31.0))
        assert abs(y - x * (w + (1 - w) / 8)) <= 2.0 ** -20 * x
    assert parts[0] == f[0] and abs(parts[-1] * 8 - f[-1]) <= 2.0 ** -22 * f[-1]
    assert lib.rope_frequencies(2, 10.0) == [1.0]


def test_frequency_refusals():
    s = lambda *a: status(lib.rope_frequencies, *a)  # noqa: E731
    inf, nan = math.inf, math.nan
    for a in ((0, 1e4), (-2, 1e4), (3, 1e4), (1026, 1e4), (64, 1.0), (64, nan), (64, inf), (64, 1e4, 0.5), (64, 1e4, inf), (64, 1e4, 2.0, -1.0),
              (64, 1e4, 2.0, inf), (64, 1e4, 2.0, 4096.0, 0.0, 32.0), (64, 1e4, 2.0, 4096.0, 32.0, 32.0), (64, 1e4, 2.0, 4096.0, 1.0, inf),
              (64, 1e4, 2.0, 4096.0, nan, 32.0)):
        assert s(*a) == -2, a


def test_frequencies_of_a_size_past_a_c_int():
    # Refused, neither cut to 32 bits (which would write past a list made for the number given) nor given room for.
    for n in (1 << 20, (1 << 32) + 64, 64 - (1 << 32), 1 << 45):
        assert status(lib.rope_frequencies, n, 1e4) == -2, n
    assert len(lib.rope_frequencies(1024, 1e4)) == 512
