"""CPU checks that a workspace made for the largest batch serves every smaller one: a server asks once.  The calls run in a
process that sees no GPU: -7 is a launch that failed there, after every check of the arguments."""
import os
import subprocess
import sys

import bit_weight_only_03_amd as lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def statuses(code):
    out = subprocess.run([sys.executable, "-c", "import ctypes, bit_weight_only_03_amd as L\nlib, p = L._lib_get(), 4096\n" + code],
                         env=dict(os.environ, HIP_VISIBLE_DEVICES="-1"), capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert out.returncode == 0, out.stderr[-500:]
    return [int(v) for v in out.stdout.split()]


def test_lora_of_fewer_rows():
    for K in (8, 200, 5120, 17408, 100000):
        for R, parts in ((8, 1), (16, 1), (16, 3), (64, 1), (64, 2), (104, 4), (256, 1), (256, 4)):
            last = 0
            for M in [*range(1, 1100), *range(1100, 20000, 37), 65536, 1 << 20]:
                need = lib.lora_workspace_bytes(M, 1024, K, R, parts)
                assert need >= last, (M, K, R, parts)
                last = need
    # at most four times what one slice of these rows takes
    assert lib.lora_workspace_bytes(4096, 7168, 5120, 16, 3) <= lib.W4A16_WORKSPACE_HEAD_BYTES + 4 * 4096 * 3 * 16 * 4
    got = statuses("for most, N, K, R in ((4096, 256, 5120, 16), (600, 64, 100000, 256), (64, 264, 17408, 32)):\n"
                   "    need = L.lora_workspace_bytes(most, N, K, R)\n"
                   "    for M in (1, 2, 15, 16, 17, 40, 63, 64, 65, 300, 511, 512, 513, 4095, 4096):\n"
                   "        if M <= most: print(lib.lora_add(p, 1, K, p, p, None, None, 1, p, None, p, 1, N, None, 1, M, N, K, R, p, need, None))\n"
                   "    print(lib.lora_add(p, 1, K, p, p, None, None, 1, p, None, p, 1, N, None, 1, most, N, K, R, p, need - 1, None))\n")
    assert got.count(-5) == 3 and set(got) == {-5, -7}, got


def test_prefix_attn_of_a_smaller_batch():
    q = lib.prefix_attn_workspace_bytes
    sizes = dict(B=(1, 2, 3, 7, 16, 39, 40, 61, 64, 256, 1000, 3000), T=(1, 2, 7, 64), P=(0, 1, 32, 33, 300, 777, 7000, 7500, 8192, 131000, 1 << 30),
                 L=(0, 31, 100, 300, 480, 700, 1000, 8000, 1 << 30))
    for Hq, Hkv, D in ((40, 8, 128), (16, 16, 64), (8, 1, 256), (128, 4, 128)):
        need = {(B, T, P, n): q(B, T, Hq, Hkv, D, P, n) for B in sizes["B"] for T in sizes["T"] for P in sizes["P"] for n in sizes["L"]}
        for at, (name, v) in enumerate(sizes.items()):
            up = dict(zip(v, v[1:]))
            for key, b in need.items():
                if key[at] in up:
                    assert b <= need[(*key[:at], up[key[at]], *key[at + 1:])], (key, name)
    got = statuses("for most, T, P, n in ((64, 1, 8192, 700), (256, 4, 16384, 300), (16, 7, 300, 9000)):\n"
                   "    need = L.prefix_attn_workspace_bytes(most, T, 40, 8, 128, P, n)\n"
                   "    call = lambda B, P, n, have: print(lib.prefix_attn(p, 5120, p, p, 1, 1, 16, 0, 128, 0, p, p, P, p, 1000, p, n, p, 0.1, p, None, B, T, 40, 8, 128, p, have, None))\n"
                   "    [call(B, P // c, n // d, need) for B in (1, 2, 16, 39, 40, 61, 64, 200, 256) if B <= most for c in (1, 2, 50, 1000) for d in (1, 3, 1000)]\n"
                   "    call(most, P, n, need - 1)\n")
    assert got.count(-5) == 3 and set(got) == {-5, -7}, got
