"""Host-side checks of the gfx950 assembly of the 8-bit layer's and the tree
attention's kernels: nothing spills to scratch, no register is split off to the
accumulation file (which would put a move at every use of a sum), and inline
assembly holds waits alone."""
import os
import re
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_weight_only_03_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
SOURCES = ["w8a8_rows.hip", "w8a8_gemm.hip", "tree_attn.hip"]

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")


def compile_asm(src):
    from bit_weight_only_03_amd.build import SOURCE_FLAGS
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "o.s")
        cmd = [HIPCC, "-O3", "-std=c++17", "--offload-arch=gfx950", "--cuda-device-only", "-S", "-Xclang", "-target-feature",
               "-Xclang", "-packed-fp32-ops", *SOURCE_FLAGS.get(src, []), "-o", out, os.path.join(CSRC, src)]
        res = subprocess.run(cmd, capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-2000:]
        return open(out).read()


@pytest.fixture(scope="module")
def asm():
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        return dict(zip(SOURCES, ex.map(compile_asm, SOURCES)))


@pytest.mark.parametrize("src", SOURCES)
def test_no_scratch_no_spills_no_accumulation_registers(asm, src):
    text = asm[src]
    sizes = [int(v) for v in re.findall(r"\.private_segment_fixed_size: (\d+)", text)]
    spills = [int(v) for v in re.findall(r"\.vgpr_spill_count: (\d+)", text)]
    assert sizes and not any(sizes) and not any(spills)
    assert "v_accvgpr" not in text
    assert not re.search(r"v_pk_(add|mul|fma)_f32", text)


@pytest.mark.parametrize("src", SOURCES)
def test_inline_assembly_holds_waits_alone(asm, src):
    for block in re.findall(r";;#ASMSTART\n(.*?);;#ASMEND", asm[src], re.S):
        for line in block.split("\n"):
            assert not line.strip() or line.strip().startswith("s_waitcnt"), line


def test_products_wait_for_no_younger_load(asm):
    # In a tiled kernel's loop the only wait for vector loads without any
    # allowed to be under way is none: each counts the younger ones.
    text = asm["w8a8_gemm.hip"]
    kernels = re.findall(r"^(_ZN\S*w8a8_tiled_kernel\S*):.*?\.Lfunc_end", text, re.S | re.M)
    assert len(kernels) == 4
    for m in re.finditer(r"^_ZN\S*w8a8_tiled_kernel\S*:.*?\.Lfunc_end", text, re.S | re.M):
        body = m.group(0)
        loop = body[body.index("s_barrier"):]
        loop = loop[:loop.index("s_cbranch")]
        waits = [int(v) for v in re.findall(r"vmcnt\((\d+)\)", loop)]
        assert waits and min(waits) >= 2, waits
        assert loop.count("v_mfma") >= 8
