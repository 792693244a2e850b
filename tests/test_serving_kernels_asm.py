"""Host-side checks of the gfx950 assembly of the rotary append's, the adapters' and the
shared-prefix attention's kernels: nothing spills to scratch, no packed fp32 arithmetic, inline
assembly holds waits alone, and products read their operands without a register's detour."""
import os
import re
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_new_kernels_asm import HIPCC, compile_asm

SOURCES = ["rope_append.hip", "lora.hip", "prefix_attn.hip"]

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")


@pytest.fixture(scope="module")
def asm():
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        return dict(zip(SOURCES, ex.map(compile_asm, SOURCES)))


def kernels(text):
    """Name and body of each kernel."""
    return [(m.group(1), m.group(0)) for m in re.finditer(r"^(_ZN\S*_kernel\S*):.*?\.Lfunc_end", text, re.S | re.M)]


@pytest.mark.parametrize("src", SOURCES)
def test_no_scratch_no_spills_no_packed_fp32(asm, src):
    text = asm[src]
    sizes = [int(v) for v in re.findall(r"\.private_segment_fixed_size: (\d+)", text)]
    spills = [int(v) for v in re.findall(r"\.vgpr_spill_count: (\d+)", text)]
    assert kernels(text) and len(sizes) == len(kernels(text)) and not any(sizes) and not any(spills)
    assert not re.search(r"v_pk_(add|mul|fma)_f32", text)


@pytest.mark.parametrize("src", SOURCES)
def test_inline_assembly_holds_waits_alone(asm, src):
    for block in re.findall(r";;#ASMSTART\n(.*?);;#ASMEND", asm[src], re.S):
        for line in block.split("\n"):
            assert not line.strip() or line.strip().startswith("s_waitcnt"), line


@pytest.mark.parametrize("src", SOURCES)
def test_no_register_is_split_off_to_the_accumulation_file(asm, src):
    # Heads of 256 alone keep some of their sums there.
    for name, body in kernels(asm[src]):
        assert "Li256E" in name or "v_accvgpr" not in body, name


@pytest.mark.parametrize("src", SOURCES)
def test_buffers_are_uniform(asm, src):
    # A buffer descriptor that the compiler takes for different in each lane costs a loop around every access.
    for name, body in kernels(asm[src]):
        for m in re.finditer(r"v_readfirstlane_b32[^\n]*\n(?:[^\n]*\n){0,12}?[^\n]*s_and_saveexec_b64[^\n]*\n(?:[^\n]*\n){0,6}?[^\n]*buffer_", body):
            raise AssertionError((name, m.group(0)))
