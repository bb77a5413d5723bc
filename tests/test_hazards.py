"""The wait states in front of loads into LDS (rotated_bit_amd/hazards.py): the
check on listings with a known answer, and on the library that is built here."""
import os

import pytest

from rotated_bit_amd import hazards as Z

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OBJECT = os.path.join(ROOT, "rotated_bit_amd", "_build", "fp8_gemm.hip.o")
LOAD = "buffer_load_dwordx4 v1, s[4:7], s9 offen lds"


def found(*lines):
    text = "0000000000001000 <kernel>:\n"
    for line in lines:
        text += f"{line}\n" if "<" in line else f"\t{line}   // 000000001000: BF800000\n"
    bad, loads = Z.violations(text)
    assert loads == sum(line.endswith(" lds") for line in lines)
    return bad


M0 = ("s_mov_b32 m0, s2", "s_nop 0")


@pytest.mark.parametrize("write,hit", [
    ("v_readlane_b32 s4, v9, 3", True), ("v_readlane_b32 s7, v9, 3", True),
    ("v_readfirstlane_b32 s9, v9", True), ("v_readlane_b32 s8, v9, 3", False),
    ("v_cmp_gt_u32_e64 s[6:7], 8, v2", True), ("v_cmp_gt_u32_e64 s[8:9], 8, v2", True),
    ("v_cmp_gt_u32_e64 s[10:11], 8, v2", False), ("v_add_u32_e32 v4, s4, v2", False),
    ("v_add_co_u32_e64 v0, s[4:5], v2, v3", True), ("s_mov_b32 s4, s20", False),
    ("v_readfirstlane_b32 m0, v3", True),
])
def test_writes_of_scalars(write, hit):
    assert bool(found(write, *M0, LOAD)) == hit
    assert bool(found(write, "s_nop 1", *M0, LOAD)) == hit          # four wait states
    assert not found(write, "s_nop 2", *M0, LOAD)                   # five
    assert not found(write, "s_add_i32 s2, s2, 1", "s_mov_b32 s3, 0", "v_nop", *M0, LOAD)


def test_m0_needs_one():
    assert found("s_mov_b32 m0, s2", LOAD)
    assert not found("s_mov_b32 m0, s2", "s_nop 0", LOAD)
    assert not found("s_mov_b32 m0, s2", "v_add_u32_e32 v1, s4, v1", LOAD)


def test_paths():
    # round a loop, over a branch, and not through an unconditional one
    loop = ["0000000000001010 <L0>:", *M0, LOAD, "v_readlane_b32 s5, v9, 0", "s_cbranch_scc1 L0",
            "s_endpgm"]
    assert found(*loop)
    assert not found(*loop[:-2], "s_nop 1", *loop[-2:])
    over = ["v_readlane_b32 s5, v9, 0", "s_cbranch_scc1 L1", "s_nop 7",
            "0000000000001020 <L1>:", *M0, LOAD, "s_endpgm"]
    assert found(*over)
    away = ["v_readlane_b32 s5, v9, 0", "s_branch L2", "0000000000001020 <L1>:", *M0, LOAD,
            "0000000000001030 <L2>:", "s_endpgm"]
    assert not found(*away)
    # another function's end is no way in
    assert not found("v_readlane_b32 s5, v9, 0", "0000000000002000 <other>:", *M0, LOAD)
    with pytest.raises(ValueError):
        found("s_cbranch_scc1 L9", LOAD)


@pytest.mark.skipif(not os.path.exists(OBJECT), reason="no object files of a build here")
def test_the_library_that_is_built():
    assert Z.check_object(OBJECT) > 0
