"""The check of wait states in the package's own machine code
(adamw_optimizer_step_amd/wait_states.py): distances between instructions that the
compiler does not see, as one of them stands in inline assembly."""
import os

import pytest

from adamw_optimizer_step_amd import _lib as L
from adamw_optimizer_step_amd import wait_states as W

MFMA8 = "v_mfma_scale_f32_16x16x128_f8f6f4 v[170:173], v[6:9], v[22:29], v[170:173], v200, v18 op_sel_hi:[0,0,0] cbsz:4"
MFMA4 = "v_mfma_scale_f32_16x16x128_f8f6f4 v[170:173], v[6:9], v[22:25], v[170:173], v200, v18 op_sel_hi:[0,0,0] cbsz:4 blgp:4"


def listing(*code):
    """The lines as llvm-objdump prints them, 8 bytes each; a branch names its target's line."""
    out = ["0000000000001000 <k>:"]
    for n, line in enumerate(code):
        to = ""
        if isinstance(line, tuple):
            line, at = line
            to = f" <k+0x{8 * at:x}>" if at else " <k>"
        out.append(f"\t{line:<58} // {0x1000 + 8 * n:012X}: D3AC0000 000225C8{to}")
    return "\n".join(out)


@pytest.mark.parametrize("write", ["v_mov_b64_e32 v[172:173], s[0:1]", "v_mov_b32_e32 v170, 0", "v_lshrrev_b32_e32 v200, v229, v49", "v_mov_b32_e32 v18, 1",
                                   "v_bitop3_b32 v29, v55, v35, v55 bitop3:0xc", "v_perm_b32 v6, v1, v2, v3", "v_permlane16_swap_b32_e32 v1, v7"])
@pytest.mark.parametrize("between,short", [([], True), (["s_nop 0"], True), (["s_waitcnt lgkmcnt(0)"], True), (["s_nop 1"], False), (["v_mov_b32_e32 v1, 0"] * 2, False)])
def test_vector_results_reach_a_matrix_instruction_after_two_states(write, between, short):
    assert bool(W.violations(listing(write, *between, MFMA8))) == short


def test_other_registers_and_memory_are_no_matter():
    assert W.violations(listing("v_mov_b32_e32 v174, 0", "ds_read_b128 v[6:9], v226 offset:4096", "s_mov_b32 s18, 1", MFMA8)) == []


@pytest.mark.parametrize("mfma,least", [(MFMA8, 12), (MFMA4, 8)])
@pytest.mark.parametrize("use", ["v_cvt_pk_bf16_f32 v1, v170, v171", "global_store_dwordx4 v[0:1], v[170:173], off", "v_mov_b32_e32 v173, 0", "v_mfma_f32_16x16x4_f32 v[0:3], v170, v4, v[0:3]",
                                 "v_mfma_scale_f32_16x16x128_f8f6f4 v[172:175], v[6:9], v[22:29], v[172:175], v200, v18 op_sel_hi:[0,0,0] cbsz:4"])
def test_matrix_results_settle(mfma, least, use):
    assert W.violations(listing(mfma, f"s_nop {least - 2}", use))
    assert W.violations(listing(mfma, f"s_nop {least - 1}", use)) == []


def test_accumulating_in_place_needs_no_distance():
    assert W.violations(listing(MFMA8, MFMA8)) == []
    assert W.violations(listing(MFMA8, MFMA8.replace("v[170:173], v[6:9]", "v[2:5], v[6:9]"))) == []


def test_every_path_counts():
    wait = "s_nop 15"
    assert W.violations(listing("v_mov_b32_e32 v170, 0", ("s_cbranch_scc1 3", 3), wait, MFMA8))                 # over the wait
    assert W.violations(listing(MFMA8, wait, "v_mov_b32_e32 v170, 0", ("s_branch 65532", 0)))                # back to the start
    assert W.violations(listing("v_mov_b32_e32 v170, 0", ("s_branch 2", 3), MFMA8, wait, MFMA8)) == []
    assert W.violations(listing("v_mov_b32_e32 v170, 0", "s_endpgm", MFMA8)) == []


def test_scalar_addresses_from_vector_instructions_and_m0():
    copy = "global_load_lds_dwordx4 v2, s[34:35]"
    for write in ("v_readfirstlane_b32 s35, v1", "v_cmp_lt_i32_e64 s[34:35], v1, v2"):
        assert W.violations(listing(write, "s_nop 3", copy))
        assert W.violations(listing(write, "s_nop 4", copy)) == []
    assert W.violations(listing("s_add_u32 s34, s1, s2", copy)) == []
    assert W.violations(listing("s_mov_b32 m0, s80", copy))
    assert W.violations(listing("s_mov_b32 m0, s80", "s_nop 0", copy)) == []


def test_the_built_library_keeps_its_distances():
    if not os.path.exists(L.LIB_PATH) or not os.path.exists(W.OBJDUMP):
        pytest.skip("no library or no disassembler")
    text = W.disassemble(L.LIB_PATH)
    assert text.count(W.MFMA_SCALE) > 500 and text.count("global_load_lds_dwordx4") > 100    # the code is there
    assert W.violations(text) == []
