"""The build's check of kernels whose inline assembly names accumulation registers: a
listing in which the compiler itself uses one is refused."""
import os
import re

import pytest

from fp8_block_scaled_x128_amd import build

GOOD = """
_ZN1k_otherILi1EEvv:
	v_accvgpr_write_b32 a3, v1
.Lfunc_end0:
_ZN9k_i8_tileILi4ELi4ELb0EEvv:             ; @_ZN9k_i8_tile
; %bb.0:
	v_add_u32_e32 v1, v2, v3               ; a0 in a comment
	;;#ASMSTART
	v_mfma_i32_32x32x32_i8 a[0:15], v[0:3], v[4:7], a[0:15]
	;;#ASMEND
	global_store_dwordx4 v0, v[4:7], s[0:1]
	s_endpgm
.Lfunc_end1:
	v_accvgpr_read_b32 v1, a3
"""
BAD = ["	v_accvgpr_write_b32 a255, v1", "	v_accvgpr_read_b32 v9, a0", "	global_load_dwordx4 a[4:7], v1, s[0:1]",
       "	v_mfma_i32_16x16x64_i8 a[0:3], v[0:3], v[4:7], a[0:3]"]
KERNELS = build.OWN_ACCUMULATORS["int8_gemm.hip"]


def test_listing_without_them_passes():
    build.check_accumulators(GOOD, KERNELS)
    build.check_accumulators(GOOD.replace("k_i8_tileI", "k_i8_tile_pairI"), KERNELS)


@pytest.mark.parametrize("line", BAD)
def test_listing_with_one_is_refused(line):
    with pytest.raises(RuntimeError, match="k_i8_tile"):
        build.check_accumulators(GOOD.replace("	s_endpgm", line + "\n	s_endpgm"), KERNELS)
    build.check_accumulators(GOOD.replace("ILi4ELi4E", "ILi2ELi2E") + GOOD.replace("	s_endpgm", "	s_nop 0"), KERNELS)


def test_listing_without_the_kernels_is_refused():
    with pytest.raises(RuntimeError, match="no kernel"):
        build.check_accumulators(GOOD.replace("k_i8_tile", "k_i8_title"), KERNELS)


def test_every_source_that_owns_registers_is_checked():
    owners = set()
    for name in os.listdir(build.CSRC):
        with open(os.path.join(build.CSRC, name)) as f:
            if re.search(r'asm[^;]*"[^"]*\ba(\[|\d)', f.read()):
                owners.add(name)
    assert owners == set(build.OWN_ACCUMULATORS)
