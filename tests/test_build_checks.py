"""The build's check of the assembly listings, on planted listings."""
import pytest

from dynamic_short_convolution_amd import build

JOIN = """
	s_and_saveexec_b64 s[2:3], vcc
	s_cbranch_execz .LBB29_15
; %bb.14:                               ;   in Loop: Header=BB29_11 Depth=1
	global_load_dwordx4 v[34:37], v[2:3], off
	s_waitcnt vmcnt(0)
	ds_write_b128 v0, v[34:37]
.LBB29_15:                              ;   in Loop: Header=BB29_11 Depth=1
{before}
	s_or_b64 exec, exec, s[2:3]
	scratch_load_dword v0, off, off offset:108 ; 4-byte Folded Reload
	s_cbranch_vccnz .LBB29_33
"""
SHORT = """
	s_and_saveexec_b64 s[2:3], vcc
; %bb.98:
	ds_read_b32 v58, v49 offset:1020
; %bb.99:
{before}
	s_or_b64 exec, exec, s[2:3]
	s_endpgm
"""


@pytest.mark.parametrize("listing", [JOIN, SHORT])
@pytest.mark.parametrize("before", ["\tscratch_store_dwordx4 off, v[78:81], off offset:16 ; 16-byte Folded Spill",
                                    "\ts_mov_b32 s91, s16\n\tv_accvgpr_write_b32 a46, v234          ;  Reload Reuse",
                                    "\tv_mov_b32_e32 v7, v9"])
def test_copies_before_the_mask_is_restored_are_found(listing, before):
    (found,) = build.misplaced_vector_code(listing.format(before=before))
    assert before.split("\n")[-1].split(";")[0].strip() in found


@pytest.mark.parametrize("listing", [JOIN, SHORT])
@pytest.mark.parametrize("before", ["", "\ts_mov_b32 s91, s16", "\tv_writelane_b32 v255, s3, 4", "\tv_readlane_b32 s3, v255, 4",
                                    "\ts_xor_b64 exec, exec, s[4:5]\n\tv_mov_b32_e32 v7, v9"])
def test_scalar_code_is_not(listing, before):
    """Scalar copies, lanes of a register that holds scalars, and code under a mask of its own."""
    assert build.misplaced_vector_code(listing.format(before=before)) == []


def test_a_branch_body_is_not():
    """A block that ends in the restoring because the join has been merged into the body."""
    assert build.misplaced_vector_code("""
	s_and_saveexec_b64 s[0:1], vcc
	s_cbranch_execnz .LBB1_119
	s_endpgm
.LBB1_119:
	v_lshlrev_b64 v[4:5], 8, v[0:1]
	global_store_dword v[4:5], v50, off
	s_or_b64 exec, exec, s[0:1]
	s_endpgm
""") == []
