"""The build's check of kernels that count vector-memory instructions."""
import os
import re

import pytest

from mixture_experts_layer_macs_amd import build

REMARK = """linear.hip:1:1: remark: Function Name: {name} [-Rpass-analysis=kernel-resource-usage]
linear.hip:1:1: remark:     VGPRs: 200 [-Rpass-analysis=kernel-resource-usage]
linear.hip:1:1: remark:     ScratchSize [bytes/lane]: {size} [-Rpass-analysis=kernel-resource-usage]
linear.hip:1:1: remark:     Occupancy [waves/SIMD]: 1 [-Rpass-analysis=kernel-resource-usage]
"""


def test_scratch_check():
    src = "linear.hip"
    good = REMARK.format(name="_ZN3moe3lin10mma_kernelEv", size=0)
    other = REMARK.format(name="_ZN3moe3lin11join_kernelEv", size=16)
    build._check_scratch(src, other + good)
    with pytest.raises(RuntimeError, match="16 bytes of scratch"):
        build._check_scratch(src, good + REMARK.format(name="_ZN3moe3lin10mma_kernelEi", size=16))


@pytest.mark.parametrize("remarks", ["", "linear.hip:1:1: remark: scratch size 0 in mma_kernel\n",
                                     REMARK.format(name="_ZN3moe3lin11join_kernelEv", size=0)])
def test_scratch_check_needs_a_kernel_to_look_at(remarks):
    with pytest.raises(RuntimeError, match="name no kernel"):
        build._check_scratch("linear.hip", remarks)


ASM = """_ZN3moe3lin10mma_kernelEv:
{write}
{between}	buffer_load_dwordx4 v8, s[0:3], s22 offen lds
"""


@pytest.mark.parametrize("write", ["\tv_readfirstlane_b32 s2, v35", "\tv_readlane_b32 s22, v1, s5",
                                   "\tv_cmp_lt_i32_e64 s[2:3], v1, v2", "\tv_mad_u64_u32 v[2:3], s[0:1], v1, v2, v[4:5]"])
def test_hazard_check(write):
    near = "".join(f"\tv_mov_b32 v{i}, 0\n.Lx:\n\t; a comment\n" for i in range(4))
    with pytest.raises(RuntimeError, match="4 wait states"):
        build._check_hazards("linear.hip", ASM.format(write=write, between=near))
    build._check_hazards("linear.hip", ASM.format(write=write, between=near + "\ts_mov_b32 s40, 1\n"))
    build._check_hazards("linear.hip", ASM.format(write=write, between="\ts_nop 4\n"))
    build._check_hazards("linear.hip", ASM.format(write=write.replace("s2", "s42").replace("s[2:3]", "s[8:9]").replace(
        "s[0:1]", "s[8:9]"), between=""))


def test_hazard_check_needs_a_load_to_look_at():
    with pytest.raises(RuntimeError, match="no direct-to-LDS load"):
        build._check_hazards("linear.hip", "_Zx:\n\ts_endpgm\n")


@pytest.mark.parametrize("write,states", [("\ts_add_i32 m0, s2, 0x400", 1), ("\ts_mov_b32 m0, s2", 1),
                                          ("\tv_readfirstlane_b32 m0, v35", 5)])
def test_hazard_check_of_the_lds_address(write, states):
    """A load takes its LDS address from M0: one wait state behind a scalar
    instruction that writes it, five behind a vector instruction."""
    near = "".join(f"\ts_add_i32 s{40 + i}, m0, 1\n" for i in range(states - 1))
    with pytest.raises(RuntimeError, match=f" {states - 1} wait states"):
        build._check_hazards("linear.hip", ASM.format(write=write, between=near))
    build._check_hazards("linear.hip", ASM.format(write=write, between=near + "\ts_nop 0\n"))
    build._check_hazards("linear.hip", ASM.format(write=write, between=near + "\ts_cmp_eq_u32 m0, 0\n"))


LOOP = """_ZN3moe3lin10mma_kernelEv:
	s_mov_b32 m0, 0
	s_branch .LBB0_2
.LBB0_1:
{first}	s_cbranch_scc1 .LBB0_3
	s_nop 4
.LBB0_2:
	s_nop 4
	{back}
	s_nop 4
{last}.LBB0_3:
	buffer_load_dwordx4 v8, s[0:3], s22 offen lds
	s_endpgm
"""


def test_hazard_check_follows_branches():
    """What a jump leads past the instructions in between, and what stands before
    a jump that is always taken."""
    check = lambda **k: build._check_hazards("linear.hip", LOOP.format(**{  # noqa: E731
        "first": "", "back": "s_cbranch_scc0 .LBB0_1", "last": "", **k}))
    check()
    near = "\tv_readfirstlane_b32 s22, v1\n"
    with pytest.raises(RuntimeError, match="s22, v1' writes 1 wait states"):
        check(first=near)                                          # behind a jump
    with pytest.raises(RuntimeError, match="s22, v1' writes 0 wait states"):
        check(last=near)                                           # in the text's order
    check(first=near + "\ts_nop 3\n")
    check(last=near + "\ts_branch .LBB0_2\n")                      # not on the way to the load
    check(first="\ts_mov_b32 m0, s1\n")                            # the jump itself is the wait state


def test_hazard_check_of_two_kernels():
    """What ends a kernel is not on the way into the next one."""
    end = "_Za:\n\tv_readfirstlane_b32 s22, v1\n"
    load = "_Zb:\n\tbuffer_load_dwordx4 v8, s[0:3], s22 offen lds\n"
    build._check_hazards("linear.hip", end + "\ts_endpgm\n" + load)
    build._check_hazards("linear.hip", end + load)


def test_every_source_with_inline_loads_is_checked():
    """A source that includes dma.h, itself or through its headers, issues them."""
    def includes(name):
        with open(os.path.join(build.CSRC, name)) as f:
            own = re.findall(r'#include "([^"/]+)"', f.read())
        return set(own).union(*(includes(n) for n in own))
    assert {s for s in build.SOURCES if "dma.h" in includes(s)} == set(build.DIRECT)
    assert set(build.COUNTED) <= set(build.DIRECT)
