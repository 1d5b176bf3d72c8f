"""The build's check of kernels that count vector-memory instructions."""
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
