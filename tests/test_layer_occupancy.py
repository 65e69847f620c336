"""The LoRA-gradient kernels wait for memory: what hides it is a second workgroup on every CU.  Every rank and
format has to leave room for two (160 KiB of LDS and 512 registers per SIMD lane); the compiler's report shows it."""
import os
import re

import pytest

from segmented_gather_matvec_amd import build
from tests.test_kernel_resources import _device_asm


@pytest.fixture(scope="module")
def gradient_kernels(tmp_path_factory):
    try:
        build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    asm = _device_asm(os.path.join(build.CSRC, "sgmv_lowrank.hip"), str(tmp_path_factory.mktemp("asm")))
    out = {}
    for block in re.split(r"\n\s+- \.agpr_count:", asm)[1:]:
        field = lambda k: re.search(r"\.%s:\s+(\S+)" % k, block).group(1)  # noqa: E731
        m = re.search(r"sgmv_lora_grad_kernelINS_\d(B?F16)ELi(\d+)E", field("name"))
        if m:
            out[m.group(1), int(m.group(2))] = int(field("group_segment_fixed_size")), int(field("vgpr_count"))
    return out


@pytest.mark.parametrize("dtype", ["F16", "BF16"])
@pytest.mark.parametrize("rank", [8, 16, 32, 64])
def test_two_workgroups_of_a_lora_gradient_share_a_cu(gradient_kernels, dtype, rank):
    lds, vgprs = gradient_kernels[dtype, rank]
    assert 2 * lds <= 160 << 10
    assert 2 * vgprs <= 512      # four waves a workgroup, one on each SIMD
