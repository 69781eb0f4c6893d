"""Kernels whose warps share out their launch's registers are held to the number of them when they are built."""
import os
import re

import pytest

from speculative_decoding_hybrid_gb300 import build

REPORT = """ptxas info    : 0 bytes gmem, 440 bytes cmem[4]
ptxas info    : Compiling entry function '_ZN1_18prompt_join_kernelILi64ELb0EEEvNS_4ArgsE' for 'sm_103a'
ptxas info    : Function properties for _ZN1_18prompt_join_kernelILi64ELb0EEEvNS_4ArgsE
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used 61 registers, used 0 barriers
ptxas info    : Compiling entry function '_ZN1_20prompt_attend_kernelILi64EEEvNS_4ArgsE' for 'sm_103a'
ptxas info    : Function properties for _ZN1_20prompt_attend_kernelILi64EEEvNS_4ArgsE
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used %d registers, used 1 barriers, 2032 bytes smem
"""


def test_another_number_of_registers_is_no_build():
    build.check_registers(REPORT % 168)
    build.check_registers("")
    for used in (160, 255):
        with pytest.raises(RuntimeError, match="prompt_attend_kernelILi64.* has %d registers.* 168" % used):
            build.check_registers(REPORT % used)


def test_the_number_is_the_source_s():
    with open(os.path.join(build.CSRC, "prompt_attend.cu")) as f:
        assert re.findall(r"kLaunchRegs = (\d+)", f.read()) == [str(build.LAUNCH_REGISTERS["prompt_attend_kernel"])]
