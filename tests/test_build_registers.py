"""The build's check of kernels whose warps share out the launch's registers."""
import os
import re

import pytest

from pagedattention_kv_cache_pa_b200 import _build

REPORT = """ptxas info    : 77 bytes gmem
ptxas info    : Compiling entry function '_ZN2pa19prefill_wide_kernelILi128ELb1EEEv' for 'sm_100a'
ptxas info    : Function properties for _ZN2pa19prefill_wide_kernelILi128ELb1EEEv
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used %d registers, used 1 barriers
ptxas info    : Compiling entry function '_ZN2pa17wide_merge_kernelILi128EEEv' for 'sm_100a'
ptxas info    : Function properties for _ZN2pa17wide_merge_kernelILi128EEEv
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used 32 registers, used 0 barriers
"""


def test_reports():
    assert _build.check_registers(REPORT % 128, "prefill_wide_kernel", 128) == 1
    for text in (REPORT % 126, REPORT % 136, "", (REPORT % 128) + (REPORT % 120)):
        with pytest.raises(RuntimeError, match="registers"):
            _build.check_registers(text, "prefill_wide_kernel", 128)


def test_the_kernel_and_the_build_name_the_same_number():
    for src, (kernel, want) in _build.LAUNCH_REGISTERS.items():
        with open(os.path.join(_build.CSRC, src)) as f:
            text = f.read()
        assert kernel in text and re.search(r"kLaunchRegs = %d\b" % want, text)
