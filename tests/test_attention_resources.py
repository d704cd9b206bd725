"""Compile the attention kernels for gfx950 and check their registers: a spill
inside their loops costs scratch traffic beside every matrix instruction (the
first dkdv kernel spilled 24 registers and ran 1.5 times slower than without).
CPU only (hipcc cross-compiles)."""
import os
import re
import shutil
import subprocess

import pytest

from blockwise_fp8_gemm_bfp8_amd import build as bfp8_build

KERNELS = {"attention.hip": ["attention_forward_kernelILi64", "attention_forward_kernelILi128",
                             "attention_stream_kernelILi64", "attention_stream_kernelILi128",
                             "attention_join_kernel", "attention_join_splits_kernel"],
           "attention_bwd.hip": ["attention_stats_kernel", "attention_sum_kernel",
                                 "attention_backward_kernelILi64",
                                 "attention_backward_kernelILi128"],
           "rope.hip": ["rope_table_kernel", "rope_kernelItLi8ELb0", "rope_kernelItLi4ELb1",
                        "rope_kernelIfLi4ELb0", "rope_kernelIfLi2ELb1"]}


@pytest.mark.parametrize("source", list(KERNELS))
def test_kernels_do_not_spill(source, tmp_path):
    if shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("hipcc not available")
    out = tmp_path / "out.s"
    subprocess.run([bfp8_build.hipcc(), *bfp8_build.compile_flags(), "-x", "hip", "-S",
                    "--cuda-device-only", os.path.join(bfp8_build.CSRC, source), "-o", str(out)],
                   check=True, capture_output=True)
    asm = out.read_text()
    blocks = re.split(r"\n  - ", asm[asm.index("amdhsa.kernels:"):])[1:]
    for kernel in KERNELS[source]:
        found = [b for b in blocks if re.search(r"\.name:\s+\S*" + kernel, b)]
        assert len(found) == 1, kernel
        get = lambda k: int(re.search(r"\." + k + r":\s+(\d+)", found[0]).group(1))
        assert get("vgpr_spill_count") == 0 and get("private_segment_fixed_size") == 0, kernel
        assert get("group_segment_fixed_size") <= 160 * 1024, kernel
