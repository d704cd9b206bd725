"""Compile the layer kernels for gfx950 and check their registers: none spills.
CPU only (hipcc cross-compiles)."""
import os
import re
import shutil
import subprocess

import pytest

from blockwise_fp8_gemm_bfp8_amd import build as bfp8_build


@pytest.mark.parametrize("source,least", [("norm.hip", 70), ("glu.hip", 20), ("clip.hip", 5)])
def test_kernels_do_not_spill(source, least, tmp_path):
    if shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("hipcc not available")
    out = tmp_path / "out.s"
    subprocess.run([bfp8_build.hipcc(), *bfp8_build.compile_flags(), "-x", "hip", "-S",
                    "--cuda-device-only", os.path.join(bfp8_build.CSRC, source), "-o", str(out)],
                   check=True, capture_output=True)
    asm = out.read_text()
    blocks = re.split(r"\n  - ", asm[asm.index("amdhsa.kernels:"):])[1:]
    kernels = [b for b in blocks if re.search(r"\.name:", b)]
    assert len(kernels) >= least
    for b in kernels:
        name = re.search(r"\.name:\s+(\S+)", b).group(1)
        get = lambda k: int(re.search(r"\." + k + r":\s+(\d+)", b).group(1))
        assert get("vgpr_spill_count") == 0 and get("private_segment_fixed_size") == 0, name
        assert get("group_segment_fixed_size") <= 64 * 1024, name
