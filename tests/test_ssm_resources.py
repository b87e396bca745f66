"""The scan's, the step's and the norms' gfx950 kernels keep their state in registers (no scratch) and fit the
blocks a CU that they are written for into its 160 KB of shared memory.

A spill in the scan's loops waits for every load before it, so the rows of the next chunk, which are loaded ahead,
stop being ahead (the backward took a fifth longer with 56 bytes of scratch).  Not meant: the forms for rows that are not
aligned, which hold a tile's elements one by one, and the norms' backward of groups above 16384 channels (4 pieces of 8
channels a thread in 128 registers).  CPU only: hipcc cross-compiles for gfx950.
"""
import os
import re
import shutil
import subprocess

import pytest

from causal_depthwise_conv1d_width_amd import build

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None, reason="needs hipcc")

LDS = 160 * 1024


def test_no_scratch_and_blocks_fit(tmp_path):
    procs = {}
    for src in (s for s in build.SSM_SOURCES if s.endswith(".hip")):  # the sources compile concurrently
        out = tmp_path / (src + ".s")
        cmd = ["hipcc", *build.hipcc_flags(), "-x", "hip", "--cuda-device-only", "-S",
               os.path.join(build.CSRC, src), "-o", str(out)]
        procs[src] = (subprocess.Popen(cmd, stdout=subprocess.DEVNULL, stderr=subprocess.PIPE, text=True), out)
    bad, seen = {}, set()
    for src, (proc, out) in procs.items():
        _, err = proc.communicate()
        assert proc.returncode == 0, f"{src}: hipcc failed\n{err}"
        for name, body in re.findall(r"\.amdhsa_kernel (\S+)\n(.*?)\.end_amdhsa_kernel", out.read_text(), re.S):
            lds = int(re.search(r"\.amdhsa_group_segment_fixed_size (\d+)", body).group(1))
            scratch = int(re.search(r"\.amdhsa_private_segment_fixed_size (\d+)", body).group(1))
            ints, flags = [int(v) for v in re.findall(r"Li(\d+)E", name)], re.findall(r"Lb([01])E", name)
            kernel = re.search(r"(ssm|gated|residual|norm)_\w+?_kernel", name).group(0)
            seen.add(kernel)
            if kernel.startswith("ssm") and flags[:1] == ["0"] and kernel != "ssm_join_kernel":
                continue
            if kernel.endswith("norm_bwd_kernel") and ints[:2] == [1024, 4]:
                continue
            blocks = 2 if kernel == "ssm_scan_bwd_kernel" and ints[0] <= 128 else 1
            if scratch or lds * blocks > LDS:
                bad[name] = (lds, scratch)
    assert {"ssm_scan_fwd_kernel", "ssm_scan_bwd_kernel", "ssm_states_kernel", "ssm_step_kernel",
            "gated_norm_bwd_kernel", "residual_norm_fwd_kernel"} <= seen
    assert not bad, f"kernels with (LDS bytes, scratch bytes per lane): {bad}"
