"""The delta rule's, the layer norm's and the slot copies' gfx950 kernels keep their state in registers (no scratch) and fit
their blocks into a CU's 160 KB of shared memory.

A spill in the walks waits for every load before it, so that the next chunk's tiles stop being ahead.  Not meant: the chunk
kernel, whose blocks run three to a CU with a few of its addresses spilled outside its inner products; the backward's chunk
kernel of states past 128 columns, which holds two tiles' gradients in registers; and the layer norm's backward above 8192
channels (2 or 4 pieces of 8 channels a thread, with both parameters' sums, in 128 registers).  CPU only: hipcc cross-compiles for gfx950.
"""
import os
import re
import shutil
import subprocess

import pytest

from causal_depthwise_conv1d_width_amd import build

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None, reason="needs hipcc")

LDS = 160 * 1024
# blocks a CU that the kernels are written for
BLOCKS = {"delta_chunk_kernel": 3, "delta_walks_kernel": 2}


def test_no_scratch_and_blocks_fit(tmp_path):
    procs = {}
    for src in (s for s in build.DELTA_SOURCES if s.endswith(".hip")):  # the sources compile concurrently
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
            ints = [int(v) for v in re.findall(r"Li(\d+)E", name)]
            kernel = re.search(r"(delta|layer|slots)_\w*?kernel", name).group(0)
            seen.add(kernel)
            spills = kernel in ("delta_chunk_kernel", "delta_scan_bwd_wide_kernel") or (
                kernel == "layer_norm_bwd_kernel" and ints[0] == 1024 and ints[1] > 1)
            wide = ints and ints[0] > 128
            if (scratch and not spills) or lds * (1 if wide else BLOCKS.get(kernel, 1)) > LDS:
                bad[name] = (lds, scratch)
    assert {"delta_chunk_kernel", "delta_scan_fwd_kernel", "delta_scan_fwd_wide_kernel", "delta_walks_kernel",
            "delta_scan_bwd_kernel", "delta_scan_bwd_wide_kernel", "delta_step_kernel", "layer_norm_fwd_kernel",
            "layer_norm_bwd_kernel", "slots_kernel"} <= seen
    assert not bad, f"kernels with (LDS bytes, scratch bytes per lane): {bad}"
