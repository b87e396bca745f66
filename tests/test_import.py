"""Importing the package, its library loader, its build and its workloads needs no torch (CPU only): they serve
programs that have none, and torch takes seconds to load."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "causal_depthwise_conv1d_width_amd"


def run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_import_without_torch():
    run(f"import sys; sys.modules['torch'] = None; import {PKG} as cc; from {PKG} import _lib, build, workloads; "
        "assert set(cc.__all__) <= set(dir(cc))")


def test_every_name_is_there():
    run(f"import {PKG} as cc; assert all(hasattr(cc, n) for n in cc.__all__); "
        f"from {PKG} import ssm; assert cc.ssm_scan_fwd is ssm.ssm_scan_fwd; assert not hasattr(cc, 'nothing')")
    run(f"from {PKG} import *; ssm_scan_fwd, gated_norm_bwd, conv1d_fwd, SsmGrads")
