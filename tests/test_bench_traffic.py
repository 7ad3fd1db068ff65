"""The committed HBM counter and matrix-core summaries belong to the kernels that
are there: the benchmark reports measured traffic only while a summary's digest
equals that of the kernel's source, so a summary left behind by a change of the
source (or of a header it shares with others) would silently end the report.

CPU only: nothing here touches a GPU.
"""
from __future__ import annotations

import os
import re

import pytest

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = "moe_layer_route_amd/csrc/"
# summary stem -> (kernel source, the benchmark's name of the summary where the file's own is not it)
KERNELS = {"gemv": ("gemv.hip", None), "gemm": ("gemm.hip", None), "mxfp4": ("mxfp4.hip", None),
           "mxfp4_gemm": ("mxfp4_gemm.hip", None), "fp8_gemv": ("fp8.hip", "fp8_gemv"),
           "fp8_gemm": ("fp8_gemm.hip", "fp8_gemm")}


def _summaries(pattern):
    names = sorted(os.listdir(os.path.join(ROOT, "profiles")))
    return [m for m in (re.fullmatch(pattern, n) for n in names) if m]


@pytest.mark.parametrize("stem,workload", [(m[1], m[2]) for m in _summaries(r"counters_(\w+)_(c\d)\.txt")])
def test_traffic_is_reported(stem, workload):
    file, name = KERNELS[stem]
    with open(os.path.join(ROOT, "profiles", f"counters_{stem}_{workload}.txt")) as fh:
        want = float(re.search(r"^hbm_bytes_per_launch=(\d+)$", fh.read(), re.M)[1])
    assert bench._traffic(CSRC + file, workload, stem=name) == want


def test_default_workloads_have_a_summary():
    """The headline (bf16, prefill) and the decode workload beside it."""
    assert bench._traffic(CSRC + "gemm.hip", "c5") and bench._traffic(CSRC + "gemv.hip", "c2")


@pytest.mark.parametrize("stem", [m[1] for m in _summaries(r"mfma_(\w+?)_c3_c5\.md")])
def test_matrix_core_summaries_are_current(stem):
    with open(os.path.join(ROOT, "profiles", f"mfma_{stem}_c3_c5.md")) as fh:
        digest = re.search(r"source_digest=([0-9a-f]{16})", fh.read())[1]
    assert digest == bench._source_digest(bench._kernel_sources(CSRC + KERNELS[stem][0]))


def test_digest_covers_the_formats_header():
    """A change of the MXFP4 device helpers is a change of the kernel that includes them."""
    assert bench._kernel_sources(CSRC + "mxfp4.hip") == [CSRC + f for f in ("mxfp4.hip", "device_common.h", "mxfp4_device.h")]
    assert bench._kernel_sources(CSRC + "gemm.hip") == [CSRC + "gemm.hip", CSRC + "device_common.h"]
