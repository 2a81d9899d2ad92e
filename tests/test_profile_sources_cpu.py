"""The bench reports a kernel's profiled DRAM traffic while the sources that
kernel is compiled from are those of its profile: its translation unit and
the headers it includes, not whatever else the library holds."""
import json
import os
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

HEADLINE = ["gemv_bf16_bf16_M1_K4096_N12288", "gemv_q8_0_bf16_M1_K4096_N12288", "gemv_q4_0_q8_1_M1_K4096_N12288",
            "gemm_q4_0_bf16_M512_K4096_N14336"]


@pytest.fixture
def csrc(tmp_path):
    return shutil.copytree(bench.CSRC, tmp_path / "csrc")


@pytest.mark.parametrize("key", HEADLINE)
def test_other_kernels_sources_leave_a_profile_valid(csrc, key):
    before = bench.source_hash(key, csrc)
    assert before == bench.source_hash(key)
    for name in ("attn_q8_0.cu", "bqg_attn.cuh", "bqg_attn_tc.cuh", "bqg_kv.cu", "bqg_kv.cuh", "bqg_layer.cu"):
        with open(csrc / name, "a") as f:
            f.write("// changed\n")
    (csrc / "another.cuh").write_text("// new\n")
    assert bench.source_hash(key, csrc) == before


@pytest.mark.parametrize("key,name", [(HEADLINE[0], "gemv_bf16.cu"), (HEADLINE[0], "bqg_gemv.cuh"), (HEADLINE[1], "bqg_common.cuh"),
                                      (HEADLINE[2], "bqg_gemv_mma.cuh"), (HEADLINE[3], "bqg_gemm.cu"), (HEADLINE[3], "bqg_tc.cuh")])
def test_its_own_sources_do_not(csrc, key, name):
    before = bench.source_hash(key, csrc)
    with open(csrc / name, "a") as f:
        f.write("// changed\n")
    assert bench.source_hash(key, csrc) != before


@pytest.mark.parametrize("key", json.load(open(os.path.join(ROOT, "profiles", "traffic.json"))))
def test_every_profiled_kernel_has_its_sources(key):
    assert len(bench.source_hash(key)) == 16
