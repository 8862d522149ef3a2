"""The debug build (every kernel checks its global addresses against the operands
that the host validated) passes the tests of the operators around a layer's
products with a clean device status, in a child process that loads it."""

import os
import subprocess
import sys

import pytest

from strided_gemm_gb300 import build as sgbuild

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CASES = ["test_quantise_against_the_definition", "test_fp8_sizes", "test_fp8_layouts_alpha_accumulate_and_sharing",
         "test_rope_against_64_bits", "test_rope_in_place", "test_workspaces_are_kept_to", "test_shared_against_64_bits",
         "test_shared_by_many", "test_shared_strided_operands", "test_a_decode_step_of_forked_sequences"]


def test_debug_build_passes_the_layers_cases_with_clean_status():
    path = sgbuild.build(debug=True)
    env = dict(os.environ, SBGEMM_LIBRARY=path, SBGEMM_CHECK_STATUS="1")
    code = ("import strided_gemm_gb300 as sg, sys; "
            f"assert sg.LIB_PATH == {path!r}, sg.LIB_PATH; "
            "import pytest; sys.exit(pytest.main(sys.argv[1:]))")
    r = subprocess.run([sys.executable, "-c", code, *(f"tests/test_layers_gpu.py::{c}" for c in CASES), "-m", "gpu", "-x",
                        "-q", "-p", "no:cacheprovider"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert " passed" in out and " failed" not in out, out[-2000:]
