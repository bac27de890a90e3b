"""The work list of the ragged attention kernel (csrc/kvq_ragged_plan.h, the same
header that the kernel includes), checked on random batches on the host: costs
and prefixes in closed form against sums block by block, the steps of a block
against the tokens that its rows attend (windows, rows before the context's
start), and the shares: every step of every block in exactly one piece, the
pieces of a block in adjacent CTAs, at most one unfinished piece at either end
of a share (the two places that a CTA has in the workspace).
"""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "int8_quantized_paged_quantize_b200", "csrc")


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    out = str(tmp_path_factory.mktemp("native") / "ragged_plan_check")
    subprocess.run([gxx, "-O2", "-std=c++17", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover", "-I", CSRC,
                    "-o", out, os.path.join(HERE, "native", "ragged_plan_check.cpp")], check=True)
    return out


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_random_batches(exe, seed):
    p = subprocess.run([exe, str(seed), "1500"], capture_output=True, text=True)
    assert p.returncode == 0, p.stdout + p.stderr
    ok, pieces, cut = p.stdout.split()
    assert ok == "ok" and int(pieces) > 10000 and int(cut) > 1000
