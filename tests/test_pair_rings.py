"""What the waits of gemm_pair_kernel's dequantizing warps rest on, walked through on the host
with the kernel's own plan, walk and ring sizes (pair_rings.cu): no GPU needed."""
import os
import subprocess

import pytest

from weight_only_quantization_rtn_b200 import build as w4build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = tmp_path_factory.mktemp("rings") / "pair_rings"
    subprocess.check_call([w4build.nvcc(), *w4build.ARCH, "-O2", "-std=c++17", "--expt-relaxed-constexpr", "-o", str(exe),
                           os.path.join(HERE, "pair_rings.cu")])
    return str(exe)


def test_every_wait_knows_the_phase_before(walk):
    r = subprocess.run([walk], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_walk_finds_turns_that_start_anew(walk):
    """Groups that begin every segment with their own k-th block may wait a ring's length too far."""
    r = subprocess.run([walk, "1"], capture_output=True, text=True)
    assert r.returncode == 1 and "A slot" in r.stdout, r.stdout


def test_decode_shares_and_ready_flags(tmp_path):
    exe = tmp_path / "decode_shares"
    subprocess.check_call([w4build.nvcc(), *w4build.ARCH, "-O2", "-std=c++17", "--expt-relaxed-constexpr", "-o", str(exe),
                           os.path.join(HERE, "decode_shares.cu")])
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
