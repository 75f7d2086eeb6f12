"""One report does not hide another: the device error word keeps a bit for each kind."""
import os
import subprocess

import pytest
import torch

import workloads
import weight_only_quantization_rtn_b200 as w4
from weight_only_quantization_rtn_b200 import build as w4build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_both_kinds_in_one_word(tmp_path):
    exe = tmp_path / "device_errors"
    subprocess.check_call([w4build.nvcc(), *w4build.ARCH, "-O2", "-std=c++17", "--expt-relaxed-constexpr", "-o", str(exe),
                           os.path.join(HERE, "device_errors.cu")])
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_bad_ids_of_many_calls_are_one_report():
    w4build.build()
    w = w4.quantize(workloads.make_weight(10, 64, 0.02, 1).cuda(), 64, False)
    ids = torch.tensor([3, 10, 11, 12], device="cuda")
    for _ in range(3):
        w4.embedding(ids, *w, g=64)
        w4.embedding_grad(torch.ones(4, 64, dtype=torch.bfloat16, device="cuda"), ids, 10)
    assert w4.device_error() == 2 and w4.device_error() == 0
