"""A wait of the norm kernels' row feed that runs out is reported and ends the block's rows; it
does not go on with what lies in shared memory."""
import ctypes
import os
import subprocess

import pytest
import torch

from activation_implicit_gemm_gb300 import _build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    so = str(tmp_path_factory.mktemp("probe") / "row_feed_probe.so")
    subprocess.check_call([_build.nvcc(), *_build.ARCH, "-O3", "-std=c++17", "-shared",
                           "-Xcompiler", "-fPIC", "-I", os.path.join(_build.ROOT, "include"),
                           os.path.join(HERE, "row_feed_probe.cu"), "-o", so])
    return ctypes.CDLL(so)


def run(probe, rows, asked):
    x = torch.randn(rows, 64, device="cuda")
    y = torch.full((rows, 64), 7.0, device="cuda")
    ok = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    args = [ctypes.c_void_p(t.data_ptr()) for t in (x, y, ok)]
    assert probe.run_probe(*args, rows, asked) == 0
    words = []
    for _ in range(2):
        word = ctypes.c_uint(99)
        assert probe.read_probe(ctypes.byref(word)) == 0
        words.append(word.value)
    return x, y, ok.tolist(), words


def test_rows_that_were_asked_for(probe):
    x, y, ok, words = run(probe, 37, 2)
    assert torch.equal(x, y) and ok == [1, 1] and words == [0, 0]


def test_a_wait_that_runs_out(probe):
    x, y, ok, words = run(probe, 7, 1)
    assert ok == [1, 0] and words == [1, 0]  # reported once
    assert torch.equal(x[::2], y[::2]) and (y[1::2] == 7.0).all()
    x, y, ok, words = run(probe, 9, 2)  # the device goes on as before
    assert torch.equal(x, y) and ok == [1, 1] and words == [0, 0]
