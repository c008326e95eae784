"""GPU: the bounded end of an SM pair whose CTAs stopped after different numbers of copies."""
import ctypes
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "microscaling_fp4_quantization_mxfp4_b200", "csrc")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("pair_settle") / "pair_settle.so")
    subprocess.run(["nvcc", "-O3", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-gencode", "arch=compute_100a,code=sm_100a",
                    "-I", CSRC, os.path.join(HERE, "cuda", "pair_settle.cu"), "-o", out], check=True, capture_output=True)
    lib = ctypes.CDLL(out)
    lib.pair_settle.argtypes = [ctypes.c_uint32] * 5 + [ctypes.c_void_p]
    return lib


@pytest.mark.parametrize("delay_ns", [0, 50000])
@pytest.mark.parametrize("slots, done", [(2, 0), (4, 4), (7, 3), (7, 15)])
def test_pair_settles(lib, slots, done, delay_ns):
    out = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for mine in range(done, done + slots + 1):
        for peers in range(done, done + slots + 1):
            out.zero_()
            torch.cuda.synchronize()
            assert lib.pair_settle(slots, done, mine, peers, delay_ns, out.data_ptr()) == 0
            torch.cuda.synchronize()
            assert int(out) == 1, (slots, done, mine, peers)
