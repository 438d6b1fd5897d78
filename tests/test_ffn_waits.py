"""Barrier waits of the tensor-core kernels are given up after two seconds.  What
takes longer without anything being broken must not count."""
import ctypes
import os
import subprocess

import pytest
import torch

import ffn_ref as R

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def early_producer(tmp_path_factory):
    from moe_deferred_finalize_gb300 import build
    so = str(tmp_path_factory.mktemp("producer") / "early_producer.so")
    subprocess.run([build._nvcc(), "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-shared",
                    "-Xcompiler", "-fPIC", os.path.join(HERE, "early_producer.cu"), "-o", so],
                   check=True, capture_output=True)
    fn = ctypes.CDLL(so).early_producer
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64,
                   ctypes.c_void_p]
    return fn


def rand(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(shape, dtype=BF16, device="cuda").normal_(0.0, scale, generator=g)


@pytest.mark.parametrize("T,N,K", [(64, 264, 8192), (2000, 1000, 264)])
def test_a_long_kernel_in_front_is_no_lost_wait(cuda_lib, early_producer, T, N, K):
    """A kernel that opens its dependent launch at once and then runs for 2.5
    seconds on one SM: the product starts beside it on the others and waits.
    k in parts on single CTAs; pairs."""
    x, w = rand(1, T, K), rand(2, N, K, scale=K ** -0.5)
    late = torch.zeros_like(x)
    cuda_lib.linear(late, w)
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    assert early_producer(late.data_ptr(), x.data_ptr(), x.numel(), 2_500_000_000, stream) == 0
    got = cuda_lib.linear(late, w)
    assert cuda_lib.lost_waits() == 0
    R.check(got, R.linear(x, w))
