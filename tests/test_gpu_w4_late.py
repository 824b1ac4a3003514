"""4-bit products behind a kernel that lets them start early and then runs for longer than their own waits last."""
import ctypes
import subprocess

import pytest
import torch

import q8_block_quantized_gemv_gb300 as q8
from q8_block_quantized_gemv_gb300 import build as q8build

pytestmark = pytest.mark.gpu

# Triggers its dependents at once, ends after `clocks` of its SM, and only then writes the activations.
LATE = r"""
#include <cuda_runtime.h>
__global__ void late(const uint4 *from, uint4 *to, int count, long long clocks) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long t0 = clock64();
    while (clock64() - t0 < clocks) __nanosleep(1000);
    for (int i = threadIdx.x; i < count; i += blockDim.x) to[i] = from[i];
}
extern "C" int run_late(const void *from, void *to, int bytes, long long clocks, void *stream) {
    late<<<1, 256, 0, (cudaStream_t)stream>>>((const uint4 *)from, (uint4 *)to, bytes / 16, clocks);
    return (int)cudaGetLastError();
}
"""
CLOCKS = 4_600_000_000  # 2.2 seconds at 2.07 GHz; the products wait for 4e9


@pytest.fixture(scope="module")
def late(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    q8build.build()
    at = tmp_path_factory.mktemp("late")
    (at / "late.cu").write_text(LATE)
    subprocess.run([q8build.nvcc(), *q8build.ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", str(at / "late.so"), str(at / "late.cu")],
                   check=True, capture_output=True)
    lib = ctypes.CDLL(str(at / "late.so"))
    lib.run_late.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p]
    yield lib
    assert q8.device_fault(clear=True) == 0


@pytest.mark.parametrize("m,K,constant", [(3, 1024, True), (40, 1024, False), (40, 4096, True), (200, 8192, True)])
def test_products_wait_for_a_late_kernel(late, m, K, constant):
    N, group = 300, 64
    g = torch.Generator("cuda").manual_seed(m)
    codes = torch.randint(0, 256, (K // 2, N), dtype=torch.uint8, device="cuda", generator=g)
    w = q8.Weight4(codes, (torch.rand((K // group, N), device="cuda", generator=g) * 0.02).half())
    x = torch.randn((m, K), device="cuda", generator=g).bfloat16()
    want = q8.gemv4(x, w)
    to = torch.zeros_like(x)
    y = torch.full_like(want, 7.0)
    late.run_late(x.data_ptr(), to.data_ptr(), 16, 0, torch.cuda.current_stream().cuda_stream)  # loaded before it counts
    torch.cuda.synchronize()
    assert late.run_late(x.data_ptr(), to.data_ptr(), x.numel() * 2, CLOCKS, torch.cuda.current_stream().cuda_stream) == 0
    q8.gemv4(to, w, y=y, constant_weights=constant)
    torch.cuda.synchronize()
    assert q8.device_fault() == 0 and torch.equal(y, want)
