"""A launch that fails returns its error once: the operators whose launches are checked by the runtime's last error must not
find it there afterwards.  (A launch with more threads than a block may have never reaches the GPU: the host refuses it.)"""
import subprocess

import pytest

from gpu_util import need_gpu
from sparse_mla_decode_combine_gb300 import build as b

pytestmark = pytest.mark.gpu

PROGRAM = r"""
#include <cstdio>
#include "fp4.h"
struct Params { int n; };
__global__ void kernel(const Params p) { (void)p; }
int main()
{
    const Params p{1};
    (void)cudaGetLastError();
    const cudaError_t e = dsv4::launch_dependent(kernel, dim3(1), 4096, 0, nullptr, p);
    const cudaError_t left = cudaPeekAtLastError();
    std::printf("%d %d\n", (int)(e != cudaSuccess), (int)left);
    return 0;
}
"""


def test_a_failed_launch_leaves_no_error_behind(tmp_path):
    need_gpu()
    src = tmp_path / "launch.cu"
    src.write_text(PROGRAM)
    exe = str(tmp_path / "launch")
    subprocess.run([b._nvcc(), *b.ARCH, "-std=c++17", "-I", b.CSRC, str(src), "-o", exe], check=True, capture_output=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()
    assert out == ["1", "0"]
