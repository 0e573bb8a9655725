"""No GPU: the build refuses kernels that use local memory where they must not."""
import os

import pytest

from linear_attention_sequence_device_gb300 import build

SPILLS = """
// 64 values a thread live at the same time, in %d registers
__global__ void __launch_bounds__(1024, %d) many(const float* x, float* y) {
    float v[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = x[threadIdx.x + 1024 * i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 64; ++i) y[threadIdx.x + 1024 * i] = v[63 - i] * v[i];
}
"""
INDEXED = """
__global__ void indexed(const int* at, float* y) {
    float v[64];
    for (int i = 0; i < 64; ++i) v[i] = sinf((float)(i * at[0]));
    y[threadIdx.x] = v[at[threadIdx.x] & 63];
}
"""
CLEAN = "__global__ void clean(float* y) { y[threadIdx.x] *= 2.f; }"


@pytest.mark.parametrize("text", [SPILLS % (32, 2), INDEXED], ids=["spills", "indexed"])
def test_kernels_in_local_memory_do_not_build(tmp_path, text):
    src, obj = str(tmp_path / "vocab_loss.cu"), str(tmp_path / "x.o")
    with open(src, "w") as f:
        f.write(text)
    with pytest.raises(RuntimeError, match="local memory"):
        build.compile_unit(src, obj)
    assert not os.path.exists(obj)


def test_kernels_in_registers_build(tmp_path):
    src, obj = str(tmp_path / "vocab_loss.cu"), str(tmp_path / "x.o")
    with open(src, "w") as f:
        f.write(CLEAN)
    assert build.local_memory(build.compile_unit(src, obj)) == {} and os.path.exists(obj)


def test_the_product_kernel_is_in_registers(tmp_path):
    """Every instance of it is in the report that the build reads, without stack or spills."""
    out = build.compile_unit(os.path.join(build.CSRC, "vocab_loss.cu"), str(tmp_path / "x.o"))
    assert out.count("bytes stack frame") >= 20 and "vocab_gemm_kernel" in out
    assert build.local_memory(out) == {}


def test_report():
    out = ("ptxas info    : Compiling entry function 'f' for 'sm_103a'\nptxas info    : Function properties for f\n"
           "    8 bytes stack frame, 4 bytes spill stores, 12 bytes spill loads\n"
           "ptxas info    : Compiling entry function 'g' for 'sm_103a'\nptxas info    : Function properties for g\n"
           "    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads\n")
    assert build.local_memory(out) == {"f": (8, 4, 12)}
