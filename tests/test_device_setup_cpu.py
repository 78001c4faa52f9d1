"""The library's set-up of a device, on the host: an operator that the device
cannot hold is refused alone.  The API's own sources, with a device that the
test makes up and stand-ins for the kernels' files."""
import subprocess

import pytest

from mixture_experts_ffn_gate_gb300 import _build

pytestmark = pytest.mark.cpu

SOURCE = r"""
#include <cuda_runtime.h>
#include <stdio.h>
static cudaError_t one_device(int *d) { *d = 0; return cudaSuccess; }
static cudaError_t attribute(int *v, cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
#define cudaGetDevice one_device
#define cudaDeviceGetAttribute attribute
#include "moe_ffn_api.cu"
static int g_pairs, g_gate, g_ortho;
namespace moe {
cudaError_t routing_init_device() { return cudaSuccess; }
cudaError_t decode_init_device() { return cudaSuccess; }
cudaError_t decode_fused_init_device() { return cudaSuccess; }
cudaError_t gemm_init_device() { return cudaSuccess; }
cudaError_t bwd_init_device() { return cudaSuccess; }
cudaError_t ortho_init_device(int *pairs)
{
    *pairs = g_pairs;
    return g_pairs < 0 ? cudaErrorInvalidValue : cudaSuccess;
}
size_t ortho_workspace_bytes(int64_t, int64_t, int64_t) { return 256; }
cudaError_t launch_gate(const GateCall &, int, cudaStream_t) { ++g_gate; return cudaSuccess; }
cudaError_t launch_orthogonalize(const OrthoCall &, void *, int, cudaStream_t) { ++g_ortho; return cudaSuccess; }
}
int main(int argc, char **argv)
{
    g_pairs = argv[1][0] == '-' ? -1 : argv[1][0] - '0';
    void *const p = (void *)0x10000;
    const int gate = moe_gate_forward((float *)p, nullptr, 4, 16, 2, nullptr, (int32_t *)p, (float *)p, nullptr, nullptr);
    const int ortho = moe_orthogonalize(p, MOE_F32, 1, 64, 64, 5, 3.4445f, -4.775f, 2.0315f, 1e-7f, 1.0f, p, p, 256,
                                        nullptr);
    printf("%d %d %d %d", gate, g_gate, ortho, g_ortho);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("setup")
    (d / "api.cu").write_text(SOURCE)
    flags = [_build._nvcc(), *_build.ARCH, "-O0", "-std=c++17", "--expt-relaxed-constexpr", "-w", "-I", _build.INCLUDE, "-I",
             _build.CSRC]
    objs = []
    for src in (d / "api.cu", f"{_build.CSRC}/moe_block_api.cu"):
        objs.append(str(d / f"{len(objs)}.o"))
        subprocess.run([*flags, "-c", str(src), "-o", objs[-1]], check=True)
    subprocess.run([_build._nvcc(), *_build.ARCH, "-cudart", "static", *objs, "-o", str(d / "setup"), "-Xlinker",
                    "--unresolved-symbols=ignore-all"], check=True)
    return str(d / "setup")


@pytest.mark.parametrize("pairs,ortho", [("2", "0 1"), ("0", "3 0"), ("-", "3 0")])
def test_only_the_orthogonalisation_needs_a_pair(program, pairs, ortho):
    """The gate runs (status 0, one launch) whatever the pairs; without one,
    or where they cannot be found out, the orthogonalisation is refused (MOE_ERR_CUDA)."""
    out = subprocess.run([program, pairs], check=True, capture_output=True, text=True).stdout
    assert out == f"0 1 {ortho}"
