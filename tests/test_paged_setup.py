"""What a call needs before its first launch, with the CUDA calls of the set-up
faked: no GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "long_context_exact_ring_gb300", "csrc")

# A compiler that gave the paged attention kernels too few registers, on a
# device where everything else succeeds.
PROGRAM = r"""
#include <cuda.h>
#include <cuda_runtime.h>
static int fake_device(int* d) { *d = 0; return 0; }
static void* fake_encoder;
static cudaError_t fake_entry(void** fn, cudaDriverEntryPointQueryResult* q)
{
    *fn = (void*)&fake_encoder;
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
static cudaError_t fake_address(void** a) { *a = (void*)&fake_encoder; return cudaSuccess; }
static cudaError_t fake_count(int* n) { *n = 152; return cudaSuccess; }
static cudaError_t fake_registers(cudaFuncAttributes* a) { *a = {}; a->numRegs = 100; return cudaSuccess; }
#define cudaGetDevice(d) (cudaError_t)fake_device(d)
#define cudaGetDriverEntryPointByVersion(name, fn, version, flags, q) fake_entry(fn, q)
#define cudaGetSymbolAddress(a, symbol) fake_address(a)
#define cudaDeviceGetAttribute(n, attribute, dev) fake_count(n)
#define cudaFuncSetAttribute(...) cudaSuccess
#define cudaFuncGetAttributes(a, ...) fake_registers(a)
#define cudaThreadExchangeStreamCaptureMode(m) (void)0
#include "ring_attn.cu"

int main()
{
    DeviceState* st = nullptr;
    // what the ring calls need
    if (device_state(&st) != RA_OK) { std::printf("ring calls: %s\n", g_last_error); return 1; }
    // the attention itself says so, before a launch
    char* x = (char*)(1 << 20);
    const int rc = paged_attn_fwd(x, nullptr, x, nullptr, x, nullptr, (int*)x, 8, (int*)x, (int*)x, x, nullptr, (float*)x,
                                  RA_BF16, 2, 4, 8, 2, 128, 32, 16, 8, 4, 1, 0.1f, x, (size_t)1 << 30, nullptr);
    if (rc != RA_ERR_CUDA || !std::strstr(g_last_error, "paged attention")) { std::printf("%d %s\n", rc, g_last_error); return 2; }
    return 0;
}
"""


def test_ring_calls_do_not_depend_on_the_paged_kernels(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src, exe = tmp_path / "setup.cu", tmp_path / "setup"
    src.write_text(PROGRAM)
    # device code is compiled no further than the host needs it
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=compute_103a", "-O0", "-std=c++17", "--expt-relaxed-constexpr",
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
