"""Host-side behaviour of the paged-cache entry points (no GPU)."""
import os
import subprocess

from conftest import ROOT

PKG = os.path.join(ROOT, "movement_primitives_gb300")

FAILING_LAUNCH = r"""
#include <cuda_runtime.h>
static cudaError_t pending = cudaSuccess;
static cudaError_t fake_launch(const cudaLaunchConfig_t *, const void *, void **) {
    return pending = cudaErrorInvalidValue;
}
static cudaError_t fake_last() {
    const cudaError_t e = pending;
    pending = cudaSuccess;
    return e;
}
#define cudaLaunchKernelExC fake_launch
#define cudaGetLastError fake_last
#include "cache_common.cuh"
int main() {
    int arg = 0;
    if (lc::launch_after(nullptr, 1, 32, 0, nullptr, &arg) != LC_ERR_CUDA) return 1;
    return lc::finish_launch() == LC_OK ? 0 : 2;
}
"""


def test_a_failed_launch_leaves_no_error_for_the_next_call(tmp_path):
    """The runtime keeps a launch's error until it is read; the next call's check may not be the one that reads it."""
    from movement_primitives_gb300 import build
    src, exe = tmp_path / "launch.cu", tmp_path / "launch"
    src.write_text(FAILING_LAUNCH)
    subprocess.run([build.nvcc(), "-std=c++17", *build.ARCH, "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(PKG, "csrc"), str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
