"""How a product is cut on devices that differ, against a CUDA runtime that answers for them (no GPU: launches are noted,
not made, and no device is visible).  The cut decides the order of a result's sums, so it may depend on the device of
the call and on nothing that was asked before."""
import os
import subprocess
import sys

import pytest

k3 = pytest.importorskip("lossless_bf16_weight_k3huf_gb300")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RUNTIME = r"""
#include <cuda.h>
#include <cuda_runtime_api.h>
static int device, fail;
extern "C" {
int noted[2];
void use(int dev, int failing) { device = dev, fail = failing; }
cudaError_t cudaGetDevice(int *d) { *d = device; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, enum cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *, enum cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
// device 0 has room for a cluster wherever it has SMs; device 1 for a third of those, device 2 for none but small ones
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *, const cudaLaunchConfig_t *c) {
    if (fail) return cudaErrorUnknown;
    const int size = int(c->attrs[0].val.clusterDim.x);
    *n = device == 0 ? 152 / size : device == 1 ? 50 / size : size <= 2 ? 152 / size : 1;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *, void **) {
    noted[0] = int(c->gridDim.x), noted[1] = c->numAttrs ? int(c->attrs[0].val.clusterDim.x) : 0;
    return cudaSuccess;
}
static CUresult encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                       CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) { return CUDA_SUCCESS; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **f, unsigned int, unsigned long long, cudaDriverEntryPointQueryResult *r) {
    *f = (void *)encode, *r = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
}
"""

CALLS = """
import ctypes, sys
import lossless_bf16_weight_k3huf_gb300 as k3
fake, lib, P = ctypes.CDLL(sys.argv[1]), k3._lib(), 1 << 20
assert ctypes.cast(ctypes.CDLL(None).cudaLaunchKernelExC, ctypes.c_void_p).value == ctypes.cast(fake.cudaLaunchKernelExC, ctypes.c_void_p).value
noted = (ctypes.c_int * 2).in_dll(fake, "noted")
for step in sys.argv[2:]:
    dev, _, failing = step.partition("!")
    fake.use(int(dev), int(failing or 0))
    for n, rows, cols in ((186, 3176, 9960), (100, 1000, 4096), (300, 2000, 8192), (3, 8192, 8192)):
        assert lib.k3huf_linear(P, cols, n, 2 * P, cols, rows, cols, None, 0, 0, None, 0, 3 * P, rows, 1, None, 0, 0, None, 0, 4 * P, None) == 0
        print(step, n, *noted)
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    k3._build.build()
    where = tmp_path_factory.mktemp("runtime")
    (where / "runtime.cpp").write_text(RUNTIME)
    so = str(where / "runtime.so")
    subprocess.run(["g++", "-shared", "-fPIC", "-I", os.path.join(k3._build._cuda_home(), "include"), str(where / "runtime.cpp"), "-o", so], check=True)

    def run(*steps):
        """Cuts by step: device, or device!1 where the query for its clusters fails."""
        out = subprocess.run([sys.executable, "-c", CALLS, so, *steps], cwd=ROOT, check=True, capture_output=True, text=True, env={**os.environ, "LD_PRELOAD": so, "CUDA_VISIBLE_DEVICES": ""}).stdout
        cuts = [[] for _ in steps]
        for k, line in enumerate(out.splitlines()):
            cuts[k // 4].append(line.split()[1:])
        return cuts

    return run


def test_a_cut_depends_on_its_device_alone(run):
    alone = [run(d)[0] for d in "012"]
    assert alone[0] != alone[1] and alone[1] != alone[2] and alone[0] != alone[2]
    assert run("0", "1", "2", "0") == [*alone, alone[0]]
    assert run("2", "1", "0", "2") == [*alone[::-1], alone[2]]


def test_a_query_that_fails_is_asked_again(run):
    assert run("2!1", "2", "2!1")[1:] == [run("2")[0]] * 2


def test_devices_beyond_those_that_are_kept(run):
    """Their SMs were taken for one, and the cut divided by the pairs that one SM makes."""
    assert run("70") == run("2") and run("1", "70", "0", "70")[1::2] == run("2") * 2
