"""A launch that the CUDA runtime refuses comes back as an error of the call, and as nothing else: the runtime's own
record of it is cleared, so the next user of CUDA in the process does not meet it.  The refusal is made on the host:
while a blocking stream is being captured, the runtime takes no launch on the default stream."""
import ctypes
import glob
import os

import pytest

import oracle
import workloads

torch = pytest.importorskip("torch")
k3 = pytest.importorskip("lossless_bf16_weight_k3huf_gb300")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.fixture(scope="module")
def runtime():
    """The CUDA runtime that the library is linked with."""
    k3._build.build()
    k3._lib()
    with open("/proc/self/maps") as f:
        used = {line.split()[-1] for line in f if "libcudart" in line}
    for path in sorted(used):
        if os.path.dirname(path) in {os.path.dirname(os.path.realpath(p)) for p in glob.glob("/usr/local/cuda*/lib64/libcudart.so*")}:
            return ctypes.CDLL(path)
    return ctypes.CDLL(sorted(used)[0])


def empty(*shape, dtype=torch.float32):
    return torch.zeros(*shape, device="cuda", dtype=dtype)


def calls():
    st = empty(1, dtype=torch.int32)
    ids = torch.tensor([1, 0, 2], device="cuda")
    blob = oracle.encode_layer([workloads.normal_tensor((10, 64), 0.02, 3)])
    hdr, layer, rows = blob[: k3.layer_info(blob)["hdr_bytes"]], torch.from_numpy(blob).cuda(), empty(3, 64, dtype=torch.bfloat16)
    table, scratch = empty(10, 64), empty(k3.embed_grad_scratch_bytes(2000, 10, 64), dtype=torch.uint8)
    many, dy = torch.zeros(2000, dtype=torch.int64, device="cuda"), empty(2000, 64)
    x, lp = empty(3, 500), empty(3)

    def adapters(n, rank, cols, rows, grad):
        bf = torch.bfloat16
        v, a, b = empty(n, cols, dtype=bf), empty(2, rank, cols, dtype=bf), empty(2, rank, rows, dtype=bf)
        i, scales, y = empty(n, dtype=torch.int32), empty(2), empty(n, rows, dtype=bf)
        sc = empty(k3.adapter_scratch_bytes(n, 2, rank, cols, rows, grad=grad), dtype=torch.uint8)
        if not grad:
            return lambda s: k3.adapter_apply(v, a, b, i, scales, y, sc, st, stream=s)
        da, db, dx = empty(*a.shape), empty(*b.shape), empty(n, cols)
        return lambda s: k3.adapter_grad(v, a, b, i, scales, y, da, db, sc, st, dx=dx, stream=s)

    return {"embed_layer": lambda s: k3.embed_layer(hdr, layer, 0, 64, ids, rows, st, stream=s),
            "embed_grad few": lambda s: k3.embed_grad(ids, dy[:3], table, scratch, st, accumulate=True, stream=s),
            "embed_grad": lambda s: k3.embed_grad(many, dy, table, scratch, st, stream=s),
            "adapter_apply few": adapters(3, 8, 64, 32, False), "adapter_apply any": adapters(3, 8, 63, 31, False),
            "adapter_apply tiles": adapters(2100, 64, 1024, 1032, False), "adapter_grad": adapters(200, 16, 64, 128, True),
            "token_logprobs": lambda s: k3.token_logprobs(x, ids, lp, st, stream=s),
            "token_logprobs_grad": lambda s: k3.token_logprobs_grad(x, ids, lp, lp, x, st, stream=s)}


@pytest.mark.parametrize("name", ["embed_layer", "embed_grad few", "embed_grad", "adapter_apply few", "adapter_apply any", "adapter_apply tiles",
                                  "adapter_grad", "token_logprobs", "token_logprobs_grad"])
def test_a_refused_launch_leaves_no_error_behind(runtime, name):
    call = calls()[name]
    call(0)
    torch.cuda.synchronize()
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert runtime.cudaStreamCreate(ctypes.byref(stream)) == 0
    try:
        assert runtime.cudaStreamBeginCapture(stream, 0) == 0
        try:
            with pytest.raises(k3.K3HufError) as e:
                call(0)
            left = runtime.cudaPeekAtLastError()
        finally:
            runtime.cudaStreamEndCapture(stream, ctypes.byref(graph))
    finally:
        runtime.cudaStreamDestroy(stream)
        runtime.cudaGetLastError()                       # (the capture's own)
    assert e.value.code == k3.E_CUDA and left == 0
    call(0)
    torch.cuda.synchronize()
