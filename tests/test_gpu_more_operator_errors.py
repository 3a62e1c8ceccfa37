"""Launches that the CUDA runtime refuses, for the products, the control of logits and distillation: an error of the call
and nothing left behind, as for the operators beside them."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
k3 = pytest.importorskip("lossless_bf16_weight_k3huf_gb300")

from test_gpu_operator_errors import empty, runtime  # noqa: E402,F401

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
BF = torch.bfloat16


def calls():
    st = empty(1, dtype=torch.int32)
    made = {}

    def product(name, n, rows, cols):
        x, w, y, dz = empty(n, cols, dtype=BF), empty(rows, cols, dtype=BF), empty(n, rows), empty(n, rows, dtype=BF)
        sc = empty(k3.linear_scratch_bytes(n, rows, cols, grad=True), dtype=torch.uint8)
        dx, dw = empty(n, cols), empty(rows, cols)
        made["linear " + name] = lambda s: k3.linear(x, w, y, st, scratch=sc, stream=s)
        made["linear_grad " + name] = lambda s: k3.linear_grad(x, w, dz, st, dx=dx, dw=dw, scratch=sc, stream=s)

    product("few", 3, 128, 256)
    product("pair", 600, 1024, 256)
    product("odd", 40, 100, 77)
    z, dz, bias = empty(40, 100, dtype=BF), empty(40, 100, dtype=BF), empty(100)
    x, o, lp, ids, t = empty(3, 5000), empty(3, 5000), empty(3), empty(3, 4, dtype=torch.int32), empty(3, 4)
    many, many_out = empty(200, 300), empty(200, 300)
    history = torch.zeros(10, dtype=torch.int64, device="cuda")
    spans, more = torch.tensor([[0, 3, 9]] * 3, device="cuda"), torch.tensor([[0, 3, 9]] * 200, device="cuda")
    made["linear_dz"] = lambda s: k3.linear_dz(z, z, dz, act="silu", dbias=bias, stream=s)
    made["control few"] = lambda s: k3.logits_control(x, o, st, history=history, spans=spans, stream=s)
    made["control many"] = lambda s: k3.logits_control(many, many_out, st, history=history, spans=more, stream=s)
    most = 2 * torch.cuda.get_device_properties(0).multi_processor_count + 9
    rows, rows_out, of_rows = empty(most, 300, dtype=BF), empty(most, 300), torch.tensor([[0, 3, 9]] * most, device="cuda")
    made["control in two launches"] = lambda s: k3.logits_control(rows, rows_out, st, history=history, spans=of_rows, stream=s)
    made["distill"] = lambda s: k3.distill(x, ids, t, lp, st, stream=s)
    made["distill_grad"] = lambda s: k3.distill_grad(x, ids, t, lp, lp, o, st, stream=s)
    return made


@pytest.mark.parametrize("name", ["linear few", "linear_grad few", "linear pair", "linear_grad pair", "linear odd", "linear_grad odd", "linear_dz", "control few",
                                  "control many", "distill", "distill_grad"])
def test_a_refused_launch_leaves_no_error_behind(runtime, name):  # noqa: F811
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


def test_a_refused_launch_of_two_leaves_no_error_behind(runtime):  # noqa: F811
    test_a_refused_launch_leaves_no_error_behind(runtime, "control in two launches")
