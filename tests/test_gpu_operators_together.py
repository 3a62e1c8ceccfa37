"""The example that runs the operators together on one coded checkpoint, against the same step in plain fp32 and fp64 on
the decoded weights.  The hidden state and the gradient between the operators are bf16 (2^-9 of each value at most) and
the softmax multiplies what they err by; the gradients after them are allowed 3% in the 2-norm, and what does not pass
through them is compared closely."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
k3 = pytest.importorskip("lossless_bf16_weight_k3huf_gb300")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example():
    k3._build.build()
    spec = importlib.util.spec_from_file_location("example", os.path.join(ROOT, "examples", "adapters_on_coded_weights.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.main()
    table, w, head = (torch.from_numpy(t.view("int16")).cuda().view(torch.bfloat16).view(-1, m.WIDTH) for t in r["tensors"])
    x = (table[r["tokens"]].float() * torch.tensor(m.WIDTH ** 0.5, device="cuda")).to(torch.bfloat16)
    assert torch.equal(x, r["x"])
    a, b = (v.double().detach().requires_grad_() for v in (r["a"], r["b"]))
    rows = table.double().detach().requires_grad_()
    i = r["adapter"].long()
    on = (i >= 0).double()[:, None]
    xd = rows[r["tokens"]] * m.WIDTH ** 0.5

    def step(xin):
        low = torch.einsum("nc,nrc->nr", xin, a[i.clamp(min=0)]) * r["scales"].double()[i.clamp(min=0)][:, None] * on
        return xin @ w.double().T + torch.einsum("nr,nro->no", low, b[i.clamp(min=0)])

    y = step(x.double())
    assert float((r["y"].double() - y.detach()).norm() / y.detach().norm()) < 1e-5
    logp = torch.log_softmax(step(xd) @ head.double().T, 1).gather(1, r["wanted"][:, None]).sum()
    logp.backward()
    want = torch.log_softmax(r["logits"].double(), 1).gather(1, r["wanted"][:, None])[:, 0]
    assert float((r["logprob"].double() - want).abs().max()) < 1e-4
    for got, ref in ((r["da"], a.grad), (r["db"], b.grad), (r["drows"], rows.grad)):
        assert float((got.double() - ref).norm() / ref.norm()) < 0.03
