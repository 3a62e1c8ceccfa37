"""The example that runs the products, the control of logits and distillation together, against the same step in 64 bits on
the decoded weights.  What passes between the operators is bf16 (2^-9 of each value at most, several times over), and the
softmax multiplies what it errs by: the gradients are allowed 4% in the 2-norm; what does not pass through bf16 tensors of
this step is compared closely."""
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
    spec = importlib.util.spec_from_file_location("head_example", os.path.join(ROOT, "examples", "head_and_losses.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.main()
    w0, w1, w2 = (torch.from_numpy(t.view("int16")).cuda().view(torch.bfloat16).view(-1, m.WIDTH).double() for t in r["tensors"])
    x, a, b, bias = (r[k].double().detach().requires_grad_() for k in ("x", "a", "b", "bias"))
    i = r["adapter"].long()
    on = (i >= 0).double()[:, None]
    low = torch.einsum("nc,nrc->nr", x, a[i.clamp(min=0)]) * r["scales"].double()[i.clamp(min=0)][:, None] * on
    u = x @ w0.T + torch.einsum("nr,nro->no", low, b[i.clamp(min=0)])
    v = torch.nn.functional.silu(u @ w1.T + bias) + u
    logits = v @ w2.T
    assert float((r["logits"].double() - logits.detach()).norm() / logits.detach().norm()) < 0.01
    # the loss of the step's own logits, closely; and the whole step's gradients
    ids, t = r["top_ids"].long(), r["top_lp"].double()

    def loss_of(z):
        logp = torch.log_softmax(z * m.SCALE, 1)
        q = t.exp()
        rest = 1 - q.sum(1)
        taken = torch.zeros_like(logp, dtype=torch.bool).scatter_(1, ids, True)
        return (q * (t - logp.gather(1, ids))).sum(1) + rest * (torch.log(rest) - torch.logsumexp(logp.masked_fill(taken, -float("inf")), 1))

    assert float((r["loss"].double() - loss_of(r["logits"].double())).abs().max()) < 2e-6
    loss_of(logits).sum().backward()
    for got, ref in ((r["da"], a.grad), (r["db"], b.grad), (r["dbias"], bias.grad), (r["dx"], x.grad)):
        assert float((got.double() - ref).norm() / ref.norm()) < 0.04
    # the controlled logits and their alternatives
    c = r["logits"][-m.REQUESTS:].double().clone()
    for k, (lo, split, hi) in enumerate(r["spans"].tolist()):
        seen = torch.unique(r["history"][lo:hi])
        c[k, seen] = torch.where(c[k, seen] > 0, c[k, seen] / 1.3, c[k, seen] * 1.3)
        kinds, times = torch.unique(r["history"][split:hi], return_counts=True)
        c[k, kinds] -= 0.3 * times
        c[k, [7, 9]] = -float("inf")
        if int(r["state"][k]) >= 0:
            j = torch.arange(m.VOCAB, device="cuda")
            c[k, ((r["words"][int(r["state"][k])].long()[j // 32] >> (j % 32)) & 1) == 0] = -float("inf")
    assert torch.equal(torch.isinf(c), torch.isinf(r["chosen"]))
    fine = torch.isfinite(c)
    assert float((r["chosen"].double() - c)[fine].abs().max()) < 1e-5
    want = torch.log_softmax(r["chosen"].double(), 1).topk(m.TOP, dim=1)
    assert torch.equal(want.indices.int(), r["next_ids"]) and float((want.values - r["next_lp"]).abs().max()) < 1e-5
