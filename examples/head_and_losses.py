"""From decoded weights to logits, the next token's choice, and a step of distillation.

A checkpoint (a projection with adapters, a block with its activation and residual, a head) is coded; a step over
many tokens decodes each weight before it uses it:

    tokens -> projection + adapters -> block: act(x W^T + bias) + x -> head -> logits
    serving: the last tokens' logits, controlled (penalties, biases, a grammar's mask), scored with alternatives
    tuning:  a teacher's alternatives -> loss of the student's logits -> gradients back through head, block and adapters

    python examples/head_and_losses.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import lossless_bf16_weight_k3huf_gb300 as k3  # noqa: E402
import workloads  # noqa: E402

TOKENS, WIDTH, VOCAB, ADAPTERS, RANK, REQUESTS, TOP, SCALE = 160, 1024, 5003, 3, 8, 4, 12, 0.9
BF = torch.bfloat16


def main():
    dev = torch.device("cuda", 0)
    tensors = [workloads.normal_tensor((WIDTH, WIDTH), WIDTH ** -0.5, 1), workloads.normal_tensor((WIDTH, WIDTH), WIDTH ** -0.5, 2),
               workloads.normal_tensor((VOCAB, WIDTH), 1.5 * WIDTH ** -0.5, 3)]
    blob = k3.encode_layer_gpu([torch.from_numpy(t.view(np.int16)).to(dev) for t in tensors])
    first = blob[: 1 << 16].cpu().numpy()
    hdr = first[: k3.layer_info(first)["hdr_bytes"]].copy()
    status = torch.zeros(1, dtype=torch.int32, device=dev)

    def weight(t):
        w = torch.empty(k3.tensor_info(hdr, t)["n_values"], dtype=BF, device=dev)
        k3.decode_tensor(hdr, blob, t, w, status)
        return w.view(-1, WIDTH)

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device=dev)

    g = torch.Generator(device=dev).manual_seed(0)

    def normal(*shape, std=1.0, dtype=BF):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    x, bias = normal(TOKENS, WIDTH), normal(WIDTH, std=0.3, dtype=torch.float32)
    a, b = normal(ADAPTERS, RANK, WIDTH, std=WIDTH ** -0.5), normal(ADAPTERS, RANK, WIDTH, std=0.2)
    scales = torch.full((ADAPTERS,), 2.0, device=dev)
    adapter = torch.randint(-1, ADAPTERS, (TOKENS,), generator=g, device=dev).to(torch.int32)
    scratch = empty(k3.adapter_scratch_bytes(TOKENS, ADAPTERS, RANK, WIDTH, WIDTH, grad=True), dtype=torch.uint8)

    # forward: every product over all tokens, the block's z kept for its gradient
    u, v, z = empty(TOKENS, WIDTH, dtype=BF), empty(TOKENS, WIDTH, dtype=BF), empty(TOKENS, WIDTH, dtype=BF)
    k3.linear(x, weight(0), u, status)
    k3.adapter_apply(x, a, b, adapter, scales, u, scratch, status, base=u)
    k3.linear(u, weight(1), v, status, bias=bias, act="silu", residual=u, z=z)
    logits = empty(TOKENS, VOCAB)
    k3.linear(v, weight(2), logits, status)

    # serving: the last tokens of four requests
    chosen = logits[-REQUESTS:].clone()
    history = torch.randint(0, VOCAB, (60,), generator=g, device=dev)
    spans = torch.tensor([[0, 5, 20], [20, 30, 30], [30, 40, 60], [60, 60, 60]], device=dev)
    penalty = torch.full((REQUESTS,), 1.3, device=dev)
    words = torch.randint(-2 ** 31, 2 ** 31 - 1, (2, (VOCAB + 31) // 32), generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    state = torch.tensor([0, -1, 1, 0], dtype=torch.int32, device=dev)
    banned = torch.tensor([7, 9], device=dev)
    k3.logits_control(chosen, chosen, status, history=history, spans=spans, repetition=penalty, frequency=penalty - 1.0, bias_ids=banned,
                      bias_values=torch.full((2,), -float("inf"), device=dev), bias_spans=torch.tensor([[0, 2]] * REQUESTS, device=dev), mask=words, mask_rows=state)
    next_ids, next_lp, lp = empty(REQUESTS, TOP, dtype=torch.int32), empty(REQUESTS, TOP), empty(REQUESTS)
    k3.token_logprobs(chosen, torch.full((REQUESTS,), -1, device=dev), lp, status, top_ids=next_ids, top_logprobs=next_lp)

    # tuning: a teacher's alternatives, the loss, and the gradients; the coded weights are frozen
    teacher = logits + normal(TOKENS, VOCAB, std=0.7, dtype=torch.float32)
    top_ids, top_lp, unscored = empty(TOKENS, TOP, dtype=torch.int32), empty(TOKENS, TOP), torch.full((TOKENS,), -1, device=dev)
    k3.token_logprobs(teacher, unscored, empty(TOKENS), status, top_ids=top_ids, top_logprobs=top_lp, scale=SCALE)
    loss, lse, log_rest = empty(TOKENS), empty(TOKENS), empty(TOKENS)
    k3.distill(logits, top_ids, top_lp, loss, status, lse=lse, log_rest=log_rest, mode="rest", scale=SCALE)
    dlogits = empty(TOKENS, VOCAB)
    k3.distill_grad(logits, top_ids, top_lp, lse, torch.ones(TOKENS, device=dev), dlogits, status, log_rest=log_rest, mode="rest", scale=SCALE)

    def back(w, dz):
        dx = empty(TOKENS, WIDTH)
        k3.linear_grad(None, w, dz, status, dx=dx, scratch=empty(k3.linear_scratch_bytes(TOKENS, w.shape[0], WIDTH, grad=True), dtype=torch.uint8))
        return dx

    dv = back(weight(2), dlogits.to(BF))
    dz, dbias = empty(TOKENS, WIDTH, dtype=BF), empty(WIDTH)
    k3.linear_dz(z, dv, dz, act="silu", dbias=dbias)
    du = (back(weight(1), dz) + dv).to(BF)                                  # ... and the residual's
    da, db, dx = empty(*a.shape), empty(*b.shape), empty(TOKENS, WIDTH)
    k3.adapter_grad(x, a, b, adapter, scales, du, da, db, scratch, status, dx=dx, dx_base=back(weight(0), du))

    torch.cuda.synchronize()
    assert status.item() == 0, f"status {status.item()}"
    for r in range(REQUESTS):
        print(f"request {r}: best tokens {next_ids[r, :4].tolist()}  log p {[round(v, 3) for v in next_lp[r, :4].tolist()]}")
    print(f"mean loss {loss.mean().item():.5f}; gradient norms: a {da.norm().item():.4g}, b {db.norm().item():.4g}, bias {dbias.norm().item():.4g}, "
          f"input {dx.norm().item():.4g}")
    return {"tensors": tensors, "x": x, "bias": bias, "a": a, "b": b, "scales": scales, "adapter": adapter, "logits": logits, "teacher": teacher, "top_ids": top_ids,
            "top_lp": top_lp, "loss": loss, "da": da, "db": db, "dbias": dbias, "dx": dx, "chosen": chosen, "history": history, "spans": spans, "penalty": penalty,
            "words": words, "state": state, "next_ids": next_ids, "next_lp": next_lp}


if __name__ == "__main__":
    main()
