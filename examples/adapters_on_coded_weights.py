"""One decode step and one tuning step on a coded checkpoint.

The checkpoint (an embedding table, one projection, an output head) stays coded in device memory.  A batch of requests,
each with a low-rank adapter or none, goes through it:

    rows of the coded table -> coded projection + adapters -> coded head -> log probabilities of the next tokens

and the gradient of their sum goes back to the logits, the adapters and the embedding rows; the coded weights are frozen.

    python examples/adapters_on_coded_weights.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import lossless_bf16_weight_k3huf_gb300 as k3  # noqa: E402
import workloads  # noqa: E402

VOCAB, WIDTH, REQUESTS, ADAPTERS, RANK, TOP = 4096, 8192, 4, 3, 16, 5


def main():
    dev = torch.device("cuda", 0)
    # the checkpoint: tensor 0 the table, 1 the projection, 2 the head, each with a code table of its own
    tensors = [workloads.normal_tensor((VOCAB, WIDTH), 0.02, 1), workloads.normal_tensor((WIDTH, WIDTH), WIDTH ** -0.5, 2),
               workloads.normal_tensor((VOCAB, WIDTH), 0.05, 3)]
    blob = k3.encode_layer_gpu([torch.from_numpy(t.view(np.int16)).to(dev) for t in tensors])
    head = blob[: 1 << 16].cpu().numpy()
    hdr = head[: k3.layer_info(head)["hdr_bytes"]].copy()
    print(f"checkpoint: {sum(t.nbytes for t in tensors) / 1e6:.0f} MB of bf16, {blob.numel() / 1e6:.0f} MB coded")

    g = torch.Generator(device=dev).manual_seed(0)
    a = (torch.randn(ADAPTERS, RANK, WIDTH, generator=g, device=dev) * WIDTH ** -0.5).to(torch.bfloat16)
    b = (torch.randn(ADAPTERS, RANK, WIDTH, generator=g, device=dev) * 0.1).to(torch.bfloat16)
    scales = torch.full((ADAPTERS,), 2.0, device=dev)
    adapter = torch.tensor([0, 2, -1, 2], dtype=torch.int32, device=dev)      # the third request has none
    tokens = torch.tensor([17, 4000, 17, 9], device=dev)
    wanted = torch.tensor([5, 99, 1234, 7], device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)

    def floats(*shape):
        return torch.empty(*shape, device=dev)

    # forward
    x = torch.empty(REQUESTS, WIDTH, dtype=torch.bfloat16, device=dev)
    k3.embed_layer(hdr, blob, 0, WIDTH, tokens, x, status, scale=WIDTH ** 0.5)
    y = floats(REQUESTS, WIDTH)
    scratch = torch.empty(k3.adapter_scratch_bytes(REQUESTS, ADAPTERS, RANK, WIDTH, WIDTH, grad=True), dtype=torch.uint8, device=dev)
    k3.adapter_apply(x, a, b, adapter, scales, y, scratch, status)            # y = the adapters' part ...
    k3.gemv_layer_batch(hdr, blob, 1, WIDTH, x, y, status)                    # ... + W x, which accumulates
    h = y.to(torch.bfloat16)
    logits = floats(REQUESTS, VOCAB)
    k3.gemv_layer_batch(hdr, blob, 2, WIDTH, h, logits, status, zero_y=True)
    logprob, entropy, lse, top = floats(REQUESTS), floats(REQUESTS), floats(REQUESTS), floats(REQUESTS, TOP)
    top_ids = torch.empty(REQUESTS, TOP, dtype=torch.int32, device=dev)
    k3.token_logprobs(logits, wanted, logprob, status, entropy=entropy, lse=lse, top_ids=top_ids, top_logprobs=top)

    # backward: d(sum of log probabilities); the frozen weights are decoded where a product needs them whole
    def weight(t):
        info = k3.tensor_info(hdr, t)
        w = torch.empty(info["n_values"], dtype=torch.bfloat16, device=dev)
        k3.decode_tensor(hdr, blob, t, w, status)
        return w.view(-1, WIDTH)

    dlogits = torch.empty_like(logits)
    k3.token_logprobs_grad(logits, wanted, lse, torch.ones(REQUESTS, device=dev), dlogits, status)
    dy = (dlogits @ weight(2).float()).to(torch.bfloat16)
    da, db, dx = floats(*a.shape), floats(*b.shape), floats(REQUESTS, WIDTH)
    k3.adapter_grad(x, a, b, adapter, scales, dy, da, db, scratch, status, dx=dx, dx_base=dy.float() @ weight(1).float())
    drows = floats(VOCAB, WIDTH)
    grad_scratch = torch.empty(k3.embed_grad_scratch_bytes(REQUESTS, VOCAB, WIDTH), dtype=torch.uint8, device=dev)
    k3.embed_grad(tokens, dx, drows, grad_scratch, status, scale=WIDTH ** 0.5)

    torch.cuda.synchronize()
    assert status.item() == 0, f"status {status.item()}"
    for i in range(REQUESTS):
        print(f"request {i}: adapter {adapter[i].item():2d}  log p {logprob[i].item():8.3f}  entropy {entropy[i].item():6.3f}  "
              f"top {top_ids[i].tolist()}")
    print(f"gradient norms: a {da.norm().item():.4g}, b {db.norm().item():.4g}, table {drows.norm().item():.4g}")
    return {"x": x, "y": y, "logits": logits, "logprob": logprob, "da": da, "db": db, "drows": drows, "tokens": tokens, "adapter": adapter,
            "a": a, "b": b, "scales": scales, "tensors": tensors, "wanted": wanted}


if __name__ == "__main__":
    main()
