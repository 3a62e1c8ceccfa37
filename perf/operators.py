"""Cases of the operators that stand next to the coded weights: rows of a coded embedding table with their gradient, the
low-rank adapters of many requests beside a shared projection with theirs, and the log probabilities of given tokens,
with entropy and top alternatives, with theirs.

`own` false computes them in their plain form, elementary torch operations in 32 bits; `own` true makes the calls that
a user of the package makes.  A frozen checkpoint is kept coded, so with `own` true the embedding table is encoded when
it is prepared, once, as it would be when the checkpoint is loaded; everything else is the same tensors on both sides."""
import math

import torch

own = False

_BF16, _F32 = "bf16", "f32"
_TYPES = {_BF16: torch.bfloat16, _F32: torch.float32}


def listed():
    return [
        # one decode step of 32 requests: the new tokens' rows of a coded table, as wide as the trunk's 8192 columns
        {"name": "embed decode 32", "op": "embed", "n": 32, "vocab": 32768, "cols": 8192, "out": _BF16},
        # a narrow table (the trunk's 576 columns) whose rows start anywhere in a chunk, an odd vocabulary, fp32 out
        {"name": "embed 1001x576 fp32", "op": "embed", "n": 1001, "vocab": 50021, "cols": 576, "out": _F32},
        # a prefill or a training step's lookup
        {"name": "embed prefill 8192", "op": "embed", "n": 8192, "vocab": 65536, "cols": 8192, "out": _BF16},
        # a small step of tuning adds into the gradient that it holds, from pass to pass
        {"name": "embed grad 515 add", "op": "embed_grad", "n": 515, "vocab": 32003, "cols": 2048, "dy": _F32, "add": True},
        # a training step writes the whole table's gradient
        {"name": "embed grad 8192", "op": "embed_grad", "n": 8192, "vocab": 32768, "cols": 8192, "dy": _BF16, "add": False},
        # decode steps: every request has its adapter (or none); fp32 beside the fp32 output of the coded projection
        {"name": "adapter decode 4", "op": "adapter", "n": 4, "adapters": 8, "rank": 16, "cols": 8192, "rows": 8192, "y": _F32},
        {"name": "adapter decode 192", "op": "adapter", "n": 192, "adapters": 64, "rank": 16, "cols": 8192, "rows": 8192, "y": _F32},
        # a prefill of a few long requests into the trunk's widest projection
        {"name": "adapter prefill 8192", "op": "adapter", "n": 8192, "adapters": 6, "rank": 64, "cols": 8192, "rows": 24576, "y": _BF16},
        # a tuning step: gradients of both factors and of the input, an odd number of tokens
        {"name": "adapter grad 4099", "op": "adapter_grad", "n": 4099, "adapters": 4, "rank": 32, "cols": 8192, "rows": 8192, "y": _BF16},
        # one decode step of 8 requests, the answer's log probabilities with alternatives
        {"name": "logprob decode 8", "op": "logprob", "n": 8, "vocab": 131072, "top": 8, "x": _F32, "banned": 0.1},
        # scoring a long text
        {"name": "logprob score 4095", "op": "logprob", "n": 4095, "vocab": 131072, "top": 20, "x": _BF16, "banned": 0.0},
        # the gradient of a policy's log probabilities and entropy
        {"name": "logprob grad 2047", "op": "logprob_grad", "n": 2047, "vocab": 131072, "x": _BF16, "banned": 0.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "adapter", "adapter", "adapter_grad", "logprob", "logprob_grad"])
    if op in ("embed", "embed_grad"):
        cols = _log(rng, 128, 16384)
        if rng.random() < 0.8:
            cols = -(-cols // 8) * 8
        if op == "embed":
            vocab = _log(rng, 1000, min(131072, (1 << 29) // cols))
            return {"op": op, "n": min(_log(rng, 1, 16384), (1 << 26) // cols), "vocab": vocab, "cols": cols, "out": rng.choice([_BF16, _F32])}
        vocab = _log(rng, 1000, min(131072, (1 << 28) // cols))
        return {"op": op, "n": min(_log(rng, 1, 16384), (1 << 26) // cols), "vocab": vocab, "cols": cols, "dy": rng.choice([_BF16, _F32]), "add": rng.random() < 0.4}
    if op in ("adapter", "adapter_grad"):
        cols, rows = (8 * _log(rng, 64, 1024 if op == "adapter_grad" else 2048) for _ in range(2))
        rank = rng.choice([4, 8, 12, 16, 16, 32, 32, 64, 64, 128])
        n = _log(rng, 1, 4096) if op == "adapter" else _log(rng, 16, 4096)
        adapters = _log(rng, 1, 32 if n > 256 else 128)
        return {"op": op, "n": n, "adapters": max(1, min(adapters, 2048 // rank)), "rank": rank, "cols": cols, "rows": rows, "y": rng.choice([_BF16, _F32])}
    vocab = _log(rng, 1000, 160000)
    n = max(1, min(_log(rng, 1, 8192), (1 << 28) // vocab))
    c = {"op": op, "n": n, "vocab": vocab, "x": rng.choice([_BF16, _F32]), "banned": rng.choice([0.0, 0.1, 0.9])}
    if op == "logprob":
        c["top"] = rng.choice([0, 1, 5, 8, 20, 32])
    return c


def _tokens(g, n, vocab):
    """Token ids with the long-tailed counts of text: the logarithm of the id is uniform."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(vocab)).long() - 1).clamp_(0, vocab - 1)


def _inputs(case, seed):
    """What both sides start from, made on the GPU from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=_BF16):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(_TYPES[dtype])

    op, n = case["op"], case["n"]
    if op == "embed":
        vocab, cols = case["vocab"], case["cols"]
        table = torch.randn(vocab, cols, generator=g, device="cuda", dtype=torch.float32)
        table.mul_(torch.exp(math.log(0.02) + 0.5 * torch.randn(vocab, 1, generator=g, device="cuda")))
        return {"table": table.to(torch.bfloat16), "ids": _tokens(g, n, vocab), "scale": math.sqrt(cols)}
    if op == "embed_grad":
        vocab, cols = case["vocab"], case["cols"]
        s = {"ids": _tokens(g, n, vocab), "dy": normal(n, cols, std=0.01, dtype=case["dy"]), "scale": math.sqrt(cols)}
        if case["add"]:
            s["held"] = normal(vocab, cols, std=0.1, dtype=_F32)
        return s
    if op in ("adapter", "adapter_grad"):
        S, r, cols, rows = case["adapters"], case["rank"], case["cols"], case["rows"]
        # -1 is a token whose request has no adapter; long inputs are runs of tokens of one request, short ones a decode
        # step's requests in the order they came
        if n > 256:
            cuts = torch.randint(0, n, (2 * S,), generator=g, device="cuda")
            run_of = (torch.arange(n, device="cuda")[:, None] >= cuts.sort().values[None, :]).sum(1)
            ids = torch.randint(-1, S, (2 * S + 1,), generator=g, device="cuda")[run_of]
        else:
            ids = torch.randint(-1, S, (n,), generator=g, device="cuda")
        s = {"ids": ids.to(torch.int32), "x": normal(n, cols), "a": normal(S, r, cols, std=cols ** -0.5), "b": normal(S, r, rows, std=r ** -0.5),
             "scales": torch.rand(S, generator=g, device="cuda") * 1.5 + 0.5}
        if op == "adapter":
            s["base"] = normal(n, rows, dtype=case["y"])
        else:
            s["dy"] = normal(n, rows, std=0.05)
            s["dx_base"] = normal(n, cols, std=0.05, dtype=case["y"])
        return s
    vocab = case["vocab"]
    x = normal(n, vocab, std=3.0, dtype=case["x"])
    if case["banned"]:
        # tokens that a constraint bans: every row keeps at least one
        ban = torch.rand(n, vocab, generator=g, device="cuda") < case["banned"]
        ban[:, vocab // 2] = False
        x.masked_fill_(ban, -math.inf)
        del ban
    tokens = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    tokens = torch.where(torch.rand(n, generator=g, device="cuda") < 0.5, x.argmax(1), tokens)  # half of them likely ones
    tokens = torch.where(x.gather(1, tokens[:, None])[:, 0] == -math.inf, torch.full_like(tokens, vocab // 2), tokens)
    tokens[(torch.rand(n, generator=g, device="cuda") < 0.03)] = -1  # places of the text that are not scored
    s = {"x": x, "tokens": tokens, "scale": 0.8}
    if op == "logprob_grad":
        # what the forward pass kept: the log of the sum of exponentials and the entropy
        xs = x.float() * s["scale"]
        s["lse"] = torch.logsumexp(xs, 1)
        p = torch.exp(xs - s["lse"][:, None])
        s["entropy"] = s["lse"] - torch.where(p > 0, p * xs, torch.zeros_like(p)).sum(1)
        s["g_logprob"] = torch.randn(n, generator=g, device="cuda")
        s["g_entropy"] = torch.randn(n, generator=g, device="cuda") * 0.01
        del xs, p
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op, n = case["op"], case["n"]
    s["case"] = case
    if not own:
        return s
    import lossless_bf16_weight_k3huf_gb300 as k3

    def out(*shape, dtype=_F32):
        return torch.empty(*shape, device="cuda", dtype=dtype if isinstance(dtype, torch.dtype) else _TYPES[dtype])

    # the buffers that a user's program keeps from step to step: outputs, the status word, scratch
    s["k3"], s["status"] = k3, torch.zeros(1, dtype=torch.int32, device="cuda")
    if op == "embed":
        s["blob"] = k3.encode_layer_gpu([s.pop("table")])
        head = s["blob"][: 1 << 16].cpu().numpy()
        s["hdr"] = head[: k3.layer_info(head)["hdr_bytes"]].copy()
        s["y"] = out(n, case["cols"], dtype=case["out"])
    elif op == "embed_grad":
        s["grad"] = s["held"] if case["add"] else out(case["vocab"], case["cols"])
        s["scratch"] = out(k3.embed_grad_scratch_bytes(n, case["vocab"], case["cols"]), dtype=torch.uint8)
    elif op == "adapter":
        s["y"] = out(n, case["rows"], dtype=case["y"])
        s["scratch"] = out(k3.adapter_scratch_bytes(n, case["adapters"], case["rank"], case["cols"], case["rows"]), dtype=torch.uint8)
    elif op == "adapter_grad":
        s["dx"] = out(n, case["cols"], dtype=case["y"])
        s["da"], s["db"] = (out(*s[k].shape) for k in ("a", "b"))
        s["scratch"] = out(k3.adapter_scratch_bytes(n, case["adapters"], case["rank"], case["cols"], case["rows"], grad=True), dtype=torch.uint8)
    elif op == "logprob":
        s["logprob"], s["entropy"], s["lse"] = out(n), out(n), out(n)
        if case["top"]:
            s["top_ids"], s["top_logprobs"] = out(n, case["top"], dtype=torch.int32), out(n, case["top"])
    else:
        s["dx"] = out(n, case["vocab"], dtype=case["x"])
    return s


def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s, s["case"])


def _run_own(s):
    k3, op = s["k3"], s["case"]["op"]
    if op == "embed":
        k3.embed_layer(s["hdr"], s["blob"], 0, s["case"]["cols"], s["ids"], s["y"], s["status"], scale=s["scale"])
        return s["y"]
    if op == "embed_grad":
        k3.embed_grad(s["ids"], s["dy"], s["grad"], s["scratch"], s["status"], scale=s["scale"], accumulate=s["case"]["add"])
        return s["grad"]
    if op == "adapter":
        k3.adapter_apply(s["x"], s["a"], s["b"], s["ids"], s["scales"], s["y"], s["scratch"], s["status"], base=s["base"])
        return s["y"]
    if op == "adapter_grad":
        k3.adapter_grad(s["x"], s["a"], s["b"], s["ids"], s["scales"], s["dy"], s["da"], s["db"], s["scratch"], s["status"], dx=s["dx"], dx_base=s["dx_base"])
        return {"da": s["da"], "db": s["db"], "dx": s["dx"]}
    if op == "logprob":
        k3.token_logprobs(s["x"], s["tokens"], s["logprob"], s["status"], entropy=s["entropy"], lse=s["lse"],
                          top_ids=s.get("top_ids"), top_logprobs=s.get("top_logprobs"), scale=s["scale"])
        return {k: s[k] for k in ("logprob", "entropy", "lse", "top_ids", "top_logprobs") if k in s}
    k3.token_logprobs_grad(s["x"], s["tokens"], s["lse"], s["g_logprob"], s["dx"], s["status"], entropy=s["entropy"],
                           g_entropy=s["g_entropy"], scale=s["scale"])
    return s["dx"]


# ---- the plain forms -----------------------------------------------------------------------------------------------

def _plain_embed(s, c):
    return (s["table"][s["ids"]].float() * s["scale"]).to(_TYPES[c["out"]])


def _plain_embed_grad(s, c):
    grad = s["held"] if c["add"] else torch.zeros(c["vocab"], c["cols"], device="cuda")
    return grad.index_add_(0, s["ids"], s["dy"].float() * s["scale"])


def _shrink(v, w, ids, S, r):
    """v times every adapter's factor, kept where the token's own adapter is."""
    h = v.float() @ w.float().view(S * r, -1).T
    mine = ids[:, None] == torch.arange(S, device="cuda").repeat_interleave(r)[None, :]
    return torch.where(mine, h, torch.zeros_like(h))


def _plain_adapter(s, c):
    S, r = c["adapters"], c["rank"]
    h = _shrink(s["x"], s["a"], s["ids"], S, r) * s["scales"].repeat_interleave(r)
    return (s["base"].float() + h @ s["b"].float().view(S * r, -1)).to(_TYPES[c["y"]])


def _plain_adapter_grad(s, c):
    S, r = c["adapters"], c["rank"]
    each = s["scales"].repeat_interleave(r)
    h = _shrink(s["x"], s["a"], s["ids"], S, r) * each
    dh = _shrink(s["dy"], s["b"], s["ids"], S, r) * each
    dx = s["dx_base"].float() + dh @ s["a"].float().view(S * r, -1)
    return {"da": (dh.T @ s["x"].float()).view(S, r, -1), "db": (h.T @ s["dy"].float()).view(S, r, -1), "dx": dx.to(_TYPES[c["y"]])}


def _plain_logprob(s, c):
    x = s["x"].float()
    xs = x * s["scale"]
    m = xs.amax(1, keepdim=True)
    e = torch.exp(xs - m)
    total = e.sum(1, keepdim=True)
    lse = (m + torch.log(total))[:, 0]
    p = e / total
    entropy = -torch.where(p > 0, p * (xs - lse[:, None]), torch.zeros_like(p)).sum(1)
    scored = s["tokens"] >= 0
    at = xs.gather(1, s["tokens"].clamp(min=0)[:, None])[:, 0]
    got = {"logprob": torch.where(scored, at - lse, torch.zeros_like(at)), "entropy": entropy, "lse": lse}
    if c["top"]:
        # larger values first, ties to the lower index: one whole number holds both
        bits = (x + 0.0).view(torch.int32)
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
        key = order * 4294967296 + (c["vocab"] - 1 - torch.arange(c["vocab"], device="cuda"))
        top = c["vocab"] - 1 - (key.topk(c["top"], dim=1).values & 0xFFFFFFFF)
        got["top_ids"] = top.to(torch.int32)
        got["top_logprobs"] = xs.gather(1, top) - lse[:, None]
    return got


def _plain_logprob_grad(s, c):
    lp = s["x"].float() * s["scale"] - s["lse"][:, None]
    p = torch.exp(lp)
    scored = s["tokens"] >= 0
    g = torch.where(scored, s["g_logprob"], torch.zeros_like(s["g_logprob"]))[:, None]
    gh = s["g_entropy"][:, None]
    d = torch.where(p > 0, -p * (g + gh * (lp + s["entropy"][:, None])), torch.zeros_like(p))
    d.scatter_add_(1, s["tokens"].clamp(min=0)[:, None], g)
    return (d * s["scale"]).to(_TYPES[c["x"]])


_PLAIN = {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "adapter": _plain_adapter, "adapter_grad": _plain_adapter_grad,
          "logprob": _plain_logprob, "logprob_grad": _plain_logprob_grad}


# ---- what a pass cannot do without ---------------------------------------------------------------------------------

def _used(count, kinds):
    """Kinds that `count` equal draws from `kinds` are expected to meet."""
    return kinds * (1.0 - (1.0 - 1.0 / kinds) ** count)


def work(case):
    op, n = case["op"], case["n"]
    if op in ("embed", "embed_grad"):
        vocab, cols = case["vocab"], case["cols"]
        # ids with a uniform logarithm: id i has probability log((i + 2) / (i + 1)) / log(vocab)
        rows = sum(1.0 - (1.0 - math.log1p(1.0 / (i + 1)) / math.log(vocab)) ** n for i in range(vocab))
        if op == "embed":
            # a coded value of such a table takes about 10.9 bits
            return {"bytes": 8 * n + rows * cols * 1.36 + n * cols * (2 if case["out"] == _BF16 else 4), "flops": n * cols}
        held = 2 * rows * cols * 4 if case["add"] else vocab * cols * 4
        return {"bytes": 8 * n + n * cols * (2 if case["dy"] == _BF16 else 4) + held, "flops": 2 * n * cols}
    if op in ("adapter", "adapter_grad"):
        S, r, cols, rows = case["adapters"], case["rank"], case["cols"], case["rows"]
        kinds = _used(2 * S if n > 256 else n, S) * r * (cols + rows)
        y = 2 if case["y"] == _BF16 else 4
        if op == "adapter":
            return {"bytes": 4 * n + 2 * n * cols + 2 * kinds + 2 * y * n * rows, "flops": 2 * n * r * (cols + rows)}
        return {"bytes": 4 * n + 2 * n * (cols + rows) + 2 * kinds + 2 * y * n * cols + 4 * S * r * (cols + rows), "flops": 2 * n * r * (3 * cols + 2 * rows)}
    vocab, w = case["vocab"], 2 if case["x"] == _BF16 else 4
    if op == "logprob":
        return {"bytes": n * (vocab * w + 20 + 8 * case["top"]), "flops": 6 * n * vocab}
    return {"bytes": n * (2 * vocab * w + 24), "flops": 8 * n * vocab}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def exact(case, seed):
    s, op, n = _inputs(case, seed), case["op"], case["n"]
    if op == "embed":
        return s["table"].index_select(0, s["ids"]).double() * s["scale"]
    if op == "embed_grad":
        want = s["held"].double() if case["add"] else torch.zeros(case["vocab"], case["cols"], dtype=torch.float64, device="cuda")
        kinds, place = torch.unique(s["ids"], return_inverse=True)
        sums = torch.zeros(len(kinds), case["cols"], dtype=torch.float64, device="cuda")
        sums.index_add_(0, place, s["dy"].double())
        want[kinds] += sums * s["scale"]
        return want
    if op in ("adapter", "adapter_grad"):
        y = s["base"].double() if op == "adapter" else s["dx_base"].double()
        da, db = (torch.zeros(s[k].shape, dtype=torch.float64, device="cuda") for k in ("a", "b"))
        for i in range(case["adapters"]):
            t = (s["ids"] == i).nonzero()[:, 0]
            if not len(t):
                continue
            scale, x, a, b = s["scales"][i].double(), s["x"][t].double(), s["a"][i].double(), s["b"][i].double()
            if op == "adapter":
                y[t] += scale * ((x @ a.T) @ b)
                continue
            dy = s["dy"][t].double()
            dh = scale * (dy @ b.T)
            y[t] += dh @ a
            da[i], db[i] = dh.T @ x, scale * ((x @ a.T).T @ dy)
        return y if op == "adapter" else {"da": da, "db": db, "dx": y}
    parts = []
    for i in range(0, n, 256):  # 256 rows at a time
        z = s["x"][i: i + 256].double() * s["scale"]
        logp = torch.log_softmax(z, 1)
        p = logp.exp()
        t = s["tokens"][i: i + 256]
        plogp = torch.where(p > 0, p * logp, torch.zeros_like(p))
        h = -plogp.sum(1)
        if op == "logprob":
            lp = torch.where(t >= 0, logp.gather(1, t.clamp(min=0)[:, None])[:, 0], torch.zeros_like(h))
            parts.append((lp, h, torch.logsumexp(z, 1)) + ((logp.topk(case["top"], dim=1).values,) if case["top"] else ()))
            continue
        g = torch.where(t >= 0, s["g_logprob"][i: i + 256], torch.zeros_like(s["g_logprob"][i: i + 256])).double()[:, None]
        d = -p * g - s["g_entropy"][i: i + 256].double()[:, None] * (plogp + p * h[:, None])
        d.scatter_add_(1, t.clamp(min=0)[:, None], g)
        parts.append((d * s["scale"],))
    whole = [torch.cat(v) for v in zip(*parts)]
    if op == "logprob_grad":
        return whole[0]
    got = dict(zip(("logprob", "entropy", "lse", "top_logprobs"), whole))
    return {**got, "top_ids": None} if case["top"] else got
