"""Cases of the operators from a decoded weight to its logits and what is done with them: the matrix product with bias,
activation and residual in its epilogue (the many-token companion of the coded matrix-vector product, the base that the
adapters add to) with its gradients, the control of logits before a token is chosen (penalties for repeated tokens,
biases, grammar masks), and distillation from a teacher's top log probabilities with its gradient.

`own` false computes them in their plain form, elementary torch operations in 32 bits; `own` true makes the calls that
a user of the package makes.  Both start from the same tensors."""
import math

import torch

own = False

_BF16, _F32 = "bf16", "f32"
_TYPES = {_BF16: torch.bfloat16, _F32: torch.float32}
_ACTS = ("none", "relu", "silu", "gelu")


def listed():
    return [
        # a decode step of three requests through one square projection of the trunk, the residual stream in fp32
        {"name": "linear decode 3", "op": "linear", "n": 3, "rows": 8192, "cols": 8192, "act": "none", "bias": "", "res": True, "z": False, "y": _F32},
        # a short prompt through the trunk's narrow input, an odd number of tokens, its activation, z kept for the backward pass
        {"name": "linear 777 silu", "op": "linear", "n": 777, "rows": 8192, "cols": 576, "act": "silu", "bias": _BF16, "res": False, "z": True, "y": _BF16},
        # a prefill through the trunk's widest projection
        {"name": "linear prefill 8192", "op": "linear", "n": 8192, "rows": 24576, "cols": 8192, "act": "gelu", "bias": _F32, "res": False, "z": False, "y": _BF16},
        # a tuning step of that projection: what the activation passes back, and the bias's gradient
        {"name": "linear grad silu 4095", "op": "linear_grad", "n": 4095, "rows": 24576, "cols": 0, "act": "silu", "y": _BF16, "add": False},
        # ... and the two products behind it, at a square projection of the trunk
        {"name": "linear grad 4096", "op": "linear_grad", "n": 4096, "rows": 8192, "cols": 8192, "act": "none", "y": _BF16, "add": False},
        # one decode step of 8 requests: penalties and biases where the logits lie
        {"name": "control decode 8", "op": "control", "n": 8, "vocab": 131072, "x": _F32, "y": "", "history": 4000, "drafts": 1, "bias": 50, "allowed": 0.0, "id": "i32"},
        # drafted tokens of 15 requests, four rows each over one history, under a grammar, an odd vocabulary
        {"name": "control drafts 60", "op": "control", "n": 60, "vocab": 50021, "x": _BF16, "y": _F32, "history": 1500, "drafts": 4, "bias": 20, "allowed": 0.05, "id": "i64"},
        # a large batch of structured answers
        {"name": "control batch 1024", "op": "control", "n": 1024, "vocab": 131072, "x": _BF16, "y": _BF16, "history": 3000, "drafts": 1, "bias": 100, "allowed": 0.9, "id": "i32"},
        # a small step of a small student, the teacher's alternatives taken as the whole distribution
        {"name": "distill 33", "op": "distill", "n": 33, "vocab": 32003, "x": _F32, "top": 8, "mode": "normalised"},
        # a training step's texts: 20 alternatives and the rest of the mass
        {"name": "distill 4095", "op": "distill", "n": 4095, "vocab": 131072, "x": _BF16, "top": 20, "mode": "rest"},
        # gradients: fp32 logits of an odd vocabulary, and a training step's
        {"name": "distill grad 515", "op": "distill_grad", "n": 515, "vocab": 50021, "x": _F32, "top": 32, "mode": "given"},
        {"name": "distill grad 2047", "op": "distill_grad", "n": 2047, "vocab": 131072, "x": _BF16, "top": 20, "mode": "rest"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "control", "control", "distill", "distill_grad"])
    if op in ("linear", "linear_grad"):
        rows, cols = _log(rng, 64, 24576), _log(rng, 64, 16384)
        if rng.random() < 0.75:
            rows, cols = -(-rows // 8) * 8, -(-cols // 8) * 8
        n = max(1, min(_log(rng, 1, 8192), (1 << 37) // (rows * cols)))
        act, y = rng.choice(_ACTS), rng.choice([_BF16, _F32])
        if op == "linear":
            return {"op": op, "n": n, "rows": rows, "cols": cols, "act": act, "bias": rng.choice(["", _BF16, _F32]), "res": rng.random() < 0.5,
                    "z": act != "none" and rng.random() < 0.5, "y": y}
        if rng.random() < 0.4:
            return {"op": op, "n": n, "rows": rows, "cols": 0, "act": rng.choice(_ACTS[1:]), "y": y, "add": rng.random() < 0.3}
        return {"op": op, "n": n, "rows": rows, "cols": cols, "act": "none", "y": y, "add": rng.random() < 0.3}
    vocab = _log(rng, 1000, 160000)
    x = rng.choice([_BF16, _F32])
    if op == "control":
        n = max(1, min(_log(rng, 1, 1024), (1 << 27) // vocab))
        return {"op": op, "n": n, "vocab": vocab, "x": x, "y": rng.choice(["", _BF16, _F32]), "history": min(_log(rng, 1, 32768), (1 << 23) // n),
                "drafts": rng.choice([1, 1, 4, 5]), "bias": rng.choice([0, 10, 300]), "allowed": rng.choice([0.0, 0.02, 0.5, 0.98]), "id": rng.choice(["i32", "i64"])}
    n = max(1, min(_log(rng, 1, 8192), (1 << 28) // vocab))
    return {"op": op, "n": n, "vocab": vocab, "x": x, "top": rng.choice([1, 5, 8, 20, 32, 64]), "mode": rng.choice(["given", "normalised", "rest"])}


def _inputs(case, seed):
    """What both sides start from, made on the GPU from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=_BF16):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(_TYPES[dtype])

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def tokens(n, vocab):
        """Token ids with the long-tailed counts of text: the logarithm of the id is uniform."""
        u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
        return (torch.exp(u * math.log(vocab)).long() - 1).clamp_(0, vocab - 1)

    op, n = case["op"], case["n"]
    if op == "linear":
        rows, cols = case["rows"], case["cols"]
        s = {"x": normal(n, cols), "w": normal(rows, cols, std=cols ** -0.5)}
        if case["bias"]:
            s["bias"] = normal(rows, std=0.5, dtype=case["bias"])
        if case["res"]:
            s["res"] = normal(n, rows, dtype=case["y"])
        return s
    if op == "linear_grad":
        rows, cols = case["rows"], case["cols"]
        if not cols:
            s = {"z": normal(n, rows), "dy": normal(n, rows, std=0.05, dtype=case["y"])}
            if case["add"]:
                s["held"] = normal(rows, dtype=_F32)
            return s
        s = {"x": normal(n, cols), "w": normal(rows, cols, std=cols ** -0.5), "dz": normal(n, rows, std=0.05)}
        if case["add"]:
            s["held"] = normal(rows, cols, std=0.1, dtype=_F32)
        return s
    vocab = case["vocab"]
    if op == "control":
        ids = torch.int32 if case["id"] == "i32" else torch.int64
        s = {"x": normal(n, vocab, std=3.0, dtype=case["x"])}
        # requests with histories of their own lengths, some of them new; drafted rows see a few tokens more than the one before
        reqs, row = -(-n // case["drafts"]), torch.arange(n, device="cuda")
        length = (uniform(reqs) * case["history"] * (uniform(reqs) < 0.95)).long() + case["drafts"]
        end = length.cumsum(0)
        begin = (end - length)[row // case["drafts"]]
        upto = end[row // case["drafts"]] - case["drafts"] + 1 + row % case["drafts"]
        split = begin + ((upto - begin) * uniform(n)).long()
        s["history"] = tokens(int(end[-1]), vocab).to(ids)
        s["spans"] = torch.stack([begin, split, upto], 1).contiguous()
        s["repetition"] = 1.0 + 0.3 * uniform(n)
        s["frequency"], s["presence"] = uniform(n) * 0.5, uniform(n) * 0.8
        if case["bias"]:
            # ids of a row differ
            step = max(1, vocab // case["bias"])
            place = torch.arange(case["bias"], device="cuda") * step + torch.randint(0, step, (n, 1), generator=g, device="cuda")
            s["bias_ids"] = place[:, : vocab // step].reshape(-1).to(ids)
            per = s["bias_ids"].numel() // n
            s["bias_values"] = torch.randn(n * per, generator=g, device="cuda") * 5.0
            s["bias_spans"] = torch.stack([row * per, (row + 1) * per], 1).contiguous()
        if case["allowed"]:
            # grammar states that rows share; some rows are free
            states = min(n, 64)
            words = (vocab + 31) // 32
            bits = (uniform(states, words * 32) < case["allowed"]).view(states, words, 32).long()
            packed = (bits << torch.arange(32, device="cuda")).sum(2)
            s["mask"] = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).to(torch.int32)
            state = torch.randint(0, states, (n,), generator=g, device="cuda")
            s["mask_rows"] = torch.where(uniform(n) < 0.1, torch.full_like(state, -1), state).to(torch.int32)
        return s
    x = normal(n, vocab, std=3.0, dtype=case["x"])
    s = {"x": x, "scale": 0.8}
    teacher = x.float().mul_(0.9)
    teacher.add_(torch.randn(n, vocab, generator=g, device="cuda"), alpha=0.7).mul_(s["scale"])
    # the teacher's logits themselves where its alternatives are taken as the whole, else its log probabilities
    top, ids = teacher.topk(case["top"], dim=1)
    if case["mode"] != "normalised":
        top = top - torch.logsumexp(teacher, 1, keepdim=True)
    del teacher
    ids = ids.to(torch.int32)
    # texts of several lengths: rows of no token, and rows with fewer alternatives
    keep = (uniform(n) * 1.1 * case["top"]).long() + 1
    keep[uniform(n) < 0.03] = 0
    ids[torch.arange(case["top"], device="cuda")[None, :] >= keep[:, None]] = -1
    s["top_ids"], s["top"] = ids, top.contiguous()
    if op == "distill_grad":
        # what the forward pass kept
        s["lse"], s["log_rest"] = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        for i in range(0, n, 512):
            z = x[i: i + 512].double() * s["scale"]
            lse = torch.logsumexp(z, 1)
            at = ids[i: i + 512].long()
            z.scatter_(1, at.clamp(min=0), torch.where(at < 0, z.gather(1, at.clamp(min=0)), torch.full_like(at, -math.inf, dtype=torch.float64)))
            # (a padded place may have put back the first token's logit: take it out again where it is one of the row's)
            first = (at == 0).any(1)
            z[:, 0] = torch.where(first, torch.full_like(lse, -math.inf), z[:, 0])
            s["lse"][i: i + 512] = lse
            s["log_rest"][i: i + 512] = torch.logsumexp(z, 1) - lse
        s["g"] = torch.randn(n, generator=g, device="cuda")
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
    if op == "linear":
        s["y"] = out(n, case["rows"], dtype=case["y"])
        if case["z"]:
            s["z"] = out(n, case["rows"], dtype=_BF16)
        s["scratch"] = out(k3.linear_scratch_bytes(n, case["rows"], case["cols"]), dtype=torch.uint8)
    elif op == "linear_grad" and not case["cols"]:
        s["dz"] = out(n, case["rows"], dtype=_BF16)
        s["dbias"] = s["held"] if case["add"] else out(case["rows"])
    elif op == "linear_grad":
        s["dx"] = out(n, case["cols"], dtype=case["y"])
        s["dw"] = s["held"] if case["add"] else out(case["rows"], case["cols"])
        s["scratch"] = out(k3.linear_scratch_bytes(n, case["rows"], case["cols"], grad=True), dtype=torch.uint8)
    elif op == "control":
        s["y"] = out(n, case["vocab"], dtype=case["y"]) if case["y"] else s["x"]
    elif op == "distill":
        s["loss"], s["lse"], s["log_rest"] = out(n), out(n), out(n) if case["mode"] == "rest" else None
    else:
        s["dx"] = out(n, case["vocab"], dtype=case["x"])
        if case["mode"] != "rest":
            s["log_rest"] = None
    return s


def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s, s["case"])


def _run_own(s):
    k3, c = s["k3"], s["case"]
    op = c["op"]
    if op == "linear":
        k3.linear(s["x"], s["w"], s["y"], s["status"], bias=s.get("bias"), residual=s.get("res"), act=c["act"], z=s.get("z"), scratch=s["scratch"])
        return {k: s[k] for k in ("y", "z") if k in s}
    if op == "linear_grad" and not c["cols"]:
        k3.linear_dz(s["z"], s["dy"], s["dz"], act=c["act"], dbias=s["dbias"], accumulate=c["add"])
        return {"dz": s["dz"], "dbias": s["dbias"]}
    if op == "linear_grad":
        k3.linear_grad(s["x"], s["w"], s["dz"], s["status"], dx=s["dx"], dw=s["dw"], scratch=s["scratch"], accumulate=c["add"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "control":
        k3.logits_control(s["x"], s["y"], s["status"], history=s["history"], spans=s["spans"], repetition=s["repetition"], frequency=s["frequency"],
                          presence=s["presence"], bias_ids=s.get("bias_ids"), bias_values=s.get("bias_values"), bias_spans=s.get("bias_spans"),
                          mask=s.get("mask"), mask_rows=s.get("mask_rows"))
        return s["y"]
    if op == "distill":
        k3.distill(s["x"], s["top_ids"], s["top"], s["loss"], s["status"], lse=s["lse"], log_rest=s["log_rest"], mode=c["mode"], scale=s["scale"])
        return {k: s[k] for k in ("loss", "lse", "log_rest") if s[k] is not None}
    k3.distill_grad(s["x"], s["top_ids"], s["top"], s["lse"], s["g"], s["dx"], s["status"], log_rest=s["log_rest"], mode=c["mode"], scale=s["scale"])
    return s["dx"]


# ---- the plain forms -----------------------------------------------------------------------------------------------

def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        q = 1 / (1 + torch.exp(-z))
        return q * (1 + z * (1 - q))
    if act == "gelu":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_linear(s, c):
    z = s["x"].float() @ s["w"].float().T
    if c["bias"]:
        z += s["bias"].float()
    y = _act(z, c["act"])
    if c["res"]:
        y = y + s["res"].float()
    got = {"y": y.to(_TYPES[c["y"]])}
    if c["z"]:
        got["z"] = z.to(torch.bfloat16)
    return got


def _plain_linear_grad(s, c):
    if not c["cols"]:
        dz = s["dy"].float() * _act_slope(s["z"].float(), c["act"])
        dbias = dz.sum(0)
        return {"dz": dz.to(torch.bfloat16), "dbias": s["held"].add_(dbias) if c["add"] else dbias}
    dz = s["dz"].float()
    dw = dz.T @ s["x"].float()
    return {"dx": (dz @ s["w"].float()).to(_TYPES[c["y"]]), "dw": s["held"].add_(dw) if c["add"] else dw}


def _counts(s, n, vocab):
    """For every row and token: how often the row's output holds it, and whether its prompt or output does."""
    begin, split, end = s["spans"].unbind(1)
    length = end - begin
    row = torch.repeat_interleave(torch.arange(n, device="cuda"), length)
    at = torch.arange(len(row), device="cuda") - (length.cumsum(0) - length)[row] + begin[row]
    place = row * vocab + s["history"][at].long()
    seen = torch.zeros(n * vocab, dtype=torch.bool, device="cuda")
    seen[place] = True
    count = torch.zeros(n * vocab, dtype=torch.int32, device="cuda")
    count.index_add_(0, place, (at >= split[row]).to(torch.int32))
    return seen.view(n, vocab), count.view(n, vocab)


def _plain_control(s, c):
    n, vocab = c["n"], c["vocab"]
    seen, count = _counts(s, n, vocab)
    v = s["x"].float()
    r = s["repetition"][:, None]
    v = torch.where(seen, torch.where(v > 0, v / r, v * r), v)
    v = v - s["frequency"][:, None] * count - torch.where(count > 0, s["presence"][:, None], torch.zeros_like(v))
    if c["bias"]:
        row = torch.repeat_interleave(torch.arange(n, device="cuda"), s["bias_spans"][:, 1] - s["bias_spans"][:, 0])
        bias = torch.zeros(n * vocab, device="cuda")
        bias[row * vocab + s["bias_ids"].long()] = s["bias_values"]
        v += bias.view(n, vocab)
    if c["allowed"]:
        ok = ((s["mask"][:, :, None] >> torch.arange(32, dtype=torch.int32, device="cuda")) & 1).bool().flatten(1)[:, :vocab]
        v = torch.where(ok[s["mask_rows"].clamp(min=0).long()] | (s["mask_rows"] < 0)[:, None], v, torch.full_like(v, -math.inf))
    return s["x"].copy_(v) if not c["y"] else v.to(_TYPES[c["y"]])


def _teacher(s, c):
    """The teacher's probabilities (zero where there is none), their logarithms (zero likewise) and the rest's mass."""
    on = s["top_ids"] >= 0
    t = torch.where(on, s["top"], torch.full_like(s["top"], -math.inf)).double()
    if c["mode"] == "normalised":
        m = torch.where(on.any(1), t.amax(1), torch.zeros_like(t[:, 0]))[:, None]
        t = t - m - torch.log(torch.exp(t - m).sum(1, keepdim=True))
    q = torch.where(on, torch.exp(t), torch.zeros_like(t))
    rest = (1 - q.sum(1)).clamp(min=0) if c["mode"] == "rest" else torch.zeros_like(q[:, 0])
    return on, q, torch.where(on, t, torch.zeros_like(t)), rest


def _plain_distill(s, c):
    # (in 64 bits: the loss is what is left of terms far larger than it)
    z = s["x"].double() * s["scale"]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    on, q, t, rest = _teacher(s, c)
    at = s["top_ids"].clamp(min=0).long()
    top = torch.where(on, z.gather(1, at), torch.zeros_like(q))
    log_sum = torch.log(e.sum(1, keepdim=True))
    loss = (q * (t - torch.where(on, top - m - log_sum, torch.zeros_like(top)))).sum(1)
    got = {"lse": (m + log_sum)[:, 0]}
    if c["mode"] == "rest":
        mine = torch.zeros_like(z, dtype=torch.bool)
        row = torch.arange(c["n"], device="cuda")[:, None].expand_as(at)
        mine[row[on], at[on]] = True
        log_rest = torch.log(torch.where(mine, torch.zeros_like(e), e).sum(1)) - log_sum[:, 0]
        got["log_rest"] = log_rest
        loss = loss + torch.where(rest > 0, rest * (torch.log(rest) - log_rest), torch.zeros_like(rest))
        loss = torch.where(on.any(1), loss, torch.zeros_like(loss))
    return {"loss": loss.float(), **{k: v.float() for k, v in got.items()}}


def _plain_distill_grad(s, c):
    p = torch.exp(s["x"].float() * s["scale"] - s["lse"][:, None])
    on, q, _, rest = _teacher(s, c)
    g = torch.where(on.any(1), s["g"], torch.zeros_like(s["g"]))[:, None]
    total = (q.sum(1) + rest).float()[:, None]
    at = s["top_ids"].clamp(min=0).long()
    if c["mode"] == "rest":
        share = (rest / torch.exp(s["log_rest"].double())).float()[:, None]
        mine = torch.zeros_like(p, dtype=torch.bool)
        row = torch.arange(c["n"], device="cuda")[:, None].expand_as(at)
        mine[row[on], at[on]] = True
        d = p * torch.where(mine, total, total - share)
    else:
        d = p * total
    d.scatter_add_(1, at, -q.float())
    return (d * (g * s["scale"])).to(_TYPES[c["x"]])


_PLAIN = {"linear": _plain_linear, "linear_grad": _plain_linear_grad, "control": _plain_control, "distill": _plain_distill,
          "distill_grad": _plain_distill_grad}


# ---- what a pass cannot do without ---------------------------------------------------------------------------------

def work(case):
    op, n = case["op"], case["n"]
    if op in ("linear", "linear_grad"):
        rows, cols, y = case["rows"], case["cols"], 2 if case["y"] == _BF16 else 4
        if op == "linear":
            each = y + (y if case["res"] else 0) + (2 if case["z"] else 0)
            return {"bytes": 2 * (n + rows) * cols + each * n * rows + {"": 0, _BF16: 2, _F32: 4}[case["bias"]] * rows, "flops": 2 * n * rows * cols}
        if not cols:
            return {"bytes": (2 + y + 2) * n * rows + (8 if case["add"] else 4) * rows, "flops": 8 * n * rows}
        return {"bytes": 2 * (n * cols + rows * cols + n * rows) + y * n * cols + (8 if case["add"] else 4) * rows * cols, "flops": 4 * n * rows * cols}
    vocab, w = case["vocab"], 2 if case["x"] == _BF16 else 4
    if op == "control":
        ids = 4 if case["id"] == "i32" else 8
        # tokens with a uniform logarithm: token i has probability log((i + 2) / (i + 1)) / log(vocab); half of the longest history on average
        length = max(1, case["history"] // 2)
        kinds = sum(1.0 - (1.0 - math.log1p(1.0 / (i + 1)) / math.log(vocab)) ** length for i in range(vocab)) + case["bias"]
        lists = length * ids / case["drafts"] + case["bias"] * (ids + 4) + 64
        mask = min(n, 64) * vocab / 8 if case["allowed"] else 0
        if case["y"]:
            # where a grammar bans a token its logit need not be read
            read = 0.1 + 0.9 * case["allowed"] if case["allowed"] else 1.0
            return {"bytes": n * (lists + vocab * (read * w + (2 if case["y"] == _BF16 else 4))) + mask, "flops": 6 * n * kinds}
        banned = 0.9 * (1 - case["allowed"]) if case["allowed"] else 0.0
        return {"bytes": n * (lists + kinds * 2 * w * (1 - banned) + banned * vocab * w) + mask, "flops": 6 * n * kinds}
    if op == "distill":
        return {"bytes": n * (vocab * w + 12 + 8 * case["top"]), "flops": 4 * n * vocab}
    return {"bytes": n * (2 * vocab * w + 12 + 8 * case["top"]), "flops": 4 * n * vocab}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def exact(case, seed):
    s, op, n = _inputs(case, seed), case["op"], case["n"]
    if op == "linear":
        y, z = [], []
        w = s["w"].double().T.contiguous()
        for i in range(0, n, 2048):  # 2048 tokens at a time
            v = torch.mm(s["x"][i: i + 2048].double(), w)
            if "bias" in s:
                v = v + s["bias"].double()[None, :]
            z.append(v)
            a = case["act"]
            if a == "relu":
                v = v * (v > 0)
            elif a == "silu":
                v = v * torch.sigmoid(v)
            elif a == "gelu":
                # (1 + tanh u) / 2 is the logistic function of 2 u
                v = v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * v * (1 + 0.044715 * v ** 2))
            y.append(v + s["res"][i: i + 2048].double() if "res" in s else v)
        return {"y": torch.cat(y), "z": torch.cat(z)} if case["z"] else {"y": torch.cat(y)}
    if op == "linear_grad" and not case["cols"]:
        z = s["z"].double().requires_grad_()
        a = case["act"]
        y = {"relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
             "gelu": lambda: z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * z * (1 + 0.044715 * z ** 2))}[a]()
        dz, = torch.autograd.grad(y, z, s["dy"].double())
        dbias = dz.sum(0)
        return {"dz": dz, "dbias": dbias + s["held"].double() if case["add"] else dbias}
    if op == "linear_grad":
        dz = s["dz"].double()
        dw = torch.mm(dz.T, s["x"].double())
        return {"dx": torch.mm(dz, s["w"].double()), "dw": dw + s["held"].double() if case["add"] else dw}
    if op == "control":
        out = s["x"].double()
        spans = s["spans"].tolist()
        for i in range(n):
            b, m, e = spans[i]
            v = out[i]
            r, f, p = (s[k][i].double() for k in ("repetition", "frequency", "presence"))
            seen = torch.unique(s["history"][b:e].long())
            v[seen] = torch.where(v[seen] > 0, v[seen] / r, v[seen] * r)
            kinds, times = torch.unique(s["history"][m:e].long(), return_counts=True)
            v[kinds] -= f * times + p
            if case["bias"]:
                lo, hi = (int(k) for k in s["bias_spans"][i])
                v[s["bias_ids"][lo:hi].long()] += s["bias_values"][lo:hi].double()
            if case["allowed"] and int(s["mask_rows"][i]) >= 0:
                words = s["mask"][int(s["mask_rows"][i])].long() & 0xFFFFFFFF
                j = torch.arange(case["vocab"], device="cuda")
                v[((words[j // 32] >> (j % 32)) & 1) == 0] = -math.inf
        return out
    parts = []
    for i in range(0, n, 256):  # 256 rows at a time
        logits = s["x"][i: i + 256].double().requires_grad_(op == "distill_grad")
        ids, t = s["top_ids"][i: i + 256].long(), s["top"][i: i + 256].double()
        on = ids >= 0
        t = t.masked_fill(~on, -math.inf)
        if case["mode"] == "normalised":
            t = torch.log_softmax(t, 1).masked_fill(~on, -math.inf)
        q = t.exp()
        logp = torch.log_softmax(logits * s["scale"], 1)
        taken = torch.zeros(logp.shape, dtype=torch.int32, device="cuda").scatter_add_(1, ids.clamp(min=0), on.int()) > 0
        kl = torch.where(on, q * (t.masked_fill(~on, 0) - logp.gather(1, ids.clamp(min=0))), torch.zeros_like(q)).sum(1)
        log_rest = torch.logsumexp(logp.masked_fill(taken, -math.inf), 1)
        if case["mode"] == "rest":
            rest = (1 - q.sum(1)).clamp(min=0)
            kl = kl + torch.where(rest > 0, rest * (torch.log(rest.clamp(min=1e-300)) - log_rest), torch.zeros_like(rest))
        kl = torch.where(on.any(1), kl, torch.zeros_like(kl))
        if op == "distill":
            parts.append((kl.detach(), torch.logsumexp(logits * s["scale"], 1)) + ((log_rest,) if case["mode"] == "rest" else ()))
        else:
            parts.append(torch.autograd.grad(kl, logits, s["g"][i: i + 256].double()))
    whole = [torch.cat(v) for v in zip(*parts)]
    return whole[0] if op == "distill_grad" else dict(zip(("loss", "lse", "log_rest"), whole))
