"""Log probabilities of given tokens with entropy and top alternatives, and their gradient, against the formulas in
64 bits (the scaled logits are the fp32 products on both sides).

With Z the largest |z - max| that still counts (its exponential is not 0 in fp32: at most 104) and V the vocabulary,
an exponential errs by a few units plus the rounding of its argument, about (4 + 2 Z) 2^-24 of itself, and a sum of V of
them by at most (V / 64 + 16) 2^-24 more (64 or more partial sums); lse by that and the roundings of m and of itself.
The top alternatives are compared exactly."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
k3 = pytest.importorskip("lossless_bf16_weight_k3huf_gb300")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
E = 2.0 ** -24
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    k3._build.build()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def forward(x, tokens, top, scale=1.0):
    n = x.shape[0]
    f = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    lp, ent, lse, st = f(n), f(n), f(n), status()
    ti = torch.full((n, top), -9, dtype=torch.int32, device="cuda") if top else None
    tl = f(n, top) if top else None
    k3.token_logprobs(x, tokens, lp, st, entropy=ent, lse=lse, top_ids=ti, top_logprobs=tl, scale=scale)
    torch.cuda.synchronize()
    return lp, ent, lse, ti, tl, int(st.item())


def reference(x, tokens, top, scale):
    z = (x.float() * np.float32(scale)).double()
    lse = torch.logsumexp(z, 1)
    logp = torch.log_softmax(z, 1)                      # (shifted by the largest first: lse alone cannot hold -3e38 + 8)
    p = logp.exp()
    ent = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
    lp = torch.where(tokens >= 0, logp.gather(1, tokens.clamp(min=0)[:, None])[:, 0], torch.zeros_like(lse))
    raw = x.float().cpu().numpy().astype(np.float64)
    order = np.lexsort((np.broadcast_to(np.arange(raw.shape[1]), raw.shape), -raw), axis=1)[:, :top] if top else None
    return z, lse, logp, p, ent, lp, order


def tolerances(z, lse, logp, p, ent, lp):
    V = z.shape[1]
    m = z.amax(1)
    arg = 2 * torch.clamp(m[:, None] - z, max=104.0)
    t_sum = ((4 + arg) * p).sum(1) * E + (V / 64 + 16) * E
    t_lse = t_sum + 2 * E * (m.abs() + lse.abs() + 1)
    spread = torch.where(p > 0, p * (m[:, None] - z), torch.zeros_like(p))
    t_ent = 3 * t_sum + (spread * (8 + arg)).sum(1) * E + (V / 64 + 32) * E * (1 + spread.sum(1))
    t_lp = t_lse + 4 * E * (lp.abs() + m.abs())
    return t_lse, t_ent, t_lp


def check(x, tokens, top, scale=1.0):
    lp, ent, lse, ti, tl, st = forward(x, tokens, top, scale)
    z, r_lse, logp, p, r_ent, r_lp, order = reference(x, tokens.long(), top, scale)
    t_lse, t_ent, t_lp = tolerances(z, r_lse, logp, p, r_ent, torch.where(r_lp.isinf(), torch.zeros_like(r_lp), r_lp))
    assert st == 0
    assert bool(((lse.double() - r_lse).abs() <= t_lse).all())
    assert bool(((ent.double() - r_ent).abs() <= t_ent).all())
    off = torch.where(r_lp == -INF, (lp != -INF).double(), (lp.double() - r_lp).abs())
    assert bool((off <= t_lp).all())
    if top:
        assert np.array_equal(ti.cpu().numpy(), order)
        r_tl = logp.gather(1, torch.from_numpy(order.copy()).cuda())
        off = torch.where(r_tl == -INF, (tl != -INF).double(), (tl.double() - r_tl).abs())
        assert bool((off <= (t_lse + 4 * E * z.amax(1).abs())[:, None] + 4 * E * torch.where(r_tl.isinf(), torch.zeros_like(r_tl), r_tl).abs()).all())


def logits(n, V, dtype, seed, std=3.0, banned=0.0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(n, V + pad, generator=g, device="cuda") * std).to(dtype)[:, :V]
    if banned:
        x[torch.rand(n, V, generator=g, device="cuda") < banned] = -INF
        x[:, V // 2] = 0.25
    tokens = torch.randint(0, V, (n,), generator=g, device="cuda")
    return x, tokens


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,V", [(1, 1), (3, 2), (2, 7), (5, 64), (4, 255), (3, 1000), (2, 4097), (40, 513), (7, 32003), (1, 131072), (2, 150001), (300, 1024), (700, 2053)])
def test_forward_matches_the_formula(n, V, dtype):
    for top in (0, 1, 5, 20, 64):
        if top > V:
            continue
        x, tokens = logits(n, V, dtype, n * 13 + V + top, banned=0.0 if top != 5 else 0.6)
        tokens[0] = -1 if n > 1 else tokens[0]
        check(x, tokens, top, scale=0.7 if top else 1.0)
        check(x, tokens.to(torch.int32), top, scale=1.3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties_go_to_the_lower_index(dtype):
    x = torch.zeros(6, 9000, device="cuda", dtype=dtype)
    x[1, 4000:] = 1.0
    x[2] = torch.randint(0, 3, (9000,), device="cuda").to(dtype)
    x[3, ::2] = -0.0                                    # equal to 0
    x[4] = torch.arange(9000, device="cuda").to(dtype)   # ascending: every value a new largest
    x[5] = -torch.arange(9000, device="cuda").to(dtype)
    for top in (1, 8, 33, 64):
        check(x, torch.arange(6, device="cuda"), top)


@pytest.mark.parametrize("top", [24, 25, 64])
@pytest.mark.parametrize("n,V", [(700, 9000), (20, 70000), (650, 70000), (5, 64), (4, 200)])
def test_many_alternatives(n, V, top):
    gen = torch.Generator("cuda").manual_seed(n + V + top)
    x = torch.rand(n, V, generator=gen, device="cuda").argsort(1).float() / V          # (no two alike)
    _, _, _, ti, tl, st = forward(x, torch.zeros(n, dtype=torch.int64, device="cuda"), top)
    want = torch.topk(x, top, dim=1)
    assert st == 0
    assert torch.equal(ti.long(), want.indices)
    got = torch.log_softmax(x.double(), 1).gather(1, want.indices)
    # (as in the docstring, with Z = 1 and values up to 1 + log V)
    assert (tl - got).abs().max() <= (6 + V / 64 + 16 + 4 * (2 + np.log(V))) * E


@pytest.mark.parametrize("many", [400, 1000, 2300, 2336, 2368, 2400, 2500, 4096])
def test_many_values_above_the_first_ones(many):
    """A part of a row that rises above all before it: up to that many candidates at once."""
    n, V = 640, 70000
    gen = torch.Generator("cuda").manual_seed(many)
    x = -torch.rand(n, V, generator=gen, device="cuda")
    x[:, 4096:4096 + many] = 1 + torch.rand(n, many, generator=gen, device="cuda").argsort(1).float() / 64
    _, _, _, ti, _, st = forward(x, torch.zeros(n, dtype=torch.int64, device="cuda"), 20)
    assert st == 0
    assert torch.equal(ti.long(), torch.topk(x, 20, dim=1).indices)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_rows_and_lowest_values(dtype):
    V = 5000
    low = torch.finfo(dtype).min
    x, tokens = logits(6, V, dtype, 3)
    x[0, 1:] = -INF                                     # one logit left: probability 1, entropy 0
    x[1, :] = low                                       # all at the type's lowest value: uniform
    x[2, 10:] = low
    x[3, :] = -INF
    x[3, 17:19] = 2.0
    x[4, 5:] = -INF                                     # fewer logits than alternatives
    tokens[:] = torch.tensor([0, 3, 4, 17, 4999, 9], device="cuda")
    check(x, tokens, 8)
    check(x, tokens, 64, scale=0.5)
    check(x, torch.tensor([3, 3, 2000, 3, 3, -1], device="cuda"), 3)   # masked tokens: log probability -infinity
    big = torch.full((2, V), low, device="cuda", dtype=dtype)
    big[0, 7] = torch.finfo(dtype).max
    lp, ent, lse, ti, tl, st = forward(big, torch.tensor([7, 0], device="cuda"), 2)
    assert st == 0 and lp[0].item() == 0.0 and ent[0].item() == 0.0 and ti[0, 0].item() == 7 and ti[0, 1].item() == 0


def test_rows_with_nothing_left_and_non_finite_ones():
    x = torch.full((4, 3000), -INF, device="cuda")
    x[1, 5] = float("nan")
    x[2, 9] = INF
    x[3] = 1.0
    lp, ent, lse, ti, tl, st = forward(x, torch.tensor([4, 4, 4, 4], device="cuda"), 3)
    assert st == 0
    assert lse[0].item() == -INF and lp[0].item() == -INF and ent[0].item() == 0.0
    assert ti[0].tolist() == [0, 1, 2] and bool((tl[0] == -INF).all())
    assert bool(lse[1].isnan()) and bool(ent[1].isnan()) and bool(lse[2].isnan() | lse[2].isinf()) and bool(ent[2].isnan())
    assert abs(lse[3].item() - (1 + np.log(3000))) < 1e-5 and ti[3].tolist() == [0, 1, 2]


def test_strides_offsets_and_tokens_past_the_vocabulary():
    for dtype in (torch.bfloat16, torch.float32):
        for pad in (1, 3, 8):
            x, tokens = logits(9, 1001, dtype, pad, pad=pad)
            check(x, tokens, 4)
            wide, tokens = logits(9, 4000, dtype, pad)
            check(wide[:, pad: pad + 2500], tokens % 2500, 4)   # rows that start anywhere
    x, tokens = logits(3, 100, torch.float32, 1)
    tokens[1] = 100
    lp, *_, st = forward(x, tokens, 0)
    assert st == k3.ST_TOKEN and lp[1].item() == 0.0
    assert forward(x[:0], tokens[:0], 5)[-1] == 0


def backward(x, tokens, lse, ent, g, h, scale, out=None):
    d = torch.full(x.shape, float("nan"), device="cuda", dtype=x.dtype) if out is None else out
    st = status()
    k3.token_logprobs_grad(x, tokens, lse, g, d, st, entropy=ent if h is not None else None, g_entropy=h, scale=scale)
    torch.cuda.synchronize()
    return d, int(st.item())


def backward_ref(x, tokens, lse, ent, g, h, scale):
    z = (x.float() * np.float32(scale)).double()
    lp = z - lse.double()[:, None]
    p = lp.exp()
    on = tokens >= 0
    gg = torch.where(on, g.double(), torch.zeros_like(g.double()))[:, None]
    hh = (h.double() if h is not None else torch.zeros_like(g.double()))[:, None]
    inner = torch.where(p > 0, lp + ent.double()[:, None], torch.zeros_like(lp))
    d = -p * (gg + hh * inner)
    mag = p * (gg.abs() + hh.abs() * (torch.where(p > 0, lp.abs(), torch.zeros_like(lp)) + ent.double().abs()[:, None]))
    d.scatter_add_(1, tokens.clamp(min=0)[:, None], gg)
    # an exponential errs by its argument's rounding and a few units; every other operation by one unit
    err = E * (16 + 2 * (torch.where(p > 0, z.abs(), torch.zeros_like(z)) + lse.double().abs()[:, None])) * mag + 4 * E * d.abs()
    return scale * d, scale * err + 2.0 ** -126 * scale       # (fp32 exponentials below 2^-126 may go to 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,V", [(1, 1), (3, 7), (2, 1000), (5, 4097), (3, 32003), (1, 131072), (300, 520)])
def test_gradient_matches_the_formula(n, V, dtype):
    for banned in (0.0, 0.5):
        x, tokens = logits(n, V, dtype, V + n, banned=banned)
        if n > 1:
            tokens[1] = -1
        scale = 0.8
        _, _, lse, *_ = (v for v in forward(x, tokens, 0, scale))
        ent = forward(x, tokens, 0, scale)[1]
        gen = torch.Generator(device="cuda").manual_seed(4)
        g, h = torch.randn(n, generator=gen, device="cuda"), torch.randn(n, generator=gen, device="cuda")
        for hh in (h, None):
            d, st = backward(x, tokens, lse, ent, g, hh, scale)
            want, tol = backward_ref(x, tokens, lse, ent, g, hh, scale)
            assert st == 0
            assert bool(((d.double() - want).abs() <= tol + (2.0 ** -8 if dtype == torch.bfloat16 else E) * want.abs()).all())
        inplace = x.clone()
        d2, _ = backward(inplace, tokens, lse, ent, g, None, scale, out=inplace)
        assert torch.equal(d2, d)


def test_gradient_of_masked_rows_strides_and_bad_tokens():
    x, tokens = logits(5, 1003, torch.float32, 9, pad=5)
    x[0] = -INF
    x[1, 1:] = -INF
    x[2, 5:] = torch.finfo(torch.float32).min
    tokens[:] = torch.tensor([-1, 0, 3, 1003, 7], device="cuda")
    *_, st = forward(x, tokens, 0)
    assert st == k3.ST_TOKEN
    lp, ent, lse, *_ = forward(x, tokens, 0)
    g, h = torch.ones(5, device="cuda"), torch.ones(5, device="cuda")
    wide = torch.full((5, 1100), 3.0, device="cuda")
    d, st = backward(x, tokens, lse, ent, g, h, 1.0, out=wide[:, :1003])
    assert st == k3.ST_TOKEN and bool((wide[:, 1003:] == 3.0).all())
    want, tol = backward_ref(x[1:3], tokens[1:3], lse[1:3], ent[1:3], g[1:3], h[1:3], 1.0)
    assert bool(((d[1:3].double() - want).abs() <= tol + E * want.abs()).all())
    assert bool((d[0] == 0).all()) and bool(d[1:].isfinite().all())


def test_gradient_against_differences():
    """Central differences of the formula in 64 bits along random directions, step 1e-4: their truncation error is
    1e-8 / 6 of a third derivative of order 10 or less, their rounding about 1e-11."""
    x, tokens = logits(6, 300, torch.float32, 21, std=1.0)
    scale = 0.9
    lp, ent, lse, *_ = forward(x, tokens, 0, scale)
    gen = torch.Generator(device="cuda").manual_seed(8)
    g, h = torch.randn(6, generator=gen, device="cuda"), torch.randn(6, generator=gen, device="cuda")
    d, _ = backward(x, tokens, lse, ent, g, h, scale)

    def loss(v):
        logp = torch.log_softmax(v * scale, 1)
        return float((g.double() * logp.gather(1, tokens[:, None])[:, 0] - h.double() * (logp.exp() * logp).sum(1)).sum())

    for seed in range(3):
        step = torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64)
        slope = (loss(x.double() + 1e-4 * step) - loss(x.double() - 1e-4 * step)) / 2e-4
        got = float((d.double() * step).sum())
        assert abs(got - slope) <= 1e-5 * float((d.double().abs() * step.abs()).sum()) + 1e-6


def test_refusals():
    x, tokens = logits(3, 50, torch.float32, 1)
    lp, st = torch.empty(3, device="cuda"), status()
    for bad in (0.0, -1.0, INF, float("nan")):
        with pytest.raises(k3.K3HufError) as e:
            k3.token_logprobs(x, tokens, lp, st, scale=bad)
        assert e.value.code == k3.E_ARG
    for top in (51, 65):
        with pytest.raises(k3.K3HufError):
            forward(torch.zeros(3, 50 if top == 51 else 100, device="cuda"), tokens, top)
    with pytest.raises(ValueError):
        k3.token_logprobs(x, tokens, lp, st, top_ids=torch.empty(3, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        k3.token_logprobs(x, tokens[:2], lp, st)
    with pytest.raises(TypeError):
        k3.token_logprobs(x.half(), tokens, lp, st)
    with pytest.raises(TypeError):
        k3.token_logprobs_grad(x, tokens, lp, lp, x.to(torch.bfloat16), st)
    with pytest.raises(k3.K3HufError):
        k3.token_logprobs_grad(x, tokens, lp, lp, torch.empty_like(x), st, g_entropy=lp)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [0.8, 1.0, 1.7, 0.3])
def test_gradient_of_rows_at_the_lowest_value(dtype, scale):
    """Rows whose mask leaves nothing, with the type's lowest value for the mask.  lse, about -3e38, does not hold the
    log of the count, so p is known to lie in [0, 1] only; a row that nothing is asked of has gradient 0, and no
    gradient is beyond scale (|g| + |h| entropy + |h|)."""
    n, V = 64, 777
    x, tokens = logits(n, V, dtype, 5)
    low = torch.finfo(dtype).min
    x[:32] = low
    if dtype == torch.float32:                           # masks near the lowest value, whose products round either way
        x[:32] = low * torch.linspace(0.5, 1.0, 32, device="cuda")[:, None]
    tokens[::2] = -1
    lp, ent, lse, *_ = forward(x, tokens, 0, scale)
    g, h = torch.full((n,), 2.0, device="cuda"), torch.full((n,), -3.0, device="cuda")
    for hh in (None, h):
        d, st = backward(x, tokens, lse, ent, g, hh, scale)
        assert st == 0 and bool(d.isfinite().all())
        if hh is None:
            assert bool((d[::2] == 0).all())
        room = scale * (2.0 + (3.0 * (ent.double() + 1) if hh is not None else 0.0)) * (1 + 2.0 ** -8)
        assert bool((d.double().abs() <= (room[:, None] if hh is not None else room)).all())
    want, tol = backward_ref(x[32:], tokens[32:], lse[32:], ent[32:], g[32:], h[32:], scale)
    assert bool(((d[32:].double() - want).abs() <= tol + (2.0 ** -8 if dtype == torch.bfloat16 else E) * want.abs()).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [40, 3000, 70000])
def test_a_nan_or_infinity_reaches_every_statistic(dtype, V):
    """Also the log probability of a token whose own logit is -infinity, and those of the alternatives."""
    x, _ = logits(4, V, dtype, 6)
    x[:3, 1::2] = -INF
    x[0, 5] = float("nan")
    x[1, V // 2] = INF
    tokens = torch.tensor([3, 3, 3, 3], device="cuda")   # (a banned one, but in the last row)
    for top in (0, 4):
        lp, ent, lse, ti, tl, st = forward(x, tokens, top)
        assert st == 0
        for v in (lp, ent, lse) + ((tl,) if top else ()):
            assert bool(v[:2].isnan().all())
            assert not bool(v[2:].isnan().any())
        assert lp[2].item() == -INF


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_largest_scales(dtype):
    """Any finite scale: at the largest every logit below the largest one has probability 0."""
    x = torch.zeros(3, 500, device="cuda", dtype=dtype)
    x[0, :] = -1.0
    x[0, 7] = 0.0
    x[2, 100:] = -0.5
    tokens = torch.tensor([7, 3, 99], device="cuda")
    for scale in (1e38, 2.4e38, 3.4e38):
        lp, ent, lse, ti, tl, st = forward(x, tokens, 2, scale)
        assert st == 0 and lp[0].item() == 0.0 and ent[0].item() == 0.0 and lse[0].item() == 0.0
        for row, count in ((1, 500), (2, 100)):
            want = np.log(count)
            for got in (-lp[row].item(), ent[row].item(), lse[row].item()):
                # (a sum of ones; see the docstring at the top with Z = 0)
                assert abs(got - want) <= (4 + 500 / 64 + 32) * E * (1 + want)
        assert ti[0].tolist() == [7, 0] and ti[1].tolist() == [0, 1]
