"""Distillation from a teacher's top alternatives, and its gradient, against the formulas in 64 bits.

With Z the largest |z - max| that still counts (at most 104) an exponential of the sum errs by about (4 + 2 Z) 2^-24 of
itself, and a sum of V of them by (V / 64 + 16) 2^-24 more (64 or more partial sums); so does its logarithm, absolutely.
The loss adds, in 64 bits, Q times the error of the row's sum and q_r times that of the rest's, and is rounded once.
In the gradient the exponent z - lse (- log p_r) of an fp32 lse errs by 2^-24 of each of its terms' magnitudes, a few times
over; what it multiplies is computed in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
k3 = pytest.importorskip("lossless_bf16_weight_k3huf_gb300")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
E = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: E}
INF = float("inf")
MODES = ("given", "normalised", "rest")


@pytest.fixture(scope="module", autouse=True)
def built():
    k3._build.build()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def make(n, V, top, seed, dtype=F32, pad=0, std=3.0, none=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(n, V + pad, generator=g, device="cuda") * std).to(dtype)[:, :V]
    teacher = x.float() + 0.7 * torch.randn(n, V, generator=g, device="cuda")
    t, ids = torch.log_softmax(teacher, 1).topk(top, dim=1)
    ids = ids.to(torch.int32)
    drop = torch.rand(n, top, generator=g, device="cuda") < none
    ids[drop] = -1
    return x, ids.contiguous(), t.contiguous()


def parts(x, ids, t, mode, scale):
    """z, log p, the alternatives' (valid, q, log q), log p_r, q_r, and which tokens they are."""
    z = x.double() * float(torch.tensor(scale, dtype=F32))
    logp = torch.log_softmax(z, 1)
    logp = torch.where((z == -INF).all(1, keepdim=True), torch.full_like(z, -INF), logp)
    on = (ids >= 0) & (ids < x.shape[1])
    at = torch.where(on, ids, torch.zeros_like(ids)).long()
    t = t.double().masked_fill(~on, -INF)
    if mode == "normalised":
        some = (t > -INF).any(1, keepdim=True)
        t = torch.where(some, torch.log_softmax(torch.where(some, t, torch.zeros_like(t)), 1), t).masked_fill(~on, -INF)
    q = t.exp()
    taken = torch.zeros(x.shape, dtype=torch.int32, device="cuda").scatter_add_(1, at, on.int()) > 0
    log_rest = torch.logsumexp(logp.masked_fill(taken, -INF), 1)
    rest = (1 - q.sum(1)).clamp(min=0) if mode == "rest" else torch.zeros_like(log_rest)
    return z, logp, on, at, q, t, log_rest, rest, taken


def run(x, ids, t, mode, scale, **more):
    n = x.shape[0]
    f = lambda: torch.full((n,), 9.0, device="cuda")  # noqa: E731
    loss, lse, log_rest, st = f(), f(), f() if mode == "rest" else None, status()
    k3.distill(x, ids, t, loss, st, lse=lse, log_rest=log_rest, mode=mode, scale=scale, **more)
    torch.cuda.synchronize()
    return loss, lse, log_rest, int(st)


def sum_error(z, keep):
    """Of the logarithm of the sum of exp(z) over `keep`."""
    V = z.shape[1]
    z = z.masked_fill(~keep, -INF)
    m = z.amax(1, keepdim=True)
    p = torch.softmax(torch.where(m == -INF, torch.zeros_like(z), z), 1)
    arg = 2 * torch.clamp(torch.nan_to_num(m - z, nan=104.0, posinf=104.0), max=104.0)
    return ((4 + arg) * p).sum(1) * E + (V / 64 + 16) * E


def close(got, want, bound, what):
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    wild = torch.isinf(want) | torch.isnan(want)
    bound = torch.nan_to_num(bound, nan=0.0)                # (of a row with NaN: no room where its result is one)
    assert bool((got.double()[torch.isinf(want)] == want[torch.isinf(want)]).all()), what
    off = (got.double() - want).abs() - bound - HALF[got.dtype] * (want.abs() + bound)
    assert bool((off[~wild] <= 0).all()), f"{what}: {float(off[~wild].max())} over its bound"


def check(x, ids, t, mode, scale=1.0, want_status=0):
    loss, lse, log_rest, st = run(x, ids, t, mode, scale)
    assert st == want_status
    z, logp, on, at, q, tt, r_rest, rest, taken = parts(x, ids, t, mode, scale)
    counts = on & (q > 0)
    want = torch.where(counts, q * (tt.masked_fill(~counts, 0) - logp.gather(1, at)), torch.zeros_like(q)).sum(1)
    if mode == "rest":
        want = want + torch.where(rest > 0, rest * (torch.log(rest.clamp(min=1e-300)) - r_rest), torch.zeros_like(rest))
    want = torch.where(on.any(1), want, torch.zeros_like(want))
    e_all, e_rest = sum_error(z, torch.ones_like(taken)), sum_error(z, ~taken)
    r_lse = torch.logsumexp(z, 1)
    close(lse, r_lse, e_all + 2 * E * r_lse.abs(), "lse")
    close(loss, want, q.sum(1) * e_all + rest * (e_rest + e_all) + 1e-12 * (q * tt.masked_fill(~counts, 0).abs()).sum(1), "loss")
    if mode == "rest":
        close(log_rest, r_rest, e_rest + e_all, "log_rest")
    return loss, lse, log_rest


def check_grad(x, ids, t, mode, scale=1.0, in_place=False, out_pad=0, want_status=0, least=1e-37):
    n, V = x.shape
    _, lse, log_rest, _ = run(x, ids, t, mode, scale)
    g = torch.Generator(device="cuda").manual_seed(n * 7 + V)
    gl = torch.randn(n, generator=g, device="cuda")
    z, logp, on, at, q, tt, r_rest, rest, taken = parts(x, ids, t, mode, scale)
    some = on.any(1)
    gl[~some] = float("nan")                                # not read
    whole = torch.full((n, V + out_pad), 7.0, dtype=x.dtype, device="cuda")
    out, src = whole[:, :V], x
    if in_place:
        out.copy_(x)
        src = out
    st = status()
    k3.distill_grad(src, ids, t, lse, gl, out, st, log_rest=log_rest, mode=mode, scale=scale)
    torch.cuda.synchronize()
    assert int(st) == want_status and bool((whole[:, V:] == 7.0).all())
    p = logp.exp()
    Q = (q.sum(1) + rest)[:, None]
    gs = torch.where(some, gl.double(), torch.zeros_like(rest))[:, None] * float(torch.tensor(scale, dtype=F32))
    qs = torch.zeros_like(p).scatter_add_(1, at, torch.where(on, q, torch.zeros_like(q)))
    share = torch.zeros_like(p)
    if mode == "rest":
        share = torch.where(taken, share, rest[:, None] * torch.exp(torch.where(r_rest == -INF, torch.full_like(r_rest, -1e9), logp.amax(1) * 0)[:, None] +
                                                                     logp - torch.where(r_rest == -INF, torch.zeros_like(r_rest), r_rest)[:, None]))
    want = torch.where(some[:, None], gs * (Q * p - qs - share), torch.zeros_like(p))
    far = z.abs().masked_fill(z == -INF, 0) + torch.nan_to_num(torch.logsumexp(z, 1), neginf=0).abs()[:, None] + torch.nan_to_num(r_rest, neginf=0).abs()[:, None] + 8
    bound = gs.abs() * (4 * E * far * (Q * p + share) + 2 * E * qs)
    close(out, want, bound + least, "dlogits")
    return out


SIZES = [(1, 1, 1), (2, 2, 2), (3, 7, 3), (4, 64, 5), (3, 255, 20), (5, 1000, 64), (2, 4097, 33), (40, 513, 8), (7, 32003, 20), (1, 131072, 64), (2, 150001, 32), (400, 1024, 8)]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,V,top", SIZES)
def test_matches_the_formula(n, V, top, dtype, mode):
    x, ids, t = make(n, V, top, n + V + top, dtype)
    check(x, ids, t, mode)
    check(x, ids, t, mode, scale=0.7)
    check_grad(x, ids, t, mode, scale=0.7)
    x, ids, t = make(n, V, top, n + V + top + 1, dtype, pad=3)
    check(x, ids, t, mode, scale=1.3)
    check_grad(x, ids, t, mode, scale=1.3, out_pad=3)
    check_grad(x, ids, t, mode, in_place=True)
    check_grad(x, ids, t, mode, out_pad=1)


@pytest.mark.parametrize("mode", MODES)
def test_rows_without_alternatives(mode):
    x, ids, t = make(6, 5000, 8, 1)
    ids[1], ids[4, 1:] = -1, -1
    loss, _, _ = check(x, ids, t, mode)
    assert float(loss[1]) == 0.0
    d = check_grad(x, ids, t, mode)
    assert bool((d[1] == 0).all())
    x[1, 7] = float("nan")                                  # a row of no text: its loss and gradient stay 0
    loss, _, _ = check(x, ids, t, mode)
    assert float(loss[1]) == 0.0
    assert bool((check_grad(x, ids, t, mode)[1] == 0).all())


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_token_listed_twice(mode, dtype):
    x, ids, t = make(5, 3000, 40, 2, dtype, none=0.0)
    t -= 2.0                                                # (so that some mass is left)
    ids[0, 5] = ids[0, 3]
    ids[1, 39] = ids[1, 0]
    ids[2, 30:36] = ids[2, 2]
    ids[3, :] = 17
    check(x, ids, t, mode)
    check_grad(x, ids, t, mode)
    check_grad(x, ids, t, mode, in_place=True)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_alternatives_alike_and_far_apart(mode, dtype):
    """64 alternatives: listed twice, in either half of the list; in neighbouring places, and as far apart as makes a row's
    vectors fall together; of log-probabilities near 0 to far below what 32 bits hold."""
    V, r = 262149, np.random.default_rng(17)
    x, _, _ = make(5, V, 64, seed=23, dtype=dtype)
    ids = np.zeros((5, 64), dtype=np.int64)
    for row in range(5):
        j = r.integers(0, 65000, 8)
        ids[row] = np.concatenate([j, j + 65536, j + 131072, j + 131073, j + 196608, j + 7, r.permutation(j), r.permutation(j + 131072)])
        ids[row] = ids[row][r.permutation(64)]
    t = r.choice([-1000.0, -100.0, -85.5, -79.5, -20.0, -7.0], (5, 64))
    t[0] = -6.0 + r.random(64)
    t[1] = -79.0 - r.random(64)
    t[2, 5], t[3, 40], t[4, 60] = -0.25, -0.5, -INF
    ids, t = torch.from_numpy(ids).cuda().to(torch.int32), torch.from_numpy(t).cuda().float()
    check(x, ids, t, mode, scale=1.3)
    check_grad(x, ids, t, mode, scale=1.3)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("n,V,dtype,pad", [(1000, 3000, BF, 0), (1000, 3000, F32, 5), (300, 50021, F32, 0), (700, 50021, BF, 3), (2000, 700, BF, 1)])
def test_gradient_of_more_pieces_than_ctas(n, V, dtype, pad, mode):
    """Each CTA works on several pieces: the next one's factors and logits are fetched, and this one's alternatives written,
    while it is at work; rows without alternatives lie between."""
    x, ids, t = make(n, V, 20, n + V, dtype, pad=pad)
    ids[::7] = -1
    ids[3::11, 4] = ids[3::11, 17]
    a = check_grad(x, ids, t, mode, scale=0.9)
    b = check_grad(x, ids, t, mode, scale=0.9, in_place=True)
    c = check_grad(x, ids, t, mode, scale=0.9, out_pad=1)           # (rows that do not sit alike: one value at a time)
    assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,V", [(5, 60013), (310, 262149), (5, 262149), (500, 60013)])
def test_vectors_that_hold_alternatives_carry_the_rest(n, V, dtype, shift):
    """The stream passes over the 16-byte vectors that may hold an alternative, and another warp adds what else they hold.
    Here that is all there is: the other tokens lie e^-60 below.  One vector lost, or added twice, is 1/700 of the sum or
    more.  Its terms, fewer than 400, and zeros are added: 2^-24 of it each, with a few units of every exponential."""
    E_, r = (4 if dtype == F32 else 8), np.random.default_rng(V)
    cycle = (128 if V <= 65536 else 256) * 64                       # vectors after which a thread's bits come round
    width = (V + 15) // 8 * 8
    buf = torch.full((n, width), -60.0, dtype=dtype, device="cuda")
    x5, ids5 = np.full((5, V), -60.0), np.zeros((5, 64), dtype=np.int64)
    for row in range(5):
        j = r.integers(0, min(V // 4, cycle * E_) - 16, 8)
        step = cycle * E_ if 3 * cycle * E_ < V else V // 4
        ids5[row] = np.concatenate([j, j + step, j + 2 * step, j + 2 * step + 1, j + 3 * step, j + 7, r.permutation(j), r.permutation(j + 2 * step)])
        if row % 2:
            ids5[row] = r.integers(0, V, 64)
        ids5[row] = ids5[row][r.permutation(64)]
        ids5[row, :2] = 0, V - 1                                    # (the row's ends, whose vectors are not whole)
        taken = set(ids5[row].tolist())
        homes = {(i + shift) // E_ % cycle for i in taken}
        k = 0
        for home in homes:
            for at in range(home, (V + shift + E_ - 1) // E_, cycle):
                inside = [e for e in range(at * E_ - shift, at * E_ - shift + E_) if 0 <= e < V and e not in taken]
                if inside:
                    x5[row, r.choice(inside)] = (k % 8) / 16 - 0.25
                    k += 1
        assert 8 < k < 400
        x5[row, list(taken)] = r.integers(-16, 16, len(taken)) / 16
    x = buf[:, shift:shift + V]
    x.copy_(torch.from_numpy(x5).cuda().to(dtype).repeat(n // 5, 1))
    assert x.data_ptr() % 16 == shift * x.element_size()
    ids = torch.from_numpy(ids5).cuda().to(torch.int32).repeat(n // 5, 1).contiguous()
    t = (-5.0 - torch.rand(5, 64, generator=torch.Generator(device="cuda").manual_seed(V), device="cuda")).repeat(n // 5, 1).contiguous()
    loss, lse, log_rest, st = run(x, ids, t, "rest", 1.0)
    assert st == 0
    z, logp, on, at, q, tt, r_rest, rest, _ = parts(x[:5], ids[:5], t[:5], "rest", 1.0)
    assert bool((rest > 0.1).all())
    want = (q * (tt - logp.gather(1, at))).sum(1) + rest * (torch.log(rest) - r_rest)
    bound = (400 + 16 + 4 + 2 * 2) * E                              # (exponents of 2 at most)
    for got, ref, b, what in ((lse, torch.logsumexp(z, 1), bound, "lse"), (log_rest, r_rest, 2 * bound, "log_rest"), (loss, want, 3 * bound, "loss")):
        close(got, ref.repeat(n // 5), torch.full((n,), b, dtype=torch.float64, device="cuda") + 1e-9, what)
        assert torch.equal(got, got[:5].repeat(n // 5))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_small_rest_keeps_its_digits(dtype):
    """The alternatives hold nearly all of p: the rest's sum is not a difference."""
    x, ids, t = make(4, 9000, 4, 3, dtype, none=0.0)
    top = ids.long()
    x.scatter_(1, top, x.gather(1, top) + 30)
    check(x, ids, t, "rest")
    check_grad(x, ids, t, "rest")
    # ... and the other way round: tokens of hardly any p
    low = x.float().topk(4, dim=1, largest=False).indices.to(torch.int32)
    check(x, low, t, "rest")
    check_grad(x, low, t, "rest")
    x[:, :] = -INF                                          # nothing but the alternatives
    x.scatter_(1, top, torch.randn(4, 4, device="cuda").to(dtype))
    t = torch.log_softmax(t, 1).contiguous()
    for mode in ("given", "normalised"):
        check(x, ids, t, mode)
        check_grad(x, ids, t, mode)
    half = (t - 1.0).contiguous()                           # q_r above 0 against p_r 0
    loss, _, log_rest, _ = run(x, ids, half, "rest", 1.0)
    assert bool((loss == INF).all()) and bool((log_rest == -INF).all())
    check_grad(x, ids, half, "rest")


def below(n, V, top, gap, scale, dtype, seed):
    """Rows whose alternatives lie at least `gap` scaled units above every other token."""
    x, ids, t = make(n, V, top, seed, dtype, none=0.0)
    at = ids.long()
    high = x.float().clone()
    high.scatter_(1, at, high.gather(1, at) + gap / scale)
    return high.to(dtype), ids, t


def rest_apart(x, ids, t, scale):
    """Loss, lse and log_rest against 64 bits.  An exponent scale * x is taken with the scale times log2 e in 32 bits: 2^-24
    of it, which both sides of a difference of logits share, so 2^-24 of the difference; what else errs is as in check()."""
    loss, lse, log_rest, st = run(x, ids, t, "rest", scale)
    assert st == 0
    z, logp, on, at, q, tt, r_rest, rest, taken = parts(x, ids, t, "rest", scale)
    e_all, e_rest = sum_error(z, torch.ones_like(taken)), sum_error(z, ~taken)
    lp = logp.gather(1, at)
    want = (q * (tt - lp)).sum(1) + rest * (torch.log(rest) - r_rest)
    assert bool((rest > 0).all())
    close(lse, torch.logsumexp(z, 1), e_all + 2 * E * torch.logsumexp(z, 1).abs(), "lse")
    close(log_rest, r_rest, e_rest + e_all + E * r_rest.abs(), "log_rest")
    close(loss, want, q.sum(1) * e_all + rest * (e_rest + e_all) + E * ((q * lp.abs()).sum(1) + rest * r_rest.abs()) + 1e-12 * (q * tt.abs()).sum(1), "loss")
    return loss, lse, log_rest


@pytest.mark.parametrize("scale", [1.0, 10.0])
@pytest.mark.parametrize("gap", [70.0, 85.0, 100.0, 1000.0, 30000.0])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,V", [(4, 3000), (3, 20011), (2, 140000), (1000, 1500)])
def test_a_rest_far_below_the_alternatives(n, V, dtype, gap, scale):
    """p_r far below the smallest fp32 number: its logarithm, the loss and the gradient are finite all the same.  A CTA per
    row, and clusters."""
    x, ids, t = below(n, V, 4, gap, scale, dtype, n + V)
    loss, _, log_rest = rest_apart(x, ids, t, scale)
    assert bool((log_rest < -gap / 2).all()) and bool(torch.isfinite(log_rest).all()) and bool(torch.isfinite(loss).all())
    # (exponentials below 2^-126 are 0: times scale |g| (Q + q_r) at most, with |g| < 6 here and Q + q_r < 2)
    least = 2.0 ** -126 * scale * 12
    for in_place in (False, True):
        d = check_grad(x, ids, t, "rest", scale=scale, in_place=in_place, least=least)
        assert bool(torch.isfinite(d.float()).all())
    # ... and the alternatives as far below the others
    x, ids, t = below(n, V, 4, -gap, scale, dtype, n + V + 1)
    rest_apart(x, ids, t, scale)
    check_grad(x, ids, t, "rest", scale=scale, least=least)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_what_the_sum_errs_by_cancels_between_near_distributions(dtype):
    """With d what the other tokens' sum errs by, relative to itself, the loss errs by (p_r - q_r) d: both of its logarithms
    take the same sum.  Its exponentials err by 1 x 2^-24 in the root mean square, nearly all to one side, and their rounded
    arguments to both, so d is 2 x 2^-24 at most in that mean over the rows; half a unit of the loss is its own rounding.
    (Sums that are rounded apart err by a third of a unit, 1.6 times this bound.)"""
    x, ids, t = make(512, 131072, 20, 41, dtype, none=0.0)
    loss, _, log_rest, _ = run(x, ids, t, "rest", 1.0)
    _, logp, _, at, q, tt, r_rest, rest, _ = parts(x, ids, t, "rest", 1.0)
    want = (q * (tt - logp.gather(1, at))).sum(1) + rest * (torch.log(rest) - r_rest)

    def rms(v):
        return float(v.pow(2).mean().sqrt())

    assert rms(loss.double() - want) <= 2 * E * rms(r_rest.exp() - rest) + E * rms(want)


def test_infinite_terms():
    x, ids, t = make(6, 4000, 8, 4, none=0.0)
    at = ids.long()
    x[0, at[0, 2]] = -INF                                   # p 0 against a q above 0
    x[1, at[1, 2]], t[1, 2] = -INF, -INF                    # ... against q 0
    x[2] = -INF                                             # no logit at all
    x[3, 11] = float("nan")
    x[4, 12] = INF
    for mode in ("given", "normalised"):
        loss, lse, _, st = run(x, ids, t, mode, 1.0)
        assert st == 0
        assert float(loss[0]) == INF and bool(torch.isfinite(loss[1])) and float(loss[2]) == INF and float(lse[2]) == -INF
        assert bool(torch.isnan(loss[3:5]).all()) and bool(torch.isnan(lse[3:5]).all()) and bool(torch.isfinite(loss[5]))
        keep = torch.tensor([0, 1, 2, 5], device="cuda")
        check_grad(x[keep], ids[keep].contiguous(), t[keep].contiguous(), mode)
    loss, lse, log_rest, st = run(x, ids, t, "rest", 1.0)
    assert float(loss[0]) == INF and bool(torch.isfinite(loss[1])) and float(log_rest[2]) == -INF and bool(torch.isnan(log_rest[3:5]).all())
    t[0, :] = -INF                                          # a teacher of probability 0 for all of them
    loss, _, _, _ = run(x, ids, t, "normalised", 1.0)
    assert float(loss[0]) == 0.0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_masks_of_the_lowest_value(dtype):
    x, ids, t = make(4, 3000, 8, 5, dtype, none=0.0)
    low = torch.finfo(dtype).min
    rest = torch.ones(4, 3000, dtype=torch.bool, device="cuda").scatter_(1, ids.long(), False)
    x[0, rest[0]] = low
    x[1, :1500] = low
    for mode in MODES:
        loss, lse, log_rest, _ = run(x[1:], ids[1:].contiguous(), t[1:].contiguous(), mode, 0.9)
        assert bool(torch.isfinite(lse).all())
    x[2] = low                                              # a whole row of them: every p 1 / V
    loss, lse, _, _ = run(x, ids, t, "normalised", 1.0)
    assert bool(torch.isfinite(loss[0])) and abs(float(loss[2]) - float((torch.log_softmax(t[2].double(), 0).exp() *
                                                                        (torch.log_softmax(t[2].double(), 0) + torch.log(torch.tensor(3000.0, dtype=torch.float64)).cuda())).sum())) < 1e-5
    d = torch.empty_like(x)
    k3.distill_grad(x, ids, t, lse, torch.ones(4, device="cuda"), d, status(), mode="normalised")
    assert bool(torch.isfinite(d.float()).all())


def test_scales_of_every_size():
    """The smallest and the largest scales, with logits as far apart as fp32 holds."""
    x, ids, t = make(3, 3000, 8, 11, none=0.0)
    x[1, ::2], x[1, 1::2] = -3.4e38, 3.3e38
    for scale in (1e-44, 1e-38, 1e-36, 1e-20, 1e10, 3e38):
        for mode in MODES:
            loss, lse, _, _ = run(x, ids, t, mode, scale)
            assert not bool(torch.isnan(loss).any()) and not bool(torch.isnan(lse).any()), (scale, mode)
    check(x[:1], ids[:1].contiguous(), t[:1].contiguous(), "rest", scale=1e-30)


def test_status_of_ids_past_the_vocabulary():
    x, ids, t = make(5, 700, 6, 6)
    ids[3, 2] = 700
    ids[4, 0] = 2 ** 31 - 1
    for mode in MODES:
        check(x, ids, t, mode, want_status=k3.ST_TOKEN)
        check_grad(x, ids, t, mode, want_status=k3.ST_TOKEN)


@pytest.mark.parametrize("mode", MODES)
def test_gradient_against_differences(mode):
    x, ids, t = make(3, 300, 6, 7, none=0.0)
    ids[1, 4] = -1
    _, lse, log_rest, _ = run(x, ids, t, mode, 0.8)
    d, st = torch.empty_like(x), status()
    k3.distill_grad(x, ids, t, lse, torch.ones(3, device="cuda"), d, st, log_rest=log_rest, mode=mode, scale=0.8)

    def loss(x):
        z, logp, on, at, q, tt, r_rest, rest, taken = parts(x, ids, t, mode, 0.8)
        kl = torch.where(on, q * (tt.masked_fill(~on, 0) - logp.gather(1, at)), torch.zeros_like(q)).sum()
        return float(kl + (rest * (torch.log(rest.clamp(min=1e-300)) - r_rest)).sum() if mode == "rest" else kl)

    g = torch.Generator(device="cuda").manual_seed(1)
    for _ in range(4):
        v = torch.randn(3, 300, generator=g, device="cuda", dtype=torch.float64)
        slope = (loss(x.double() + 1e-5 * v) - loss(x.double() - 1e-5 * v)) / 2e-5
        got = float((d.double() * v).sum())
        assert abs(got - slope) <= 1e-5 * float((d.double() * v).abs().sum()) + 1e-6


def test_from_the_log_probabilities_of_a_teacher():
    """The teacher's alternatives as token_logprobs gives them: a student that equals it has loss 0 against itself, of
    what the alternatives' fp32 logarithms hold, and no gradient."""
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(9, 6000, generator=g, device="cuda") * 3
    n, top = 9, 20
    tokens = torch.zeros(n, dtype=torch.int64, device="cuda")
    lp, st = torch.empty(n, device="cuda"), status()
    ids, t = torch.empty(n, top, dtype=torch.int32, device="cuda"), torch.empty(n, top, device="cuda")
    k3.token_logprobs(x, tokens, lp, st, top_ids=ids, top_logprobs=t)
    loss, lse, log_rest, _ = run(x, ids, t, "rest", 1.0)
    assert float(loss.abs().max()) < 1e-5
    d = torch.empty_like(x)
    k3.distill_grad(x, ids, t, lse, torch.ones(n, device="cuda"), d, st, log_rest=log_rest, mode="rest")
    assert float(d.abs().max()) < 1e-5 and int(st) == 0


def test_same_bits_graphs_streams_and_no_rows():
    x, ids, t = make(3, 131072, 20, 9, BF)
    a = run(x, ids, t, "rest", 0.8)
    b = run(x, ids, t, "rest", 0.8)
    assert all(torch.equal(u, v) for u, v in zip(a[:3], b[:3]))
    loss, lse, log_rest, st = torch.empty(3, device="cuda"), torch.empty(3, device="cuda"), torch.empty(3, device="cuda"), status()
    d = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k3.distill(x, ids, t, loss, st, lse=lse, log_rest=log_rest, mode="rest", scale=0.8)
        k3.distill_grad(x, ids, t, lse, loss, d, st, log_rest=log_rest, mode="rest", scale=0.8)
    graph.replay()
    first = d.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d.zero_()
        graph.replay()
    side.synchronize()
    assert torch.equal(loss, a[0]) and torch.equal(d, first) and int(st) == 0
    none = torch.empty(0, 50, device="cuda")
    z = torch.empty(0, device="cuda")
    k3.distill(none, torch.empty(0, 4, dtype=torch.int32, device="cuda"), torch.empty(0, 4, device="cuda"), z, st)
    k3.distill_grad(none, torch.empty(0, 4, dtype=torch.int32, device="cuda"), torch.empty(0, 4, device="cuda"), z, z, none, st)
