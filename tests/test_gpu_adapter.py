"""Low-rank adapters of many requests and their gradients, against the formulas in 64 bits.

Products of bf16 values are exact in fp32; what rounds is the additions, by at most u = 2^-23 of the running sum each
(a tensor-core accumulation may truncate), one for every 8 products or fewer partial sums, the rank-wide intermediate
(kept to 2^-16 of itself at least where the result is bf16, to 2^-22 where it is fp32) and the result.  With M the same formula over
magnitudes, the tests allow (K / 8 + 64) u M for every contraction of length K on the way, plus the result's rounding:
2^-8 of it for bf16, u for fp32."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
k3 = pytest.importorskip("lossless_bf16_weight_k3huf_gb300")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
U = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def built():
    k3._build.build()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def make(n, S, r, cols, rows, seed, kind="mixed"):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    if kind == "runs":
        ids = torch.randint(-1, S, (n,), generator=g, device="cuda").sort().values
    elif kind == "one":
        ids = torch.full((n,), S - 1, device="cuda")
    elif kind == "none":
        ids = torch.full((n,), -1, device="cuda")
    else:
        ids = torch.randint(-1, S, (n,), generator=g, device="cuda")
    return {"x": normal(n, cols), "a": normal(S, r, cols, std=cols ** -0.5), "b": normal(S, r, rows, std=r ** -0.5),
            "scales": torch.rand(S, generator=g, device="cuda") + 0.5, "ids": ids.to(torch.int32), "dy": normal(n, rows)}


def scratch_for(s, grad=False):
    S, r, cols = s["a"].shape
    size = k3.adapter_scratch_bytes(s["ids"].numel(), S, r, cols, s["b"].shape[2], grad=grad)
    return torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xEE)


def apply(s, y, base=None):
    st = status()
    k3.adapter_apply(s["x"], s["a"], s["b"], s["ids"], s["scales"], y, scratch_for(s), st, base=base)
    torch.cuda.synchronize()
    return int(st.item())


def slack(K):
    return (K / 8 + 64) * U


def rounding(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


def reference(s, base):
    """(y, tolerance before y's own rounding) in 64 bits."""
    n, rows = s["dy"].shape
    S, r, cols = s["a"].shape
    y = base.double().clone() if base is not None else torch.zeros(n, rows, dtype=torch.float64, device="cuda")
    tol = U * y.abs()
    for i in range(S):
        t = (s["ids"] == i).nonzero()[:, 0]
        x, a, b, c = s["x"][t].double(), s["a"][i].double(), s["b"][i].double(), s["scales"][i].double()
        y[t] += c * (x @ a.T) @ b
        h = c * (x @ a.T).abs()
        kept = 2.0 ** -15
        tol[t] += c * slack(cols) * (x.abs() @ a.abs().T) @ b.abs() + (slack(r) + kept) * h @ b.abs()
    return y, tol


SHAPES = [(1, 1, 1, 8, 8), (1, 3, 16, 512, 640), (5, 4, 8, 1000, 264), (17, 9, 12, 768, 2056), (33, 2, 64, 576, 8192), (70, 40, 4, 8192, 576),
          (129, 3, 128, 264, 328), (200, 64, 16, 1024, 1024), (300, 5, 32, 2048, 1024), (513, 7, 16, 72, 80), (1000, 2, 64, 1024, 776),
          (300, 100, 20, 128, 256), (400, 3, 7, 640, 648), (260, 4, 16, 333, 1001), (9, 2, 5, 7, 3), (3, 2, 33, 1, 1), (1200, 1, 128, 136, 64)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["mixed", "runs"])
@pytest.mark.parametrize("n,S,r,cols,rows", SHAPES)
def test_apply_matches_the_formula(n, S, r, cols, rows, kind, dtype):
    s = make(n, S, r, cols, rows, n * 31 + cols, kind)
    base = torch.randn(n, rows, device="cuda").to(dtype)
    for b in (base, None):
        y = torch.full((n, rows), float("nan"), device="cuda", dtype=dtype)
        assert apply(s, y, b) == 0
        want, tol = reference(s, b)
        tol = tol + rounding(dtype) * want.abs()
        assert bool(((y.double() - want).abs() <= tol).all())
        again = torch.empty_like(y)
        apply(s, again, b)
        assert torch.equal(again, y)                     # the same bits every time


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["mixed", "runs", "one"])
@pytest.mark.parametrize("n,S,r,cols,rows", [(2100, 3, 64, 1024, 1032), (1300, 40, 128, 520, 776), (4001, 2, 48, 600, 264), (9000, 6, 16, 512, 576)])
def test_apply_to_many_tokens(n, S, r, cols, rows, kind, dtype):
    """Enough factor rows for the tensor-core tiles (over 300 MB): several adapters per tile, ranks of one and two
    blocks, padded ranks, ragged last tiles."""
    s = make(n, S, r, cols, rows, n + cols, kind)
    base = torch.randn(n, rows, device="cuda").to(dtype)
    for b in (base, None):
        y = torch.full((n, rows), float("nan"), device="cuda", dtype=dtype)
        assert apply(s, y, b) == 0
        want, tol = reference(s, b)
        assert bool(((y.double() - want).abs() <= tol + rounding(dtype) * want.abs()).all())
        again = torch.empty_like(y)
        apply(s, again, b)
        assert torch.equal(again, y)
        if dtype == torch.float32:
            assert float((y.double() - want).norm() / want.norm()) < 2e-6


def test_fp32_result_keeps_fp32_precision():
    """The rank-wide intermediate is not rounded to 16 bits on the way to an fp32 result: the whole output is within
    2e-6 of the formula in the 2-norm (fp32 sums of 1024 terms err by about 1e-6 or less; a bf16 intermediate by 2e-3,
    two bf16 parts by about 3e-6)."""
    for n in (16, 700):
        s = make(n, 3, 32, 1024, 1024, 5, "runs")
        s["ids"].clamp_(min=0)
        y = torch.empty(n, 1024, device="cuda")
        assert apply(s, y) == 0
        want, _ = reference(s, None)
        assert float((y.double() - want).norm() / want.norm()) < 2e-6


@pytest.mark.parametrize("kind", ["one", "none"])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_one_adapter_or_none(kind, n):
    s = make(n, 5, 16, 256, 512, 3, kind)
    base = torch.randn(n, 512, device="cuda")
    y = torch.empty_like(base)
    assert apply(s, y, base) == 0
    want, tol = reference(s, base)
    assert bool(((y.double() - want).abs() <= tol + U * want.abs()).all())
    if kind == "none":
        assert torch.equal(y, base)


@pytest.mark.parametrize("n", [6, 300])
def test_in_place_strides_and_ids_past_the_pool(n):
    s = make(n, 4, 16, 512, 264, 8)
    for dtype, pad in ((torch.float32, 3), (torch.bfloat16, 8), (torch.bfloat16, 1)):
        wide_x = torch.randn(n, 512 + pad, device="cuda").to(torch.bfloat16)
        s["x"] = wide_x[:, :512]
        wide_y = torch.randn(n, 264 + pad, device="cuda").to(dtype)
        y, before = wide_y[:, :264], wide_y.clone()
        s["ids"][1], s["ids"][2] = 4, 1 << 20             # past the pool: no adapter, and the status bit
        assert apply(s, y, y) == k3.ST_TOKEN
        want, tol = reference(s, before[:, :264])
        assert bool(((y.double() - want).abs() <= tol + rounding(dtype) * want.abs()).all())
        assert torch.equal(wide_y[:, 264:], before[:, 264:])
        assert torch.equal(y[1:3], before[1:3, :264])


def test_no_tokens():
    s = make(0, 2, 8, 64, 64, 1)
    assert apply(s, torch.empty(0, 64, device="cuda")) == 0
    da, db = torch.full((2, 8, 64), 5.0, device="cuda"), torch.full((2, 8, 64), 5.0, device="cuda")
    k3.adapter_grad(s["x"], s["a"], s["b"], s["ids"], s["scales"], s["dy"], da, db, scratch_for(s, True), status(), accumulate=True)
    assert bool((da == 5).all()) and bool((db == 5).all())
    k3.adapter_grad(s["x"], s["a"], s["b"], s["ids"], s["scales"], s["dy"], da, db, scratch_for(s, True), status())
    assert bool((da == 0).all()) and bool((db == 0).all())


# --- gradients ------------------------------------------------------------------

def grads(s, dtype=torch.float32, base=None, held=None, want_dx=True):
    da, db = (torch.full(s[k].shape, float("nan"), device="cuda") for k in ("a", "b"))
    if held is not None:
        da.copy_(held[0])
        db.copy_(held[1])
    dx = torch.full(s["x"].shape, float("nan"), device="cuda", dtype=dtype) if want_dx else None
    st = status()
    k3.adapter_grad(s["x"], s["a"], s["b"], s["ids"], s["scales"], s["dy"], da, db, scratch_for(s, True), st, dx=dx,
                    dx_base=base if want_dx else None, accumulate=held is not None)
    torch.cuda.synchronize()
    return da, db, dx, int(st.item())


def grad_reference(s, base=None, held=None):
    n, rows = s["dy"].shape
    S, r, cols = s["a"].shape
    zero = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")  # noqa: E731
    dx = base.double().clone() if base is not None else zero(n, cols)
    da, db = (h.double().clone() for h in held) if held is not None else (zero(S, r, cols), zero(S, r, rows))
    t_dx, t_da, t_db = U * dx.abs(), U * da.abs(), U * db.abs()
    kept = 2.0 ** -15
    for i in range(S):
        t = (s["ids"] == i).nonzero()[:, 0]
        x, a, b, c, dy = s["x"][t].double(), s["a"][i].double(), s["b"][i].double(), s["scales"][i].double(), s["dy"][t].double()
        h, dh = c * x @ a.T, c * dy @ b.T
        e_h, e_dh = c * slack(cols) * (x.abs() @ a.abs().T), c * slack(rows) * (dy.abs() @ b.abs().T)
        dx[t] += dh @ a
        t_dx[t] += (e_dh + (slack(r) + kept) * dh.abs()) @ a.abs()
        da[i] += dh.T @ x
        t_da[i] += (e_dh + slack(8 * len(t)) * dh.abs()).T @ x.abs()
        db[i] += h.T @ dy
        t_db[i] += (e_h + slack(8 * len(t)) * h.abs()).T @ dy.abs()
    return (da, t_da + U * da.abs()), (db, t_db + U * db.abs()), (dx, t_dx)


def close(got, want_tol, dtype=torch.float32):
    want, tol = want_tol
    return bool(((got.double() - want).abs() <= tol + rounding(dtype) * want.abs()).all())


@pytest.mark.parametrize("kind", ["mixed", "runs"])
@pytest.mark.parametrize("n,S,r,cols,rows", SHAPES)
def test_gradients_match_the_formula(n, S, r, cols, rows, kind):
    s = make(n, S, r, cols, rows, n * 17 + rows, kind)
    for dtype in (torch.float32, torch.bfloat16):
        base = torch.randn(n, cols, device="cuda").to(dtype)
        da, db, dx, st = grads(s, dtype, base)
        ra, rb, rx = grad_reference(s, base)
        assert st == 0 and close(da, ra) and close(db, rb) and close(dx, rx, dtype)
        da2, db2, dx2, _ = grads(s, dtype, base)
        assert torch.equal(da, da2) and torch.equal(db, db2) and torch.equal(dx, dx2)
    held = (torch.randn(S, r, cols, device="cuda"), torch.randn(S, r, rows, device="cuda"))
    da, db, dx, st = grads(s, held=held, want_dx=False)
    ra, rb, _ = grad_reference(s, held=held)
    assert st == 0 and dx is None and close(da, ra) and close(db, rb)


def test_gradients_against_differences():
    """L = sum y * dY is linear in either factor alone and in x, so central differences along random directions of the
    formula in 64 bits are exact up to rounding; the kernels' gradients have the same inner products."""
    s = make(50, 4, 8, 96, 72, 11)
    g = torch.Generator(device="cuda").manual_seed(2)
    names = ("a", "b", "x")
    at = {k: s[k].double() for k in names}
    step = {k: torch.randn(s[k].shape, generator=g, device="cuda", dtype=torch.float64) for k in names}

    def loss(v):
        i = s["ids"].long()
        on = (i >= 0).double()
        h = torch.einsum("nc,nrc->nr", v["x"], v["a"][i.clamp(min=0)]) * (s["scales"].double()[i.clamp(min=0)] * on)[:, None]
        return float((torch.einsum("nr,nro->no", h, v["b"][i.clamp(min=0)]) * s["dy"].double()).sum())

    da, db, dx, _ = grads(s)
    refs = dict(zip(names, grad_reference(s)))
    for k, got in zip(names, (da, db, dx)):
        slope = (loss({**at, k: at[k] + step[k]}) - loss({**at, k: at[k] - step[k]})) / 2
        room = float(((refs[k][1] + U * refs[k][0].abs()) * step[k].abs()).sum())
        assert abs(float((got.double() * step[k]).sum()) - slope) <= room + 1e-8 * abs(slope)


@pytest.mark.parametrize("n,r", [(12, 16), (300, 16), (300, 96), (300, 5)])
def test_no_token_meets_another_adapters_values(n, r):
    """Infinities and NaN in one adapter, and in the inputs of the tokens that use it, stay with those tokens: the
    others' results are the very ones that finite values there give."""
    S, cols, rows = 5, 264, 328
    good = make(n, S, r, cols, rows, 40 + r)
    bad = {k: v.clone() for k, v in good.items()}
    bad["a"][2, :, 7] = float("inf")
    bad["b"][2, r - 1] = float("nan")
    hit = good["ids"] == 2
    bad["x"][hit] = float("nan")
    bad["dy"][hit] = float("-inf")
    none = good["ids"] < 0
    bad["x"][none], bad["dy"][none] = float("nan"), float("inf")
    for dtype in (torch.float32, torch.bfloat16):
        base = torch.randn(n, rows, device="cuda").to(dtype)
        y, z = torch.empty_like(base), torch.empty_like(base)
        assert apply(good, y, base) == 0 and apply(bad, z, base) == 0
        assert torch.equal(y[~hit], z[~hit]) and torch.equal(z[none], base[none])
        want, got = grads(good, dtype), grads(bad, dtype)
        keep = [i for i in range(S) if i != 2]
        assert torch.equal(want[0][keep], got[0][keep]) and torch.equal(want[1][keep], got[1][keep])
        assert torch.equal(want[2][~hit], got[2][~hit])
        assert bool((got[2][none] == 0).all())


def test_refusals():
    s = make(4, 2, 8, 64, 32, 1)
    y, st, sc = torch.empty(4, 32, device="cuda"), status(), scratch_for(s)
    args = (s["x"], s["a"], s["b"], s["ids"], s["scales"])
    with pytest.raises(k3.K3HufError) as e:
        k3.adapter_apply(*args, y, sc[: sc.numel() - 1], st)
    assert e.value.code == k3.E_ARG
    with pytest.raises(ValueError):
        k3.adapter_apply(*args, y[:, :31], sc, st)
    with pytest.raises(TypeError):
        k3.adapter_apply(s["x"].float(), *args[1:], y, sc, st)
    with pytest.raises(TypeError):
        k3.adapter_apply(*args, y, sc, st, base=y.to(torch.bfloat16))
    with pytest.raises(TypeError):
        k3.adapter_apply(*args[:3], s["ids"].long(), s["scales"], y, sc, st)
    with pytest.raises(ValueError):
        k3.adapter_apply(s["x"], s["a"][:, :4], *args[2:], y, sc, st)
    wide = make(4, 1, 129, 64, 32, 1)
    with pytest.raises(k3.K3HufError):
        k3.adapter_scratch_bytes(4, 1, 129, 64, 32)
    with pytest.raises(k3.K3HufError):
        k3.adapter_apply(wide["x"], wide["a"], wide["b"], wide["ids"], wide["scales"], y, sc, st)
    with pytest.raises(ValueError):
        k3.adapter_grad(*args, s["dy"], torch.empty(2, 8, 64, device="cuda"), torch.empty(2, 8, 32, device="cuda"), scratch_for(s, True), st,
                        dx_base=torch.empty(4, 64, device="cuda"))


@pytest.mark.parametrize("rank", [16, 33, 96, 5])
def test_accumulating_leaves_unused_adapters_alone(rank):
    """Adapters without a token keep every bit of what is held (-0 too, which adding 0 would make +0), whatever the
    form; those with one get held + their sum."""
    S, n, cols, rows = 9, 300, 264, 328
    s = make(n, S, rank, cols, rows, rank)
    s["ids"] = torch.where(s["ids"] % 4 == 1, s["ids"], torch.full_like(s["ids"], -1))         # adapters 1 and 5
    wide_x = torch.zeros(n, cols + 1, dtype=torch.bfloat16, device="cuda")
    wide_x[:, 1:] = s["x"]
    for x in (s["x"], wide_x[:, 1:]):                    # on 16 bytes, and not
        s["x"] = x
        held = tuple(torch.randn(s[k].shape, device="cuda") for k in ("a", "b"))
        for h in held:
            h[:, :, ::3] = -0.0
        da, db, _, st = grads(s, held=held, want_dx=False)
        ra, rb, _ = grad_reference(s, held=held)
        assert st == 0 and close(da, ra) and close(db, rb)
        unused = [i for i in range(S) if i not in (1, 5)]
        for got, h in ((da, held[0]), (db, held[1])):
            assert torch.equal(got[unused].view(torch.int32), h[unused].view(torch.int32))
        da, db, _, st = grads(s, want_dx=False)          # not accumulating, they get zeros
        assert st == 0 and bool((da[unused] == 0).all()) and bool((db[unused] == 0).all())


@pytest.mark.parametrize("form", ["few", "tiles", "any"])
def test_intermediates_beyond_the_largest_bf16(form):
    """A rank-wide intermediate that overflows fp32 is an infinity, and so is what it gives with finite factors; one
    between the largest bf16 and the largest fp32 value is finite, and so is what it gives."""
    n, S, r, cols, rows = (2100, 3, 64, 1024, 1032) if form == "tiles" else (40, 3, 64, 1024, 1032)
    s = make(n, S, r, cols, rows, 77)
    s["scales"].fill_(1.0)
    s["ids"][5], s["ids"][6] = 1, 2
    # token 5: 2^120 2^10; token 6: 2^127 (2 - 2^-7 + 2^-8 + 2^-9), rounded to bf16 an infinity
    s["x"][5], s["x"][6] = 0, 0
    s["a"][1, :, 0], s["a"][2, :, :3] = 0, 0
    s["x"][5, 0], s["a"][1, 0, 0] = 2.0 ** 120, 2.0 ** 10
    s["x"][6, :3] = 2.0 ** 127
    s["a"][2, 0, :3] = torch.tensor([2 - 2.0 ** -7, 2.0 ** -8, 2.0 ** -9], device="cuda").to(torch.bfloat16)
    s["b"][2] *= 2.0 ** -100
    s["b"][1][s["b"][1] == 0] = 1.0                      # (0 times infinity is NaN)
    s["dy"][5], s["dy"][6] = 0, 0
    if form == "any":
        wide = torch.zeros(n, cols + 1, dtype=torch.bfloat16, device="cuda")
        wide[:, 1:] = s["x"]
        s["x"] = wide[:, 1:]
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.full((n, rows), float("nan"), device="cuda", dtype=dtype)
        assert apply(s, y) == 0
        assert torch.equal(y[5].float(), torch.sign(s["b"][1, 0].float()) * float("inf"))
        want = float(np.float32(2.0 ** 127 * (2 - 2.0 ** -9))) * s["b"][2, 0].double()
        # (the other rank rows' factors are 0 times theirs)
        got = y[6].double()
        assert bool(((got - want).abs() <= (2.0 ** -15 + rounding(dtype)) * want.abs()).all())
    # the same in the gradients: dh of token 5 overflows, of token 6 lies in between
    s = make(n, S, r, cols, rows, 78)
    s["scales"].fill_(1.0)
    s["ids"][s["ids"] == 1] = 0                          # token 5 alone has adapter 1, token 6 adapter 2
    s["ids"][s["ids"] == 2] = 0
    s["ids"][5], s["ids"][6] = 1, 2
    s["dy"][5], s["dy"][6] = 0, 0
    s["b"][1, :, 0], s["b"][2, :, :3] = 0, 0
    s["dy"][5, 0], s["b"][1, 0, 0] = 2.0 ** 120, 2.0 ** 10
    s["dy"][6, :3] = 2.0 ** 127
    s["b"][2, 0, :3] = torch.tensor([2 - 2.0 ** -7, 2.0 ** -8, 2.0 ** -9], device="cuda").to(torch.bfloat16)
    s["a"][2] *= 2.0 ** -100
    s["x"][6] *= 2.0 ** -100
    s["a"][1][s["a"][1] == 0] = 1.0
    s["x"][5][s["x"][5] == 0] = 1.0
    if form == "any":
        wide = torch.zeros(n, cols + 1, dtype=torch.bfloat16, device="cuda")
        wide[:, 1:] = s["x"]
        s["x"] = wide[:, 1:]
    da, db, dx, st = grads(s)
    dh = float(np.float32(2.0 ** 127 * (2 - 2.0 ** -9)))
    assert st == 0
    assert torch.equal(dx[5], torch.sign(s["a"][1, 0].float()) * float("inf"))
    assert torch.equal(da[1, 0], torch.sign(s["x"][5].float()) * float("inf")) and bool((da[1, 1:] == 0).all())
    for got, factor in ((dx[6], s["a"][2, 0]), (da[2, 0], s["x"][6])):
        want = dh * factor.double()
        assert bool(((got.double() - want).abs() <= 2.0 ** -15 * want.abs()).all())


def test_more_rows_than_a_grid_has_column_blocks():
    """One token and 34 million rows: few enough factor bytes for the form of few tokens, whose grid takes 65535
    blocks of 512 rows."""
    rows = 65535 * 512 + 8
    s = make(1, 1, 1, 8, 8, 3)
    s["ids"].fill_(0)
    s["b"] = (torch.arange(rows, device="cuda") % 251 - 125).to(torch.bfloat16).view(1, 1, rows)
    h = float((s["x"].double() @ s["a"][0].double().T * s["scales"].double()[0]).item())
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.full((1, rows), float("nan"), device="cuda", dtype=dtype)
        st = status()
        k3.adapter_apply(s["x"], s["a"], s["b"], s["ids"], s["scales"], y, scratch_for(s), st)
        torch.cuda.synchronize()
        want = s["b"][0].double() * h
        assert st.item() == 0
        # (eight products; see the docstring at the top)
        scale = float(s["scales"][0].double() * (s["x"].double().abs() @ s["a"][0].double().abs().T).item())
        tol = s["b"][0].double().abs() * ((slack(8) + slack(1)) * scale + 2.0 ** -15 * abs(h)) + rounding(dtype) * want.abs()
        assert bool(((y.double() - want).abs() <= tol).all())


# --- the tensor-core forms where the tests above run the others: over 300 MB of factor rows -------------------------

MANY = (2100, 4, 64, 1024, 1032)                         # 553 MB; a ragged last tile, rows that end inside a column tile


@pytest.mark.parametrize("dtype,pad", [(torch.float32, 4), (torch.bfloat16, 8), (torch.float32, 64)])
def test_tiles_in_place_strides_and_ids_past_the_pool(dtype, pad):
    n, S, r, cols, rows = MANY
    s = make(n, S, r, cols, rows, 81)
    wide_x = torch.randn(n, cols + 8, device="cuda").to(torch.bfloat16)
    s["x"] = wide_x[:, :cols]
    wide_y = torch.randn(n, rows + pad, device="cuda").to(dtype)
    y, before = wide_y[:, :rows], wide_y.clone()
    past = torch.tensor([1, 130, 2099], device="cuda")
    s["ids"][past] = torch.tensor([S, 1 << 20, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    assert apply(s, y, y) == k3.ST_TOKEN
    want, tol = reference(s, before[:, :rows])
    assert bool(((y.double() - want).abs() <= tol + rounding(dtype) * want.abs()).all())
    assert torch.equal(wide_y[:, rows:], before[:, rows:])
    assert torch.equal(y[past], before[past, :rows])


@pytest.mark.parametrize("kind", ["one", "none"])
def test_tiles_of_one_adapter_or_none(kind):
    n, S, r, cols, rows = MANY
    s = make(n, S, r, cols, rows, 82, kind)
    for dtype in (torch.float32, torch.bfloat16):
        base = torch.randn(n, rows, device="cuda").to(dtype)
        for b in (base, None):
            y = torch.full_like(base, float("nan"))
            assert apply(s, y, b) == 0
            want, tol = reference(s, b)
            assert bool(((y.double() - want).abs() <= tol + rounding(dtype) * want.abs()).all())
            if kind == "none":
                assert torch.equal(y, base if b is not None else torch.zeros_like(base))


@pytest.mark.parametrize("r", [64, 96, 50])
def test_tiles_keep_adapters_apart(r):
    """As test_no_token_meets_another_adapters_values, forward."""
    n, S, _, cols, rows = MANY
    good = make(n, S, r, cols, rows, 83 + r)
    bad = {k: v.clone() for k, v in good.items()}
    bad["a"][2, :, 7] = float("inf")
    bad["b"][2, r - 1] = float("nan")
    hit, none = good["ids"] == 2, good["ids"] < 0
    bad["x"][hit] = float("nan")
    bad["x"][none] = float("inf")
    for dtype in (torch.float32, torch.bfloat16):
        base = torch.randn(n, rows, device="cuda").to(dtype)
        y, z = torch.empty_like(base), torch.empty_like(base)
        assert apply(good, y, base) == 0 and apply(bad, z, base) == 0
        assert torch.equal(y[~hit], z[~hit]) and torch.equal(z[none], base[none])


def test_tiles_keep_fp32_precision():
    """As test_fp32_result_keeps_fp32_precision: two bf16 parts of a normal intermediate are off by 2.4e-6 of it in the
    2-norm, and so is what they give; three hold all of its 24 bits.  dx is the same product."""
    n, S, r, cols, rows = MANY
    s = make(n, S, r, cols, rows, 84, "runs")
    s["ids"].clamp_(min=0)
    y = torch.empty(n, rows, device="cuda")
    assert apply(s, y) == 0
    want, _ = reference(s, None)
    assert float((y.double() - want).norm() / want.norm()) < 2e-6
    for shape in (MANY, (300, 3, 32, 1024, 1032), (260, 2, 128, 520, 264)):
        s = make(*shape, 85, "runs")
        s["ids"].clamp_(min=0)
        _, _, dx, st = grads(s)
        want, _ = grad_reference(s)[2]
        assert st == 0 and float((dx.double() - want).norm() / want.norm()) < 2e-6


@pytest.mark.parametrize("dtype,pad", [(torch.float32, 4), (torch.bfloat16, 8)])
@pytest.mark.parametrize("n,r", [(300, 16), (270, 80)])
def test_gradients_in_place_strides_and_ids_past_the_pool(n, r, dtype, pad):
    """dx_base is dx; rows of x, dy and dx further apart than their columns; ids past the pool, which take no part."""
    S, cols, rows = 5, 264, 328
    s = make(n, S, r, cols, rows, 86)
    s["x"] = torch.randn(n, cols + 8, device="cuda").to(torch.bfloat16)[:, :cols]
    s["dy"] = torch.randn(n, rows + 16, device="cuda").to(torch.bfloat16)[:, :rows]
    past = torch.tensor([0, 129, n - 1], device="cuda")
    s["ids"][past] = torch.tensor([S, 1 << 20, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    wide = torch.randn(n, cols + pad, device="cuda").to(dtype)
    dx, before = wide[:, :cols], wide.clone()
    da, db = (torch.full(s[k].shape, float("nan"), device="cuda") for k in ("a", "b"))
    st = status()
    k3.adapter_grad(s["x"], s["a"], s["b"], s["ids"], s["scales"], s["dy"], da, db, scratch_for(s, True), st, dx=dx, dx_base=dx)
    torch.cuda.synchronize()
    ra, rb, rx = grad_reference(s, before[:, :cols])
    assert st.item() == k3.ST_TOKEN
    assert close(da, ra) and close(db, rb) and close(dx, rx, dtype)
    assert torch.equal(wide[:, cols:], before[:, cols:]) and torch.equal(dx[past], before[past, :cols])


@pytest.mark.parametrize("form", ["few", "tiles", "any"])
def test_tokens_without_an_adapter_keep_the_base_bits(form):
    """y = base, to the sign of its zeros; the same of dx."""
    n, S, r, cols, rows = MANY if form == "tiles" else (40, 3, 16, 264, 328)
    s = make(n, S, r, cols, rows, 91)
    s["ids"][::3] = -1
    if form == "any":
        wide = torch.zeros(n, cols + 1, dtype=torch.bfloat16, device="cuda")
        wide[:, 1:] = s["x"]
        s["x"] = wide[:, 1:]
    none = s["ids"] < 0
    for dtype, bits in ((torch.float32, torch.int32), (torch.bfloat16, torch.int16)):
        base, dx_base = torch.randn(n, rows, device="cuda").to(dtype), torch.randn(n, cols, device="cuda").to(dtype)
        base[:, ::5], dx_base[:, ::5] = -0.0, -0.0
        y = torch.empty_like(base)
        assert apply(s, y, base) == 0
        assert torch.equal(y[none].view(bits), base[none].view(bits))
        dx = grads(s, dtype, dx_base)[2]
        assert torch.equal(dx[none].view(bits), dx_base[none].view(bits))
