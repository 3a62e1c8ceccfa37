"""The product with bias, activation and residual in its epilogue, and its gradients, against the formulas in 64 bits.

Products of bf16 values are exact in fp32.  A sum of K of them is taken in steps of 16, and each step rounds (or cuts
off) what it holds to 24 bits: at most 2^-23 of S, the sum of the products' magnitudes, per step, so
(K / 16 + 16) 2^-23 S with the additions of partial sums.  The epilogue adds the bias and the residual (2^-24 of what
they give, each), and an activation passes an error on at most 1.2 times (its largest slope) and errs by a few units of
its value: 8 x 2^-24 of |z|.  A result in bf16 is rounded once, by 2^-8 of itself at most."""
import math

import pytest

torch = pytest.importorskip("torch")
k3 = pytest.importorskip("lossless_bf16_weight_k3huf_gb300")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
E = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: E}


@pytest.fixture(scope="module", autouse=True)
def built():
    k3._build.build()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def normal(*shape, seed, dtype=BF, std=1.0, pad=0):
    """A matrix (its rows `pad` elements apart) or a vector."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = (torch.randn(*shape[:-1], shape[-1] + pad, generator=g, device="cuda") * std).to(dtype)
    return v[..., : shape[-1]]


def scratch(n, rows, cols, grad=False, any=True):
    return torch.empty(k3.linear_scratch_bytes(n, rows, cols, grad=grad, any=any), dtype=torch.uint8, device="cuda")


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def sum_bound(a, b):
    """Bound of the error of a @ b.T."""
    K = a.shape[1]
    return (K / 16 + 16) * 2 * E * (a.double().abs() @ b.double().abs().T)


def check(got, want, bound, what):
    off = (got.double() - want).abs() - bound - HALF[got.dtype] * (want.abs() + bound)
    assert bool((off <= 0).all()), f"{what}: {float(off.max())} over its bound at {int(off.argmax())}"


def forward(n, rows, cols, act="none", y_type=BF, bias=None, res=False, z_type=None, pad=(0, 0, 0, 0), seed=1, any=True):
    x, w = normal(n, cols, seed=seed, pad=pad[0]), normal(rows, cols, seed=seed + 1, std=cols ** -0.5, pad=pad[1])
    b = None if bias is None else normal(rows, seed=seed + 2, dtype=bias)
    r = normal(n, rows, seed=seed + 3, dtype=y_type, pad=pad[2]) if res else None
    y = torch.full((n, rows + pad[3]), 7.0, dtype=y_type, device="cuda")
    z = None if z_type is None else torch.full((n, rows), 7.0, dtype=z_type, device="cuda")
    st = status()
    k3.linear(x, w, y[:, :rows], st, bias=b, residual=r, act=act, z=z, scratch=scratch(n, rows, cols, any=any))
    torch.cuda.synchronize()
    assert int(st) == 0
    assert bool((y[:, rows:] == 7.0).all())
    want = x.double() @ w.double().T + (0 if b is None else b.double())
    bound = sum_bound(x, w) + E * want.abs()
    if z is not None:
        check(z, want, bound, "z")
    bound = 1.2 * bound + 8 * E * want.abs()
    want = act64(want, act) + (0 if r is None else r.double())
    check(y[:, :rows], want, bound + E * want.abs(), "y")
    return y


SIZES = [(1, 1, 1), (1, 128, 64), (2, 7, 3), (3, 200, 130), (16, 129, 65), (17, 64, 1000), (33, 576, 8192), (64, 1000, 72), (65, 300, 513), (129, 130, 127),
         (257, 1000, 200), (300, 8192, 576), (1000, 520, 1048), (5, 8192, 8192), (2000, 3000, 712)]


@pytest.mark.parametrize("n,rows,cols", SIZES)
def test_forward(n, rows, cols):
    forward(n, rows, cols)
    forward(n, rows, cols, act="silu", y_type=F32, bias=BF, res=True, z_type=BF, seed=5)
    forward(n, rows, cols, act="gelu", y_type=BF, bias=F32, res=True, z_type=F32, pad=(8, 16, 3, 5), seed=9)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("n", [2, 40, 300])
def test_epilogues(act, n):
    for y_type in (BF, F32):
        for bias in (None, BF, F32):
            for res in (False, True):
                forward(n, 200, 320, act=act, y_type=y_type, bias=bias, res=res, seed=n)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_hold_what_the_header_says(act):
    """An fp32 exponential of u errs by (2 + 1.2 |u|) units of 2^-23 (its rounded exponent), a quotient by two; GELU's u by
    three roundings more.  So (8 + 2.4 |u|) 2^-24 of the value for SiLU, (8 + 6 |u|) for GELU, and, as the exponential is no
    part of the value where it is small, 8 x 2^-24 of |z|; a quotient by more than 2^126 is 0."""
    z = torch.cat([torch.linspace(-100, 100, 2000001, device="cuda"), -torch.logspace(-6, 2, 1000001, device="cuda"), torch.logspace(-6, 30, 1000001, device="cuda")])
    z = z[: z.numel() // 8 * 8].contiguous()
    n = z.numel()
    one, w, y, st = torch.ones(1, 8, dtype=BF, device="cuda"), torch.zeros(n, 8, dtype=BF, device="cuda"), torch.empty(1, n, device="cuda"), status()
    k3.linear(one, w, y, st, bias=z, act=act)                       # (products of 0: z is the bias)
    z = z.double()
    u = z if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    want = z / (1 + torch.exp(-u))
    off = (y[0].double() - want).abs()
    assert bool((off <= (8 + (2.4 if act == "silu" else 6) * u.abs().clamp(max=200)) * E * want.abs() + 2.0 ** -119).all())
    assert bool((off <= 8 * E * z.abs() + 2.0 ** -119).all()) and int(st) == 0


@pytest.mark.parametrize("pad", [(1, 0, 0, 0), (0, 3, 0, 0), (5, 7, 1, 1)])
def test_rows_of_any_alignment(pad):
    for n in (1, 4, 70, 300):
        forward(n, 260, 333, pad=pad)
        forward(n, 260, 336, pad=pad)
    # addresses that are no multiple of 16
    x, w = normal(9, 73, seed=1).contiguous()[:, 1:], normal(50, 73, seed=2).contiguous()[:, 1:]
    y, st = torch.empty(9, 50, device="cuda"), status()
    k3.linear(x, w, y, st, scratch=scratch(9, 50, 72))
    check(y, x.double() @ w.double().T, sum_bound(x, w), "y")
    assert int(st) == 0


def test_what_lies_between_rows_is_not_read_or_written():
    """Rows that start on 16 bytes and end inside a block of 16: NaN behind them takes no part, and stays."""
    for n, rows, cols in ((300, 261, 333), (5, 261, 333), (300, 515, 1001), (2000, 1030, 77)):
        x, w, dz = (normal(a, b, seed=a + b, std=0.3) for a, b in ((n, cols), (rows, cols), (n, rows)))
        def spread(v):
            held = torch.full((v.shape[0], (v.shape[1] + 15) // 8 * 8), float("nan"), dtype=BF, device="cuda")
            held[:, : v.shape[1]] = v
            return held[:, : v.shape[1]]
        for y_type in (BF, F32):
            y, st = torch.full((n, (rows + 15) // 8 * 8), 7.0, dtype=y_type, device="cuda"), status()
            k3.linear(spread(x), spread(w), y[:, :rows], st)
            check(y[:, :rows], x.double() @ w.double().T, sum_bound(x, w), "y")
            assert bool((y[:, rows:] == 7.0).all())
            dx, dw = torch.full((n, (cols + 15) // 8 * 8), 7.0, dtype=y_type, device="cuda"), torch.empty(rows, cols, device="cuda")
            k3.linear_grad(spread(x), spread(w), spread(dz), st, dx=dx[:, :cols], dw=dw)
            check(dx[:, :cols], dz.double() @ w.double(), sum_bound(dz, w.T), "dx")
            check(dw, dz.double().T @ x.double(), sum_bound(dz.T, x.T), "dw")
            assert bool((dx[:, cols:] == 7.0).all()) and int(st) == 0


def test_residual_in_place_and_one_row():
    x, w = normal(40, 320, seed=1), normal(200, 320, seed=2, std=0.05)
    for y_type in (BF, F32):
        r = normal(40, 200, seed=3, dtype=y_type)
        y, st = r.clone(), status()
        k3.linear(x, w, y, st, residual=y, act="silu")
        want = act64(x.double() @ w.double().T, "silu") + r.double()
        check(y, want, 1.2 * sum_bound(x, w) + 16 * E * want.abs(), "y")
    # one token of a strided view: its row's stride does not matter
    one = normal(3, 333, seed=4)[1:2, :320]
    y, st = torch.empty(1, 200, device="cuda"), status()
    k3.linear(one, w, y, st, scratch=scratch(1, 200, 320))
    check(y, one.double() @ w.double().T, sum_bound(one, w), "y")


def test_infinities_and_nan_stay_in_their_rows():
    x, w = normal(70, 192, seed=1), normal(150, 192, seed=2, std=0.1)
    x[3, 5], x[10, 0], w[20, 7] = float("inf"), float("nan"), float("-inf")
    y, st = torch.empty(70, 150, device="cuda"), status()
    k3.linear(x, w, y, st)
    want = x.double() @ w.double().T
    assert torch.equal(torch.isnan(want), torch.isnan(y))
    assert torch.equal(torch.isinf(want), torch.isinf(y)) and bool((want[torch.isinf(want)] == y[torch.isinf(want)].double()).all())
    fine = torch.isfinite(want)
    xf, wf = torch.nan_to_num(x.float(), 0, 0, 0), torch.nan_to_num(w.float(), 0, 0, 0)
    assert bool(((y.double() - want).abs()[fine] <= (sum_bound(xf, wf) + E * want.abs())[fine]).all())


@pytest.mark.parametrize("y_type", [BF, F32])
@pytest.mark.parametrize("n,rows,cols", [(1003, 4104, 192), (4001, 2056, 576), (300, 8200, 64), (2570, 1000, 1100)])
def test_residuals_of_large_results(n, rows, cols, y_type):
    """Rows of a residual that start on 16 bytes and rows that do not, tiles that end inside; in place, bit for bit the same."""
    for pad in (0, 1):
        forward(n, rows, cols, act="silu", y_type=y_type, bias=F32, res=True, z_type=BF, pad=(0, 0, pad, 0), seed=n + pad)
    x, w, r = normal(n, cols, seed=1, dtype=BF), normal(rows, cols, seed=2, dtype=BF), normal(n, rows, seed=3, dtype=y_type)
    st, y, room = status(), torch.empty_like(r), scratch(n, rows, cols)
    k3.linear(x, w, y, st, residual=r, act="gelu", scratch=room)
    k3.linear(x, w, r, st, residual=r, act="gelu", scratch=room)
    assert torch.equal(y, r) and int(st) == 0


def test_fp32_results_hold_long_sums():
    """All products positive: steps that round to one side add up.  Every 32 steps of 16 the sum leaves the tensor core,
    so the error is at most that of 32 steps and of K / 512 additions to nearest."""
    n, rows, cols = 40, 256, 32768
    x, w = normal(n, cols, seed=1).abs(), normal(rows, cols, seed=2, std=0.01).abs()
    y, st = torch.empty(n, rows, device="cuda"), status()
    k3.linear(x, w, y, st)
    want = x.double() @ w.double().T
    assert bool(((y.double() - want).abs() <= ((32 + 4) * 2 + cols / 512) * E * want).all())


def test_a_contraction_of_several_runs():
    n, rows, cols = 20, 130, 66000                              # bf16 results leave the tensor core every 65536 values
    x, w = normal(n, cols, seed=1), normal(rows, cols, seed=2, std=0.01)
    y, st = torch.empty(n, rows, dtype=BF, device="cuda"), status()
    k3.linear(x, w, y, st)
    check(y, x.double() @ w.double().T, sum_bound(x, w), "y")
    x, dz = normal(140000, 40, seed=3), normal(140000, 24, seed=4)
    dw = torch.empty(24, 40, device="cuda")
    k3.linear_grad(x, None, dz, st, dw=dw)
    check(dw, dz.double().T @ x.double(), sum_bound(dz.T, x.T), "dw")
    big, small = normal(300, 140000, seed=5), normal(260, 140000, seed=6, std=0.01)
    y = torch.empty(300, 260, dtype=BF, device="cuda")
    k3.linear(big, small, y, st)
    check(y, big.double() @ small.double().T, sum_bound(big, small), "y of pairs")
    assert int(st) == 0


def grads(n, rows, cols, dx_type=BF, add=False, pad=(0, 0, 0), seed=1, want=("dx", "dw")):
    x, w, dz = normal(n, cols, seed=seed, pad=pad[0]), normal(rows, cols, seed=seed + 1, std=0.1, pad=pad[1]), normal(n, rows, seed=seed + 2, pad=pad[2])
    dx = torch.full((n, cols), 7.0, dtype=dx_type, device="cuda")
    held = normal(rows, cols, seed=seed + 3, dtype=F32).contiguous()
    dw, st = held.clone(), status()
    k3.linear_grad(x if "dw" in want else None, w if "dx" in want else None, dz, st, dx=dx if "dx" in want else None, dw=dw if "dw" in want else None,
                   scratch=scratch(n, rows, cols, grad=True), accumulate=add)
    torch.cuda.synchronize()
    assert int(st) == 0
    if "dx" in want:
        check(dx, dz.double() @ w.double(), sum_bound(dz, w.T), "dx")
    if "dw" in want:
        ref = dz.double().T @ x.double()
        check(dw, ref + (held.double() if add else 0), sum_bound(dz.T, x.T) + E * ref.abs(), "dw")
    return dx, dw


@pytest.mark.parametrize("n,rows,cols", SIZES)
def test_gradients(n, rows, cols):
    grads(n, rows, cols)
    grads(n, rows, cols, dx_type=F32, add=True, pad=(8, 0, 16), seed=4)
    grads(n, rows, cols, pad=(1, 2, 3), seed=4)


def test_gradients_of_one_side_and_of_no_token():
    grads(70, 200, 136, want=("dx",))
    grads(70, 200, 136, want=("dw",))
    dw, st = torch.full((20, 30), 3.0, device="cuda"), status()
    none = torch.empty(0, 20, dtype=BF, device="cuda")
    k3.linear_grad(torch.empty(0, 30, dtype=BF, device="cuda"), None, none, st, dw=dw, accumulate=True)
    assert bool((dw == 3.0).all())
    k3.linear_grad(torch.empty(0, 30, dtype=BF, device="cuda"), None, none, st, dw=dw)
    assert bool((dw == 0.0).all())
    db = torch.full((20,), 3.0, device="cuda")
    k3.linear_dz(none, none, none, dbias=db)
    assert bool((db == 0.0).all())


def slope64(z, act):
    z = z.detach().requires_grad_()
    return torch.autograd.grad(act64(z, act).sum(), z)[0]


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("n,rows,pad", [(1, 1, 0), (3, 8, 0), (5, 130, 3), (200, 72, 8), (1000, 129, 0), (2000, 2048, 0), (17, 5000, 8)])
def test_dz(act, n, rows, pad):
    """act' errs by a few units: 16 x 2^-24 of 1 + |z| (its terms); the bias's sum by one unit per addition, along a
    thread's tokens and then over the partial sums, of the magnitudes' sum."""
    for z_type, dy_type, add in ((BF, BF, False), (F32, F32, True), (BF, F32, False)):
        z, dy = normal(n, rows, seed=n, dtype=z_type, std=3.0, pad=pad), normal(n, rows, seed=n + 1, dtype=dy_type, pad=pad)
        dz = torch.full((n, rows + pad), 7.0, dtype=BF, device="cuda")
        held = normal(rows, seed=n + 2, dtype=F32).contiguous()
        db = held.clone()
        k3.linear_dz(z, dy, dz[:, :rows], act=act, dbias=db, accumulate=add)
        want = dy.double() * slope64(z.double(), act)
        bound = 16 * E * (1 + z.double().abs()) * dy.double().abs()
        check(dz[:, :rows], want, bound, "dz")
        assert bool((dz[:, rows:] == 7.0).all())
        off = (db.double() - want.sum(0) - (held.double() if add else 0)).abs()
        tol = bound.sum(0) + (n / 16 + 32) * E * (want.abs().sum(0) + bound.sum(0)) + 2 * E * held.double().abs()
        assert bool((off <= tol).all())


def test_dz_in_place_without_bias_and_far_out():
    z, dy = normal(50, 64, seed=1), normal(50, 64, seed=2)
    for act in ("silu", "gelu"):
        want = dy.double() * slope64(z.double(), act)
        for into in ("dy", "z"):
            a, b = z.clone(), dy.clone()
            k3.linear_dz(a, b, b if into == "dy" else a, act=act)
            check(b if into == "dy" else a, want, 16 * E * (1 + z.double().abs()) * dy.double().abs(), into)
        far = torch.tensor([[1e30, -1e30, float("inf"), float("-inf"), 90.0, -90.0, 0.0, -0.0]], device="cuda")
        out = torch.empty(1, 8, dtype=BF, device="cuda")
        k3.linear_dz(far, torch.ones(1, 8, device="cuda"), out, act=act)
        assert torch.allclose(out.float().cpu(), torch.tensor([[1.0, 0.0, 1.0, 0.0, 1.0, 0.0, 0.5, 0.5]]), atol=1e-30)
        far[0, 0] = float("nan")
        k3.linear_dz(far, torch.ones(1, 8, device="cuda"), out, act=act)
        assert bool(torch.isnan(out[0, 0])) and not bool(torch.isnan(out[0, 1:]).any())


def test_gradient_against_differences():
    """d loss / d (x, w, bias) for loss = sum(g act(x w^T + bias)), along one direction each, by central differences in 64
    bits; dz is rounded to bf16 (2^-8 of each) before the products."""
    n, rows, cols, act = 24, 40, 56, "gelu"
    x, w, b, g = normal(n, cols, seed=1), normal(rows, cols, seed=2, std=0.2), normal(rows, seed=3, dtype=F32), normal(n, rows, seed=4)
    y, z, st = torch.empty(n, rows, device="cuda"), torch.empty(n, rows, device="cuda"), status()
    k3.linear(x, w, y, st, bias=b, act=act, z=z)
    dz, db = torch.empty(n, rows, dtype=BF, device="cuda"), torch.empty(rows, device="cuda")
    k3.linear_dz(z, g, dz, act=act, dbias=db)
    dx, dw = torch.empty(n, cols, device="cuda"), torch.empty(rows, cols, device="cuda")
    k3.linear_grad(x, w, dz, st, dx=dx, dw=dw)

    def loss(x, w, b):
        return float((g.double() * act64(x @ w.T + b, act)).sum())

    at = [x.double(), w.double(), b.double()]
    for k, got in enumerate((dx, dw, db)):
        d = normal(*got.shape, seed=10 + k, dtype=F32).double()
        h = 1e-5
        hi, lo = ([v + s * h * d if i == k else v for i, v in enumerate(at)] for s in (1, -1))
        slope = (loss(*hi) - loss(*lo)) / (2 * h)
        # the products' terms, each off by 2^-8 of itself at most
        each = dz.double().abs()
        room = (each @ w.double().abs() if k == 0 else each.T @ x.double().abs() if k == 1 else each.sum(0)) * d.abs()
        assert abs(float((got.double() * d).sum()) - slope) <= 2.0 ** -8 * float(room.sum()) + 1e-6 * abs(slope)


def test_same_bits_on_every_call_streams_and_graphs():
    n, rows, cols = 9, 700, 1600                                # a contraction shared by a cluster's CTAs
    x, w = normal(n, cols, seed=1), normal(rows, cols, seed=2, std=0.02)
    y, st = torch.empty(n, rows, device="cuda"), status()
    k3.linear(x, w, y, st)
    first = y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            y.zero_()
            k3.linear(x, w, y, st)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, first)
    dz = normal(n, rows, seed=3)
    dx, dw, sc = torch.empty(n, cols, device="cuda"), torch.zeros(rows, cols, device="cuda"), scratch(n, rows, cols, grad=True, any=False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k3.linear(x, w, y, st)
        k3.linear_grad(x, w, dz, st, dx=dx, dw=dw, scratch=sc, accumulate=True)
    y.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, first) and int(st) == 0
    ref = dz.double().T @ x.double()
    check(dw, 2 * ref, 2 * sum_bound(dz.T, x.T) + 4 * E * ref.abs(), "dw twice")


def test_decoded_weight_and_the_coded_product_agree():
    """The many-token product on a decoded tensor, and the coded matrix-vector product on its container."""
    import numpy as np
    import workloads
    rows, cols = 96, 8192
    t = workloads.normal_tensor((rows, cols), cols ** -0.5, 5)
    blob = k3.encode_layer([t])
    info = k3.layer_info(blob)
    hdr, d_blob, st = blob[: info["hdr_bytes"]], torch.from_numpy(blob).cuda(), status()
    w = torch.empty(rows * cols, dtype=BF, device="cuda")
    k3.decode_tensor(hdr, d_blob, 0, w, st)
    assert np.array_equal(w.view(torch.int16).cpu().numpy().view(np.uint16), t.reshape(-1))
    x = normal(4, cols, seed=1)
    y, v = torch.empty(4, rows, device="cuda"), torch.empty(4, rows, device="cuda")
    k3.linear(x, w.view(rows, cols), y, st)
    k3.gemv_layer_batch(hdr, d_blob, 0, cols, x, v, st, zero_y=True)
    want, bound = x.double() @ w.view(rows, cols).double().T, sum_bound(x, w.view(rows, cols))
    check(y, want, bound, "linear")
    assert bool(((v.double() - want).abs() <= cols * E * (x.double().abs() @ w.view(rows, cols).double().abs().T)).all())
    assert int(st) == 0


@pytest.mark.parametrize("n,rows,cols", [(1, 100, 4096), (9, 200, 3000), (40, 333, 5000), (100, 130, 9000), (1300, 17, 64), (2500, 40, 128)])
def test_warps_that_part_meet_again_at_the_clusters_barriers(n, rows, cols):
    """Contractions that clusters share, of tiles whose last columns or lanes lie outside, and sums of slopes over clusters
    with half a warp of columns: warps part in these before they meet the cluster.  Every call gives the same bits."""
    x, w, z, dy = normal(n, cols, seed=1), normal(rows, cols, seed=2, std=cols ** -0.5), normal(n, rows, seed=3, dtype=F32), normal(n, rows, seed=4)
    b, room, st = normal(rows, seed=5, dtype=F32), scratch(n, rows, cols, grad=True), status()
    first = None
    for _ in range(10):
        y, dx, dw = torch.empty(n, rows, device="cuda"), torch.empty(n, cols, device="cuda"), torch.empty(rows, cols, device="cuda")
        dz, db = torch.empty(n, rows, dtype=BF, device="cuda"), torch.empty(rows, device="cuda")
        k3.linear(x, w, y, st, bias=b, act="silu", scratch=room)
        k3.linear_dz(z, dy, dz, act="silu", dbias=db)
        k3.linear_grad(x, w, dz, st, dx=dx, dw=dw, scratch=room)
        now = (y, dz, db, dx, dw)
        first = first or now
        assert all(torch.equal(a, c) for a, c in zip(first, now))
    assert int(st) == 0
    want = x.double() @ w.double().T + b.double()
    check(first[0], act64(want, "silu"), 1.2 * (sum_bound(x, w) + E * want.abs()) + 8 * E * want.abs(), "y")
    want = dy.double() * slope64(z.double(), "silu")
    bound = 16 * E * (1 + z.double().abs()) * dy.double().abs()
    check(first[1], want, bound, "dz")
    assert bool(((first[2].double() - want.sum(0)).abs() <= bound.sum(0) + (n / 16 + 32) * E * (want.abs().sum(0) + bound.sum(0))).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,rows,cols,pad", [(3, 300, 1000, 0), (40, 520, 320, 0), (1003, 4104, 192, 0), (1003, 4104, 192, 1)])
def test_z_over_the_residual(n, rows, cols, pad, dtype):
    """z may be written where the residual is read, of the same type and stride: bit for bit what separate buffers give."""
    x, w, r = normal(n, cols, seed=1), normal(rows, cols, seed=2, std=0.05), normal(n, rows, seed=3, dtype=dtype, pad=pad)
    z, st = torch.empty(n, rows + pad, dtype=dtype, device="cuda")[:, :rows], status()
    y, over = torch.empty(n, rows, dtype=dtype, device="cuda"), torch.empty(n, rows, dtype=dtype, device="cuda")
    k3.linear(x, w, y, st, residual=r, act="silu", z=z)
    k3.linear(x, w, over, st, residual=r, act="silu", z=r)
    assert torch.equal(y, over) and torch.equal(z, r) and int(st) == 0


def signs(n, K, seed):
    """n x K values, zero but for one of each 16 along K, which is 1 or -1; and their sums over each 64."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    at = torch.arange(0, K, 16, device="cuda")
    at = at + (torch.rand(len(at), generator=g, device="cuda") * (K - at).clamp(max=16)).long()
    v = torch.randint(0, 2, (n, len(at)), generator=g, device="cuda").float() * 2 - 1
    x = torch.zeros(n, K, dtype=BF, device="cuda")
    x[:, at] = v.to(BF)
    return x, torch.zeros(n, (K + 63) // 64, device="cuda").index_add_(1, at // 64, v)


def steps_of(m, K):
    """m x K: row r is 1 where k / 64 is r modulo m."""
    k = torch.arange(K, device="cuda")
    w = torch.zeros(m, K, dtype=BF, device="cuda")
    w[k // 64 % m, k] = 1
    return w


def by_step(sums, m):
    """What such a product gives: whole numbers, exact in bf16 up to 256."""
    want = torch.zeros(sums.shape[0], m, device="cuda").index_add_(1, torch.arange(sums.shape[1], device="cuda") % m, sums)
    assert float(want.abs().max()) <= 256
    return want


@pytest.mark.parametrize("n,rows,cols", [(2048, 2048, 66000), (600, 3000, 66000), (20, 130, 530000), (1000, 1000, 132000), (300, 2000, 70000), (7, 1000, 140000)])
def test_every_step_of_several_runs_counts_once(n, rows, cols):
    """Results from single steps of the contraction, bit for bit: runs of 65536 values and of 512, in pairs of CTAs (the
    first two shapes) and where a cluster shares them."""
    x, sums = signs(n, cols, seed=n)
    w, want, st = steps_of(rows, cols), by_step(sums, rows), status()
    for y_type in (BF, F32):
        y = torch.empty(n, rows, dtype=y_type, device="cuda")
        k3.linear(x, w, y, st)
        assert torch.equal(y.float(), want), y_type
    # the same sums as dz W
    w = w.T.contiguous()
    for dx_type in (BF, F32):
        dx = torch.empty(n, rows, dtype=dx_type, device="cuda")
        k3.linear_grad(None, w, x, st, dx=dx, scratch=scratch(n, cols, rows, grad=True))
        assert torch.equal(dx.float(), want), dx_type
    # ... and, over the tokens, as dz^T x
    if n * rows <= 1 << 20:
        dw = torch.empty(n, rows, device="cuda")
        k3.linear_grad(w, None, x.T.contiguous(), st, dw=dw, scratch=scratch(cols, n, rows, grad=True))
        assert torch.equal(dw, want)
    assert int(st) == 0
