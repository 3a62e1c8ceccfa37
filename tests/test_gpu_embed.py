"""Rows of a coded embedding table and the gradient of the lookup.

The lookup is exact: the decoded value times the fp32 scale, rounded once, so
it is compared bit for bit with the oracle's decode.  The gradient is a sum of
c fp32 terms per row (c tokens of that id) and a product with the scale, each
rounded by at most 2^-24 of the sum of magnitudes: the tests allow
(c + 4) 2^-24 of scale x sum |dY|."""
import numpy as np
import pytest

import oracle
import workloads

torch = pytest.importorskip("torch")
k3 = pytest.importorskip("lossless_bf16_weight_k3huf_gb300")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.fixture(scope="module", autouse=True)
def built():
    k3._build.build()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def table_of(blob, tensor, cols):
    rc, out = oracle.decode_layer(blob)
    assert rc == 0
    t = k3.tensor_info(blob, tensor)
    w = out[t["out_offset"]: t["out_offset"] + 2 * t["n_values"]].view(np.int16).copy()
    return torch.from_numpy(w).view(torch.bfloat16).reshape(-1, cols)


def expect(table, ids, scale, dtype):
    rows = table.shape[0]
    i = torch.as_tensor(ids, dtype=torch.int64)
    ok = (i >= 0) & (i < rows)
    y = table[i.clamp(0, rows - 1)].float() * np.float32(scale)
    return torch.where(ok[:, None], y, torch.zeros_like(y)).to(dtype)


def lookup(blob, tensor, cols, ids, scale=1.0, dtype=torch.bfloat16, id_dtype=torch.int64, pad=0):
    hdr = blob[: k3.layer_info(blob)["hdr_bytes"]]
    d = torch.from_numpy(blob).cuda()
    i = torch.as_tensor(ids, dtype=id_dtype).cuda()
    whole = torch.full((len(ids), cols + pad), 7.0, dtype=dtype, device="cuda")
    out = whole[:, :cols]
    st = status()
    k3.embed_layer(hdr, d, tensor, cols, i, out, st, scale=scale)
    torch.cuda.synchronize()
    assert bool((whole[:, cols:] == 7.0).all())
    return out.cpu(), int(st.item())


def same_bits(a, b):
    view = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    return torch.equal(a.contiguous().view(view), b.contiguous().view(view))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(40, 8192), (129, 576), (300, 257), (1000, 1), (77, 24), (5, 4096), (9, 10000), (64, 256), (33, 2056)])
def test_rows_match_the_oracle(rows, cols, dtype):
    w = workloads.normal_tensor((rows, cols), 0.02, rows * 7 + cols)
    blob = oracle.encode_layer([w])
    rng = np.random.default_rng(cols)
    for n in (1, 3, 50):
        ids = rng.integers(0, rows, n)
        got, st = lookup(blob, 0, cols, ids, scale=1.7, dtype=dtype)
        assert st == 0
        assert same_bits(got, expect(table_of(blob, 0, cols), ids, 1.7, dtype))


@pytest.mark.parametrize("chunk,sub", [(4096, 256), (4096, 0), (512, 64), (100, 20), (1000, 1000), (7, 1), (8192, 256)])
def test_any_container_layout(chunk, sub):
    ts = [workloads.heavy_tail(seed=5, n=40 * 640).reshape(40, 640), workloads.normal_tensor((33, 96), 0.5, 9)]
    blob = oracle.encode_layer(ts, chunk_syms=chunk, sub_syms=sub)
    ids = np.random.default_rng(3).integers(0, 33, 25)
    for tensor, cols in ((0, 640), (1, 96), (1, 32)):
        got, st = lookup(blob, tensor, cols, ids, scale=0.5)
        assert st == 0
        assert same_bits(got, expect(table_of(blob, tensor, cols), ids, 0.5, torch.bfloat16))


@pytest.mark.parametrize("chunk,sub", [(4096, 256), (3000, 100)])
def test_rows_across_a_stripe_boundary(chunk, sub):
    cols = 3001                                        # does not divide 2^25
    rows = (1 << 25) // cols + 3
    w = workloads.normal_tensor((rows, cols), 0.02, 12).reshape(rows, cols)
    blob = k3.encode_layer([w], chunk_syms=chunk, sub_syms=sub)
    ids = [rows - 1, rows - 2, rows - 3, rows - 4, rows - 5, 0, 17]
    got, st = lookup(blob, 0, cols, ids)
    assert st == 0
    want = torch.from_numpy(np.ascontiguousarray(w[ids]).view(np.int16)).view(torch.bfloat16)
    assert same_bits(got, want)


def test_ids_none_past_the_table_and_repeated():
    w = workloads.normal_tensor((50, 320), 0.02, 21)
    blob = oracle.encode_layer([w])
    ids = [-1, 3, 3, 3, -7, 49, 0]
    for id_dtype in (torch.int32, torch.int64):
        got, st = lookup(blob, 0, 320, ids, id_dtype=id_dtype, pad=5)
        assert st == 0
        assert same_bits(got, expect(table_of(blob, 0, 320), ids, 1.0, torch.bfloat16))
        got, st = lookup(blob, 0, 320, ids + [50], id_dtype=id_dtype)
        assert st == k3.ST_TOKEN
        assert same_bits(got, expect(table_of(blob, 0, 320), ids + [50], 1.0, torch.bfloat16))
    assert lookup(blob, 0, 320, [1 << 40], id_dtype=torch.int64)[1] == k3.ST_TOKEN
    got, st = lookup(blob, 0, 320, [])
    assert st == 0 and got.shape == (0, 320)


@pytest.mark.parametrize("pad", [0, 1, 8])
def test_output_strides(pad):
    w = workloads.normal_tensor((31, 584), 0.02, 22)
    blob = oracle.encode_layer([w])
    ids = np.arange(31)[::-1].copy()
    for dtype in (torch.bfloat16, torch.float32):
        got, st = lookup(blob, 0, 584, ids, scale=3.0, dtype=dtype, pad=pad)
        assert st == 0 and same_bits(got, expect(table_of(blob, 0, 584), ids, 3.0, dtype))


def test_single_symbol_and_wide_tables():
    """A table whose high bytes are all equal (one 1-bit code), and one with every high byte."""
    one = np.full((20, 512), 0x3F80, np.uint16) + np.arange(512, dtype=np.uint16)[None, :] % 64
    every = np.random.default_rng(1).integers(0, 1 << 16, (64, 512)).astype(np.uint16)
    every[(every & 0x7F80) == 0x7F80] &= 0x3FFF         # (no NaN: their products need not keep their bits)
    for w in (one, every):
        blob = oracle.encode_layer([w])
        ids = np.arange(w.shape[0])
        got, st = lookup(blob, 0, 512, ids)
        assert st == 0 and same_bits(got, expect(table_of(blob, 0, 512), ids, 1.0, torch.bfloat16))


def test_corrupt_stream_sets_a_status_bit_and_stays_inside():
    """Flipped bits in the container's index and stream, on a copy that the host header does not see."""
    w = workloads.heavy_tail(seed=8, n=64 * 1024).reshape(64, 1024)
    blob = oracle.encode_layer([w])
    info = k3.layer_info(blob)
    first = info["hdr_bytes"]
    rng = np.random.default_rng(4)
    for at in list(range(first, first + 32, 4)) + [int(v) for v in rng.integers(first + 32, first + 3000, 12)]:
        bad = blob.copy()
        bad[at] ^= 0x41
        d = torch.from_numpy(bad).cuda()
        out = torch.empty((64, 1024), dtype=torch.bfloat16, device="cuda")
        st = status()
        k3.embed_layer(blob[:first], d, 0, 1024, torch.arange(64, device="cuda"), out, st)
        torch.cuda.synchronize()
        same = same_bits(out.cpu(), expect(table_of(blob, 0, 1024), np.arange(64), 1.0, torch.bfloat16))
        assert st.item() != 0 or same or at >= first + 32  # (a flipped code may decode to another whole stream)


def test_on_a_stream_of_its_own():
    w = workloads.normal_tensor((100, 1024), 0.02, 31)
    blob = oracle.encode_layer([w])
    hdr = blob[: k3.layer_info(blob)["hdr_bytes"]]
    d = torch.from_numpy(blob).cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.empty((100, 1024), dtype=torch.bfloat16, device="cuda")
    st = status()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ids = torch.arange(100, device="cuda").flip(0).contiguous()
        k3.embed_layer(hdr, d, 0, 1024, ids, out, st)
    side.synchronize()
    assert st.item() == 0 and same_bits(out.cpu(), expect(table_of(blob, 0, 1024), np.arange(100)[::-1].copy(), 1.0, torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("chunk,sub", [(4096, 32), (4096, 8), (1024, 16), (960, 96), (3000, 24)])
def test_sub_streams_that_are_no_whole_rounds(chunk, sub, dtype):
    """Sub-streams whose length is not a multiple of the 64 values that are decoded and stored at a time, enough of
    them that warps take 32 whole ones at once: nothing beyond a sub-stream is written, in the rows or behind them."""
    rows, cols = 64, 9600
    w = workloads.normal_tensor((rows, cols), 0.02, chunk + sub)
    blob = k3.encode_layer([w], chunk_syms=chunk, sub_syms=sub)
    n = 200 if sub <= 32 else 600                        # 600 rows of 100 or more: over 45000 units
    ids = np.random.default_rng(sub).integers(0, rows, n)
    buf = torch.full(((n + 1) * cols,), 7.0, dtype=dtype, device="cuda")
    out, st = buf[: n * cols].view(n, cols), status()
    k3.embed_layer(blob[: k3.layer_info(blob)["hdr_bytes"]], torch.from_numpy(blob).cuda(), 0, cols, torch.as_tensor(ids).cuda(), out, st, scale=1.7)
    torch.cuda.synchronize()
    table = torch.from_numpy(w.view(np.int16)).view(torch.bfloat16).reshape(rows, cols)
    assert st.item() == 0
    assert bool((buf[n * cols:] == 7.0).all())
    assert same_bits(out.cpu(), expect(table, ids, 1.7, dtype))


@pytest.mark.parametrize("chunk", [(1 << 25) + 1, 1 << 31, (1 << 32) - (1 << 25), (1 << 32) - (1 << 25) + 1, (1 << 32) - 1])
def test_chunks_longer_than_a_stripe(chunk):
    """One chunk and one sub-stream per stripe, up to the largest chunk size that the header holds."""
    w = workloads.normal_tensor((10, 64), 0.02, 17)
    blob = oracle.encode_layer([w], chunk_syms=chunk, sub_syms=256)
    ids = [9, 0, 3, -1, 3]
    for dtype in (torch.bfloat16, torch.float32):
        got, st = lookup(blob, 0, 64, ids, scale=0.5, dtype=dtype)
        assert st == 0
        assert same_bits(got, expect(table_of(blob, 0, 64), ids, 0.5, dtype))


def big_table(rows, cols, kind):
    if kind == "normal":
        return workloads.normal_tensor((rows, cols), 0.02, rows + cols)
    w = np.random.default_rng(rows).integers(0, 1 << 16, (rows, cols)).astype(np.uint16)   # 8-bit codes
    w[(w & 0x7F80) == 0x7F80] &= 0x3FFF                  # (no NaN)
    return w


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,cols,kind", [(400, 8192, "normal"), (1000, 8192, "normal"), (1500, 8192, "normal"), (4000, 8192, "normal"),
                                         (1500, 8191, "normal"), (3000, 8192, "bytes"), (1500, 8200, "bytes"), (1500, 8191, "bytes")])
def test_calls_that_fill_the_gpu(n, cols, kind, dtype):
    """8, 16 and 32 units per item, items past a warp's first, whole rows or rows that start anywhere, and bits that
    take several passes ("bytes": 32 units of 16 pieces), some of them of no row."""
    rows = 500
    w = big_table(rows, cols, kind)
    blob = k3.encode_layer([w])
    rng = np.random.default_rng(n)
    ids = rng.integers(0, rows, n)
    for none in (False, True):
        if none:
            ids[rng.random(n) < 0.1] = -1
        buf = torch.full(((n + 1) * cols,), 7.0, dtype=dtype, device="cuda")
        out, st = buf[: n * cols].view(n, cols), status()
        k3.embed_layer(blob[: k3.layer_info(blob)["hdr_bytes"]], torch.from_numpy(blob).cuda(), 0, cols, torch.as_tensor(ids).cuda(), out, st, scale=0.5)
        torch.cuda.synchronize()
        table = torch.from_numpy(w.view(np.int16)).view(torch.bfloat16).reshape(rows, cols)
        assert st.item() == 0 and bool((buf[n * cols:] == 7.0).all())
        assert same_bits(out.cpu(), expect(table, ids, 0.5, dtype))


def test_corrupt_indexes_are_found():
    """Every flipped bit of a chunk's or a sub-stream's first bit sets a status bit where the rows meet the whole of
    it (the sub-stream before it, or the chunk's last, does not end where the next begins); nothing behind the rows is
    written, with these or with flipped bits of the stream."""
    rows, cols = 64, 1024
    w = workloads.heavy_tail(seed=8, n=rows * cols).reshape(rows, cols)
    blob = oracle.encode_layer([w])
    hdr = k3.layer_info(blob)["hdr_bytes"]
    chunks, subs = rows * cols // 4096, 15               # 15 recorded starts in each chunk of 16 sub-streams
    first = hdr + 32
    index = first + 4 * chunks + 2 * chunks * subs
    rng = np.random.default_rng(9)
    flips = [(first + 4 * c, 1 << int(rng.integers(0, 8))) for c in range(chunks)]
    flips += [(int(at), 1 << int(rng.integers(0, 8))) for at in rng.integers(first + 4 * chunks, index, 40)]
    stream = [(int(at), 0xFF) for at in rng.integers(index + 16, index + 4000, 20)]
    for at, mask in flips + stream:
        bad = blob.copy()
        bad[at] ^= mask
        buf = torch.full(((rows + 1) * cols,), 7.0, dtype=torch.bfloat16, device="cuda")
        st = status()
        k3.embed_layer(blob[:hdr], torch.from_numpy(bad).cuda(), 0, cols, torch.arange(rows, device="cuda"), buf[: rows * cols].view(rows, cols), st)
        torch.cuda.synchronize()
        assert bool((buf[rows * cols:] == 7.0).all())
        assert at >= index or st.item() != 0, (at - first, mask)


# --- gradient -----------------------------------------------------------------

def grad_of(ids, dy, rows, scale, held=None, id_dtype=torch.int64):
    n, cols = dy.shape
    g = torch.full((rows, cols), float("nan"), device="cuda") if held is None else held.clone()
    scratch = torch.empty(k3.embed_grad_scratch_bytes(n, rows, cols), dtype=torch.uint8, device="cuda").fill_(0xEE)
    st = status()
    k3.embed_grad(torch.as_tensor(ids, dtype=id_dtype).cuda(), dy, g, scratch, st, scale=scale, accumulate=held is not None)
    torch.cuda.synchronize()
    return g, int(st.item())


def grad_ref(ids, dy, rows, scale, held=None):
    """(gradient in 64 bits, tolerance)"""
    d = dy.double().cpu().numpy()
    want = np.zeros((rows, d.shape[1])) if held is None else held.double().cpu().numpy()
    mag, count = np.zeros_like(want), np.zeros(rows)
    for t, i in enumerate(ids):
        if 0 <= i < rows:
            want[i] += float(np.float32(scale)) * d[t]
            mag[i] += abs(scale) * np.abs(d[t])
            count[i] += 1
    tol = (count + 4)[:, None] * 2.0 ** -24 * mag + (2.0 ** -23 * np.abs(want) if held is not None else 0)
    return want, tol


def long_tail(rng, n, rows):
    return (np.exp(rng.random(n) * np.log(rows)).astype(np.int64) - 1).clip(0, rows - 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,rows,cols", [(1, 5, 8), (2, 3, 1), (40, 7, 33), (300, 1000, 64), (1025, 300, 136), (3000, 11, 24),
                                         (5000, 40000, 8), (20000, 999, 40), (33, 70000, 4), (513, 2, 2050)])
def test_gradient_matches_the_formula(n, rows, cols, dtype):
    rng = np.random.default_rng(n + rows)
    ids = long_tail(rng, n, rows)
    ids[rng.random(n) < 0.05] = -1
    dy = torch.from_numpy(rng.standard_normal((n, cols)).astype(np.float32)).to(dtype).cuda()
    for held in (None, torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).cuda()):
        g, st = grad_of(ids, dy, rows, 2.5, held)
        assert st == 0
        want, tol = grad_ref(ids, dy, rows, 2.5, held)
        assert np.all(np.abs(g.double().cpu().numpy() - want) <= tol)
        again, _ = grad_of(ids, dy, rows, 2.5, held)
        assert torch.equal(again, g)                    # the same bits every time


def test_gradient_of_one_repeated_id_and_of_none():
    dy = torch.randn(4097, 72, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    for ids, rows in (([3] * 4097, 9), ([-1] * 4097, 9), ([0] * 2000 + [8] * 2097, 9)):
        g, st = grad_of(ids, dy, rows, 1.0)
        want, tol = grad_ref(ids, dy, rows, 1.0)
        assert st == 0 and np.all(np.abs(g.double().cpu().numpy() - want) <= tol)
    g, st = grad_of([2, 9, 1 << 33], dy[:3], 9, 1.0)
    want, tol = grad_ref([2], dy[:1], 9, 1.0)
    assert st == k3.ST_TOKEN and np.all(np.abs(g.double().cpu().numpy() - want) <= tol)
    g, st = grad_of([], dy[:0], 9, 1.0)
    assert st == 0 and bool((g == 0).all())
    held = torch.ones(9, 72, device="cuda")
    assert torch.equal(grad_of([], dy[:0], 9, 1.0, held)[0], held)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,rows,cols", [(1100, 60, 1032), (3000, 4000, 2056), (2000, 37, 3001), (17000, 300, 1056)])
def test_gradient_of_wide_tables(n, rows, cols, dtype):
    """More than 1024 tokens and columns: several slabs of columns, for ids with few tokens and for those with many;
    17000 tokens take two blocks."""
    rng = np.random.default_rng(n + cols)
    ids = long_tail(rng, n, rows)
    ids[rng.random(n) < 0.05] = -1
    ids[: 40] = rows - 1                                 # (more than 32 of the last id too)
    dy = torch.from_numpy(rng.standard_normal((n, cols)).astype(np.float32)).to(dtype).cuda()
    for held in (None, torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).cuda()):
        g, st = grad_of(ids, dy, rows, 0.7, held)
        assert st == 0
        want, tol = grad_ref(ids, dy, rows, 0.7, held)
        assert np.all(np.abs(g.double().cpu().numpy() - want) <= tol)
        again, _ = grad_of(ids, dy, rows, 0.7, held)
        assert torch.equal(again, g)
        if held is not None:
            unused = np.setdiff1d(np.arange(rows), ids)
            assert torch.equal(g[unused], held[unused])


def test_gradient_strides_and_int32_ids():
    rng = np.random.default_rng(5)
    for pad in (1, 4, 8):
        whole = torch.randn(200, 48 + pad, device="cuda").to(torch.bfloat16)
        dy = whole[:, :48]
        ids = rng.integers(0, 37, 200)
        g, st = grad_of(ids, dy, 37, 0.3, id_dtype=torch.int32)
        want, tol = grad_ref(ids, dy, 37, 0.3)
        assert st == 0 and np.all(np.abs(g.double().cpu().numpy() - want) <= tol)


def test_gradient_against_differences():
    """The lookup is linear in the table, so a central difference of L = sum out * dY along a random direction is exact
    up to 64-bit rounding; the kernel's gradient must have the same inner product with the direction."""
    rng = np.random.default_rng(6)
    rows, cols, n, scale = 40, 56, 90, 1.25
    w, direction = rng.standard_normal((rows, cols)), rng.standard_normal((rows, cols))
    ids = rng.integers(0, rows, n)
    dy = torch.from_numpy(rng.standard_normal((n, cols)).astype(np.float32)).cuda()
    d = dy.double().cpu().numpy()

    def loss(table):
        return float((scale * table[ids] * d).sum())

    slope = (loss(w + direction) - loss(w - direction)) / 2
    g, _ = grad_of(ids, dy, rows, scale)
    _, tol = grad_ref(ids, dy, rows, scale)
    got = float((g.double().cpu().numpy() * direction).sum())
    assert abs(got - slope) <= float((tol * np.abs(direction)).sum()) + 1e-9


def test_refusals():
    blob = oracle.encode_layer([workloads.normal_tensor((10, 64), 0.02, 3)])
    hdr = blob[: k3.layer_info(blob)["hdr_bytes"]]
    d, st = torch.from_numpy(blob).cuda(), status()
    ids, out = torch.arange(4, device="cuda"), torch.empty((4, 64), dtype=torch.bfloat16, device="cuda")
    for tensor, cols in ((1, 64), (0, 63)):
        with pytest.raises(k3.K3HufError) as e:
            k3.embed_layer(hdr, d, tensor, cols, ids, torch.empty((4, cols), dtype=torch.bfloat16, device="cuda"), st)
        assert e.value.code == k3.E_ARG
    with pytest.raises(k3.K3HufError):
        k3.embed_layer(hdr, d, 0, 64, ids, out, st, layer_bytes=blob.size - 1)
    with pytest.raises(ValueError):
        k3.embed_layer(hdr, d, 0, 64, ids, out[:3], st)
    with pytest.raises(ValueError):
        k3.embed_layer(hdr, d, 0, 64, ids, torch.empty((64, 4), dtype=torch.bfloat16, device="cuda").T, st)
    with pytest.raises(TypeError):
        k3.embed_layer(hdr, d, 0, 64, ids, out.half(), st)
    with pytest.raises(TypeError):
        k3.embed_layer(hdr, d, 0, 64, ids.float(), out, st)
    with pytest.raises(TypeError):
        k3.embed_layer(hdr, d, 0, 64, ids, out.cpu(), st)
    dy, g = torch.zeros(4, 64, device="cuda"), torch.zeros(10, 64, device="cuda")
    scratch = torch.empty(k3.embed_grad_scratch_bytes(4, 10, 64), dtype=torch.uint8, device="cuda")
    with pytest.raises(k3.K3HufError):
        k3.embed_grad(ids, dy, g, scratch[: scratch.numel() - 1], st)
    with pytest.raises(TypeError):
        k3.embed_grad(ids, dy, g.double(), scratch, st)
    with pytest.raises(ValueError):
        k3.embed_grad(ids, dy[:, :32], g, scratch, st)
