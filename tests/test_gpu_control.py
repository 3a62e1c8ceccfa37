"""Penalties for repeated tokens, biases and grammar masks on logits, against the formula in 64 bits, row by row.

The kernel's fp32 value takes at most one rounding per operation: of the scaled logit, of frequency x count, and of each
difference and sum, every one at most 2^-24 of the magnitudes that went in; 8 x 2^-24 of their sum covers them.  The
result is rounded once more, to its type."""
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


@pytest.fixture(scope="module", autouse=True)
def built():
    k3._build.build()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def pack(bits):
    """Rows of truth values as int32 words."""
    n, V = bits.shape
    words = (V + 31) // 32
    b = np.zeros((n, words * 32), dtype=np.uint8)
    b[:, :V] = bits
    return torch.from_numpy(np.packbits(b, axis=1, bitorder="little").view(np.int32).copy()).cuda()


def case(n, V, seed, x_type=F32, history=40, bias=5, allowed=None, ids=torch.int64, pad=0):
    """Inputs as the call takes them, with the truth values of the mask."""
    r = np.random.default_rng(seed)
    x = torch.from_numpy(r.normal(size=(n, V + pad)).astype(np.float32) * 3).cuda().to(x_type)[:, :V]
    c = {}
    if history is not None:
        length = r.integers(0, history + 1, n)
        length[0] = history
        ends = np.cumsum(length)
        tokens = np.minimum(np.exp(r.uniform(0, np.log(V + 1), ends[-1])).astype(np.int64) - 1, V - 1)
        tokens[r.random(len(tokens)) < 0.05] = -1                       # padding
        split = ends - length + (length * r.random(n)).astype(np.int64)
        c["history"] = torch.from_numpy(tokens).cuda().to(ids)
        c["spans"] = torch.from_numpy(np.stack([ends - length, split, ends], 1)).cuda()
        for k, lo, hi in (("repetition", 0.8, 1.5), ("frequency", -0.2, 0.6), ("presence", -0.5, 0.9)):
            c[k] = torch.from_numpy(r.uniform(lo, hi, n).astype(np.float32)).cuda()
    if bias:
        count = r.integers(0, bias + 1, n)
        count[-1] = bias
        ends = np.cumsum(count)
        b = np.concatenate([r.choice(V, k, replace=False) for k in np.minimum(count, V)])
        ends = np.cumsum(np.minimum(count, V))
        c["bias_ids"] = torch.from_numpy(b).cuda().to(ids)
        c["bias_values"] = torch.from_numpy(r.normal(size=len(b)).astype(np.float32) * 4).cuda()
        c["bias_spans"] = torch.from_numpy(np.stack([ends - np.minimum(count, V), ends], 1)).cuda()
    bits = None
    if allowed is not None:
        states = max(1, n // 2)
        bits = r.random((states, V)) < allowed
        c["mask"] = pack(bits)
        rows = r.integers(-1, states, n).astype(np.int32)
        c["mask_rows"] = torch.from_numpy(rows).cuda()
    return x, c, bits


def reference(x, c, bits):
    n, V = x.shape
    v = x.double().cpu().numpy().copy()
    room = np.abs(np.where(np.isfinite(v), v, 0))
    get = {k: t.cpu().numpy() for k, t in c.items()}
    for t in range(n):
        if "history" in get:
            a, s, e = get["spans"][t]
            h = get["history"]
            prompt, output = h[a:s], h[s:e]
            prompt, output = prompt[(prompt >= 0) & (prompt < V)], output[(output >= 0) & (output < V)]
            seen = np.unique(np.concatenate([prompt, output])).astype(np.int64)
            if "repetition" in get:
                rep = np.float64(get["repetition"][t])
                v[t, seen] = np.where(v[t, seen] > 0, v[t, seen] / rep, v[t, seen] * rep)
            room[t, seen] += np.abs(np.where(np.isfinite(v[t, seen]), v[t, seen], 0))
            kinds, times = np.unique(output, return_counts=True)
            kinds = kinds.astype(np.int64)
            f = np.float64(get["frequency"][t]) if "frequency" in get else 0.0
            p = np.float64(get["presence"][t]) if "presence" in get else 0.0
            v[t, kinds] -= f * times + p
            room[t, kinds] += 2 * np.abs(f * times) + abs(p)
        if "bias_ids" in get:
            a, e = get["bias_spans"][t]
            last = {}
            for i in range(a, e):
                if 0 <= get["bias_ids"][i] < V:
                    last[int(get["bias_ids"][i])] = float(get["bias_values"][i])
            for j, b in last.items():
                v[t, j] += b
                room[t, j] += abs(b) if np.isfinite(b) else 0
        if bits is not None:
            state = get["mask_rows"][t] if "mask_rows" in get else t
            if state >= 0:
                v[t, ~bits[state]] = -INF
    return v, room


def check(x, c, bits, out_type=F32, in_place=False, pad=0, stream=None):
    n, V = x.shape
    want, room = reference(x, c, bits)
    if in_place:
        whole = torch.full((n, V + pad), 7.0, dtype=x.dtype, device="cuda")
        whole[:, :V] = x
        out, src = whole[:, :V], whole[:, :V]
    else:
        whole = torch.full((n, V + pad), 7.0, dtype=out_type, device="cuda")
        out, src = whole[:, :V], x
    st = status()
    k3.logits_control(src, out, st, **c)
    torch.cuda.synchronize()
    assert bool((whole[:, V:] == 7.0).all())
    got = out.double().cpu().numpy()
    assert np.array_equal(np.isnan(want), np.isnan(got))
    same = np.isinf(want) | np.isnan(want)
    assert np.array_equal(want[np.isinf(want)], got[np.isinf(want)])
    off = np.abs(np.where(same, 0, got) - np.where(same, 0, want))
    assert (off <= 8 * E * room + HALF[out.dtype] * (np.abs(np.where(same, 0, want)) + 8 * E * room)).all(), off.max()
    return int(st)


SIZES = [(1, 1), (3, 2), (2, 7), (4, 8), (3, 31), (2, 33), (5, 1000), (7, 8191), (3, 8192), (4, 8193), (2, 16389), (3, 50021), (2, 131072), (1, 150001), (300, 517)]


@pytest.mark.parametrize("x_type", [BF, F32])
@pytest.mark.parametrize("n,V", SIZES)
def test_matches_the_formula(n, V, x_type):
    for k, (out_type, in_place, allowed, pad) in enumerate([(F32, False, None, 0), (BF, False, 0.5, 0), (x_type, True, None, 0), (x_type, True, 0.9, 3), (F32, False, 0.02, 5),
                                                            (BF, False, 0.97, 8)]):
        x, c, bits = case(n, V, seed=n + V + k, x_type=x_type, allowed=allowed, ids=(torch.int32, torch.int64)[k % 2], pad=(0, 8, 1)[k % 3])
        assert check(x, c, bits, out_type=out_type, in_place=in_place, pad=pad) == 0


@pytest.mark.parametrize("history", [0, 1, 3, 257, 5000, 70000])
def test_histories_of_every_length(history):
    for n, V, in_place in ((1, 32003, False), (4, 32003, True), (40, 1000, False)):
        if history * n > 300000:
            continue
        x, c, bits = case(n, V, seed=history + n, history=history)
        assert check(x, c, bits, in_place=in_place) == 0


def test_every_token_touched():
    """More touched tokens than are looked after at once, and more than 2^16 of a part."""
    r = np.random.default_rng(3)
    for V in (131072, 150001):
        x, c, _ = case(2, V, seed=11, history=10, bias=4)
        all_of_them = np.concatenate([r.permutation(V), r.integers(0, V, 5000)])
        c["history"] = torch.from_numpy(all_of_them.astype(np.int32)).cuda()
        c["spans"] = torch.tensor([[0, 60000, len(all_of_them)], [V // 3, V // 2, V]], device="cuda")
        for in_place in (False, True):
            assert check(x, c, None, in_place=in_place) == 0


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("n", [3, 200, 400])
def test_long_rows_of_different_tokens(n, ids):
    """Rows that differ in how many tokens they touch, fewer and more than are looked after at once; ids that are none, within."""
    V, r = 40011, np.random.default_rng(n)
    x, c, bits = case(n, V, seed=n, x_type=BF, history=5, bias=40, allowed=0.6, ids=ids)
    length = r.integers(0, 7001, n)
    length[:3] = 30011, 0, 8192
    ends = np.cumsum(length)
    tokens = r.integers(0, V, ends[-1])
    c["history"] = torch.from_numpy(tokens).cuda().to(ids)
    c["spans"] = torch.from_numpy(np.stack([ends - length, ends - length // 2, ends], 1)).cuda()
    assert check(x, c, bits) == 0
    # (an id past the vocabulary is no token, and -1 none either)
    at = torch.from_numpy(r.choice(20000, 50, replace=False)).cuda()
    c["history"][at] = -1
    assert check(x, c, bits) == 0
    want, got, st = torch.empty_like(x), torch.empty_like(x), status()
    k3.logits_control(x, want, st, **c)
    assert int(st) == 0
    c["history"][at[0]] = V if ids == torch.int32 else 1 << 33
    k3.logits_control(x, got, st, **c)
    assert torch.equal(got, want) and int(st) == k3.ST_TOKEN


def test_each_part_alone():
    for drop in (("repetition",), ("frequency",), ("presence",), ("repetition", "frequency", "presence"), ("bias_ids", "bias_values", "bias_spans"),
                 ("history", "spans", "repetition", "frequency", "presence"), ("mask", "mask_rows")):
        for in_place in (False, True):
            x, c, bits = case(5, 9001, seed=3, allowed=0.6)
            for k in drop:
                c.pop(k)
            if "mask" in drop:
                bits = None
            assert check(x, c, bits, in_place=in_place) == 0
    x, _, _ = case(5, 9001, seed=3)
    assert check(x, {}, None) == 0 and check(x, {}, None, in_place=True) == 0          # nothing to do
    x, c, bits = case(6, 9001, seed=4, allowed=0.6)
    r = np.random.default_rng(1)
    bits = r.random((6, 9001)) < 0.5
    c["mask"] = pack(bits)
    c.pop("mask_rows")                                                                 # row t's own mask
    assert check(x, c, bits) == 0


def test_untouched_logits_keep_their_value():
    x, c, _ = case(4, 20011, seed=5, x_type=BF, history=10, bias=2)
    x[0, 5], x[1, 19999], x[2, 300] = INF, -INF, -0.0
    out, st = torch.empty_like(x), status()
    k3.logits_control(x, out, st, **c)
    touched = torch.zeros_like(x, dtype=torch.bool)
    for t in range(4):
        a, _, e = c["spans"][t].tolist()
        h = c["history"][a:e]
        touched[t, h[h >= 0].long()] = True
        a, e = c["bias_spans"][t].tolist()
        touched[t, c["bias_ids"][a:e].long()] = True
    assert torch.equal(out.view(torch.int16)[~touched], x.view(torch.int16)[~touched])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,V", [(3, 20011), (40, 1000), (700, 3001)])
def test_untouched_nan_keep_their_bits(n, V, dtype):
    """NaN of either sign and any payload: copied, copied to rows that sit otherwise, in place beside banned tokens."""
    bits = (torch.int16, (0x7FC0, -0x40, 0x7F81, -1, 0x7FFF, -0x7F)) if dtype == BF else (torch.int32, (0x7FC00000, -0x400000, 0x7F800001, -1, 0x7FABCDEF, -0x7FFFFF))
    for k, (allowed, in_place, pad) in enumerate([(None, False, 0), (0.6, False, 0), (0.6, False, 3), (None, False, 1), (0.9, True, 0), (0.5, True, 5)]):
        x, c, allow = case(n, V, seed=n + k, x_type=dtype, history=20, bias=3, allowed=allowed, pad=pad if in_place else 0)
        r = np.random.default_rng(k)
        where = torch.from_numpy(r.random((n, V)) < 0.2).cuda()
        some = torch.tensor(bits[1], dtype=bits[0], device="cuda")[torch.from_numpy(r.integers(0, 6, (n, V))).cuda()]
        x = x.contiguous()
        x.view(bits[0])[where] = some[where]
        keep = torch.ones(n, V, dtype=torch.bool, device="cuda")
        for t in range(n):
            a, _, e = c["spans"][t].tolist()
            h = c["history"][a:e].long()
            keep[t, h[h >= 0]] = False
            a, e = c["bias_spans"][t].tolist()
            keep[t, c["bias_ids"][a:e].long()] = False
        banned = torch.zeros_like(keep)
        if allow is not None:
            state = c["mask_rows"].long()
            banned = ~torch.from_numpy(allow).cuda()[state.clamp(min=0)] & (state >= 0)[:, None]
        whole = torch.zeros(n, V + pad, dtype=dtype, device="cuda")
        out, st = whole[:, :V], status()
        if in_place:
            out.copy_(x)
        assert not in_place or torch.equal(out.contiguous().view(bits[0]), x.view(bits[0]))
        k3.logits_control(out if in_place else x, out, st, **c)
        got = out.contiguous()
        assert torch.equal(got.view(bits[0])[keep & ~banned], x.view(bits[0])[keep & ~banned]) and bool((got[banned] == -INF).all()) and int(st) == 0


def test_infinities_nan_and_masks_of_nothing():
    x, c, bits = case(6, 700, seed=6, allowed=0.5)
    x[0, :50] = -INF
    x[1, :50] = INF
    x[2, :50] = float("nan")
    x[3] = torch.finfo(F32).min
    bits[:] = False                                                                    # every state bans everything
    c["mask"] = pack(bits)
    assert check(x, c, bits) == 0
    assert check(x, c, bits, in_place=True) == 0
    bits[:] = True
    c["mask"] = pack(bits)
    c["bias_values"][:3] = -INF
    for in_place in (False, True):
        assert check(x, c, bits, in_place=in_place) == 0
    # the words' bits past the vocabulary mean nothing
    c["mask"][:, -1] |= -1 << (700 % 32)
    assert check(x, c, bits) == 0


def test_a_token_listed_twice_takes_its_last_bias():
    x = torch.zeros(2, 5000, device="cuda")
    ids = torch.tensor([7, 4999, 7, 7, 0, 4999], device="cuda")
    values = torch.tensor([1.0, 2.0, 3.0, 4.0, 5.0, 6.0], device="cuda")
    c = {"bias_ids": ids, "bias_values": values, "bias_spans": torch.tensor([[0, 6], [0, 3]], device="cuda")}
    out, st = torch.empty_like(x), status()
    k3.logits_control(x, out, st, **c)
    assert out[0, [0, 7, 4999]].tolist() == [5.0, 4.0, 6.0] and out[1, [0, 7, 4999]].tolist() == [0.0, 3.0, 2.0]
    # many entries of one token, over several threads
    many = torch.full((3000,), 11, dtype=torch.int32, device="cuda")
    k3.logits_control(x, out, st, bias_ids=many, bias_values=torch.arange(3000, device="cuda").float(), bias_spans=torch.tensor([[0, 3000], [5, 100]], device="cuda"))
    assert out[:, 11].tolist() == [2999.0, 99.0] and int((out != 0).sum()) == 2


def test_rows_share_lists():
    """Drafted tokens: rows of one request see more and more of the same history."""
    r = np.random.default_rng(0)
    V = 3000
    x, _, _ = case(5, V, seed=1)
    c = {"history": torch.from_numpy(r.integers(0, V, 400).astype(np.int32)).cuda(),
         "spans": torch.tensor([[0, 300, 395 + k] for k in range(5)], device="cuda"),
         "repetition": torch.full((5,), 1.2, device="cuda"), "frequency": torch.full((5,), 0.3, device="cuda"),
         "bias_ids": torch.tensor([1, 2, 3], device="cuda"), "bias_values": torch.tensor([1.0, -1.0, 2.0], device="cuda"),
         "bias_spans": torch.tensor([[0, 3]] * 5, device="cuda")}
    assert check(x, c, None) == 0


def test_status_of_bad_ids_spans_and_masks():
    x, c, bits = case(4, 900, seed=8, allowed=0.5)
    good = {k: v.clone() for k, v in c.items()}
    c["history"][3] = 900
    c["bias_ids"][0] = 1 << 40
    want = status()
    out = torch.empty_like(x)
    k3.logits_control(x, out, want, **c)
    assert int(want) == k3.ST_TOKEN
    for key, value in (("spans", torch.tensor([-1, 0, 2], device="cuda")), ("spans", torch.tensor([0, 1 << 40, 1 << 41], device="cuda")),
                       ("spans", torch.tensor([5, 3, 10], device="cuda")), ("spans", torch.tensor([5, 12, 10], device="cuda"))):
        c = {k: v.clone() for k, v in good.items()}
        c[key][1] = value
        assert check_bad(x, c, bits, 1, "spans", [0, 0, 0]) == k3.ST_INDEX
    c = {k: v.clone() for k, v in good.items()}
    c["bias_spans"][2] = torch.tensor([0, 1 << 30], device="cuda")
    assert check_bad(x, c, bits, 2, "bias_spans", [0, 0]) == k3.ST_INDEX
    c = {k: v.clone() for k, v in good.items()}
    c["mask_rows"][3] = len(bits)
    assert check_bad(x, c, bits, 3, "mask_rows", -1) == k3.ST_INDEX


def check_bad(x, c, bits, row, key, as_if):
    """The call's status; its result must be that of the row's part left out."""
    out, st = torch.empty_like(x), status()
    k3.logits_control(x, out, st, **c)
    fixed = {k: v.clone() for k, v in c.items()}
    fixed[key][row] = torch.tensor(as_if, device="cuda").to(fixed[key].dtype)
    want, none = torch.empty_like(x), status()
    k3.logits_control(x, want, none, **fixed)
    assert torch.equal(out, want) and int(none) == 0
    return int(st)


def test_graph_streams_and_no_rows():
    x, c, bits = case(6, 40000, seed=9, allowed=0.7, history=500)
    out, st = torch.empty_like(x), status()
    k3.logits_control(x, out, st, **c)
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k3.logits_control(x, out, st, **c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.zero_()
        graph.replay()
    side.synchronize()
    assert torch.equal(out, first) and int(st) == 0
    none = torch.empty(0, 40000, device="cuda")
    k3.logits_control(none, none, st)


def two_launches():
    return 2 * torch.cuda.get_device_properties(0).multi_processor_count + 9


@pytest.mark.parametrize("x_type,out_type,in_place,history,bias,allowed", [
    (BF, BF, True, 60, 5, 0.7), (F32, F32, True, 60, 5, 0.03), (F32, BF, False, 60, 5, 0.9), (BF, F32, False, 60, 5, None), (BF, BF, False, None, 0, 0.5),
    (F32, F32, True, None, 0, 0.5), (F32, F32, True, 200, 8, None), (BF, BF, False, None, 6, 0.5), (F32, F32, False, None, 0, None)])
@pytest.mark.parametrize("V", [517, 9001, 40016])
def test_many_rows_in_two_launches(V, x_type, out_type, in_place, history, bias, allowed):
    """More rows than the GPU holds at once: the stream and the lists are launches of their own, the second beginning while
    the first one ends.  With and without either, in place and not, of either type."""
    n = two_launches() if V > 9001 else 700
    x, c, bits = case(n, V, seed=V + n, x_type=x_type, history=history, bias=bias, allowed=allowed, pad=V % 3)
    assert check(x, c, bits, out_type=out_type, in_place=in_place, pad=V % 2) == 0


def test_many_rows_of_long_lists():
    """... whose rows touch more tokens than the lists' launch looks after at once, beside rows that touch none."""
    n, V, r = two_launches(), 30011, np.random.default_rng(3)
    x, c, bits = case(n, V, seed=5, x_type=BF, history=3, bias=3, allowed=0.8)
    length = r.integers(0, 200, n)
    length[[0, 7, n - 1]] = 20000, 9000, 15000
    ends = np.cumsum(length)
    c["history"] = torch.from_numpy(r.integers(0, V, ends[-1])).cuda()
    c["spans"] = torch.from_numpy(np.stack([ends - length, ends - length // 3, ends], 1)).cuda()
    for in_place in (False, True):
        assert check(x, c, bits, out_type=BF, in_place=in_place) == 0


@pytest.mark.parametrize("in_place", [False, True])
def test_two_launches_in_a_graph(in_place):
    """Captured, replayed one after the other over other logits: each replay gives what the call gives."""
    n, V = two_launches(), 9001
    x, c, _ = case(n, V, seed=9, x_type=BF, history=300, allowed=0.7)
    held, out, st = x.clone(), torch.empty_like(x), status()
    if in_place:
        out = held
    graph = torch.cuda.CUDAGraph()
    k3.logits_control(x.clone(), torch.empty_like(x), st, **c)
    with torch.cuda.graph(graph):
        k3.logits_control(held, out, st, **c)
    for k in range(5):
        now = x.roll(k, 1) * (1 + k)
        held.copy_(now)
        want = torch.empty_like(x)
        k3.logits_control(now, want, st, **c)
        graph.replay()
        assert torch.equal(out, want), k
    assert int(st) == 0


def test_refusals_of_the_binding():
    x, c, _ = case(3, 100, seed=1, allowed=0.5)
    out, st = torch.empty_like(x), status()
    for bad in ({"history": c["history"]}, {"repetition": c["repetition"]}, {"bias_ids": c["bias_ids"]}, {"mask_rows": c["mask_rows"]}, {**c, "spans": c["spans"][:2]},
                {**c, "mask": c["mask"][:, :-1].contiguous()}, {**c, "bias_values": c["bias_values"][:-1]}):
        with pytest.raises((ValueError, k3.K3HufError)):
            k3.logits_control(x, out, st, **bad)
    with pytest.raises(TypeError):
        k3.logits_control(x, out, st, **{**c, "spans": c["spans"].int()})
    with pytest.raises(TypeError):
        k3.logits_control(x.half(), out, st)
    with pytest.raises(ValueError):
        k3.logits_control(x, out[:2], st)
