"""Refusals of the operators next to the coded weights, on CPU: every call below returns before it touches a device, so
the device addresses are placeholders."""
import ctypes

import numpy as np
import pytest

import oracle
import workloads

k3 = pytest.importorskip("lossless_bf16_weight_k3huf_gb300")
P = 1 << 20                                             # a placeholder address, aligned to everything


@pytest.fixture(scope="module")
def lib():
    k3._build.build()
    return k3._lib()


def test_embed_layer(lib):
    blob = oracle.encode_layer([workloads.normal_tensor((10, 64), 0.02, 3)])

    def call(blob=blob, hdr=None, layer=P, size=None, tensor=0, cols=64, ids=P, ib=8, n=4, out=P, ot=0, stride=64, st=P):
        h = np.ascontiguousarray(blob if hdr is None else hdr)
        return lib.k3huf_embed_layer(h.ctypes.data, h.size, layer, blob.size if size is None else size, tensor, cols, ids, ib, n, 1.0, out, ot,
                                     stride, st, None)

    assert call(n=0) == k3.OK
    bad = blob.copy()
    bad[0] ^= 1
    assert call(hdr=bad) == k3.E_FORMAT and call(hdr=blob[:100]) == k3.E_FORMAT
    for kw in (dict(layer=None), dict(layer=P + 8), dict(size=blob.size - 1), dict(tensor=1), dict(cols=0), dict(cols=63), dict(ids=None),
               dict(ids=P + 4), dict(ib=2), dict(out=None), dict(out=P + 1), dict(ot=2), dict(stride=63), dict(st=None), dict(st=P + 2)):
        assert call(**kw) == k3.E_ARG, kw


def test_embed_grad(lib):
    need = k3.embed_grad_scratch_bytes(4, 10, 64)

    def call(ids=P, ib=8, n=4, dy=P, dt=0, stride=64, rows=10, cols=64, grad=P, scratch=P, size=need, st=P, flags=0):
        return lib.k3huf_embed_grad(ids, ib, n, dy, dt, stride, rows, cols, 1.0, grad, scratch, size, st, flags, None)

    for kw in (dict(ids=None), dict(ids=P + 4), dict(ib=3), dict(dy=None), dict(dy=P + 1), dict(dt=7), dict(stride=63), dict(rows=0), dict(cols=0),
               dict(grad=None), dict(grad=P + 2), dict(scratch=None), dict(scratch=P + 16), dict(size=need - 1), dict(st=None), dict(flags=1),
               dict(n=1 << 40)):
        assert call(**kw) == k3.E_ARG, kw
    assert call(n=0, ids=None, dy=None, flags=k3.ACCUMULATE) == k3.OK


def adapters(**kw):
    v = dict(a=P, b=P, scales=P, n_adapters=2, rank=8, cols=64, rows=32)
    v.update(kw)
    return k3.Adapters(*(v[f] for f, _ in k3.Adapters._fields_))


BAD_ADAPTERS = (dict(a=None), dict(b=None), dict(scales=None), dict(n_adapters=0), dict(rank=0), dict(rank=129), dict(cols=0), dict(rows=0),
                dict(a=P + 1), dict(scales=P + 2))


def test_adapter_apply(lib):
    need = k3.adapter_scratch_bytes(4, 2, 8, 64, 32)

    def call(ad=None, x=P, xs=64, ids=P, n=4, base=P, bs=32, y=P, ys=32, yt=1, scratch=P, size=need, st=P):
        ad = adapters() if ad is None else ad
        return lib.k3huf_adapter_apply(ctypes.addressof(ad), x, xs, ids, n, base, bs, y, ys, yt, scratch, size, st, None)

    assert call(n=0) == k3.OK
    for kw in BAD_ADAPTERS:
        assert call(ad=adapters(**kw)) == k3.E_ARG, kw
    for kw in (dict(x=None), dict(x=P + 1), dict(xs=63), dict(ids=None), dict(ids=P + 2), dict(base=P + 2), dict(bs=31), dict(y=None), dict(y=P + 2),
               dict(ys=31), dict(yt=2), dict(scratch=None), dict(scratch=P + 16), dict(size=need - 1), dict(st=None), dict(bs=40)):
        assert call(**kw) == k3.E_ARG, kw
    assert lib.k3huf_adapter_apply(None, P, 64, P, 4, None, 0, P, 32, 1, P, need, P, None) == k3.E_ARG


def test_adapter_grad(lib):
    need = k3.adapter_scratch_bytes(4, 2, 8, 64, 32, grad=True)

    def call(ad=None, x=P, xs=64, ids=P, n=4, dy=P, ys=32, base=None, bs=0, dx=P, ds=64, dt=1, da=P, db=P, scratch=P, size=need, st=P, flags=0):
        ad = adapters() if ad is None else ad
        return lib.k3huf_adapter_grad(ctypes.addressof(ad), x, xs, ids, n, dy, ys, base, bs, dx, ds, dt, da, db, scratch, size, st, flags, None)

    for kw in BAD_ADAPTERS:
        assert call(ad=adapters(**kw)) == k3.E_ARG, kw
    for kw in (dict(x=None), dict(xs=63), dict(ids=None), dict(dy=None), dict(dy=P + 1), dict(ys=31), dict(base=P, bs=63), dict(base=P + 2, bs=64),
               dict(base=P, bs=64, dx=None), dict(base=P, bs=72), dict(dx=P + 2), dict(ds=63), dict(dt=9), dict(da=None), dict(db=None), dict(da=P + 2),
               dict(scratch=None), dict(size=need - 1), dict(st=None), dict(flags=8)):
        assert call(**kw) == k3.E_ARG, kw


def test_token_logprobs(lib):
    def call(x=P, t=1, stride=50, n=3, vocab=50, scale=1.0, tok=P, ib=8, lp=P, ent=P, lse=P, top=2, ti=P, tl=P, st=P):
        return lib.k3huf_token_logprobs(x, t, stride, n, vocab, scale, tok, ib, lp, ent, lse, top, ti, tl, st, None)

    assert call(n=0) == k3.OK
    for kw in (dict(x=None), dict(x=P + 2), dict(t=2), dict(stride=49), dict(vocab=0), dict(vocab=1 << 31, stride=1 << 31), dict(scale=0.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-1.0), dict(tok=None), dict(tok=P + 4), dict(ib=1), dict(lp=None), dict(lp=P + 2),
               dict(ent=P + 2), dict(lse=P + 2), dict(top=51), dict(top=65, vocab=100, stride=100), dict(ti=None), dict(tl=None), dict(st=None)):
        assert call(**kw) == k3.E_ARG, kw


def test_token_logprobs_grad(lib):
    def call(x=P, t=1, stride=50, n=3, vocab=50, scale=1.0, tok=P, ib=8, lse=P, ent=P, g=P, h=P, d=P, ds=50, st=P):
        return lib.k3huf_token_logprobs_grad(x, t, stride, n, vocab, scale, tok, ib, lse, ent, g, h, d, ds, st, None)

    assert call(n=0) == k3.OK
    for kw in (dict(x=None), dict(x=P + 2), dict(t=2), dict(stride=49), dict(vocab=0), dict(scale=0.0), dict(tok=None), dict(ib=1), dict(lse=None),
               dict(ent=None), dict(g=None), dict(d=None), dict(d=P + 2), dict(ds=49), dict(ds=60), dict(st=None), dict(h=P + 2)):
        assert call(**kw) == k3.E_ARG, kw


def test_scratch_sizes_grow_with_the_tokens():
    assert k3.embed_grad_scratch_bytes(0, 1, 1) <= k3.embed_grad_scratch_bytes(1 << 16, 1 << 18, 8192)
    assert k3.adapter_scratch_bytes(1, 1, 1, 1, 1) <= k3.adapter_scratch_bytes(1 << 16, 64, 128, 8192, 8192, grad=True)
    for args in ((4, 0, 64), (4, 10, 0)):
        with pytest.raises(k3.K3HufError):
            k3.embed_grad_scratch_bytes(*args)


def test_linear(lib):
    def call(x=P, xs=64, n=4, w=P, ws=64, rows=32, cols=64, bias=P, bt=0, act=1, res=P, rs=32, y=P, ys=32, yt=1, z=P + 64, zs=32, zt=0, scratch=None, size=0, st=P):
        return lib.k3huf_linear(x, xs, n, w, ws, rows, cols, bias, bt, act, res, rs, y, ys, yt, z, zs, zt, scratch, size, st, None)

    assert call(n=0) == k3.OK and call(n=0, x=None, w=None, y=None, z=None, res=None, bias=None) == k3.OK
    for kw in (dict(x=None), dict(x=P + 1), dict(xs=63), dict(n=1 << 31), dict(w=None), dict(w=P + 1), dict(ws=63), dict(rows=0), dict(rows=1 << 31),
               dict(cols=0), dict(cols=1 << 31, xs=1 << 31, ws=1 << 31), dict(bias=P + 1), dict(bt=1, bias=P + 2), dict(bt=2), dict(act=4), dict(res=P + 2),
               dict(rs=31), dict(rs=40), dict(y=None), dict(y=P + 2), dict(ys=31), dict(yt=2), dict(z=P + 1), dict(zs=31), dict(zt=2), dict(zt=1, z=P + 2),
               dict(st=None), dict(st=P + 2), dict(scratch=P + 16, size=1 << 20), dict(z=P, y=P, zt=1)):
        assert call(**kw) == k3.E_ARG, kw
    # rows that do not start on 16 bytes need their copies' room
    need = k3.linear_scratch_bytes(4, 32, 64, any=True)
    assert k3.linear_scratch_bytes(4, 32, 64) == 0 and k3.linear_scratch_bytes(4, 32, 63) == need
    for kw in (dict(xs=65, ws=65), dict(xs=65, ws=65, scratch=P, size=need - 1), dict(xs=65), dict(ws=65), dict(x=P + 2), dict(w=P + 8)):
        assert call(**kw) == k3.E_ARG, kw


def test_linear_dz(lib):
    def call(z=P, zt=0, zs=32, dy=P + 64, dyt=0, dys=32, n=4, rows=32, act=2, dz=P + 128, dzs=32, db=P, flags=0):
        return lib.k3huf_linear_dz(z, zt, zs, dy, dyt, dys, n, rows, act, dz, dzs, db, flags, None)

    assert call(n=0, db=None) == k3.OK and call(n=0, flags=k3.ACCUMULATE) == k3.OK
    for kw in (dict(z=None), dict(z=P + 1), dict(zt=1, z=P + 2), dict(zt=2), dict(zs=31), dict(dy=None), dict(dy=P + 1), dict(dyt=3), dict(dys=31),
               dict(n=1 << 31), dict(rows=0), dict(act=4), dict(dz=None), dict(dz=P + 1), dict(dzs=31), dict(db=P + 2), dict(flags=1), dict(dz=P, zs=40),
               dict(dz=P, zt=1), dict(dz=P + 64, dys=40), dict(dz=P + 64, dyt=1)):
        assert call(**kw) == k3.E_ARG, kw


def test_linear_grad(lib):
    def call(x=P, xs=64, n=4, w=P, ws=64, rows=32, cols=64, dz=P, dzs=32, dx=P, dxs=64, dxt=0, dw=P, scratch=None, size=0, st=P, flags=0):
        return lib.k3huf_linear_grad(x, xs, n, w, ws, rows, cols, dz, dzs, dx, dxs, dxt, dw, scratch, size, st, flags, None)

    assert call(n=0, dw=None) == k3.OK and call(n=0, flags=k3.ACCUMULATE) == k3.OK
    for kw in (dict(x=None), dict(x=P + 1), dict(xs=63), dict(n=1 << 31), dict(w=None), dict(w=P + 1), dict(ws=63), dict(rows=0), dict(cols=0), dict(dz=None),
               dict(dz=P + 1), dict(dzs=31), dict(dx=P + 1), dict(dxt=1, dx=P + 2), dict(dxt=2), dict(dxs=63), dict(dw=P + 2), dict(dx=None, dw=None), dict(st=None),
               dict(flags=8), dict(scratch=P + 16, size=1 << 20), dict(xs=65), dict(ws=65), dict(dzs=33)):
        assert call(**kw) == k3.E_ARG, kw
    need = k3.linear_scratch_bytes(4, 32, 64, grad=True, any=True)
    assert call(xs=65, ws=65, dzs=33, scratch=P, size=need - 1) == k3.E_ARG


def test_logits_control(lib):
    full = dict(history=P, spans=P, n_history=100, history_id_bytes=8, bias_id_bytes=4, repetition=P, frequency=P, presence=P, bias_ids=P, bias_values=P,
                bias_spans=P, n_bias=9, mask=P, mask_rows=P, n_masks=2, mask_stride=2)

    def call(x=P, t=1, stride=50, n=3, vocab=50, out=P + 4096, ot=0, os=50, st=P, control=True, **kw):
        c = k3.Control(**{**full, **kw})
        return lib.k3huf_logits_control(ctypes.addressof(c) if control else None, x, t, stride, n, vocab, out, ot, os, st, None)

    assert call(n=0) == k3.OK and call(n=0, x=None, out=None) == k3.OK
    for kw in (dict(control=False), dict(x=None), dict(x=P + 2), dict(t=2), dict(stride=49), dict(vocab=0), dict(vocab=1 << 31, stride=1 << 31, os=1 << 31),
               dict(n=1 << 31), dict(out=None), dict(out=P + 1), dict(ot=2), dict(os=49), dict(out=P), dict(out=P, ot=1, os=60), dict(st=None), dict(st=P + 2),
               dict(spans=None), dict(spans=P + 4), dict(n_history=(1 << 30) + 1), dict(history_id_bytes=2), dict(history=P + 4), dict(repetition=P + 2),
               dict(frequency=P + 1), dict(presence=P + 2), dict(bias_ids=P + 2), dict(bias_id_bytes=3), dict(bias_values=None), dict(bias_values=P + 2),
               dict(bias_spans=None), dict(bias_spans=P + 4), dict(n_bias=(1 << 30) + 1), dict(mask=P + 2), dict(mask_rows=P + 2), dict(mask_stride=1), dict(mask_rows=None)):
        assert call(**kw) == k3.E_ARG, kw


def test_distill(lib):
    def call(x=P, t=1, stride=50, n=3, vocab=50, scale=1.0, ids=P, lp=P, top=5, mode=2, loss=P, lse=P, rest=P, st=P):
        return lib.k3huf_distill(x, t, stride, n, vocab, scale, ids, lp, top, mode, loss, lse, rest, st, None)

    assert call(n=0) == k3.OK
    for kw in (dict(x=None), dict(x=P + 2), dict(t=2), dict(stride=49), dict(n=1 << 27), dict(vocab=0), dict(vocab=1 << 31, stride=1 << 31), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(ids=None), dict(ids=P + 2), dict(lp=None), dict(lp=P + 1), dict(top=0),
               dict(top=65), dict(mode=3), dict(mode=0), dict(mode=1), dict(loss=None), dict(loss=P + 2), dict(lse=P + 2), dict(rest=P + 2), dict(st=None)):
        assert call(**kw) == k3.E_ARG, kw


def test_distill_grad(lib):
    def call(x=P, t=1, stride=50, n=3, vocab=50, scale=1.0, ids=P, lp=P, top=5, mode=2, lse=P, rest=P, g=P, d=P, ds=50, st=P):
        return lib.k3huf_distill_grad(x, t, stride, n, vocab, scale, ids, lp, top, mode, lse, rest, g, d, ds, st, None)

    assert call(n=0) == k3.OK
    for kw in (dict(x=None), dict(x=P + 2), dict(t=2), dict(stride=49), dict(n=1 << 27), dict(vocab=0), dict(scale=0.0), dict(ids=None), dict(lp=None), dict(top=0),
               dict(top=65), dict(mode=3), dict(mode=0), dict(rest=None), dict(rest=P + 2), dict(lse=None), dict(lse=P + 1), dict(g=None), dict(g=P + 2),
               dict(d=None), dict(d=P + 2), dict(ds=49), dict(ds=60), dict(st=None)):
        assert call(**kw) == k3.E_ARG, kw


def test_products_refuse_outputs_over_their_inputs(lib):
    """Every argument at an address of its own, but for the one pair that is named."""
    x, w, bias, res, y, z, dz, dx, dw, dy, db = (P + (k << 16) for k in range(11))

    def linear(x=x, w=w, bias=bias, res=res, y=y, z=z, zs=32, zt=0):
        return lib.k3huf_linear(x, 32, 4, w, 32, 32, 32, bias, 0, 1, res, 32, y, 32, 0, z, zs, zt, None, 0, P, None)

    for kw in (dict(y=x), dict(y=w), dict(y=bias), dict(y=z), dict(z=x), dict(z=w), dict(z=bias), dict(z=res, zt=1), dict(z=res, zs=40)):
        assert linear(**kw) == k3.E_ARG, kw

    def grad(x=x, w=w, dz=dz, dx=dx, dw=dw):
        return lib.k3huf_linear_grad(x, 32, 4, w, 32, 32, 32, dz, 32, dx, 32, 0, dw, None, 0, P, 0, None)

    for kw in (dict(dx=x), dict(dx=dz), dict(dx=dz, dw=None), dict(dx=w), dict(dx=w, dw=None), dict(dx=dw), dict(dw=x), dict(dw=x, dx=None), dict(dw=dz),
               dict(dw=dz, dx=None), dict(dw=w)):
        assert grad(**kw) == k3.E_ARG, kw

    def slope(db):
        return lib.k3huf_linear_dz(z, 0, 32, dy, 0, 32, 4, 32, 2, dz, 32, db, 0, None)

    for at in (z, dy, dz):
        assert slope(at) == k3.E_ARG


def test_products_refuse_one_argument_at_a_time(lib):
    """The refusals of each argument, with all others as they should be."""
    x, w, bias, res, y, z, dz, dx, dw = (P + (k << 16) for k in range(9))

    def linear(x=x, xs=64, n=4, w=w, ws=64, rows=32, cols=64, bias=bias, bt=0, act=1, res=res, rs=32, y=y, ys=32, yt=1, z=z, zs=32, zt=0, scratch=None, size=0, st=P):
        return lib.k3huf_linear(x, xs, n, w, ws, rows, cols, bias, bt, act, res, rs, y, ys, yt, z, zs, zt, scratch, size, st, None)

    need = k3.linear_scratch_bytes(4, 32, 64, any=True)
    for kw in (dict(x=None), dict(x=x + 1), dict(xs=63), dict(n=1 << 31), dict(w=None), dict(w=w + 1), dict(ws=63), dict(rows=0), dict(rows=1 << 31, ys=1 << 31, rs=1 << 31, zs=1 << 31),
               dict(cols=0), dict(cols=1 << 31, xs=1 << 31, ws=1 << 31), dict(bias=bias + 1), dict(bt=1, bias=bias + 2), dict(bt=2), dict(act=4), dict(res=res + 2),
               dict(rs=31), dict(res=y, rs=40), dict(y=None), dict(y=y + 2), dict(ys=31), dict(yt=2), dict(z=z + 1), dict(zs=31), dict(zt=2), dict(zt=1, z=z + 2),
               dict(st=None), dict(st=P + 2), dict(scratch=P + 16, size=1 << 20), dict(xs=65, ws=65), dict(xs=65, ws=65, scratch=P, size=need - 1), dict(xs=65),
               dict(ws=65), dict(x=x + 2), dict(w=w + 8)):
        assert linear(**kw) == k3.E_ARG, kw

    def grad(x=x, xs=64, n=4, w=w, ws=64, rows=32, cols=64, dz=dz, dzs=32, dx=dx, dxs=64, dxt=0, dw=dw, scratch=None, size=0, st=P, flags=0):
        return lib.k3huf_linear_grad(x, xs, n, w, ws, rows, cols, dz, dzs, dx, dxs, dxt, dw, scratch, size, st, flags, None)

    need = k3.linear_scratch_bytes(4, 32, 64, grad=True, any=True)
    for kw in (dict(x=None), dict(x=x + 1), dict(xs=63), dict(n=1 << 31), dict(w=None), dict(w=w + 1), dict(ws=63), dict(rows=0), dict(cols=0), dict(dz=None),
               dict(dz=dz + 1), dict(dzs=31), dict(dx=dx + 1), dict(dxt=1, dx=dx + 2), dict(dxt=2), dict(dxs=63), dict(dw=dw + 2), dict(dx=None, dw=None), dict(st=None),
               dict(flags=8), dict(scratch=P + 16, size=1 << 20), dict(xs=65), dict(ws=65), dict(dzs=33), dict(xs=65, ws=65, dzs=33, scratch=P, size=need - 1)):
        assert grad(**kw) == k3.E_ARG, kw
