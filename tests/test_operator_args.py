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
