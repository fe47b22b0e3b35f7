"""Host-side checks of the entry points around the attention (rotary
positions, norms, pool copies): bad arguments are refused before anything is
launched.  Pointers are fake addresses that are never dereferenced; a call that
passes its checks ends with LA2_ERR_CUDA here, where there is no GPU to launch
on, and is made only where that is so."""
import ctypes

import pytest
import torch

import causal_linear_attention_fwd_b200 as la2
from causal_linear_attention_fwd_b200 import _binding as B

INV, UNS, OK = B.LA2_ERR_INVALID, B.LA2_ERR_UNSUPPORTED, B.LA2_OK
MB = 1 << 20
(Q, K, V, F, POS, RQ, RK, RV, O, G, W, U, DU, DO, DG, DW, WS, H, Y, N, HN, DH, DY, PW, DPW,
 SRC, DST) = [(i + 1) * 64 * MB for i in range(27)]
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake addresses")


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return la2.library()


class Heads(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("batch", ctypes.c_int64), ("head", ctypes.c_int64),
                ("row", ctypes.c_int64)]


def heads(p, batch, head, row):
    return None if p is None else ctypes.byref(Heads(p, batch, head, row))


def rotary(lib, q=Q, k=K, v=V, f=F, pos=None, kind=0, rq=RQ, rk=RK, rv=RV, flags=0, Bn=2, Hn=4, Hk=2,
           L=10, d=64, e=128, r=32, dt=B.LA2_BF16, back=False, row=1024, head=None, batch=None):
    s = lambda p, w: heads(p, row * L if batch is None else batch, w if head is None else head, row)  # noqa: E731
    if back:
        return lib.la2_rotary_backward(rq, rk, rv, f, pos, kind, s(q, d), s(k, d), s(v, e), 1.0, flags,
                                       Bn, Hn, Hk, L, d, e, r, dt, None)
    return lib.la2_rotary(s(q, d), s(k, d), s(v, e), f, pos, kind, rq, rk, rv, 1.0, flags, Bn, Hn, Hk, L,
                          d, e, r, dt, None)


@pytest.mark.parametrize("back", [False, True])
def test_rotary_validation(lib, back):
    f = lambda **kw: rotary(lib, back=back, **kw)  # noqa: E731
    for bad in (dict(Bn=-1), dict(L=-1), dict(r=33), dict(r=0), dict(r=66), dict(flags=2), dict(kind=3),
                dict(Hk=3), dict(Hk=0), dict(q=None), dict(k=None), dict(f=None), dict(rq=None), dict(rk=None),
                dict(rv=None), dict(v=None), dict(kind=1), dict(pos=POS), dict(rq=RQ + 8), dict(f=F + 4),
                dict(pos=POS + 4, kind=2), dict(q=Q + 1), dict(row=-1), dict(head=-64), dict(rq=Q),
                dict(rk=Q + 16), dict(rv=F), dict(rk=POS, pos=POS, kind=1)):
        if back and bad in (dict(rq=RQ), ):
            continue
        if back and set(bad) == {"rk", "pos", "kind"}:
            bad = dict(k=POS, pos=POS, kind=1)     # a gradient over the positions
        if back and bad == dict(rv=F):
            bad = dict(v=F)
        assert f(**bad) == INV, bad
    for bad in (dict(d=96), dict(e=32), dict(dt=7)):
        assert f(**bad) == UNS, bad
    for empty in (dict(Bn=0), dict(L=0), dict(Hn=0, Hk=0)):
        assert f(**empty) == OK, empty
    assert f(rv=None, v=None, e=0, L=0) == OK


def test_rotary_outputs_apart(lib):
    """Results of the forward may not meet; gradients may be slices of one
    buffer side by side, but neither overlap nor fold onto themselves."""
    assert rotary(lib, rk=RQ) == INV
    assert rotary(lib, rk=RQ + 2 * 4 * 10 * 64 * 2 - 16) == INV
    f = lambda **kw: rotary(lib, back=True, **kw)  # noqa: E731
    assert f(k=Q) == INV                                 # the same place
    assert f(k=Q + 4 * 64 * 2 - 16) == INV               # k's first columns are q's last
    assert f(k=Q + 1024 * 2 - 64) == INV                 # k of a row reaches into the next row's q
    assert f(row=255) == INV                             # q's four heads of 64 fill 256
    assert f(row=128) == INV                             # rows of a tensor on one another
    assert f(head=32) == INV                             # heads on one another
    assert f(batch=1024) == INV                          # batches on one another


@no_gpu
def test_rotary_slices_of_one_buffer_pass_the_checks(lib):
    f = lambda **kw: rotary(lib, back=True, **kw)  # noqa: E731
    assert f(k=Q + 4 * 64 * 2, v=Q + 6 * 64 * 2) == B.LA2_ERR_CUDA
    # one after another in each head: [B, L, H, 3, 64]
    assert f(k=Q + 128, v=Q + 256, e=64, Hk=4, head=192, row=4 * 192) == B.LA2_ERR_CUDA
    assert f(k=Q + 112, v=Q + 256, e=64, Hk=4, head=192, row=4 * 192) == INV
    assert f(k=Q + 128, v=Q + 272, e=64, Hk=4, head=192, row=4 * 192) == INV


def gated(lib, o=O, gate=G, sb=5000, sl=500, w=W, u=U, eps=1e-6, flags=0, Bn=2, Hn=3, L=10, e=64,
          dt=B.LA2_BF16):
    return lib.la2_gated_norm(o, gate, sb, sl, w, u, eps, flags, Bn, Hn, L, e, dt, None)


def gated_back(lib, du=DU, o=O, gate=G, sb=5000, sl=500, w=W, do=DO, dg=DG, tb=1920, tl=192, dw=DW, eps=1e-6,
               flags=0, Bn=2, Hn=3, L=10, e=64, dt=B.LA2_BF16, ws=WS, wsb=MB):
    return lib.la2_gated_norm_backward(du, o, gate, sb, sl, w, do, dg, tb, tl, dw, eps, flags, Bn, Hn, L, e, dt,
                                       ws, wsb, None)


def test_gated_norm_validation(lib):
    both = (dict(Bn=-1), dict(L=-2), dict(eps=0.0), dict(eps=float("nan")), dict(flags=8), dict(flags=16),
            dict(flags=2 | 4), dict(sb=-1), dict(o=None), dict(o=O + 4), dict(gate=G + 1), dict(w=W + 4))
    for bad in both:
        assert gated(lib, **bad) == INV, bad
        assert gated_back(lib, **bad) == INV, bad
    for bad in (dict(e=32), dict(dt=5), dict(Hn=257, flags=2)):
        assert gated(lib, **bad) == UNS and gated_back(lib, **bad) == UNS, bad
    for bad in (dict(u=None), dict(u=U + 2), dict(u=O), dict(u=W), dict(u=G + 64)):
        assert gated(lib, **bad) == INV, bad
    for bad in (dict(du=None), dict(do=None), dict(dg=None), dict(gate=None), dict(do=DU), dict(do=O),
                dict(dg=G), dict(dg=DO), dict(dw=DG), dict(ws=None), dict(wsb=64), dict(ws=DU), dict(ws=WS + 8),
                dict(tl=191), dict(tb=1919), dict(tb=-1), dict(dw=DW + 4), dict(dw=W)):
        assert gated_back(lib, **bad) == INV, bad
    for empty in (dict(Bn=0), dict(L=0), dict(Hn=0)):
        assert gated(lib, **empty) == OK and gated_back(lib, dw=None, **empty) == OK


def residual(lib, h=H, hd=B.LA2_F32, y=Y, w=W, pw=None, hn=HN, n=N, eps=1e-6, flags=0, rows=10, D=64,
             dt=B.LA2_BF16):
    return lib.la2_residual_norm(h, hd, y, w, pw, hn, n, 1.0, 1.0, eps, flags, rows, D, dt, None)


def residual_back(lib, dn=DU, dhn=DG, hn=HN, hd=B.LA2_F32, y=Y, w=W, pw=PW, dh=DH, dy=DY, dw=DW, dpw=DPW,
                  eps=1e-6, flags=8, rows=10, D=64, dt=B.LA2_BF16, ws=WS, wsb=MB):
    return lib.la2_residual_norm_backward(dn, dhn, hn, hd, y, w, pw, dh, dy, dw, dpw, 1.0, 1.0, eps, flags, rows, D,
                                          dt, ws, wsb, None)


def test_residual_norm_validation(lib):
    for bad in (dict(rows=-1), dict(D=0), dict(eps=0.0), dict(flags=1), dict(flags=16)):
        assert residual(lib, **bad) == INV and residual_back(lib, **bad) == INV, bad
    for bad in (dict(D=16385), dict(dt=3), dict(hd=9), dict(hd=B.LA2_BF16, dt=B.LA2_F32)):
        assert residual(lib, **bad) == UNS and residual_back(lib, **bad) == UNS, bad
    for bad in (dict(h=None), dict(n=None), dict(hn=None), dict(y=None), dict(y=None, hn=None, flags=8),
                dict(pw=PW), dict(h=H + 8), dict(n=N + 8), dict(n=H), dict(hn=Y), dict(n=HN), dict(hn=W),
                dict(hn=H + 16), dict(n=Y + 16)):
        assert residual(lib, **bad) == INV, bad
    for bad in (dict(dn=None), dict(hn=None), dict(y=None), dict(dh=None), dict(flags=0), dict(dh=HN), dict(dy=DU),
                dict(dy=DG), dict(dy=Y), dict(dh=DG + 16), dict(dw=W), dict(dpw=DW), dict(ws=None), dict(wsb=100),
                dict(ws=DH), dict(dy=DY + 4)):
        assert residual_back(lib, **bad) == INV, bad
    assert residual(lib, rows=0) == OK
    assert residual_back(lib, rows=0, dw=None, dpw=None) == OK


@no_gpu
def test_norms_in_place_pass_the_checks(lib):
    assert residual(lib, hn=H, n=Y) == B.LA2_ERR_CUDA
    assert residual(lib, y=None, hn=None) == B.LA2_ERR_CUDA
    assert residual_back(lib, dh=DG) == B.LA2_ERR_CUDA
    assert residual_back(lib, dhn=None, dy=None) == B.LA2_ERR_CUDA
    assert gated(lib, gate=None) == B.LA2_ERR_CUDA


def test_norm_workspace_sizes(lib):
    size = lambda op, *a: lib.la2_workspace_size(op, *a, B.LA2_BF16)  # noqa: E731
    g, r = B.LA2_OP_GATED_NORM_BACKWARD, B.LA2_OP_RESIDUAL_NORM_BACKWARD
    assert size(r, 1, 1, 1, 100, 0) == 104 * 4 * 2                  # one row of partial sums for each weight, aligned
    assert size(r, 1, 1, 3, 16384, 0) == 3 * 16384 * 4 * 2
    assert size(r, 1, 1, 1 << 33, 64, 0) == size(r, 1, 1, 1 << 20, 64, 0)   # bounded by the GPU
    assert size(r, 1, 1, 5, 16385, 0) == 0 and size(r, 1, 1, 0, 64, 0) == 0
    assert size(g, 1, 4, 1, 64, 128) == 4 * 128 * 4
    assert size(g, 1, 4, 1, 64, 96) == 0 and size(g, 0, 4, 1, 64, 64) == 0
    assert size(g, 8, 1024, 8192, 64, 128) > 0                      # per head only: no limit on the row


def pool(lib, a=Q, na=8, b=Q, nb=8, src=SRC, dst=DST, n=4, layers=1, Hn=1, d=64, e=64):
    return lib.la2_pool_copy(a, na, b, nb, src, dst, n, layers, Hn, d, e, None)


def test_pool_copy_validation(lib):
    for bad in (dict(n=-1), dict(layers=-1), dict(Hn=-1), dict(na=-1), dict(nb=-1), dict(a=None), dict(b=None),
                dict(src=None), dict(dst=None), dict(src=SRC + 2), dict(a=Q + 4), dict(b=Q + 16384),
                dict(a=Q + 16384), dict(nb=7), dict(src=Q + 64), dict(b=K, dst=K + 16), dict(b=K, src=K + 7 * 16384)):
        assert pool(lib, **bad) == INV, bad
    for bad in (dict(d=32), dict(e=80), dict(n=4097)):
        assert pool(lib, **bad) == UNS, bad
    for empty in (dict(n=0), dict(layers=0), dict(Hn=0)):
        assert pool(lib, **empty) == OK


def test_bindings_refuse_host_tensors(lib):
    x = torch.zeros(1, 2, 3, 64)
    f = torch.zeros(32, dtype=torch.float64)
    i = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: la2.rotary(x, x, f), lambda: la2.rotary_backward(x, x, f), lambda: la2.gated_norm(x),
                 lambda: la2.gated_norm_backward(x.view(1, 3, 128), x), lambda: la2.residual_norm(x),
                 lambda: la2.residual_norm_backward(x, x), lambda: la2.pool_copy(x, i, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
