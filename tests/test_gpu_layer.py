"""GPU parity of the operators around the attention against fp64 references
(tests/layer_ref.py): rotary positions, gated norm, residual norm and pool
copies, forward and backward, over the shapes, layouts and values where they
can go wrong.

Tolerances, elementwise: half a step of the output's type at the reference
value, plus the fp32 arithmetic's error, a multiple of 2^-24 times the
magnitudes that enter (K below):
  rotation   an angle less its whole turns keeps 2^-26 turns = 2^-23.3 rad, the
             sine and cosine 2 ulp, the scale, two products and a sum 1 each:
             under 8 * 2^-24 of |a| + |b|; a shared head's sum of `rep` terms
             adds rep - 1 roundings; fp64 angles of positions up to 2^30 err by
             2^30 * 3 * 2^-53 turns, under 2^-20 rad: 16 * 2^-24 more.
  norms      a sum of D <= 16,384 squares: at most 32 terms in a thread, 10
             levels of a tree, 32 more: under 80 roundings, half of it in
             the root; exponential and quotient under 2 ^ 5 steps for |g| <= 8;
             products: under 128 * 2^-24 of the terms that are added.
  weights    R rows: R + 128 roundings of the sum of the terms' magnitudes.
"""
import pytest
import torch

import causal_linear_attention_fwd_b200 as la2
import layer_ref as ref
from layer_ref import F32, close, d64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=FP, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


# ------------------------------------------------------------------ rotary
def fused(g, B, L, H, Hk, d, e, dtype, pad, per_head=False):
    """q, k, v as views of one token-major buffer; pad extra columns before
    them make rows that no 16-byte piece fits when odd."""
    if per_head:  # [B,L,H,3,d]: q, k, v of a head side by side
        x = randn(g, B, L, H * 3 * d + pad, dtype=dtype)
        y = x[..., pad:].view(B, L, H, 3, d) if pad == 0 else x[..., pad:].unflatten(-1, (H, 3, d))
        return x, *(y[..., i, :].transpose(1, 2) for i in range(3))
    x = randn(g, B, L, H * d + Hk * (d + e) + pad, dtype=dtype)
    cut = lambda at, n, w: x[..., at:at + n * w].unflatten(-1, (n, w)).transpose(1, 2)  # noqa: E731
    return x, cut(pad, H, d), cut(pad + H * d, Hk, d), cut(pad + (H + Hk) * d, Hk, e)


def make_positions(kind, g, B, L, far):
    if kind == "none":
        return None
    hi = 1 << (30 if far else 12)
    return torch.randint(-5, hi, (B,) if kind == "start" else (B, L), generator=g, device=DEV)


ROTARY = [
    # B, H, Hk, L, d, e, r, pad, positions
    (1, 1, 1, 1, 64, 64, 64, 0, "none"),
    (3, 4, 4, 1, 128, 128, 64, 0, "start"),
    (2, 4, 2, 33, 128, 64, 128, 0, "table"),
    (2, 6, 1, 17, 64, 128, 16, 0, "start"),
    (1, 5, 5, 130, 128, 128, 32, 8, "none"),
    (2, 4, 1, 9, 64, 64, 2, 0, "table"),       # one pair: value by value
    (2, 3, 3, 21, 128, 64, 20, 0, "none"),     # half of r not a multiple of 8
    (2, 8, 4, 7, 64, 128, 62, 3, "start"),     # rows off the 16-byte grid
    (1, 64, 8, 5, 128, 128, 128, 0, "start"),
    (70, 2, 2, 1, 64, 64, 32, 0, "table"),
]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", ROTARY)
def test_rotary(case, interleaved, dtype):
    B, H, Hk, L, d, e, r, pad, kind = case
    g = gen(sum(case[:8]))
    _, q, k, v = fused(g, B, L, H, Hk, d, e, dtype, pad)
    pos = make_positions(kind, g, B, L, far=r > 16)
    f, scale = la2.rotary_frequencies(r, scaling="by_parts", factor=4.0, original_length=512, device=DEV)
    got = la2.rotary(q, k, f, pos, v=v, interleaved=interleaved, scale=scale)
    assert la2.last_device_error() == 0
    want = ref.rotary(d64(q), d64(k), d64(v), f, pos, interleaved, scale)
    sizes = [ref.pair_size(d64(x), r // 2, scale, interleaved) for x in (q, k)]
    sizes[1] = sizes[1].repeat_interleave(H // Hk, 1)
    for name, y, z, s in zip("qk", got, want, sizes):
        assert y.is_contiguous() and y.dtype == dtype
        close(name, y, z, dtype, 24 * F32 * s)
    assert torch.equal(got[2], v.repeat_interleave(H // Hk, 1))   # copied, bit for bit
    if r < d:
        assert torch.equal(got[0][..., r:], q[..., r:])
    # without v, into the caller's buffers, the same bits
    outs = [torch.empty_like(t) for t in got[:2]]
    again = la2.rotary(q, k, f, pos, interleaved=interleaved, scale=scale, out=outs)
    assert len(again) == 2 and torch.equal(outs[0], got[0]) and torch.equal(outs[1], got[1])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", ROTARY)
def test_rotary_backward(case, interleaved, dtype):
    B, H, Hk, L, d, e, r, pad, kind = case
    g = gen(1 + sum(case[:8]))
    x, gq, gk, gv = fused(g, B, L, H, Hk, d, e, dtype, pad)
    before = x.clone()
    dq, dk, dv = (randn(g, B, H, L, n, dtype=dtype) for n in (d, d, e))
    pos = make_positions(kind, g, B, L, far=r > 16)
    f, scale = la2.rotary_frequencies(r, device=DEV)[0], 1.25
    how = dict(interleaved=interleaved, scale=scale)
    la2.rotary_backward(dq, dk, f, pos, dv=dv, kv_heads=Hk, out=(gq, gk, gv), **how)
    assert la2.last_device_error() == 0
    assert torch.equal(x[..., :pad], before[..., :pad])           # beside the slices: untouched
    leaves = [torch.zeros(B, n, L, w, dtype=torch.float64, requires_grad=True)
              for n, w in ((H, d), (Hk, d), (Hk, e))]
    outs = ref.rotary(*leaves, f, pos, interleaved, scale)
    want = ref.grads(outs, [d64(t) for t in (dq, dk, dv)], leaves)
    rep = H // Hk
    total = lambda t: d64(t).abs().unflatten(1, (Hk, rep)).sum(2)  # noqa: E731
    sq = ref.pair_size(d64(dq), r // 2, scale, interleaved)
    sk = ref.pair_size(total(dk), r // 2, scale, interleaved)
    close("gq", gq, want[0], dtype, 24 * F32 * sq)
    close("gk", gk, want[1], dtype, (24 + rep) * F32 * sk + rep * F32 * total(dk))
    close("gv", gv, want[2], dtype, rep * F32 * total(dv))
    # default outputs: token-major buffers, the same bits
    a, b = la2.rotary_backward(dq, dk, f, pos, kv_heads=Hk, **how)
    assert a.transpose(1, 2).is_contiguous() and torch.equal(a, gq) and torch.equal(b, gk)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_rotary_heads_side_by_side_and_expanded(dtype):
    """q, k, v of each head side by side [B,L,H,3,d]; a k head expanded with
    stride 0; head-major inputs; a head axis outside the rows."""
    g = gen(5)
    B, L, H, d = 2, 19, 4, 64
    x, q, k, v = fused(g, B, L, H, H, d, d, dtype, 0, per_head=True)
    f, _ = la2.rotary_frequencies(64, device=DEV)
    rq, rk, rv = la2.rotary(q, k, f, v=v)
    c = [t.contiguous() for t in (q, k, v)]
    assert all(torch.equal(a, b) for a, b in zip((rq, rk, rv), la2.rotary(c[0], c[1], f, v=c[2])))
    one = c[1][:, :1]
    wide = la2.rotary(q, one.expand(B, H, L, d), f)[1]
    assert torch.equal(wide, la2.rotary(q, one, f)[1])
    la2.rotary_backward(rq, rk, f, dv=rv, out=(q, k, v))          # back into the same buffer
    size = ref.pair_size(d64(c[0]), 32, 1.0, False)
    close("there and back", q, d64(c[0]), dtype, ref.HALF[dtype] * 3 * size + 48 * F32 * size)
    assert torch.equal(v, c[2])
    la2.last_device_error()


def test_rotary_refuses():
    g = gen(6)
    f, _ = la2.rotary_frequencies(64, device=DEV)
    q = randn(g, 2, 4, 8, 64, dtype=BF)
    k = randn(g, 2, 2, 8, 64, dtype=BF)
    bad = [lambda: la2.rotary(q, k[:, :, :4], f), lambda: la2.rotary(q, k.float(), f),
           lambda: la2.rotary(q, k[..., ::2], f), lambda: la2.rotary(q, k, f.float()),
           lambda: la2.rotary(q, k, f, torch.zeros(3, dtype=torch.int64, device=DEV)),
           lambda: la2.rotary(q, k, f, torch.zeros(2, dtype=torch.int32, device=DEV)),
           lambda: la2.rotary(q, k.cpu(), f), lambda: la2.rotary(q, randn(g, 2, 3, 8, 64, dtype=BF), f),
           lambda: la2.rotary(q, k, f, out=(q.clone(),)),
           lambda: la2.rotary_backward(q, q, f, kv_heads=3)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(la2.LA2Error):     # r above d
        la2.rotary(q, k, torch.zeros(33, dtype=torch.float64, device=DEV))
    with pytest.raises(la2.LA2Error):     # an output over an input
        la2.rotary(q, k, f, out=(q, torch.empty_like(q)))
    with pytest.raises(la2.LA2Error):     # gradients on top of one another
        la2.rotary_backward(q, q.clone(), f, out=(torch.empty_like(q),) * 2)
    e = torch.empty(2, 1, 8, 64, device=DEV, dtype=BF).expand(2, 4, 8, 64)
    with pytest.raises(la2.LA2Error):     # a gradient whose heads share their place
        la2.rotary_backward(q, q.clone(), f, out=(torch.empty_like(q), e))
    with pytest.raises(TypeError):
        la2.rotary(q.half(), k.half(), f)


def test_empty_calls():
    """No rows, no heads or no requests: empty results, zero weight gradients."""
    f, _ = la2.rotary_frequencies(64, device=DEV)
    for B, H, L in ((0, 2, 3), (2, 2, 0), (2, 0, 3)):
        x = torch.empty(B, H, L, 64, device=DEV)
        assert la2.rotary(x, x, f)[1].shape == x.shape
        assert la2.rotary_backward(x, x, f)[0].shape == x.shape
        u = la2.gated_norm(x, torch.empty(B, L, H * 64, device=DEV))
        assert u.shape == (B, L, H * 64)
        w = torch.ones(64, device=DEV)
        do, dg, dw = la2.gated_norm_backward(u, x, u, w)
        assert do.shape == x.shape and dg.shape == u.shape and torch.equal(dw, torch.zeros_like(w))
    h = torch.empty(0, 24, device=DEV)
    w = torch.ones(24, device=DEV)
    assert la2.residual_norm(h, h, w)[1].shape == h.shape
    dh, dy, dw, _ = la2.residual_norm_backward(h, h, h, w)
    assert dh.shape == dy.shape == h.shape and torch.equal(dw, torch.zeros_like(w))
    pool = torch.ones(3, 1, 64, 64, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    assert bool((la2.pool_copy(pool, none, none) == 1).all())


# ------------------------------------------------------------------ gated norm
GATED = [
    # B, H, L, e, per_head, weight, gate, activation, pad
    (1, 1, 1, 64, True, "shared", True, "silu", 0),
    (2, 4, 33, 128, True, "full", True, "sigmoid", 0),
    (1, 6, 50, 64, True, "shared", True, "silu", 8),
    (3, 5, 7, 128, True, "none", True, "silu", 3),
    (2, 64, 3, 128, True, "full", False, "silu", 0),
    (1, 20, 301, 64, True, "shared", False, "sigmoid", 0),
    (2, 48, 40, 64, True, "shared", True, "sigmoid", 1),
    (1, 1, 5, 64, False, "full", True, "silu", 0),
    (2, 4, 130, 128, False, "full", True, "silu", 0),       # a warp per row
    (2, 5, 33, 128, False, "none", True, "sigmoid", 5),
    (1, 32, 21, 128, False, "full", True, "sigmoid", 0),
    (2, 33, 9, 128, False, "full", True, "silu", 0),
    (1, 128, 5, 128, False, "full", False, "silu", 0),      # the widest row
    (1, 2, 700, 128, False, "full", True, "silu", 0),
    (1, 3, 2500, 64, True, "full", True, "silu", 0),
]


def gated_inputs(case, dtype, seed):
    B, H, L, e, per_head, weight, gate, act, pad = case
    g = gen(seed)
    o = randn(g, B, H, L, e, dtype=dtype, scale=2.0)
    if L > 2:
        o[:, :, 1] = 0                                    # a row that was masked away
        o[:, :, 2] *= 1e-4
    z = randn(g, B, L, pad + H * e, dtype=dtype, scale=1.5).clamp(-8, 8)[..., pad:] if gate else None
    w = None if weight == "none" else 1 + randn(g, e if weight == "shared" else H * e, scale=0.3)
    return g, o, z, w, dict(activation=act, per_head=per_head, eps=1e-5)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("case", GATED)
def test_gated_norm(case, dtype):
    g, o, z, w, how = gated_inputs(case, dtype, 11)
    u = la2.gated_norm(o, z, w, **how)
    assert la2.last_device_error() == 0
    want = ref.gated_norm(d64(o), d64(z), d64(w), how["activation"], how["per_head"], 1e-5)
    close("u", u, want, dtype, 128 * F32 * want.abs())
    if case[2] > 2:
        assert bool((u[:, 1] == 0).all())
    buf = torch.empty_like(u)
    assert la2.gated_norm(o, z, w, out=buf, **how) is buf and torch.equal(buf, u)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("case", GATED)
def test_gated_norm_backward(case, dtype):
    B, H, L, e, per_head, weight, gate, act, pad = case
    g, o, z, w, how = gated_inputs(case, dtype, 12)
    du = randn(g, B, L, H * e, dtype=dtype)
    do, dg, dw = la2.gated_norm_backward(du, o, z, w, **how)
    assert la2.last_device_error() == 0
    leaves = [ref.leaf(t) for t in (o, z, w)]
    up = d64(du)
    want = ref.grads([ref.gated_norm(*leaves, act, per_head, 1e-5)], [up], leaves)
    # magnitudes of the terms that are added
    x = d64(o).transpose(1, 2)
    dims = (3,) if per_head else (2, 3)
    rstd = ((x * x).mean(dims, keepdim=True) + 1e-5).rsqrt()
    y = (x * rstd).abs()
    s = torch.sigmoid(d64(z)).unflatten(-1, (H, e)) if gate else None
    a = torch.ones_like(y) if not gate else (s * d64(z).unflatten(-1, (H, e)) if act == "silu" else s)
    ww = torch.ones(H, e, dtype=torch.float64) if w is None else d64(w).repeat(H if weight == "shared" else 1).reshape(H, e)
    dy = (up.unflatten(-1, (H, e)) * ww * a).abs()
    size = (rstd * (dy + y * (dy * y).mean(dims, keepdim=True))).transpose(1, 2)
    close("do", do, want[0], dtype, 128 * F32 * size)
    if gate:
        zz = d64(z).unflatten(-1, (H, e)).abs()
        slope = s * (1 + zz) if act == "silu" else s     # its terms, added up
        close("dgate", dg, want[1], dtype, 128 * F32 * ((up.unflatten(-1, (H, e)) * ww).abs() * y * slope).flatten(2))
    else:
        assert dg is None
    if w is not None:
        terms = (up.unflatten(-1, (H, e)) * a).abs() * y
        rows = B * L * (H if weight == "shared" else 1)
        total = terms.sum((0, 1, 2) if weight == "shared" else (0, 1)).flatten()
        close("dw", dw, want[2], FP, (rows + 128) * F32 * total)
    else:
        assert dw is None
    # into the caller's tensors (the gate's a slice), the same bits
    wide = torch.full((B, L, H * e + 7), 3.0, device=DEV, dtype=dtype)
    outs = (torch.empty_like(do), wide[..., 7:] if gate else None)
    again = la2.gated_norm_backward(du, o, z, w, out=outs, **how)
    assert torch.equal(outs[0], do) and bool((wide[..., :7] == 3).all())
    assert not gate or torch.equal(outs[1], dg)
    assert w is None or torch.equal(again[2], dw)        # a fixed order of summation


def test_gated_norm_non_finite_rows_stay_alone():
    g = gen(13)
    for per_head in (True, False):
        o, z = randn(g, 1, 4, 9, 64, dtype=BF), randn(g, 1, 9, 256, dtype=BF)
        clean = la2.gated_norm(o, z, per_head=per_head)
        o[:, :, 3], o[:, :, 5], z[:, 7] = float("nan"), float("inf"), float("-inf")
        got = la2.gated_norm(o, z, per_head=per_head)
        keep = [0, 1, 2, 4, 6, 8]
        assert torch.equal(got[:, keep], clean[:, keep])
        assert bool(got[:, 3].isnan().all()) and bool(got[:, 5].isnan().all())
        far = z.clone()
        far[:, 7] = -3e38                                 # the lowest values: sigmoid 0
        low = la2.gated_norm(o, far, per_head=per_head, activation="sigmoid")
        assert bool((low[:, 7] == 0).all())


def test_gated_norm_refuses():
    g = gen(14)
    o = randn(g, 1, 2, 4, 64)
    z, w = randn(g, 1, 4, 128), torch.ones(64, device=DEV)
    bad = [lambda: la2.gated_norm(o, z[:, :3]), lambda: la2.gated_norm(o, z.to(BF)),
           lambda: la2.gated_norm(o, z, w, per_head=False), lambda: la2.gated_norm(o, z, w.double()),
           lambda: la2.gated_norm(o, z, activation="tanh"), lambda: la2.gated_norm(o.cpu(), z),
           lambda: la2.gated_norm(o.transpose(2, 3), z), lambda: la2.gated_norm(o, z, torch.ones(65, device=DEV)),
           lambda: la2.gated_norm(o, torch.zeros(1, 4, 256, device=DEV)[..., ::2]),
           lambda: la2.gated_norm_backward(z[:, :2], o, z, w),
           lambda: la2.gated_norm_backward(z, o, z, w, out=(torch.empty_like(o), None))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(la2.LA2Error):
        la2.gated_norm(o, z, eps=0.0)
    with pytest.raises(la2.LA2Error):     # another head size
        la2.gated_norm(randn(g, 1, 2, 4, 32))
    with pytest.raises(la2.LA2Error):     # a row wider than a CTA holds
        la2.gated_norm(randn(g, 1, 129, 1, 128), per_head=False)
    with pytest.raises(la2.LA2Error):     # too small a workspace
        la2.gated_norm_backward(z, o, z, w, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(la2.LA2Error):     # rows of the gradient on one another
        la2.gated_norm_backward(z, o, z, w, out=(torch.empty_like(o), torch.empty(1, 1, 128, device=DEV).expand(1, 4, 128)))


# ------------------------------------------------------------------ residual norm
RESIDUAL = [
    # N, D, y type, h type, post, weights
    (1, 1, FP, FP, False, True), (3, 7, BF, BF, True, True), (5, 8, FP, FP, True, True),
    (300, 64, BF, FP, False, True), (4, 512, BF, BF, True, False), (3, 513, FP, FP, True, True),
    (7, 520, BF, BF, False, True), (601, 1111, FP, FP, False, True), (33, 2049, BF, FP, True, True),
    (1300, 256, BF, BF, True, True), (65, 4096, BF, BF, False, True), (9, 4096, BF, FP, True, True),
    (9, 4104, FP, FP, True, True), (5, 16384, BF, BF, True, True), (4, 16384, FP, FP, True, True),
    (5003, 99, BF, FP, True, True), (2600, 505, FP, FP, True, True), (4001, 3, BF, BF, False, True),
    (901, 1700, BF, BF, False, True), (400, 5001, BF, BF, True, True), (350, 4095, BF, FP, True, True),
    (340, 9001, FP, FP, False, True), (5, 4097, BF, BF, True, True), (2, 2043, BF, FP, True, False),
    (3, 16383, BF, FP, True, True), (3, 16383, FP, FP, False, False), (700, 8192, BF, FP, False, True),
]


def residual_inputs(case, seed):
    N, D, dt, hd, post, weights = case
    g = gen(seed)
    h, y = randn(g, N, D, dtype=hd, scale=3.0), randn(g, N, D, dtype=dt, scale=0.5)
    if N > 2:
        y[1] = 0
        h[2] *= 1e-3
    w = 1 + randn(g, D, scale=0.3) if weights else None
    pw = 1 + randn(g, D, scale=0.3) if weights and post else None
    return g, h, y, w, dict(post_norm=post, post_weight=pw, alpha=0.75, beta=-1.5, eps=1e-5)


def ref_residual(h, y, w, how):
    return ref.residual_norm(h, y, w, how["post_norm"], how["post_weight"], how["alpha"], how["beta"], how["eps"])


@pytest.mark.parametrize("case", RESIDUAL)
def test_residual_norm(case):
    N, D, dt, hd, post, weights = case
    g, h, y, w, how = residual_inputs(case, 21)
    hn, n = la2.residual_norm(h, y, w, **how)
    assert la2.last_device_error() == 0 and hn.dtype == hd and n.dtype == dt
    how64 = {**how, "post_weight": d64(how["post_weight"])}
    want_h, want_n = ref_residual(d64(h), d64(y), d64(w), how64)
    size = how["alpha"] * d64(h).abs() + (want_h - how["alpha"] * d64(h)).abs()
    close("h_new", hn, want_h, hd, 128 * F32 * size)
    r = (want_h.pow(2).mean(-1, keepdim=True) + 1e-5).rsqrt()
    ww = 1.0 if w is None else d64(w).abs()
    # n's error: its own, h's terms through the norm, and the norm's through theirs
    drift = (size * want_h.abs()).mean(-1, keepdim=True) * r * r
    close("n", n, want_n, dt, 128 * F32 * (r * ww * size + want_n.abs() * (1 + drift)))
    # in place: the same bits
    hh, yy = h.clone(), y.clone()
    la2.residual_norm(hh, yy, w, out=(hh, yy), **how)
    assert torch.equal(hh, hn) and torch.equal(yy, n)
    # the norm alone
    same, alone = la2.residual_norm(h, None, w, eps=1e-5, dtype=dt)
    assert same is h
    close("norm", alone, ref.residual_norm(d64(h), None, d64(w), False, None, 1, 1, 1e-5)[1], dt,
          128 * F32 * d64(alone).abs())


@pytest.mark.parametrize("upstream", [True, False])
@pytest.mark.parametrize("case", RESIDUAL)
def test_residual_norm_backward(case, upstream):
    N, D, dt, hd, post, weights = case
    g, h, y, w, how = residual_inputs(case, 22)
    al, be, eps = how["alpha"], how["beta"], how["eps"]
    hn = h                                                # the stored sum: any values
    dn = randn(g, N, D, dtype=dt)
    up = randn(g, N, D, dtype=hd) if upstream else None
    dh, dy, dw, dpw = la2.residual_norm_backward(dn, hn, y if post else None, w, dh_new=up, **how)
    assert la2.last_device_error() == 0
    # the two stages of the chain rule, each by autograd over the formulas
    x, ww = ref.leaf(hn), ref.leaf(w)
    dx, want_w = ref.grads([ref.residual_norm(x, None, ww, False, None, 1, 1, eps)[1]], [d64(dn)], [x, ww])
    dH = dx + (0 if up is None else d64(up))
    z, pw = ref.leaf(y), ref.leaf(how["post_weight"])
    p = ref.rms(z, eps, (-1,)) if post else z * 1.0
    p = p if pw is None else p * pw
    want_y, want_p = ref.grads([p], [be * dH], [z, pw])
    with torch.no_grad():
        one = torch.ones(D, dtype=torch.float64)
        r = (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
        xn, s = (x * r).abs(), (d64(dn) * (one if w is None else d64(w))).abs()
        size = r * (s + xn * (s * xn).mean(-1, keepdim=True)) + (0 if up is None else d64(up).abs())
        close("dh", dh, al * dH, hd, 128 * F32 * al * size)
        if post:
            ry = (z.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
            zn, pp = (z * ry).abs(), (one if pw is None else pw).abs()
            t = abs(be) * size * pp
            close("dy", dy, want_y, dt, 256 * F32 * ry * (t + zn * (t * zn).mean(-1, keepdim=True)))
        else:
            close("dy", dy, want_y, dt, 128 * F32 * abs(be) * size)
        if w is not None:
            close("dw", dw, want_w, FP, (N + 128) * F32 * (d64(dn).abs() * xn).sum(0))
        if pw is not None:
            close("dpw", dpw, want_p, FP, (N + 256) * F32 * (abs(be) * size * zn).sum(0))
        assert (dw is None) == (w is None) and (dpw is None) == (pw is None)
    # in place over the upstream gradient, without dy: the same bits
    if upstream:
        over = up.clone()
        a, b, c, _ = la2.residual_norm_backward(dn, hn, y if post else None, w, dh_new=over, out=(over, None),
                                                want_dy=False, **how)
        assert b is None and torch.equal(over, dh) and (w is None or torch.equal(c, dw))


def test_residual_norm_shapes_and_non_finite_rows():
    g = gen(23)
    h, y = randn(g, 2, 3, 5, 72, dtype=BF), randn(g, 2, 3, 5, 72, dtype=BF)
    a, b = la2.residual_norm(h, y, post_norm=True)
    c, d = la2.residual_norm(h.view(30, 72), y.view(30, 72), post_norm=True)
    assert a.shape == h.shape and torch.equal(a.view(30, 72), c) and torch.equal(b.view(30, 72), d)
    h.view(30, 72)[4], y.view(30, 72)[9] = float("nan"), float("inf")
    a2, b2 = la2.residual_norm(h, y, post_norm=True)
    keep = [i for i in range(30) if i not in (4, 9)]
    assert torch.equal(a2.view(30, 72)[keep], c[keep]) and torch.equal(b2.view(30, 72)[keep], d[keep])
    assert bool(b2.view(30, 72)[[4, 9]].isnan().all())


def test_residual_norm_refuses():
    g = gen(24)
    h, y, w = randn(g, 4, 64), randn(g, 4, 64), torch.ones(64, device=DEV)
    bad = [lambda: la2.residual_norm(h, y[:3]), lambda: la2.residual_norm(h, y, w[:63]),
           lambda: la2.residual_norm(h, y, w.to(BF)), lambda: la2.residual_norm(h, y, w, post_weight=w),
           lambda: la2.residual_norm(h, None, w, post_norm=True), lambda: la2.residual_norm(h, None, w, alpha=2.0),
           lambda: la2.residual_norm(h, y, dtype=BF), lambda: la2.residual_norm(h.t(), None),
           lambda: la2.residual_norm_backward(y, h, None, w, post_norm=True),
           lambda: la2.residual_norm_backward(y[:2], h, None, w),
           lambda: la2.residual_norm_backward(y, h, None, w, dh_new=h.to(BF))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(la2.LA2Error):     # a narrower stream than the block's output
        la2.residual_norm(h.to(BF), y)
    with pytest.raises(la2.LA2Error):
        la2.residual_norm(torch.zeros(1, 16385, device=DEV))
    with pytest.raises(la2.LA2Error):
        la2.residual_norm(h, y, eps=-1.0)
    with pytest.raises(la2.LA2Error):     # n over h
        la2.residual_norm(h, y, out=(torch.empty_like(h), h))
    with pytest.raises(la2.LA2Error):
        la2.residual_norm_backward(y, h, None, w, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


# ------------------------------------------------------------------ pool copies
def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def moves(kind, P, N, seed):
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(P, generator=g)[:N]
    if kind == "cycle":
        return torch.roll(perm, 1), perm
    if kind == "fork":
        return perm[:1].expand(N).clone(), perm
    if kind == "beams":
        return perm[torch.randint(0, N, (N,), generator=g)], perm
    src = torch.sort(perm).values.clone()                 # compact; some cleared, some not moved
    dst = torch.arange(N)
    src[N // 2::3] = -1
    dst[N // 3::5] = -1
    return src, dst


@pytest.mark.parametrize("kind", ["cycle", "fork", "beams", "compact"])
@pytest.mark.parametrize("shape,N", [((4, 1, 64, 64), 1), ((5, 3, 64, 128), 4), ((40, 2, 128, 128), 37),
                                     ((3, 9, 1, 64, 64), 7), ((700, 1, 64, 64), 600),
                                     ((2, 1100, 1, 64, 64), 1050), ((4200, 1, 64, 64), 4096)])
def test_pool_copy(kind, shape, N):
    pool = randn(gen(31), *shape)
    src, dst = moves(kind, shape[-4], N, 32 + N)
    want = ref.pool_copy(pool.cpu(), src, dst)
    out = la2.pool_copy(pool, src.int().to(DEV), dst.int().to(DEV))
    assert la2.last_device_error() == 0 and out is pool
    assert torch.equal(pool.cpu(), want)


def test_pool_copy_between_pools_and_bad_slots():
    g = gen(33)
    pool, other = randn(g, 6, 2, 64, 64), randn(g, 9, 2, 64, 64)
    keep = other.clone()
    want = ref.pool_copy(pool.cpu(), torch.tensor([8, -1, 0]), torch.tensor([0, 2, 5]), source=other.cpu())
    # slots past either pool are skipped and reported; the others move
    la2.pool_copy(pool, i32([8, -1, 9, 0, 3]), i32([0, 2, 1, 5, 6]), source=other)
    assert la2.last_device_error() == 1 and la2.last_device_error() == 0
    assert torch.equal(pool.cpu(), want) and torch.equal(other, keep)
    la2.pool_copy(pool, i32([0, 1]), i32([-1, -7]))       # no move at all
    assert la2.last_device_error() == 0 and torch.equal(pool.cpu(), want)


def test_pool_copy_past_32_bits():
    """A pool of more than 4 GiB: slots at both ends trade places."""
    P = 1100
    pool = torch.zeros(P, 64, 128, 128, device=DEV)
    for s in (0, 1, 1023, 1024, P - 1):
        pool[s] = torch.arange(s, s + 64, device=DEV)[:, None, None].float()
    src, dst = [P - 1, 0, 1024, 1], [0, P - 1, 1, 1024]
    want = {d: pool[s].clone() for s, d in zip(src, dst)}
    la2.pool_copy(pool, i32(src), i32(dst))
    assert la2.last_device_error() == 0
    assert all(torch.equal(pool[d], w) for d, w in want.items())
    assert bool((pool[1023] == torch.arange(1023, 1087, device=DEV)[:, None, None]).all())
    assert float(pool[2:1023].abs().max()) == 0


def test_pool_copy_refuses():
    pool = torch.zeros(4, 1, 64, 64, device=DEV)
    bad = [lambda: la2.pool_copy(pool, i32([0]), i32([0, 1])), lambda: la2.pool_copy(pool.to(BF), i32([0]), i32([1])),
           lambda: la2.pool_copy(pool, i32([0]).long(), i32([1])), lambda: la2.pool_copy(pool[0], i32([0]), i32([1])),
           lambda: la2.pool_copy(pool, i32([0]), i32([1]), source=torch.zeros(4, 2, 64, 64, device=DEV)),
           lambda: la2.pool_copy(pool, torch.zeros(1, dtype=torch.int32), i32([1]))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    many = torch.zeros(4097, dtype=torch.int32, device=DEV)
    with pytest.raises(la2.LA2Error):
        la2.pool_copy(pool, many, many)
    with pytest.raises(la2.LA2Error):     # pools that partly overlap
        la2.pool_copy(pool[1:], i32([0]), i32([1]), source=pool[:3])


# ------------------------------------------------------------------ how they are called
def all_calls(seed):
    """Every entry point once, on its own inputs; returns a callable and its results' tensors."""
    g = gen(seed)
    B, H, Hk, L, d = 2, 4, 2, 65, 64
    f, _ = la2.rotary_frequencies(64, device=DEV)
    x, q, k, v = fused(g, B, L, H, Hk, d, d, BF, 0)
    o, z, w = randn(g, B, H, L, d, dtype=BF), randn(g, B, L, H * d, dtype=BF), torch.ones(H * d, device=DEV)
    h, y = randn(g, B, L, 512), randn(g, B, L, 512, dtype=BF)
    hw, pool = torch.ones(512, device=DEV), randn(g, 8, H, d, d)
    src, dst = i32([1, 0, 2, 5]), i32([0, 1, 3, 6])

    def call(stream=None):
        r = list(la2.rotary(q, k, f, v=v, stream=stream))
        r += la2.rotary_backward(*r[:2], f, dv=r[2], kv_heads=Hk, stream=stream)
        r.append(la2.gated_norm(o, z, w, stream=stream))
        r += la2.gated_norm_backward(r[-1], o, z, w, stream=stream)
        r += la2.residual_norm(h, y, hw, post_norm=True, post_weight=hw, stream=stream)
        r += la2.residual_norm_backward(r[-1], r[-2], y, hw, dh_new=h, post_norm=True, post_weight=hw, stream=stream)
        r.append(la2.pool_copy(pool.clone(), src, dst, stream=stream))
        return r
    return call


def test_other_streams_and_graphs():
    call = all_calls(41)
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                         # the current stream is another one
        got = call()
        named = call(stream=side)                         # and given by name
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(a, b) for a, b in zip(want, named))
    graphs, results = [], []
    for seed in (41, 42):                                 # two graphs, replayed in turn and over again
        c = all_calls(seed)
        with torch.cuda.stream(side):
            c()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(c())
        graphs.append(graph)
    for t in results[0] + results[1]:
        t.zero_()
    for graph in graphs + graphs[::-1]:
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, results[0]))
    assert all(torch.equal(a, b) for a, b in zip(all_calls(42)(), results[1]))
    assert la2.last_device_error() == 0


def test_two_calls_at_once():
    """The same calls on two streams at once, over and over: no call shares
    anything with another."""
    calls = [all_calls(61), all_calls(62)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(calls[i]())
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(want[i], r))
    assert la2.last_device_error() == 0


def test_gate_shared_by_the_batch():
    """A gate with stride 0 over the batch, and one head's o of one token."""
    g = gen(63)
    o, z = randn(g, 3, 2, 5, 64, dtype=BF), randn(g, 1, 5, 128, dtype=BF)
    du = randn(g, 3, 5, 128, dtype=BF)
    wide = z.expand(3, 5, 128)
    for per_head in (True, False):
        assert torch.equal(la2.gated_norm(o, wide, per_head=per_head),
                           la2.gated_norm(o, wide.contiguous(), per_head=per_head))
        a = la2.gated_norm_backward(du, o, wide, per_head=per_head)
        b = la2.gated_norm_backward(du, o, wide.contiguous(), per_head=per_head)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])   # one gradient per use


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 values: their last rows equal those of a call
    on these rows alone."""
    g = gen(64)
    for D in (8192, 8191):                                # N * D just above 2^31
        N = (1 << 31) // D + 40
        keep = 8 + N % 8                                  # rows that begin at the same place in a 16-byte piece
        h, y = (torch.empty(N, D, device=DEV, dtype=BF).normal_(generator=g) for _ in range(2))
        w = torch.ones(D, device=DEV)
        hn, n = la2.residual_norm(h, y, w, post_norm=True)
        tail = lambda t: t[-keep:].clone()  # noqa: E731
        a, b = la2.residual_norm(tail(h), tail(y), w, post_norm=True)
        assert torch.equal(hn[-keep:], a) and torch.equal(n[-keep:], b)
        dh, dy, _, _ = la2.residual_norm_backward(n, hn, y, w, dh_new=h, post_norm=True)
        c, d, _, _ = la2.residual_norm_backward(b, a, tail(y), w, dh_new=tail(h), post_norm=True)
        assert torch.equal(dh[-keep:], c) and torch.equal(dy[-keep:], d)
        del h, y, hn, n, dh, dy
        torch.cuda.empty_cache()
    H, e, keep = 32, 64, 9
    L = (1 << 31) // (H * e) + 50
    o, z = torch.empty(1, H, L, e, device=DEV, dtype=BF), torch.empty(1, L, H * e, device=DEV, dtype=BF)
    o.normal_(generator=g)
    z.normal_(generator=g)
    for per_head in (True, False):
        u = la2.gated_norm(o, z, per_head=per_head)
        end = la2.gated_norm(o[:, :, -keep:].contiguous(), z[:, -keep:].contiguous(), per_head=per_head)
        assert torch.equal(u[:, -keep:], end)
        do, dz, _ = la2.gated_norm_backward(u, o, z, per_head=per_head)
        ref_do, ref_dz, _ = la2.gated_norm_backward(end, o[:, :, -keep:].contiguous(), z[:, -keep:].contiguous(), per_head=per_head)
        assert torch.equal(do[:, :, -keep:], ref_do) and torch.equal(dz[:, -keep:], ref_dz)
        del u, do, dz
    f, _ = la2.rotary_frequencies(e, device=DEV)
    q = z.unflatten(-1, (H, e)).transpose(1, 2)
    pos = torch.arange(L, device=DEV)[None] % 1000
    rq, rk = la2.rotary(q, q[:, :1], f, pos)
    a, b = la2.rotary(q[:, :, -keep:], q[:, :1, -keep:], f, pos[:, -keep:].contiguous())
    assert torch.equal(rq[:, :, -keep:], a) and torch.equal(rk[:, :, -keep:], b)
    gq, gk = la2.rotary_backward(rq, rk, f, pos, kv_heads=4)
    c, d = la2.rotary_backward(a, b, f, pos[:, -keep:].contiguous(), kv_heads=4)
    assert torch.equal(gq[:, :, -keep:], c) and torch.equal(gk[:, :, -keep:], d)
    assert la2.last_device_error() == 0


def test_directional_derivatives():
    """The kernels' gradients along random directions against central
    differences of the fp64 losses (fp32 inputs: 1e-5 of the gradient's and
    direction's norms bounds the kernels' 2^-24 errors and the differences')."""
    g = gen(51)
    B, H, L, e = 1, 3, 6, 64
    o, z, w, du = randn(g, B, H, L, e), randn(g, B, L, H * e), 1 + randn(g, H * e, scale=.2), randn(g, B, L, H * e)
    for per_head in (True, False):
        got = la2.gated_norm_backward(du, o, z, w, per_head=per_head)
        xs = [d64(t) for t in (o, z, w)]
        loss = lambda *a: float((ref.gated_norm(*a, "silu", per_head, 1e-6) * d64(du)).sum())  # noqa: E731,B023
        for i in range(3):
            t = d64(randn(g, *xs[i].shape))
            at = lambda s: loss(*[x + s * t if j == i else x for j, x in enumerate(xs)])  # noqa: E731,B023
            diff, dot = (at(1e-5) - at(-1e-5)) / 2e-5, float((d64(got[i]) * t).sum())
            assert abs(diff - dot) <= 1e-5 * float(d64(got[i]).norm() * t.norm())
    h, y, pw, hw = randn(g, 4, 96), randn(g, 4, 96), 1 + randn(g, 96, scale=.2), 1 + randn(g, 96, scale=.2)
    un, uh = randn(g, 4, 96), randn(g, 4, 96)
    how = dict(post_norm=True, alpha=0.8, beta=1.1)
    hn, _ = la2.residual_norm(h, y, hw, post_weight=pw, **how)
    dh, dy, dw, dpw = la2.residual_norm_backward(un, hn, y, hw, dh_new=uh, post_weight=pw, **how)
    xs = [d64(t) for t in (h, y, hw, pw)]

    def loss(h, y, w, p):
        a, b = ref.residual_norm(h, y, w, True, p, 0.8, 1.1, 1e-6)
        return float((a * d64(uh)).sum() + (b * d64(un)).sum())
    for i, grad in enumerate((dh, dy, dw, dpw)):
        t = d64(randn(g, *xs[i].shape))
        at = lambda s: loss(*[x + s * t if j == i else x for j, x in enumerate(xs)])  # noqa: E731,B023
        diff, dot = (at(1e-5) - at(-1e-5)) / 2e-5, float((d64(grad) * t).sum())
        assert abs(diff - dot) <= 1e-5 * float(d64(grad).norm() * t.norm())
