"""The fp64 references of the operators around the attention: against finite
differences, closed forms of the gradients and hand values."""
import math

import pytest
import torch

import causal_linear_attention_fwd_b200 as la2
import layer_ref as ref


def gen(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_by_hand_and_by_complex_products(interleaved):
    x = gen(1, 2, 3, 5, 8)
    f = torch.tensor([1.0, 0.25], dtype=torch.float64)
    pos = torch.tensor([0, 1000], dtype=torch.int64)
    q, k, v = ref.rotary(x, x[:, :1], x[:, 1:2], f, pos, interleaved, 1.5)
    assert torch.equal(q[..., 4:], x[..., 4:]) and torch.equal(v, x[:, 1:2].expand(2, 3, 5, 8))
    assert torch.equal(k[:, 0], k[:, 2])
    a, b = (slice(0, 4, 2), slice(1, 4, 2)) if interleaved else (slice(0, 2), slice(2, 4))
    p = pos[:, None].double() + torch.arange(5)
    z = torch.complex(x[..., a].contiguous(), x[..., b].contiguous())
    z = z * torch.polar(torch.full((2, 1, 5, 2), 1.5, dtype=torch.float64), (p[..., None] * f)[:, None])
    assert torch.allclose(q[..., a], z.real, atol=1e-13) and torch.allclose(q[..., b], z.imag, atol=1e-13)
    # position 0 turns nothing
    assert torch.allclose(q[0, :, 0, :4], 1.5 * x[0, :, 0, :4], atol=0)


def test_rotary_products_depend_on_the_distance_alone():
    f, _ = la2.rotary_frequencies(64, device="cpu")
    q, k = gen(2, 1, 1, 1, 64), gen(3, 1, 1, 1, 64)
    at = lambda x, p: ref.rotary(x, x, None, f, torch.tensor([p]), False, 1.0)[0]  # noqa: E731
    near, far = (at(q, 17 + s) * at(k, 5 + s) for s in (0, 1 << 20))
    assert abs(float(near.sum() - far.sum())) < 1e-8


def test_rotary_frequencies():
    f, s = la2.rotary_frequencies(8, 10000.0, device="cpu")
    assert s == 1.0 and torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64))
    g, _ = la2.rotary_frequencies(8, scaling="linear", factor=4.0, device="cpu")
    assert torch.equal(g, f / 4)
    g, _ = la2.rotary_frequencies(8, scaling="base", factor=4.0, device="cpu")
    assert g[0] == 1.0 and math.isclose(float(g[-1]), 0.001 / 4, rel_tol=1e-12)
    g, s = la2.rotary_frequencies(128, scaling="by_parts", factor=8.0, original_length=4096, device="cpu")
    f, _ = la2.rotary_frequencies(128, device="cpu")
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns > 32], f[turns > 32])
    assert torch.allclose(g[turns < 1], f[turns < 1] / 8, rtol=1e-14)
    assert bool((g <= f).all()) and bool((g >= f / 8 * (1 - 1e-12)).all())
    assert math.isclose(s, 1 + 0.1 * math.log(8))
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, factor=0.5),
                dict(rotary_dim=8, scaling="else"), dict(rotary_dim=8, base=1.0),
                dict(rotary_dim=8, scaling="by_parts", fast=1.0)):
        with pytest.raises(ValueError):
            la2.rotary_frequencies(**bad, device="cpu")


@pytest.mark.parametrize("per_head", [True, False])
@pytest.mark.parametrize("kind", ["silu", "sigmoid"])
@pytest.mark.parametrize("shared", [True, False])
def test_gated_norm_gradients(per_head, kind, shared):
    if shared and not per_head:
        shared = False
    B, H, L, e, eps = 2, 3, 2, 4, 1e-3
    o, g, w, up = gen(1, B, H, L, e), gen(2, B, L, H * e), gen(3, e if shared else H * e), gen(4, B, L, H * e)
    f = lambda *x: ref.gated_norm(*x, kind, per_head, eps)  # noqa: E731
    leaves = [t.clone().requires_grad_() for t in (o, g, w)]
    assert torch.autograd.gradcheck(f, leaves)
    do, dg, dw = ref.grads([f(*leaves)], [up], leaves)
    # the closed forms
    z, ww = g.reshape(B, L, H, e), (w.repeat(H) if shared else w).reshape(H, e)
    dims = (3,) if per_head else (2, 3)
    x = o.transpose(1, 2)
    rstd = ((x * x).mean(dims, keepdim=True) + eps).rsqrt()
    y, s, u = x * rstd, torch.sigmoid(z), up.reshape(B, L, H, e)
    a, da = (z * s, s * (1 + z * (1 - s))) if kind == "silu" else (s, s * (1 - s))
    dy = u * ww * a
    assert torch.allclose(do, (rstd * (dy - y * (dy * y).mean(dims, keepdim=True))).transpose(1, 2))
    assert torch.allclose(dg, (u * ww * y * da).reshape(B, L, -1))
    assert torch.allclose(dw, (u * a * y).sum((0, 1, 2) if shared else (0, 1)).flatten())


@pytest.mark.parametrize("post", [True, False])
def test_residual_norm_gradients(post):
    N, D, eps, al, be = 3, 5, 1e-3, 0.7, -1.3
    h, y, w, pw, un, uh = (gen(i, *s) for i, s in enumerate([(N, D), (N, D), (D,), (D,), (N, D), (N, D)]))
    f = lambda h, y, w, pw: ref.residual_norm(h, y, w, post, pw if post else None, al, be, eps)  # noqa: E731
    leaves = [t.clone().requires_grad_() for t in (h, y, w, pw)]
    assert torch.autograd.gradcheck(f, leaves)
    hn, n = f(*leaves)
    dh, dy, dw, dpw = ref.grads([hn, n], [uh, un], leaves)
    with torch.no_grad():
        r = (hn.pow(2).mean(1, keepdim=True) + eps).rsqrt()
        x, s = hn * r, un * w
        dH = uh + r * (s - x * (s * x).mean(1, keepdim=True))
        assert torch.allclose(dh, al * dH) and torch.allclose(dw, (un * x).sum(0))
        if not post:
            assert torch.allclose(dy, be * dH)
            return
        ry = (y.pow(2).mean(1, keepdim=True) + eps).rsqrt()
        yn, z = y * ry, be * dH * pw
        assert torch.allclose(dy, ry * (z - yn * (z * yn).mean(1, keepdim=True)))
        assert torch.allclose(dpw, (be * dH * yn).sum(0))


def test_rotary_gradient():
    q, k, v = gen(1, 1, 4, 2, 8), gen(2, 1, 2, 2, 8), gen(3, 1, 2, 2, 4)
    f = torch.tensor([0.9, 0.2, 0.01], dtype=torch.float64)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    for inter in (False, True):
        g = lambda q, k, v: tuple(ref.rotary(q, k, v, f, torch.tensor([7]), inter, 1.2))  # noqa: E731,B023
        assert torch.autograd.gradcheck(g, leaves)


def test_pool_copy_reference():
    p = torch.arange(5.0)[:, None, None, None].expand(5, 1, 2, 2).contiguous()
    src, dst = torch.tensor([1, 0, 0, -1, 4]), torch.tensor([0, 1, 2, 3, -1])
    assert ref.pool_copy(p, src, dst)[:, 0, 0, 0].tolist() == [1, 0, 0, 0, 4]
