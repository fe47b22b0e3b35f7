"""fp64 references of the operators around the attention (rotary positions,
gated norm, residual norm, pool copies), written from their formulas on the
CPU, with the magnitudes that their rounding errors scale with.  Gradients come
from torch's autograd over these forward formulas; tests/test_layer_ref_cpu.py
holds them against finite differences and the closed forms."""
from __future__ import annotations

import torch

F32 = 2.0 ** -24                                    # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def d64(t):
    return None if t is None else t.detach().cpu().double()


def positions_of(positions, B, L):
    p = torch.arange(L, dtype=torch.float64).expand(B, L)
    if positions is None:
        return p
    q = d64(positions)
    return q[:, None] + p if q.dim() == 1 else q


def rotate(x, angle, scale, interleaved):
    """x [B,n,L,w] fp64, angle [B,L,r/2]: the first r columns turned."""
    half = angle.shape[-1]
    c, s = (f(angle)[:, None] * scale for f in (torch.cos, torch.sin))
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack((a * c - b * s, a * s + b * c), dim=-1).reshape(*x.shape[:-1], 2 * half)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat((a * c - b * s, a * s + b * c), dim=-1)
    return torch.cat((y, x[..., 2 * half:]), dim=-1)


def pair_size(x, half, scale, interleaved):
    """|a| + |b| of each value's pair, times the scale; 0 where nothing turns."""
    m = torch.zeros_like(x)
    if interleaved:
        s = x[..., 0:2 * half:2].abs() + x[..., 1:2 * half:2].abs()
        m[..., 0:2 * half:2], m[..., 1:2 * half:2] = s, s
    else:
        s = x[..., :half].abs() + x[..., half:2 * half].abs()
        m[..., :half], m[..., half:2 * half] = s, s
    return m * scale


def rotary(q, k, v, inv_freq, positions, interleaved, scale):
    B, H, L, _ = q.shape
    rep = H // k.shape[1]
    angle = positions_of(positions, B, L)[..., None] * d64(inv_freq)
    out = [rotate(q, angle, scale, interleaved),
           rotate(k, angle, scale, interleaved).repeat_interleave(rep, 1)]
    return out + ([] if v is None else [v.repeat_interleave(rep, 1)])


def activate(g, kind):
    s = torch.sigmoid(g)
    return g * s if kind == "silu" else s


def rms(x, eps, dims):
    return x / torch.sqrt((x * x).mean(dims, keepdim=True) + eps)


def gated_norm(o, gate, weight, kind, per_head, eps):
    """o [B,H,L,e] -> u [B,L,H*e]."""
    B, H, L, e = o.shape
    y = rms(o.transpose(1, 2), eps, (3,) if per_head else (2, 3))
    if weight is not None:
        y = y * (weight if weight.numel() == H * e else weight.repeat(H)).reshape(H, e)
    if gate is not None:
        y = y * activate(gate.reshape(B, L, H, e), kind)
    return y.reshape(B, L, H * e)


def residual_norm(h, y, weight, post_norm, post_weight, alpha, beta, eps):
    if y is not None:
        p = rms(y, eps, (-1,)) if post_norm else y
        if post_weight is not None:
            p = p * post_weight
        h = alpha * h + beta * p
    n = rms(h, eps, (-1,))
    return h, n if weight is None else n * weight


def grads(outs, ups, wrt):
    """Gradients of sum(out * up) for the tensors wrt (None kept)."""
    loss = sum((o * u).sum() for o, u in zip(outs, ups) if u is not None)
    got = iter(torch.autograd.grad(loss, [t for t in wrt if t is not None], allow_unused=True))
    return [None if t is None else next(got) for t in wrt]


def leaf(t):
    return None if t is None else d64(t).requires_grad_()


def close(name, got, ref, dtype, slack):
    """|got - ref| <= half a step of dtype at ref + slack (elementwise)."""
    got, ref = got.detach().cpu().double(), ref.detach()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    bound = HALF[dtype] * ref.abs() * (1 + 2.0 ** -6) + slack + 1e-37
    bad = ~((got - ref).abs() <= bound)
    if bool(bad.any()):
        i = int(torch.argmax(((got - ref).abs() / bound).nan_to_num(nan=1e30).flatten()))
        raise AssertionError(f"{name}: {int(bad.sum())} of {ref.numel()} off; worst got "
                             f"{got.flatten()[i]:.9g} for {ref.flatten()[i]:.9g}, bound "
                             f"{bound.flatten()[i]:.3g}")


def pool_copy(pool, src, dst, source=None):
    """pool [P,...] or [layers,P,...] by the definition, one move after another from a copy."""
    old = (pool if source is None else source).clone()
    new = pool.clone()
    for a, b in zip(src.tolist(), dst.tolist()):
        if b >= 0:
            if pool.dim() == 5:
                new[:, b] = old[:, a] if a >= 0 else 0.0
            else:
                new[b] = old[a] if a >= 0 else 0.0
    return new
