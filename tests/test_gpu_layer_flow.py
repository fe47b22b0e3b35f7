"""The operators around the attention used together, as a layer and a server
use them: a training step of one attention layer against fp64 autograd over
the same formulas (the attention's part by the oracle), and a decode loop over a
state pool whose requests are forked, reordered and compacted."""
import numpy as np
import pytest
import torch

import causal_linear_attention_fwd_b200 as la2
import layer_ref as ref
from causal_linear_attention_fwd_b200 import inputs
from gpu_util import check
from layer_ref import d64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float32


def randn(g, *shape, dtype=FP, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def layer_forward(p, h, positions):
    """One layer on the residual stream h [B,L,D], as its user writes it: norm,
    projection, rotary positions, attention, gated norm, output projection,
    residual sum and next norm.  Returns everything the backward needs."""
    B, L, D = h.shape
    H, Hk, d = p["H"], p["Hk"], p["d"]
    _, n1 = la2.residual_norm(h, None, p["w1"], dtype=p["dt"])
    x = n1 @ p["win"]                                            # [B,L,(H+2Hk)d + Hd]
    cut = lambda at, n: x[..., at:at + n * d].unflatten(-1, (n, d)).transpose(1, 2)  # noqa: E731
    q, k, v = cut(0, H), cut(H * d, Hk), cut((H + Hk) * d, Hk)
    gate = x[..., (H + 2 * Hk) * d:]
    rq, rk, rv = la2.rotary(q, k, p["f"], positions, v=v, scale=p["scale"])
    o = la2.forward(rq, rk, rv, p["lam"])
    u = la2.gated_norm(o, gate, p["wg"])
    y = u @ p["wout"]
    h2, n2 = la2.residual_norm(h, y, p["w2"], post_norm=True, post_weight=p["wp"], alpha=p["alpha"], beta=p["beta"])
    return dict(n1=n1, x=x, gate=gate, rq=rq, rk=rk, rv=rv, o=o, u=u, y=y, h2=h2, n2=n2)


def layer_backward(p, h, positions, s, dn2, dh2):
    """Gradients of the layer's weights and input, call by call."""
    B, L, D = h.shape
    H, Hk, d = p["H"], p["Hk"], p["d"]
    dh, dy, dw2, dwp = la2.residual_norm_backward(dn2, s["h2"], s["y"], p["w2"], dh_new=dh2, post_norm=True,
                                                  post_weight=p["wp"], alpha=p["alpha"], beta=p["beta"])
    du = dy @ p["wout"].T
    dwout = s["u"].flatten(0, 1).T @ dy.flatten(0, 1)
    dx = torch.empty_like(s["x"])
    cut = lambda at, n: dx[..., at:at + n * d].unflatten(-1, (n, d)).transpose(1, 2)  # noqa: E731
    do = torch.empty_like(s["o"])
    _, _, dwg = la2.gated_norm_backward(du, s["o"], s["gate"], p["wg"], out=(do, dx[..., (H + 2 * Hk) * d:]))
    dq, dk, dv = la2.backward(s["rq"], s["rk"], s["rv"], p["lam"], do)
    la2.rotary_backward(dq, dk, p["f"], positions, dv=dv, kv_heads=Hk, scale=p["scale"],
                        out=(cut(0, H), cut(H * d, Hk), cut((H + Hk) * d, Hk)))
    dn1 = dx @ p["win"].T
    dwin = s["n1"].flatten(0, 1).T @ dx.flatten(0, 1)
    dh1, _, dw1, _ = la2.residual_norm_backward(dn1, h, None, p["w1"], dh_new=dh, want_dy=False)
    return dict(dh=dh1, dw1=dw1, dwin=dwin, dwg=dwg, dwout=dwout, dw2=dw2, dwp=dwp)


@pytest.mark.parametrize("dtype,stream", [(FP, FP), (BF, BF), (BF, FP)])
def test_training_step_of_a_layer(orc, dtype, stream):
    g = torch.Generator(device=DEV).manual_seed(3)
    B, L, H, Hk, d, D = 2, 75, 4, 2, 64, 136
    f, scale = la2.rotary_frequencies(d, scaling="by_parts", factor=4.0, original_length=64, device=DEV)
    p = dict(H=H, Hk=Hk, d=d, dt=dtype, f=f, scale=scale, alpha=0.9, beta=0.4, lam=inputs.decay_lambdas(H, DEV),
             w1=1 + randn(g, D, scale=.1), w2=1 + randn(g, D, scale=.1), wp=1 + randn(g, D, scale=.1),
             wg=1 + randn(g, d, scale=.1), win=randn(g, D, (2 * H + 2 * Hk) * d, dtype=dtype, scale=D ** -.5),
             wout=randn(g, H * d, D, dtype=dtype, scale=(H * d) ** -.5))
    p["win"][:, :(H + Hk) * d] *= d ** -.25
    h, positions = randn(g, B, L, D, dtype=stream), torch.tensor([0, 1 << 20], device=DEV)
    dn2, dh2 = randn(g, B, L, D, dtype=dtype), randn(g, B, L, D, dtype=stream)
    s = layer_forward(p, h, positions)
    got = layer_backward(p, h, positions, s, dn2, dh2)
    torch.cuda.synchronize()
    assert la2.last_device_error() == 0

    # the same layer in fp64: the attention by its quadratic form (held to the
    # oracle below), everything else by the references' formulas
    leaves = {n: ref.leaf(t) for n, t in (("h", h), ("w1", p["w1"]), ("win", p["win"]), ("wg", p["wg"]),
                                          ("wout", p["wout"]), ("w2", p["w2"]), ("wp", p["wp"]))}
    x = ref.residual_norm(leaves["h"], None, leaves["w1"], False, None, 1, 1, 1e-6)[1] @ leaves["win"]
    cut = lambda at, n: x[..., at:at + n * d].unflatten(-1, (n, d)).transpose(1, 2)  # noqa: E731
    rq, rk, rv = ref.rotary(cut(0, H), cut(H * d, Hk), cut((H + Hk) * d, Hk), f, positions, False, scale)
    t = torch.arange(L)
    apart = t[:, None] - t
    mask = torch.where(apart >= 0, d64(p["lam"])[:, None, None] ** apart.clamp(min=0), 0.0)
    attention = lambda q, k, v: ((q @ k.transpose(-1, -2)) * mask) @ v  # noqa: E731
    o = attention(rq, rk, rv)
    # the oracle takes fp32 inputs: both on the rounded ones
    low = [a.detach().float() for a in (rq, rk, rv)]
    held, _ = orc.forward(*(np.ascontiguousarray(a.numpy()) for a in low), d64(p["lam"]).numpy(), None,
                          want_state=True)
    assert np.abs(held - attention(*(a.double() for a in low)).numpy()).max() <= 1e-12 * np.abs(held).max()
    u = ref.gated_norm(o, x[..., (H + 2 * Hk) * d:], leaves["wg"], "silu", True, 1e-6)
    h2, n2 = ref.residual_norm(leaves["h"], u @ leaves["wout"], leaves["w2"], True, leaves["wp"], .9, .4, 1e-6)
    want = ref.grads([h2, n2], [d64(dh2), d64(dn2)], list(leaves.values()))
    # fp32: the attention's bar.  bf16: some ten tensors in a row are rounded to
    # 2^-8 of their values, each independent of the others, so their errors
    # add in squares to 2^-8 / sqrt(3) * sqrt(10) of the norm, under 1e-2 each;
    # products of them with cancelling sums (weight gradients) take 3 times that
    tol = {FP: 1e-4, BF: 3e-2}[dtype]
    pairs = [("h2", s["h2"], h2), ("n2", s["n2"], n2)]
    pairs += [(n, got[n], w) for n, w in zip(("dh", "dw1", "dwin", "dwg", "dwout", "dw2", "dwp"), want)]
    for name, a, b in pairs:
        a, b = d64(a), b.detach()
        rel = float((a - b).norm() / b.norm())
        assert rel <= tol, f"{name}: {rel:.2e} of the norm"


@pytest.mark.parametrize("layers", [1, 3])
def test_decode_over_a_pool_that_forks_and_moves(orc, layers):
    """Prefill two requests, fork one of them twice, decode, reorder the beams
    (two go on from one parent), compact, decode again: every request's
    outputs are those of the oracle run over its own history of tokens."""
    H, d, P, T0 = 3, 64, 9, 20
    lam = inputs.decay_lambdas(H, DEV)
    lam_h = d64(lam).numpy()
    f, scale = la2.rotary_frequencies(32, device=DEV)
    pool = torch.full((layers, P, H, d, d), 7.0, device=DEV)   # left over from earlier requests
    move = lambda s, t: la2.pool_copy(pool, *(torch.tensor(x, dtype=torch.int32, device=DEV) for x in (s, t)))  # noqa: E731
    g = torch.Generator(device=DEV).manual_seed(8)
    history = {}                                              # slot -> list of (q, k, v) per layer, as fed

    def feed(slots, T, prefill=False):
        B = len(slots)
        start = torch.tensor([0 if prefill else history[s][0][0].shape[1] for s in slots], device=DEV)
        table = torch.tensor(slots, dtype=torch.int32, device=DEV)
        outs = []
        for layer in range(layers):
            x = randn(g, B, T, 3 * H * d, dtype=BF, scale=d ** -.25)
            q, k, v = (x[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)).transpose(1, 2) for i in range(3))
            rq, rk, rv = la2.rotary(q, k, f, start, v=v, scale=scale)
            if prefill:
                o = la2.forward_pool(rq, rk, rv, lam, pool[layer], table)
            else:
                o = la2.decode_tokens(rq, rk, rv, lam, pool[layer], table)
            u = la2.gated_norm(o)
            outs.append(u)
            for i, s in enumerate(slots):
                past = history.setdefault(s, [None] * layers)
                new = [t[i] for t in (rq, rk, rv)]
                past[layer] = new if past[layer] is None or prefill else [torch.cat(z, 1) for z in zip(past[layer], new)]
        for layer in range(layers):
            for i, s in enumerate(slots):
                q, k, v = (np.ascontiguousarray(d64(t)[None].numpy()) for t in history[s][layer])
                o = torch.from_numpy(orc.forward(q, k, v, lam_h, None, want_state=True)[0])[:, :, -T:]
                want = ref.gated_norm(o, None, None, "silu", True, 1e-6)[0]
                check(f"layer {layer} slot {s}", outs[layer][i], want.numpy(), BF)

    def moved(src, dst):
        move(src, dst)
        old = {s: [list(x) if x else x for x in v] for s, v in history.items()}
        for a, b in zip(src, dst):
            if a < 0:
                history.pop(b, None)
            elif a in old:
                history[b] = [list(x) for x in old[a]]

    feed([4, 6], T0, prefill=True)
    moved([4, 4], [0, 8])                     # fork
    feed([4, 0, 8, 6], 1)
    moved([8, 8, 4], [4, 0, 8])               # beams: 4 and 0 go on from 8, 8 from 4
    feed([0, 4, 8], 5)
    moved([6, 8, 4, -1, -1], [1, 2, 3, 6, 8])  # compact, and clear what is left behind
    history[6] = [[torch.empty(H, 0, d, device=DEV, dtype=BF)] * 3 for _ in range(layers)]
    feed([0, 1, 2, 3, 6], 2)                  # slot 6: a new request from a cleared state
    assert la2.last_device_error() == 0
    assert float((pool[:, 5] - 7).abs().max()) == 0 and float((pool[:, 7] - 7).abs().max()) == 0
