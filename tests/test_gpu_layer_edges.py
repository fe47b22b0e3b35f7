"""The operators around the attention where their plans, launches and numbers
meet their limits: rows that two CTAs share, threads that call at once, gates
far out, streams given by name.  Tolerances as in test_gpu_layer.py unless a
test derives its own."""
import math

import pytest
import torch

import causal_linear_attention_fwd_b200 as la2
import layer_ref as ref
from layer_ref import F32, close, d64
from test_gpu_layer import BF, DEV, FP, gated_inputs, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("case", [
    (2, 129, 3, 64, False, "full", True, "silu", 0),        # uneven shares: 65 heads and 64
    (2, 255, 3, 64, False, "full", True, "sigmoid", 3),
    (1, 131, 5, 64, False, "none", False, "silu", 0),
    (2, 65, 3, 128, False, "full", True, "silu", 1)])
def test_gated_norm_wide_rows_of_odd_heads(case, dtype):
    """Rows of more than 8,192 columns, which two CTAs share, of an odd number
    of heads: u, do and dgate against the formulas, and what stands in front of
    and behind them left as it was."""
    B, H, L, e, per_head, weight, gate, act, pad = case
    g, o, z, w, how = gated_inputs(case, dtype, 15)
    du = randn(g, B, L, H * e, dtype=dtype)
    guard = 4096                                          # values around each output

    def walled(*shape):
        n = math.prod(shape)
        flat = torch.full((n + 2 * guard,), 3.0, device=DEV, dtype=dtype)
        return flat, flat[guard:guard + n].view(shape)
    bufs = [walled(B, L, H * e), walled(B, H, L, e), walled(B, L, H * e)]
    u = la2.gated_norm(o, z, w, out=bufs[0][1], **how)
    do, dg, dw = la2.gated_norm_backward(du, o, z, w, out=(bufs[1][1], bufs[2][1] if gate else None), **how)
    assert la2.last_device_error() == 0
    for flat, _ in bufs:
        assert bool((flat[:guard] == 3).all()) and bool((flat[-guard:] == 3).all())
    leaves = [ref.leaf(t) for t in (o, z, w)]
    up = d64(du)
    want_u = ref.gated_norm(*leaves, act, per_head, 1e-5)
    want = ref.grads([want_u], [up], leaves)
    close("u", u, want_u, dtype, 128 * F32 * want_u.detach().abs())
    x = d64(o).transpose(1, 2)
    rstd = ((x * x).mean((2, 3), keepdim=True) + 1e-5).rsqrt()
    y = (x * rstd).abs()
    zz = d64(z).unflatten(-1, (H, e)) if gate else None
    s = torch.sigmoid(zz) if gate else None
    a = torch.ones_like(y) if not gate else (s * zz if act == "silu" else s)
    ww = torch.ones(H, e, dtype=torch.float64) if w is None else d64(w).reshape(H, e)
    dy = (up.unflatten(-1, (H, e)) * ww * a).abs()
    size = (rstd * (dy + y * (dy * y).mean((2, 3), keepdim=True))).transpose(1, 2)
    close("do", do, want[0], dtype, 128 * F32 * size)
    if gate:
        slope = s * (1 + zz.abs()) if act == "silu" else s
        close("dgate", dg, want[1], dtype, 128 * F32 * ((up.unflatten(-1, (H, e)) * ww).abs() * y * slope).flatten(2))
    if w is not None:
        close("dw", dw, want[2], FP, (B * L + 128) * F32 * ((up.unflatten(-1, (H, e)) * a).abs() * y).sum((0, 1)).flatten())
