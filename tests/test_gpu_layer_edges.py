"""The operators around the attention where their plans, launches and numbers
meet their limits: rows that two CTAs share, threads that call at once, gates
far out, streams given by name.  Tolerances as in test_gpu_layer.py unless a
test derives its own."""
import math
import os
import struct
import subprocess
import sys
import threading

import pytest
import torch

import causal_linear_attention_fwd_b200 as la2
import layer_ref as ref
from layer_ref import F32, close, d64
from test_gpu_layer import BF, DEV, FP, gated_inputs, gen, randn

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


def test_host_threads_at_different_sizes():
    """Two host threads whose calls run the same kernels with different amounts
    of shared memory: rows of 2,560 and 4,096 columns, 16 and 128 turned columns
    with shared heads.  The C entries in a close loop, where one thread's set-up
    falls into another's: every call is launched and right."""
    g = gen(71)
    lib, rows, B, H, L, d = la2.library(), 2, 1, 2, 3, 64
    jobs = []
    for D, r in ((2560, 16), (4096, 64)):
        h, y = randn(g, rows, D), randn(g, rows, D, dtype=BF)
        dq, dk, f = randn(g, B, H, L, d), randn(g, B, H, L, d), la2.rotary_frequencies(r, device=DEV)[0]
        want = [*la2.residual_norm(h, y), *la2.rotary_backward(dq, dk, f, kv_heads=1)]
        outs = [torch.zeros_like(t) for t in want]
        p = [t.data_ptr() for t in outs]
        side = torch.cuda.Stream()
        head = struct.Struct("=qqqq").pack
        gq, gk = (head(x.data_ptr(), *x.stride()[:3]) for x in outs[2:])
        norm = (h.data_ptr(), 0, y.data_ptr(), None, None, p[0], p[1], 1.0, 1.0, 1e-6, 0, rows, D, 1, side.cuda_stream)
        turn = (dq.data_ptr(), dk.data_ptr(), None, f.data_ptr(), None, 0, gq, gk, None, 1.0, 0, B, H, 1, L, d, d, r, 0,
                side.cuda_stream)
        jobs.append((norm, turn, outs, want, (h, y, dq, dk, f, side)))
    torch.cuda.synchronize()
    start, codes = threading.Barrier(2), [set(), set()]

    def loop(i):
        norm, turn = jobs[i][:2]
        start.wait()
        for call, args in ((lib.la2_residual_norm, norm), (lib.la2_rotary_backward, turn)):
            for _ in range(20000):
                codes[i].add(call(*args))
    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{0}, {0}]
    for _, _, outs, want, _ in jobs:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert la2.last_device_error() == 0


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("activation", ["silu", "sigmoid"])
@pytest.mark.parametrize("per_head", [True, False])
def test_gates_far_out(per_head, activation, dtype):
    """Gates to +-104 and beyond.  o is +-1, so a row's norm is the one number r
    that the call without a gate gives, and u = +-r a(g) errs by the gate's own
    steps.  In units of 2^-24 of the value:
      fp32   the power of two 4 (2^-22), its correction 1, 1 + e^-|g| 1, the
             reciprocal and the product 1 each, times r 1, times g (silu) 1: 10;
             where the result is subnormal, 4 last places (2^-149) of the
             sigmoid, which silu multiplies by g.
      bf16   (|g| + 4) 2 by the approximate instructions and 3 for the products,
             half a step of the type, and below g = -87 the sigmoid's less than
             2^-126 left out.
    The gradient of g: the sigmoid's 8, 1 - s with s's 8 and 1 of its own, one
    product with g and one sum, four products: under 24 of its terms; a result
    below 2^-126 is off by half a step of the type's subnormals (2^-134, 2^-150).
    do = r (dy - y mean(dy y)) is linear in the sigmoid, so what a sigmoid leaves
    out enters as r (|up| lost + |y| mean(|up| lost |y|))."""
    g = gen(72)
    B, H, L, e = 1, 4, 40, 64
    o = torch.where(torch.rand(B, H, L, e, generator=g, device=DEV) < 0.5, -1.0, 1.0).to(dtype)
    z = torch.empty(B, L, H * e, device=DEV).uniform_(-104, 104, generator=g)
    z[:, :10] = torch.linspace(-104, -80, 10 * H * e, device=DEV).view(10, H * e)
    z[0, 10, :10] = torch.tensor([20., -20., 60., -60., 86., -86., 90., -90., 1e4, -1e4], device=DEV)
    z = z.to(dtype)
    du = randn(g, B, L, H * e, dtype=dtype)
    how = dict(activation=activation, per_head=per_head)
    r = d64(la2.gated_norm(o.float(), **how)).abs()
    assert bool((r == r.flatten()[0]).all())
    u = la2.gated_norm(o, z, **how)
    do, dg, _ = la2.gated_norm_backward(du, o, z, **how)
    assert la2.last_device_error() == 0
    zz, y, silu = d64(z), d64(o).transpose(1, 2).flatten(2) * r, activation == "silu"
    s = torch.sigmoid(zz)
    a = s * zz if silu else s
    times = 1 + zz.abs() if silu else torch.ones_like(zz)
    if dtype == FP:
        slack, lost = 10 * F32, 4 * 2.0 ** -149 * times
    else:
        slack, lost = ref.HALF[BF] + (2 * zz.abs() + 11) * F32, torch.where(zz < -87, 2.0 ** -126 * times, 0.0)
    off = (d64(u) - y * a).abs()
    bad = off > (1 + 2.0 ** -6) * slack * (y * a).abs() + lost
    assert not bool(bad.any()), (int(bad.sum()), zz[bad][:4], (off / (y * a).abs())[bad][:4] / F32)
    slope = s * (1 + zz * (1 - s)) if silu else s * (1 - s)
    up = d64(du)
    terms, want = (up * y).abs() * s * times, up * y * slope
    step = 24 * F32 if dtype == FP else (2 * zz.abs() + 24) * F32
    bound = ref.HALF[dtype] * want.abs() * (1 + 2.0 ** -6) + step * terms + (lost + 2.0 ** -149) * (1 + up.abs()) * 2
    bound = bound + (2.0 ** -150 if dtype == FP else 2.0 ** -134)
    off = (d64(dg) - want).abs()
    assert bool((off <= bound).all()), (off / bound).max()
    dy = (up * a).abs()
    over = lambda t: t.unflatten(-1, (H, e)).mean(-1 if per_head else (-2, -1), keepdim=True).expand(B, L, H, e).flatten(2)  # noqa: E731
    want = r * (up * a - y * over(up * a * y))
    size = r * (dy + y.abs() * over(dy * y.abs()))
    turn = lambda t: t.unflatten(-1, (H, e)).transpose(1, 2)  # noqa: E731
    far = 0 if dtype == FP else 2 * 104 * F32
    left = r * (up.abs() * lost + y.abs() * over(up.abs() * lost * y.abs()))
    close("do", do, turn(want), dtype, turn((128 * F32 + far) * size + left))


def busy(stream):
    """Keeps a stream at work for some 20 ms."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(40_000_000)


def same_size(tensors):
    """New tensors of these sizes on the current stream, filled with 7: they take
    the memory that has come free."""
    return [torch.full_like(t, 7, memory_format=torch.contiguous_format) for t in tensors for _ in range(2)]


@pytest.mark.parametrize("call", ["gated", "residual"])
def test_scratch_of_a_call_on_a_named_stream(call):
    """A backward named for a busy stream that is not the current one: what the
    current stream allocates after the return meets neither its scratch nor its
    results, and the weights' gradients are right."""
    g = gen(73)
    side = torch.cuda.Stream()
    if call == "gated":
        o, z, w, du = randn(g, 2, 4, 300, 64), randn(g, 2, 300, 256), 1 + randn(g, 256, scale=.2), randn(g, 2, 300, 256)
        run = lambda **kw: la2.gated_norm_backward(du, o, z, w, **kw)  # noqa: E731
        n = la2.workspace_size(la2.LA2_OP_GATED_NORM_BACKWARD, 2, 4, 300, 64, 64, FP)
    else:
        h, y, dn, w = randn(g, 500, 1024), randn(g, 500, 1024), randn(g, 500, 1024), 1 + randn(g, 1024, scale=.2)
        run = lambda **kw: la2.residual_norm_backward(dn, h, y, w, dh_new=y, post_norm=True, post_weight=w, **kw)  # noqa: E731
        n = la2.workspace_size(la2.LA2_OP_RESIDUAL_NORM_BACKWARD, 1, 1, 500, 1024, 1024, FP)
    want = run()
    torch.cuda.synchronize()
    busy(side)
    got = run(stream=side)
    others = same_size([torch.empty(n // 4, device=DEV) for _ in range(4)] + list(got))
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in others)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_memory_of_a_call_on_a_named_stream():
    """Inputs dropped while a named stream has yet to read them, and results
    dropped while the caller's has: neither's memory is handed out before."""
    g = gen(74)
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    B, H, L, d = 2, 4, 200, 64
    f, _ = la2.rotary_frequencies(d, device=DEV)
    src, dst = torch.tensor([1, 0], dtype=torch.int32, device=DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    x = [randn(g, B, H, L, d) for _ in range(3)]
    z, w, pool = randn(g, B, L, H * d), 1 + randn(g, H * d, scale=.2), randn(g, 3, H, d, d)

    def all_of(stream=None):
        q, k, v = (t.clone() for t in x)
        zz, ww, h = z.clone(), w.clone(), z + 1
        main.synchronize()
        if stream is not None:
            busy(stream)
        kw = dict(stream=stream)
        r = list(la2.rotary(q, k, f.clone(), v=v, **kw))
        r += la2.rotary_backward(q, k, f.clone(), dv=v, **kw)
        r.append(la2.gated_norm(v, zz, ww, **kw))
        r += la2.gated_norm_backward(zz, v, zz, ww, **kw)
        r += la2.residual_norm(h, zz, ww, **kw)
        r += la2.residual_norm_backward(zz, h, None, ww, **kw)[:3]
        copy = pool.clone()
        main.synchronize()
        r.append(la2.pool_copy(copy, src.clone(), dst.clone(), **kw))
        return r
    want = all_of()
    torch.cuda.synchronize()
    got = all_of(side)                                    # its inputs are dropped by now
    taken = same_size(x + [z, w, pool, f.float(), src])
    main.wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    del taken, got
    got = all_of(side)
    main.wait_stream(side)
    busy(main)
    kept = [t.clone() for t in got]                       # read when main gets there
    shapes = [torch.empty(t.shape, device="meta") for t in got]
    del got
    with torch.cuda.stream(side):
        over = [torch.full(s.shape, 7.0, device=DEV) for s in shapes for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))
    assert len(over) == 2 * len(want) and la2.last_device_error() == 0


@pytest.mark.parametrize("D", [64, 99, 2048, 5001, 16384])
def test_one_tensor_as_stream_and_block_output(D):
    """h and y one tensor, and an output over both; the gradients of n and h' one
    tensor, and dh over both: the bits of the call on copies."""
    g = gen(75)
    x, w = randn(g, 300, D), 1 + randn(g, D, scale=.2)
    how = dict(post_norm=True, post_weight=w, alpha=0.5, beta=2.0)
    hn, n = la2.residual_norm(x, x.clone(), w, **how)
    for which in (0, 1):
        y = x.clone()
        outs = (y, torch.empty_like(y)) if which == 0 else (torch.empty_like(y), y)
        la2.residual_norm(y, y, w, out=outs, **how)
        assert torch.equal(outs[0], hn) and torch.equal(outs[1], n)
    up = randn(g, 300, D)
    want = la2.residual_norm_backward(up, hn, x, w, dh_new=up.clone(), **how)
    over = up.clone()
    got = la2.residual_norm_backward(over, hn, x, w, dh_new=over, out=(over, None), **how)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert la2.last_device_error() == 0


@pytest.mark.parametrize("D", [96, 99, 2048, 2049, 16384])
def test_one_weight_of_two(D):
    """A norm on y with one of the two weights: the other's gradient is not made,
    and this one's has the bits of the call with ones for the other."""
    g = gen(76)
    hn, y, dn, up = (randn(g, 700, D) for _ in range(4))
    w, one = 1 + randn(g, D, scale=.2), torch.ones(D, device=DEV)
    how = dict(dh_new=up, post_norm=True)
    full = la2.residual_norm_backward(dn, hn, y, w, post_weight=one, **how)
    got = la2.residual_norm_backward(dn, hn, y, w, **how)
    assert got[3] is None and all(torch.equal(a, b) for a, b in zip(got[:3], full))
    full = la2.residual_norm_backward(dn, hn, y, one, post_weight=w, **how)
    got = la2.residual_norm_backward(dn, hn, y, None, post_weight=w, **how)
    assert got[2] is None and all(torch.equal(got[i], full[i]) for i in (0, 1, 3))
    assert la2.last_device_error() == 0


FIRST = """
import torch
import causal_linear_attention_fwd_b200 as la2
import test_gpu_layer as t
call = t.all_calls(81)
h, y = t.randn(t.gen(82), 5, 4096), t.randn(t.gen(82), 5, 4096)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call() + list(la2.residual_norm(h, y, post_norm=True)) + list(la2.residual_norm_backward(h, y, None)[:2])
graph.replay()
torch.cuda.synchronize()
want = call() + list(la2.residual_norm(h, y, post_norm=True)) + list(la2.residual_norm_backward(h, y, None)[:2])
assert all(torch.equal(a, b) for a, b in zip(got, want)) and la2.last_device_error() == 0
print("same")
"""


def test_first_calls_of_a_process_captured():
    """No call before the capture: what a first call sets up is allowed there."""
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": os.pathsep.join((here, os.path.dirname(here)))})
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_named_stream_inside_a_capture():
    """A capture that forks to a named stream and joins it again: scratch and
    results come from the graph's memory, and every replay gives the bits of the
    eager calls."""
    g = gen(77)
    side = torch.cuda.Stream()
    o, z, du = randn(g, 2, 4, 300, 64), randn(g, 2, 300, 256), randn(g, 2, 300, 256)
    h, y, w = randn(g, 500, 1024), randn(g, 500, 1024), 1 + randn(g, 1024, scale=.2)
    q, lam = randn(g, 1, 2, 2048, 64), torch.full((2,), 0.9, device=DEV)

    def calls(stream=None):
        r = list(la2.gated_norm_backward(du, o, z, w[:256], stream=stream))
        r += la2.residual_norm_backward(h, y, y, w, dh_new=y, post_norm=True, post_weight=w, stream=stream)
        return r + list(la2.backward(q, q, q, lam, la2.forward(q, q, q, lam, stream=stream), stream=stream))
    want = calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        got = calls(side)
        main.wait_stream(side)
        kept = [t.clone() for t in got]
        more = [torch.full_like(t, 7) for t in got]
    for _ in range(3):
        for t in (*got, *kept, *more):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(kept, want))
        assert all(bool((t == 7).all()) for t in more)
    assert la2.last_device_error() == 0
