"""The attention's calls on a stream given by name that is not the current one:
scratch, inputs that are dropped and results are not handed out before their
last use."""
import pytest
import torch

import causal_linear_attention_fwd_b200 as la2
from causal_linear_attention_fwd_b200 import inputs

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
B, H, L, d, e = 1, 2, 4096, 128, 128


def busy(stream):
    """Keeps a stream at work for some 20 ms."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(40_000_000)


def calls():
    """name: (its tensors, the call on copies of them).  Split sequences, so that
    the calls that take scratch need it."""
    x = inputs.make_inputs(B, H, L, d, e, dtype=torch.bfloat16, device=DEV, seed=3, with_kv0=True)
    base = dict(q=x["q"], k=x["k"], v=x["v"], lam=inputs.fixed_lambdas((0.99, 0.5), DEV), kv0=x["kv0"], dO=x["dO"])
    packed = {n: base[n][0].contiguous() for n in ("q", "k", "v", "dO")} | {
        "lam": base["lam"], "cu": torch.tensor([0, 1000, 1000, L], device=DEV)}
    slots = torch.tensor([2], dtype=torch.int32, device=DEV)
    pool = torch.randn(3, H, d, e, device=DEV, generator=torch.Generator(DEV).manual_seed(4))
    few = {n: base[n][:, :, :5].contiguous() for n in ("q", "k", "v")} | {"lam": base["lam"], "pool": pool, "slots": slots}
    one = {n: base[n][:, :, 0].contiguous() for n in ("q", "k", "v")} | {"lam": base["lam"], "kv": pool[:1].clone()}

    def over(tensor, name, f):  # a call that works on a buffer of its own
        def run(t, **kw):
            return f(t, **kw), t[name]
        return tensor, run
    return {
        "forward": (base, lambda t, **kw: la2.forward(t["q"], t["k"], t["v"], t["lam"], t["kv0"], want_state=True, **kw)),
        "forward_noalloc": (base, lambda t, **kw: la2.forward_noalloc(t["q"], t["k"], t["v"], t["lam"], t["kv0"],
                                                                      want_state=True, **kw)),
        "backward": (base, lambda t, **kw: la2.backward(t["q"], t["k"], t["v"], t["lam"], t["dO"], t["kv0"], want_dkv0=True, **kw)),
        "forward_varlen": (packed, lambda t, **kw: la2.forward_varlen(t["q"], t["k"], t["v"], t["lam"], t["cu"],
                                                                      want_state=True, **kw)),
        "backward_varlen": (packed, lambda t, **kw: la2.backward_varlen(t["q"], t["k"], t["v"], t["lam"], t["cu"], t["dO"],
                                                                        want_dkv0=True, **kw)),
        "forward_pool": over(base | {"pool": pool, "slots": slots}, "pool", lambda t, **kw: la2.forward_pool(
            t["q"], t["k"], t["v"], t["lam"], t["pool"], t["slots"], continue_state=True, **kw)),
        "decode_tokens": over(few, "pool", lambda t, **kw: la2.decode_tokens(t["q"], t["k"], t["v"], t["lam"], t["pool"],
                                                                             t["slots"], **kw)),
        "decode_step": over(one, "kv", lambda t, **kw: la2.decode_step(t["q"], t["k"], t["v"], t["lam"], t["kv"], **kw)),
        "shard_state": (base, lambda t, **kw: la2.shard_state(t["k"], t["v"], t["lam"], **kw)),
        "state_prefix": ({"delta": pool[:, None].contiguous(), "lam": base["lam"]},
                         lambda t, **kw: la2.state_prefix(t["delta"], t["lam"], 64, **kw)),
        "backward_shard": (base, lambda t, **kw: la2.backward_shard(t["q"], t["k"], t["v"], t["lam"], t["dO"], t["kv0"],
                                                                    want_dkv0=True, **kw)),
        "dlambda": (base, lambda t, **kw: la2.dlambda(t["q"], t["k"], t["v"], t["lam"], t["dO"], t["kv0"], **kw)),
        "dlambda_whole": (base, lambda t, **kw: la2.dlambda(t["q"], t["k"], t["v"], t["lam"], t["dO"], t["kv0"],
                                                            chunked=False, **kw)),
        "feature_map": (base, lambda t, **kw: la2.feature_map(t["q"], t["k"], **kw)),
        "feature_map_backward": (base, lambda t, **kw: la2.feature_map_backward(t["q"], t["k"], t["q"], t["k"], **kw)),
    }


def same(name, got, want):
    """Equal; the decay gradients, whose chunks are added in any order, to the
    library's bar for them."""
    if name.startswith("dlambda"):
        return bool(((got[0] - want[0]).abs() <= 1e-3 * want[0].abs()).all())
    return all(torch.equal(a, b) for a, b in zip(got, want))


def flat(r):
    return [y for x in r for y in flat(x)] if isinstance(r, (tuple, list)) else [r]


@pytest.mark.parametrize("name", [
    "forward", "forward_noalloc", "backward", "forward_varlen", "backward_varlen", "forward_pool", "decode_tokens",
    "decode_step", "shard_state", "state_prefix", "backward_shard", "dlambda", "dlambda_whole", "feature_map",
    "feature_map_backward"])
def test_named_stream(name):
    data, call = calls()[name]
    copies = lambda: {n: t.clone() for n, t in data.items()}  # noqa: E731
    want = flat(call(copies()))
    torch.cuda.synchronize()
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    sizes = [torch.empty_like(t, device="meta") for t in [*data.values(), *want]]
    scratch = [la2.workspace_size(op, B, H, L, d, e, torch.bfloat16) for op in
               (la2.LA2_OP_FORWARD, la2.LA2_OP_BACKWARD, la2.LA2_OP_SHARD_STATE, la2.LA2_OP_DLAMBDA)]
    assert all(scratch)

    def fill():
        new = [torch.empty(s.shape, dtype=s.dtype, device=DEV) for s in sizes for _ in range(2)]
        new += [torch.empty(n, dtype=torch.uint8, device=DEV) for n in scratch]
        return [t.fill_(7) for t in new]
    own = copies()
    torch.cuda.synchronize()
    busy(side)
    got = flat(call(own, stream=side))
    del own                                               # before the named stream has read it
    new = fill()
    torch.cuda.synchronize()
    assert same(name, got, want)
    assert all(bool((t == 7).all()) for t in new)
    del got, new
    own = copies()
    torch.cuda.synchronize()
    got = flat(call(own, stream=side))
    main.wait_stream(side)
    busy(main)
    kept = [t.clone() for t in got]                       # when the current stream gets there
    del got, own                                          # and is dropped before
    with torch.cuda.stream(side):
        new = fill()
    torch.cuda.synchronize()
    assert same(name, kept, want)
    assert len(new) and la2.last_device_error() == 0
