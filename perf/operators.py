"""The operators around the attention calls, as a layer and a server use them.

  rotary          positions turned into rotations of q and k, read out of a
                  fused token-major projection and written head-major for the
                  attention (k and v heads shared by several q heads repeated);
                  backward: the attention's gradients taken back into the
                  fused projection's layout
  gated_norm      the attention's output (head-major) normed per head or over
                  the whole row, times an activated gate, token-major for the
                  output projection; forward and backward
  residual_norm   the scaled residual sum after a block (the block's output
                  normed first if wanted) and the norm before the next block;
                  forward and backward
  pool_copy       recurrent states copied, forked, reordered, compacted and
                  cleared between the slots of a serving pool

`own = False` computes them with elementary torch operations, `own = True`
with this repository's package.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
DEV = "cuda"
MOST_BYTES = 3.3e9  # what the largest listed case moves


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token for each of 64 requests far into their texts, half of
        # each head rotated: the smallest call, between two products of a
        # decode step
        dict(name="rotary_decode", op="rotary", dir="fwd", B=64, H=16, Hk=16, L=1, d=128, e=128,
             r=64, interleaved=False, pos="start", scaled=True, dtype="bf16"),
        # a long prompt's q, k, v from one fused projection, at the
        # benchmark's 65,536 x 32 token-heads
        dict(name="rotary_prompt", op="rotary", dir="fwd", B=1, H=32, Hk=32, L=65536, d=128, e=128,
             r=128, interleaved=False, pos="none", scaled=True, dtype="bf16"),
        # training with k and v heads shared by four q heads, odd length,
        # packed documents' positions
        dict(name="rotary_train_bwd", op="rotary", dir="bwd", B=4, H=32, Hk=8, L=4097, d=128, e=64,
             r=96, interleaved=True, pos="table", scaled=False, dtype="bf16"),
        # one token for each of 256 requests x 64 heads
        dict(name="gated_norm_decode", op="gated_norm", dir="fwd", B=256, H=64, L=1, e=128,
             per_head=True, shared=True, activation="silu", dtype="bf16"),
        # the benchmark's B 8 x H 32 x L 8,192 point, one norm over the row
        dict(name="gated_norm_train", op="gated_norm", dir="fwd", B=8, H=32, L=8192, e=128,
             per_head=False, shared=False, activation="sigmoid", dtype="bf16"),
        # training: B 4 x L 2,048 rows and a ragged one, norm per head
        dict(name="gated_norm_train_bwd", op="gated_norm", dir="bwd", B=4, H=32, L=2049, e=128,
             per_head=True, shared=False, activation="silu", dtype="bf16"),
        # a decode step's rows
        dict(name="residual_norm_decode", op="residual_norm", dir="fwd", N=256, D=8192, post=True,
             stream="f32", dtype="bf16"),
        # training rows of 32 heads x 128, residual stream in 16 bits
        dict(name="residual_norm_train", op="residual_norm", dir="fwd", N=65536, D=4096, post=False,
             stream="bf16", dtype="bf16"),
        dict(name="residual_norm_train_bwd", op="residual_norm", dir="bwd", N=16384, D=4096, post=True,
             stream="f32", dtype="bf16"),
        # a small model in 32 bits whose width no vector divides
        dict(name="residual_norm_odd_bwd", op="residual_norm", dir="bwd", N=2999, D=1111, post=False,
             stream="f32", dtype="f32"),
        # beam search at 64 requests x 4 beams, 64 heads: each beam goes on
        # from its parent's state
        dict(name="pool_beams", op="pool_copy", P=272, H=64, d=128, e=128, layers=1, N=256,
             what="beams"),
        # a batch compacted to the pool's front, new requests cleared: small
        # states, several layers in one pool
        dict(name="pool_compact", op="pool_copy", P=96, H=8, d=64, e=64, layers=6, N=37,
             what="compact"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Another case of the ranges that the listed ones stand for."""
    while True:
        op = rng.choice(["rotary", "gated_norm", "residual_norm", "pool_copy"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        direction = rng.choice(["fwd", "bwd"])
        if op in ("rotary", "gated_norm"):
            H = rng.choice([1, 2, 4, 6, 8, 12, 16, 20, 32, 64])
            B = _log_int(rng, 1, 64)
            L = 1 if rng.random() < 0.25 else _log_int(rng, 2, 20000)
            e = rng.choice([64, 128])
        if op == "rotary":
            d = rng.choice([64, 128])
            r = rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)])
            case = dict(op=op, dir=direction, B=B, H=H,
                        Hk=rng.choice([x for x in range(1, H + 1) if H % x == 0]), L=L, d=d, e=e, r=r,
                        interleaved=rng.random() < 0.5, pos=rng.choice(["none", "start", "table"]),
                        scaled=rng.random() < 0.5, dtype=dtype)
        elif op == "gated_norm":
            per_head = rng.random() < 0.5
            case = dict(op=op, dir=direction, B=B, H=H, L=L, e=e, per_head=per_head,
                        shared=per_head and rng.random() < 0.5,
                        activation=rng.choice(["silu", "sigmoid"]), dtype=dtype)
        elif op == "residual_norm":
            D = _log_int(rng, 64, 16384)
            if rng.random() < 0.6:
                D = max(8, D // 8 * 8)
            case = dict(op=op, dir=direction, N=_log_int(rng, 1, 65536), D=D, post=rng.random() < 0.5,
                        stream="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]), dtype=dtype)
        else:
            N = _log_int(rng, 1, 600)
            case = dict(op=op, P=N + _log_int(rng, 1, 400), H=rng.choice([1, 2, 4, 8, 16, 32, 64]),
                        d=rng.choice([64, 128]), e=rng.choice([64, 128]),
                        layers=rng.choice([1, 1, 1, 2, 6]), N=N,
                        what=rng.choice(["beams", "compact", "shuffle"]))
            if case["P"] * case["layers"] * case["H"] * case["d"] * case["e"] * 4 > MOST_BYTES:
                continue
        if work(case)["bytes"] <= MOST_BYTES:
            return case


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(shape, dtype, g, scale=1.0):
    x = torch.empty(shape, dtype=dtype, device=DEV)
    x.normal_(0.0, scale, generator=g)
    return x


def _heads(x, first, n, width):
    """n heads of `width` columns from column `first` of a token-major [B,L,.] buffer, as [B,n,L,width]."""
    B, L, _ = x.shape
    return x[..., first:first + n * width].view(B, L, n, width).transpose(1, 2)


def _frequencies(r, scaled):
    """base^(-2i/r); scaled: the wavelengths a longer context cannot tell
    apart slowed down by a factor of 8, with a ramp between."""
    f = [10000.0 ** (-2.0 * i / r) for i in range(r // 2)]
    if scaled:
        turns = [8192.0 * x / (2.0 * math.pi) for x in f]
        keep = [min(1.0, max(0.0, (t - 1.0) / 31.0)) for t in turns]
        f = [x * (k + (1.0 - k) / 8.0) for x, k in zip(f, keep)]
    return torch.tensor(f, dtype=torch.float64, device=DEV)


def _parents(case, seed):
    """(src, dst) of a pool's moves, int32; every dst once."""
    rng = np.random.default_rng(int(seed) + 77)
    N, P = case["N"], case["P"]
    if case["what"] == "beams":  # groups of four slots, each going on from one of its group's
        slots = rng.permutation(P)[:N]
        group = np.arange(N) // 4 * 4
        src = slots[np.minimum(group + rng.integers(0, 4, N), N - 1)]
        return src.astype(np.int32), slots.astype(np.int32)
    if case["what"] == "compact":  # the live slots to the pool's front, in order; the last fifth cleared
        live = np.sort(rng.permutation(P)[:N])
        src = live.copy()
        src[N - N // 5:] = -1
        return src.astype(np.int32), np.arange(N, dtype=np.int32)
    slots = rng.permutation(P)[:N]  # a cycle through all of them
    return np.roll(slots, 1).astype(np.int32), slots.astype(np.int32)


def prepare(case, seed):
    g = _gen(seed)
    op, s = case["op"], dict(case)
    dt = DT.get(case.get("dtype"))
    if op == "rotary":
        B, H, Hk, L, d, e = (case[n] for n in ("B", "H", "Hk", "L", "d", "e"))
        s["width"] = H * d + Hk * (d + e)
        if case["dir"] == "fwd":
            x = _randn((B, L, s["width"]), dt, g)
            s["q"], s["k"], s["v"] = (_heads(x, 0, H, d), _heads(x, H * d, Hk, d),
                                      _heads(x, (H + Hk) * d, Hk, e))
        else:
            s["dq"], s["dk"], s["dv"] = (_randn((B, H, L, n), dt, g) for n in (d, d, e))
        s["inv_freq"] = _frequencies(case["r"], case["scaled"])
        s["scale"] = 1.0 + 0.1 * math.log(8.0) if case["scaled"] else 1.0
        if case["pos"] == "start":    # tokens so far of each request
            s["positions"] = torch.randint(0, 1 << 20, (B,), generator=g, device=DEV)
        elif case["pos"] == "table":  # documents packed into rows: positions begin again inside a row
            s["positions"] = (torch.arange(L, device=DEV)[None]
                              + torch.randint(0, 1 << 17, (B, 1), generator=g, device=DEV)) % 1777
        else:
            s["positions"] = None
    elif op == "gated_norm":
        B, H, L, e = (case[n] for n in ("B", "H", "L", "e"))
        s["o"] = _randn((B, H, L, e), dt, g, 2.0)
        s["o"][:, :, L // 2] *= 1e-3              # a row early in a text: a small state, small outputs
        if L > 3:
            s["o"][0, :, 3] = 0                   # a padded row
        s["gate"] = _randn((B, L, 2 * H * e), dt, g, 1.5)[..., H * e:]
        s["weight"] = 1.0 + _randn((e if case["shared"] else H * e,), torch.float32, g, 0.2)
        if case["dir"] == "bwd":
            s["du"] = _randn((B, L, H * e), dt, g)
    elif op == "residual_norm":
        N, D, hd = case["N"], case["D"], DT[case["stream"]]
        s["y"] = _randn((N, D), dt, g, 0.5)
        s["alpha"], s["beta"] = 1.0, 0.35
        s["weight"] = 1.0 + _randn((D,), torch.float32, g, 0.2)
        s["post_weight"] = 1.0 + _randn((D,), torch.float32, g, 0.2) if case["post"] else None
        if case["dir"] == "fwd":
            s["h"] = _randn((N, D), hd, g, 3.0)
        else:
            s["h_new"] = _randn((N, D), hd, g, 3.0)
            s["dn"], s["dh_new"] = _randn((N, D), dt, g), _randn((N, D), hd, g)
    else:
        P, H, d, e, layers = (case[n] for n in ("P", "H", "d", "e", "layers"))
        s["pool"] = _randn((layers, P, H, d, e) if layers > 1 else (P, H, d, e), torch.float32, g)
        src, dst = _parents(case, seed)
        s["src"], s["dst"] = torch.from_numpy(src).to(DEV), torch.from_numpy(dst).to(DEV)
    return s


# ------------------------------------------------------------- the plain forms
def _angles(s, B, L, sign):
    t = torch.arange(L, device=DEV)
    p = s["positions"]
    p = t[None] if p is None else (p[:, None] + t if p.dim() == 1 else p)
    # 64 bits: a far position's angle has more digits than 32 bits hold
    a = p.double()[:, None, :, None] * s["inv_freq"]
    return (a.cos() * s["scale"]).float(), (sign * a.sin() * s["scale"]).float()


def _rotate(x, r, cos, sin, interleaved):
    x = x.float()
    a, rest = x[..., :r], x[..., r:]
    if interleaved:
        u, w = a[..., 0::2], a[..., 1::2]
        y = torch.stack((u * cos - w * sin, u * sin + w * cos), -1).flatten(-2)
    else:
        u, w = a[..., :r // 2], a[..., r // 2:]
        y = torch.cat((u * cos - w * sin, u * sin + w * cos), -1)
    return torch.cat((y, rest), -1)


def _repeat(x, times):
    return x if times == 1 else x[:, :, None].expand(-1, -1, times, -1, -1).flatten(1, 2)


def _plain_rotary(s):
    B, H, Hk, L, r = s["B"], s["H"], s["Hk"], s["L"], s["r"]
    dt = DT[s["dtype"]]
    if s["dir"] == "fwd":
        cos, sin = _angles(s, B, L, 1.0)
        q = _rotate(s["q"], r, cos, sin, s["interleaved"]).to(dt)
        k = _rotate(s["k"], r, cos, sin, s["interleaved"]).to(dt)
        return q, _repeat(k, H // Hk).contiguous(), _repeat(s["v"], H // Hk).contiguous()
    cos, sin = _angles(s, B, L, -1.0)
    shared = lambda x: x.float().view(B, Hk, H // Hk, L, -1).sum(2)  # noqa: E731
    gq = _rotate(s["dq"], r, cos, sin, s["interleaved"])
    gk = _rotate(shared(s["dk"]), r, cos, sin, s["interleaved"])
    return torch.cat([x.transpose(1, 2).flatten(2) for x in (gq, gk, shared(s["dv"]))], -1).to(dt)


def _act(gate, kind):
    sig = 1.0 / (1.0 + torch.exp(-gate))
    if kind == "sigmoid":
        return sig, sig * (1.0 - sig)
    return gate * sig, sig * (1.0 + gate * (1.0 - sig))


def _plain_gated_norm(s):
    B, H, L, e = s["B"], s["H"], s["L"], s["e"]
    o = s["o"].float().transpose(1, 2)                                  # [B,L,H,e]
    gate = s["gate"].float().view(B, L, H, e)
    w = s["weight"].expand(H, e) if s["shared"] else s["weight"].view(H, e)
    over = (-1,) if s["per_head"] else (-2, -1)
    rstd = torch.rsqrt((o * o).mean(over, keepdim=True) + 1e-6)
    y = o * rstd
    a, da = _act(gate, s["activation"])
    if s["dir"] == "fwd":
        return (y * w * a).to(s["o"].dtype).flatten(2)
    du = s["du"].float().view(B, L, H, e)
    dgate = du * w * y * da
    dy = du * w * a
    do = rstd * (dy - y * (dy * y).mean(over, keepdim=True))
    dw = (du * a * y).sum((0, 1, 2) if s["shared"] else (0, 1)).flatten()
    dt = s["o"].dtype
    return do.to(dt).transpose(1, 2).contiguous(), dgate.to(dt).flatten(2), dw


def _normed(x):
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    return x * rstd, rstd


def _plain_residual_norm(s):
    y, dt, hd = s["y"].float(), DT[s["dtype"]], DT[s["stream"]]
    if s["dir"] == "fwd":
        p = _normed(y)[0] * s["post_weight"] if s["post"] else y
        h = s["alpha"] * s["h"].float() + s["beta"] * p
        return h.to(hd), (_normed(h)[0] * s["weight"]).to(dt)
    hn, rstd = _normed(s["h_new"].float())
    dn = s["dn"].float()
    dhn = dn * s["weight"]
    dH = s["dh_new"].float() + rstd * (dhn - hn * (dhn * hn).mean(-1, keepdim=True))
    dp = s["beta"] * dH
    out = [(s["alpha"] * dH).to(hd), None, (dn * hn).sum(0)]
    if s["post"]:
        yn, ry = _normed(y)
        dyn = dp * s["post_weight"]
        out[1] = (ry * (dyn - yn * (dyn * yn).mean(-1, keepdim=True))).to(dt)
        out.append((dp * yn).sum(0))
    else:
        out[1] = dp.to(dt)
    return tuple(out)


def _plain_pool_copy(s):
    pool, src, dst = s["pool"], s["src"].long(), s["dst"].long()
    dim = pool.dim() - 4
    taken = pool.index_select(dim, src.clamp(min=0))
    taken.mul_((src >= 0).to(pool.dtype).view(-1, 1, 1, 1))
    pool.index_copy_(dim, dst, taken)
    return pool


def run(s):
    op = s["op"]
    if not own:
        return {"rotary": _plain_rotary, "gated_norm": _plain_gated_norm,
                "residual_norm": _plain_residual_norm, "pool_copy": _plain_pool_copy}[op](s)
    import causal_linear_attention_fwd_b200 as la2
    if op == "rotary":
        how = dict(interleaved=s["interleaved"], scale=s["scale"])
        if s["dir"] == "fwd":
            return la2.rotary(s["q"], s["k"], s["inv_freq"], s["positions"], v=s["v"], **how)
        B, H, Hk, L, d, e = (s[n] for n in ("B", "H", "Hk", "L", "d", "e"))
        x = torch.empty((B, L, s["width"]), dtype=s["dq"].dtype, device=s["dq"].device)
        la2.rotary_backward(s["dq"], s["dk"], s["inv_freq"], s["positions"], dv=s["dv"], kv_heads=Hk,
                            out=(_heads(x, 0, H, d), _heads(x, H * d, Hk, d),
                                 _heads(x, (H + Hk) * d, Hk, e)), **how)
        return x
    if op == "gated_norm":
        how = dict(activation=s["activation"], per_head=s["per_head"], eps=1e-6)
        if s["dir"] == "fwd":
            return la2.gated_norm(s["o"], s["gate"], s["weight"], **how)
        return la2.gated_norm_backward(s["du"], s["o"], s["gate"], s["weight"], **how)
    if op == "residual_norm":
        how = dict(post_norm=s["post"], post_weight=s["post_weight"], alpha=s["alpha"], beta=s["beta"],
                   eps=1e-6)
        if s["dir"] == "fwd":
            return la2.residual_norm(s["h"], s["y"], s["weight"], **how)
        dh, dy, dw, dpw = la2.residual_norm_backward(s["dn"], s["h_new"], s["y"], s["weight"],
                                                     dh_new=s["dh_new"], **how)
        return (dh, dy, dw, dpw) if s["post"] else (dh, dy, dw)
    return la2.pool_copy(s["pool"], s["src"], s["dst"])


# ---------------------------------------------------------------- what it costs
def work(case):
    """Bytes: each input read once, each output written once.  Operations:
    the multiplications and additions of the formulas."""
    op = case["op"]
    es = SIZE.get(case.get("dtype"), 4)
    if op == "rotary":
        B, H, Hk, L, d, e, r = (case[n] for n in ("B", "H", "Hk", "L", "d", "e", "r"))
        few, full = B * L * (H * d + Hk * (d + e)), B * L * H * (2 * d + e)
        table = {"none": 0, "start": 8 * B, "table": 8 * B * L}[case["pos"]]
        ops = 3 * B * L * r * (H + Hk) + (B * L * (d + e) * (H - Hk) if case["dir"] == "bwd" else 0)
        return {"bytes": (few + full) * es + table + 4 * r, "flops": ops}
    if op == "gated_norm":
        n = case["B"] * case["L"] * case["H"] * case["e"]
        w = 4 * (case["e"] if case["shared"] else case["H"] * case["e"])
        if case["dir"] == "fwd":
            return {"bytes": 3 * n * es + w, "flops": 9 * n}
        return {"bytes": 5 * n * es + 2 * w, "flops": 22 * n}
    if op == "residual_norm":
        n, hs = case["N"] * case["D"], SIZE[case["stream"]]
        w = 4 * case["D"] * (2 if case["post"] else 1)
        if case["dir"] == "fwd":
            return {"bytes": n * (2 * es + 2 * hs) + w, "flops": n * (11 if case["post"] else 7)}
        post = 1 if case["post"] else 0
        return {"bytes": n * (2 * es + 3 * hs) + post * n * es + 2 * w, "flops": n * (14 + 11 * post)}
    src, dst = _parents(case, 0)
    moved = src != dst
    row = case["layers"] * case["H"] * case["d"] * case["e"] * 4
    reads = len(set(src[moved & (src >= 0)].tolist()))
    return {"bytes": (reads + int(moved.sum())) * row + 8 * case["N"], "flops": 0}


# --------------------------------------------------------- the definition, 64 bits
def _exact_turn(x, r, phase, interleaved):
    """Pairs as complex numbers, multiplied by the phase."""
    x = x.double().clone()
    first = slice(0, r, 2) if interleaved else slice(0, r // 2)
    second = slice(1, r, 2) if interleaved else slice(r // 2, r)
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * phase
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_rotary(s):
    B, H, Hk, L, r = s["B"], s["H"], s["Hk"], s["L"], s["r"]
    pos = torch.zeros((B, L), dtype=torch.float64, device=DEV)
    if s["positions"] is None or s["positions"].dim() == 1:
        pos += torch.arange(L, dtype=torch.float64, device=DEV)
    if s["positions"] is not None:
        pos += s["positions"].double().reshape(B, -1)
    angle = (pos[..., None] * s["inv_freq"])[:, None]
    back = s["dir"] == "bwd"
    phase = torch.polar(torch.full_like(angle, s["scale"]), -angle if back else angle)
    of_head = torch.arange(H, device=DEV) // (H // Hk)
    if not back:
        return (_exact_turn(s["q"], r, phase, s["interleaved"]),
                _exact_turn(s["k"], r, phase, s["interleaved"])[:, of_head], s["v"].double()[:, of_head])
    gather = lambda x: torch.zeros((B, Hk, *x.shape[2:]), dtype=torch.float64, device=DEV).index_add_(  # noqa: E731
        1, of_head, x.double())
    parts = (_exact_turn(s["dq"], r, phase, s["interleaved"]),
             _exact_turn(gather(s["dk"]), r, phase, s["interleaved"]), gather(s["dv"]))
    return torch.cat([x.permute(0, 2, 1, 3).reshape(B, L, -1) for x in parts], 2)


def _exact_rms(x, dims):
    return (x.pow(2).sum(dims, keepdim=True) / math.prod(x.shape[i] for i in dims) + 1e-6).sqrt()


def _exact_gated_norm(s):
    B, H, L, e = s["B"], s["H"], s["L"], s["e"]
    o = s["o"].double()                                                 # [B,H,L,e]
    z = s["gate"].double().reshape(B, L, H, e).permute(0, 2, 1, 3)
    w = s["weight"].double().reshape(-1, e)[:, None]                    # [H or 1, 1, e]
    dims = (3,) if s["per_head"] else (1, 3)
    rms = _exact_rms(o, dims)
    sig = torch.special.expit(z)
    act, slope = (z * sig, sig + z * sig * (1 - sig)) if s["activation"] == "silu" else (sig, sig - sig * sig)
    token_major = lambda x: x.permute(0, 2, 1, 3).reshape(B, L, H * e)  # noqa: E731
    if s["dir"] == "fwd":
        return token_major(o / rms * w * act)
    up = s["du"].double().reshape(B, L, H, e).permute(0, 2, 1, 3)
    n = math.prod(o.shape[i] for i in dims)
    t = up * w * act
    do = t / rms - o * (t * o).sum(dims, keepdim=True) / (n * rms ** 3)
    dw = (up * act * o / rms).sum((0, 2))                               # [H,e]
    return do, token_major(up * w * o / rms * slope), dw.sum(0) if s["shared"] else dw.reshape(-1)


def _exact_residual_norm(s):
    y, w = s["y"].double(), s["weight"].double()
    pw = s["post_weight"].double() if s["post"] else None
    ry = _exact_rms(y, (1,)) if s["post"] else None
    if s["dir"] == "fwd":
        h = s["h"].double() * s["alpha"] + (y / ry * pw if s["post"] else y) * s["beta"]
        return h, h / _exact_rms(h, (1,)) * w
    D = y.shape[1]
    h, dn = s["h_new"].double(), s["dn"].double()
    rh = _exact_rms(h, (1,))
    t = dn * w
    total = s["dh_new"].double() + t / rh - h * (t * h).sum(1, keepdim=True) / (D * rh ** 3)
    dw, dp = (dn * h / rh).sum(0), total * s["beta"]
    if not s["post"]:
        return total * s["alpha"], dp, dw
    t = dp * pw
    dy = t / ry - y * (t * y).sum(1, keepdim=True) / (D * ry ** 3)
    return total * s["alpha"], dy, dw, (dp * y / ry).sum(0)


def _exact_pool_copy(s):
    pool = s["pool"] if s["pool"].dim() == 5 else s["pool"][None]
    new = pool.double()
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        new[:, b] = pool[:, a].double() if a >= 0 else 0.0
    return new if s["pool"].dim() == 5 else new[0]


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "gated_norm": _exact_gated_norm,
            "residual_norm": _exact_residual_norm, "pool_copy": _exact_pool_copy}[case["op"]](s)
