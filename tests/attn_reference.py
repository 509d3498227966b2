"""fp64 definitions of the linear attention, one token after another, with the
sums of absolute values that bounds are made of.

Bounds.  Let u = 2^-24 and U = 2^-8, the half steps of fp32 and bf16.  Every
result is a sum of products; `big` is the same sum over absolute values of all
its terms (the recurrences run on |q|, |k|, |v|, |dO|, |h0|, |dh_last|).  fp32
sums, decays (two roundings of exp2 and of its argument each) and products add
at most one u of `big` for each term or step on the way: a sum over dk or dv
(up to 128), over a block (up to 64), one update a block, a dozen for decays:
c = (dk + dv + 200 + 4 blocks) u.  With bf16 io, one operand of each product
that ends in a bf16 result is rounded to bf16, U of `big`, and the result
itself, U of it:
    bf16 results   U |r| + (U + c) big
    fp32 results   c big
The decays' gradient is taken from sums over a block's tokens, whose terms
cancel: there `big` is that sum over the whole block."""
import torch

U24, U8 = 2.0 ** -24, 2.0 ** -8


def expand(s):
    """q, k (heads of their own), v, keep [b, L, H] and the starts, in fp64."""
    H = s["v"].shape[2]
    r = H // s["k"].shape[2]
    q, k = (s[n].double().repeat_interleave(r, 2) for n in ("q", "k"))
    b, L = q.shape[:2]
    g = s["g"].double().expand(b, L, H)
    cut = torch.zeros(b, L, dtype=torch.bool, device=q.device) if s.get("reset") is None else \
        s["reset"] != 0
    cut = cut.unsqueeze(-1) | (g < -104.0)
    return q, k, s["v"].double(), g.exp(), cut


def forward(s, scale):
    """o [b, L, H, dv], the states after each token [L] and the first one."""
    q, k, v, keep, cut = expand(s)
    b, L, H, dk = q.shape
    S = torch.zeros(b, H, dk, v.shape[-1], dtype=torch.float64, device=q.device) \
        if s.get("h0") is None else s["h0"].double()
    first, states, o = S, [], torch.empty_like(v)
    for t in range(L):
        kept = torch.where(cut[:, t, :, None, None], 0.0, keep[:, t, :, None, None] * S)
        S = kept + k[:, t, :, :, None] * v[:, t, :, None, :]
        states.append(S)
        o[:, t] = scale * (q[:, t, :, :, None] * S).sum(-2)
    return o, states, first


def backward(s, scale, states, first, do, dh_last=None):
    """dict of the gradients, those of q and k for each head of v, and dg for
    each token."""
    q, k, v, keep, cut = expand(s)
    L = q.shape[1]
    do = do.double()
    d = {n: torch.empty_like(x) for n, x in (("dq", q), ("dk", k), ("dv", v), ("dg", keep))}
    R = torch.zeros_like(first) if dh_last is None else dh_last.double()
    for t in range(L - 1, -1, -1):
        R = R + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        d["dq"][:, t] = scale * (states[t] * do[:, t, :, None, :]).sum(-1)
        d["dk"][:, t] = (R * v[:, t, :, None, :]).sum(-1)
        d["dv"][:, t] = (R * k[:, t, :, :, None]).sum(-2)
        before = states[t - 1] if t else first
        live = torch.where(cut[:, t, :, None, None], 0.0, keep[:, t, :, None, None] * R)
        d["dg"][:, t] = torch.where(cut[:, t, :, None, None], 0.0, live * before).sum((-1, -2))
        R = live
    d["dh0"] = R
    return d


def absolute(s):
    return {n: x.abs() if n in ("q", "k", "v", "h0") and x is not None else x
            for n, x in s.items()}


def const(s, io):
    block = 64 if io == "bf16" else 32
    blocks = -(-s["q"].shape[1] // block)
    return (s["k"].shape[-1] + s["v"].shape[-1] + 200 + 4 * blocks) * U24


def bound(ref, big, c, io):
    return c * big + (U8 * (ref.abs() + big) if io == "bf16" else 0.0) + 1e-30


def per_block(x, io):
    """Sums over the blocks of tokens (dim 1), for every token of them."""
    n = 64 if io == "bf16" else 32
    L = x.shape[1]
    y = torch.nn.functional.pad(x, (0, 0, 0, -L % n)).unflatten(1, (-1, n)).sum(2, keepdim=True)
    return y.expand(-1, -1, n, -1).flatten(1, 2)[:, :L]


def shared(x, kheads):
    return x.unflatten(2, (kheads, -1)).sum(3)


def check(got, want, lim, what):
    err = (got.double() - want).abs()
    bad = ~(err <= lim)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                             f"{float((err / lim).nan_to_num(nan=1e30).max()):.3g} bounds; first at {i}: "
                             f"got {float(got[i])} want {float(want[i])}")


def check_forward(s, scale, io, o, h_last):
    ref, states, first = forward(s, scale)
    c = const(s, io)
    big, bigs, _ = forward(absolute(s), abs(scale))
    check(o, ref, bound(ref, big, c, io), "o")
    if h_last is not None:
        check(h_last, states[-1], bound(states[-1], bigs[-1], c, "f32"), "h_last")
    return states, first, bigs


def check_backward(s, scale, io, states, first, bigs, do, dh_last, got):
    a = absolute(s)
    hk = s["k"].shape[2]
    big0 = torch.zeros_like(first) if s.get("h0") is None else a["h0"].double()
    want = backward(s, scale, states, first, do, dh_last)
    big = backward(a, abs(scale), bigs, big0, do.abs(), None if dh_last is None else dh_last.abs())
    c = const(s, io)
    for n in ("dq", "dk"):
        check(got[n], shared(want[n], hk), bound(shared(want[n], hk), shared(big[n], hk), 2 * c, io), n)
    check(got["dv"], want["dv"], bound(want["dv"], big["dv"], 2 * c, io), "dv")
    q, k, *_ = expand(a)
    tokens = per_block((q * big["dq"]).sum(-1) + (k * big["dk"]).sum(-1), io) + big["dg"]
    if s["g"].dim() == 1:
        check(got["dg"], want["dg"].sum((0, 1)), 3 * c * tokens.sum((0, 1)) + 1e-30, "dg")
    else:
        check(got["dg"], want["dg"], 3 * c * tokens + 1e-30, "dg")
    if got.get("dh0") is not None:
        check(got["dh0"], want["dh0"], bound(want["dh0"], big["dh0"], 2 * c, "f32"), "dh0")
