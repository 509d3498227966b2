"""Linear attention (ms_linear_attn_fwd / _bwd / _step) against its fp64
definition; bounds in attn_reference."""
import math

import pytest
import torch

import attn_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
IO = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(b, L, H, Hk, dk, dv, io, start=False, reset=False, fixed=False, seed=0, rate=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    s = {"q": n(b, L, Hk, dk).to(IO[io]), "k": n(b, L, Hk, dk).to(IO[io]),
         "v": n(b, L, H, dv).to(IO[io])}
    s["g"] = -rate * torch.exp(n(H) if fixed else n(b, L, H)) * 0.1
    s["h0"] = n(b, H, dk, dv) if start else None
    s["reset"] = (torch.rand(b, L, generator=g, device=DEV) < 0.05).to(torch.uint8) \
        if reset else None
    do = n(b, L, H, dv).to(IO[io])
    dh = n(b, H, dk, dv) if start else None
    return s, do, dh


def both(gpu, s, do, dh, scale=0.3, **kw):
    b, L, H, dv = s["v"].shape
    h_last = torch.full((b, H, s["k"].shape[3], dv), float("nan"), device=DEV)
    states = gpu.linear_attn_states(s["k"], s["v"])
    o = gpu.linear_attn_fwd(s["q"], s["k"], s["v"], s["g"], scale=scale, reset=s["reset"],
                            h0=s["h0"], h_last=h_last, states=states, **kw)
    d = gpu.linear_attn_bwd(s["q"], s["k"], s["v"], s["g"], do, states, scale=scale,
                            reset=s["reset"], dh_last=dh, **kw)
    return o, h_last, d


# b, L, heads, kheads, dk, dv: one token, edges of blocks of 32 and 64 and of tiles of
# 16 and 64 channels, several blocks, enough of them for segments
SHAPES = [(1, 1, 1, 1, 1, 1), (3, 1, 4, 2, 64, 64), (2, 5, 2, 1, 3, 7), (1, 31, 1, 1, 17, 16),
          (1, 64, 2, 2, 64, 64), (2, 65, 4, 2, 40, 72), (1, 129, 3, 3, 128, 128),
          (3, 97, 6, 3, 65, 66), (1, 700, 2, 1, 16, 100), (2, 520, 3, 1, 100, 20),
          (1, 1100, 1, 1, 128, 65)]
KINDS = [(False, False, False), (True, True, False), (True, False, True), (False, True, True)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward_and_backward(gpu, shape, io):
    for k, (start, reset, fixed) in enumerate(KINDS):
        s, do, dh = inputs(*shape, io, start, reset, fixed, seed=10 + k)
        o, h_last, d = both(gpu, s, do, dh)
        states, first, bigs = ref.check_forward(s, 0.3, io, o, h_last)
        ref.check_backward(s, 0.3, io, states, first, bigs, do, dh, d)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_decays(gpu, io):
    """Decays that differ by many orders, none at all, growth, and ones that
    are 0 (which drop the state)."""
    s, do, dh = inputs(2, 150, 3, 1, 24, 40, io, start=True, seed=3)
    g = s["g"]
    g[:, ::7] = -60.0
    g[:, 3::11] = 0.0
    g[:, 5::13] = 0.05
    g[0, 70] = -math.inf
    g[1, 64] = -500.0
    o, h_last, d = both(gpu, s, do, dh)
    states, first, bigs = ref.check_forward(s, 0.3, io, o, h_last)
    ref.check_backward(s, 0.3, io, states, first, bigs, do, dh, d)
    assert (d["dg"][0, 70] == 0).all() and (d["dg"][1, 64] == 0).all()
    # a decay of 0 is a reset
    t = dict(s, g=g.clone(), reset=torch.zeros(2, 150, dtype=torch.uint8, device=DEV))
    t["g"][0, 70] = t["g"][1, 64] = -1.0
    t["reset"][0, 70] = t["reset"][1, 64] = 1
    o2, h2, d2 = both(gpu, t, do, dh)
    assert torch.equal(o, o2) and torch.equal(h_last, h2)
    for n in d:
        assert torch.equal(d[n], d2[n]), n


def test_gradient_against_differences(gpu):
    """Central differences of the fp64 forward along a random direction of each
    input: truncation 1e-10 relative at step 1e-5, rounding 1e-10; the kernels'
    bound is c of the sum of |gradient| |direction|, for which its square root
    many random terms leave far more room than 1e-4."""
    s, do, dh = inputs(2, 100, 4, 2, 12, 20, "f32", True, True, False, seed=7)
    _, _, d = both(gpu, s, do, dh)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)

    def loss(t):
        o, states, _ = ref.forward(t, 0.3)
        return float((o * do.double()).sum() + (states[-1] * dh.double()).sum())

    for n in ("q", "k", "v", "g", "h0"):
        x = s[n].double()
        w = torch.randn(x.shape, generator=gen, device=DEV, dtype=torch.float64)
        eps = 1e-5
        diff = (loss(dict(s, **{n: x + eps * w})) - loss(dict(s, **{n: x - eps * w}))) / (2 * eps)
        grad = d["d" + n].double()
        lim = 1e-5 * float((grad * w).abs().sum()) + 1e-6
        assert abs(float((grad * w).sum()) - diff) <= lim, n


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["k", "v"])
def test_what_is_not_finite_stays_behind(gpu, io, where):
    """Tokens that are NaN or infinite reach nothing ahead of them and nothing
    behind a reset: all else is as the definition has it."""
    s, do, dh = inputs(2, 200, 2, 1, 20, 36, io, start=True, seed=4)
    s["reset"] = torch.zeros(2, 200, dtype=torch.uint8, device=DEV)
    s["reset"][0, 50] = s["reset"][0, 130] = s["reset"][1, 128] = 1
    s[where][0, 40, 0, 3] = math.nan
    s[where][1, 100, 0, 5] = math.inf
    s["h0"][1, 1, 2, 2] = math.nan
    o, h_last, d = both(gpu, s, do, dh)
    want, states, first = ref.forward(s, 0.3)
    clean = dict(s, **{where: s[where].nan_to_num(0, 0, 0)}, h0=s["h0"].nan_to_num(0))
    big, bigs, _ = ref.forward(ref.absolute(clean), 0.3)
    c = ref.const(s, io)
    fine = torch.isfinite(want)
    assert torch.isfinite(o[fine]).all() and not torch.isfinite(o[~fine]).any()
    ref.check(torch.where(fine, o.double(), 0.0), torch.where(fine, want, 0.0),
              ref.bound(torch.where(fine, want, 0.0), big, c, io), "o")
    assert torch.isfinite(h_last).all()  # both rows end behind a reset
    ref.check(h_last, states[-1], ref.bound(states[-1], bigs[-1], c, "f32"), "h_last")
    w = ref.backward(s, 0.3, states, first, do, dh)
    a = ref.absolute(clean)
    bd = ref.backward(a, 0.3, bigs, a["h0"].double(), do.abs(), dh.abs())
    for n in ("dq", "dk"):
        w[n], bd[n] = ref.shared(w[n], 1), ref.shared(bd[n], 1)
    for n in ("dq", "dk", "dv", "dg"):
        fine = torch.isfinite(w[n])
        assert torch.isfinite(d[n][fine]).all(), n
        if n != "dg":
            ref.check(torch.where(fine, d[n].double(), 0.0), torch.where(fine, w[n], 0.0),
                      ref.bound(torch.where(fine, w[n], 0.0), bd[n], 2 * c, io), n)


@pytest.mark.parametrize("where", ["q", "do"])
def test_queries_that_are_not_finite(gpu, where):
    """A query or gradient that is not finite reaches its own output and what is
    ahead of it in its document only."""
    s, do, dh = inputs(1, 200, 2, 2, 20, 36, "bf16", seed=5)
    s["reset"] = torch.zeros(1, 200, dtype=torch.uint8, device=DEV)
    s["reset"][0, 90] = 1
    (s["q"] if where == "q" else do)[0, 120, 1, 3] = math.nan
    o, h_last, d = both(gpu, s, do, None)
    want, states, first = ref.forward(s, 0.3)
    w = ref.backward(s, 0.3, states, first, do)
    w["o"], d["o"] = want, o
    for n in ("o", "dq", "dk", "dv", "dg"):
        assert torch.equal(torch.isfinite(w[n]), torch.isfinite(d[n])), n


def test_slices_and_pieces(gpu):
    """Columns of one wider tensor are read in place; a sequence in two pieces,
    the state over the first's, is the whole's."""
    b, L, H, Hk, dk, dv = 2, 150, 4, 2, 24, 40
    s, do, _ = inputs(b, L, H, Hk, dk, dv, "bf16", seed=8)
    wide = torch.randn(b, L, 2 * Hk * dk + H * dv + 3, device=DEV).to(torch.bfloat16)
    at = 0
    t = dict(s)
    for n, x in (("q", Hk * dk), ("k", Hk * dk), ("v", H * dv)):
        wide[..., at:at + x] = s[n].flatten(2)
        t[n] = wide[..., at:at + x].unflatten(-1, s[n].shape[2:])
        at += x
    o, h, d = both(gpu, s, do, None)
    o2, h2, d2 = both(gpu, t, do, None)
    assert torch.equal(o, o2) and torch.equal(h, h2)
    for n in d:
        assert torch.equal(d[n], d2[n]), n
    state = torch.zeros(b, H, dk, dv, device=DEV)
    part = lambda x, i, j: x[:, i:j].contiguous()  # noqa: E731
    for i, j in ((0, 64), (64, 150)):
        gpu.linear_attn_fwd(*(part(s[n], i, j) for n in ("q", "k", "v", "g")), scale=0.3, h0=state,
                            h_last=state)
    assert torch.equal(state, h)  # whole blocks: the same steps


def test_the_same_again_and_on_another_stream(gpu):
    s, do, dh = inputs(2, 300, 6, 2, 64, 64, "bf16", True, True, seed=9)
    o, h, d = both(gpu, s, do, dh)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, h2, d2 = both(gpu, s, do, dh, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(h, h2)
    for n in d:
        assert torch.equal(d[n], d2[n]), n


def test_captured(gpu):
    """Forward and backward in a graph, replayed on other inputs among eager
    work."""
    s, do, dh = inputs(1, 600, 3, 1, 40, 64, "bf16", True, True, seed=11)
    s2, do2, dh2 = inputs(1, 600, 3, 1, 40, 64, "bf16", True, True, seed=12)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both(gpu, s, do, dh)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, h, d = both(gpu, s, do, dh)
    for k in range(4):
        src, dsrc, hsrc = (s2, do2, dh2) if k % 2 else inputs(1, 600, 3, 1, 40, 64, "bf16", True,
                                                               True, seed=20 + k)
        for n in ("q", "k", "v", "g", "h0", "reset"):
            s[n].copy_(src[n])
        do.copy_(dsrc)
        dh.copy_(hsrc)
        graph.replay()
        wo, wh, wd = both(gpu, src, dsrc, hsrc)
        torch.cuda.synchronize()
        assert torch.equal(o, wo) and torch.equal(h, wh)
        for n in d:
            assert torch.equal(d[n], wd[n]), n


def test_two_calls_at_once(gpu):
    """Calls on two streams side by side, each with a workspace of its own."""
    a, da, ha = inputs(1, 3000, 2, 1, 64, 64, "bf16", True, True, seed=13)
    b, db, hb = inputs(1, 2500, 2, 2, 100, 40, "f32", True, False, seed=14)
    want = both(gpu, a, da, ha), both(gpu, b, db, hb)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got = [both(gpu, *args, stream=s) for args, s in zip(((a, da, ha), (b, db, hb)), streams)]
        torch.cuda.synchronize()
        for (o, h, d), (wo, wh, wd) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(h, wh)
            for n in d:
                assert torch.equal(d[n], wd[n]), n


# ---- steps ---------------------------------------------------------------------------------

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1, 1), (3, 1, 4, 1, 64, 64), (2, 5, 2, 2, 33, 70),
                                   (2, 16, 3, 1, 128, 128), (1, 37, 2, 1, 100, 6),
                                   (1, 64, 1, 1, 17, 127)], ids=lambda s: "x".join(map(str, s)))
def test_step(gpu, shape, io):
    """Bounds: the state is updated token by token, two roundings each."""
    for fixed in (False, True):
        s, _, _ = inputs(*shape, io, True, False, fixed, seed=30)
        if not fixed and shape[1] > 4:
            s["g"][0, 3] = -math.inf
        h = s["h0"].clone()
        o = gpu.linear_attn_step(h, s["q"], s["k"], s["v"], s["g"], scale=0.3)
        ref.check_forward(s, 0.3, io, o, h)
        kept = s["h0"].clone()
        o2 = gpu.linear_attn_step(kept, s["q"], s["k"], s["v"], s["g"], scale=0.3, update=False)
        assert torch.equal(o, o2) and torch.equal(kept, s["h0"])
        assert gpu.linear_attn_step(kept, None, s["k"], s["v"], s["g"]) is None
        assert torch.equal(kept, h)


def test_step_counts(gpu):
    b, T = 7, 6
    s, _, _ = inputs(b, T, 4, 2, 20, 36, "bf16", True, seed=31)
    counts = torch.tensor([0, 1, 2, 6, 5, -3, 99], dtype=torch.int32, device=DEV)
    h, o = s["h0"].clone(), torch.full((b, T, 4, 36), 7.0, dtype=torch.bfloat16, device=DEV)
    gpu.linear_attn_step(h, s["q"], s["k"], s["v"], s["g"], scale=0.3, counts=counts, o=o)
    for i, n in enumerate([0, 1, 2, 6, 5, 0, 6]):
        row = {k: x[i:i + 1, :n].contiguous() if k in "qkvg" else x for k, x in s.items()}
        assert (o[i, n:] == 7.0).all()
        hi = s["h0"][i:i + 1].clone()
        if n:
            oi = gpu.linear_attn_step(hi, row["q"], row["k"], row["v"], row["g"], scale=0.3)
            assert torch.equal(o[i:i + 1, :n], oi)
        assert torch.equal(h[i:i + 1], hi)


def test_step_captured(gpu):
    s, _, _ = inputs(4, 1, 4, 1, 64, 64, "bf16", True, seed=32)
    h = s["h0"].clone()
    gpu.linear_attn_step(h, s["q"], s["k"], s["v"], s["g"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = gpu.linear_attn_step(h, s["q"], s["k"], s["v"], s["g"])
    h.copy_(s["h0"])
    want = s["h0"].clone()
    for _ in range(3):
        graph.replay()
        w = gpu.linear_attn_step(want, s["q"], s["k"], s["v"], s["g"])
        torch.cuda.synchronize()
        assert torch.equal(h, want) and torch.equal(o, w)


# ---- as an operation -------------------------------------------------------------------------

def test_autograd(gpu):
    s, do, dh = inputs(2, 70, 4, 2, 16, 24, "f32", True, True, seed=40)
    leaves = {n: s[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "h0")}
    # transposed and broadcast arguments are copied
    k = leaves["k"].transpose(1, 2).contiguous().transpose(1, 2)
    o, h = gpu.linear_attn(leaves["q"], k, leaves["v"], leaves["g"], leaves["h0"], scale=0.3,
                           reset=s["reset"], return_last=True)
    ((o * do).sum() + (h * dh).sum()).backward()
    _, _, d = both(gpu, s, do, dh)
    for n, x in leaves.items():
        assert torch.equal(x.grad, d["d" + n]), n
    fixed = torch.full((4,), -0.2, device=DEV, requires_grad=True)
    gpu.linear_attn(s["q"], s["k"], s["v"], fixed, scale=0.3).sum().backward()
    wide = torch.full((2, 70, 4), -0.2, device=DEV, requires_grad=True)
    gpu.linear_attn(s["q"], s["k"], s["v"], wide, scale=0.3).sum().backward()
    torch.testing.assert_close(fixed.grad, wide.grad.sum((0, 1)), rtol=1e-4, atol=1e-3)
    with pytest.raises(RuntimeError):
        o = gpu.linear_attn(s["q"], s["k"], s["v"], wide)
        g, = torch.autograd.grad(o.sum(), wide, create_graph=True)
        torch.autograd.grad(g.sum(), wide)


def test_refusals(gpu):
    s, do, dh = inputs(2, 40, 4, 2, 16, 24, "bf16", seed=41)
    q, k, v, g = (s[n] for n in "qkvg")
    fwd = gpu.linear_attn_fwd
    for bad in ((q.float(), k, v, g), (q, k.float(), v, g), (q, k, v, g.double())):
        with pytest.raises(TypeError):
            fwd(*bad)
    for bad in ((q[:, 1:], k, v, g), (q, k, v[:, 1:], g), (q, k, v, g[:, 1:].contiguous()),
                (q.cpu(), k, v, g), (q, k, v.expand(2, 40, 4, 24)[:1].expand(2, 40, 4, 24), g),
                (q, k, v.transpose(1, 2), g), (q, k, v, g.transpose(1, 2)), (q, None, v, g),
                (None, k, v, g)):
        with pytest.raises((ValueError, TypeError)):
            fwd(*bad)
    with pytest.raises(gpu.MsError):
        fwd(q, k, v[:, :, :3].contiguous(), g[:, :, :3].contiguous())  # 2 does not divide 3
    with pytest.raises(gpu.MsError):
        fwd(q, k, v, g, scale=math.inf)
    with pytest.raises((ValueError, TypeError)):
        fwd(q, k, v, g, h0=torch.zeros(2, 4, 16, 23, device=DEV))
    with pytest.raises((ValueError, TypeError)):
        gpu.linear_attn_bwd(q, k, v, g, do, torch.zeros(5, device=DEV))
    h = torch.zeros(2, 4, 16, 24, device=DEV)
    with pytest.raises(gpu.MsError):
        gpu.linear_attn_step(h, None, k, v, g, update=False)
    long = inputs(1, 65, 1, 1, 4, 4, "f32")[0]
    with pytest.raises(gpu.MsError):
        gpu.linear_attn_step(torch.zeros(1, 1, 4, 4, device=DEV), long["q"], long["k"], long["v"],
                             long["g"])
    wide = inputs(1, 2, 1, 1, 129, 4, "f32")[0]
    with pytest.raises(gpu.MsError):
        fwd(wide["q"], wide["k"], wide["v"], wide["g"])
