"""The gated linear recurrence (ms_gated_scan_fwd / _bwd, ms_gated_step)
against its fp64 definition.

Bounds: the library's own (helpers.bound: fp32 1e-4 (1 + |ref|), bf16 2 ulp +
1e-3) for y and the state.  A decay of up to 0.999 remembers about 1000 steps,
and each step's decay carries at most one rounding of exp2 (2^-23): 1.2e-4 of
the state's size in the worst case, a few 1e-6 as they fall.  Gradients:
lm_reference.grad_bound."""
import numpy as np
import pytest
import torch

import lm_reference as ref
from helpers import assert_within

pytestmark = pytest.mark.gpu
DEV = "cuda"
IO = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(b, L, d, io, gate, start, reset, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    keep = 0.9 + 0.099 * torch.rand(d, generator=g, device=DEV)
    s = {k: n(b, L, d).to(IO[io]) for k in ("x", "r", "i", "dy")}
    s["lam"] = torch.log(torch.expm1(-torch.log(keep) / 8.0))
    s["z"] = n(b, L, d).to(IO[io]) if gate else None
    s["h0"] = n(b, d) if start else None
    s["dh_last"] = n(b, d) if start else None
    s["reset"] = (torch.rand(b, L, generator=g, device=DEV) < 0.02).to(torch.uint8) \
        if reset else None
    return s


# b, L, d: one step, block edges of 16 / 64 / 128, several blocks; channel
# counts of whole vectors, of none (below four), and with a tail
SHAPES = [(1, 1, 1), (3, 1, 64), (2, 31, 3), (1, 32, 32), (2, 33, 33), (1, 127, 5), (2, 129, 100),
          (1, 255, 64), (3, 256, 7), (1, 257, 36), (2, 1000, 66), (1, 2500, 2), (70, 5, 40)]
KINDS = [(False, False, False), (True, True, False), (True, False, True), (False, True, True)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward_and_backward(gpu, shape, io):
    b, L, d = shape
    for k, (gate, start, reset) in enumerate(KINDS):
        s = inputs(b, L, d, io, gate, start, reset, seed=100 + k)
        hl = torch.full((b, d), float("nan"), device=DEV)
        states = gpu.gated_scan_states(s["x"])
        y = gpu.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], s["z"], reset=s["reset"],
                               h0=s["h0"], h_last=hl, states=states)
        yr, hs, hr = ref.gated_forward(s["x"], s["r"], s["i"], s["lam"], s["z"], s["h0"],
                                       s["reset"])
        assert_within(y, yr.numpy(), io, f"y {gate, start, reset}")
        assert_within(hl, hr.numpy(), "f32", f"h_last {gate, start, reset}")
        first = torch.zeros(b, 1, d, dtype=torch.float64) if s["h0"] is None else \
            s["h0"].cpu().double().unsqueeze(1)
        before = torch.cat([first, hs[:, :-1]], 1)[:, ::16]
        assert_within(states, before.numpy(), "f32", "states")
        got = gpu.gated_scan_bwd(s["x"], s["r"], s["i"], s["lam"], s["dy"], states, s["z"],
                                 reset=s["reset"], dh_last=s["dh_last"])
        want = ref.gated_backward(s["x"], s["r"], s["i"], s["lam"], s["dy"], s["z"], s["h0"],
                                  s["dh_last"], s["reset"])
        assert (got["dz"] is None) == (s["z"] is None)
        for name, w in want.items():
            o = io if name in ("dx", "dr", "di", "dz") else "f32"
            ref.assert_close(got[name], w.numpy(), ref.grad_bound(w.numpy(), o),
                             f"{name} {gate, start, reset}")


def test_gradient_against_differences(gpu):
    """Central differences of the fp64 forward along a random direction of
    every input.  Step 1e-6: truncation about 1e-12, rounding about 1e-9 of a
    loss of order 10; the GPU's fp32 gradient adds 1e-6 of the sum of
    |gradient| |direction|."""
    s = inputs(2, 150, 12, "f32", True, True, True, seed=7)
    names = ("x", "r", "i", "lam", "z", "h0")
    states = gpu.gated_scan_states(s["x"])
    gpu.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], s["z"], reset=s["reset"], h0=s["h0"],
                       states=states)
    got = gpu.gated_scan_bwd(s["x"], s["r"], s["i"], s["lam"], s["dy"], states, s["z"],
                             reset=s["reset"], dh_last=s["dh_last"])
    v64 = {k: s[k].cpu().double() for k in names}

    def loss(v):
        y, _, hl = ref.gated_forward(v["x"], v["r"], v["i"], v["lam"], v["z"], v["h0"], s["reset"])
        return float((y * s["dy"].cpu().double()).sum() + (hl * s["dh_last"].cpu().double()).sum())

    rng = torch.Generator().manual_seed(3)
    for k in names:
        v = torch.randn(v64[k].shape, generator=rng, dtype=torch.float64)
        e = 1e-6
        diff = (loss({**v64, k: v64[k] + e * v}) - loss({**v64, k: v64[k] - e * v})) / (2 * e)
        g = got["d" + k].cpu().double()
        lim = 1e-5 * float((g.abs() * v.abs()).sum()) + 1e-6
        assert abs(float((g * v).sum()) - diff) <= lim, (k, float((g * v).sum()), diff)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_steps_equal_the_scan(gpu, io):
    s = inputs(3, 70, 50, io, True, True, False, seed=11)
    hl = s["h0"].clone()
    y = gpu.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], s["z"], h0=hl, h_last=hl)  # aliased
    yr, _, hr = ref.gated_forward(s["x"], s["r"], s["i"], s["lam"], s["z"], s["h0"])
    h = s["h0"].clone()
    for t in range(70):
        yt = gpu.gated_step(h, *(s[k][:, t].contiguous() for k in ("x", "r", "i")), s["lam"],
                            s["z"][:, t].contiguous())
        assert_within(yt, yr[:, t].numpy(), io, f"y_t {t}")
    assert_within(h, hr.numpy(), "f32", "h")
    assert_within(hl, hr.numpy(), "f32", "h_last over h0")
    assert_within(y, yr.numpy(), io, "y")


def test_pieces_equal_the_whole(gpu):
    s = inputs(2, 600, 70, "f32", False, True, True, seed=12)
    yr, _, hr = ref.gated_forward(s["x"], s["r"], s["i"], s["lam"], None, s["h0"], s["reset"])
    h, parts = s["h0"].clone(), []
    for t0, t1 in ((0, 1), (1, 300), (300, 600)):
        p = {k: s[k][:, t0:t1].contiguous() for k in ("x", "r", "i", "reset")}
        hn = torch.empty_like(h)
        parts.append(gpu.gated_scan_fwd(p["x"], p["r"], p["i"], s["lam"], reset=p["reset"], h0=h,
                                        h_last=hn))
        h = hn
    assert_within(torch.cat(parts, 1), yr.numpy(), "f32", "y")
    assert_within(h, hr.numpy(), "f32", "h_last")


@pytest.mark.parametrize("d", [40, 37])
def test_extreme_gates(gpu, d):
    """Gates far out (decay exactly 0 and 1), rates far out, zero inputs:
    results stay those of the definition, and gradients finite."""
    s = inputs(2, 90, d, "f32", True, True, False, seed=13)
    s["r"][:, 5] = 200.0
    s["r"][:, 9] = -200.0
    s["r"][0, 20:30] = -90.0
    s["i"][:, 7] = -150.0
    s["i"][:, 8] = 150.0
    s["lam"][0], s["lam"][1], s["lam"][2], s["lam"][3] = -80.0, -30.0, 60.0, -120.0
    s["x"][1] = 0.0
    hl, states = torch.empty(2, d, device=DEV), gpu.gated_scan_states(s["x"])
    y = gpu.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], s["z"], h0=s["h0"], h_last=hl,
                           states=states)
    yr, _, hr = ref.gated_forward(s["x"], s["r"], s["i"], s["lam"], s["z"], s["h0"])
    assert_within(y, yr.numpy(), "f32")
    assert_within(hl, hr.numpy(), "f32")
    got = gpu.gated_scan_bwd(s["x"], s["r"], s["i"], s["lam"], s["dy"], states, s["z"],
                             dh_last=s["dh_last"])
    want = ref.gated_backward(s["x"], s["r"], s["i"], s["lam"], s["dy"], s["z"], s["h0"],
                              s["dh_last"])
    for name, w in want.items():
        assert torch.isfinite(got[name]).all(), name
        ref.assert_close(got[name], w.numpy(), ref.grad_bound(w.numpy(), "f32"), name)


def test_nan_and_infinity_stay_where_they_belong(gpu):
    """A NaN reaches its own channel from its step on, and not past a reset."""
    s = inputs(2, 400, 44, "f32", False, True, False, seed=14)
    s["reset"] = torch.zeros(2, 400, dtype=torch.uint8, device=DEV)
    s["reset"][:, 300] = 1
    s["reset"][1, 50] = 1
    s["x"][0, 100, 3] = float("nan")
    s["x"][0, 130, 9] = float("inf")
    s["h0"][1, 5] = float("nan")
    hl, states = torch.empty(2, 44, device=DEV), gpu.gated_scan_states(s["x"])
    y = gpu.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], reset=s["reset"], h0=s["h0"],
                           h_last=hl, states=states)
    yr, _, hr = ref.gated_forward(s["x"], s["r"], s["i"], s["lam"], None, s["h0"], s["reset"])
    assert torch.isnan(y[0, 100:300, 3]).all() and torch.isfinite(y[0, 300:, 3]).all()
    assert torch.isinf(y[0, 130:300, 9]).all() and torch.isfinite(y[0, 300:, 9]).all()
    assert torch.isnan(y[1, :50, 5]).all() and torch.isfinite(y[1, 50:, 5]).all()
    rest = torch.isfinite(yr)
    assert (torch.isfinite(y).cpu() == rest).all()
    assert_within(torch.where(rest.to(DEV), y, torch.zeros_like(y)),
                  torch.where(rest, yr, torch.zeros_like(yr)).numpy(), "f32")
    assert_within(hl, hr.numpy(), "f32")
    # backward: no gradient crosses the reset either
    s["dy"][0, 350, 7] = float("nan")
    g = gpu.gated_scan_bwd(s["x"], s["r"], s["i"], s["lam"], s["dy"], states, reset=s["reset"])
    assert torch.isnan(g["dx"][0, 300:351, 7]).all()
    assert torch.isfinite(g["dx"][0, :300, 7]).all() and torch.isfinite(g["dx"][0, 351:, 7]).all()
    assert torch.isfinite(g["dr"][0, 300:, 3]).all() and torch.isfinite(g["dx"][0, :, 3]).all()


def test_repeats_bit_for_bit_also_on_another_stream(gpu):
    s = inputs(2, 3000, 72, "bf16", True, True, True, seed=15)

    def call(stream=None):
        hl, st = torch.empty(2, 72, device=DEV), gpu.gated_scan_states(s["x"])
        y = gpu.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], s["z"], reset=s["reset"],
                               h0=s["h0"], h_last=hl, states=st, stream=stream)
        g = gpu.gated_scan_bwd(s["x"], s["r"], s["i"], s["lam"], s["dy"], st, s["z"],
                               reset=s["reset"], dh_last=s["dh_last"], stream=stream)
        return [y, hl] + [g[k] for k in sorted(g)]

    first = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        again = call(stream)
        torch.cuda.synchronize()
        for p, q in zip(first, again):
            assert torch.equal(p, q)


def test_side_by_side_on_streams(gpu):
    """Scans of many blocks on several streams at once, each with a workspace of
    its own, beside matrix products that take the rest of the chip: every block's
    wait for earlier ones ends, and the bits are those of a scan alone."""
    sets = [inputs(*shape, "bf16", True, False, True, seed=40 + k)
            for k, shape in enumerate(((1, 20000, 64), (4, 5000, 320), (2, 9000, 100)))]
    a = torch.randn(4096, 4096, device=DEV, dtype=torch.bfloat16)

    def run(s):
        states = gpu.gated_scan_states(s["x"])
        y = gpu.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], s["z"], reset=s["reset"],
                               states=states)
        g = gpu.gated_scan_bwd(s["x"], s["r"], s["i"], s["lam"], s["dy"], states, s["z"],
                               reset=s["reset"])
        return [y] + [g[k] for k in sorted(g)]

    alone = [run(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(len(sets) + 1)]
    for _ in range(5):
        got = []
        with torch.cuda.stream(streams[-1]):
            for _ in range(4):
                a @ a
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                got.append(run(s))
        torch.cuda.synchronize()
        for one, other in zip(alone, got):
            for u, v in zip(one, other):
                assert torch.equal(u, v)


def test_in_a_graph(gpu):
    s = inputs(1, 5000, 40, "bf16", True, True, True, seed=16)
    io = gpu.MS_BF16
    y, hl, st = torch.empty_like(s["x"]), torch.empty(1, 40, device=DEV), \
        gpu.gated_scan_states(s["x"])
    wf = torch.empty(max(1, gpu.gated_scan_workspace_bytes(1, 5000, 40, io)), dtype=torch.uint8,
                     device=DEV)
    wb = torch.empty(gpu.gated_scan_bwd_workspace_bytes(1, 5000, 40, io), dtype=torch.uint8,
                     device=DEV)

    def call():
        gpu.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], s["z"], reset=s["reset"], h0=s["h0"],
                           y=y, h_last=hl, states=st, workspace=wf)
        return gpu.gated_scan_bwd(s["x"], s["r"], s["i"], s["lam"], s["dy"], st, s["z"],
                                  reset=s["reset"], dh_last=s["dh_last"], workspace=wb)

    want = {k: v.clone() for k, v in call().items()}
    yw, hw = y.clone(), hl.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for rep in range(3):
        for t in (y, hl, st, *out.values()):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, yw) and torch.equal(hl, hw), rep
        for k in want:
            assert torch.equal(out[k], want[k]), (rep, k)
        call()
        torch.cuda.synchronize()


def test_autograd(gpu):
    s = inputs(2, 80, 24, "f32", True, True, False, seed=17)
    t = {k: s[k].clone().requires_grad_() for k in ("x", "r", "i", "lam", "z", "h0")}
    y, hl = gpu.gated_scan(t["x"], t["r"], t["i"], t["lam"], t["z"], t["h0"], return_last=True)
    ((y * s["dy"]).sum() + (hl * s["dh_last"]).sum()).backward()
    want = ref.gated_backward(s["x"], s["r"], s["i"], s["lam"], s["dy"], s["z"], s["h0"],
                              s["dh_last"])
    for k in t:
        w = want["d" + k].numpy()
        ref.assert_close(t[k].grad, w, ref.grad_bound(w, "f32"), k)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,off,ld", [(64, 0, 320), (36, 3, 155), (33, 1, 140), (2, 1, 11), (8, 8, 41)])
def test_slices_of_a_wider_tensor(gpu, io, d, off, ld):
    """x, r, i and z as columns of one projection, at offsets of any alignment:
    the same bits as from contiguous copies."""
    s = inputs(3, 150, d, io, True, True, True, seed=d)
    wide = torch.full((3, 150, ld), float("nan"), device=DEV).to(IO[io])
    for k, name in enumerate(("x", "r", "i", "z")):
        wide[:, :, off + k * d:off + (k + 1) * d] = s[name]
    v = [wide[:, :, off + k * d:off + (k + 1) * d] for k in range(4)]
    c = [s[k] for k in ("x", "r", "i", "z")]
    out = []
    for x, r, i, z in (c, v):
        states, hl = gpu.gated_scan_states(x), torch.empty(3, d, device=DEV)
        y = gpu.gated_scan_fwd(x, r, i, s["lam"], z, reset=s["reset"], h0=s["h0"], h_last=hl,
                               states=states)
        g = gpu.gated_scan_bwd(x, r, i, s["lam"], s["dy"], states, z, reset=s["reset"],
                               dh_last=s["dh_last"])
        h = s["h0"].clone()
        yt = gpu.gated_step(h, x[:, 7], r[:, 7], i[:, 7], s["lam"], z[:, 7]) \
            if x is v[0] else gpu.gated_step(h, *(t[:, 7].contiguous() for t in (x, r, i)),
                                             s["lam"], z[:, 7].contiguous())
        out.append([y, hl, states, h, yt] + [g[k] for k in sorted(g)])
    for a, b in zip(*out):
        assert torch.equal(a, b)
    # one pitch for all
    with pytest.raises(ValueError, match="contiguous"):
        gpu.gated_scan_fwd(v[0], c[1], v[2], s["lam"])
    # gradients reach the wider tensor
    leaf = wide.nan_to_num().requires_grad_()
    x, r, i, z = (leaf[:, :, off + k * d:off + (k + 1) * d] for k in range(4))
    gpu.gated_scan(x, r, i, s["lam"], z, s["h0"], reset=s["reset"]).backward(s["dy"])
    g = gpu.gated_scan_bwd(*c[:3], s["lam"], s["dy"], out[0][2], c[3], reset=s["reset"])
    for k, name in enumerate(("dx", "dr", "di", "dz")):
        assert torch.equal(leaf.grad[:, :, off + k * d:off + (k + 1) * d], g[name])


def test_refusals(gpu):
    s = inputs(2, 10, 8, "f32", False, False, False)
    x, r, i, lam = s["x"], s["r"], s["i"], s["lam"]
    with pytest.raises(TypeError):
        gpu.gated_scan_fwd(x.half(), r, i, lam)
    with pytest.raises(TypeError):
        gpu.gated_scan_fwd(x, r.bfloat16(), i, lam)
    with pytest.raises(ValueError, match="shape"):
        gpu.gated_scan_fwd(x, r[:, :9].contiguous(), i, lam)
    with pytest.raises(ValueError, match="contiguous"):
        gpu.gated_scan_fwd(x.transpose(0, 1).contiguous().transpose(0, 1), r, i, lam)
    with pytest.raises(ValueError, match="device"):
        gpu.gated_scan_fwd(x.cpu(), r, i, lam)
    with pytest.raises(ValueError, match="states"):
        gpu.gated_scan_bwd(x, r, i, lam, s["dy"], None)
    for c in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(gpu.MsError, match="sharpness"):
            gpu.gated_scan_fwd(x, r, i, lam, c=c)
    with pytest.raises(gpu.MsError, match="seqlen"):
        gpu.gated_scan_fwd(x[:, :0], r[:, :0], i[:, :0], lam)
    with pytest.raises(gpu.MsError, match="16-byte"):
        flat = torch.zeros(2 * 10 * 8 + 1, device=DEV)[1:].view(2, 10, 8)
        gpu.gated_scan_fwd(flat, r, i, lam)
    with pytest.raises(gpu.MsError, match="workspace"):
        gpu.gated_scan_bwd(x, r, i, lam, s["dy"], gpu.gated_scan_states(x),
                           workspace=torch.empty(1, dtype=torch.uint8, device=DEV))
    np.testing.assert_equal(gpu.gated_scan_states(x).shape, (2, 1, 8))


def test_calls_on_two_streams_in_turn(gpu):
    """A call on another stream takes no memory that the current stream has
    freed (its queue may still use it): calls in turn, with nothing between them,
    give the bits of calls alone."""
    side = torch.cuda.Stream()
    s = inputs(2, 6000, 136, "bf16", True, False, True, seed=18)
    t = inputs(2, 6000, 136, "bf16", True, False, True, seed=19)

    def run(v, stream=None):
        states = gpu.gated_scan_states(v["x"], stream=stream)
        y = gpu.gated_scan_fwd(v["x"], v["r"], v["i"], v["lam"], v["z"], reset=v["reset"],
                               states=states, stream=stream)
        g = gpu.gated_scan_bwd(v["x"], v["r"], v["i"], v["lam"], v["dy"], states, v["z"],
                               reset=v["reset"], stream=stream)
        return [y] + [g[k] for k in sorted(g) if g[k] is not None]

    want = run(s), run(t)
    torch.cuda.synchronize()
    n = gpu.gated_scan_bwd_workspace_bytes(2, 6000, 136, gpu.MS_BF16)
    m = gpu.lm._marshal()
    for stream in (side, side.cuda_stream):
        freed = torch.empty(n, dtype=torch.uint8, device=DEV)
        at = freed.data_ptr()
        del freed
        call = gpu.lm._Call(m, s["x"], stream)
        assert call.workspace(None, n)[0].data_ptr() != at
        assert call.empty(torch.uint8, n).data_ptr() != at
        assert call.together(torch.uint8, (n,))[0].data_ptr() != at
    for _ in range(8):
        got = [(run(s), run(t, side)) for _ in range(3)]
        torch.cuda.synchronize()
        for one in got:
            for a, b in zip(want, one):
                assert all(torch.equal(p, q) for p, q in zip(a, b))


def same_with_nan(p, q):
    n, m = torch.isnan(p), torch.isnan(q)
    return torch.equal(n, m) and torch.equal(p.masked_fill(n, 0), q.masked_fill(m, 0))


@pytest.mark.parametrize("d", [44, 45, 3])
def test_fast_decays_are_no_resets(gpu, d):
    """Decays of 0.06: their product over a block is 0, which cuts nothing off.
    Resets that are all zero give what no resets give, and what is not finite
    stays so up to a reset, also beside a decay that is NaN itself."""
    L = 700
    s = inputs(2, L, d, "f32", False, True, False, seed=20)
    s["lam"][::2], s["lam"][1], s["lam"][d - 1] = 0.0, 0.0, 0.0
    s["r"] *= 0.1
    nan, inf = float("nan"), float("inf")
    s["x"][0, 100, 0], s["x"][1, 130, 0] = nan, inf
    s["h0"][1, 1] = nan
    s["r"][0, 298, 1] = nan
    s["dy"][0, 650, d - 1], s["dh_last"][1, d - 1] = nan, inf
    zeros = torch.zeros(2, L, dtype=torch.uint8, device=DEV)

    def run(reset):
        hl, states = torch.empty(2, d, device=DEV), gpu.gated_scan_states(s["x"])
        y = gpu.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], reset=reset, h0=s["h0"],
                               h_last=hl, states=states)
        g = gpu.gated_scan_bwd(s["x"], s["r"], s["i"], s["lam"], s["dy"], states, reset=reset,
                               dh_last=s["dh_last"])
        return {"y": y, "h_last": hl, "states": states, **{k: g[k] for k in g if g[k] is not None}}

    none, zero = run(None), run(zeros)
    for k in none:
        assert same_with_nan(none[k], zero[k]), k
    y, hl, dx = zero["y"], zero["h_last"], zero["dx"]
    assert torch.isnan(y[0, 100:, 0]).all() and torch.isnan(hl[0, 0])
    assert not torch.isfinite(y[1, 130:, 0]).any() and not torch.isfinite(hl[1, 0])
    assert torch.isnan(y[1, :, 1]).all() and torch.isnan(y[0, 298:, 1]).all()
    assert torch.isnan(dx[0, :651, d - 1]).all() and torch.isfinite(dx[0, 651:, d - 1]).all()
    assert not torch.isfinite(dx[1, :, d - 1]).any()
    # the same with resets at 300 and, in the second row, at 60
    cut = zeros.clone()
    cut[:, 300], cut[1, 60] = 1, 7
    got = run(cut)
    yr, _, hr = ref.gated_forward(s["x"], s["r"], s["i"], s["lam"], None, s["h0"], cut)
    rest = torch.isfinite(yr)
    assert rest[:, 300:].all() and (torch.isfinite(got["y"]).cpu() == rest).all()
    assert_within(torch.where(rest.to(DEV), got["y"], torch.zeros_like(y)),
                  torch.where(rest, yr, torch.zeros_like(yr)).numpy(), "f32")
    assert_within(got["h_last"], hr.numpy(), "f32")
    dx = got["dx"]
    assert torch.isnan(dx[0, 300:651, d - 1]).all() and not torch.isfinite(dx[1, 300:, d - 1]).any()
    assert torch.isfinite(dx[:, :300, d - 1]).all() and torch.isfinite(dx[0, 651:, d - 1]).all()
    assert torch.isfinite(got["dh0"][:, d - 1]).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gradients_off_16_bytes(gpu, io):
    """Gradients as torch.cat hands them on, resets and rates inside a larger
    buffer: contiguous, aligned to their element."""
    s = inputs(3, 41, 37, io, True, True, True, seed=21)
    off = {}
    for k in ("dy", "dh_last", "reset", "lam"):
        off[k] = torch.cat([s[k].flatten()[:1], s[k].flatten()])[1:].view(s[k].shape)
        assert off[k].data_ptr() % 16
    leaves = [{k: s[k].clone().requires_grad_() for k in ("x", "r", "i", "lam", "z", "h0")}
              for _ in range(2)]
    for t, v in zip(leaves, (s, off)):
        # t["lam"] itself is aligned; the raw calls below take the one that is not
        y, hl = gpu.gated_scan(t["x"], t["r"], t["i"], t["lam"], t["z"], t["h0"],
                               reset=v["reset"], return_last=True)
        if v is off:
            pad = lambda u: torch.cat([u.new_zeros(1), u.flatten()])  # noqa: E731
            ((pad(y) * pad(s["dy"])).sum() + (pad(hl) * pad(s["dh_last"])).sum()).backward()
        else:
            torch.autograd.backward([y, hl], [s["dy"], s["dh_last"]])
    for k in leaves[0]:
        assert torch.equal(leaves[0][k].grad, leaves[1][k].grad), k
    out = []
    for v in (s, off):
        states = gpu.gated_scan_states(s["x"])
        y = gpu.gated_scan_fwd(s["x"], s["r"], s["i"], v["lam"], s["z"], reset=v["reset"],
                               h0=s["h0"], states=states)
        g = gpu.gated_scan_bwd(s["x"], s["r"], s["i"], v["lam"], v["dy"], states, s["z"],
                               reset=v["reset"], dh_last=v["dh_last"])
        h = s["h0"].clone()
        yt = gpu.gated_step(h, *(s[k][:, 3].contiguous() for k in ("x", "r", "i")), v["lam"])
        out.append([y, h, yt] + [g[k] for k in sorted(g)])
    for a, b in zip(*out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,off", [(36, 3), (33, 1), (64, 0), (2, 1), (10, 0)])
def test_slices_of_one_row(gpu, io, d, off):
    """One row has no distance to the next, and is still a slice of a wider one."""
    s = inputs(1, 1, d, io, True, True, False, seed=d)
    wide = torch.zeros(1, 1, 4 * d + off + 5, device=DEV).to(IO[io])
    v = [wide[..., off + k * d:off + (k + 1) * d] for k in range(4)]
    for a, name in zip(v, ("x", "r", "i", "z")):
        a.copy_(s[name])
    out = []
    for x, r, i, z in ([s[k] for k in ("x", "r", "i", "z")], v):
        h, states, hl = s["h0"].clone(), gpu.gated_scan_states(x), torch.empty(1, d, device=DEV)
        y = gpu.gated_scan_fwd(x, r, i, s["lam"], z, h0=s["h0"], h_last=hl, states=states)
        g = gpu.gated_scan_bwd(x, r, i, s["lam"], s["dy"], states, z, dh_last=s["dh_last"])
        yt = gpu.gated_step(h, x[0], r[0], i[0], s["lam"], z[0])
        assert_within(yt, y[0].double().cpu().numpy(), io)
        assert_within(h, hl.double().cpu().numpy(), "f32")
        out.append([y, hl, states, h, yt] + [g[k] for k in sorted(g)])
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_autograd_takes_slices_of_the_resets(gpu):
    s = inputs(3, 50, 24, "f32", False, False, True, seed=22)
    wide = torch.cat([s["reset"], torch.ones_like(s["reset"][:, :3])], 1)
    a, b = (gpu.gated_scan(s["x"], s["r"], s["i"], s["lam"], reset=v)
            for v in (wide[:, :50], wide.bool()[:, :50].contiguous()))
    assert torch.equal(a, b)


def second_order(outputs, inputs):
    """First-order gradients that have a graph; differentiating them raises."""
    loss = sum((o * o).sum() for o in outputs)
    grads = torch.autograd.grad(loss, inputs, create_graph=True)
    plain = torch.autograd.grad(sum((o * o).sum() for o in outputs), inputs, retain_graph=True)
    for a, b in zip(grads, plain):
        assert torch.equal(a.detach(), b)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        sum((g * g).sum() for g in grads).backward()


def test_second_derivatives_are_refused(gpu):
    """A gradient penalty would silently lose what goes through these."""
    s = inputs(2, 30, 16, "f32", True, True, False, seed=23)
    t = [s[k].clone().requires_grad_() for k in ("x", "r", "i", "lam", "z", "h0")]
    second_order(gpu.gated_scan(*t, return_last=True), t)
    w = torch.randn(20, 16, device=DEV, requires_grad=True)
    second_order([gpu.embed(torch.arange(5, device=DEV), w)], [w])
    x = torch.randn(4, 30, device=DEV, requires_grad=True)
    second_order(gpu.token_logprobs(x, torch.arange(4, device=DEV))[:2], [x])


def test_default_stream_by_its_handle(gpu):
    s = inputs(2, 3000, 72, "bf16", True, False, False, seed=24)
    want = gpu.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], s["z"])
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        assert gpu.lm._Call(gpu.lm._marshal(), s["x"], 0).other == torch.cuda.default_stream()
        got = gpu.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], s["z"], stream=0)
    torch.cuda.synchronize()
    assert torch.equal(want, got)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_autograd_off_16_bytes(gpu, io):
    """The differentiable operations take what begins at its element's alignment."""
    def off(t):
        return torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)

    s = inputs(2, 40, 33, io, True, True, False, seed=25)
    names = ("x", "r", "i", "lam", "z", "h0")
    grads = []
    for f in (lambda t: t.clone(), off):
        t = [f(s[k]).requires_grad_() for k in names]
        assert f is not off or all(v.data_ptr() % 16 for v in t)
        torch.autograd.backward(gpu.gated_scan(*t, return_last=True), [s["dy"], s["dh_last"]])
        w = f(s["x"][0]).requires_grad_()
        gpu.embed(torch.arange(9, device=DEV), w).backward(s["dy"][0, :9])
        v = f(s["x"][1]).requires_grad_()
        lp, ent = gpu.token_logprobs(v, torch.arange(40, device=DEV) % 33)[:2]
        torch.autograd.backward([lp, ent], [s["h0"].flatten()[:40], s["h0"].flatten()[20:60]])
        grads.append([k.grad for k in (*t, w, v)])
    for a, b in zip(*grads):
        assert torch.equal(a, b)
