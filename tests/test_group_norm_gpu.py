"""The group norm of each row's channels (ms_group_norm_fwd / _bwd) against its
fp64 definition.

Bounds.  u = 2^-24.  A sum over a group's n channels adds at most n u relative
to the sum of absolute values (trees and 4 or 8 values a lane: far less); the
gate has a handful of roundings (exp2, its argument up to 2^7, a reciprocal):
150 u.  So with c = (2 n + 300) u, a result is off by at most c times the same
expression over absolute values, where a mean is taken off plus what the
values' own size loses in that.  bf16 results add their rounding, 2^-8."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
U24, U8 = 2.0 ** -24, 2.0 ** -8


def inputs(rows, groups, size, io, gate, weight, bias, seed=0, shift=0.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    c = groups * size
    return {"x": (2 * n(rows, c) + shift).to(IO[io]), "z": n(rows, c).to(IO[io]) if gate else None,
            "weight": 1 + 0.3 * n(c) if weight else None, "bias": n(c) if bias else None,
            "dy": n(rows, c).to(IO[io])}


def definition(s, groups, center, gate_first, eps):
    """{result: (value, size of what it is made of)}"""
    x, dy = s["x"].double(), s["dy"].double()
    rows, c = x.shape
    view = lambda t: t.reshape(-1, groups, c // groups)  # noqa: E731
    x, dy = view(x), view(dy)
    w = view(s["weight"].double()) if s["weight"] is not None else torch.ones_like(x[:1])
    b = view(s["bias"].double()) if s["bias"] is not None else torch.zeros_like(x[:1])
    z = view(s["z"].double()) if s["z"] is not None else None
    gate = z * z.sigmoid() if z is not None else torch.ones_like(x)
    slope = z.sigmoid() * (1 + z * (1 - z.sigmoid())) if z is not None else None
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    first = gate_first and z is not None
    u = x * gate if first else x
    cc = u - mean(u) if center else u
    f = (mean(cc * cc) + eps).rsqrt()
    hat = cc * f
    # absolute sizes: of u's own rounding against what is left beside its mean
    ahat = (u.abs() + (mean(u.abs()) if center else 0)) * f
    out = {}
    pre, apre = hat * w + b, ahat * w.abs() + b.abs()
    post = torch.ones_like(x) if first else gate
    out["y"] = pre * post, apre * post.abs()
    d = dy * post
    out["dweight"] = (d * hat).sum(0), (d.abs() * ahat).sum(0)
    out["dbias"] = d.sum(0), d.abs().sum(0)
    e = d * w
    ae = e.abs()
    du = f * (e - hat * mean(e * hat) - (mean(e) if center else 0))
    adu = f * (ae + ahat * mean(ae * ahat) + (mean(ae) if center else 0))
    # the factor itself is as uncertain as the mean square of ahat against hat's
    adu = adu * mean(ahat * ahat).clamp_min(1.0)
    out["y"] = out["y"][0], out["y"][1] * mean(ahat * ahat).clamp_min(1.0)
    if z is not None:
        if first:
            out["dz"] = du * x * slope, adu * x.abs() * (1 + z.abs())
        else:
            out["dz"] = dy * pre * slope, dy.abs() * apre * (1 + z.abs())
    out["dx"] = du * (gate if first else 1), adu * (gate.abs() if first else 1)
    return {k: (v.flatten(-2).squeeze(0) if k[:2] in ("dw", "db") else v.reshape(rows, c),
                a.flatten(-2).squeeze(0) if k[:2] in ("dw", "db") else a.reshape(rows, c))
            for k, (v, a) in out.items()}


def compare(got, want, size, rows, io, name):
    value, big = want
    c = (2 * size + 300 + (rows if name in ("dweight", "dbias") else 0)) * U24
    if name in ("dweight", "dbias"):
        io = "f32"
    lim = 2 * c * big + (U8 * value.abs() if io == "bf16" else 0) + 1e-30
    err = (got.double() - value).abs()
    bad = ~(err <= lim)
    assert not bad.any(), (name, int(bad.sum()), float((err / lim).max()))


# rows, groups, size: one value, part of a vector, lanes 1 to 64, 2 to 4 vectors a
# lane, a workgroup, the largest; groups that do not fill a wave's lanes
SHAPES = [(1, 1, 1), (3, 5, 3), (70, 24, 64), (5, 7, 73), (33, 3, 128), (9, 2, 250), (4, 1, 512),
          (6, 1, 1000), (17, 1, 1536), (2, 2, 2049), (3, 1, 5000), (2, 1, 8192), (4500, 1, 8),
          (1, 64, 16)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward_and_backward(gpu, shape, io):
    rows, groups, size = shape
    for k, (gate, first, center, weight, bias) in enumerate(
            [(False, False, True, True, True), (True, False, False, True, False),
             (True, True, True, True, True), (True, True, False, False, False),
             (True, False, True, False, True)]):
        s = inputs(rows, groups, size, io, gate, weight, bias, seed=k, shift=0.5 * center)
        kw = {"center": center, "gate_first": first, "eps": 1e-3}
        y = gpu.group_norm_fwd(s["x"], groups, s["weight"], s["bias"], s["z"], **kw)
        d = gpu.group_norm_bwd(s["x"], s["dy"], groups, s["weight"], s["bias"], s["z"], **kw)
        want = definition(s, groups, center, first, 1e-3)
        compare(y, want["y"], size, rows, io, "y")
        for n in ("dx", "dz", "dweight", "dbias"):
            given = {"dx": True, "dz": gate, "dweight": weight, "dbias": bias}[n]
            assert (d[n] is not None) == given
            if given:
                compare(d[n], want[n], size, rows, io, n)


def test_gradient_against_differences(gpu):
    """Central differences in fp64, step 1e-6 (truncation 1e-10, rounding 1e-9)."""
    s = inputs(5, 3, 20, "f32", True, True, True, seed=5)
    for center, first in ((True, False), (False, True), (True, True)):
        d = gpu.group_norm_bwd(s["x"], s["dy"], 3, s["weight"], s["bias"], s["z"], center=center,
                               gate_first=first)

        def loss(t):
            return float((definition(t, 3, center, first, 1e-5)["y"][0] * s["dy"].double()).sum())

        for n in ("x", "z", "weight", "bias"):
            g = torch.Generator(device=DEV)
            g.manual_seed(3)
            x = s[n].double()
            w = torch.randn(x.shape, generator=g, device=DEV, dtype=torch.float64)
            diff = (loss(dict(s, **{n: x + 1e-6 * w})) - loss(dict(s, **{n: x - 1e-6 * w}))) / 2e-6
            grad = d["d" + n].double()
            lim = 1e-5 * float((grad * w).abs().sum()) + 1e-6
            assert abs(float((grad * w).sum()) - diff) <= lim, (n, center, first)


def test_rows_by_themselves(gpu):
    """Constant and zero rows, and a row that is not finite, which stays alone."""
    s = inputs(6, 2, 40, "f32", False, True, True, seed=6)
    s["x"][0] = 0
    s["x"][1] = 3.0
    s["x"][3, 50] = math.nan
    y = gpu.group_norm_fwd(s["x"], 2, s["weight"], s["bias"])
    assert torch.equal(y[0], s["bias"])
    # a mean of equal values is them to 2^-24 n, over the root of eps
    assert ((y[1] - s["bias"]).abs() <= 3.0 * 80 * U24 / 1e-5 ** 0.5 * s["weight"].abs()).all()
    assert torch.isnan(y[3, 40:]).all() and torch.isfinite(y[3, :40]).all()
    assert torch.isfinite(y[[0, 1, 2, 4, 5]]).all()
    empty = gpu.group_norm_fwd(s["x"][:0], 2, s["weight"], s["bias"])
    assert empty.shape == (0, 80)
    d = gpu.group_norm_bwd(s["x"][:0], s["dy"][:0], 2, s["weight"], s["bias"])
    assert (d["dweight"] == 0).all() and (d["dbias"] == 0).all()


def test_slices_shapes_streams_graphs(gpu):
    s = inputs(60, 4, 24, "bf16", True, True, True, seed=7)
    wide = torch.zeros(60, 2 * 96 + 5, dtype=torch.bfloat16, device=DEV)
    wide[:, 3:99], wide[:, 99:195] = s["x"], s["z"]
    x, z = wide[:, 3:99], wide[:, 99:195]
    args = (4, s["weight"], s["bias"])
    y = gpu.group_norm_fwd(s["x"], *args, s["z"])
    assert torch.equal(y, gpu.group_norm_fwd(x, *args, z))
    d = gpu.group_norm_bwd(s["x"], s["dy"], *args, s["z"])
    d2 = gpu.group_norm_bwd(x.unflatten(0, (3, 20)), s["dy"].unflatten(0, (3, 20)), *args,
                            z.unflatten(0, (3, 20)))
    for n in d:
        assert torch.equal(d[n].flatten(), d2[n].flatten()), n
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    d3 = gpu.group_norm_bwd(x, s["dy"], *args, z, stream=side)
    side.synchronize()
    for n in d:
        assert torch.equal(d[n], d3[n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg = gpu.group_norm_bwd(x, s["dy"], *args, z)
    for _ in range(3):
        wide.copy_(torch.randn(wide.shape, device=DEV))
        graph.replay()
        w = gpu.group_norm_bwd(x, s["dy"], *args, z)
        torch.cuda.synchronize()
        for n in w:
            assert torch.equal(dg[n], w[n]), n


def test_autograd(gpu):
    s = inputs(30, 3, 20, "f32", True, True, True, seed=8)
    leaves = {n: s[n].clone().requires_grad_() for n in ("x", "weight", "bias", "z")}
    y = gpu.group_norm(leaves["x"].t().contiguous().t(), 3, leaves["weight"], leaves["bias"],
                       leaves["z"], center=False)
    y.backward(s["dy"].t().contiguous().t())
    d = gpu.group_norm_bwd(s["x"], s["dy"], 3, s["weight"], s["bias"], s["z"], center=False)
    for n, x in leaves.items():
        assert torch.equal(x.grad, d["d" + n]), n
    x = s["x"].clone().requires_grad_()
    gpu.group_norm(x, 3).sum().backward()
    assert x.grad.shape == x.shape


def test_gradients_of_absent_weights(gpu):
    """The C ABI gives dweight and dbias also where weight and bias are 1 and 0
    by their absence."""
    s = inputs(50, 3, 40, "f32", True, False, False, seed=9)
    out = [torch.full((50, 120), float("nan"), device=DEV) for _ in range(2)]
    dw, db = (torch.full((120,), float("nan"), device=DEV) for _ in range(2))
    n = gpu.group_norm_bwd_workspace_bytes(50, 3, 40, 0)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    rc = gpu.load().ms_group_norm_bwd(
        s["x"].data_ptr(), 120, None, None, s["z"].data_ptr(), 120, 1, 0, 1e-3, s["dy"].data_ptr(),
        out[0].data_ptr(), out[1].data_ptr(), dw.data_ptr(), db.data_ptr(), 50, 3, 40, 0,
        ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    want = definition(s, 3, True, False, 1e-3)
    for name, got in (("dx", out[0]), ("dz", out[1]), ("dweight", dw), ("dbias", db)):
        compare(got, want[name], 40, 50, "f32", name)


def test_refusals(gpu):
    s = inputs(6, 2, 40, "bf16", True, True, True)
    x, z, w = s["x"], s["z"], s["weight"]
    f = gpu.group_norm_fwd
    for bad in (lambda: f(x, 3, w), lambda: f(x, 0), lambda: f(x.cpu(), 2), lambda: f(x.t(), 2),
                lambda: f(x, 2, w[:40]), lambda: f(x, 2, w, None, z[:5]),
                lambda: f(x, 2, w, None, z.t().contiguous().t()),
                lambda: f(x[:, :1].expand(6, 80), 2)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for bad in (lambda: f(x, 2, w.double()), lambda: f(x, 2, w, None, z.float()),
                lambda: f(x.half(), 2)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: f(x, 2, w, eps=0.0), lambda: f(x, 2, w, eps=math.nan),
                lambda: f(x, 2, w, gate_first=True),
                lambda: f(torch.zeros(1, 8193, device=DEV), 1),
                lambda: gpu.group_norm_bwd(x, s["dy"], 2, w,
                                           workspace=torch.zeros(8, device=DEV))):
        with pytest.raises(gpu.MsError):
            bad()
