"""The group norm where a wave or a workgroup goes down several rows: more rows
than 2048 workgroups (1280 in the backward of groups wider than a wave) take one
each.  Definition and bounds are those of test_group_norm_gpu."""
import pytest
import torch

from test_group_norm_gpu import DEV, compare, definition, inputs

pytestmark = pytest.mark.gpu

# rows, groups, size: groups of a workgroup with 1, 2, 4 and 8 vectors a lane, one to
# three rows of a workgroup, with columns beside each other; a wave's with 1 and 2
# vectors, some lanes or all of them; rows that do not fill the last pass
WIDE = [(4100, 1, 1536), (300, 16, 1100), (2600, 1, 2049), (2500, 1, 4500), (1400, 2, 530)]
NARROW = [(9000, 1, 64), (9001, 3, 73), (8500, 1, 1000), (20000, 1, 8), (17000, 1, 300)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", WIDE + NARROW, ids=lambda s: "x".join(map(str, s)))
def test_many_rows(gpu, shape, io):
    rows, groups, size = shape
    for k, (gate, first, center) in enumerate(
            [(False, False, False), (True, False, False), (True, True, False), (True, True, True),
             (False, False, True)]):
        s = inputs(rows, groups, size, io, gate, True, k % 2 == 0, seed=20 + k, shift=0.5 * center)
        kw = {"center": center, "gate_first": first, "eps": 1e-3}
        args = groups, s["weight"], s["bias"]
        y = gpu.group_norm_fwd(s["x"], *args, s["z"], **kw)
        d = gpu.group_norm_bwd(s["x"], s["dy"], *args, s["z"], **kw)
        want = definition(s, groups, center, first, 1e-3)
        compare(y, want["y"], size, rows, io, "y")
        for n, x in d.items():
            if x is not None:
                compare(x, want[n], size, rows, io, n)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(6000, 1, 1536), (2100, 2, 2600)], ids=lambda s: "x".join(map(str, s)))
def test_a_row_is_the_same_among_others(gpu, shape, io):
    """A row's result does not depend on which rows a workgroup takes with it:
    rows of quite different sizes, whose sums must not meet, many times over."""
    rows, groups, size = shape
    s = inputs(rows, groups, size, io, True, True, True, seed=31)
    s["x"] *= torch.logspace(-3, 3, 7, device=DEV)[torch.arange(rows, device=DEV) % 7, None].to(
        s["x"].dtype)
    for center in (False, True):
        kw = {"center": center, "eps": 1e-6}
        args = groups, s["weight"], s["bias"]
        alone = [{n: s[n][i:i + 1000].contiguous() for n in ("x", "z", "dy")}
                 for i in range(0, rows, 1000)]
        want = torch.cat([gpu.group_norm_fwd(p["x"], *args, p["z"], **kw) for p in alone])
        grads = [gpu.group_norm_bwd(p["x"], p["dy"], *args, p["z"], **kw) for p in alone]
        first = gpu.group_norm_bwd(s["x"], s["dy"], *args, s["z"], **kw)
        for _ in range(10):
            assert torch.equal(gpu.group_norm_fwd(s["x"], *args, s["z"], **kw), want)
            d = gpu.group_norm_bwd(s["x"], s["dy"], *args, s["z"], **kw)
            for n in ("dx", "dz"):
                assert torch.equal(d[n], torch.cat([g[n] for g in grads])), n
            for n in ("dweight", "dbias"):
                assert torch.equal(d[n], first[n]), n
