"""Documents packed into one sequence (resets): nothing of one reaches another's
results, not by a rounding, and not where a log decay is no number."""
import math

import pytest
import torch

import attn_reference as ref
from test_linear_attn_gpu import both, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def packed(io, starts, L=700, heads=4, kheads=2, dk=40, dv=72, seed=0):
    """Inputs of one sequence whose documents start at `starts` (and at 0)."""
    s, do, _ = inputs(1, L, heads, kheads, dk, dv, io, seed=seed)
    s["reset"] = torch.zeros(1, L, dtype=torch.uint8, device=DEV)
    s["reset"][0, starts] = 1
    return s, do


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, 3e38], ids=["nan", "inf", "3e38"])
def test_decays_that_are_no_numbers(gpu, io, bad):
    """A log decay that is NaN, infinite or past all exponents makes nothing of
    the documents ahead of it and behind it other than it is: the same bits as
    with a decay in its place."""
    starts = [10, 23, 24, 100, 130, 300]
    s, do = packed(io, starts, seed=1)
    want = both(gpu, s, do, None)
    t = dict(s, g=s["g"].clone())
    t["g"][0, 5, 1] = t["g"][0, 110, 0] = t["g"][0, 250] = bad
    t["g"][0, 24, 2] = bad  # that of a document's first token is not looked at
    o, h, d = both(gpu, t, do, None)
    spoilt = [(0, 10), (100, 130), (130, 300)]
    fine = torch.ones(700, dtype=torch.bool, device=DEV)
    for i, j in spoilt:
        fine[i:j] = False
    assert torch.equal(h, want[1]) and torch.isfinite(h).all()
    assert torch.equal(o[:, fine], want[0][:, fine])
    for n in ("dq", "dk", "dv"):
        assert torch.equal(d[n][:, fine], want[2][n][:, fine]), n
    # in the document itself: outputs ahead of it, and all of the other heads
    assert torch.equal(o[:, :5], want[0][:, :5]) and torch.equal(o[:, 130:250], want[0][:, 130:250])
    assert torch.equal(o[:, :24, [0, 2, 3]], want[0][:, :24, [0, 2, 3]])
    if not math.isfinite(bad):
        assert torch.isnan(o[:, 250:300]).all()
    # among tokens that are not finite either
    t["k"] = s["k"].clone()
    t["k"][0, 3, 0, 1] = t["k"][0, 105, 1, 0] = math.nan
    o, h, d = both(gpu, t, do, None)
    assert torch.isfinite(h).all()
    for x in (o, d["dq"], d["dk"], d["dv"]):
        assert torch.isfinite(x[:, fine]).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, 3e38], ids=["nan", "inf", "3e38"])
def test_gradients_beside_decays_that_are_no_numbers(gpu, io, bad):
    """The gradients of the decays, too, are those of their own document: sums
    over a block's tokens stop at its ends."""
    s, do = packed(io, [10, 40, 70, 120], L=150, seed=5)
    want = both(gpu, s, do, None)[2]["dg"]
    for token, (i, j) in ((5, (0, 10)), (20, (10, 40)), (100, (70, 120)), (130, (120, 150))):
        t = dict(s, g=s["g"].clone())
        t["g"][0, token] = bad
        dg = both(gpu, t, do, None)[2]["dg"]
        assert torch.equal(dg[:, :i], want[:, :i]) and torch.equal(dg[:, j:], want[:, j:])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_documents_do_not_meet(gpu, io):
    """A document's results are the same bits whatever lies in the others of its
    block, also where sums over theirs are large or overflow."""
    s, do = packed(io, [20, 50, 90], L=150, seed=2)
    o, h, d = both(gpu, s, do, None)
    other, odo = packed(io, [20, 50, 90], L=150, seed=3)
    for size in (1.0, 1e12, 1e37):
        for i, j in ((0, 20), (20, 50), (50, 90), (90, 150)):
            keep = torch.zeros(150, dtype=torch.bool, device=DEV)
            keep[i:j] = True
            t = dict(s)
            for n in ("q", "k", "v", "g"):
                t[n] = torch.where(keep.view(1, -1, *(1,) * (s[n].dim() - 2)), s[n], other[n])
            # 4.6 at the most times 1e37 is finite
            tdo = torch.where(keep.view(1, -1, 1, 1), do, (odo.float() * size).to(do.dtype))
            assert torch.isfinite(tdo).all()
            to, th, td = both(gpu, t, tdo, None)
            assert torch.equal(to[:, i:j], o[:, i:j]), (size, i)
            if j == 150:
                assert torch.equal(th, h)
            for n in ("dq", "dk", "dv", "dg"):
                assert torch.equal(td[n][:, i:j], d[n][:, i:j]), (size, i, n)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_infinities(gpu, io):
    """An infinite key among positive numbers makes infinite sums: o and the state
    have them.  Gradients are finite where the definition's are and only there."""
    s, do, _ = inputs(1, 200, 4, 2, 40, 36, io, seed=4)
    for n in ("q", "k", "v"):
        s[n] = s[n].abs() + 0.125
    do = do.abs() + 0.125
    s["g"] = s["g"].clamp_min(-0.5)
    for where, value in ((("k", (0, 3, 0, 5)), math.inf), (("do", (0, 100, 1, 7)), math.inf)):
        t, tdo = dict(s, k=s["k"].clone()), do.clone()
        (t["k"] if where[0] == "k" else tdo)[where[1]] = value
        o, h, d = both(gpu, t, tdo, None)
        want, states, first = ref.forward(t, 0.3)
        w = ref.backward(t, 0.3, states, first, tdo)
        for x, y in ((o, want), (h, states[-1])):
            assert not torch.isnan(y).any() and not torch.isnan(x).any()
            assert torch.equal(torch.isposinf(x), torch.isposinf(y))
        for n in ("dq", "dk"):
            w[n] = ref.shared(w[n], 2)
        for n in ("dq", "dk", "dv", "dg"):
            assert torch.equal(torch.isfinite(d[n]), torch.isfinite(w[n])), (where, n)
