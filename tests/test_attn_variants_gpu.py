"""Variants of the kernels that are taken by size, at sizes that take them: two
workgroups of the forward a CU, states past the caches, longer pieces of a
vocabulary."""
import math

import pytest
import torch

import attn_reference as ref
from test_linear_attn_gpu import both, inputs
from test_verify_gpu import inputs as drafts
from test_verify_gpu import run

pytestmark = pytest.mark.gpu
DEV = "cuda"

# dk > 64 and more than 256 workgroups: rows of whole vectors and not, sequences that
# are cut (8 and 16 heads' columns, 64 and 32 segments) and not
PAIRS = [(3, 150, 88, 44, 72, 64), (3, 97, 44, 1, 101, 66), (2, 200, 66, 66, 128, 128)]
LONG = [(1, 8500, 4, 2, 72, 100), (2, 8300, 4, 1, 65, 128)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", PAIRS + LONG, ids=lambda s: "x".join(map(str, s)))
def test_two_workgroups_a_cu(gpu, shape, io):
    b, L, H, Hk, dk, dv = shape
    assert b * H * ((dv + 63) // 64) > 256 or L > 8000
    kinds = [(True, True, False), (False, False, True)]
    for k, (start, reset, fixed) in enumerate(kinds if L < 8000 else kinds[:1]):
        s, do, dh = inputs(*shape, io, start, reset, fixed, seed=70 + k)
        if L > 8000:  # memories that outlast a segment
            s["g"] = s["g"] * 0.02
        o, h_last, d = both(gpu, s, do, dh)
        states, first, bigs = ref.check_forward(s, 0.3, io, o, h_last)
        ref.check_backward(s, 0.3, io, states, first, bigs, do, dh, d)
        # the same in pieces of whole blocks, which take other variants
        part = s["h0"].clone() if start else torch.zeros(b, H, dk, dv, device=DEV)
        outs = []
        for i in range(0, L, 64):
            t = {n: s[n][:, i:i + 64].contiguous() for n in ("q", "k", "v")}
            g = s["g"] if fixed else s["g"][:, i:i + 64].contiguous()
            r = None if s["reset"] is None else s["reset"][:, i:i + 64].contiguous()
            outs.append(gpu.linear_attn_fwd(t["q"], t["k"], t["v"], g, scale=0.3, reset=r, h0=part,
                                            h_last=part))
            if i >= 512:
                break
        got = torch.cat(outs, 1)
        n = got.shape[1]
        t = dict(s, **{m: s[m][:, :n] for m in ("q", "k", "v")})
        t["g"] = s["g"] if fixed else s["g"][:, :n]
        t["reset"] = None if s["reset"] is None else s["reset"][:, :n]
        want, big = (ref.forward(x, 0.3)[0] for x in (t, ref.absolute(t)))
        ref.check(got, want, ref.bound(want, big, ref.const(s, io), io), "o in pieces")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["q", "k", "v"])
def test_not_finite_with_two_a_cu(gpu, io, where):
    """The token-by-token path of that variant: its queries wait in LDS and are
    asked for late."""
    s, _, _ = inputs(3, 150, 88, 88, 72, 60, io, True, seed=80)
    s["reset"] = torch.zeros(3, 150, dtype=torch.uint8, device=DEV)
    s["reset"][0, 50] = s["reset"][1, 128] = s["reset"][2, 90] = 1
    s[where][0, 40, :, 3] = math.nan
    s[where][1, 100, 5, 5] = math.nan
    s[where][2, 64, 7, 0] = -math.inf
    h_last = torch.empty(3, 88, 72, 60, device=DEV)
    o = gpu.linear_attn_fwd(s["q"], s["k"], s["v"], s["g"], scale=0.3, reset=s["reset"],
                            h0=s["h0"], h_last=h_last)
    want, states, _ = ref.forward(s, 0.3)
    clean = dict(s, **{where: s[where].nan_to_num(0, 0, 0)})
    big, bigs, _ = ref.forward(ref.absolute(clean), 0.3)
    c, fine = ref.const(s, io), torch.isfinite(want)
    assert not fine.all() and torch.equal(torch.isfinite(o), fine)
    ref.check(torch.where(fine, o.double(), 0.0), torch.where(fine, want, 0.0),
              ref.bound(torch.where(fine, want, 0.0), big, c, io), "o")
    ref.check(h_last, states[-1], ref.bound(states[-1], bigs[-1], c, "f32"), "h_last")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("dv", [128, 126])
def test_step_on_a_large_state(gpu, io, dv):
    """States above 64 MB go past the caches: twice in turn, and read again by
    what does not."""
    b, H, Hk, dk = 320, 8, 2, 64
    assert b * H * dk * dv * 4 > 64e6
    s, _, _ = inputs(b, 1, H, Hk, dk, dv, io, True, seed=90)
    h = s["h0"].clone()
    for k in range(2):
        before = h.clone()
        t = dict(s, h0=before)
        o = gpu.linear_attn_step(h, s["q"], s["k"], s["v"], s["g"], scale=0.3)
        ref.check_forward(t, 0.3, io, o, h)
        kept = before.clone()
        o2 = gpu.linear_attn_step(kept, s["q"], s["k"], s["v"], s["g"], scale=0.3, update=False)
        assert torch.equal(o, o2) and torch.equal(kept, before)
        # the small state's variant, by parts of the batch
        for i in (0, 200):
            part = {n: s[n][i:i + 20].contiguous() for n in ("q", "k", "v", "g")}
            hp = before[i:i + 20].contiguous()
            op = gpu.linear_attn_step(hp, *part.values(), scale=0.3)
            assert torch.equal(op, o[i:i + 20]) and torch.equal(hp, h[i:i + 20])
    counts = torch.arange(b, device=DEV, dtype=torch.int32) % 2
    before = h.clone()
    gpu.linear_attn_step(h, None, s["k"], s["v"], s["g"], counts=counts)
    gpu.linear_attn_step(before, None, s["k"], s["v"], s["g"])
    assert torch.equal(h[1::2], before[1::2])


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("shape", [(300, 1, 8200), (600, 1, 8200), (150, 2, 30001), (2, 64, 20000)],
                         ids=lambda s: "x".join(map(str, s)))
def test_longer_pieces(gpu, shape, drafted):
    """More than 1024 pieces of 2048 values: pieces of 4096 and 8192; many drafts
    whose rows are in many parts."""
    run(gpu, drafts(*shape, "bf16", drafted, seed=100 + shape[0]), 1.0)
