"""Verification of drafted tokens where scale times a logit is large or tiny: a
scale that makes nearly greedy choices, logits far from 0, masks beside them."""
import math

import pytest
import torch

from test_verify_gpu import definition, inputs, softmax

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(gpu, args, scale):
    """As in test_verify_gpu, but for draws that no probabilities of finite
    precision settle.  Exponentials are right to 2.3e-12 (the first term left out
    of the cubic of 2^r, (ln 2 / 256)^4 / 24), so p and q each to 5e-12 with their
    sums, and what is left of p - q, of mass `left`, to 1e-11 in all: a border
    inside it moves by up to 1e-11 / left of the whole.  With 1e-9 to the next
    border a draw is settled from left = 0.01 on; below, where nearly equal
    distributions refuse a draft that neither would have drawn, it has to be a
    token that p has at all."""
    logits, ids, u, draft = args
    r = {n: x.cpu() for n, x in gpu.verify_drafts(logits, ids, u, draft, scale=scale).items()}
    tokens, count, logprob, near = definition(logits, ids, u, draft, scale)
    assert near > 1e-9, "choose another seed: a number lies on a border"
    assert torch.equal(r["count"].long(), count)
    for i in range(len(count)):
        t = int(count[i])
        p = softmax(logits[i, t].cpu(), scale)
        if p is not None and t < logits.shape[1] - 1 and draft is not None:
            q = softmax(draft[i, t].cpu(), scale)
            if q is not None and 0 < (p - q).clamp_min(0).sum() < 0.01:
                v = int(r["tokens"][i, t])
                assert p[v] > 0
                tokens[i, t], logprob[i, t] = v, p[v].log()
    assert torch.equal(r["tokens"].long(), tokens)
    err = (r["logprob"].double() - logprob).abs()
    assert (err <= 2.0 ** -23 * logprob.abs() + 1e-10).all()
    return r


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("scale", [2.0 ** -120, 2.0 ** -40, 1e3, 1e6, 1e8, 1e9, 2.0 ** 100],
                         ids=lambda s: f"{s:.0e}")
def test_scales(gpu, scale, drafted, io):
    args = inputs(6, 3, 3001, io, drafted, seed=1)
    logits, ids, u, draft = args
    run(gpu, args, scale)
    logits[:, :, 1000:2000] = -math.inf
    logits[:, :, 2500:] = torch.finfo(logits.dtype).min
    if drafted:
        draft[:, :, 200:300] = -math.inf
    run(gpu, args, scale)
    # drafts that a greedy choice takes
    ids.copy_(logits[:, :3].float().argmax(-1))
    if drafted:
        draft.copy_(logits[:, :3])
    r = run(gpu, args, scale)
    if scale >= 1e3 and drafted:
        assert (r["count"] == 3).all()


@pytest.mark.parametrize("scale", [1.0, 0.5, 16.0])
def test_logits_far_from_zero(gpu, scale):
    """Logits of 2e10 lie 2048 apart in fp32: the largest has all mass."""
    logits, ids, u, draft = inputs(4, 3, 1000, "f32", seed=2)
    for x in (logits, draft):
        x.mul_(2e10 / 8).add_(2e10)
    logits[:, :, 100:200] = -math.inf
    ids.copy_(logits[:, :3].argmax(-1))
    draft.scatter_(2, ids.unsqueeze(-1), 1e12)
    r = run(gpu, (logits, ids, u, draft), scale)
    # a probability of 1 comes out as 2^x / s with s = 2^x, |x| <= 2^-17 what the
    # rounding of 5e11 left: its log to a few 2^-53, besides the 2.3e-12 of run()
    assert (r["count"] == 3).all() and (r["logprob"].abs() <= 1e-11).all()
    # and at 1e7, where they are 1 apart
    logits, ids, u, draft = inputs(4, 3, 1000, "f32", seed=3)
    logits.mul_(4.0).add_(1e7)
    draft.mul_(4.0).sub_(3e7)
    run(gpu, (logits, ids, u, draft), scale)


def test_all_at_the_lowest_value(gpu):
    """A row of the type's lowest value is even; masks of -inf in it are none."""
    for dtype in ("f32", "bf16"):
        logits, ids, u, _ = inputs(3, 2, 500, dtype, seed=4)
        logits.fill_(torch.finfo(logits.dtype).min)
        logits[:, :, 100:300] = -math.inf
        for scale in (2.0 ** -110, 1.0, 1e20):
            run(gpu, (logits, ids, u, None), scale)
