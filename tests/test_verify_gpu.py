"""Verification of drafted tokens (ms_verify_drafts) against its definition in
fp64, exactly where whole numbers come out: inputs whose numbers fall within
1e-9 of a border are not drawn (checked by the reference)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
IO = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(b, T, V, io, drafted=True, seed=0, std=2.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    logits = (std * n(b, T + 1, V)).to(IO[io])
    draft = (0.9 * logits[:, :T].float() + 0.8 * n(b, T, V)).to(IO[io]) if drafted else None
    noise = -torch.log(-torch.log(torch.rand(b, T, V, generator=g, device=DEV).clamp(1e-20, 1 - 1e-7)))
    x = draft.float() if drafted else 2 * logits[:, :T].float()
    ids = (x + noise).argmax(-1) if T else torch.zeros(b, 0, dtype=torch.int64, device=DEV)
    return logits, ids, torch.rand(b, T + 1, generator=g, device=DEV), draft


def softmax(row, scale):
    """Probabilities of a row in fp64, None where it has none."""
    x = row.double() * scale
    if not (x < math.inf).all() or x.max() == -math.inf:
        return None
    e = (x - x.max()).exp()
    return e / e.sum()


def definition(logits, ids, u, draft, scale):
    logits, ids, u = logits.cpu(), ids.cpu(), u.double().cpu()
    draft = None if draft is None else draft.cpu()
    b, T1, V = logits.shape
    tokens = torch.full((b, T1), -1, dtype=torch.int64)
    count = torch.zeros(b, dtype=torch.int64)
    logprob = torch.zeros(b, T1, dtype=torch.float64)
    near = 1.0
    for i in range(b):
        t = 0
        while True:
            p = softmax(logits[i, t], scale)
            if t == T1 - 1:
                left = p
                break
            x = int(ids[i, t])
            q = torch.zeros(V, dtype=torch.float64)
            if draft is None:
                if 0 <= x < V:
                    q[x] = 1.0
            else:
                q = softmax(draft[i, t], scale)
            there = 0 <= x < V and p is not None and q is not None
            if there and p[x] > 0:
                near = min(near, abs(float(u[i, t] * q[x] / p[x]) - 1))
            if there and u[i, t] * q[x] < p[x]:
                tokens[i, t], logprob[i, t] = x, p[x].log()
                t += 1
                continue
            left = None if p is None else p if q is None else (p - q).clamp_min(0)
            break
        count[i] = t
        if p is None:
            continue
        if left.sum() <= 0:
            left = p
        sums = left.cumsum(0)
        border = u[i, T1 - 1] * sums[-1]
        # masses of 0 sum to exactly 0, on either side: no border of a number of 0
        far = (sums / sums[-1] - u[i, T1 - 1]).abs()[sums > 0]
        near = min(near, float(far.min()))
        past = (sums > border).nonzero()
        v = int(past[0]) if len(past) else int((left > 0).nonzero()[-1])
        tokens[i, t], logprob[i, t] = v, p[v].log()
    return tokens, count, logprob, near


def run(gpu, args, scale=1.0, **kw):
    logits, ids, u, draft = args
    r = gpu.verify_drafts(logits, ids, u, draft, scale=scale, **kw)
    tokens, count, logprob, near = definition(logits, ids, u, draft, scale)
    assert near > 1e-9, "choose another seed: a number lies on a border"
    assert torch.equal(r["count"].cpu().long(), count)
    assert torch.equal(r["tokens"].cpu().long(), tokens)
    # fp64, rounded once
    err = (r["logprob"].cpu().double() - logprob).abs()
    assert (err <= 2.0 ** -23 * logprob.abs() + 1e-10).all()
    return r


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 0, 300), (3, 2, 5), (5, 4, 999), (40, 3, 64),
                                   (2, 64, 37), (1, 4, 50280), (2, 3, 131072), (3, 7, 4097)],
                         ids=lambda s: "x".join(map(str, s)))
def test_against_the_definition(gpu, shape, drafted, io):
    run(gpu, inputs(*shape, io, drafted, seed=sum(shape)), 1.0)
    run(gpu, inputs(*shape, io, drafted, seed=sum(shape) + 1), 0.75)


def test_all_accepted_and_none(gpu):
    logits, ids, u, draft = inputs(4, 5, 200, "f32", seed=3)
    r = run(gpu, (logits, ids, u, logits[:, :5].contiguous()))  # q = p
    assert (r["count"] == 5).all()
    low = logits.clone()
    low[:, :5].scatter_(2, ids.unsqueeze(-1), -math.inf)
    r = run(gpu, (low, ids, u, draft))
    assert (r["count"] == 0).all()


def test_masks_and_rows_that_are_none(gpu):
    logits, ids, u, draft = inputs(9, 3, 500, "bf16", seed=4)
    logits[:, :, 100:350] = -math.inf
    logits[5, :, 350:] = torch.finfo(torch.bfloat16).min
    draft[3, 1] = -math.inf
    draft[4, 0, 7] = math.nan
    draft[6, 0, 7] = math.inf
    logits[1, 0] = -math.inf
    logits[2, 0, 499] = math.nan
    logits[7, 3] = math.nan
    logits[8, 0, 0] = math.inf
    ids[0, 0], ids[0, 1] = 200, 9  # masked
    ids[7] = logits[7, :3].float().argmax(-1)
    u[7, :3] = 0.0
    r = run(gpu, (logits, ids, u, draft))
    tokens = r["tokens"].cpu()
    assert (tokens[1] == -1).all() and (tokens[2] == -1).all() and (tokens[8] == -1).all()
    assert int(r["count"][7]) == 3 and int(tokens[7, 3]) == -1


def test_ids_outside_and_numbers_at_the_ends(gpu):
    logits, ids, u, draft = inputs(6, 2, 4100, "f32", seed=5)
    ids[0, 0], ids[1, 0], ids[2, 1] = -1, 4100, 1 << 40
    u[:, 2] = torch.tensor([0.0, 1 - 2.0 ** -24, 0.5, 0.0, 1 - 2.0 ** -24, 0.25])
    logits[3:, :, :10] = -math.inf  # a draw of 0 is the first with any mass
    logits[4, :, 4000:] = -math.inf
    run(gpu, (logits, ids, u, draft))
    run(gpu, (logits, ids, u, None))
    run(gpu, (logits, ids.to(torch.int32), u, draft))
    # numbers that are not below 1 draw the last token with mass
    u[:, 2] = 1.0
    r = gpu.verify_drafts(logits, ids, u, draft)
    assert (r["tokens"] < 4100).all() and (r["tokens"].amax(1) >= 0).all()


def test_a_draw_of_a_large_row(gpu):
    """Every piece of a row is searched: one token holds nearly all mass."""
    V = 300000
    logits = torch.full((8, 1, V), -20.0, device=DEV)
    places = torch.tensor([0, 1, 4095, 4096, 131071, 262144, V - 2, V - 1], device=DEV)
    logits[torch.arange(8, device=DEV), 0, places] = 20.0
    u = torch.full((8, 1), 0.5, device=DEV)
    r = gpu.verify_drafts(logits, torch.zeros(8, 0, dtype=torch.int64, device=DEV), u)
    assert torch.equal(r["tokens"][:, 0].long(), places)


def test_strided_streams_graphs(gpu):
    logits, ids, u, draft = inputs(4, 3, 1001, "bf16", seed=6)
    wide = torch.zeros(4, 4, 1010, dtype=torch.bfloat16, device=DEV)
    wide[..., 3:1004] = logits
    want = run(gpu, (logits, ids, u, draft))
    for r in (gpu.verify_drafts(wide[..., 3:1004], ids, u, draft),):
        for n in want:
            assert torch.equal(r[n], want[n])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    r = gpu.verify_drafts(logits, ids, u, draft, stream=side)
    side.synchronize()
    for n in want:
        assert torch.equal(r[n], want[n])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = gpu.verify_drafts(logits, ids, u, draft)
    for k in range(4):
        for x, y in zip((logits, ids, u, draft), inputs(4, 3, 1001, "bf16", seed=10 + k)):
            x.copy_(y)
        graph.replay()
        w = gpu.verify_drafts(logits, ids, u, draft)
        torch.cuda.synchronize()
        for n in w:
            assert torch.equal(r[n], w[n])


def test_refusals(gpu):
    logits, ids, u, draft = inputs(2, 3, 100, "f32")
    f = gpu.verify_drafts
    for bad in (lambda: f(logits.cpu(), ids, u, draft), lambda: f(logits[0], ids, u, draft),
                lambda: f(logits, ids[:, :2], u, draft), lambda: f(logits, ids, u[:, :3], draft),
                lambda: f(logits, ids, u, draft[:, :2]), lambda: f(logits, ids, None, draft),
                lambda: f(logits, ids.t().contiguous().t(), u, draft),
                lambda: f(logits.transpose(1, 2), ids, u, draft),
                lambda: f(logits[:, :0], ids[:, :0], u[:, :0])):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for bad in (lambda: f(logits, ids.float(), u, draft), lambda: f(logits, ids, u.double(), draft),
                lambda: f(logits, ids, u, draft.bfloat16()), lambda: f(logits.half(), ids, u)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: f(logits, ids, u, draft, scale=0.0),
                lambda: f(logits, ids, u, draft, scale=math.inf),
                lambda: f(logits, ids, u, draft, workspace=torch.zeros(4, device=DEV)),
                lambda: f(torch.zeros(1, 66, 4, device=DEV),
                          torch.zeros(1, 65, dtype=torch.int64, device=DEV),
                          torch.zeros(1, 66, device=DEV))):
        with pytest.raises(gpu.MsError):
            bad()
    r = f(logits[:0], ids[:0], u[:0], draft[:0])
    assert r["tokens"].shape == (0, 4)
