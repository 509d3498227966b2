"""Token log probabilities, entropy, alternatives and their gradient against
fp64.

Bounds.  A term 2^d carries |d| 2^-23 + 2^-23 of its value (the rounding of d
and of exp2); weighted by the terms themselves that is a few 2^-23 for the sum,
and the differences x - max and the logarithm add 2^-24 of their values: 1e-5
(1 + |ref|) leaves a factor of about ten.  The gradient adds the rounding of
lse and of its exponent, 2^-23 (|x| + |log p|) of p: 2e-5 of the value and of
the row's largest upstream gradient times scale, and half a bf16 ulp (2^-8
covers it) where it is bf16.  Token numbers are equal."""
import math

import numpy as np
import pytest
import torch

import lm_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
IO = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(rows, vocab, io, seed, std=2.5, pad=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    buf = (torch.randn(rows, vocab + pad, generator=g, device=DEV) * std).to(IO[io])
    t = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    return buf[:, :vocab], t


def upstream(rows, seed, size=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(rows, generator=g, device=DEV) * size for _ in range(2)]


def check(gpu, logits, targets, top=0, scale=1.0):
    got = gpu.token_logprobs_fwd(logits, targets, top=top, scale=scale)
    want = ref.logprobs(logits, targets, top, scale)
    for k in ("logprob", "entropy", "lse", "top_logprob"):
        w = want[k].numpy()
        ref.assert_close(got[k], w, 1e-5 * (1 + np.abs(np.where(np.isfinite(w), w, 0))), k)
    assert torch.equal(got["top_id"].cpu().long(), want["top_id"]), "top_id"
    return got


def check_grad(gpu, logits, targets, gl, gh, scale=1.0, out=None):
    r = gpu.token_logprobs_fwd(logits, targets, scale=scale)
    want = ref.logprobs_grad(logits, targets, gl, gh, scale).numpy()
    io = logits.dtype
    keep = logits.clone()
    got = gpu.token_logprobs_bwd(logits, targets, r["stats"], r["entropy"], gl, gh, scale=scale,
                                 dlogits=out)
    up = np.zeros(len(want))
    for t in (gl, gh):
        if t is not None:
            up = np.maximum(up, np.abs(t.cpu().double().numpy()))
    lim = 2e-5 * (np.abs(want) + scale * up[:, None])
    if io == torch.bfloat16:
        lim = lim + 2.0 ** -8 * np.abs(want)
    ref.assert_close(got, want, lim, "dlogits")
    return keep


# vocabularies around the vector (4, 8), wave and block sizes, odd ones, and
# ones long enough to be split over workgroups
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (2, 7), (5, 8), (4, 9), (3, 63), (2, 64),
                                        (6, 257), (3, 1023), (2, 2048), (5, 4099), (2, 8193),
                                        (3, 32001), (1, 70000), (1100, 513)])
def test_sizes(gpu, rows, vocab, io):
    x, t = make(rows, vocab, io, seed=rows * vocab)
    for top in sorted({0, 1, min(5, vocab), min(64, vocab)}):
        check(gpu, x, t, top=top, scale=1.0 if top else 0.7)
    gl, gh = upstream(rows, 1)
    check_grad(gpu, x, t, gl, gh, scale=1.3)
    check_grad(gpu, x, t, gl, None)
    check_grad(gpu, x, None, None, gh)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_strided_rows(gpu, io, pad):
    x, t = make(6, 5001, io, seed=3, pad=pad)
    check(gpu, x, t.int(), top=20)
    gl, gh = upstream(6, 2)
    check_grad(gpu, x, t, gl, gh)
    out = torch.empty(6, 5001 + 11, device=DEV, dtype=IO[io])[:, :5001]
    check_grad(gpu, x, t.int(), gl, gh, out=out)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [5, 700, 20000])
def test_masks(gpu, vocab, io):
    x, t = make(8, vocab, io, seed=4)
    lowest = torch.finfo(IO[io]).min
    t = t.long()
    x[0] = -math.inf                       # nothing left
    x[1] = lowest                          # the type's lowest everywhere: uniform
    x[2, :] = -math.inf
    x[2, vocab // 2] = 1.5                 # one token left
    t[2] = vocab // 2
    x[3, : vocab - 2] = -math.inf          # a few left, at the end
    x[4, 1:] = lowest                      # one token and the lowest
    t[4] = 0
    x[5, ::2] = -math.inf
    t[5] = 0                               # the target itself is masked
    t[6] = -100                            # no target
    t[7] = vocab                           # no target
    for top in (0, min(5, vocab)):
        got = check(gpu, x, t, top=top)
    assert got["entropy"][0] == 0 and got["logprob"][0] == -math.inf
    assert abs(float(got["entropy"][1]) - math.log(vocab)) <= 1e-5 * (1 + math.log(vocab))
    assert got["logprob"][2] == 0 and got["entropy"][2] == 0
    for size in (1.0, 10.0):  # with the lowest: gradients times log p past fp32's range
        gl, gh = upstream(8, 3, size)
        check_grad(gpu, x, t, gl, gh)


@pytest.mark.parametrize("vocab", [64, 100, 3000, 60000])
def test_ties_and_orders(gpu, vocab):
    """Equal logits rank by token; rows that rise, fall, are constant, or hold
    their largest values in one lane's share."""
    x, t = make(9, vocab, "bf16", seed=5)
    k = torch.arange(vocab, device=DEV).float()
    x[0] = 0.0
    x[1] = (k / vocab).bfloat16()
    x[2] = (-k / vocab).bfloat16()
    x[3] = (torch.round(x[3].float())).bfloat16()   # few values, many ties
    x[4] = 0.0
    x[4, ::2] = -0.0                                 # -0 and 0 are equal
    x[5] = -math.inf
    x[5, vocab - 1] = 1.0
    x[6] = (k % 512 < 8).bfloat16() * 3              # one lane's vectors
    x[7, :] = 100.0
    x[8] = (k / vocab * 200 - 100).bfloat16()
    for top in (1, 20, 64):
        check(gpu, x, t, top=top)


def test_nan_and_infinity(gpu):
    x, t = make(4, 9000, "f32", seed=6)
    x[1, 4000] = float("nan")
    x[2, 4000] = float("inf")
    got = gpu.token_logprobs_fwd(x, t, top=3)
    for k in ("logprob", "entropy", "lse"):
        assert torch.isnan(got[k][1]) and torch.isnan(got[k][2]), k
        assert torch.isfinite(got[k][0]) and torch.isfinite(got[k][3]), k
    assert got["top_id"][2, 0] == 4000 and 4000 not in got["top_id"][1].tolist()
    y = torch.full((1, 40), float("nan"), device=DEV)
    y[0, 7], y[0, 9] = 1.0, 2.0
    assert gpu.token_logprobs_fwd(y, top=4)["top_id"].tolist() == [[9, 7, -1, -1]]
    big = torch.full((1, 300), 3.0e38, device=DEV)
    big[0, 5:] = -3.0e38
    check(gpu, big, torch.zeros(1, dtype=torch.int64, device=DEV), top=5)


def test_gradient_in_place_and_differences(gpu):
    x, t = make(5, 1001, "f32", seed=8)
    gl, gh = upstream(5, 4)
    r = gpu.token_logprobs_fwd(x, t, scale=0.8)
    apart = gpu.token_logprobs_bwd(x, t, r["stats"], r["entropy"], gl, gh, scale=0.8)
    y = x.clone()
    gpu.token_logprobs_bwd(y, t, r["stats"], r["entropy"], gl, gh, scale=0.8, dlogits=y)
    assert torch.equal(apart, y)
    # central differences of the fp64 definition: truncation and rounding about
    # 1e-9, the fp32 gradient 2e-5 of sum |g| |v| at most
    v = torch.randn(5, 1001, generator=torch.Generator().manual_seed(2), dtype=torch.float64)

    def loss(z):
        w = ref.logprobs(z, t, 0, 0.8)
        return float((w["logprob"] * gl.cpu().double() + w["entropy"] * gh.cpu().double()).sum())

    e = 1e-5
    diff = (loss(x.cpu().double() + e * v) - loss(x.cpu().double() - e * v)) / (2 * e)
    g = apart.cpu().double()
    assert abs(float((g * v).sum()) - diff) <= 2e-5 * float((g.abs() * v.abs()).sum()) + 1e-7


def test_repeats_on_another_stream_and_in_a_graph(gpu):
    x, t = make(3, 50001, "bf16", seed=9)
    first = gpu.token_logprobs_fwd(x, t, top=10)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        again = gpu.token_logprobs_fwd(x, t, top=10, stream=stream)
        torch.cuda.synchronize()
        for k in first:
            assert torch.equal(first[k], again[k]), k
    ws = torch.empty(max(1, gpu.token_logprobs_workspace_bytes(3, 50001, 10, gpu.MS_BF16)),
                     dtype=torch.uint8, device=DEV)
    gl = torch.ones(3, device=DEV)
    d = torch.empty(3, 50001, dtype=x.dtype, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gpu.token_logprobs_fwd(x, t, top=10, workspace=ws)
        gpu.token_logprobs_bwd(x, t, out["stats"], out["entropy"], gl, gl, dlogits=d)
    want = gpu.token_logprobs_bwd(x, t, first["stats"], first["entropy"], gl, gl)
    for rep in range(3):
        for k in out:
            out[k].fill_(-7)
        ws.fill_(0xa5 + rep)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in first:
            assert torch.equal(first[k], out[k]), (rep, k)
        assert torch.equal(d, want), rep
        gpu.token_logprobs_fwd(x, t, top=10)
        torch.cuda.synchronize()


def test_autograd(gpu):
    x, t = make(6, 300, "f32", seed=10)
    x = x.clone().requires_grad_()
    lp, ent, top_lp, top_id = gpu.token_logprobs(x, t, top=4, scale=1.5)
    assert not top_lp.requires_grad and top_id.dtype == torch.int32
    (-lp.mean() - 0.1 * ent.mean()).backward()
    gl, gh = torch.full((6,), -1 / 6.0, device=DEV), torch.full((6,), -0.1 / 6, device=DEV)
    w = ref.logprobs_grad(x, t, gl, gh, 1.5).numpy()
    ref.assert_close(x.grad, w, 2e-5 * (np.abs(w) + 0.25), "grad")


def test_refusals(gpu):
    x, t = make(3, 40, "f32", seed=11)
    with pytest.raises(ValueError, match="device"):
        gpu.token_logprobs_fwd(x.cpu(), t)
    with pytest.raises(TypeError):
        gpu.token_logprobs_fwd(x.half(), t)
    with pytest.raises(ValueError, match="contiguous"):
        gpu.token_logprobs_fwd(torch.zeros(40, 3, device=DEV).t(), t)
    with pytest.raises(ValueError, match="overlapping"):
        gpu.token_logprobs_fwd(torch.zeros(40, device=DEV).expand(3, 40), t)
    with pytest.raises(TypeError, match="targets"):
        gpu.token_logprobs_fwd(x, t.float())
    with pytest.raises(ValueError, match="shape"):
        gpu.token_logprobs_fwd(x, t[:2])
    for top in (-1, 41, 65):
        with pytest.raises(gpu.MsError):
            gpu.token_logprobs_fwd(x, t, top=top)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(gpu.MsError, match="scale"):
            gpu.token_logprobs_fwd(x, t, scale=scale)
    with pytest.raises(gpu.MsError, match="16-byte"):
        gpu.token_logprobs_fwd(torch.zeros(3, 44, device=DEV)[:, 1:41], t)
    r = gpu.token_logprobs_fwd(x, t)
    with pytest.raises(gpu.MsError, match="targets"):
        gpu.token_logprobs_bwd(x, None, r["stats"], None, torch.ones(3, device=DEV))
    with pytest.raises(gpu.MsError, match="entropy"):
        gpu.token_logprobs_bwd(x, t, r["stats"], None, None, torch.ones(3, device=DEV))
    none = gpu.token_logprobs_fwd(x[:0], t[:0], top=2)
    assert none["logprob"].shape == (0,) and none["top_id"].shape == (0, 2)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_plans(gpu, io):
    """One workgroup a row, one of many waves, and rows split over workgroups,
    on both sides of the sizes where one gives way to the other."""
    for rows, vocab in ((1, 4100), (2, 57344), (2, 57345), (1, 114689), (95, 120000), (96, 120000),
                        (256, 9001), (257, 9001), (512, 4500)):
        x, t = make(rows, vocab, io, seed=rows + vocab)
        for top in (0, 7, 33, 64) if rows < 90 else (33,):
            check(gpu, x, t, top=top)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(6, 50280), (300, 50280), (6, 131072), (100, 131072),
                                        (300, 131072)])
def test_many_infinities(gpu, rows, vocab, io):
    """Rows of +inf, in one workgroup of few or many waves and in splits: NaN
    results, the lowest tokens that hold one as alternatives; other rows as ever."""
    x, t = make(rows, vocab, io, seed=rows + vocab)
    k = torch.arange(vocab, device=DEV)
    x[0] = math.inf
    x[1, ::2] = math.inf
    x[2] = torch.where(k > vocab // 2, math.inf, k / vocab).to(IO[io])
    x[3, vocab - 3:] = math.inf
    x[4, 7::16] = math.inf
    x[4, ::3] = float("nan")
    raw = x[:6].cpu().float().numpy()
    ids = np.argsort(np.where(np.isnan(raw), np.inf, -raw), axis=1, kind="stable")
    for top in (1, 5, 64):
        got = gpu.token_logprobs_fwd(x, t, top=top)
        for name in ("logprob", "entropy", "lse", "top_logprob"):
            assert torch.isnan(got[name][:5]).all(), name
            assert torch.isfinite(got[name][5:]).all(), name
        assert (got["top_id"][:6].cpu().numpy() == ids[:, :top]).all()
    gl, gh = upstream(rows, 5)
    r = gpu.token_logprobs_fwd(x, t)
    d = gpu.token_logprobs_bwd(x, t, r["stats"], r["entropy"], gl, gh)
    assert torch.isfinite(d[5:]).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_targets_and_gradients_off_16_bytes(gpu, io):
    """Targets after the first of a text, and gradients as torch.cat hands them
    on: contiguous, aligned to their element."""
    x, t = make(12, 3001, io, seed=12)
    for u in (t[1:], t.int()[1:]):
        assert u.data_ptr() % 16
        check(gpu, x[:11], u, top=5)
    a, b = (v.clone().requires_grad_() for v in (x[:5], x[5:11]))
    lp, ent = (torch.cat(v) for v in zip(gpu.token_logprobs(a, t[:5])[:2],
                                         gpu.token_logprobs(b, t[6:12])[:2]))
    gl, gh = upstream(11, 6)
    (lp * gl + ent * gh).sum().backward()
    for v, u, k in ((a, t[:5], slice(0, 5)), (b, t[6:12], slice(5, 11))):
        r = gpu.token_logprobs_fwd(v.detach(), u)
        want = gpu.token_logprobs_bwd(v.detach(), u, r["stats"], r["entropy"], gl[k].clone(),
                                      gh[k].clone())
        assert torch.equal(v.grad, want)


def test_autograd_takes_slices_of_a_token_tensor(gpu):
    x, _ = make(7, 200, "f32", seed=13)
    tokens = torch.randint(0, 200, (7, 5), generator=torch.Generator().manual_seed(3)).to(DEV)
    a, b = (gpu.token_logprobs(x, t)[0] for t in (tokens[:, 2], tokens[:, 2].contiguous()))
    assert torch.equal(a, b)
