"""The linear attention's operators together, as a program uses them: a layer
trained, a prompt and single tokens after it, and drafted tokens verified; and
offsets that pass 32 bits."""
import pytest
import torch

from test_verify_gpu import definition

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, HK, DK, DV, V, W = 4, 2, 16, 24, 97, 32  # heads, their keys', sizes, vocabulary, width


class Layer(torch.nn.Module):
    """Embedding, one layer and a head: heads normalised and gated."""

    def __init__(self, ms):
        super().__init__()
        self.ms = ms
        g = torch.Generator(device=DEV)
        g.manual_seed(0)
        p = lambda *s: torch.nn.Parameter(0.3 * torch.randn(s, generator=g, device=DEV))  # noqa: E731
        self.table, self.weight, self.out = p(V, W), p(H * DV), p(H * DV, W)
        self.proj = p(W, 2 * HK * DK + 2 * H * DV)
        self.g = torch.nn.Parameter(torch.tensor([-0.5, -0.1, -0.02, -0.005], device=DEV))

    def parts(self, ids, ms=None):
        x = self.ms.embed(ids, self.table, scale=1.0)
        p = x @ self.proj
        q, k, v, z = p.split([HK * DK, HK * DK, H * DV, H * DV], -1)  # read where they are
        return x, q.unflatten(-1, (HK, DK)), k.unflatten(-1, (HK, DK)), \
            v.unflatten(-1, (H, DV)), z

    def finish(self, x, o, z):
        y = self.ms.group_norm(o.flatten(-2), H, 1 + self.weight, None, z, center=False)
        return (x + y @ self.out) @ self.table.t()

    def forward(self, ids, reset=None, h0=None):
        x, q, k, v, z = self.parts(ids)
        o, h = self.ms.linear_attn(q, k, v, self.g, h0, scale=0.25, reset=reset, return_last=True)
        return self.finish(x, o, z), h


def plain(m, ids, reset):
    """The same in torch, in fp64."""
    t = {n: p.detach().double().requires_grad_() for n, p in m.named_parameters()}
    x = t["table"][ids]
    q, k, v, z = (x @ t["proj"]).split([HK * DK, HK * DK, H * DV, H * DV], -1)
    s = {"q": q.unflatten(-1, (HK, DK)), "k": k.unflatten(-1, (HK, DK)),
         "v": v.unflatten(-1, (H, DV))}
    q, k = (s[n].repeat_interleave(H // HK, 2) for n in ("q", "k"))
    keep = t["g"].exp().expand(*ids.shape, H) * (1 - reset.double()).unsqueeze(-1)
    S, o = 0.0, []
    for i in range(ids.shape[1]):
        S = S * keep[:, i, :, None, None] + k[:, i, :, :, None] * s["v"][:, i, :, None, :]
        o.append(0.25 * (q[:, i, :, :, None] * S).sum(-2))
    o = torch.stack(o, 1)
    y = o * (o.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    y = y.flatten(-2) * (1 + t["weight"]) * torch.nn.functional.silu(z)
    return (x + y @ t["out"]) @ t["table"].t(), t


def test_trained(gpu):
    """Loss and every gradient against the fp64 program.  fp32 throughout: sums
    over at most 3 x 75 tokens and 200 channels, three products deep; 1e-3 of
    the largest gradient is far above 2^-24 times their lengths (1e-5)."""
    m = Layer(gpu)
    ids = torch.randint(0, V, (3, 75), device=DEV)
    reset = (torch.rand(3, 75, device=DEV) < 0.05).to(torch.uint8)
    target = torch.randint(0, V, (225,), device=DEV)
    logits, _ = m(ids, reset)
    logp, *_ = gpu.token_logprobs(logits.flatten(0, 1), target)
    (-logp.mean()).backward()
    want, t = plain(m, ids, reset)
    loss = torch.nn.functional.cross_entropy(want.flatten(0, 1), target)
    loss.backward()
    assert abs(float(-logp.mean().detach()) - float(loss.detach())) < 1e-4
    for n, p in m.named_parameters():
        err = (p.grad.double() - t[n].grad).abs().max() / t[n].grad.abs().max()
        assert err < 1e-3, (n, float(err))


@torch.no_grad()
def test_served(gpu):
    """A prompt in one piece, then token by token: the same logits as all at
    once, to the bound of fp32 states (1e-4 of their size)."""
    m = Layer(gpu)
    ids = torch.randint(0, V, (2, 70), device=DEV)
    whole, _ = m(ids)
    logits, h = m(ids[:, :64])
    torch.testing.assert_close(logits, whole[:, :64], rtol=1e-4, atol=1e-4)
    for i in range(64, 70):
        x, q, k, v, z = m.parts(ids[:, i:i + 1])
        o = gpu.linear_attn_step(h, q, k, v, m.g, scale=0.25)
        torch.testing.assert_close(m.finish(x, o, z)[:, 0], whole[:, i], rtol=1e-4, atol=1e-4)


@torch.no_grad()
def test_drafted(gpu):
    """Drafted tokens scored ahead from the state, verified, and the accepted
    ones taken in: the states are those of the text that came out."""
    m = Layer(gpu)
    b, n = 5, 4
    prompt = torch.randint(0, V, (b, 33), device=DEV)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(7)
    text = [row.tolist() for row in prompt]
    _, h = m(prompt[:, :-1])
    last = prompt[:, -1]
    for _ in range(6):
        draft_logits = 0.5 * torch.randn(b, n, V, generator=gen, device=DEV)
        drafts = draft_logits.argmax(-1)
        ids = torch.cat([last[:, None], drafts], 1)
        before = h.clone()
        x, q, k, v, z = m.parts(ids)
        o = gpu.linear_attn_step(h, q, k, v, m.g, scale=0.25, update=False)
        assert torch.equal(h, before)
        logits = m.finish(x, o, z)
        u = torch.rand(b, n + 1, generator=gen, device=DEV)
        r = gpu.verify_drafts(logits, drafts, u, draft_logits)
        tokens, count, _, near = definition(logits, drafts, u, draft_logits, 1.0)
        assert near > 1e-9
        assert torch.equal(r["tokens"].cpu().long(), tokens)
        gpu.linear_attn_step(h, None, k, v, m.g, counts=r["count"] + 1)
        for i, row in enumerate(r["tokens"].tolist()):
            text[i] += [t for t in row if t >= 0]
        last = torch.tensor([row[-1] for row in text], device=DEV)
    for i, row in enumerate(text):
        _, want = m(torch.tensor([row[:-1]], device=DEV))
        torch.testing.assert_close(h[i:i + 1], want, rtol=1e-4, atol=1e-4)


def test_state_in_its_own_place(gpu):
    """h_last over h0 where the sequence is cut into segments, whose last one may
    be done before the first begins."""
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    for io in (torch.float32, torch.bfloat16):
        q, k, v = (rnd(1, 9000, 2, 64).to(io) for _ in range(3))
        decay = -0.001 * torch.rand(1, 9000, 2, generator=g, device=DEV)
        h0 = rnd(1, 2, 64, 64)
        want = torch.empty_like(h0)
        o = gpu.linear_attn_fwd(q, k, v, decay, h0=h0, h_last=want)
        for _ in range(5):
            h = h0.clone()
            assert torch.equal(gpu.linear_attn_fwd(q, k, v, decay, h0=h, h_last=h), o)
            assert torch.equal(h, want)


def test_past_32_bits(gpu):
    """v and o of more than 2^31 values: the last sequences are what they are by
    themselves."""
    b, L, heads, dk, dv = 1100, 64, 256, 8, 120
    assert b * L * heads * dv > 1 << 31
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    q, k = rnd(b, L, 1, dk), rnd(b, L, 1, dk)
    v = torch.zeros(b, L, heads, dv, dtype=torch.bfloat16, device=DEV)
    v[-2:] = rnd(2, L, heads, dv)
    decay = -torch.rand(heads, generator=g, device=DEV)
    o = gpu.linear_attn_fwd(q, k, v, decay)
    alone = gpu.linear_attn_fwd(q[-2:].contiguous(), k[-2:].contiguous(), v[-2:].contiguous(), decay)
    assert torch.equal(o[-2:], alone)
    assert not o[:-2].any()
    y = gpu.group_norm_fwd(o.flatten(2).flatten(0, 1), heads, center=False)
    want = gpu.group_norm_fwd(alone.flatten(2).flatten(0, 1), heads, center=False)
    assert torch.equal(y[-2 * L:], want)
