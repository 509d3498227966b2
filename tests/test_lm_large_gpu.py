"""The language-model operators past 2^31 elements (any index or byte offset
kept in 32 bits would wrap), buffers' margins, and the timing hooks.

Large cases are compared where the offsets are large, against the same
definition on a small piece: after a reset the recurrence knows nothing of what
came before, tokens and rows are independent.  Bounds are those of the
operators' own tests."""
import numpy as np
import pytest
import torch

import lm_reference as ref
from helpers import assert_within

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def test_gated_scan_past_2_31_elements(gpu):
    L, d, tail = (1 << 21) + 37, 1024, 300
    g = gen(1)
    x, r, i, dy = (torch.empty(1, L, d, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
                   for _ in range(4))
    keep = 0.9 + 0.099 * torch.rand(d, generator=g, device=DEV)
    lam = torch.log(torch.expm1(-torch.log(keep) / 8.0))
    reset = torch.zeros(1, L, dtype=torch.uint8, device=DEV)
    reset[0, L - tail] = 1
    states, h_last = gpu.gated_scan_states(x), torch.empty(1, d, device=DEV)
    y = gpu.gated_scan_fwd(x, r, i, lam, reset=reset, h_last=h_last, states=states)
    got = gpu.gated_scan_bwd(x, r, i, lam, dy, states, reset=reset)
    assert torch.isfinite(got["dlam"]).all() and torch.isfinite(states).all()
    ch = torch.tensor([0, 63, 64, 500, d - 1], device=DEV)
    for cut in (slice(0, tail), slice(L - tail, L)):  # both ends
        p = {k: v[:, cut].index_select(2, ch) for k, v in (("x", x), ("r", r), ("i", i))}
        rs = reset[:, cut]
        yr, _, hr = ref.gated_forward(p["x"], p["r"], p["i"], lam[ch], reset=rs)
        assert_within(y[:, cut].index_select(2, ch), yr.numpy(), "bf16", f"y {cut}")
    assert_within(h_last[:, ch], hr.numpy(), "f32", "h_last")
    want = ref.gated_backward(p["x"], p["r"], p["i"], lam[ch], dy[:, cut].index_select(2, ch),
                              reset=rs)
    for k in ("dx", "dr", "di"):
        w = want[k].numpy()
        ref.assert_close(got[k][:, cut].index_select(2, ch), w, ref.grad_bound(w, "bf16"), k)


def test_gated_step_past_2_31_elements(gpu):
    b, d = 65537, 32776  # 2^31 + 5.6e5 states, 8.6 GB
    assert b * d > 2**31
    g = gen(2)
    x = torch.empty(b, d, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    h = torch.empty(b, d, device=DEV).normal_(generator=g)
    lam = torch.randn(d, generator=g, device=DEV)
    before = h[-3:].clone()
    y = gpu.gated_step(h, x, x, x, lam)
    t = x[-3:].unsqueeze(1)
    yr, _, hr = ref.gated_forward(t, t, t, lam, h0=before)
    assert_within(y[-3:], yr[:, 0].numpy(), "bf16")
    assert_within(h[-3:], hr.numpy(), "f32", "h")


def test_embedding_past_2_31_elements(gpu):
    rows, dim, n = (1 << 20) + 77, 2056, (1 << 20) + 5
    assert rows * dim > 2**31 and n * dim > 2**31
    g = gen(3)
    w = torch.empty(rows, dim, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    ids = torch.randint(0, rows, (n,), generator=g, device=DEV)
    ids[-1], ids[-2], ids[-3] = rows - 1, 0, rows - 1
    out = gpu.embed_fwd(ids, w, scale=2.0)
    for cut in (slice(0, 1000), slice(n - 1000, n)):
        assert torch.equal(out[cut], w[ids[cut]] * 2)
    # gradient: out serves as dy; rows at both ends of the table
    dw = gpu.embed_bwd(ids, out, rows, grad_dtype=torch.float32, dweight=None)
    for row in (0, 1, rows // 2, rows - 2, rows - 1):
        dy = out[ids == row].double()
        want, size = dy.sum(0), dy.abs().sum(0)
        err = (dw[row].double() - want).abs()
        assert (err <= (len(dy) + 1) * 2.0 ** -24 * size).all(), row


def test_logprobs_past_2_31_elements(gpu):
    rows, vocab, ld = 42000, 51200, 51211
    assert rows * vocab > 2**31
    g = gen(4)
    buf = torch.empty(rows, ld, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    logits = buf[:, :vocab]
    t = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    got = gpu.token_logprobs_fwd(logits, t, top=3)
    gl = torch.randn(rows, generator=g, device=DEV)
    keep = [(cut, logits[cut].float().cpu()) for cut in (slice(0, 3), slice(rows - 3, rows))]
    margin = buf[:, vocab:].clone()
    gpu.token_logprobs_bwd(logits, t, got["stats"], got["entropy"], gl, dlogits=logits)
    assert torch.equal(buf[:, vocab:], margin)  # nothing between the rows is written
    for cut, x in keep:
        want = ref.logprobs(x, t[cut], 3)
        for k in ("logprob", "entropy", "lse", "top_logprob"):
            v = want[k].numpy()
            ref.assert_close(got[k][cut], v, 1e-5 * (1 + np.abs(v)), k)
        assert torch.equal(got["top_id"][cut].cpu().long(), want["top_id"])
        grad = ref.logprobs_grad(x, t[cut], gl[cut], None).numpy()
        up = np.abs(gl[cut].cpu().double().numpy())[:, None]
        ref.assert_close(logits[cut], grad, 2e-5 * (np.abs(grad) + up) + 2.0 ** -8 * np.abs(grad),
                         "dlogits")


class Margins:
    """Buffers inside larger ones of a known byte."""

    def __init__(self):
        self.all = []

    def __call__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((256 + n + 256,), 0xA5, dtype=torch.uint8, device=DEV)
        self.all.append((raw, n))
        return raw[256:256 + n].view(dtype).view(shape)

    def check(self):
        for raw, n in self.all:
            assert (raw[:256] == 0xA5).all() and (raw[256 + n:] == 0xA5).all()


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_nothing_is_written_outside_the_buffers(gpu, io):
    """Odd sizes; given workspaces are of exactly the size asked for."""
    code = gpu.MS_BF16 if io == torch.bfloat16 else gpu.MS_F32
    g, f32 = gen(5), torch.float32
    for b, L, d in ((1, 1, 1), (2, 130, 3), (2, 1030, 37), (3, 257, 101)):
        m = Margins()
        x = torch.randn(b, L, d, generator=g, device=DEV).to(io)
        lam = torch.randn(d, generator=g, device=DEV)
        n = gpu.gated_scan_workspace_bytes(b, L, d, code)
        h, states = m((b, d), f32), m((b, -(-L // 16), d), f32)
        h.zero_()
        gpu.gated_scan_fwd(x, x, x, lam, x, y=m((b, L, d), io), h0=h, h_last=h, states=states,
                           workspace=m((n,), torch.uint8) if n else None)
        n = gpu.gated_scan_bwd_workspace_bytes(b, L, d, code)
        gpu.gated_scan_bwd(x, x, x, lam, x, states, x, workspace=m((n,), torch.uint8))
        gpu.gated_step(h, x[:, 0].contiguous(), x[:, 0].contiguous(), x[:, 0].contiguous(), lam,
                       y_t=m((b, d), io))
        m.check()
    for n, rows, dim in ((1, 1, 1), (77, 10, 5), (5000, 33, 19), (4097, 3, 261)):
        m = Margins()
        w = torch.randn(rows, dim, generator=g, device=DEV).to(io)
        ids = torch.randint(0, rows, (n,), generator=g, device=DEV)
        out = gpu.embed_fwd(ids, w, out=m((n, dim), io))
        size = gpu.embed_bwd_workspace_bytes(n, rows, dim, code)
        for gd in (f32, torch.bfloat16):
            gpu.embed_bwd(ids, out, rows, dweight=m((rows, dim), gd),
                          workspace=m((size,), torch.uint8))
        m.check()
    for rows, vocab, top in ((1, 1, 1), (3, 77, 5), (2, 33333, 64), (7, 9000, 0)):
        m = Margins()
        x = m((rows, vocab), io)
        x.copy_(torch.randn(rows, vocab, generator=g, device=DEV))
        t = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
        n = gpu.token_logprobs_workspace_bytes(rows, vocab, top, code)
        r = gpu.token_logprobs_fwd(x, t, top=top, workspace=m((n,), torch.uint8) if n else None)
        gpu.token_logprobs_bwd(x, t, r["stats"], r["entropy"], r["logprob"], r["entropy"],
                               dlogits=m((rows, vocab), io))
        m.check()


def test_launches_are_timed(gpu):
    x = torch.randn(2, 2000, 128, device=DEV)
    lam = torch.randn(128, device=DEV)
    states, h = gpu.gated_scan_states(x), torch.zeros(2, 128, device=DEV)
    x_t = x[:, 0].contiguous()
    w = torch.randn(40, 128, device=DEV)
    ids = torch.arange(5000, device=DEV) % 40
    t = torch.zeros(3, dtype=torch.int64, device=DEV)
    logits, long = torch.randn(3, 30000, device=DEV), torch.randn(3, 90000, device=DEV)
    # (call, launches of each phase)
    calls = [(lambda: gpu.gated_scan_fwd(x, x, x, lam, states=states), {"prep": 1, "main": 1}),
             (lambda: gpu.gated_scan_bwd(x, x, x, lam, x, states),
              {"prep": 1, "main": 1, "reduce": 1}),
             (lambda: gpu.gated_step(h, x_t, x_t, x_t, lam), {"step": 1}),
             (lambda: gpu.embed_fwd(ids, w), {"main": 1}),
             (lambda: gpu.embed_bwd(ids, torch.ones(5000, 128, device=DEV), 40),
              {"main": 1, "reduce": 1}),
             (lambda: gpu.token_logprobs_fwd(logits, t, top=5), {"main": 1}),
             (lambda: gpu.token_logprobs_fwd(long, t, top=5), {"main": 1, "reduce": 1})]
    for k, (call, want) in enumerate(calls):
        gpu.profile_begin(1)
        call()
        prof = gpu.profile_end()
        assert prof["calls"] == 1, k
        for phase, n in want.items():
            assert prof[phase]["launches"] == n and prof[phase]["mean_ms"] > 0, (k, phase, prof)
