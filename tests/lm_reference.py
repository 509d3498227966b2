"""Plain fp64 references (CPU) of the language-model operators, written from
their definitions, and the bounds the GPU results are held to."""
from __future__ import annotations

import numpy as np
import torch

F64 = torch.float64


def to64(t):
    return None if t is None else t.detach().cpu().double()


# ---- gated linear recurrence ------------------------------------------------------------

def gated_coeffs(r, lam, c):
    """a and sqrt(1 - a^2), with 1 - a^2 = -expm1(2 log a) (no cancellation)."""
    rate = c * torch.where(lam > 30, lam, torch.log1p(torch.exp(torch.clamp(lam, max=30))))
    la = -rate * torch.sigmoid(r)
    return la, torch.exp(la), torch.sqrt(-torch.expm1(2 * la))


def gated_forward(x, r, i, lam, z=None, h0=None, reset=None, c=8.0):
    """(y, h of every step, h_last), timestep by timestep."""
    x, r, i, lam, z, h0 = map(to64, (x, r, i, lam, z, h0))
    la, a, n = gated_coeffs(r, lam, c)
    b = n * torch.sigmoid(i) * x
    h = torch.zeros_like(x[:, 0]) if h0 is None else h0.clone()
    hs = torch.empty_like(x)
    for t in range(x.shape[1]):
        past = a[:, t] * h
        if reset is not None:
            past = torch.where(reset[:, t].cpu().bool().unsqueeze(1), torch.zeros_like(past), past)
        h = past + b[:, t]
        hs[:, t] = h
    y = hs if z is None else hs * z * torch.sigmoid(z)
    return y, hs, h


def gated_backward(x, r, i, lam, dy, z=None, h0=None, dh_last=None, reset=None, c=8.0):
    """Gradients by the chain rule through a and sqrt(1 - a^2) apart; where a
    is 1 to fp64 (la == 0) the root's term is its limit, 0."""
    _, hs, _ = gated_forward(x, r, i, lam, z, h0, reset, c)
    x, r, i, lam, dy, z, h0, dh_last = map(to64, (x, r, i, lam, dy, z, h0, dh_last))
    la, a, n = gated_coeffs(r, lam, c)
    sr, si = torch.sigmoid(r), torch.sigmoid(i)
    B, L, d = x.shape
    keep = torch.ones(B, L, 1, dtype=F64)
    if reset is not None:
        keep = 1 - reset.cpu().bool().double().unsqueeze(2)
    out = {}
    gy = dy
    if z is not None:
        sz = torch.sigmoid(z)
        out["dz"] = dy * hs * sz * (1 + z * (1 - sz))
        gy = dy * z * sz
    g = torch.empty_like(x)
    m = torch.zeros(B, d, dtype=F64) if dh_last is None else dh_last.clone()
    for t in range(L - 1, -1, -1):
        g[:, t] = gy[:, t] + m
        m = g[:, t] * a[:, t] * keep[:, t]
    first = torch.zeros(B, 1, d, dtype=F64) if h0 is None else h0.unsqueeze(1)
    hprev = torch.cat([first, hs[:, :-1]], 1)
    out["dx"] = g * n * si
    out["di"] = g * n * x * si * (1 - si)
    dla = g * keep * a * hprev + torch.where(n > 0, -g * si * x * a * a / n, torch.zeros_like(n))
    sp = torch.where(lam > 30, lam, torch.log1p(torch.exp(torch.clamp(lam, max=30))))
    out["dr"] = dla * -c * sp * sr * (1 - sr)
    out["dlam"] = (dla * -c * sr).sum((0, 1)) * torch.sigmoid(lam)
    out["dh0"] = m
    return out


# ---- token log probabilities -------------------------------------------------------------

def log_softmax(x, scale):
    """(log p, lse) beside each row's largest logit; all -inf: -inf and -inf."""
    top = x.amax(1, keepdim=True)
    m = torch.where(torch.isneginf(top), torch.zeros_like(top), top)
    d = (x - m) * scale
    s = torch.log(torch.exp(d).sum(1, keepdim=True))
    dead = torch.isneginf(top)
    lp = torch.where(dead, torch.full_like(d, -torch.inf), d - s)
    return lp, (m * scale + s).squeeze(1)


def logprobs(logits, targets, top=0, scale=1.0):
    x = to64(logits)
    lp, lse = log_softmax(x, scale)
    p = torch.exp(lp)
    ent = -torch.where(p == 0, torch.zeros_like(p), p * lp).sum(1)
    chosen = torch.zeros(x.shape[0], dtype=F64)
    for k, t in enumerate(targets.tolist() if targets is not None else []):
        if 0 <= t < x.shape[1]:
            chosen[k] = lp[k, t]
    raw = to64(logits).numpy() + 0.0
    # stable sort of the negated values: largest first, lower token first
    ids = torch.from_numpy(np.argsort(-raw, axis=1, kind="stable")[:, :top].copy())
    return {"logprob": chosen, "entropy": ent, "lse": lse, "top_id": ids,
            "top_logprob": torch.gather(lp, 1, ids)}


def logprobs_grad(logits, targets, dlogprob, dentropy, scale=1.0):
    x = to64(logits)
    lp, lse = log_softmax(x, scale)
    p = torch.exp(lp)
    ent = -torch.where(p == 0, torch.zeros_like(p), p * lp).sum(1, keepdim=True)
    g = torch.zeros_like(x)
    if dlogprob is not None:
        gl = to64(dlogprob).clone()
        ok = (targets.cpu() >= 0) & (targets.cpu() < x.shape[1])
        gl[~ok] = 0
        g -= gl.unsqueeze(1) * p
        rows = torch.nonzero(ok).squeeze(1)
        g[rows, targets.cpu()[rows].long()] += gl[rows]
    if dentropy is not None:
        plp = torch.where(p == 0, torch.zeros_like(p), p * (lp + ent))
        g -= to64(dentropy).unsqueeze(1) * plp
    g[torch.isneginf(lse)] = 0
    return g * scale


# ---- bounds --------------------------------------------------------------------------------

def grad_bound(ref, io):
    """Gradients: 2e-4 of the value and of the tensor's RMS (the scan's own
    bound for fp32 gradients), and half a bf16 ulp (2^-8 of the value covers
    it with the rounding of the value itself) where they are rounded to bf16."""
    ref = np.asarray(ref, dtype=np.float64)
    rms = np.sqrt(np.mean(ref * ref)) if ref.size else 0.0
    lim = 2e-4 * (np.abs(ref) + rms) + 1e-30
    return lim + (2.0 ** -8 * np.abs(ref) if io == "bf16" else 0.0)


def assert_close(got, ref, lim, what):
    got = got.detach().cpu().double().numpy()
    ref = np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    finite = np.isfinite(ref)
    assert (np.isnan(got) == np.isnan(ref)).all(), f"{what}: NaN in other places"
    inf = ~finite & ~np.isnan(ref)
    assert (got[inf] == ref[inf]).all(), f"{what}: infinities differ"
    err = np.abs(got - np.where(finite, ref, 0))
    lim = np.broadcast_to(lim, ref.shape)
    bad = finite & ~(err <= lim)
    if bad.any():
        k = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; first at {k}: got "
                             f"{got[k]} ref {ref[k]} bound {lim[k]}")
