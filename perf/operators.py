"""Cases of the language-model operators beside the scan: the gated linear recurrence (forward,
training pass, single-token step), the embedding lookup with its gradient, and the log
probabilities of given tokens with entropy and top alternatives.

Each case is timed in a plain form (elementary torch operations in fp32, rounded once at the end)
and, with ``own`` set, through the framework's entry points.  ``exact`` is the definition in fp64.
"""
import math

import torch

own = False

DEV = "cuda"
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
SHARPNESS = 8.0  # c of the recurrence: a = exp(-c softplus(lam) sigmoid(r))


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # prefill of the 130M layer's shape, with the output gate
        {"name": "recur_layer", "op": "recur", "batch": 8, "L": 2048, "d": 1536, "io": "bf16",
         "gate": True, "start": False, "reset": False},
        # one long document continued from a state: few channels, the sequence has to be split
        {"name": "recur_long", "op": "recur", "batch": 1, "L": 131072, "d": 1536, "io": "bf16",
         "gate": False, "start": True, "reset": False},
        # a training step's forward and backward of the 130M layer's shape
        {"name": "recur_train", "op": "recur_train", "batch": 8, "L": 2048, "d": 1536,
         "io": "bf16", "gate": True, "start": False, "reset": False},
        # training on packed documents in fp32: ragged length, a channel count of no tile, resets
        {"name": "recur_train_packed", "op": "recur_train", "batch": 3, "L": 1999, "d": 1000,
         "io": "f32", "gate": False, "start": True, "reset": True},
        # one decode step of the decode workload's batch and width
        {"name": "recur_step", "op": "recur_step", "batch": 256, "d": 5120, "io": "bf16",
         "gate": True},
        # the tokens of a training batch looked up in a 50k table
        {"name": "embed_batch", "op": "embed", "n": 16384, "rows": 50280, "d": 768, "io": "bf16",
         "ids": "i64", "scaled": True},
        # the gradient of that table: word frequencies, a few tokens hold much of the batch
        {"name": "embed_grad", "op": "embed_grad", "n": 16384, "rows": 50280, "d": 768,
         "io": "bf16", "ids": "i64", "scaled": True},
        # the gradient of a wide 256k table from a large batch, in fp32
        {"name": "embed_grad_large", "op": "embed_grad", "n": 131072, "rows": 256000, "d": 2048,
         "io": "f32", "ids": "i32", "scaled": False},
        # one request's next token: log probability, entropy and five alternatives
        {"name": "logp_one", "op": "logp", "rows": 1, "vocab": 50280, "io": "f32", "top": 5,
         "pad": 0, "masked": False, "warm": False},
        # a serving batch over a 128k vocabulary, banned tokens, temperature, twenty alternatives
        {"name": "logp_serve", "op": "logp", "rows": 64, "vocab": 131072, "io": "bf16",
         "top": 20, "pad": 0, "masked": True, "warm": True},
        # scoring given text (perplexity) with alternatives
        {"name": "logp_score", "op": "logp", "rows": 8192, "vocab": 50280, "io": "bf16",
         "top": 5, "pad": 0, "masked": False, "warm": False},
        # the loss and its gradient, odd vocabulary in rows padded to whole vectors
        {"name": "logp_train", "op": "logp_train", "rows": 8192, "vocab": 32001, "io": "bf16",
         "pad": 7, "masked": False, "warm": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["recur", "recur", "recur_train", "recur_train", "recur_step", "embed",
                     "embed_grad", "embed_grad", "logp", "logp", "logp_train"])
    io = rng.choice(["bf16", "bf16", "f32"])
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("recur", "recur_train"):
        d = _log(rng, 64, 5120)
        d = d if rng.random() < 0.3 else max(8, d // 8 * 8)
        L = _log(rng, 1, 131072)
        most = 1 << 26 if op == "recur" else 1 << 25
        L = min(L, most // d)
        batch = max(1, min(_log(rng, 1, 64), most // (d * L)))
        return {"op": op, "batch": batch, "L": L, "d": d, "io": io, "gate": flip(),
                "start": flip(), "reset": rng.random() < 0.3}
    if op == "recur_step":
        return {"op": op, "batch": _log(rng, 1, 512), "d": _log(rng, 64, 5120), "io": io,
                "gate": flip()}
    if op in ("embed", "embed_grad"):
        d = _log(rng, 64, 4096)
        d = d if rng.random() < 0.3 else max(8, d // 8 * 8)
        n, rows = _log(rng, 1, 131072), _log(rng, 256, 256000)
        while n * d > 1 << 28:
            n //= 2
        while rows * d > 1 << 28:
            rows //= 2
        return {"op": op, "n": n, "rows": rows, "d": d, "io": io,
                "ids": rng.choice(["i64", "i32"]), "scaled": flip()}
    vocab = _log(rng, 256, 256000)
    rows = _log(rng, 1, 8192)
    while rows * vocab > 1 << 28:
        rows //= 2
    case = {"op": op, "rows": rows, "vocab": vocab, "io": io,
            "pad": rng.choice([0, 0, (-vocab) % 8, 3]), "masked": rng.random() < 0.3,
            "warm": flip()}
    if op == "logp":
        case["top"] = rng.choice([0, 1, 5, 20, 64])
    return case


# ---- what a user's program has in hand -----------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, io = case["op"], IO[case["io"]]
    s = {"case": case}

    def normal(*shape, std=1.0, dtype=io):
        return torch.randn(shape, generator=g, device=DEV).mul_(std).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    if op.startswith("recur"):
        b, d = case["batch"], case["d"]
        # decays exp(-c softplus(lam)) spread over 0.9 .. 0.999, as such layers are started
        keep = 0.9 + 0.099 * uniform(d)
        s["lam"] = torch.log(torch.expm1(-torch.log(keep) / SHARPNESS))
        if op == "recur_step":
            for k in ("x", "r", "i"):
                s[k] = normal(b, d)
            s["z"] = normal(b, d) if case["gate"] else None
            s["h"] = normal(b, d, dtype=torch.float32)
            return s
        L = case["L"]
        for k in ("x", "r", "i"):
            s[k] = normal(b, L, d)
        s["z"] = normal(b, L, d) if case["gate"] else None
        s["h0"] = normal(b, d, dtype=torch.float32) if case["start"] else None
        s["reset"] = (uniform(b, L) < 1.0 / 256).to(torch.uint8) if case["reset"] else None
        if op == "recur_train":
            s["dy"] = normal(b, L, d)
            s["dh_last"] = normal(b, d, dtype=torch.float32) if case["start"] else None
        return s
    if op.startswith("embed"):
        n, rows, d = case["n"], case["rows"], case["d"]
        # word frequencies fall as 1 / rank; ranks are spread over the table
        rank = torch.exp(uniform(n).double() * math.log(rows)).long().sub_(1).clamp_(0, rows - 1)
        names = torch.randperm(rows, generator=g, device=DEV)
        s["ids"] = names[rank].to(torch.int64 if case["ids"] == "i64" else torch.int32)
        s["scale"] = math.sqrt(d) if case["scaled"] else 1.0
        if op == "embed":
            s["weight"] = normal(rows, d, std=0.02)
        else:
            s["dy"] = normal(n, d)
        return s
    rows, vocab = case["rows"], case["vocab"]
    buf = normal(rows, vocab + case["pad"], std=2.5)
    if case["masked"]:  # one token in a hundred is banned
        banned = uniform(vocab + case["pad"]) < 0.01
        buf.masked_fill_(banned, -math.inf)
    s["logits"] = buf[:, :vocab]
    s["scale"] = 1.25 if case["warm"] else 1.0
    s["targets"] = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    if op == "logp_train":
        s["dlogprob"] = torch.full((rows,), -1.0 / rows, device=DEV)
        s["dentropy"] = torch.full((rows,), -0.01 / rows, device=DEV)
    return s


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return (_own if own else _plain)[op](state)


def _scan_plain(A, B):
    """h_t = A_t h_{t-1} + B_t along dim 1, by doubling (inclusive, from zero)."""
    A, B = A.clone(), B.clone()
    step, L = 1, A.shape[1]
    while step < L:
        B[:, step:] += A[:, step:] * B[:, :-step]
        A[:, step:] = A[:, step:] * A[:, :-step]
        step *= 2
    return B


def _gates_plain(s):
    x, r, i = s["x"].float(), s["r"].float(), s["i"].float()
    sr, si = torch.sigmoid(r), torch.sigmoid(i)
    sp = torch.logaddexp(s["lam"], torch.zeros_like(s["lam"]))
    la = -SHARPNESS * sp * sr
    a = torch.exp(la)
    norm = torch.sqrt(-torch.expm1(2 * la))
    return x, sr, si, sp, la, a, norm


def _recur_forward_plain(s):
    x, sr, si, sp, la, a, norm = _gates_plain(s)
    A = a if s["reset"] is None else a * (s["reset"] == 0).unsqueeze(-1)
    B = norm * si * x
    if s["h0"] is not None:
        B[:, 0] += A[:, 0] * s["h0"]
    return _scan_plain(A, B), A, (x, sr, si, sp, la, a, norm)


def _recur_plain(s):
    h, _, _ = _recur_forward_plain(s)
    y = h
    if s["z"] is not None:
        z = s["z"].float()
        y = h * (z * torch.sigmoid(z))
    return {"y": y.to(s["x"].dtype), "h_last": h[:, -1].contiguous()}


def _recur_train_plain(s):
    h, A, (x, sr, si, sp, la, a, norm) = _recur_forward_plain(s)
    io = s["x"].dtype
    out = {}
    gh = s["dy"].float()
    y = h
    if s["z"] is not None:
        z = s["z"].float()
        sz = torch.sigmoid(z)
        y = h * (z * sz)
        out["dz"] = (gh * h * sz * (1 + z * (1 - sz))).to(io)
        gh = gh * (z * sz)
    out["y"] = y.to(io)
    if s["dh_last"] is not None:
        gh = gh.clone()
        gh[:, -1] += s["dh_last"]
    # lambda_t = gh_t + A_{t+1} lambda_{t+1}: the same scan over reversed time
    Anext = torch.cat([A[:, 1:], torch.zeros_like(A[:, :1])], dim=1)
    lam = _scan_plain(Anext.flip(1), gh.flip(1)).flip(1)
    first = s["h0"].unsqueeze(1) if s["h0"] is not None else torch.zeros_like(h[:, :1])
    hprev = torch.cat([first, h[:, :-1]], dim=1)
    ratio = torch.where(norm > 0, la / norm, torch.zeros_like(la))
    q = lam * (A * hprev * la - si * x * a * a * ratio)
    out["dx"] = (lam * norm * si).to(io)
    out["di"] = (lam * norm * x * si * (1 - si)).to(io)
    out["dr"] = (q * (1 - sr)).to(io)
    out["dlam"] = q.sum(dim=(0, 1)) * torch.sigmoid(s["lam"]) / sp
    if s["h0"] is not None:
        out["dh0"] = A[:, 0] * lam[:, 0]
    return out


def _recur_step_plain(s):
    x, sr, si, sp, la, a, norm = _gates_plain(s)
    s["h"].copy_(a * s["h"] + norm * si * x)
    y = s["h"]
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    return {"y": y.to(s["x"].dtype), "h": s["h"]}


def _embed_plain(s):
    return (s["weight"][s["ids"].long()].float() * s["scale"]).to(s["weight"].dtype)


def _embed_grad_plain(s):
    dw = torch.zeros(s["case"]["rows"], s["case"]["d"], device=DEV)
    dw.index_add_(0, s["ids"].long(), s["dy"].float() * s["scale"])
    return dw.to(s["dy"].dtype)


def _logp_forward_plain(s):
    x = s["logits"].float() * s["scale"]
    top = x.amax(dim=1, keepdim=True)
    e = torch.exp(x - top)
    lse = torch.log(e.sum(dim=1, keepdim=True)) + top
    logp = x - lse
    p = torch.exp(logp)
    entropy = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(dim=1)
    return logp, p, entropy, logp.gather(1, s["targets"].unsqueeze(1)).squeeze(1)


def _logp_plain(s):
    logp, _, entropy, chosen = _logp_forward_plain(s)
    out = {"logprob": chosen, "entropy": entropy}
    k, vocab = s["case"]["top"], s["case"]["vocab"]
    if k:
        # order by (logit descending, token ascending): unique whole-number keys
        bits = s["logits"].float().add(0.0).contiguous().view(torch.int32).long()
        key = torch.where(bits < 0, -(bits & 0x7fffffff), bits)
        key = key * (1 << 20) + (vocab - 1 - torch.arange(vocab, device=DEV))
        ids = torch.topk(key, k, dim=1).values
        ids = vocab - 1 - (ids & ((1 << 20) - 1))
        out["top_id"] = ids.to(torch.int32)
        out["top_logprob"] = logp.gather(1, ids)
    return out


def _logp_train_plain(s):
    logp, p, entropy, chosen = _logp_forward_plain(s)
    gl, gh = s["dlogprob"].unsqueeze(1), s["dentropy"].unsqueeze(1)
    plp = torch.where(p > 0, p * (logp + entropy.unsqueeze(1)), torch.zeros_like(p))
    grad = -gl * p - gh * plp
    grad.scatter_add_(1, s["targets"].unsqueeze(1), gl)
    return {"logprob": chosen, "entropy": entropy,
            "dlogits": (grad * s["scale"]).to(s["logits"].dtype)}


_plain = {"recur": _recur_plain, "recur_train": _recur_train_plain,
          "recur_step": _recur_step_plain, "embed": _embed_plain,
          "embed_grad": _embed_grad_plain, "logp": _logp_plain, "logp_train": _logp_train_plain}


def _ms():
    import selective_state_space_81_amd as ms
    return ms


def _recur_own(s):
    x = s["x"]
    h_last = torch.empty(x.shape[0], x.shape[2], dtype=torch.float32, device=DEV)
    y = _ms().gated_scan_fwd(x, s["r"], s["i"], s["lam"], s["z"], c=SHARPNESS, reset=s["reset"],
                             h0=s["h0"], h_last=h_last)
    return {"y": y, "h_last": h_last}


def _recur_train_own(s):
    ms = _ms()
    states = ms.gated_scan_states(s["x"])
    y = ms.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], s["z"], c=SHARPNESS,
                          reset=s["reset"], h0=s["h0"], states=states)
    g = ms.gated_scan_bwd(s["x"], s["r"], s["i"], s["lam"], s["dy"], states, s["z"], c=SHARPNESS,
                          reset=s["reset"], dh_last=s["dh_last"], want_dh0=s["h0"] is not None)
    out = {"dx": g["dx"], "dr": g["dr"], "di": g["di"], "dlam": g["dlam"], "y": y}
    if s["z"] is not None:
        out["dz"] = g["dz"]
    if s["h0"] is not None:
        out["dh0"] = g["dh0"]
    return out


def _recur_step_own(s):
    y = _ms().gated_step(s["h"], s["x"], s["r"], s["i"], s["lam"], s["z"], c=SHARPNESS)
    return {"y": y, "h": s["h"]}


def _embed_own(s):
    return _ms().embed_fwd(s["ids"], s["weight"], scale=s["scale"])


def _embed_grad_own(s):
    return _ms().embed_bwd(s["ids"], s["dy"], s["case"]["rows"], scale=s["scale"])


def _logp_own(s):
    k = s["case"]["top"]
    r = _ms().token_logprobs_fwd(s["logits"], s["targets"], top=k, scale=s["scale"])
    out = {"logprob": r["logprob"], "entropy": r["entropy"]}
    if k:
        out["top_id"], out["top_logprob"] = r["top_id"], r["top_logprob"]
    return out


def _logp_train_own(s):
    ms = _ms()
    r = ms.token_logprobs_fwd(s["logits"], s["targets"], scale=s["scale"])
    d = ms.token_logprobs_bwd(s["logits"], s["targets"], r["stats"], r["entropy"], s["dlogprob"],
                              s["dentropy"], scale=s["scale"])
    return {"logprob": r["logprob"], "entropy": r["entropy"], "dlogits": d}


_own = {"recur": _recur_own, "recur_train": _recur_train_own, "recur_step": _recur_step_own,
        "embed": _embed_own, "embed_grad": _embed_grad_own, "logp": _logp_own,
        "logp_train": _logp_train_own}


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    op, s = case["op"], SIZE[case["io"]]
    if op.startswith("recur"):
        gate = 1 if case["gate"] else 0
        if op == "recur_step":
            e = case["batch"] * case["d"]
            return {"bytes": e * (8 + s * (4 + gate)) + 4 * case["d"], "flops": 25 * e}
        e = case["batch"] * case["L"] * case["d"]
        state = 4 * case["batch"] * case["d"]
        small = 4 * case["d"] + (case["batch"] * case["L"] if case["reset"] else 0)
        if op == "recur":
            return {"bytes": e * s * (4 + gate) + small + state * (2 if case["start"] else 1),
                    "flops": 25 * e}
        # x r i [z] dy in, y dx dr di [dz] out
        return {"bytes": e * s * (8 + 2 * gate) + small + 4 * case["d"] +
                (3 * state if case["start"] else 0), "flops": 70 * e}
    if op.startswith("embed"):
        n, d = case["n"], case["d"]
        ids = n * (8 if case["ids"] == "i64" else 4)
        if op == "embed":  # a table row is read once, however often it is asked for
            return {"bytes": ids + (n + min(n, case["rows"])) * d * s, "flops": n * d}
        return {"bytes": ids + (n + case["rows"]) * d * s, "flops": 2 * n * d}
    e = case["rows"] * case["vocab"]
    if op == "logp":
        return {"bytes": e * s + case["rows"] * (16 + 8 * case["top"]), "flops": 6 * e}
    return {"bytes": 2 * e * s + case["rows"] * 24, "flops": 14 * e}


# ---- the definitions in 64 bits ------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "recur_step":
        t = {k: s[k].unsqueeze(1) if s[k] is not None else None for k in ("x", "r", "i", "z")}
        t |= {"lam": s["lam"], "h0": s["h"], "reset": None}
        h, _ = _exact_states(t)
        return {"y": _exact_gate(h, t["z"])[:, 0], "h": h[:, 0]}
    if op == "recur":
        h, _ = _exact_states(s)
        return {"y": _exact_gate(h, s["z"]), "h_last": h[:, -1].clone()}
    if op == "recur_train":
        return _exact_train(s)
    if op == "embed":
        return s["weight"].double()[s["ids"].long()] * s["scale"]
    if op == "embed_grad":
        dw = torch.zeros(case["rows"], case["d"], dtype=torch.float64, device=DEV)
        return dw.index_add_(0, s["ids"].long(), s["dy"].double()) * s["scale"]
    return _exact_logp(s)


def _exact_coeffs(s):
    x, r, i, lam = (s[k].double() for k in ("x", "r", "i", "lam"))
    rate = -SHARPNESS * torch.nn.functional.softplus(lam, threshold=700.0)
    la = rate * r.sigmoid()
    return x, r.sigmoid(), i.sigmoid(), rate, la, la.exp(), (-(2 * la).expm1()).sqrt()


def _exact_states(s):
    """Every h_t, one timestep after another; also the state before each."""
    x, _, si, _, _, a, norm = _exact_coeffs(s)
    if s["reset"] is not None:
        a = a * (1 - s["reset"].double()).unsqueeze(2)
    inp = norm * si * x
    del x, si, norm
    h = torch.empty_like(inp)
    now = s["h0"].double() if s["h0"] is not None else torch.zeros_like(inp[:, 0])
    start = now
    for t in range(h.shape[1]):
        torch.addcmul(inp[:, t], a[:, t], now, out=h[:, t])
        now = h[:, t]
    return h, start


def _exact_gate(h, z):
    return h if z is None else h * torch.nn.functional.silu(z.double())


def _exact_train(s):
    h, start = _exact_states(s)
    before = torch.cat([start.unsqueeze(1), h[:, :-1]], 1)
    x, sr, si, rate, la, a, norm = _exact_coeffs(s)
    live = torch.ones_like(a) if s["reset"] is None else \
        (1 - s["reset"].double()).unsqueeze(2).expand_as(a)
    dy = s["dy"].double()
    out = {"y": _exact_gate(h, s["z"])}
    if s["z"] is not None:
        z = s["z"].double()
        sz = z.sigmoid()
        out["dz"] = dy * h * (sz + z * sz * (1 - sz))
        dy = dy * z * sz
    g = torch.empty_like(h)
    now = s["dh_last"].double() if s["dh_last"] is not None else torch.zeros_like(h[:, 0])
    for t in range(h.shape[1] - 1, -1, -1):  # dL/dh_t
        g[:, t] = dy[:, t] + now
        now = g[:, t] * a[:, t] * live[:, t]
    if s["h0"] is not None:
        out["dh0"] = now
    out["dx"] = g * norm * si
    out["di"] = g * norm * x * si * (1 - si)
    dla = g * before * a * live - g * si * x * a * a / norm
    out["dr"] = dla * rate * sr * (1 - sr)
    out["dlam"] = (dla * sr).sum((0, 1)) * -SHARPNESS * s["lam"].double().sigmoid()
    return out


def _exact_logp(s):
    x = s["logits"].double() * s["scale"]
    logp = torch.log_softmax(x, dim=1)
    p = torch.softmax(x, dim=1)
    entropy = torch.special.entr(p).sum(1)
    out = {"logprob": logp.gather(1, s["targets"][:, None])[:, 0], "entropy": entropy}
    if s["case"]["op"] == "logp":
        if s["case"]["top"]:
            out["top_id"] = None
            out["top_logprob"] = torch.sort(logp, dim=1, descending=True).values[
                :, :s["case"]["top"]].clone()
        return out
    hot = torch.zeros_like(p).scatter_(1, s["targets"][:, None], 1.0)
    d = s["dlogprob"].double()[:, None] * (hot - p)
    # dH/dx_v = -p_v (log p_v + H), written with entr(p) = -p log p
    d += s["dentropy"].double()[:, None] * (torch.special.entr(p) - p * entropy[:, None])
    out["dlogits"] = d * s["scale"]
    return out
