"""Cases of the operators of a linear attention language model beside the scans: linear attention
with a decay for each head (forward, training pass, single token, drafted tokens), the group norm
of each token's channels with its gate, and the verification of drafted tokens.

Each case is timed in a plain form (elementary torch operations in fp32, rounded once at the end;
sums of decays and decisions in fp64) and, with ``own`` set, through the framework's entry points.
``exact`` is the definition in fp64.
"""
import math

import torch

own = False

DEV = "cuda"
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-5
CHUNK = 64  # tokens of a block of the plain forms


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # prefill of a layer of the 130M model's width as a state-space layer with scalar decays:
        # 24 heads of 64 channels share keys and queries of 128
        {"name": "attn_layer", "op": "attn", "batch": 8, "L": 2048, "heads": 24, "kheads": 1,
         "dk": 128, "dv": 64, "io": "bf16", "start": False, "reset": False, "fixed": False},
        # one long document continued from a state, heads of 128 with keys of their own: few
        # heads, the sequence has to be split
        {"name": "attn_long", "op": "attn", "batch": 1, "L": 131072, "heads": 12, "kheads": 12,
         "dk": 128, "dv": 128, "io": "bf16", "start": True, "reset": False, "fixed": True},
        # a training step's forward and backward, heads of 64 with keys of their own
        {"name": "attn_train", "op": "attn_train", "batch": 8, "L": 2048, "heads": 24,
         "kheads": 24, "dk": 64, "dv": 64, "io": "bf16", "start": False, "reset": False,
         "fixed": False},
        # training on packed documents in fp32: ragged length, sizes of no tile, shared keys,
        # resets, from a state
        {"name": "attn_train_packed", "op": "attn_train", "batch": 3, "L": 1999, "heads": 6,
         "kheads": 2, "dk": 40, "dv": 72, "io": "f32", "start": True, "reset": True,
         "fixed": False},
        # one decode step of the decode workload's batch
        {"name": "attn_step", "op": "attn_step", "batch": 256, "heads": 24, "kheads": 1,
         "dk": 128, "dv": 64, "tokens": 1, "io": "bf16"},
        # four drafted tokens and one more scored from the state, then the accepted ones taken in
        {"name": "attn_draft", "op": "attn_draft", "batch": 32, "heads": 24, "kheads": 1,
         "dk": 128, "dv": 64, "tokens": 5, "io": "bf16"},
        # the heads' outputs of a prefill normalised, with the layer's gate
        {"name": "norm_layer", "op": "norm", "rows": 16384, "groups": 24, "size": 64, "io": "bf16",
         "gate": True, "gate_first": False, "center": False, "bias": False},
        # the same in training, gate ahead of the norm, all channels one group
        {"name": "norm_train", "op": "norm_train", "rows": 16384, "groups": 1, "size": 1536,
         "io": "bf16", "gate": True, "gate_first": True, "center": False, "bias": False},
        # fp32, centred, with a bias, odd group size
        {"name": "norm_train_odd", "op": "norm_train", "rows": 5997, "groups": 7, "size": 73,
         "io": "f32", "gate": False, "gate_first": False, "center": True, "bias": True},
        # one token of one sequence: the launch
        {"name": "norm_token", "op": "norm", "rows": 1, "groups": 24, "size": 64, "io": "bf16",
         "gate": True, "gate_first": False, "center": False, "bias": False},
        # one request's four drafted tokens over a 50k vocabulary
        {"name": "verify_one", "op": "verify", "batch": 1, "tokens": 4, "vocab": 50280,
         "io": "f32", "pad": 0, "drafted": True, "warm": False},
        # a serving batch over a 128k vocabulary
        {"name": "verify_serve", "op": "verify", "batch": 64, "tokens": 4, "vocab": 131072,
         "io": "bf16", "pad": 0, "drafted": True, "warm": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _head_sizes(rng):
    """(heads, kheads, dk, dv)"""
    heads = _log(rng, 1, 32)
    kheads = rng.choice([heads, 1, rng.choice([k for k in range(1, heads + 1) if heads % k == 0])])
    size = lambda: rng.choice([64, 128, _log(rng, 8, 128), _log(rng, 8, 128)])  # noqa: E731
    return heads, kheads, size(), size()


def draw(rng):
    op = rng.choice(["attn", "attn", "attn_train", "attn_train", "attn_step", "attn_draft", "norm",
                     "norm_train", "norm_train", "verify", "verify"])
    io = rng.choice(["bf16", "bf16", "f32"])
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("attn", "attn_train"):
        heads, kheads, dk, dv = _head_sizes(rng)
        token = heads * (2 * dk + 2 * dv)
        most = 1 << 27 if op == "attn" else 1 << 26
        L = max(1, min(_log(rng, 1, 131072), most // token))
        batch = max(1, min(_log(rng, 1, 32), most // (token * L)))
        # states of the plain form's blocks: 1 GiB at the most
        while batch > 1 and batch * heads * -(-L // CHUNK) * dk * dv > 1 << 28:
            batch //= 2
        return {"op": op, "batch": batch, "L": L, "heads": heads, "kheads": kheads, "dk": dk,
                "dv": dv, "io": io, "start": flip(), "reset": rng.random() < 0.3,
                "fixed": rng.random() < 0.3}
    if op in ("attn_step", "attn_draft"):
        heads, kheads, dk, dv = _head_sizes(rng)
        batch = max(1, min(_log(rng, 1, 512), (1 << 26) // (heads * dk * dv)))
        return {"op": op, "batch": batch, "heads": heads, "kheads": kheads, "dk": dk, "dv": dv,
                "tokens": 1 if op == "attn_step" else _log(rng, 2, 16), "io": io}
    if op in ("norm", "norm_train"):
        size = rng.choice([64, 128, _log(rng, 4, 4096), _log(rng, 4, 4096)])
        groups = max(1, min(_log(rng, 1, 64), 8192 // size))
        rows = max(1, min(_log(rng, 1, 65536), (1 << 25) // (groups * size)))
        gate = flip()
        return {"op": op, "rows": rows, "groups": groups, "size": size, "io": io, "gate": gate,
                "gate_first": gate and flip(), "center": flip(), "bias": flip()}
    vocab, tokens = _log(rng, 256, 256000), _log(rng, 1, 12)
    batch = max(1, min(_log(rng, 1, 256), (1 << 26) // (vocab * (2 * tokens + 1))))
    return {"op": "verify", "batch": batch, "tokens": tokens, "vocab": vocab, "io": io,
            "pad": rng.choice([0, 0, (-vocab) % 8, 3]), "drafted": rng.random() < 0.8,
            "warm": flip()}


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

    if op.startswith("attn"):
        b, H, Hk, dk, dv = (case[k] for k in ("batch", "heads", "kheads", "dk", "dv"))
        L = case["L"] if "L" in case else case["tokens"]
        s["q"], s["k"] = normal(b, L, Hk, dk), normal(b, L, Hk, dk)
        s["v"] = normal(b, L, H, dv)
        s["scale"] = 1.0 / math.sqrt(dk)
        if case.get("fixed"):  # one decay a head, memories of 32 to 4096 tokens
            s["g"] = torch.log1p(-torch.exp2(-5 - 7 * uniform(H)))
        else:  # step sizes of 0.001 to 0.1 by rates of 1 to 16
            rate = torch.exp(uniform(H) * math.log(16.0))
            s["g"] = -rate * torch.exp(math.log(1e-3) + uniform(b, L, H) * math.log(100.0))
        if op in ("attn_step", "attn_draft"):
            s["h"] = normal(b, H, dk, dv, dtype=torch.float32)
            if op == "attn_draft":
                s["counts"] = torch.randint(1, L + 1, (b,), generator=g, device=DEV,
                                            dtype=torch.int32)
            return s
        s["h0"] = normal(b, H, dk, dv, dtype=torch.float32) if case["start"] else None
        s["reset"] = (uniform(b, L) < 1.0 / 256).to(torch.uint8) if case["reset"] else None
        if op == "attn_train":
            s["do"] = normal(b, L, H, dv)
            s["dh_last"] = normal(b, H, dk, dv, dtype=torch.float32) if case["start"] else None
        return s
    if op.startswith("norm"):
        rows, c = case["rows"], case["groups"] * case["size"]
        s["x"] = normal(rows, c, std=2.0)
        if case["center"]:
            s["x"] += normal(c)
        s["z"] = normal(rows, c) if case["gate"] else None
        s["weight"] = 1.0 + normal(c, std=0.2, dtype=torch.float32)
        s["bias"] = normal(c, std=0.2, dtype=torch.float32) if case["bias"] else None
        if op == "norm_train":
            s["dy"] = normal(rows, c)
        return s
    b, T, V = case["batch"], case["tokens"], case["vocab"]
    buf = normal(b, T + 1, V + case["pad"], std=2.5)
    s["logits"] = buf[..., :V]
    s["scale"] = 1.25 if case["warm"] else 1.0
    s["uniforms"] = uniform(b, T + 1)
    if case["drafted"]:  # the drafting model is near the target, and has drawn from its own
        s["draft_logits"] = (0.85 * s["logits"][:, :T].float() +
                             normal(b, T, V, std=1.0, dtype=torch.float32)).to(io)
        x = s["draft_logits"].float() * s["scale"]
    else:  # tokens looked up somewhere, mostly likely ones
        s["draft_logits"] = None
        x = s["logits"][:, :T].float() * 2.0
    noise = -torch.log(-torch.log(uniform(b, T, V).clamp_(1e-30, 1 - 1e-7)))
    s["drafts"] = (x + noise).argmax(-1)
    return s


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return (_own if own else _plain)[op](state)


def _scan_plain(A, B):
    """S_c = A_c S_{c-1} + B_c along dim 2, by doubling (inclusive, from zero)."""
    A, step = A.clone(), 1
    while step < A.shape[2]:
        B[:, :, step:] += A[:, :, step:] * B[:, :, :-step]
        A[:, :, step:] = A[:, :, step:] * A[:, :, :-step]
        step *= 2
    return B


def _blocks(x, size):
    """[b, L, H, d] -> [b, H, blocks, size, d] in fp32, padded with zeros."""
    b, L, H, d = x.shape
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, -L % size))
    return x.reshape(b, -1, size, H, d).permute(0, 3, 1, 2, 4)


def _flat(x, L):
    b, H, n, c, d = x.shape
    return x.permute(0, 2, 3, 1, 4).reshape(b, n * c, H, d)[:, :L]


def _decays(s, L, H):
    """Decays inside blocks, [b, H, blocks, size, ...]: from the keys to the queries, from the
    block's start to the queries, from the keys to its end, and from its start to its end."""
    b, g, reset = s["q"].shape[0], s["g"].double(), s.get("reset")
    size = min(CHUNK, L)
    g = _blocks64(g.expand(b, L, H) if g.dim() == 1 else g, size)
    G = torch.cumsum(g, -1)
    one = torch.ones((), device=DEV)
    if reset is None:
        start = torch.zeros_like(G, dtype=torch.int32)
    else:  # documents begun within the block
        start = torch.cumsum(_blocks64(reset.unsqueeze(-1).expand(b, L, H), size), -1).int()
    live = (start.unsqueeze(-1) == start.unsqueeze(-2)) & torch.ones(
        size, size, dtype=torch.bool, device=DEV).tril()
    D = torch.where(live, G.unsqueeze(-1) - G.unsqueeze(-2), -math.inf).float().exp()
    a = torch.where(start == 0, G.float().exp(), 0 * one)
    e = torch.where(start == start[..., -1:], (G[..., -1:] - G).float().exp(), 0 * one)
    return size, D, a, e, a[..., -1]


def _blocks64(x, size):
    b, L, H = x.shape
    x = torch.nn.functional.pad(x, (0, 0, 0, -L % size))
    return x.reshape(b, -1, size, H).permute(0, 3, 1, 2).double()


def _attn_blocks(s):
    L, H = s["v"].shape[1:3]
    r = H // s["q"].shape[2]
    size, D, a, e, gamma = _decays(s, L, H)
    q, k = (_blocks(s[n], size).repeat_interleave(r, 1) for n in ("q", "k"))
    v = _blocks(s["v"], size)
    if s.get("counts") is not None:  # what is not taken in adds nothing
        k = k * (torch.arange(L, device=DEV) < s["counts"][:, None])[:, None, None, :, None]
    own_states = (k * e.unsqueeze(-1)).transpose(-1, -2) @ v
    h0 = s.get("h0")
    if h0 is not None:
        own_states[:, :, 0] += gamma[:, :, 0, None, None] * h0
    after = _scan_plain(gamma[..., None, None], own_states)
    first = torch.zeros_like(after[:, :, :1]) if h0 is None else h0.unsqueeze(2)
    before = torch.cat([first, after[:, :, :-1]], 2)
    P = (q @ k.transpose(-1, -2)) * D
    o = (P @ v + a.unsqueeze(-1) * (q @ before)) * s["scale"]
    return L, r, size, D, a, e, gamma, q, k, v, before, after, P, o


def _attn_plain(s):
    L, *_, after, _, o = _attn_blocks(s)
    return {"o": _flat(o, L).to(s["v"].dtype), "h_last": after[:, :, -1].contiguous()}


def _attn_train_plain(s):
    L, r, size, D, a, e, gamma, q, k, v, before, after, P, o = _attn_blocks(s)
    io, scale = s["v"].dtype, s["scale"]
    out = {"o": _flat(o, L).to(io)}
    do = _blocks(s["do"], size) * scale
    # gradients of the states at the blocks' ends, from what comes behind
    own_grads = (q * a.unsqueeze(-1)).transpose(-1, -2) @ do
    last = s["dh_last"].unsqueeze(2) if s["dh_last"] is not None else \
        torch.zeros_like(own_grads[:, :, :1])
    own_grads[:, :, -1:] += gamma[:, :, -1:, None, None] * last
    grads = _scan_plain(gamma.flip(2)[..., None, None], own_grads.flip(2)).flip(2)
    R = torch.cat([grads[:, :, 1:], last], 2)
    dP = (do @ v.transpose(-1, -2)) * D
    dv = P.transpose(-1, -2) @ do + e.unsqueeze(-1) * (k @ R)
    aSdo = a.unsqueeze(-1) * (do @ before.transpose(-1, -2))
    eRv = e.unsqueeze(-1) * (v @ R.transpose(-1, -2))
    dq = dP @ k + aSdo
    dk = dP.transpose(-1, -2) @ q + eRv
    M = P * (do @ v.transpose(-1, -2))
    later = M.sum(-1) - M.sum(-2) + (q * aSdo).sum(-1)
    earlier = (k * eRv).sum(-1)
    dg = later.flip(-1).cumsum(-1).flip(-1) + earlier.cumsum(-1) - earlier + \
        (gamma * (R * before).sum((-1, -2))).unsqueeze(-1)
    dg = _flat(dg.unsqueeze(-1), L).squeeze(-1)
    if s["reset"] is not None:
        dg = dg * (1 - s["reset"].float()).unsqueeze(-1)
    b = dq.shape[0]
    shared = lambda x: _flat(x, L).reshape(b, L, -1, r, x.shape[-1]).sum(3).to(io)  # noqa: E731
    out |= {"dq": shared(dq), "dk": shared(dk), "dv": _flat(dv, L).to(io)}
    out["dg"] = dg.double().sum((0, 1)).float() if s["g"].dim() == 1 else dg
    if s["h0"] is not None:
        out["dh0"] = grads[:, :, 0].contiguous()
    return out


def _attn_step_plain(s):
    L, *_, after, _, o = _attn_blocks(s | {"h0": s["h"]})
    s["h"].copy_(after[:, :, -1])
    return {"o": _flat(o, L).to(s["v"].dtype), "h": s["h"]}


def _attn_draft_plain(s):
    L, *_, o = _attn_blocks(s | {"h0": s["h"], "counts": None})
    taken = torch.arange(L, device=DEV) < s["counts"][:, None]
    *_, after, _, _ = _attn_blocks(s | {"h0": s["h"], "g": s["g"] * taken.unsqueeze(-1)})
    s["h"].copy_(after[:, :, -1])
    return {"o": _flat(o, L).to(s["v"].dtype), "h": s["h"]}


def _norm_parts(s):
    """x (gated first or not) in groups, what is normalised of it, and the factor of that."""
    case = s["case"]
    shape = (case["rows"], case["groups"], case["size"])
    x = s["x"].float().reshape(shape)
    z = s["z"].float().reshape(shape) if s["z"] is not None else None
    if case["gate_first"]:
        x = x * (z * torch.sigmoid(z))
    c = x - x.mean(-1, keepdim=True) if case["center"] else x
    factor = torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS)
    return shape, z, c * factor, factor


def _norm_plain(s):
    shape, z, xhat, _ = _norm_parts(s)
    y = xhat * s["weight"].reshape(shape[1:])
    if s["bias"] is not None:
        y = y + s["bias"].reshape(shape[1:])
    if z is not None and not s["case"]["gate_first"]:
        y = y * (z * torch.sigmoid(z))
    return y.reshape(s["x"].shape).to(s["x"].dtype)


def _norm_train_plain(s):
    case, io = s["case"], s["x"].dtype
    shape, z, xhat, factor = _norm_parts(s)
    w = s["weight"].reshape(shape[1:])
    dy = s["dy"].float().reshape(shape)
    out = {"y": _norm_plain(s)}
    sz = torch.sigmoid(z) if z is not None else None
    after = z is not None and not case["gate_first"]
    if after:
        pre = xhat * w
        if s["bias"] is not None:
            pre = pre + s["bias"].reshape(shape[1:])
        dz = dy * pre * sz * (1 + z * (1 - sz))
        dy = dy * (z * sz)
    out["dweight"] = (dy * xhat).sum(0).flatten()
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0).flatten()
    d = dy * w
    dx = d - xhat * (d * xhat).mean(-1, keepdim=True)
    if case["center"]:
        dx = dx - d.mean(-1, keepdim=True)
    dx = dx * factor
    if case["gate_first"]:
        x = s["x"].float().reshape(shape)
        dz = dx * x * sz * (1 + z * (1 - sz))
        dx = dx * (z * sz)
    out["dx"] = dx.reshape(s["x"].shape).to(io)
    if z is not None:
        out["dz"] = dz.reshape(s["x"].shape).to(io)
    return out


def _verify_plain(s):
    # whether a number lies this side of a border or that: in fp64
    x = s["logits"].double() * s["scale"]
    b, T1, V = x.shape
    T = T1 - 1
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    ids = s["drafts"].long().unsqueeze(-1)
    if s["draft_logits"] is not None:
        y = s["draft_logits"].double() * s["scale"]
        q = torch.exp(y - y.amax(-1, keepdim=True))
        q = q / q.sum(-1, keepdim=True)
    else:
        q = torch.zeros_like(p[:, :T]).scatter_(-1, ids, 1.0)
    u = s["uniforms"].double()
    taken = u[:, :T] * q.gather(-1, ids).squeeze(-1) < p[:, :T].gather(-1, ids).squeeze(-1)
    count = taken.long().cumprod(-1).sum(-1)
    # what is left of the target's where the first draft was refused, or behind the last one
    q = torch.cat([q, torch.zeros_like(p[:, :1])], 1)
    row = count.view(b, 1, 1).expand(b, 1, V)
    left = (p.gather(1, row) - q.gather(1, row)).clamp_min(0).squeeze(1)
    sums = left.cumsum(-1)
    border = u[:, T:] * sums[:, -1:]
    drawn = (sums <= border).sum(-1)
    at = torch.arange(T1, device=DEV)
    ids = torch.cat([s["drafts"].long(), torch.zeros_like(ids[:, :1, 0])], 1)
    tokens = torch.where(at < count[:, None], ids, -1)
    tokens = torch.where(at == count[:, None], drawn[:, None], tokens)
    chosen = p.gather(-1, tokens.clamp_min(0).unsqueeze(-1)).squeeze(-1).log()
    logprob = torch.where(tokens >= 0, chosen, 0.0).float()
    return {"tokens": tokens.int(), "count": count.int(), "logprob": logprob}


_plain = {"attn": _attn_plain, "attn_train": _attn_train_plain, "attn_step": _attn_step_plain,
          "attn_draft": _attn_draft_plain, "norm": _norm_plain, "norm_train": _norm_train_plain,
          "verify": _verify_plain}


def _ms():
    import selective_state_space_81_amd as ms
    return ms


def _attn_own(s):
    b, _, H, dv = s["v"].shape
    h_last = torch.empty(b, H, s["k"].shape[3], dv, dtype=torch.float32, device=DEV)
    o = _ms().linear_attn_fwd(s["q"], s["k"], s["v"], s["g"], scale=s["scale"], reset=s["reset"],
                              h0=s["h0"], h_last=h_last)
    return {"o": o, "h_last": h_last}


def _attn_train_own(s):
    ms = _ms()
    states = ms.linear_attn_states(s["k"], s["v"])
    o = ms.linear_attn_fwd(s["q"], s["k"], s["v"], s["g"], scale=s["scale"], reset=s["reset"],
                           h0=s["h0"], states=states)
    g = ms.linear_attn_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], states, scale=s["scale"],
                           reset=s["reset"], dh_last=s["dh_last"], want_dh0=s["h0"] is not None)
    out = {"o": o, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"], "dg": g["dg"]}
    if s["h0"] is not None:
        out["dh0"] = g["dh0"]
    return out


def _attn_step_own(s):
    o = _ms().linear_attn_step(s["h"], s["q"], s["k"], s["v"], s["g"], scale=s["scale"])
    return {"o": o, "h": s["h"]}


def _attn_draft_own(s):
    ms = _ms()
    o = ms.linear_attn_step(s["h"], s["q"], s["k"], s["v"], s["g"], scale=s["scale"],
                            update=False)
    ms.linear_attn_step(s["h"], None, s["k"], s["v"], s["g"], counts=s["counts"])
    return {"o": o, "h": s["h"]}


def _norm_args(s):
    case = s["case"]
    return {"bias": s["bias"], "z": s["z"], "center": case["center"],
            "gate_first": case["gate_first"], "eps": EPS}


def _norm_own(s):
    return _ms().group_norm_fwd(s["x"], s["case"]["groups"], s["weight"], **_norm_args(s))


def _norm_train_own(s):
    ms = _ms()
    y = _norm_own(s)
    g = ms.group_norm_bwd(s["x"], s["dy"], s["case"]["groups"], s["weight"], **_norm_args(s))
    out = {"y": y, "dx": g["dx"], "dweight": g["dweight"]}
    if s["bias"] is not None:
        out["dbias"] = g["dbias"]
    if s["z"] is not None:
        out["dz"] = g["dz"]
    return out


def _verify_own(s):
    r = _ms().verify_drafts(s["logits"], s["drafts"], s["uniforms"], s["draft_logits"],
                            scale=s["scale"])
    return {"tokens": r["tokens"], "count": r["count"], "logprob": r["logprob"]}


_own = {"attn": _attn_own, "attn_train": _attn_train_own, "attn_step": _attn_step_own,
        "attn_draft": _attn_draft_own, "norm": _norm_own, "norm_train": _norm_train_own,
        "verify": _verify_own}


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    op, s = case["op"], SIZE[case["io"]]
    if op.startswith("attn"):
        b, H, Hk, dk, dv = (case[k] for k in ("batch", "heads", "kheads", "dk", "dv"))
        n = b * (case["L"] if "L" in case else case["tokens"])
        qk, v, state = n * Hk * dk * s, n * H * dv * s, 4 * b * H * dk * dv
        decays = 4 * H if case.get("fixed") else 4 * n * H
        product = 2 * n * H * dk * dv
        if op == "attn_step":
            return {"bytes": 2 * qk + 2 * v + decays + 2 * state, "flops": 2 * product}
        if op == "attn_draft":  # scored from the state, then the state read and written
            return {"bytes": 2 * qk + 2 * v + decays + 2 * state + 4 * b, "flops": 2 * product}
        more = n // H if case["reset"] else 0
        if op == "attn":
            return {"bytes": 2 * qk + 2 * v + decays + more + state * (2 if case["start"] else 1),
                    "flops": 2 * product}
        # q k v g do in, o dq dk dv dg out
        return {"bytes": 4 * qk + 4 * v + 2 * decays + more + (3 * state if case["start"] else 0),
                "flops": 7 * product}
    if op.startswith("norm"):
        e, c = case["rows"] * case["groups"] * case["size"], case["groups"] * case["size"]
        gate, small = 1 if case["gate"] else 0, 8 * c if case["bias"] else 4 * c
        if op == "norm":
            return {"bytes": e * s * (2 + gate) + small, "flops": 8 * e}
        return {"bytes": e * s * (4 + 2 * gate) + 2 * small, "flops": 25 * e}
    rows = case["batch"] * (case["tokens"] + 1 + (case["tokens"] if case["drafted"] else 0))
    e = rows * case["vocab"]
    return {"bytes": e * s + case["batch"] * (case["tokens"] + 1) * 24, "flops": 3 * e}


# ---- the definitions in 64 bits ------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attn_train":
        return _exact_attn_train(s)
    if op.startswith("attn"):
        return _exact_attn(s)
    if op.startswith("norm"):
        return _exact_norm(s)
    return _exact_verify(s)


def _exact_inputs(s):
    """q, k, v [L, b, H, d] and the decays [L, b, H, 1, 1], 0 where a document starts."""
    b, L, H, _ = s["v"].shape
    r = H // s["k"].shape[2]
    q, k = (torch.repeat_interleave(s[n].double(), r, dim=2).transpose(0, 1) for n in ("q", "k"))
    keep = torch.exp(s["g"].double()).expand(b, L, H)
    if s.get("reset") is not None:
        keep = keep * (s["reset"] == 0)[..., None]
    return q * s["scale"], k, s["v"].double().transpose(0, 1), keep.transpose(0, 1)[..., None, None]


def _exact_attn(s):
    """One token after another."""
    q, k, v, keep = _exact_inputs(s)
    name = "h" if "h" in s else "h_last"
    start = s.get("h", s.get("h0"))
    now = torch.zeros(k.shape[1:] + v.shape[-1:], dtype=torch.float64, device=DEV) \
        if start is None else start.double()
    if k.shape[0] * now.numel() > 1 << 37:
        return None
    o = torch.empty_like(v)
    final = now
    for t in range(k.shape[0]):
        now = torch.addcmul(now * keep[t], k[t, ..., None], v[t, :, :, None, :])
        torch.sum(q[t, ..., None] * now, dim=-2, out=o[t])
        if "counts" in s:
            final = torch.where((s["counts"] > t).view(-1, 1, 1, 1), now, final)
        else:
            final = now
    return {"o": o.transpose(0, 1), name: final}


def _exact_attn_train(s):
    q, k, v, keep = _exact_inputs(s)
    L, b, H, dk = k.shape
    if L * b * H * dk * v.shape[-1] > 3 << 30:  # every state is kept, and its gradient
        return None
    S = k[..., None] * v[..., None, :]
    start = s["h0"].double() if s["h0"] is not None else torch.zeros_like(S[0])
    now = start
    for t in range(L):
        S[t] += keep[t] * now
        now = S[t]
    do = s["do"].double().transpose(0, 1)
    out = {"o": (q[..., None] * S).sum(-2), "dq": (S * do[..., None, :]).sum(-1) * s["scale"]}
    R = q[..., None] * do[..., None, :]  # dL/dS_t
    now = s["dh_last"].double() if s["dh_last"] is not None else torch.zeros_like(R[0])
    for t in range(L - 1, -1, -1):
        R[t] += now
        now = keep[t] * R[t]
    if s["h0"] is not None:
        dh0 = now
    out["dk"] = (R * v[..., None, :]).sum(-1)
    out["dv"] = (R * k[..., None]).sum(-2)
    dg = torch.empty(L, b, H, dtype=torch.float64, device=DEV)
    dg[0] = (R[0] * start).sum((-1, -2))
    for t in range(1, L):
        dg[t] = (R[t] * S[t - 1]).sum((-1, -2))
    dg *= keep[..., 0, 0]
    for name in ("dq", "dk"):
        out[name] = out[name].unflatten(2, (s["k"].shape[2], -1)).sum(3)
    out = {n: x.transpose(0, 1) for n, x in out.items()}
    out["dg"] = dg.sum((0, 1)) if s["g"].dim() == 1 else dg.transpose(0, 1)
    if s["h0"] is not None:
        out["dh0"] = dh0
    return out


def _exact_norm(s):
    case = s["case"]
    n = case["size"]
    view = lambda t: t.double().unflatten(-1, (case["groups"], n))  # noqa: E731
    x, w = view(s["x"]), view(s["weight"])
    gate = slope = 1.0
    if s["z"] is not None:
        z = view(s["z"])
        gate = torch.nn.functional.silu(z)
        sig = z.sigmoid()
        slope = sig + gate * (1 - sig)
    inside = x * gate if case["gate_first"] else x
    mean = inside.mean(-1, keepdim=True) if case["center"] else 0.0
    dev = ((inside - mean).square().sum(-1, keepdim=True) / n + EPS).sqrt()
    hat = (inside - mean) / dev
    pre = hat * w + (view(s["bias"]) if s["bias"] is not None else 0.0)
    y = pre if case["gate_first"] else pre * gate
    if case["op"] == "norm":
        return y.flatten(-2)
    dy = view(s["dy"])
    out = {"y": y}
    dpre = dy if case["gate_first"] else dy * gate
    out["dweight"] = (dpre * hat).sum(0)
    if s["bias"] is not None:
        out["dbias"] = dpre.sum(0)
    dhat = dpre * w
    din = dhat - hat * (dhat * hat).sum(-1, keepdim=True) / n
    if case["center"]:
        din = din - dhat.sum(-1, keepdim=True) / n
    din = din / dev
    out["dx"] = din * gate if case["gate_first"] else din
    if s["z"] is not None:
        out["dz"] = (din * x if case["gate_first"] else dy * pre) * slope
    return {k: t.flatten(-2) for k, t in out.items()}


def _exact_verify(s):
    """One sequence and one draft after another."""
    logp = torch.log_softmax(s["logits"].double() * s["scale"], -1)
    b, T1, V = logp.shape
    logq = None if s["draft_logits"] is None else \
        torch.log_softmax(s["draft_logits"].double() * s["scale"], -1)
    drafts, uniforms = s["drafts"].tolist(), s["uniforms"].double().tolist()
    at = s["drafts"].unsqueeze(-1)
    of_p = logp[:, :-1].gather(-1, at).squeeze(-1).exp().tolist()
    of_q = [[1.0] * (T1 - 1)] * b if logq is None else logq.gather(-1, at).squeeze(-1).exp().tolist()
    out = torch.zeros(b, T1, dtype=torch.float64, device=DEV)
    for i in range(b):
        t = 0
        while t < T1 - 1 and uniforms[i][t] * of_q[i][t] < of_p[i][t]:
            out[i, t] = logp[i, t, drafts[i][t]]
            t += 1
        rest = logp[i, t].exp()
        if t < T1 - 1:
            if logq is None:
                rest[drafts[i][t]] = 0.0
            else:
                rest = torch.relu(rest - logq[i, t].exp())
        mass = torch.cumsum(rest, 0)
        drawn = torch.searchsorted(mass, mass[-1:] * uniforms[i][-1], right=True)
        out[i, t] = logp[i, t, drawn].squeeze()
    return {"tokens": None, "count": None, "logprob": out}
