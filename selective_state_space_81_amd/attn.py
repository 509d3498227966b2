"""The operators of a linear attention language model: linear attention with a
decay for each head, the group norm of each token's channels with its gate, and
the verification of drafted tokens.  Argument marshalling only, as in ``lm``
(which has the calls' streams, buffers and refusals): the work is done by the
HIP kernels behind ``include/msscan.h``.

Raw calls (``*_fwd``, ``*_bwd``, ``linear_attn_step``, ``verify_drafts``) take and
return device tensors; ``linear_attn`` and ``group_norm`` are the same as
differentiable torch operations.
"""
from __future__ import annotations

import ctypes
import functools

import selective_state_space_81_amd as ms

from . import lm

EXPORTS = ("ms_linear_attn_workspace_bytes", "ms_linear_attn_states_bytes", "ms_linear_attn_fwd",
           "ms_linear_attn_bwd_workspace_bytes", "ms_linear_attn_bwd", "ms_linear_attn_step",
           "ms_group_norm_fwd", "ms_group_norm_bwd_workspace_bytes", "ms_group_norm_bwd",
           "ms_verify_drafts_workspace_bytes", "ms_verify_drafts")

MAX_HEAD_DIM = 128  # of dk and dv
MAX_STEP_TOKENS = 64
MAX_DRAFTS = 64


def declare(lib) -> None:
    """Argument types of this module's entry points."""
    vp, f32, sz = ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
    i32, i64 = ctypes.c_int32, ctypes.c_int64
    heads = [i32, i64] + [i32] * 5  # batch, seqlen, heads, kheads, dk, dv, io
    qkv = [vp, i64] * 3 + [vp, i32, f32]  # with g, fixed and scale
    for name, res, args in (
            ("ms_linear_attn_workspace_bytes", sz, heads),
            ("ms_linear_attn_states_bytes", sz, [i32, i64] + [i32] * 4),
            ("ms_linear_attn_fwd", ctypes.c_int, qkv + [vp] * 5 + heads + [vp, sz, vp]),
            ("ms_linear_attn_bwd_workspace_bytes", sz, [i32, i64] + [i32] * 6),
            ("ms_linear_attn_bwd", ctypes.c_int, qkv + [vp] * 9 + heads + [vp, sz, vp]),
            ("ms_linear_attn_step", ctypes.c_int,
             [vp] + qkv + [vp, i32, vp] + [i32] * 7 + [vp]),
            ("ms_group_norm_fwd", ctypes.c_int,
             [vp, i64, vp, vp, vp, i64, i32, i32, f32, vp, i64, i32, i32, i32, vp]),
            ("ms_group_norm_bwd_workspace_bytes", sz, [i64, i32, i32, i32]),
            ("ms_group_norm_bwd", ctypes.c_int,
             [vp, i64, vp, vp, vp, i64, i32, i32, f32] + [vp] * 5 + [i64, i32, i32, i32, vp, sz, vp]),
            ("ms_verify_drafts_workspace_bytes", sz, [i32, i32, i64, i32, i32]),
            ("ms_verify_drafts", ctypes.c_int,
             [vp, i64, vp, i64, vp, i32, vp, f32, vp, vp, vp, i32, i32, i64, i32, vp, sz, vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args


def _pitch(m, t, name, dims, inner, text, like=None):
    """(distance of the rows, io code) of a device tensor whose last `inner`
    dimensions are a contiguous row, in like's dtype and on its device."""
    code = m.pitch(t, dims, inner)
    if code < 0:
        if not getattr(t, "is_cuda", False) or t.dim() != dims:
            raise ValueError(f"{name} must be a {text} device tensor")
        ms._io(t)
        raise ValueError(f"{name} must be contiguous, or a slice of rows that are evenly apart")
    if like is not None:
        if t.dtype != like.dtype:
            raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
        if t.device != like.device:
            raise ValueError(f"{name} is on {t.device}, not on {like.device}")
    return code >> 1, code & 1


def _need(**given):
    for name, t in given.items():
        if t is None:
            raise ValueError(f"{name} is required")


# ---- linear attention --------------------------------------------------------------------

def _chk_heads(m, q, k, v, g, reset=None):
    """Checks of what the passes share: (sizes, pitches of q, k and v, fixed, reset)."""
    import torch
    _need(k=k, v=v, g=g)
    ldk, io = _pitch(m, k, "k", 4, 2, "[batch, L, kheads, dk]")
    ldv, _ = _pitch(m, v, "v", 4, 2, "[batch, L, heads, dv]", k)
    b, L, hk, dk = k.shape
    h, dv = v.shape[2:]
    if v.shape[:2] != k.shape[:2]:
        raise ValueError(f"v must have shape {(b, L)} ahead of its heads, got {tuple(v.shape[:2])}")
    ldq = 0
    if q is not None:
        ldq, _ = _pitch(m, q, "q", 4, 2, "[batch, L, kheads, dk]", k)
        if q.shape != k.shape:
            raise ValueError(f"q must have shape {tuple(k.shape)}, got {tuple(q.shape)}")
    fixed = g.dim() == 1
    if not m.fits(k, torch.float32, (h,) if fixed else (b, L, h), g):
        lm._refuse(k.device, torch.float32, (h,) if fixed else (b, L, h), g=g)
    if reset is not None:
        if reset.dtype == torch.bool:
            reset = reset.view(torch.uint8)
        if not m.fits(k, torch.uint8, (b, L), reset):
            lm._refuse(k.device, torch.uint8, (b, L), reset=reset)
    return (b, L, h, hk, dk, dv, io), (ldq, ldk, ldv), int(fixed), reset


@functools.lru_cache(maxsize=1024)
def linear_attn_workspace_bytes(batch: int, seqlen: int, heads: int, kheads: int, dk: int,
                                dv: int, io: int) -> int:
    """ms_linear_attn_workspace_bytes: workspace of linear_attn_fwd."""
    return lm._size(ms.load().ms_linear_attn_workspace_bytes(batch, seqlen, heads, kheads, dk, dv,
                                                             io), "the linear attention")


@functools.lru_cache(maxsize=1024)
def linear_attn_bwd_workspace_bytes(batch: int, seqlen: int, heads: int, kheads: int, dk: int,
                                    dv: int, fixed: int, io: int) -> int:
    """ms_linear_attn_bwd_workspace_bytes: workspace of linear_attn_bwd."""
    return lm._size(ms.load().ms_linear_attn_bwd_workspace_bytes(
        batch, seqlen, heads, kheads, dk, dv, fixed, io), "the linear attention's backward")


@functools.lru_cache(maxsize=1024)
def linear_attn_states_bytes(batch: int, seqlen: int, heads: int, dk: int, dv: int,
                             io: int) -> int:
    """ms_linear_attn_states_bytes: what the forward keeps for the backward."""
    return lm._size(ms.load().ms_linear_attn_states_bytes(batch, seqlen, heads, dk, dv, io),
                    "the linear attention's states")


def linear_attn_states(k, v, stream=None):
    """An empty buffer for the states that linear_attn_fwd saves for
    linear_attn_bwd (its order is the kernels' own)."""
    import torch
    m = lm._marshal()
    _, io = _pitch(m, k, "k", 4, 2, "[batch, L, kheads, dk]")
    _pitch(m, v, "v", 4, 2, "[batch, L, heads, dv]", k)
    n = linear_attn_states_bytes(k.shape[0], k.shape[1], v.shape[2], k.shape[3], v.shape[3], io)
    return lm._Call(m, k, stream).empty(torch.float32, n // 4)


def _chk_states(m, k, states, sizes):
    import torch
    b, L, h, _, dk, dv, io = sizes
    n = linear_attn_states_bytes(b, L, h, dk, dv, io) // 4
    if not m.fits(k, torch.float32, (n,), states):
        lm._refuse(k.device, torch.float32, (n,), states=states)


def linear_attn_fwd(q, k, v, g, *, scale=1.0, reset=None, o=None, h0=None, h_last=None,
                    states=None, workspace=None, stream=None):
    """ms_linear_attn_fwd on torch device tensors: linear attention of q and k
    [batch, L, kheads, dk] and v [batch, L, heads, dv] with log decays g
    ([batch, L, heads] or [heads], fp32), from the state h0 [batch, heads, dk,
    dv].  kheads divides heads.  reset [batch, L] (uint8 or bool) starts new
    sequences; states (linear_attn_states) receives what the backward needs.
    q, k and v may be column slices of wider tensors.  Allocates o (and the
    workspace) when not given.  Returns o."""
    import torch
    m = lm._marshal()
    _need(q=q)
    sizes, (ldq, ldk, ldv), fixed, reset = _chk_heads(m, q, k, v, g, reset)
    b, L, h, hk, dk, dv, io = sizes
    f32 = torch.float32
    if not m.fits(k, f32, (b, h, dk, dv), h0, h_last):
        lm._refuse(k.device, f32, (b, h, dk, dv), h0=h0, h_last=h_last)
    if states is not None:
        _chk_states(m, k, states, sizes)
    if o is not None and not m.fits(k, k.dtype, (b, L, h, dv), o):
        lm._refuse(k.device, k.dtype, (b, L, h, dv), o=o)
    need = linear_attn_workspace_bytes(*sizes)
    call = lm._Call(m, k, stream)
    if o is None:
        o = call.empty(k.dtype, b, L, h, dv)
    ws, wn = call.workspace(workspace, need)
    call.run(m.linear_attn_fwd, q, ldq, k, ldk, v, ldv, g, fixed, scale, reset, o, h0, h_last,
             states, *sizes, ws, wn)
    return o


def linear_attn_bwd(q, k, v, g, do, states, *, scale=1.0, reset=None, dh_last=None,
                    workspace=None, stream=None, want_dh0=True):
    """ms_linear_attn_bwd on torch device tensors: gradients of
    linear_attn_fwd for do [batch, L, heads, dv] (and optionally dh_last), with
    the states it saved.  Returns a dict: dq, dk, dv (io dtype), dg (fp32, of
    g's shape) and dh0 (fp32)."""
    import torch
    m = lm._marshal()
    _need(q=q, do=do, states=states)
    sizes, (ldq, ldk, ldv), fixed, reset = _chk_heads(m, q, k, v, g, reset)
    b, L, h, hk, dk, dv, io = sizes
    f32, dt = torch.float32, k.dtype
    _chk_states(m, k, states, sizes)
    if not m.fits(k, dt, (b, L, h, dv), do):
        lm._refuse(k.device, dt, (b, L, h, dv), do=do)
    if not m.fits(k, f32, (b, h, dk, dv), dh_last):
        lm._refuse(k.device, f32, (b, h, dk, dv), dh_last=dh_last)
    need = linear_attn_bwd_workspace_bytes(b, L, h, hk, dk, dv, fixed, io)
    call = lm._Call(m, k, stream)
    out = {"dq": call.empty(dt, b, L, hk, dk), "dk": call.empty(dt, b, L, hk, dk),
           "dv": call.empty(dt, b, L, h, dv), "dg": call.empty(f32, *g.shape),
           "dh0": call.empty(f32, b, h, dk, dv) if want_dh0 else None}
    ws, wn = call.workspace(workspace, need)
    call.run(m.linear_attn_bwd, q, ldq, k, ldk, v, ldv, g, fixed, scale, reset, states, do,
             dh_last, out["dq"], out["dk"], out["dv"], out["dg"], out["dh0"], *sizes, ws, wn)
    return out


def linear_attn_step(h, q, k, v, g, *, scale=1.0, counts=None, update=True, o=None, stream=None):
    """ms_linear_attn_step on torch device tensors: the next tokens (1 to 64)
    of every sequence, q and k [batch, tokens, kheads, dk], v [batch, tokens,
    heads, dv], from the state h [batch, heads, dk, dv] (fp32), which is updated
    in place unless update is False.  counts [batch] (int32): how many of the
    tokens are there in each row; rows of o behind them are not written.  With q
    None only the state moves on.  Returns o (None without q)."""
    import torch
    m = lm._marshal()
    _need(h=h)
    sizes, (ldq, ldk, ldv), fixed, _ = _chk_heads(m, q, k, v, g)
    b, L, heads, hk, dk, dv, io = sizes
    if not m.fits(k, torch.float32, (b, heads, dk, dv), h):
        lm._refuse(k.device, torch.float32, (b, heads, dk, dv), h=h)
    if not m.fits(k, torch.int32, (b,), counts):
        lm._refuse(k.device, torch.int32, (b,), counts=counts)
    if o is not None and not m.fits(k, k.dtype, (b, L, heads, dv), o):
        lm._refuse(k.device, k.dtype, (b, L, heads, dv), o=o)
    call = lm._Call(m, k, stream)
    if q is None:
        o = None
    elif o is None:
        o = call.empty(k.dtype, b, L, heads, dv)
    call.run(m.linear_attn_step, h, q, ldq, k, ldk, v, ldv, g, fixed, scale, counts, int(update), o,
             *sizes)
    return o


# ---- group norm ----------------------------------------------------------------------------

def _chk_norm(m, x, groups, weight, bias, z):
    import torch
    ldx, io = _pitch(m, x, "x", x.dim(), 1, "[..., channels]")
    c = x.shape[-1]
    if groups < 1 or c % groups:
        raise ValueError(f"groups={groups} must divide the {c} channels")
    ldz = 0
    if z is not None:
        ldz, _ = _pitch(m, z, "z", x.dim(), 1, "[..., channels]", x)
        if z.shape != x.shape:
            raise ValueError(f"z must have shape {tuple(x.shape)}, got {tuple(z.shape)}")
    if not m.fits(x, torch.float32, (c,), weight, bias):
        lm._refuse(x.device, torch.float32, (c,), weight=weight, bias=bias)
    return x.numel() // c if c else 0, c // groups, ldx, ldz, io


def group_norm_fwd(x, groups, weight=None, bias=None, z=None, *, center=True, gate_first=False,
                   eps=1e-5, y=None, stream=None):
    """ms_group_norm_fwd on torch device tensors: the norm of x [..., channels]
    over each of `groups` groups of a row's channels (mean taken off with
    center), times weight plus bias ([channels] fp32), and with z (of x's shape)
    times silu(z), or of x silu(z) with gate_first.  x and z may be column slices
    of wider tensors.  Allocates y when not given.  Returns y."""
    m = lm._marshal()
    rows, size, ldx, ldz, io = _chk_norm(m, x, groups, weight, bias, z)
    if y is not None and not m.fits(x, x.dtype, tuple(x.shape), y):
        lm._refuse(x.device, x.dtype, tuple(x.shape), y=y)
    call = lm._Call(m, x, stream)
    if y is None:
        y = call.empty(x.dtype, *x.shape)
    call.run(m.group_norm_fwd, x, ldx, weight, bias, z, ldz, int(center), int(gate_first), eps, y,
             rows, groups, size, io)
    return y


@functools.lru_cache(maxsize=1024)
def group_norm_bwd_workspace_bytes(rows: int, groups: int, size: int, io: int) -> int:
    """ms_group_norm_bwd_workspace_bytes: workspace of group_norm_bwd."""
    return lm._size(ms.load().ms_group_norm_bwd_workspace_bytes(rows, groups, size, io),
                    "the group norm's backward")


def group_norm_bwd(x, dy, groups, weight=None, bias=None, z=None, *, center=True,
                   gate_first=False, eps=1e-5, workspace=None, stream=None, want_dweight=True,
                   want_dbias=True):
    """ms_group_norm_bwd on torch device tensors: gradients of group_norm_fwd
    for dy (of x's shape).  Returns a dict: dx, dz (io dtype; dz None without
    z), dweight and dbias (fp32; None where the argument was, or it is not
    wanted)."""
    import torch
    m = lm._marshal()
    _need(dy=dy)
    rows, size, ldx, ldz, io = _chk_norm(m, x, groups, weight, bias, z)
    if not m.fits(x, x.dtype, tuple(x.shape), dy):
        lm._refuse(x.device, x.dtype, tuple(x.shape), dy=dy)
    want_dweight, want_dbias = want_dweight and weight is not None, want_dbias and bias is not None
    need = group_norm_bwd_workspace_bytes(rows, groups, size, io)
    call = lm._Call(m, x, stream)
    f32, c = torch.float32, x.shape[-1]
    out = {"dx": call.empty(x.dtype, *x.shape),
           "dz": call.empty(x.dtype, *x.shape) if z is not None else None,
           "dweight": call.empty(f32, c) if want_dweight else None,
           "dbias": call.empty(f32, c) if want_dbias else None}
    if not (want_dweight or want_dbias):
        need = 0
    ws, wn = call.workspace(workspace, need)
    call.run(m.group_norm_bwd, x, ldx, weight, bias, z, ldz, int(center), int(gate_first), eps, dy,
             out["dx"], out["dz"], out["dweight"], out["dbias"], rows, groups, size, io, ws, wn)
    return out


# ---- verification of drafted tokens ------------------------------------------------------------

@functools.lru_cache(maxsize=1024)
def verify_drafts_workspace_bytes(batch: int, drafts: int, vocab: int, drafted: int,
                                  io: int) -> int:
    """ms_verify_drafts_workspace_bytes: workspace of verify_drafts."""
    return lm._size(ms.load().ms_verify_drafts_workspace_bytes(batch, drafts, vocab, drafted, io),
                    "the verification of drafts")


def verify_drafts(logits, drafts, uniforms, draft_logits=None, *, scale=1.0, workspace=None,
                  stream=None):
    """ms_verify_drafts on torch device tensors: drafts [batch, n] (int32 or
    int64) against the target's logits [batch, n + 1, vocab], with uniforms
    [batch, n + 1] (fp32, below 1) and the drafting model's logits [batch, n,
    vocab] (None: drafts without probabilities of their own).  Rows of logits
    may be strided.  Returns a dict: tokens [batch, n + 1] int32 (the accepted
    drafts, the token drawn, -1 behind it), count [batch] int32 (drafts
    accepted) and logprob [batch, n + 1] fp32."""
    import torch
    m = lm._marshal()
    ld, io = _pitch(m, logits, "logits", 3, 1, "[batch, drafts + 1, vocab]")
    b, rows, vocab = logits.shape
    n = rows - 1
    if n < 0:
        raise ValueError("logits must have a row behind the drafts")
    bits = lm._id_bits(drafts, "drafts")
    if not m.fits(logits, drafts.dtype, (b, n), drafts):
        lm._refuse(logits.device, drafts.dtype, (b, n), drafts=drafts)
    _need(uniforms=uniforms)
    if not m.fits(logits, torch.float32, (b, rows), uniforms):
        lm._refuse(logits.device, torch.float32, (b, rows), uniforms=uniforms)
    ldd = 0
    if draft_logits is not None:
        ldd, _ = _pitch(m, draft_logits, "draft_logits", 3, 1, "[batch, drafts, vocab]", logits)
        if draft_logits.shape != (b, n, vocab):
            raise ValueError(f"draft_logits must have shape {(b, n, vocab)}, "
                             f"got {tuple(draft_logits.shape)}")
        if n == 0:
            draft_logits = None
    need = verify_drafts_workspace_bytes(b, n, vocab, int(draft_logits is not None), io)
    call = lm._Call(m, logits, stream)
    tokens, count, logprob = call.together(torch.int32, (b, rows), torch.int32, (b,),
                                           torch.float32, (b, rows))
    ws, wn = call.workspace(workspace, need)
    call.run(m.verify_drafts, logits, ld, draft_logits, ldd, drafts, bits, uniforms, scale, tokens,
             count, logprob, b, n, vocab, io, ws, wn)
    return {"tokens": tokens, "count": count, "logprob": logprob}


# ---- as differentiable operations -----------------------------------------------------------

_fns = None


def _rows(m, t, inner):
    """t, or a copy where its rows are not contiguous and evenly apart."""
    return t if t is None or m.pitch(t, t.dim(), inner) >= 0 else t.contiguous()


def _taken(q, k, v, g, h0, reset):
    """The arguments of linear_attn as the raw calls take them."""
    m = lm._marshal()
    return tuple(_rows(m, t, 2) for t in (q, k, v)) + tuple(
        t if t is None else t.contiguous() for t in (g, h0, reset))


def _attend(q, k, v, g, h0, scale, reset, last, states):
    """(o, h_last or None)"""
    import torch
    h_last = None
    if last:
        (b, _, h, _, dk, dv, _), *_ = _chk_heads(lm._marshal(), q, k, v, g, reset)
        h_last = torch.empty(b, h, dk, dv, dtype=torch.float32, device=k.device)
    return linear_attn_fwd(q, k, v, g, scale=scale, reset=reset, h0=lm._aligned(h0),
                           h_last=h_last, states=states), h_last


def _functions():
    """The autograd Functions, built on first use (importing the package does
    not import torch)."""
    global _fns
    if _fns is not None:
        return _fns
    import torch
    from torch.autograd.function import once_differentiable

    class LinearAttn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, g, h0, scale, reset, last):
            q, k, v, g, h0, reset = _taken(q, k, v, g, h0, reset)
            states = linear_attn_states(k, v)
            o, h_last = _attend(q, k, v, g, h0, scale, reset, last, states)
            ctx.save_for_backward(q, k, v, g, states, reset)
            ctx.scale, ctx.start = scale, h0 is not None and ctx.needs_input_grad[4]
            ctx.set_materialize_grads(False)
            return o, h_last

        @staticmethod
        @once_differentiable
        def backward(ctx, do, dh_last):
            q, k, v, g, states, reset = ctx.saved_tensors
            do = torch.zeros(v.shape, dtype=v.dtype, device=v.device) if do is None else \
                do.contiguous()
            if dh_last is not None:
                dh_last = dh_last.contiguous()
            d = linear_attn_bwd(q, k, v, g, do, states, scale=ctx.scale, reset=reset,
                                dh_last=dh_last, want_dh0=ctx.start)
            return d["dq"], d["dk"], d["dv"], d["dg"], d["dh0"], None, None, None

    class GroupNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, groups, weight, bias, z, center, gate_first, eps):
            m = lm._marshal()
            x, z = _rows(m, x, 1), _rows(m, z, 1)
            weight, bias = (t if t is None else t.contiguous() for t in (weight, bias))
            ctx.save_for_backward(x, weight, bias, z)
            ctx.groups = groups
            ctx.how = {"center": center, "gate_first": gate_first, "eps": eps}
            return group_norm_fwd(x, groups, weight, bias, z, **ctx.how)

        @staticmethod
        @once_differentiable
        def backward(ctx, dy):
            x, weight, bias, z = ctx.saved_tensors
            d = group_norm_bwd(x, dy.contiguous(), ctx.groups, weight, bias, z, **ctx.how,
                               want_dweight=ctx.needs_input_grad[2],
                               want_dbias=ctx.needs_input_grad[3])
            return d["dx"], None, d["dweight"], d["dbias"], d["dz"], None, None, None

    _fns = (LinearAttn, GroupNorm)
    return _fns


def linear_attn(q, k, v, g, h0=None, *, scale=1.0, reset=None, return_last=False):
    """Linear attention as a differentiable torch operation (linear_attn_fwd
    with its saved states, linear_attn_bwd).  Returns o, or (o, h_last) with
    return_last; gradients (of the first order) reach q, k, v, g and h0.  Where
    none is asked for, no states are saved."""
    import torch
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad
                                       for t in (q, k, v, g, h0)):
        o, h_last = _functions()[0].apply(q, k, v, g, h0, scale, reset, return_last)
    else:
        q, k, v, g, h0, reset = _taken(q, k, v, g, h0, reset)
        o, h_last = _attend(q, k, v, g, h0, scale, reset, return_last, None)
    return (o, h_last) if return_last else o


def group_norm(x, groups, weight=None, bias=None, z=None, *, center=True, gate_first=False,
               eps=1e-5):
    """The group norm of each row's channels as a differentiable torch
    operation; gradients (of the first order) reach x, weight, bias and z."""
    return _functions()[1].apply(x, groups, weight, bias, z, center, gate_first, eps)
