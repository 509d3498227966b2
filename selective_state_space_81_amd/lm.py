"""The operators of a recurrent language model beside the scan: the gated
linear recurrence, the embedding with its gradient and the token log
probabilities.  Argument marshalling only, as in the package's ``__init__``:
the work is done by the HIP kernels behind ``include/msscan.h``.

Raw calls (``*_fwd``, ``*_bwd``, ``gated_step``) take and return device
tensors; ``gated_scan``, ``embed`` and ``token_logprobs`` are the same as
differentiable torch operations.  Work goes to the current stream of the
tensors' device, or to ``stream``; buffers allocated here are kept from reuse
until that stream has passed them.
"""
from __future__ import annotations

import ctypes
import functools
import math

import selective_state_space_81_amd as ms

EXPORTS = ("ms_gated_scan_workspace_bytes", "ms_gated_scan_states_bytes", "ms_gated_scan_fwd",
           "ms_gated_scan_bwd_workspace_bytes", "ms_gated_scan_bwd", "ms_gated_step",
           "ms_embed_fwd", "ms_embed_bwd_workspace_bytes", "ms_embed_bwd",
           "ms_token_logprobs_workspace_bytes", "ms_token_logprobs_fwd", "ms_token_logprobs_bwd")

GATED_BLOCK = 16  # steps between the saved states of the gated scan
MAX_TOP = 64      # most alternatives of token_logprobs


def declare(lib) -> None:
    """Argument types of this module's entry points."""
    vp, f32, sz = ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
    i32, i64 = ctypes.c_int32, ctypes.c_int64
    for name, res, args in (
            ("ms_gated_scan_workspace_bytes", sz, [i32, i64, i32, i32]),
            ("ms_gated_scan_states_bytes", sz, [i32, i64, i32]),
            ("ms_gated_scan_fwd", ctypes.c_int,
             [vp] * 4 + [f32] + [vp] * 6 + [i32, i64, i32, i32, vp, sz, vp]),
            ("ms_gated_scan_bwd_workspace_bytes", sz, [i32, i64, i32, i32]),
            ("ms_gated_scan_bwd", ctypes.c_int,
             [vp] * 4 + [f32] + [vp] * 11 + [i32, i64, i32, i32, vp, sz, vp]),
            ("ms_gated_step", ctypes.c_int, [vp] * 5 + [f32, vp, vp, i32, i32, i32, vp]),
            ("ms_embed_fwd", ctypes.c_int, [vp, i32, vp, f32, vp, i64, i64, i32, i32, vp]),
            ("ms_embed_bwd_workspace_bytes", sz, [i64, i64, i32, i32]),
            ("ms_embed_bwd", ctypes.c_int,
             [vp, i32, vp, f32, i64, vp, i32, i64, i64, i32, i32, vp, sz, vp]),
            ("ms_token_logprobs_workspace_bytes", sz, [i64, i64, i32, i32]),
            ("ms_token_logprobs_fwd", ctypes.c_int,
             [vp, i64, vp, i32, f32, vp, vp, vp, vp, i32, vp, vp, i64, i64, i32, vp, sz, vp]),
            ("ms_token_logprobs_bwd", ctypes.c_int,
             [vp, i64, vp, i32, f32, vp, vp, vp, vp, vp, i64, i64, i64, i32, vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args


class _Call:
    """One call's device and stream.  Allocations made for it are recorded on
    its stream when that is not the current one (their memory could otherwise
    be handed out again while the call still uses it)."""

    __slots__ = ("torch", "device", "stream", "other")

    def __init__(self, like, stream):
        import torch
        self.torch, self.device, self.other = torch, like.device, None
        # the current stream's handle, without building a Stream around it
        self.stream = torch._C._cuda_getCurrentRawStream(self.device.index)
        if stream is not None:
            given = stream if isinstance(stream, int) else stream.cuda_stream
            if given != self.stream:
                self.stream = given
                self.other = torch.cuda.ExternalStream(given, device=self.device) \
                    if isinstance(stream, int) else stream

    def empty(self, shape, dtype):
        # (empty_strided costs a third less than empty: 1.2 of 1.7 us)
        strides, n = [], 1
        for k in reversed(shape):
            strides.append(n)
            n *= k or 1
        strides.reverse()
        t = self.torch.empty_strided(shape, strides, dtype=dtype, device=self.device)
        if self.other is not None:
            t.record_stream(self.other)
        return t

    def workspace(self, given, need):
        """(pointer, bytes, tensor) of the given workspace, or of a new one."""
        if given is None and need:
            given = self.empty((need,), self.torch.uint8)
        if given is None:
            return None, 0, None
        if given.device != self.device or not given.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {self.device}")
        return given.data_ptr(), given.numel() * given.element_size(), given

    def run(self, fn, *args):
        if self.torch._C._cuda_getDevice() != self.device.index:
            with self.torch.cuda.device(self.device):
                rc = fn(*args, self.stream)
        else:
            rc = fn(*args, self.stream)
        if rc:
            ms._check(rc)


def _chk(t, name, dtype, shape, device) -> None:
    """The package's check of a tensor argument, and its device.  Written to
    cost little when all is well: a step of a few microseconds makes a dozen."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.device == device and
                     t.is_contiguous()):
        return
    ms._chk(t, name, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, not on {device}")


def _size(n: int, what: str) -> int:
    if n == ctypes.c_size_t(-1).value:
        raise ms.MsError(2, ms.load().ms_last_error().decode() or f"invalid sizes for {what}")
    return int(n)


# ---- gated linear recurrence -------------------------------------------------------------

def _chk_gated(x, r, i, lam, z, reset):
    """Checks of the arguments both passes share; (shape, device, io, reset)."""
    import torch
    if not getattr(x, "is_cuda", False) or x.dim() != 3:
        raise ValueError("x must be a [batch, L, d_inner] device tensor")
    io, shape, dev, dt = ms._io(x), x.shape, x.device, x.dtype
    _chk(x, "x", dt, shape, dev)
    _chk(r, "r", dt, shape, dev)
    _chk(i, "i", dt, shape, dev)
    _chk(lam, "lam", torch.float32, shape[2:], dev)
    _chk(z, "z", dt, shape, dev)
    if reset is not None:
        if reset.dtype == torch.bool:
            reset = reset.view(torch.uint8)
        _chk(reset, "reset", torch.uint8, shape[:2], dev)
    return shape, dev, io, reset


@functools.lru_cache(maxsize=1024)
def gated_scan_workspace_bytes(batch: int, seqlen: int, d_inner: int, io: int) -> int:
    """ms_gated_scan_workspace_bytes: workspace of gated_scan_fwd."""
    return _size(ms.load().ms_gated_scan_workspace_bytes(batch, seqlen, d_inner, io),
                 "the gated scan")


@functools.lru_cache(maxsize=1024)
def gated_scan_bwd_workspace_bytes(batch: int, seqlen: int, d_inner: int, io: int) -> int:
    """ms_gated_scan_bwd_workspace_bytes: workspace of gated_scan_bwd."""
    return _size(ms.load().ms_gated_scan_bwd_workspace_bytes(batch, seqlen, d_inner, io),
                 "the gated scan's backward")


def gated_scan_states(x, stream=None):
    """An empty buffer for the states that gated_scan_fwd saves for
    gated_scan_bwd: [batch, ceil(L / 16), d_inner] fp32."""
    import torch
    b, L, d = x.shape
    return _Call(x, stream).empty((b, -(-L // GATED_BLOCK), d), torch.float32)


def gated_scan_fwd(x, r, i, lam, z=None, *, c=8.0, reset=None, y=None, h0=None, h_last=None,
                   states=None, workspace=None, stream=None):
    """ms_gated_scan_fwd on torch device tensors: the gated linear recurrence
    of x [batch, L, d] with decay gate r, input gate i (pre-activations), rate
    lam [d] and sharpness c, optionally gated by silu(z).  reset [batch, L]
    (uint8 or bool) starts new sequences; states (gated_scan_states) receives
    what the backward needs.  Allocates y (and the workspace) when not given.
    Returns y."""
    import torch
    shape, dev, io, reset = _chk_gated(x, r, i, lam, z, reset)
    b, L, d = shape
    f32 = torch.float32
    _chk(h0, "h0", f32, (b, d), dev)
    _chk(h_last, "h_last", f32, (b, d), dev)
    _chk(y, "y", x.dtype, shape, dev)
    _chk(states, "states", f32, (b, -(-L // GATED_BLOCK), d), dev)
    call = _Call(x, stream)
    if y is None:
        y = call.empty(shape, x.dtype)
    wp, wn, keep = call.workspace(workspace, gated_scan_workspace_bytes(b, L, d, io))
    p = ms._ptr
    call.run(ms.load().ms_gated_scan_fwd, p(x), p(r), p(i), p(lam), c, p(z), p(reset), p(y), p(h0),
             p(h_last), p(states), b, L, d, io, wp, wn)
    return y


def gated_scan_bwd(x, r, i, lam, dy, states, z=None, *, c=8.0, reset=None, dh_last=None,
                   workspace=None, stream=None, want_dh0=True):
    """ms_gated_scan_bwd on torch device tensors: gradients of gated_scan_fwd
    for dy (and optionally dh_last), with the states it saved.  Returns a dict:
    dx, dr, di, dz (io dtype; dz None without z), dlam and dh0 (fp32)."""
    import torch
    shape, dev, io, reset = _chk_gated(x, r, i, lam, z, reset)
    b, L, d = shape
    f32 = torch.float32
    if states is None:
        raise ValueError("states is required (gated_scan_fwd fills it)")
    if dy is None:
        raise ValueError("dy is required")
    _chk(states, "states", f32, (b, -(-L // GATED_BLOCK), d), dev)
    _chk(dy, "dy", x.dtype, shape, dev)
    _chk(dh_last, "dh_last", f32, (b, d), dev)
    call = _Call(x, stream)
    out = {k: call.empty(shape, x.dtype) for k in ("dx", "dr", "di")}
    out["dz"] = call.empty(shape, x.dtype) if z is not None else None
    out["dlam"] = call.empty((d,), f32)
    out["dh0"] = call.empty((b, d), f32) if want_dh0 else None
    wp, wn, keep = call.workspace(workspace, gated_scan_bwd_workspace_bytes(b, L, d, io))
    p = ms._ptr
    call.run(ms.load().ms_gated_scan_bwd, p(x), p(r), p(i), p(lam), c, p(z), p(reset), p(states), p(dy),
             p(dh_last), p(out["dx"]), p(out["dr"]), p(out["di"]), p(out["dz"]), p(out["dlam"]),
             p(out["dh0"]), b, L, d, io, wp, wn)
    return out


def gated_step(h, x_t, r_t, i_t, lam, z_t=None, *, c=8.0, y_t=None, stream=None):
    """ms_gated_step on torch device tensors: one step of the recurrence for
    x_t [batch, d]; h [batch, d] fp32 is updated in place.  Returns y_t."""
    import torch
    if not getattr(x_t, "is_cuda", False) or x_t.dim() != 2:
        raise ValueError("x_t must be a [batch, d_inner] device tensor")
    io, shape, dev, dt = ms._io(x_t), x_t.shape, x_t.device, x_t.dtype
    f32 = torch.float32
    if h is None:
        raise ValueError("h is required")
    _chk(h, "h", f32, shape, dev)
    _chk(x_t, "x_t", dt, shape, dev)
    _chk(r_t, "r_t", dt, shape, dev)
    _chk(i_t, "i_t", dt, shape, dev)
    _chk(lam, "lam", f32, shape[1:], dev)
    _chk(z_t, "z_t", dt, shape, dev)
    _chk(y_t, "y_t", dt, shape, dev)
    call = _Call(x_t, stream)
    if y_t is None:
        y_t = call.empty(shape, dt)
    p = ms._ptr
    call.run(ms.load().ms_gated_step, p(h), p(x_t), p(r_t), p(i_t), p(lam), c, p(z_t), p(y_t),
             shape[0], shape[1], io)
    return y_t


# ---- embedding -----------------------------------------------------------------------------

def _id_bits(t, name: str) -> int:
    import torch
    if t.dtype == torch.int64:
        return 64
    if t.dtype == torch.int32:
        return 32
    raise TypeError(f"{name} must be int32 or int64, got {t.dtype}")


def embed_fwd(ids, weight, *, scale=1.0, out=None, stream=None):
    """ms_embed_fwd on torch device tensors: scale * weight[ids] for ids of
    any shape; ids outside the table give rows of zeros.  Returns
    [*ids.shape, dim]."""
    if not getattr(weight, "is_cuda", False) or weight.dim() != 2:
        raise ValueError("weight must be a [rows, dim] device tensor")
    io = ms._io(weight)
    rows, dim = weight.shape
    bits, dev = _id_bits(ids, "ids"), weight.device
    _chk(ids, "ids", ids.dtype, ids.shape, dev)
    _chk(weight, "weight", weight.dtype, weight.shape, dev)
    shape = (*ids.shape, dim)
    _chk(out, "out", weight.dtype, shape, dev)
    call = _Call(weight, stream)
    if out is None:
        out = call.empty(shape, weight.dtype)
    call.run(ms.load().ms_embed_fwd, ms._ptr(ids), bits, ms._ptr(weight), scale, ms._ptr(out),
             ids.numel(), rows, dim, io)
    return out


@functools.lru_cache(maxsize=1024)
def embed_bwd_workspace_bytes(n: int, rows: int, dim: int, io: int) -> int:
    """ms_embed_bwd_workspace_bytes: workspace of embed_bwd."""
    return _size(ms.load().ms_embed_bwd_workspace_bytes(n, rows, dim, io),
                 "the embedding's gradient")


def embed_bwd(ids, dy, rows, *, scale=1.0, padding=-1, grad_dtype=None, dweight=None,
              workspace=None, stream=None):
    """ms_embed_bwd on torch device tensors: the gradient [rows, dim] of the
    table of embed_fwd for dy [*ids.shape, dim], in grad_dtype (dy's when not
    given); the row `padding` gets none.  Returns dweight."""
    import torch
    if not getattr(dy, "is_cuda", False) or dy.dim() != ids.dim() + 1:
        raise ValueError("dy must be a [*ids.shape, dim] device tensor")
    io = ms._io(dy)
    bits = _id_bits(ids, "ids")
    dim, dev = dy.shape[-1], dy.device
    _chk(ids, "ids", ids.dtype, ids.shape, dev)
    _chk(dy, "dy", dy.dtype, (*ids.shape, dim), dev)
    if grad_dtype is None:
        grad_dtype = dy.dtype if dweight is None else dweight.dtype
    if grad_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"grad_dtype must be float32 or bfloat16, got {grad_dtype}")
    _chk(dweight, "dweight", grad_dtype, (rows, dim), dev)
    n = ids.numel()
    need = embed_bwd_workspace_bytes(n, rows, dim, io)
    call = _Call(dy, stream)
    if dweight is None:
        dweight = call.empty((rows, dim), grad_dtype)
    wp, wn, keep = call.workspace(workspace, need)
    call.run(ms.load().ms_embed_bwd, ms._ptr(ids), bits, ms._ptr(dy), scale, padding, ms._ptr(dweight),
             ms.MS_BF16 if grad_dtype == torch.bfloat16 else ms.MS_F32, n, rows, dim, io, wp, wn)
    return dweight


# ---- token log probabilities -----------------------------------------------------------------

def _chk_logits(logits, name="logits"):
    """A [rows, vocab] device tensor whose rows are contiguous; (rows, vocab, ld)."""
    if not getattr(logits, "is_cuda", False) or logits.dim() != 2:
        raise ValueError(f"{name} must be a [rows, vocab] device tensor")
    rows, vocab = logits.shape
    if vocab > 1 and logits.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    ld = logits.stride(0) if rows > 1 else vocab
    if ld < vocab:
        raise ValueError(f"{name} must not have overlapping rows")
    return rows, vocab, ld


def _chk_targets(targets, rows, device):
    if targets is None:
        return 64
    _chk(targets, "targets", targets.dtype, (rows,), device)
    return _id_bits(targets, "targets")


@functools.lru_cache(maxsize=1024)
def token_logprobs_workspace_bytes(rows: int, vocab: int, top: int, io: int) -> int:
    """ms_token_logprobs_workspace_bytes: workspace of token_logprobs_fwd."""
    return _size(ms.load().ms_token_logprobs_workspace_bytes(rows, vocab, top, io),
                 "the token log probabilities")


def token_logprobs_fwd(logits, targets=None, *, top=0, scale=1.0, workspace=None, stream=None):
    """ms_token_logprobs_fwd on torch device tensors: for logits [rows, vocab]
    (rows may be strided) and targets [rows], a dict of logprob (None without
    targets), entropy, lse ([rows] fp32), stats ([rows, 2] fp32, for the
    gradient), top_logprob [rows, top] fp32 and
    top_id [rows, top] int32."""
    import torch
    rows, vocab, ld = _chk_logits(logits)
    io = ms._io(logits)
    bits = _chk_targets(targets, rows, logits.device)
    f32 = torch.float32
    need = token_logprobs_workspace_bytes(rows, vocab, top, io)
    call = _Call(logits, stream)
    out = {"logprob": call.empty((rows,), f32) if targets is not None else None,
           "entropy": call.empty((rows,), f32), "lse": call.empty((rows,), f32),
           "stats": call.empty((rows, 2), f32),
           "top_logprob": call.empty((rows, top), f32),
           "top_id": call.empty((rows, top), torch.int32)}
    wp, wn, keep = call.workspace(workspace, need)
    p = ms._ptr
    call.run(ms.load().ms_token_logprobs_fwd, p(logits), ld, p(targets), bits, scale, p(out["logprob"]),
             p(out["entropy"]), p(out["lse"]), p(out["stats"]), top, p(out["top_logprob"]),
             p(out["top_id"]), rows, vocab, io, wp, wn)
    return out


def token_logprobs_bwd(logits, targets, stats, entropy=None, dlogprob=None, dentropy=None, *,
                       scale=1.0, dlogits=None, stream=None):
    """ms_token_logprobs_bwd on torch device tensors: the gradient of the
    logits for dlogprob and dentropy ([rows] fp32, either may be None), with
    the stats and entropy that token_logprobs_fwd returned.  dlogits may be
    logits.  Returns dlogits."""
    import torch
    rows, vocab, ld = _chk_logits(logits)
    io = ms._io(logits)
    dev = logits.device
    bits = _chk_targets(targets, rows, dev)
    f32 = torch.float32
    _chk(stats, "stats", f32, (rows, 2), dev)
    for t, name in ((entropy, "entropy"), (dlogprob, "dlogprob"), (dentropy, "dentropy")):
        _chk(t, name, f32, (rows,), dev)
    call = _Call(logits, stream)
    if dlogits is None:
        dlogits = call.empty((rows, vocab), logits.dtype)
    r2, v2, ldd = _chk_logits(dlogits, "dlogits")
    if dlogits.dtype != logits.dtype:
        raise TypeError(f"dlogits must be {logits.dtype}, got {dlogits.dtype}")
    if (r2, v2) != (rows, vocab):
        raise ValueError(f"dlogits must have shape {(rows, vocab)}, got {(r2, v2)}")
    if dlogits.device != dev:
        raise ValueError(f"dlogits is on {dlogits.device}, not on {dev}")
    p = ms._ptr
    call.run(ms.load().ms_token_logprobs_bwd, p(logits), ld, p(targets), bits, scale, p(stats), p(entropy),
             p(dlogprob), p(dentropy), p(dlogits), ldd, rows, vocab, io)
    return dlogits


# ---- as differentiable operations -----------------------------------------------------------

_fns = None


def _functions():
    """The autograd Functions, built on first use (importing the package does
    not import torch)."""
    global _fns
    if _fns is not None:
        return _fns
    import torch

    class GatedScan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, r, i, lam, z, h0, c, reset):
            states = gated_scan_states(x)
            h_last = torch.empty(x.shape[0], x.shape[2], dtype=torch.float32, device=x.device)
            y = gated_scan_fwd(x, r, i, lam, z, c=c, reset=reset, h0=h0, h_last=h_last,
                               states=states)
            ctx.save_for_backward(x, r, i, lam, z, states, reset)
            ctx.c, ctx.start = c, h0 is not None
            ctx.set_materialize_grads(False)
            return y, h_last

        @staticmethod
        def backward(ctx, dy, dh_last):
            x, r, i, lam, z, states, reset = ctx.saved_tensors
            dy = torch.zeros_like(x) if dy is None else dy.contiguous()
            if dh_last is not None:
                dh_last = dh_last.contiguous()
            g = gated_scan_bwd(x, r, i, lam, dy, states, z, c=ctx.c, reset=reset,
                               dh_last=dh_last, want_dh0=ctx.start)
            return g["dx"], g["dr"], g["di"], g["dlam"], g["dz"], g["dh0"], None, None

    class Embed(torch.autograd.Function):
        @staticmethod
        def forward(ctx, ids, weight, scale, padding):
            ctx.save_for_backward(ids)
            ctx.rows, ctx.scale, ctx.padding = weight.shape[0], scale, padding
            return embed_fwd(ids, weight, scale=scale)

        @staticmethod
        def backward(ctx, dy):
            ids, = ctx.saved_tensors
            return None, embed_bwd(ids, dy.contiguous(), ctx.rows, scale=ctx.scale,
                                   padding=ctx.padding), None, None

    class TokenLogprobs(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, targets, top, scale):
            r = token_logprobs_fwd(logits, targets, top=top, scale=scale)
            ctx.save_for_backward(logits, targets, r["stats"], r["entropy"])
            ctx.scale = scale
            ctx.mark_non_differentiable(r["top_logprob"], r["top_id"])
            ctx.set_materialize_grads(False)
            return r["logprob"], r["entropy"], r["top_logprob"], r["top_id"]

        @staticmethod
        def backward(ctx, dlogprob, dentropy, _dtop, _did):
            logits, targets, stats, entropy = ctx.saved_tensors
            dlogprob, dentropy = (t if t is None else t.contiguous() for t in (dlogprob, dentropy))
            return token_logprobs_bwd(logits, targets, stats, entropy, dlogprob, dentropy,
                                      scale=ctx.scale), None, None, None

    _fns = (GatedScan, Embed, TokenLogprobs)
    return _fns


def gated_scan(x, r, i, lam, z=None, h0=None, *, c=8.0, reset=None, return_last=False):
    """The gated linear recurrence as a differentiable torch operation
    (ms_gated_scan_fwd with its saved states, ms_gated_scan_bwd).  Returns y,
    or (y, h_last) with return_last; gradients reach every tensor argument
    but reset."""
    y, h_last = _functions()[0].apply(x, r, i, lam, z, h0, c, reset)
    return (y, h_last) if return_last else y


def embed(ids, weight, *, scale=None, padding=-1):
    """Embedding lookup as a differentiable torch operation; scale None means
    sqrt(dim).  The gradient of the table is dense, in its dtype; the row
    `padding` gets none."""
    if scale is None:
        scale = math.sqrt(weight.shape[1])
    return _functions()[1].apply(ids, weight, scale, padding)


def token_logprobs(logits, targets, *, top=0, scale=1.0):
    """Token log probabilities as a differentiable torch operation: (logprob,
    entropy, top_logprob, top_id); gradients reach the logits from logprob and
    entropy."""
    return _functions()[2].apply(logits, targets, top, scale)
