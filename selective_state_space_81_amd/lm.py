"""The operators of a recurrent language model beside the scan: the gated
linear recurrence, the embedding with its gradient and the token log
probabilities.  Argument marshalling only, as in the package's ``__init__``
(its quick half in C++, csrc/binding.cpp): the work is done by the HIP kernels behind ``include/msscan.h``.

Raw calls (``*_fwd``, ``*_bwd``, ``gated_step``) take and return device
tensors; ``gated_scan``, ``embed`` and ``token_logprobs`` are the same as
differentiable torch operations.  Work goes to the current stream of the
tensors' device, or to ``stream``.  Buffers allocated here belong to the stream
that the work goes to, and results are kept from reuse until the current one
has passed them too; the inputs of a call on another stream have to be ready
there, and kept until it has passed them.
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
             [vp] * 4 + [f32] + [vp] * 6 + [i32, i64, i32, i64, i32, vp, sz, vp]),
            ("ms_gated_scan_bwd_workspace_bytes", sz, [i32, i64, i32, i32]),
            ("ms_gated_scan_bwd", ctypes.c_int,
             [vp] * 4 + [f32] + [vp] * 11 + [i32, i64, i32, i64, i32, vp, sz, vp]),
            ("ms_gated_step", ctypes.c_int, [vp] * 5 + [f32, vp, vp, i32, i32, i64, i32, vp]),
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


@functools.lru_cache(maxsize=None)
def _marshal():
    """The extension module that checks, allocates and calls (csrc/binding.cpp),
    bound to the loaded library."""
    lib = ms.load()
    try:
        from selective_state_space_81_amd import _marshal as m
    except ImportError as e:
        raise ImportError("_marshal.so cannot be loaded; build it with "
                          "`python -m selective_state_space_81_amd.build`") from e
    for name in ("gated_scan_fwd", "gated_scan_bwd", "gated_step", "embed_fwd", "embed_bwd",
                 "token_logprobs_fwd", "token_logprobs_bwd"):
        m.bind(name, ctypes.cast(getattr(lib, "ms_" + name), ctypes.c_void_p).value)
    return m


class _Call:
    """One call's device and stream.  What it allocates comes from that
    stream's memory: memory that the current stream has freed may still be in
    use by work queued there, which another stream does not wait for.  Results
    are recorded on the current stream, whose work may use them."""

    __slots__ = ("torch", "m", "like", "index", "stream", "other", "current")

    def __init__(self, m, like, stream):
        import torch
        self.torch, self.m, self.like, self.other = torch, m, like, None
        self.index = like.get_device()
        # the current stream's handle, without building a Stream around it
        self.stream = torch._C._cuda_getCurrentRawStream(self.index)
        if stream is not None:
            given = stream if isinstance(stream, int) else stream.cuda_stream
            if given != self.stream:
                self.current = torch.cuda.current_stream(self.index)
                self.stream = given
                if not isinstance(stream, int):
                    self.other = stream
                elif given:
                    self.other = torch.cuda.ExternalStream(given, device=like.device)
                else:  # as an external handle 0 becomes a new stream
                    self.other = torch.cuda.default_stream(self.index)

    def _make(self, make, *args):
        if self.other is None:
            return make(self.like, *args)
        with self.torch.cuda.stream(self.other):
            return make(self.like, *args)

    def empty(self, dtype, *shape):
        t = self._make(self.m.empty, dtype, *shape)
        if self.other is not None:
            t.record_stream(self.current)
        return t

    def together(self, *dtypes_and_sizes):
        ts = self._make(self.m.together, *dtypes_and_sizes)
        if self.other is not None:
            ts[0].record_stream(self.current)  # the one allocation of all
        return ts

    def workspace(self, given, need):
        """(tensor, bytes) of the given workspace, or of a new one."""
        if given is None:
            return (self._make(self.m.empty, self.torch.uint8, need), need) if need else (None, 0)
        if given.device != self.like.device or not given.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {self.like.device}")
        return given, given.numel() * given.element_size()

    def run(self, fn, *args):
        if self.torch._C._cuda_getDevice() != self.index:
            with self.torch.cuda.device(self.index):
                rc = fn(*args, self.stream)
        else:
            rc = fn(*args, self.stream)
        if rc:
            ms._check(rc)


def _refuse(device, dtype, shape, rows=False, **given):
    """What is wrong with an argument that the extension's check refused: the
    package's check of each (rows: it may be a slice), and its device."""
    for name, t in given.items():
        if t is not None:
            if not (rows and getattr(t, "is_cuda", False) and t.dtype == dtype and
                    t.shape == shape):
                ms._chk(t, name, dtype, tuple(shape))
            if t.device != device:
                raise ValueError(f"{name} is on {t.device}, not on {device}")


def _io_of(m, x, name, dims, text):
    """The io code of a contiguous device tensor of so many dimensions."""
    io = m.io(x, dims)
    if io < 0:
        if not getattr(x, "is_cuda", False) or x.dim() != dims:
            raise ValueError(f"{name} must be a {text} device tensor")
        io = ms._io(x)
        ms._chk(x, name, x.dtype, tuple(x.shape))
    return io


def _size(n: int, what: str) -> int:
    if n == ctypes.c_size_t(-1).value:
        raise ms.MsError(2, ms.load().ms_last_error().decode() or f"invalid sizes for {what}")
    return int(n)


# ---- gated linear recurrence -------------------------------------------------------------

def _refuse_rows(dims, text, **given):
    """What is wrong with the tensors whose rows have one distance (x first)."""
    name, x = next(iter(given.items()))
    if not getattr(x, "is_cuda", False) or x.dim() != dims:
        raise ValueError(f"{name} must be a {text} device tensor")
    ms._io(x)
    for k, t in given.items():
        if t is None and k[0] != "z":
            raise ValueError(f"{k} is required")
    _refuse(x.device, x.dtype, x.shape, rows=True, **given)
    raise ValueError(f"{', '.join(given)} must be contiguous, or slices of rows that are as far "
                     "apart in one as in the other")


def _chk_gated(m, x, r, i, lam, z, reset):
    """Checks of the arguments both passes share; (shape, ld, io, reset)."""
    import torch
    code = m.rows(x, 3, r, i, z)
    if code < 0 or r is None or i is None:
        _refuse_rows(3, "[batch, L, d_inner]", x=x, r=r, i=i, z=z)
    ld, io = code >> 1, code & 1
    shape = x.shape
    if lam is None:
        raise ValueError("lam is required")
    if not m.fits(x, torch.float32, (shape[2],), lam):
        _refuse(x.device, torch.float32, shape[2:], lam=lam)
    if reset is not None:
        if reset.dtype == torch.bool:
            reset = reset.view(torch.uint8)
        if not m.fits(x, torch.uint8, (shape[0], shape[1]), reset):
            _refuse(x.device, torch.uint8, shape[:2], reset=reset)
    return shape, ld, io, reset


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
    m = _marshal()
    if m.rows(x, 3) < 0:
        _refuse_rows(3, "[batch, L, d_inner]", x=x)
    b, L, d = x.shape
    return _Call(m, x, stream).empty(torch.float32, b, -(-L // GATED_BLOCK), d)


def gated_scan_fwd(x, r, i, lam, z=None, *, c=8.0, reset=None, y=None, h0=None, h_last=None,
                   states=None, workspace=None, stream=None):
    """ms_gated_scan_fwd on torch device tensors: the gated linear recurrence
    of x [batch, L, d] with decay gate r, input gate i (pre-activations), rate
    lam [d] and sharpness c, optionally gated by silu(z).  reset [batch, L]
    (uint8 or bool) starts new sequences; states (gated_scan_states) receives
    what the backward needs.  x, r, i and z are contiguous, or column slices of
    one wider tensor (their rows as far apart in one as in the other).  Allocates y (and the workspace) when not given.
    Returns y."""
    import torch
    m = _marshal()
    shape, ld, io, reset = _chk_gated(m, x, r, i, lam, z, reset)
    b, L, d = shape
    f32 = torch.float32
    if not m.fits(x, f32, (b, d), h0, h_last):
        _refuse(x.device, f32, (b, d), h0=h0, h_last=h_last)
    if not m.fits(x, f32, (b, -(-L // GATED_BLOCK), d), states):
        _refuse(x.device, f32, (b, -(-L // GATED_BLOCK), d), states=states)
    if y is not None and not m.fits(x, x.dtype, (b, L, d), y):
        _refuse(x.device, x.dtype, shape, y=y)
    call = _Call(m, x, stream)
    if y is None:
        y = call.empty(x.dtype, b, L, d)
    ws, wn = call.workspace(workspace, gated_scan_workspace_bytes(b, L, d, io))
    call.run(m.gated_scan_fwd, x, r, i, lam, c, z, reset, y, h0, h_last, states, b, L, d, ld, io,
             ws, wn)
    return y


def gated_scan_bwd(x, r, i, lam, dy, states, z=None, *, c=8.0, reset=None, dh_last=None,
                   workspace=None, stream=None, want_dh0=True):
    """ms_gated_scan_bwd on torch device tensors: gradients of gated_scan_fwd
    for dy (and optionally dh_last), with the states it saved.  Returns a dict:
    dx, dr, di, dz (io dtype; dz None without z), dlam and dh0 (fp32)."""
    import torch
    m = _marshal()
    shape, ld, io, reset = _chk_gated(m, x, r, i, lam, z, reset)
    b, L, d = shape
    f32, dt = torch.float32, x.dtype
    if states is None:
        raise ValueError("states is required (gated_scan_fwd fills it)")
    if dy is None:
        raise ValueError("dy is required")
    if not m.fits(x, f32, (b, -(-L // GATED_BLOCK), d), states):
        _refuse(x.device, f32, (b, -(-L // GATED_BLOCK), d), states=states)
    if not m.fits(x, dt, (b, L, d), dy):
        _refuse(x.device, dt, shape, dy=dy)
    if not m.fits(x, f32, (b, d), dh_last):
        _refuse(x.device, f32, (b, d), dh_last=dh_last)
    call = _Call(m, x, stream)
    out = {k: call.empty(dt, b, L, d) for k in ("dx", "dr", "di")}
    out["dz"] = call.empty(dt, b, L, d) if z is not None else None
    out["dlam"] = call.empty(f32, d)
    out["dh0"] = call.empty(f32, b, d) if want_dh0 else None
    ws, wn = call.workspace(workspace, gated_scan_bwd_workspace_bytes(b, L, d, io))
    call.run(m.gated_scan_bwd, x, r, i, lam, c, z, reset, states, dy, dh_last, out["dx"], out["dr"],
             out["di"], out["dz"], out["dlam"], out["dh0"], b, L, d, ld, io, ws, wn)
    return out


def gated_step(h, x_t, r_t, i_t, lam, z_t=None, *, c=8.0, y_t=None, stream=None):
    """ms_gated_step on torch device tensors: one step of the recurrence for
    x_t [batch, d]; h [batch, d] fp32 is updated in place.  x_t, r_t, i_t and z_t
    may be column slices of one wider tensor.  Returns y_t."""
    import torch
    m = _marshal()
    code = m.rows(x_t, 2, r_t, i_t, z_t)
    if code < 0 or r_t is None or i_t is None:
        _refuse_rows(2, "[batch, d_inner]", x_t=x_t, r_t=r_t, i_t=i_t, z_t=z_t)
    b, d = x_t.shape
    f32 = torch.float32
    for t, name in ((h, "h"), (lam, "lam")):
        if t is None:
            raise ValueError(f"{name} is required")
    if y_t is not None and not m.fits(x_t, x_t.dtype, (b, d), y_t):
        _refuse(x_t.device, x_t.dtype, (b, d), y_t=y_t)
    if not m.fits(x_t, f32, (b, d), h):
        _refuse(x_t.device, f32, (b, d), h=h)
    if not m.fits(x_t, f32, (d,), lam):
        _refuse(x_t.device, f32, (d,), lam=lam)
    call = _Call(m, x_t, stream)
    if y_t is None:
        y_t = call.empty(x_t.dtype, b, d)
    call.run(m.gated_step, h, x_t, r_t, i_t, lam, c, z_t, y_t, b, d, code >> 1, code & 1)
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
    m = _marshal()
    io = _io_of(m, weight, "weight", 2, "[rows, dim]")
    rows, dim = weight.shape
    bits, size = _id_bits(ids, "ids"), ids.shape
    if not m.fits(weight, ids.dtype, size, ids):
        _refuse(weight.device, ids.dtype, size, ids=ids)
    if out is not None and not m.fits(weight, weight.dtype, (*size, dim), out):
        _refuse(weight.device, weight.dtype, (*size, dim), out=out)
    call = _Call(m, weight, stream)
    if out is None:
        out = call.empty(weight.dtype, *size, dim)
    call.run(m.embed_fwd, ids, bits, weight, scale, out, ids.numel(), rows, dim, io)
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
    m = _marshal()
    size = ids.shape
    io = _io_of(m, dy, "dy", len(size) + 1, "[*ids.shape, dim]")
    bits, dim = _id_bits(ids, "ids"), dy.shape[-1]
    if not m.fits(dy, ids.dtype, size, ids):
        _refuse(dy.device, ids.dtype, size, ids=ids)
    if not m.fits(dy, dy.dtype, (*size, dim), dy):
        _refuse(dy.device, dy.dtype, (*size, dim), dy=dy)
    if grad_dtype is None:
        grad_dtype = dy.dtype if dweight is None else dweight.dtype
    if grad_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"grad_dtype must be float32 or bfloat16, got {grad_dtype}")
    if dweight is not None and not m.fits(dy, grad_dtype, (rows, dim), dweight):
        _refuse(dy.device, grad_dtype, (rows, dim), dweight=dweight)
    n = ids.numel()
    need = embed_bwd_workspace_bytes(n, rows, dim, io)
    call = _Call(m, dy, stream)
    if dweight is None:
        dweight = call.empty(grad_dtype, rows, dim)
    ws, wn = call.workspace(workspace, need)
    call.run(m.embed_bwd, ids, bits, dy, scale, padding, dweight,
             ms.MS_BF16 if grad_dtype == torch.bfloat16 else ms.MS_F32, n, rows, dim, io, ws, wn)
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


def _chk_targets(m, targets, rows, logits):
    if targets is None:
        return 64
    if not m.fits(logits, targets.dtype, (rows,), targets):
        _refuse(logits.device, targets.dtype, (rows,), targets=targets)
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
    m = _marshal()
    rows, vocab, ld = _chk_logits(logits)
    io = ms._io(logits)
    bits = _chk_targets(m, targets, rows, logits)
    f32 = torch.float32
    need = token_logprobs_workspace_bytes(rows, vocab, top, io)
    call = _Call(m, logits, stream)
    each = (rows,)
    logprob, entropy, lse, stats, top_logprob, top_id = call.together(
        f32, each, f32, each, f32, each, f32, (rows, 2), f32, (rows, top), torch.int32, (rows, top))
    if targets is None:
        logprob = None
    ws, wn = call.workspace(workspace, need)
    call.run(m.token_logprobs_fwd, logits, ld, targets, bits, scale, logprob, entropy, lse, stats,
             top, top_logprob, top_id, rows, vocab, io, ws, wn)
    return {"logprob": logprob, "entropy": entropy, "lse": lse, "stats": stats,
            "top_logprob": top_logprob, "top_id": top_id}


def token_logprobs_bwd(logits, targets, stats, entropy=None, dlogprob=None, dentropy=None, *,
                       scale=1.0, dlogits=None, stream=None):
    """ms_token_logprobs_bwd on torch device tensors: the gradient of the
    logits for dlogprob and dentropy ([rows] fp32, either may be None), with
    the stats and entropy that token_logprobs_fwd returned.  dlogits may be
    logits.  Returns dlogits."""
    import torch
    m = _marshal()
    rows, vocab, ld = _chk_logits(logits)
    io = ms._io(logits)
    bits = _chk_targets(m, targets, rows, logits)
    f32 = torch.float32
    if not m.fits(logits, f32, (rows, 2), stats):
        _refuse(logits.device, f32, (rows, 2), stats=stats)
    if not m.fits(logits, f32, (rows,), entropy, dlogprob, dentropy):
        _refuse(logits.device, f32, (rows,), entropy=entropy, dlogprob=dlogprob,
                dentropy=dentropy)
    call = _Call(m, logits, stream)
    if dlogits is None:
        dlogits = call.empty(logits.dtype, rows, vocab)
    r2, v2, ldd = _chk_logits(dlogits, "dlogits")
    if dlogits.dtype != logits.dtype:
        raise TypeError(f"dlogits must be {logits.dtype}, got {dlogits.dtype}")
    if (r2, v2) != (rows, vocab):
        raise ValueError(f"dlogits must have shape {(rows, vocab)}, got {(r2, v2)}")
    if dlogits.device != logits.device:
        raise ValueError(f"dlogits is on {dlogits.device}, not on {logits.device}")
    call.run(m.token_logprobs_bwd, logits, ld, targets, bits, scale, stats, entropy, dlogprob,
             dentropy, dlogits, ldd, rows, vocab, io)
    return dlogits


# ---- as differentiable operations -----------------------------------------------------------

_fns = None


def _aligned(t):
    """t, or a copy of a tensor that begins off 16 bytes (the calls above refuse it)."""
    return t if t is None or t.data_ptr() % 16 == 0 else t.clone()


def _functions():
    """The autograd Functions, built on first use (importing the package does
    not import torch)."""
    global _fns
    if _fns is not None:
        return _fns
    import torch
    # a gradient of a gradient would be missing what came through these: refused
    from torch.autograd.function import once_differentiable

    class GatedScan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, r, i, lam, z, h0, c, reset):
            reset = None if reset is None else reset.contiguous()
            if x.is_contiguous():  # and no slice of a wider tensor, which may begin anywhere
                x, r, i, z = map(_aligned, (x, r, i, z))
            h0 = _aligned(h0)
            states = gated_scan_states(x)
            h_last = torch.empty(x.shape[0], x.shape[2], dtype=torch.float32, device=x.device)
            y = gated_scan_fwd(x, r, i, lam, z, c=c, reset=reset, h0=h0, h_last=h_last,
                               states=states)
            ctx.save_for_backward(x, r, i, lam, z, states, reset)
            ctx.c, ctx.start = c, h0 is not None
            ctx.set_materialize_grads(False)
            return y, h_last

        @staticmethod
        @once_differentiable
        def backward(ctx, dy, dh_last):
            x, r, i, lam, z, states, reset = ctx.saved_tensors
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else dy.contiguous()
            if dh_last is not None:
                dh_last = dh_last.contiguous()
            g = gated_scan_bwd(x, r, i, lam, dy, states, z, c=ctx.c, reset=reset,
                               dh_last=dh_last, want_dh0=ctx.start)
            return g["dx"], g["dr"], g["di"], g["dlam"], g["dz"], g["dh0"], None, None

    class Embed(torch.autograd.Function):
        @staticmethod
        def forward(ctx, ids, weight, scale, padding):
            ids = ids.contiguous()
            ctx.save_for_backward(ids)
            ctx.rows, ctx.scale, ctx.padding = weight.shape[0], scale, padding
            return embed_fwd(ids, _aligned(weight), scale=scale)

        @staticmethod
        @once_differentiable
        def backward(ctx, dy):
            ids, = ctx.saved_tensors
            return None, embed_bwd(ids, dy.contiguous(), ctx.rows, scale=ctx.scale,
                                   padding=ctx.padding), None, None

    class TokenLogprobs(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, targets, top, scale):
            targets = None if targets is None else targets.contiguous()
            logits = _aligned(logits)
            r = token_logprobs_fwd(logits, targets, top=top, scale=scale)
            ctx.save_for_backward(logits, targets, r["stats"], r["entropy"])
            ctx.scale = scale
            ctx.mark_non_differentiable(r["top_logprob"], r["top_id"])
            ctx.set_materialize_grads(False)
            return r["logprob"], r["entropy"], r["top_logprob"], r["top_id"]

        @staticmethod
        @once_differentiable
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
    or (y, h_last) with return_last; gradients (of the first order) reach every
    tensor argument but reset, which may be a slice of a wider one."""
    y, h_last = _functions()[0].apply(x, r, i, lam, z, h0, c, reset)
    return (y, h_last) if return_last else y


def embed(ids, weight, *, scale=None, padding=-1):
    """Embedding lookup as a differentiable torch operation for ids of any
    shape and strides; scale None means sqrt(dim).  The gradient of the table (of the
    first order) is dense, in its dtype; the row `padding` gets none."""
    if scale is None:
        scale = math.sqrt(weight.shape[1])
    return _functions()[1].apply(ids, weight, scale, padding)


def token_logprobs(logits, targets, *, top=0, scale=1.0):
    """Token log probabilities as a differentiable torch operation: (logprob,
    entropy, top_logprob, top_id) for targets of any stride; gradients (of
    the first order) reach the logits from logprob and entropy."""
    return _functions()[2].apply(logits, targets, top, scale)
