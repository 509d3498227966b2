"""Host-only checks of the language-model operators' C ABI: sizes, and every
refusal that needs no GPU (nothing is launched on any of these calls)."""
import contextlib
import ctypes
import types

import pytest
import torch

import selective_state_space_81_amd as ms

NONE = ctypes.c_size_t(-1).value
P = 16  # an aligned address that is never read


def test_sizes():
    lib = ms.load()
    assert lib.ms_gated_scan_states_bytes(2, 33, 5) == 2 * 3 * 5 * 4
    assert lib.ms_gated_scan_states_bytes(1, 16, 8) == 8 * 4
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (-1, 5, 5), (1, 1 << 31, 1)):
        assert lib.ms_gated_scan_states_bytes(*bad) == NONE
        assert lib.ms_gated_scan_workspace_bytes(*bad, 1) == NONE
        assert lib.ms_gated_scan_bwd_workspace_bytes(*bad, 1) == NONE
    assert lib.ms_gated_scan_workspace_bytes(1, 1, 1, 7) == NONE
    assert lib.ms_gated_scan_bwd_workspace_bytes(8, 2048, 1536, 1) % 256 == 0
    assert lib.ms_embed_bwd_workspace_bytes(0, 10, 8, 0) != NONE
    for bad in ((-1, 10, 8, 0), (1 << 31, 10, 8, 0), (5, 0, 8, 0), (5, 10, 0, 0), (5, 10, 8, 3)):
        assert lib.ms_embed_bwd_workspace_bytes(*bad) == NONE
    assert lib.ms_token_logprobs_workspace_bytes(0, 100, 5, 0) != NONE
    for bad in ((-1, 9, 0, 0), (1, 0, 0, 0), (1, 9, 10, 0), (1, 900, 65, 0), (1, 9, -1, 0),
                (1, 9, 0, 2)):
        assert lib.ms_token_logprobs_workspace_bytes(*bad) == NONE


def test_gated_refusals():
    lib = ms.load()

    def fwd(x=P, y=P, lam=P, c=8.0, h0=None, b=1, L=40, d=8, io=1, ld=None):
        return lib.ms_gated_scan_fwd(x, P, P, lam, c, None, None, y, h0, None, None, b, L, d,
                                     d if ld is None else ld, io, P, 1 << 40, None)

    assert fwd(x=None) == 1 and fwd(y=None) == 1 and fwd(lam=None) == 1
    assert fwd(b=0) == 2 and fwd(L=0) == 2 and fwd(d=0) == 2 and fwd(L=1 << 31) == 2
    assert fwd(io=2) == 3
    assert fwd(x=24) == 5 and fwd(h0=8) == 5
    assert fwd(ld=7) == 2 and fwd(ld=1 << 23) == 7
    assert fwd(ld=20, x=17) == 5 and fwd(ld=20, y=24) == 5  # only rows may lie off 16 bytes
    for c in (0.0, -2.0, float("inf"), float("nan")):
        assert fwd(c=c) == 2
    assert b"sharpness" in lib.ms_last_error()

    def bwd(z=None, dz=None, states=P, ws=P, n=1 << 40):
        return lib.ms_gated_scan_bwd(P, P, P, P, 8.0, z, None, states, P, None, P, P, P, dz, P,
                                     None, 1, 40, 8, 8, 1, ws, n, None)

    assert bwd(states=None) == 1 and bwd(z=P) == 1
    assert bwd(ws=None) == 6 and bwd(n=8) == 6
    assert lib.ms_gated_step(None, P, P, P, P, 8.0, None, P, 1, 8, 8, 1, None) == 1
    assert lib.ms_gated_step(P, P, P, P, P, 8.0, None, P, 0, 8, 8, 1, None) == 2
    assert lib.ms_gated_step(P, P, 20, P, P, 8.0, None, P, 1, 8, 8, 1, None) == 5


def test_embed_refusals():
    lib = ms.load()

    def fwd(ids=P, bits=64, w=P, scale=1.0, n=5, rows=10, dim=8, io=0):
        return lib.ms_embed_fwd(ids, bits, w, scale, P, n, rows, dim, io, None)

    assert fwd(ids=None) == 1 and fwd(w=None) == 1
    assert fwd(bits=16) == 3 and fwd(io=4) == 3
    assert fwd(n=-1) == 2 and fwd(rows=0) == 2 and fwd(dim=0) == 2 and fwd(dim=1 << 25) == 2
    assert fwd(scale=float("nan")) == 2
    assert fwd(w=8) == 5
    assert fwd(ids=None, n=0) == 0  # nothing to do, nothing launched

    assert lib.ms_embed_bwd_workspace_bytes(5000, 10, 8, 0) > 0

    def bwd(ids=P, dw=P, gd=0, ws=P, n=1 << 40):
        return lib.ms_embed_bwd(ids, 64, P, 1.0, -1, dw, gd, 5000, 10, 8, 0, ws, n, None)

    assert bwd(ids=None) == 1 and bwd(dw=None) == 1 and bwd(gd=5) == 3
    assert bwd(ws=None) == 6 and bwd(n=1) == 6 and bwd(ws=8) == 5


def test_logprob_refusals():
    lib = ms.load()

    def fwd(x=P, ld=40, t=P, bits=64, scale=1.0, lp=P, top=0, tl=None, ti=None, rows=3, V=40,
            io=0, ws=P):
        return lib.ms_token_logprobs_fwd(x, ld, t, bits, scale, lp, P, P, P, top, tl, ti, rows, V, io,
                                         ws, 1 << 40, None)

    assert fwd(x=None) == 1 and fwd(t=None) == 1 and fwd(top=2) == 1 and fwd(top=2, tl=P) == 1
    assert fwd(ld=39) == 2 and fwd(V=0) == 2 and fwd(rows=-1) == 2 and fwd(top=65) == 2
    assert fwd(bits=8) == 3 and fwd(io=9) == 3
    assert fwd(scale=0.0) == 2 and fwd(scale=float("inf")) == 2
    assert fwd(x=4) == 5
    assert fwd(rows=0, x=None) == 0
    # a shape that is split over workgroups, and so needs a workspace
    assert lib.ms_token_logprobs_workspace_bytes(1, 100000, 0, 0) > 0
    assert fwd(rows=1, V=100000, ld=100000, ws=None) == 6

    def bwd(x=P, t=P, stats=P, ent=P, gl=P, gh=P, d=P, ld=40, ldd=40):
        return lib.ms_token_logprobs_bwd(x, ld, t, 64, 1.0, stats, ent, gl, gh, d, ldd, 3, 40, 0,
                                         None)

    assert bwd(x=None) == 1 and bwd(stats=None) == 1 and bwd(d=None) == 1
    assert bwd(t=None) == 1 and bwd(ent=None) == 1
    assert bwd(ldd=39) == 2 and bwd(ldd=48) == 2  # over the logits with another stride


def test_launches_too_large():
    """A launch holds fewer than 2^24 workgroups of 256 threads."""
    lib = ms.load()
    # 65535 x 65539 channels, one by one
    assert lib.ms_gated_step(P, P, P, P, P, 8.0, None, P, 65535, 65539, 65539, 1, None) == 7
    assert lib.ms_gated_scan_workspace_bytes(65535, 1, 64 * 300, 1) == NONE
    assert b"2^24-1" in lib.ms_last_error()
    assert lib.ms_gated_scan_workspace_bytes(65535, 1, 64 * 200, 1) != NONE
    assert lib.ms_embed_fwd(P, 64, P, 1.0, P, (1 << 31) - 1, 10, 1 << 12, 0, None) == 7
    assert lib.ms_embed_bwd(P, 64, P, 1.0, -1, P, 0, 5, (1 << 31) - 1, 1 << 12, 0, P, 1 << 50,
                            None) == 7
    assert lib.ms_token_logprobs_fwd(P, 5, P, 64, 1.0, P, P, P, P, 0, None, None, 1 << 24, 5, 0,
                                     None, 0, None) == 7
    assert lib.ms_token_logprobs_bwd(P, 1 << 20, P, 64, 1.0, P, P, P, P, P, 1 << 20,
                                     (1 << 24) - 1, 1 << 20, 0, None) == 7


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 4, 8)
    with pytest.raises(ValueError, match="device"):
        ms.gated_scan_fwd(x, x, x, torch.zeros(8))
    with pytest.raises(ValueError, match="device"):
        ms.gated_step(x[:, 0], x[:, 0], x[:, 0], x[:, 0], torch.zeros(8))
    with pytest.raises(ValueError, match="device"):
        ms.embed_fwd(torch.zeros(3, dtype=torch.int64), torch.zeros(5, 8))
    with pytest.raises(ValueError, match="device"):
        ms.embed_bwd(torch.zeros(3, dtype=torch.int64), torch.zeros(3, 8), 5)
    with pytest.raises(ValueError, match="device"):
        ms.token_logprobs_fwd(torch.zeros(3, 8))


def test_marshalling():
    """The binding's extension module on host tensors (it looks at no memory)."""
    m = ms.lm._marshal()
    x, f32 = torch.zeros(3, 4), torch.float32
    assert m.io(x, 2) == -1 and m.rows(x, 2) == -1  # not on a device
    assert m.fits(x, torch.int32, (2,), None, torch.zeros(2, dtype=torch.int32))
    assert not m.fits(x, f32, (3,), x) and not m.fits(x, f32, (3, 5), x)
    assert not m.fits(x, f32, (4, 3), torch.zeros(3, 4).t())
    with pytest.raises(TypeError):
        m.fits(x, f32, (3, "4"), x)
    e = m.empty(x, torch.bfloat16, 2, 0, 5)
    assert e.shape == (2, 0, 5) and e.dtype == torch.bfloat16
    with pytest.raises(TypeError):
        m.empty(x, 5)
    a, b = m.together(x, f32, (5,), torch.int64, (2, 3))
    assert a.shape == (5,) and b.shape == (2, 3) and b.dtype == torch.int64
    a.fill_(1), b.fill_(2)
    assert a.sum() == 5 and b.sum() == 12 and not a._is_view()
    for bad in ((f32,), (f32, (-1,)), (f32, 5), (5, (1,))):
        with pytest.raises(TypeError):
            m.together(x, *bad)
    # wrong counts and types never reach the library
    with pytest.raises(TypeError):
        m.gated_step(x)
    with pytest.raises(TypeError):
        m.gated_step(x, x, x, x, x, "8", None, x, 3, 4, 4, 0, 0)
    with pytest.raises(OverflowError):
        m.gated_step(x, x, x, x, x, 8.0, None, x, 1 << 40, 4, 4, 0, 0)
    assert m.gated_step(x, x, x, x, x, 8.0, None, x, 0, 4, 4, 0, 0) == 2  # MS_ERR_SHAPE
    assert m.gated_step(None, x, x, x, x, 8.0, None, x, 3, 4, 4, 0, None) == 1  # MS_ERR_NULL


@pytest.mark.parametrize("shape,to", [((64,), (2, 100, 64)), ((2, 1, 64), (2, 100, 64)),
                                      ((1, 100, 64), (2, 100, 64)), ((1, 1, 64), (1, 100, 64)),
                                      ((1, 1, 64), (7, 1, 64)), ((1, 64), (8, 64)), ((1, 1), (8, 1))])
def test_expanded_rows_are_refused(shape, to):
    """A broadcast input has fewer rows in memory than its sizes say."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    m = ms.lm._marshal()
    with FakeTensorMode():  # device tensors without a device
        whole = torch.empty(to, device="cuda:0")
        wide = torch.empty(*to[:-1], 3 * to[-1] + 1, device="cuda:0")[..., to[-1]:2 * to[-1]]
        few = torch.empty(shape, device="cuda:0").expand(to)
        dims = len(to)
        assert m.rows(whole, dims) == 2 * to[-1] and m.rows(wide, dims) == 2 * (3 * to[-1] + 1)
        assert m.rows(few, dims) == -1 and m.rows(whole, dims, few) == -1
        lam = torch.empty(to[-1], device="cuda:0")
        for k in range(4):
            args = [few if j == k else whole for j in range(4)]
            with pytest.raises(ValueError, match="contiguous"):
                if dims == 2:
                    ms.gated_step(torch.empty(to, device="cuda:0"), *args[:3], lam, args[3])
                else:
                    ms.gated_scan_fwd(*args[:3], lam, args[3])


@pytest.mark.parametrize("as_int", [False, True])
def test_buffers_come_from_the_stream_of_the_call(monkeypatch, as_int):
    """What is allocated for a call on another stream is allocated there (the
    current stream's freed memory may still be in use by its queue), and results,
    not workspaces, are recorded on the current stream."""
    current, side = (types.SimpleNamespace(cuda_stream=k) for k in (1, 2))
    stack = [current]

    @contextlib.contextmanager
    def on(stream):
        stack.append(stream)
        yield
        stack.pop()

    class Made:
        def __init__(self):
            self.of, self.recorded = stack[-1], []

        def record_stream(self, stream):
            self.recorded.append(stream)

    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda k: 1, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda k=None: stack[-1])
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: {2: side}[h])
    m = types.SimpleNamespace(empty=lambda like, dtype, *shape: Made(),
                              together=lambda like, *sizes: [Made(), Made()])
    like = types.SimpleNamespace(get_device=lambda: 0, device="cuda:0")
    for stream, of in ((None, current), (current, current), (side, side)):
        given = stream.cuda_stream if as_int and stream else stream
        call = ms.lm._Call(m, like, given)
        assert call.stream == of.cuda_stream
        out, several = call.empty(torch.float32, 3), call.together(torch.float32, (3,))
        ws, n = call.workspace(None, 256)
        assert n == 256 and out.of is of and ws.of is of and all(t.of is of for t in several)
        assert stack == [current]
        there = [current] if of is side else []
        assert out.recorded == there and several[0].recorded == there and ws.recorded == []
        assert call.workspace(None, 0) == (None, 0)


def test_alignment_of_what_is_read_by_element():
    """ids, targets, resets, rates and gradients need their element's alignment
    only.  Each call is refused for something that is checked after it."""
    lib = ms.load()
    none, large = 6, 7  # no workspace, too large a launch
    many = (1 << 31) - 1

    def fwd(lam=P, reset=None):
        return lib.ms_gated_scan_fwd(P, P, P, lam, 8.0, None, reset, P, None, None, None, 1, 4000, 8,
                                     8, 1, None, 0, None)

    assert fwd() == none and fwd(lam=P + 4) == none and fwd(reset=P + 1) == none
    assert fwd(lam=P + 2) == 5

    def bwd(lam=P, reset=None, dy=P, dh_last=None, states=P, io=1):
        return lib.ms_gated_scan_bwd(P, P, P, lam, 8.0, None, reset, states, dy, dh_last, P, P, P,
                                     None, P, None, 1, 4000, 8, 8, io, None, 0, None)

    assert bwd() == none and bwd(lam=P + 4, reset=P + 3, dy=P + 2, dh_last=P + 4) == none
    assert bwd(dy=P + 4, io=0) == none and bwd(states=P + 4) == 5
    assert bwd(dy=P + 1) == 5 and bwd(dy=P + 2, io=0) == 5 and bwd(dh_last=P + 2) == 5

    def step(lam):
        return lib.ms_gated_step(P, P, P, P, lam, 8.0, None, P, 65535, 65539, 65539, 1, None)

    assert step(P + 4) == large and step(P + 2) == 5

    def lookup(ids, bits):
        return lib.ms_embed_fwd(ids, bits, P, 1.0, P, many, 10, 1 << 12, 0, None)

    assert lookup(P + 8, 64) == large and lookup(P + 4, 32) == large
    assert lookup(P + 4, 64) == 5 and lookup(P + 2, 32) == 5

    def table(ids=P, bits=64, dy=P, io=1):
        return lib.ms_embed_bwd(ids, bits, dy, 1.0, -1, P, 0, 5000, 10, 8, io, None, 0, None)

    assert table(ids=P + 8, dy=P + 2) == none and table(ids=P + 4, bits=32, dy=P + 4, io=0) == none
    assert table(ids=P + 4) == 5 and table(dy=P + 1) == 5 and table(dy=P + 2, io=0) == 5

    def logp(t, bits):
        return lib.ms_token_logprobs_fwd(P, 100000, t, bits, 1.0, P, P, P, P, 0, None, None, 1, 100000,
                                         0, None, 0, None)

    assert logp(P + 8, 64) == none and logp(P + 4, 32) == none
    assert logp(P + 4, 64) == 5 and logp(P + 1, 32) == 5

    def grad(t=P, stats=P, ent=P, gl=P, gh=P):
        return lib.ms_token_logprobs_bwd(P, 1 << 20, t, 64, 1.0, stats, ent, gl, gh, P, 1 << 20,
                                         (1 << 24) - 1, 1 << 20, 0, None)

    assert grad(t=P + 8, stats=P + 4, ent=P + 12, gl=P + 4, gh=P + 8) == large
    for bad in ("stats", "ent", "gl", "gh", "t"):
        assert grad(**{bad: P + 2}) == 5, bad


def test_handle_0_is_the_default_stream(monkeypatch):
    """torch makes a stream of its own of an external handle of 0."""
    current, default = (types.SimpleNamespace(cuda_stream=k) for k in (1, 0))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda k: 1, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda k=None: current)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda k=None: default)
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda h, device=None: types.SimpleNamespace(cuda_stream=h or 77))
    like = types.SimpleNamespace(get_device=lambda: 0, device="cuda:0")
    call = ms.lm._Call(None, like, 0)
    assert call.stream == 0 and call.other is default
    assert ms.lm._Call(None, like, 5).other.cuda_stream == 5
