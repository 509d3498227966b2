"""Host-only checks of the C ABI of the linear attention, the group norm and
the verification of drafts: sizes, and every refusal that needs no GPU (nothing
is launched on any of these calls)."""
import ctypes

import selective_state_space_81_amd as ms

NONE = ctypes.c_size_t(-1).value
P = 16  # an aligned address that is never read
INF, NAN = float("inf"), float("nan")


def test_sizes():
    lib = ms.load()
    # blocks of 64 tokens in bf16, 32 in fp32; whole tiles of 16 channels
    assert lib.ms_linear_attn_states_bytes(2, 65, 3, 17, 64, 1) == 2 * 2 * 3 * 32 * 64 * 4
    assert lib.ms_linear_attn_states_bytes(2, 65, 3, 17, 64, 0) == 2 * 3 * 3 * 32 * 64 * 4
    assert lib.ms_linear_attn_workspace_bytes(64, 4096, 24, 1, 128, 64, 1) == 0
    assert 0 < lib.ms_linear_attn_workspace_bytes(1, 100000, 2, 1, 64, 64, 1) < 1 << 30
    for bad in ((0, 5, 2, 1, 8, 8, 1), (1, 0, 2, 1, 8, 8, 1), (1, 1 << 31, 2, 1, 8, 8, 1),
                (1, 5, 0, 1, 8, 8, 1), (1, 5, 2, 0, 8, 8, 1), (1, 5, 3, 2, 8, 8, 1),
                (1, 5, 2, 4, 8, 8, 1), (1, 5, 2, 1, 0, 8, 1), (1, 5, 2, 1, 8, 0, 1),
                (1, 5, 2, 1, 129, 8, 1), (1, 5, 2, 1, 8, 129, 1), (1, 5, 2, 1, 8, 8, 2),
                (1 << 20, 5, 1 << 10, 1, 8, 8, 1)):
        assert lib.ms_linear_attn_workspace_bytes(*bad) == NONE, bad
        assert lib.ms_linear_attn_bwd_workspace_bytes(*bad[:6], 0, bad[6]) == NONE, bad
    assert lib.ms_linear_attn_bwd_workspace_bytes(2, 65, 3, 3, 17, 64, 1, 1) > \
        lib.ms_linear_attn_bwd_workspace_bytes(2, 65, 3, 3, 17, 64, 0, 1) > 0
    assert lib.ms_group_norm_bwd_workspace_bytes(0, 3, 8, 1) == 2 * 24 * 4
    for bad in ((-1, 3, 8, 1), (5, 0, 8, 1), (5, 3, 0, 1), (5, 3, 8193, 1), (5, 1 << 14, 8192, 1),
                (5, 3, 8, 7), (1 << 31, 3, 8, 1)):
        assert lib.ms_group_norm_bwd_workspace_bytes(*bad) == NONE, bad
    assert lib.ms_verify_drafts_workspace_bytes(0, 3, 100, 1, 1) == 0
    assert lib.ms_verify_drafts_workspace_bytes(2, 0, 100, 0, 1) > 0
    for bad in ((-1, 3, 100, 1, 1), (2, -1, 100, 1, 1), (2, 65, 100, 1, 1), (2, 3, 0, 1, 1),
                (2, 3, 1 << 31, 1, 1), (2, 3, 100, 1, 2), (1 << 30, 3, 100, 1, 1)):
        assert lib.ms_verify_drafts_workspace_bytes(*bad) == NONE, bad


def test_linear_attn_refusals():
    lib = ms.load()

    def fwd(q=P, k=P, v=P, g=P, o=P, ldq=16, ldk=16, ldv=32, scale=1.0, h0=None, states=None, b=1,
            L=40, h=4, hk=2, dk=8, dv=8, io=1, ws=P, n=1 << 40):
        return lib.ms_linear_attn_fwd(q, ldq, k, ldk, v, ldv, g, 0, scale, None, o, h0, None,
                                      states, b, L, h, hk, dk, dv, io, ws, n, None)

    for name in ("q", "k", "v", "g", "o"):
        assert fwd(**{name: None}) == 1, name
    assert fwd(ldq=15) == 2 and fwd(ldk=15) == 2 and fwd(ldv=31) == 2 and fwd(ldv=1 << 41) == 7
    assert fwd(scale=INF) == 2 and fwd(scale=NAN) == 2
    assert fwd(b=0) == 2 and fwd(L=0) == 2 and fwd(h=3) == 2 and fwd(io=5) == 3
    assert fwd(dk=129, ldq=512, ldk=512) == 7
    assert fwd(q=17) == 5 and fwd(q=18, o=18) == 5 and fwd(h0=8) == 5 and fwd(states=4) == 5
    assert fwd(g=18) == 5
    assert fwd(L=100000, ws=None) == 6 and fwd(L=100000, n=8) == 6
    assert b"workspace" in lib.ms_last_error()

    def bwd(do=P, dq=P, dg=P, states=P, dh0=None, ws=P, n=1 << 40):
        return lib.ms_linear_attn_bwd(P, 16, P, 16, P, 32, P, 0, 1.0, None, states, do, None, dq, P,
                                      P, dg, dh0, 1, 40, 4, 2, 8, 8, 1, ws, n, None)

    assert bwd(do=None) == 1 and bwd(dq=None) == 1 and bwd(dg=None) == 1 and bwd(states=None) == 1
    assert bwd(dq=18) == 5 and bwd(dg=20) == 5 and bwd(dh0=4) == 5 and bwd(do=17) == 5
    assert bwd(ws=None) == 6 and bwd(n=64) == 6

    def step(h=P, q=P, k=P, o=P, counts=None, update=1, T=3, ldk=16, dk=8):
        return lib.ms_linear_attn_step(h, q, 16, k, ldk, P, 32, P, 0, 1.0, counts, update, o, 2, T,
                                       4, 2, dk, 8, 1, None)

    assert step(h=None) == 1 and step(k=None) == 1 and step(o=None) == 1
    assert step(q=None, o=None, update=0) == 1
    assert step(T=0) == 2 and step(T=65) == 7 and step(ldk=15) == 2 and step(dk=0) == 2
    assert step(h=20) == 5 and step(o=20) == 5 and step(counts=18) == 5


def test_group_norm_refusals():
    lib = ms.load()

    def fwd(x=P, y=P, ldx=24, z=None, ldz=24, first=0, eps=1e-5, rows=5, groups=3, size=8, io=1):
        return lib.ms_group_norm_fwd(x, ldx, None, None, z, ldz, 1, first, eps, y, rows, groups, size,
                                     io, None)

    assert fwd(x=None) == 1 and fwd(y=None) == 1 and fwd(first=1) == 1
    assert fwd(ldx=23) == 2 and fwd(z=P, ldz=23) == 2 and fwd(rows=-1) == 2 and fwd(groups=0) == 2
    for eps in (0.0, -1.0, INF, NAN):
        assert fwd(eps=eps) == 2
    assert fwd(io=2) == 3 and fwd(size=8193, ldx=1 << 20) == 7
    assert fwd(y=24) == 5 and fwd(x=17) == 5
    assert fwd(rows=0, x=None, y=None) == 0  # nothing to do

    def bwd(dx=P, dy=P, z=None, dz=None, dw=P, ws=P, n=1 << 40, rows=5):
        return lib.ms_group_norm_bwd(P, 24, None, None, z, 24, 1, 0, 1e-5, dy, dx, dz, dw, None, rows,
                                     3, 8, 1, ws, n, None)

    assert bwd(dx=None) == 1 and bwd(dy=None) == 1 and bwd(z=P) == 1
    assert bwd(ws=None) == 6 and bwd(n=8) == 6 and bwd(dx=24) == 5 and bwd(dw=20) == 5
    assert bwd(dw=None, ws=None, rows=0) == 0


def test_verify_refusals():
    lib = ms.load()

    def f(logits=P, ld=100, q=P, ldd=100, ids=P, bits=64, u=P, scale=1.0, tokens=P, b=2, n=3,
          vocab=100, io=1, ws=P, size=1 << 40):
        return lib.ms_verify_drafts(logits, ld, q, ldd, ids, bits, u, scale, tokens, P, P, b, n, vocab,
                                    io, ws, size, None)

    assert f(logits=None) == 1 and f(ids=None) == 1 and f(u=None) == 1 and f(tokens=None) == 1
    assert f(ld=99) == 2 and f(ldd=99) == 2 and f(n=65) == 2 and f(n=-1) == 2 and f(vocab=0) == 2
    assert f(bits=16) == 3 and f(io=2) == 3
    for scale in (0.0, -1.0, INF, NAN):
        assert f(scale=scale) == 2
    assert f(logits=17) == 5 and f(ids=20) == 5 and f(u=18) == 5 and f(ws=8) == 5
    assert f(ws=None) == 6 and f(size=16) == 6
    assert f(b=0, logits=None) == 0  # nothing to do
