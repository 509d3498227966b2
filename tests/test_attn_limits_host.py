"""Limits of the linear attention's launches: each pass refuses only what it would
need too many workgroups for itself."""
import ctypes

import selective_state_space_81_amd as ms

NONE = ctypes.c_size_t(-1).value


def test_passes_have_limits_of_their_own():
    lib = ms.load()
    fwd, bwd, states = (lib.ms_linear_attn_workspace_bytes, lib.ms_linear_attn_bwd_workspace_bytes,
                        lib.ms_linear_attn_states_bytes)
    # 64 rows of 65536 tokens, 256 heads of 16 x 16: 1024 blocks a row
    assert fwd(64, 65536, 256, 1, 16, 16, 1) == 0
    assert states(64, 65536, 256, 16, 16, 1) == 64 * 1024 * 256 * 16 * 16 * 4
    # the backward takes a workgroup for each block and head of keys: 2^16, or 2^24
    assert bwd(64, 65536, 256, 1, 16, 16, 0, 1) == states(64, 65536, 256, 16, 16, 1)
    assert bwd(64, 65536, 256, 256, 16, 16, 0, 1) == NONE
    # the forward one for each head and 64 columns, whatever the blocks
    assert fwd(64, 65536, 256, 256, 16, 16, 1) == 0
    # no backward at all: 2^24 blocks
    assert states(1 << 14, 65536, 2, 16, 16, 1) == NONE
    assert fwd(1 << 14, 65536, 2, 1, 16, 16, 1) == 0


def test_python_has_the_same():
    assert ms.linear_attn_states_bytes(64, 65536, 256, 16, 16, 1) == 64 * 1024 * 256 * 16 * 16 * 4
    assert ms.linear_attn_workspace_bytes(64, 65536, 256, 256, 16, 16, 1) == 0
