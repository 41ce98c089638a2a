"""Sizes of the linear cross entropy's workspaces, on the CPU."""

import pytest

MB = 1 << 20


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("N,D,V", [(1, 4096, 128256), (17, 4096, 151936), (17, 1024, 151936), (64, 8192, 151936),
                                   (128, 2048, 200000), (200, 4096, 151936), (300, 512, 128256)])
def test_few_states_need_no_room_for_a_head_that_is_read_in_place(N, D, V, dtype):
    """Heads of whole groups of 16 bytes a row: at most 128 MB of packed tokens, the copy
    of the states and what the call itself holds."""
    from lossless_draft_verification_sample_amd import _lib
    lib = _lib.load()
    sv_f32 = dtype == 0
    packed = 128 * MB + N * D * 4
    fwd = lib.spec_verify_linear_ce_workspace_bytes(N, D, V, dtype)
    assert 0 < fwd <= packed + -(-V // 64) * N * 8 + 4 * N + 2048
    bwd = lib.spec_verify_linear_ce_backward_workspace_bytes(N, D, V, dtype, 1, 1)
    # dz of all tokens at most, and of dh's splits 128 MB or one
    assert bwd <= packed + N * (V + 256) * 4 + max(128 * MB, N * D * 4) + 2048
    assert sv_f32 or fwd < 140 * MB


def test_wide_odd_heads_keep_their_piece():
    """They are packed by every call."""
    from lossless_draft_verification_sample_amd import _lib
    lib = _lib.load()
    assert lib.spec_verify_linear_ce_workspace_bytes(17, 4095, 151936, 1) > 256 * MB
