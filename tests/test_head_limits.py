"""Host-side limits of the attn_head_* calls (no kernel is launched)."""

import numpy as np
import pytest

import bwd_causal_sdpa_b200 as A

P = 1 << 20  # a fake, aligned address


@pytest.mark.parametrize("is_bwd", [False, True])
def test_subnormal_temperatures_are_refused(is_bwd):
    """The kernels scale logits by log2(e) / temperature, which overflows below
    4.3e-39: such calls answered with NaN. Everything below the normal range is
    refused; the smallest normal number goes on to the next check."""

    def call(tau):
        if is_bwd:
            return A.attn_head_distill_bwd(P, P, P, P, tau, P, P, None, P, P, 10, 100, 64, 4, A.ATTN_F32,
                                           A.ATTN_F32, None, 0)
        return A.attn_head_distill(P, P, P, P, tau, P, P, 10, 100, 64, 4, A.ATTN_F32, None, 0)

    tiny = float(np.finfo(np.float32).tiny)
    for tau in (3e-39, 4.2e-39, 1e-38, np.nextafter(np.float32(tiny), np.float32(0))):
        assert call(float(tau)) == A.ATTN_EINVAL
    for tau in (tiny, 1e-30, 1e30, float(np.finfo(np.float32).max)):
        assert call(tau) == A.ATTN_EWORKSPACE


SIZES = [(n, v, c) for n in (1, 100, 256, 257, 300, 2048, 8192, 21504, 21505, 40000)
         for v in (1, 500, 1000, 32063, 50000, 1 << 20, 1 << 22) for c in (8, 64, 768, 2048)]


@pytest.mark.parametrize("is_bwd", [0, 1])
def test_workspaces_keep_the_stated_bounds(is_bwd):
    """What include/attn.h states, for single targets and for teachers."""
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    for n, v, c in SIZES:
        got = A.attn_head_workspace_bytes(n, v, c, 0, is_bwd)
        rows, ids = up(n), up(v)
        if is_bwd:
            dz = 3 * (96 << 20) if rows <= 21504 else 3 * 4608 * rows + (1 << 20)
            bound = dz + max(4 * rows * c, 20_000_000)
        else:
            bound = max(rows * ids // 16, 300 << 10)
        bound += rows * (2 * c + 64) + ids // 16 + 8192
        assert 0 < got <= bound, (n, v, c)
        for k in (1, 2, 4, 5, 7, 64, 1024):
            more = A.attn_head_workspace_bytes(n, v, c, k, is_bwd) - got
            assert more <= rows * (12 * k + ids // 32 + 32) + 8192, (n, v, c, k)


def test_one_piece_takes_one_buffer_of_dz():
    """256 rows of width 64 against 1000 ids: one buffer of 256 x 1024 entries of
    dz, one of the second term as large, and beside them x (32 KiB), the sums of
    dx (fp32, at most 4 parts: K blocks go 8 to a part) and the rows' arrays."""
    dz = 256 * 1024 * 2
    got = A.attn_head_workspace_bytes(256, 1000, 64, 0, 1)
    assert 2 * dz < got < 2 * dz + 256 * 64 * 2 + 4 * 256 * 64 * 4 + 256 * 64 + 8192 < 3 * dz
