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
