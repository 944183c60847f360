"""Host-side checks of the attn_head_* calls and their workspace (no kernel is
launched: every call here fails validation)."""

import pytest

import bwd_causal_sdpa_b200 as A

P = 1 << 20  # a fake, aligned address


def _ce(**kw):
    a = dict(x=P, w=P, target=P, loss=P, lse=P, N=10, V=100, C=64, workspace=P, ws_bytes=1 << 40)
    return A.attn_head_ce(**{**a, **kw})


def _ce_bwd(**kw):
    a = dict(x=P, w=P, target=P, lse=P, dloss=P, dlse=None, dx=P, dw=P, N=10, V=100, C=64,
             dw_dtype=A.ATTN_BF16, workspace=P, ws_bytes=1 << 40)
    return A.attn_head_ce_bwd(**{**a, **kw})


def _distill(**kw):
    a = dict(x=P, w=P, t_idx=P, t_logit=P, temperature=1.0, loss=P, lse=P, N=10, V=100, C=64, K=4,
             t_dtype=A.ATTN_F32, workspace=P, ws_bytes=1 << 40)
    return A.attn_head_distill(**{**a, **kw})


def _distill_bwd(**kw):
    a = dict(x=P, w=P, t_idx=P, t_logit=P, temperature=1.0, lse=P, dloss=P, dlse=P, dx=P, dw=P,
             N=10, V=100, C=64, K=4, t_dtype=A.ATTN_F32, dw_dtype=A.ATTN_F32, workspace=P,
             ws_bytes=1 << 40)
    return A.attn_head_distill_bwd(**{**a, **kw})


@pytest.mark.parametrize("call", [_ce, _ce_bwd, _distill, _distill_bwd])
def test_shared_validation(call):
    for name in ("x", "w", "lse"):
        assert call(**{name: None}) == A.ATTN_EINVAL
    for name in ("N", "V", "C"):
        assert call(**{name: 0}) == A.ATTN_EINVAL
        assert call(**{name: -8}) == A.ATTN_EINVAL
    assert call(C=60) == A.ATTN_EUNSUPPORTED          # rows not 16-byte strided
    assert call(C=(1 << 20) + 8) == A.ATTN_EUNSUPPORTED
    assert call(N=(1 << 26) + 1) == A.ATTN_EUNSUPPORTED
    assert call(V=(1 << 26) + 1) == A.ATTN_EUNSUPPORTED
    assert call(x=P + 8) == A.ATTN_EALIGN
    assert call(w=P + 2) == A.ATTN_EALIGN
    assert call(lse=P + 1) == A.ATTN_EALIGN
    assert call(workspace=P + 8) == A.ATTN_EALIGN
    assert call(workspace=None) == A.ATTN_EWORKSPACE
    assert call(ws_bytes=255) == A.ATTN_EWORKSPACE


def test_forward_validation():
    assert _ce(target=None) == A.ATTN_EINVAL
    for call in (_ce, _distill):
        assert call(loss=None) == A.ATTN_EINVAL
        assert call(loss=P + 2) == A.ATTN_EALIGN


def test_backward_validation():
    for call in (_ce_bwd, _distill_bwd):
        for name in ("dloss", "dx", "dw"):
            assert call(**{name: None}) == A.ATTN_EINVAL
        assert call(dw_dtype=3) == A.ATTN_EINVAL
        assert call(dx=P + 8) == A.ATTN_EALIGN
        assert call(dw=P + 4) == A.ATTN_EALIGN
        assert call(dlse=P + 2) == A.ATTN_EALIGN


def test_teacher_validation():
    for call in (_distill, _distill_bwd):
        assert call(t_idx=None) == A.ATTN_EINVAL
        assert call(t_logit=None) == A.ATTN_EINVAL
        assert call(K=0) == A.ATTN_EINVAL
        assert call(K=-1) == A.ATTN_EINVAL
        assert call(K=1025) == A.ATTN_EUNSUPPORTED
        for tau in (0.0, -1.0, float("inf"), float("nan"), 1e-45):
            assert call(temperature=tau) == A.ATTN_EINVAL
        assert call(t_dtype=7) == A.ATTN_EINVAL
        assert call(t_logit=P + 2) == A.ATTN_EALIGN
        assert call(t_idx=P + 2) == A.ATTN_EALIGN


def test_workspace_bytes():
    ws = A.attn_head_workspace_bytes
    for bad in ((0, 10, 64, 0), (10, 0, 64, 0), (10, 10, 0, 0), (10, 10, 60, 0), (10, 10, 64, -1),
                (10, 10, 64, 1025)):
        for b in (0, 1):
            assert ws(*bad, b) == 0
    # the forward keeps 8 bytes per 128 logits, never the logits
    assert ws(8192, 32063, 2048, 0, 0) < 8192 * 32063 * 2 // 8
    # the backward's does not grow with the vocabulary: three pieces of dz of at
    # most 96 MiB, the kept rows of x (bf16), the sums of dx (fp32), and small
    # arrays by row and by 256 vocabulary rows
    for v in (32063, 50000, 1 << 20, 1 << 22):
        got = ws(8192, v, 2048, 0, 1)
        assert got <= 3 * (96 << 20) + 8192 * 2048 * (2 + 4) + (1 << 20), v
    assert ws(8192, 32063, 2048, 0, 1) < 8192 * 32063 * 2
    # one buffer of dz where one piece holds the vocabulary
    assert ws(256, 1000, 64, 0, 1) % 256 == 0
    # units are numbered in 32 bits
    assert ws(1 << 26, 1 << 26, 64, 0, 1) == 0
    assert _ce(ws_bytes=ws(10, 100, 64, 0, 0) - 1) == A.ATTN_EWORKSPACE
    assert _ce_bwd(ws_bytes=ws(10, 100, 64, 0, 1) - 1) == A.ATTN_EWORKSPACE
    assert _distill(ws_bytes=ws(10, 100, 64, 4, 0) - 1) == A.ATTN_EWORKSPACE
    assert _distill_bwd(ws_bytes=ws(10, 100, 64, 4, 1) - 1) == A.ATTN_EWORKSPACE
