"""The output head's backward over many pieces of the vocabulary: buffers of dz
used again, sums of dx over all pieces, a shorter last piece, few and many kept
rows. Every element of dx and dW against float64 products on the device, with
the bounds of test_head_precision_gpu.py:

  D = b |dz| + (2 e + 2^-20) |a| p + 2^-20 |g| q,  b = 2^-16 (two terms) or 2^-8,
  |dx error| <= D |W| + s(V) |dz| |W| + 2^-8 |dx|,  dW likewise over the rows,

s(n) = (n / 8 + 10) 2^-23; between the pieces dx is added in fp32, a rounding
per piece that n / 8 covers (a piece has at least 1024 ids)."""

import numpy as np
import pytest

from oracle import target_lists, teacher_lists
from workloads import head_config_by_name, make_head_workload

pytestmark = pytest.mark.gpu


def _bounds(r, ids, q, dlse, dw_f32):
    """(dx, its bound, dW, its bound) in float64 on the device, some rows at a time."""
    import torch

    c = r.w.cfg
    x, W = r.x.double(), r.wt.double()
    ids, q = torch.from_numpy(ids).cuda(), torch.from_numpy(q).cuda()
    kept = (ids >= 0).any(dim=1)
    x = torch.where(kept[:, None], x, 0.0)
    dloss, dlse = r.dloss.double() * kept, dlse.double() * kept
    two = dw_f32 or int(kept.sum()) <= 256
    total = lambda n: (n / 8 + 10) * 2.0**-23  # noqa: E731
    dx, b_dx = torch.zeros_like(x), torch.zeros_like(x)
    dw, b_dw = torch.zeros_like(W), torch.zeros_like(W)
    aW = W.abs()
    step = max(32, min(1024, (1 << 26) // c.V))
    for i in range(0, c.N, step):
        s = slice(i, i + step)
        z = x[s] @ W.T / c.tau
        lse = torch.logsumexp(z, dim=1)
        p = torch.exp(z - lse[:, None]) * kept[s, None]
        at, here = ids[s].clamp(min=0), ids[s] >= 0
        share = torch.zeros_like(z).scatter_add_(1, at, q[s] * here)
        named = torch.zeros_like(z).scatter_add_(1, at, here.double()) > 0
        top = torch.where(here, q[s], -1.0).argmax(dim=1, keepdim=True)
        first = torch.zeros_like(z).scatter_(1, at.gather(1, top), 1.0) > 0
        dz = (p * (dloss + dlse)[s, None] - share * dloss[s, None]) / c.tau
        S = (x[s].abs() @ aW.T / c.tau).amax(dim=1)
        e = (c.C / 16 + 2) * 2.0**-23 * S + 2.0**-20 * (1 + lse.abs())
        slack = (2 * e + 2.0**-20)[:, None] * ((dloss + dlse)[s].abs() / c.tau)[:, None] * p
        slack += 2.0**-20 * share * dloss[s, None].abs() / c.tau
        fine = lambda where: torch.where(where, 2.0**-16, 2.0**-8)  # noqa: E731
        far = torch.ones_like(first) if two else first
        a = dz.abs()
        dx[s] = dz @ W
        b_dx[s] = ((fine(named if c.K <= 4 else far) + total(c.V)) * a + slack) @ aW
        dw += dz.T @ x[s]
        if not two and c.V > 1 << 20:  # rows are not sorted: one term in dW
            far = torch.zeros_like(first)
        b_dw += ((fine(far) + total(c.N)) * a + slack).T @ x[s].abs()
    b_dx += 2.0**-8 * dx.abs()
    if not dw_f32:
        b_dw += 2.0**-8 * dw.abs()
    return dx, b_dx, dw, b_dw


# more than 21504 rows take pieces of 2048 ids with a bf16 dW (1024 with an fp32
# one: half of that is its second term), whatever the width
@pytest.mark.parametrize("N,V,C,K,left_out,dw_f32", [
    (25000, 12500, 64, 0, 0.0, False),      # 7 pieces, the last one 212 ids
    (25000, 12500, 72, 3, 0.0, False),
    (25000, 12500, 64, 20, 0.2, False),
    (25000, 12500, 264, 3, 0.97, False),    # 750 rows kept: dx split over units
    (25000, 12500, 72, 0, 0.995, False),    # 125 kept: two terms
    (25000, 12500, 72, 9, 0.995, False),
    (25000, 61000, 64, 0, 0.5, False),      # 30 pieces
    (25000, 8300, 64, 3, 0.0, True),        # 9 pieces
    (9000, 33000, 200, 0, 0.1, False),      # longer pieces
    (9000, 33000, 72, 2, 0.93, True),
    (300, 1 << 20, 16, 0, 0.0, False),      # the most tiles that rows are sorted by
    (300, 1050000, 16, 0, 0.0, False),      # more of them
    (300, 1050000, 8, 9, 0.0, False),
    (40, 1050000, 8, 0, 0.0, False),
])
def test_every_element_over_many_pieces(N, V, C, K, left_out, dw_f32):
    import torch

    from bwd_causal_sdpa_b200 import ATTN_BF16, ATTN_F32, ATTN_OK
    from bwd_causal_sdpa_b200.runner import HeadRunner

    w = make_head_workload(head_config_by_name("head_distill_small" if K else "head_small"), N=N, V=V,
                           C=C, K=K, left_out=left_out, seed=20 + K)
    r = HeadRunner(w, dw_dtype=ATTN_F32 if dw_f32 else ATTN_BF16)
    r.ws.fill_(0xFF)  # NaN: what no unit has written shows
    r.forward()
    r.ws.fill_(0xFF)
    r.dx.fill_(7.0)
    r.dw.fill_(7.0)
    r.backward()
    assert r.status() == ATTN_OK
    ids, q = teacher_lists(w.t_idx, w.t_logit, V, w.cfg.tau) if K else target_lists(w.target, V)
    dx, b_dx, dw, b_dw = _bounds(r, ids, q, r.dlse, dw_f32)
    for name, got, ref, bound in (("dx", r.dx, dx, b_dx), ("dw", r.dw, dw, b_dw)):
        off = (got.double() - ref).abs()
        bad = ~(off <= bound + 1e-37)
        assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[:3].tolist(),
                               (off / bound)[bad].max().item())
    again = r.dx.clone(), r.dw.clone()
    r.backward()
    assert torch.equal(again[0], r.dx) and torch.equal(again[1], r.dw)
