"""How many bits of dz the gradients of the output head carry.

dz is the tensor cores' operand, in bf16 (half a step: 2^-8 relative). In two
terms, hi + lo, both bf16, what is left of an entry is half a step of lo:
2^-8 2^-8 = 2^-16. The library states where it takes two: for an fp32 dW, and
where at most 256 rows are kept; for a bf16 dW of more rows at the foremost
entry of each (the target, or a teacher's largest share); and dx gets what the
rounding takes from up to four named entries, of more of them from the foremost
one, in fp32. Bounds, element by element, as in test_head_gpu.py with that
half step in its place:

  D = b |dz| + (2 e + 2^-20) |a| p + 2^-20 |g| q,   b = 2^-16 or 2^-8,
  |dx error| <= D |W| + s |dz| |W| + 2^-8 |dx|,  dW likewise (its own rounding
  only where it is bf16),

where s = (n / 8 + 10) 2^-23 bounds a fp32 sum of two terms of n entries in
steps of 16, each cut at 24 bits.
"""

import numpy as np
import pytest

from oracle import head_dz, head_loss, head_loss_backward, target_lists, teacher_lists
from workloads import head_config_by_name, make_head_workload

pytestmark = pytest.mark.gpu


def _named(ids, q, V):
    """Shares over the vocabulary, and where the named and the foremost ids are."""
    rows = np.arange(ids.shape[0])
    share = np.zeros((ids.shape[0], V))
    named, foremost = np.zeros(share.shape, bool), np.zeros(share.shape, bool)
    here = ids >= 0
    at = np.broadcast_to(rows[:, None], ids.shape)
    np.add.at(share, (at, np.maximum(ids, 0)), np.where(here, q, 0.0))
    named[at[here], ids[here]] = True
    top = np.where(here, q, -1.0).argmax(axis=1)
    some = here.any(axis=1)
    foremost[rows[some], ids[rows, top][some]] = True
    return share, named, foremost


def _check(w, dw_f32, all_terms):
    """all_terms: at most 256 rows are kept."""
    from bwd_causal_sdpa_b200 import ATTN_BF16, ATTN_F32, ATTN_OK
    from bwd_causal_sdpa_b200.runner import HeadRunner

    c = w.cfg
    r = HeadRunner(w, dw_dtype=ATTN_F32 if dw_f32 else ATTN_BF16)
    r.forward()
    r.ws.fill_(0xFF)  # NaN: what the call has not written shows
    r.backward()
    assert r.status() == ATTN_OK
    got = r.results()
    ids, q = teacher_lists(w.t_idx, w.t_logit, c.V, c.tau) if c.K else target_lists(w.target, c.V)
    kept = (ids >= 0).any(axis=1)
    assert all_terms == (kept.sum() <= 256)
    x, W = w.x.astype(np.float64), w.w.astype(np.float64)
    x[~kept] = 0.0
    _, lse = head_loss(x, W, ids, q, c.tau)
    dz = np.abs(head_dz(x, W, ids, q, w.dloss, w.dlse, c.tau))
    dx, dw = head_loss_backward(x, W, ids, q, w.dloss, w.dlse, c.tau)
    share, named, foremost = _named(ids, q, c.V)
    S = (np.abs(x) @ np.abs(W).T / c.tau).max(axis=1)
    e = (c.C / 16 + 2) * 2.0**-23 * S + 2.0**-20 * (1 + np.abs(lse))
    p = np.exp(x @ W.T / c.tau - lse[:, None]) * kept[:, None]
    a = np.abs(w.dloss.astype(np.float64) + w.dlse) / c.tau
    slack = (2 * e + 2.0**-20)[:, None] * a[:, None] * p
    slack += 2.0**-20 * share * np.abs(w.dloss)[:, None] / c.tau
    two = all_terms or dw_f32
    b_dw = np.where(two | foremost, 2.0**-16, 2.0**-8)
    b_dx = np.where(named if c.K <= 4 else two | foremost, 2.0**-16, 2.0**-8)
    total = lambda n: (n / 8 + 10) * 2.0**-23  # noqa: E731
    b_dx = ((b_dx + total(c.V)) * dz + slack) @ np.abs(W) + 2.0**-8 * np.abs(dx)
    b_dw = ((b_dw + total(c.N)) * dz + slack).T @ np.abs(x)
    b_dw += (0.0 if dw_f32 else 2.0**-8) * np.abs(dw)
    for name, ref, bound in (("dx", dx, b_dx), ("dw", dw, b_dw)):
        off = np.abs(got[name] - ref)
        bad = ~(off <= bound + 1e-37)  # fp32 results below the normal range are flushed
        assert not bad.any(), (name, c, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                               (off / np.maximum(bound, 1e-37))[bad].max())


CONFIG = {0: "head_small", 1: "head_distill_small"}


def _workload(N, K, **kw):
    kw = {**dict(V=1000, C=200, left_out=0.0), **kw}
    w = make_head_workload(head_config_by_name(CONFIG[min(K, 1)]), N=N, K=K, seed=40 + N + K, **kw)
    # a mean over the rows: every target's dz near one value, and that at 129.5 /
    # 128, in the middle of two bf16 values (the farthest a rounding can be off)
    w.dloss[:] = np.float32(129.5 / 128 / 512)
    return w


@pytest.mark.parametrize("K", [0, 3, 40])
@pytest.mark.parametrize("N", [1, 70, 300, 700])
def test_fp32_dw_holds_two_terms(N, K):
    _check(_workload(N, K), True, N <= 256)


@pytest.mark.parametrize("K", [0, 2, 4, 5, 40])
@pytest.mark.parametrize("N,left_out", [(1, 0.0), (2, 0.0), (9, 0.5), (40, 0.0), (200, 0.1),
                                        (256, 0.0), (800, 0.7)])
def test_few_rows_hold_two_terms(N, left_out, K):
    _check(_workload(N, K, left_out=left_out), False, True)


@pytest.mark.parametrize("K", [0, 1, 3, 30])
@pytest.mark.parametrize("N,V,C,left_out", [(257, 5000, 72, 0.0), (700, 6000, 72, 0.0),
                                            (1100, 3001, 200, 0.3), (1500, 130, 64, 0.0),
                                            # narrow logits tiles, the last vocabulary tile half empty
                                            (600, 100, 64, 0.0), (450, 880, 72, 0.2),
                                            (2000, 1, 8, 0.0), (4099, 20000, 8, 0.9)])
def test_foremost_entries_of_many_rows_hold_two_terms(N, V, C, left_out, K):
    _check(_workload(N, K, V=V, C=C, left_out=left_out), False, False)


@pytest.mark.parametrize("K", [0, 1, 4])
def test_named_logits_are_rounded_sums(K):
    """z[target] = -45 as a sum of 2048 products of one sign, every other logit 0:
    loss = log(V - 1) + 45 up to e^-45 (and less the teacher's entropy). The library sums the few named logits in
    16 plain fp32 sums of 128 products; what an addition rounds off is spread over
    half a step either way. Its root mean square over all 2048 is at most
    sqrt(2048) 2^-22 / sqrt(12) (partial sums stay below 45 / 16 < 4): six times
    that, half a step (2^-19) for each of the 15 sums that join them at most, of
    which all but 7 are below 16 (2^-20, 2^-21: 2^-16 in all), and 2^-22 of the
    loss for the rest. A tensor core cuts the 128 partial sums of such a logit,
    each by up to a whole step in the same direction, 1.3e-4 on average."""
    from bwd_causal_sdpa_b200 import ATTN_OK
    from bwd_causal_sdpa_b200.runner import HeadRunner
    from workloads import round_to_bf16

    w = make_head_workload(head_config_by_name(CONFIG[min(K, 1)]), N=24, V=300, C=2048, K=K, tau=1.0,
                           left_out=0.0, ragged=False, seed=77)
    rng = np.random.default_rng(78)
    w.x[:] = round_to_bf16((1 + rng.random(w.x.shape)).astype(np.float32))
    w.w[:] = 0.0
    w.w[7] = round_to_bf16((-(1 + rng.random(2048)) * 20 / 2048).astype(np.float32))
    if K:
        w.t_idx[:] = 7  # the same id K times, each with a share of its own
    else:
        w.target[:] = 7
    z = w.x.astype(np.float64) @ w.w[7].astype(np.float64)
    assert (-64 < z).all() and (z < -32).all()
    r = HeadRunner(w)
    r.forward()
    assert r.status() == ATTN_OK
    want = np.log(299 + np.exp(z)) - z
    if K:
        _, q = teacher_lists(w.t_idx, w.t_logit, 300, 1.0)
        want += (q * np.log(q)).sum(axis=1)
    bound = 6 * np.sqrt(2048 / 12) * 2.0**-22 + 2.0**-16 + 2.0**-22 * want
    off = np.abs(r.results()["loss"] - want)
    assert (off <= bound).all(), (off.max(), bound.min())
