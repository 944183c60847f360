"""The losses of the output head against the float64 oracle.

Tolerances, element by element, from the roundings that the calls make. With
S = |x| |W|^T / tau (per logit, the sum of its absolute products):

  * a logit is a fp32 sum of C products taken 16 at a time: off by at most
    (C / 16 + 2) 2^-23 S when every partial sum is cut at 24 bits. With that,
    a few fp32 roundings of the exponent, the sum and the logarithm (2^-20
    relative to 1 + |lse|):
    e = (C / 16 + 2) 2^-23 max_v S + 2^-20 (1 + |lse|);  |lse error| <= e and
    |loss error| <= 2 e + 2^-20 |loss terms|;
  * dz = a p - g q carries exp's relative error (e of the logit and of lse,
    together 2 e, plus 2^-20) in the first term and half a bf16 step, 2^-8, in
    all; its products are fp32 sums. With
    D = 2^-8 |dz| + (2 e + 2^-20) |a| p + 2^-20 |g| q:
    |dx error| <= D |W| + 2^-14 |dz| |W| + 2^-8 |dx|, likewise dW (the last
    term only where dW is bf16), where 2^-14 bounds a fp32 sum of up to
    2^9 x 16 terms and the last terms are the output's half step.
"""

import numpy as np
import pytest

from oracle import (head_dz, head_loss, head_loss_backward, out_projection,
                    out_projection_backward, target_lists, teacher_lists)
from workloads import head_config_by_name, make_head_workload

pytestmark = pytest.mark.gpu


def _lists(w, t_logit=None):
    c = w.cfg
    if c.K:
        return teacher_lists(w.t_idx, w.t_logit if t_logit is None else t_logit, c.V, c.tau)
    return target_lists(w.target, c.V)


def _bounds(w, ids, q, loss, lse, dloss, dlse, dw_f32):
    c = w.cfg
    kept = (ids >= 0).any(axis=1)
    x = np.where(kept[:, None], w.x, 0.0).astype(np.float64)
    W = w.w.astype(np.float64)
    S = (np.abs(x) @ np.abs(W).T / c.tau).max(axis=1)
    e = (c.C / 16 + 2) * 2.0**-23 * S + 2.0**-20 * (1 + np.abs(lse))
    entropy = np.where(q > 0, q * np.abs(np.log(np.where(q > 0, q, 1.0))), 0.0).sum(axis=1)
    b_loss = 2 * e + 2.0**-20 * (entropy + np.abs(lse) + S + np.abs(loss))
    dz = head_dz(x, W, ids, q, dloss, dlse, c.tau)
    g = np.where(kept, dloss, 0.0) / c.tau
    a = np.abs(g + (0.0 if dlse is None else np.where(kept, dlse, 0.0) / c.tau))
    share = np.zeros((c.N, c.V))
    rows = np.broadcast_to(np.arange(c.N)[:, None], ids.shape)
    np.add.at(share, (rows, np.maximum(ids, 0)), np.where(ids >= 0, q, 0.0) * np.abs(g)[:, None])
    z = x @ W.T / c.tau
    p = np.exp(z - z.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    D = 2.0**-8 * np.abs(dz) + (2 * e + 2.0**-20)[:, None] * a[:, None] * p + 2.0**-20 * share
    D = np.where(kept[:, None], D, 0.0) + 2.0**-14 * np.abs(dz)
    dx, dw = head_loss_backward(x, W, ids, q, dloss, dlse, c.tau)
    b_dx = D @ np.abs(W) + 2.0**-8 * np.abs(dx)
    b_dw = D.T @ np.abs(x) + (0.0 if dw_f32 else 2.0**-8) * np.abs(dw)
    return dict(loss=b_loss, lse=e, dx=b_dx, dw=b_dw), dict(dx=dx, dw=dw)


def _check(w, t_dtype=1, dw_dtype=0, with_dlse=True, stream=None):
    import torch

    from bwd_causal_sdpa_b200 import ATTN_BF16, ATTN_F32, ATTN_OK
    from bwd_causal_sdpa_b200.runner import HeadRunner

    c = w.cfg
    r = HeadRunner(w, t_dtype=t_dtype, dw_dtype=dw_dtype, with_dlse=with_dlse, stream=stream)
    r.forward()
    r.backward()
    assert r.status() == ATTN_OK
    got = r.results()
    t_logit = None
    if c.K:
        t_logit = r.t_logit.to(torch.float64).cpu().numpy()
    assert t_dtype in (ATTN_BF16, ATTN_F32)
    ids, q = _lists(w, t_logit)
    dlse = w.dlse if with_dlse else None
    loss, lse = head_loss(w.x, w.w, ids, q, c.tau)
    bounds, ref = _bounds(w, ids, q, loss, lse, w.dloss, dlse, dw_dtype == ATTN_F32)
    ref.update(loss=loss, lse=lse)
    for name in ("loss", "lse", "dx", "dw"):
        off = np.abs(got[name] - ref[name])
        tiny = 1e-37  # fp32 results below the normal range are flushed
        bad = ~(off <= bounds[name] + tiny)
        assert not bad.any(), (name, c, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                               got[name][bad][:3], ref[name][bad][:3], bounds[name][bad][:3])
    kept = (ids >= 0).any(axis=1)
    for name in ("loss", "lse", "dx"):
        assert not got[name][~kept].any(), name
    return r, got


SIZES = [(1, 1, 8), (1, 257, 8), (2, 256, 64), (3, 255, 72), (127, 130, 136), (128, 512, 256),
         (129, 513, 200), (256, 300, 264), (257, 1000, 128), (300, 2049, 768), (600, 777, 520)]


@pytest.mark.parametrize("N,V,C", SIZES)
def test_cross_entropy_sizes(N, V, C):
    w = make_head_workload(head_config_by_name("head_small"), N=N, V=V, C=C, left_out=0.0,
                           seed=60 + N)
    _check(w)


@pytest.mark.parametrize("N,V,C", SIZES[1:])
@pytest.mark.parametrize("K,tau", [(1, 1.0), (5, 0.7), (33, 3.0)])
def test_distillation_sizes(N, V, C, K, tau):
    w = make_head_workload(head_config_by_name("head_distill_small"), N=N, V=V, C=C, K=K, tau=tau,
                           left_out=0.0, seed=70 + N)
    _check(w)


@pytest.mark.parametrize("name", ["head_small", "head_distill_small"])
@pytest.mark.parametrize("left_out", [0.0, 0.1, 0.5, 0.95, 1.0])
@pytest.mark.parametrize("N", [1, 300, 1031])
def test_left_out_rows(name, left_out, N):
    """Rows left out hold NaN and infinities, which must reach nothing."""
    w = make_head_workload(head_config_by_name(name), left_out=left_out, N=N, seed=80 + N)
    out = w.target < 0 if w.cfg.K == 0 else (w.t_idx < 0).all(axis=1)
    w.x[out] = np.where(np.arange(w.cfg.C) % 2, np.nan, np.inf)
    _check(w)


@pytest.mark.parametrize("t_dtype", [0, 1])
@pytest.mark.parametrize("dw_dtype", [0, 1])
@pytest.mark.parametrize("with_dlse", [False, True])
def test_types(t_dtype, dw_dtype, with_dlse):
    for name in ("head_small", "head_distill_small"):
        _check(make_head_workload(head_config_by_name(name)), t_dtype, dw_dtype, with_dlse)


def test_zero_upstream_rows_have_no_gradients():
    for name in ("head_small", "head_distill_small"):
        w = make_head_workload(head_config_by_name(name), left_out=0.0)
        w.dloss[::3] = 0.0
        w.dlse[::6] = 0.0  # rows 0, 6, ..: neither; rows 3, 9, ..: dlse alone
        _check(w)


@pytest.mark.parametrize("N,left_out,C", [(8200, 0.0, 64), (8200, 0.995, 64), (8200, 0.995, 72),
                                          (8200, 0.97, 520)])
def test_several_pieces_of_the_vocabulary(N, left_out, C):
    """More logits than one dz buffer holds; with few kept rows the vocabulary
    axis of dx is split too, and the last piece is shorter than the others."""
    w = make_head_workload(head_config_by_name("head_small"), N=N, V=8500, C=C, left_out=left_out)
    _check(w)


def test_many_entries_in_the_first_tile():
    """A teacher whose entries crowd a few ids, named twice and in any order."""
    w = make_head_workload(head_config_by_name("head_distill_small"), N=130, V=700, K=300,
                           ragged=False, left_out=0.0)
    w.t_idx[:] = np.random.default_rng(7).integers(0, 40, w.t_idx.shape)
    w.t_idx[:, ::7] = 699
    _check(w)


def test_teacher_entries_at_the_edges():
    w = make_head_workload(head_config_by_name("head_distill_small"), N=8, K=4, left_out=0.0,
                           ragged=False)
    w.t_idx[0] = [-1, 5, -7, 999]
    w.t_logit[0] = [np.nan, 1.0, np.inf, 2.0]        # what absent entries hold is not read
    w.t_logit[1] = [-np.inf, 0.0, -np.inf, 1.0]      # q = 0 beside others
    w.t_logit[2] = -np.inf                           # nothing left: the row is left out
    w.t_logit[3] = np.finfo(np.float32).min          # the type's lowest value everywhere
    w.t_logit[4] = [np.finfo(np.float32).min, 0, 0, 3.0]
    w.t_logit[5] = [1e4, -1e4, 9.99e3, 0.0]
    w.t_idx[6] = [255, 256, 0, 999]
    w.t_idx[7] = [3, 3, 3, 3]
    _check(w)


@pytest.mark.parametrize("scale", [1e-3, 8.0, 64.0])
def test_logit_scales(scale):
    """From flat to one-hot softmax (logits of several hundred)."""
    w = make_head_workload(head_config_by_name("head_small"))
    w.x *= np.float32(scale)
    from workloads import round_to_bf16
    w.x = round_to_bf16(w.x)
    _check(w)


def test_bad_ids_are_reported_and_absent():
    import torch

    from bwd_causal_sdpa_b200 import ATTN_EDEVICE_INPUT, ATTN_OK
    from bwd_causal_sdpa_b200.runner import HeadRunner

    for name in ("head_small", "head_distill_small"):
        w = make_head_workload(head_config_by_name(name), left_out=0.0)
        bad = make_head_workload(head_config_by_name(name), left_out=0.0)
        if w.cfg.K:
            w.t_idx[5, 0] = -1
            bad.t_idx[5, 0] = w.cfg.V
        else:
            w.target[5] = -1
            bad.target[5] = 2**31 - 1
        out = []
        for v, code in ((w, ATTN_OK), (bad, ATTN_EDEVICE_INPUT)):
            r = HeadRunner(v)
            r.forward()
            assert r.status() == code
            r.backward()
            assert r.status() == code
            out.append([getattr(r, n).clone() for n in ("loss", "lse", "dx", "dw")])
        for a, b in zip(*out):
            assert torch.equal(a, b)


def test_nan_and_infinity_in_kept_rows_stay_in_their_rows():
    import torch

    from bwd_causal_sdpa_b200.runner import HeadRunner

    w = make_head_workload(head_config_by_name("head_small"), left_out=0.0)
    clean = HeadRunner(w)
    clean.forward()
    w.x[7, 3] = np.nan
    w.x[40, 5] = np.inf
    r = HeadRunner(w)
    r.forward()
    torch.cuda.synchronize()
    rest = torch.ones(w.cfg.N, dtype=torch.bool, device="cuda")
    rest[[7, 40]] = False
    for n in ("loss", "lse"):
        a, b = getattr(r, n), getattr(clean, n)
        assert torch.isnan(a[7]) and not torch.isfinite(a[40])
        assert torch.equal(a[rest], b[rest])


@pytest.mark.parametrize("N", [40, 300])
def test_a_target_whose_logit_overflows(N):
    """A target at -inf: its loss is inf, its row's lse and every other row are
    what they are without it."""
    import torch

    from bwd_causal_sdpa_b200 import ATTN_OK
    from bwd_causal_sdpa_b200.runner import HeadRunner

    w = make_head_workload(head_config_by_name("head_small"), N=N, left_out=0.0)
    w.w[:, :2] = 0.0
    w.w[5, :2] = -1.0
    w.x[:, :2] = 0.0
    w.target[w.target == 5] = 6
    clean, _ = _check(w)
    w.x[3, :2] = np.float32(2.0**127)
    w.target[3] = 5
    r = HeadRunner(w)
    r.forward()
    assert r.status() == ATTN_OK
    z = w.x[3, 2:].astype(np.float64) @ w.w[np.arange(w.cfg.V) != 5, 2:].astype(np.float64).T
    want = np.log(np.exp(z - z.max()).sum()) + z.max()
    assert r.loss[3].item() == np.inf
    assert abs(r.lse[3].item() - want) <= 1e-5 * (1 + abs(want))
    rest = torch.arange(N, device="cuda") != 3
    assert torch.equal(r.loss[rest], clean.loss[rest]) and torch.equal(r.lse[rest], clean.lse[rest])


def test_same_call_same_bits_and_nothing_behind_is_written():
    """Outputs inside larger buffers: what lies behind them stays."""
    import torch

    import bwd_causal_sdpa_b200 as A
    from bwd_causal_sdpa_b200.runner import HeadRunner

    w = make_head_workload(head_config_by_name("head_small"), N=301, V=999, C=200)
    c = w.cfg
    r = HeadRunner(w)
    bufs = []
    for _ in range(2):
        r.ws.fill_(0xFF)  # NaN everywhere: nothing is read that the call has not written
        pad = dict(device="cuda")
        loss, lse = (torch.full((c.N + 64,), 7.0, **pad) for _ in range(2))
        dx = torch.full((c.N + 3, c.C), 7.0, dtype=torch.bfloat16, **pad)
        dw = torch.full((c.V + 3, c.C), 7.0, dtype=torch.bfloat16, **pad)
        A.check(A.attn_head_ce(r.x, r.wt, r.target, loss, lse, c.N, c.V, c.C, r.ws, r.ws_bytes))
        r.ws.fill_(0xFF)
        A.check(A.attn_head_ce_bwd(r.x, r.wt, r.target, lse, r.dloss, r.dlse, dx, dw, c.N, c.V,
                                   c.C, A.ATTN_BF16, r.ws, r.ws_bytes))
        torch.cuda.synchronize()
        for t, n in ((loss, c.N), (lse, c.N), (dx, c.N), (dw, c.V)):
            assert (t[n:] == 7.0).all() and torch.isfinite(t[:n].float()).all()
        bufs.append((loss, lse, dx, dw))
    for a, b in zip(*bufs):
        assert torch.equal(a, b)


def test_streams_and_captured_graphs():
    """Two calls at once on their own streams and workspaces, and a captured
    step replayed on inputs that changed (more rows kept than when captured)."""
    import torch

    from bwd_causal_sdpa_b200.runner import HeadRunner

    cfgs = [head_config_by_name("head_small"), head_config_by_name("head_distill_small")]
    ws = [make_head_workload(c, N=500, V=3001) for c in cfgs]
    streams = [torch.cuda.Stream() for _ in ws]
    torch.cuda.synchronize()
    rs = [HeadRunner(w, stream=s) for w, s in zip(ws, streams)]
    torch.cuda.synchronize()
    for _ in range(3):
        for r in rs:
            r.forward()
            r.backward()
    torch.cuda.synchronize()
    names = ("loss", "lse", "dx", "dw")
    alone = []
    for w in ws:
        r, _ = _check(w)
        alone.append([getattr(r, n).clone() for n in names])
    for r, ref in zip(rs, alone):
        for n, t in zip(names, ref):
            assert torch.equal(getattr(r, n), t)

    for w, ref in zip(ws, alone):
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        r = HeadRunner(w, stream=s)
        ids = r.t_idx if w.cfg.K else r.target
        good = ids.clone()
        ids.fill_(-1)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            r.forward()
            r.backward()
        g.replay()
        torch.cuda.synchronize()
        assert not r.dw.any() and not r.dx.any() and not r.loss.any()
        ids.copy_(good)
        g.replay()
        torch.cuda.synchronize()
        for n, t in zip(names, ref):
            assert torch.equal(getattr(r, n), t)


def test_large_calls_at_once():
    """Two steps whose units each fill the GPU, on streams of their own beside
    an attention: the same bits as alone, whatever share of the SMs each gets."""
    import torch

    import bwd_causal_sdpa_b200 as A
    from bwd_causal_sdpa_b200.runner import AttnRunner, HeadRunner

    ws = [make_head_workload(head_config_by_name(n), N=N, V=V, C=C, left_out=0.1, seed=95)
          for n, N, V, C in (("head_small", 4100, 20001, 256), ("head_distill_small", 3000, 9000, 520))]
    names = ("loss", "lse", "dx", "dw")
    alone = []
    for w in ws:
        r = HeadRunner(w)
        r.forward()
        r.backward()
        assert r.status() == A.ATTN_OK
        alone.append([getattr(r, n).clone() for n in names])
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    rs = [HeadRunner(w, stream=s) for w, s in zip(ws, streams)]
    at = AttnRunner(1, 8, 4096, 128, stream=streams[2])
    for t in (at.q, at.k, at.v, at.do):
        t.normal_()
    torch.cuda.synchronize()
    for _ in range(6):
        for r in rs:
            r.forward()
            r.backward()
        at.forward()
        at.backward()
    torch.cuda.synchronize()
    assert A.attn_get_status() == A.ATTN_OK
    for r, ref in zip(rs, alone):
        for n, t in zip(names, ref):
            assert torch.equal(getattr(r, n), t), n
    assert torch.isfinite(at.dq.float()).all()


def test_output_projection_feeds_the_loss():
    """The end of a training step: o -> attn_out_proj -> attn_head_ce, and back
    through attn_head_ce_bwd and attn_out_proj_bwd, against the oracle's chain
    (relative Frobenius bounds of the projections: 1e-2 for bf16 outputs)."""
    import torch

    import bwd_causal_sdpa_b200 as A
    from tests.parity import rel_fro
    from workloads import make_proj_workload, proj_config_by_name, round_to_bf16

    pw = make_proj_workload(proj_config_by_name("proj_small_d64"))
    pc = pw.cfg
    N, V, C = pc.B * pc.T, 1003, pc.C
    rng = np.random.default_rng(9)
    W = round_to_bf16((rng.standard_normal((V, C)) / np.sqrt(C)).astype(np.float32))
    target = rng.integers(0, V, N).astype(np.int32)
    target[::5] = -100
    dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", t)  # noqa: E731
    o, w_o, w = (dev(a, torch.bfloat16) for a in (pw.o, pw.w_o, W))
    tg = dev(target, torch.int32)
    dloss = torch.full((N,), 1.0 / N, device="cuda")
    y = torch.empty((pc.B, pc.T, C), dtype=torch.bfloat16, device="cuda")
    dy, d_o = torch.empty_like(y), torch.empty_like(o)
    dw_o = torch.empty(tuple(pw.w_o.shape), device="cuda")
    loss, lse = (torch.empty(N, device="cuda") for _ in range(2))
    dw = torch.empty((V, C), device="cuda")
    nb = max(A.attn_head_workspace_bytes(N, V, C, 0, b) for b in (0, 1))
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    A.check(A.attn_out_proj(o, w_o, y, pc.B, pc.T, C, pc.H, pc.D))
    A.check(A.attn_head_ce(y, w, tg, loss, lse, N, V, C, ws, nb))
    A.check(A.attn_head_ce_bwd(y, w, tg, lse, dloss, None, dy, dw, N, V, C, A.ATTN_F32, ws, nb))
    A.check(A.attn_out_proj_bwd(dy, o, w_o, d_o, dw_o, pc.B, pc.T, C, pc.H, pc.D))
    assert A.attn_get_status() == A.ATTN_OK
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    ry = out_projection(pw.o, pw.w_o)
    ids, q = target_lists(target, V)
    rl, _ = head_loss(ry.reshape(N, C), W, ids, q)
    rdx, rdw = head_loss_backward(ry.reshape(N, C), W, ids, q, np.full(N, 1.0 / N))
    rdo, rdwo = out_projection_backward(rdx.reshape(ry.shape), pw.o, pw.w_o)
    errs = {"loss": rel_fro(f(loss), rl), "dw": rel_fro(f(dw), rdw), "d_o": rel_fro(f(d_o), rdo),
            "dw_o": rel_fro(f(dw_o), rdwo)}
    assert all(e <= 1e-2 for e in errs.values()), errs


@pytest.mark.parametrize("N,K", [(200, 1024), (256, 40), (1, 40)])
def test_one_row_tile_with_a_teacher(N, K):
    """The forward that takes all rows as they are: rows left out among them
    hold NaN, ids repeat and crowd."""
    w = make_head_workload(head_config_by_name("head_distill_small"), N=N, K=K, V=1500, C=64,
                           left_out=0.3, seed=90 + N)
    out = (w.t_idx < 0).all(axis=1)
    w.x[out] = np.nan
    _check(w)


@pytest.mark.parametrize("name", ["head_small", "head_distill_small"])
@pytest.mark.parametrize("N,V,C", [(70, 900, 96), (513, 4100, 640), (1030, 2000, 1544)])
def test_workspace_of_the_stated_size_is_enough(name, N, V, C):
    """The stated bytes and no more: what follows the workspace stays, and what
    it held before does not matter."""
    import torch

    import bwd_causal_sdpa_b200 as A
    from bwd_causal_sdpa_b200.runner import HeadRunner

    w = make_head_workload(head_config_by_name(name), N=N, V=V, C=C)
    K = w.cfg.K
    ref, _ = _check(w)
    for fill in (0x00, 0xFF):
        r = HeadRunner(w)
        for is_bwd, call in ((0, r.forward), (1, r.backward)):
            nb = A.attn_head_workspace_bytes(N, V, C, K, is_bwd)
            buf = torch.full((nb + 4096,), fill, dtype=torch.uint8, device="cuda")
            buf[nb:] = 0x5A
            r.ws, r.ws_bytes = buf, nb
            call()
            torch.cuda.synchronize()
            assert (buf[nb:] == 0x5A).all()
        for n in ("loss", "lse", "dx", "dw"):
            assert torch.equal(getattr(r, n), getattr(ref, n)), n


@pytest.mark.parametrize("name,left_out", [("head_237m", 0.0), ("head_237m", 0.93),
                                           ("head_8k", 0.3), ("head_distill_8k", 0.1)])
def test_full_size_against_64_bits(name, left_out):
    """The training shapes, against plain float64 products on the device.
    Relative Frobenius bounds: dx and dW carry two independent roundings to
    bf16 of rms at most 2^-8 / sqrt(3) each: 2^-8 sqrt(2 / 3) = 3.2e-3 < 4e-3;
    loss and lse the fp32 sums of their logits (2e-6, two to three digits
    above 2^-23)."""
    import torch

    from bwd_causal_sdpa_b200 import ATTN_OK
    from bwd_causal_sdpa_b200.runner import HeadRunner

    w = make_head_workload(head_config_by_name(name), left_out=left_out)
    c = w.cfg
    r = HeadRunner(w)
    r.forward()
    r.backward()
    assert r.status() == ATTN_OK
    first = [getattr(r, n).clone() for n in ("loss", "lse", "dx", "dw")]
    for _ in range(5):  # units land on other SMs, waits fall otherwise: the same bits
        r.dx.fill_(7.0)
        r.dw.fill_(7.0)
        r.forward()
        r.backward()
        for n, t in zip(("loss", "lse", "dx", "dw"), first):
            assert torch.equal(getattr(r, n), t), n
    ids, q = _lists(w)
    ids, q = torch.from_numpy(ids).cuda(), torch.from_numpy(q).cuda()
    x, W = r.x.double(), r.wt.double()
    kept = (ids >= 0).any(dim=1)
    loss, lse = (torch.zeros(c.N, dtype=torch.float64, device="cuda") for _ in range(2))
    dx, dw = torch.zeros_like(x), torch.zeros_like(W)
    for i in range(0, c.N, 1024):
        s = slice(i, i + 1024)
        z = x[s] @ W.T / c.tau
        l = torch.logsumexp(z, dim=1)
        at = z.gather(1, ids[s].clamp(min=0))
        terms = torch.where(q[s] > 0, q[s] * (torch.log(q[s].clamp(min=1e-300)) - at + l[:, None]), 0.0)
        loss[s], lse[s] = terms.sum(dim=1) * kept[s], l * kept[s]
        g = r.dloss[s].double() * kept[s]
        dz = torch.exp(z - l[:, None]) * (g + r.dlse[s].double() * kept[s])[:, None]
        dz.scatter_add_(1, ids[s].clamp(min=0), -g[:, None] * q[s])
        dz = dz / c.tau
        dx[s] = dz @ W
        dw += dz.T @ x[s]
    for n, ref, tol in (("loss", loss, 2e-6), ("lse", lse, 2e-6), ("dx", dx, 4e-3), ("dw", dw, 4e-3)):
        err = ((getattr(r, n).double() - ref).norm() / ref.norm()).item()
        assert err <= tol, (n, err)
