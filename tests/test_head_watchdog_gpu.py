"""Failure detection in the output head's backward, without a GPU fault: a
counter that is never raised makes the waits for it run out (about 10 ms in the
watchdog build, libattn_debug.so), every role unwinds, the status word reports
ATTN_ETIMEOUT, and the next call on the same context is right. Nothing here
traps, faults or spins without a bound."""

import numpy as np
import pytest

from oracle import head_loss_backward, target_lists, teacher_lists
from tests.parity import rel_fro
from tests.test_watchdog_gpu import _debug_lib
from workloads import head_config_by_name, make_head_workload

pytestmark = pytest.mark.gpu


# what is withheld: 2, dz of the first vocabulary tile (dW and dx wait for it);
# 3, dx of the first of several pieces (dx of the second waits for it)
@pytest.mark.parametrize("name,what,N,V,C", [("head_small", 2, 300, 1000, 200),
                                             ("head_small", 2, 1500, 3000, 128),
                                             ("head_distill_small", 2, 90, 2000, 64),
                                             ("head_small", 3, 8200, 8500, 64)])
def test_a_counter_that_stays_times_out_and_the_context_survives(name, what, N, V, C):
    import torch

    import bwd_causal_sdpa_b200 as A

    lib = _debug_lib()
    w = make_head_workload(head_config_by_name(name), N=N, V=V, C=C, seed=33)
    K = w.cfg.K
    dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", t)  # noqa: E731
    x, wt = dev(w.x, torch.bfloat16), dev(w.w, torch.bfloat16)
    dloss, dlse = dev(w.dloss, torch.float32), dev(w.dlse, torch.float32)
    loss, lse = (torch.empty(N, device="cuda") for _ in range(2))
    dx, dw = torch.empty_like(x), torch.empty_like(wt)
    nb = max(lib.attn_head_workspace_bytes(N, V, C, K, b) for b in (0, 1))
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    if K:
        ids, tl = dev(w.t_idx, torch.int32), dev(w.t_logit, torch.float32)
        fwd = lambda: lib.attn_head_distill(  # noqa: E731
            p(x), p(wt), p(ids), p(tl), w.cfg.tau, p(loss), p(lse), N, V, C, K, A.ATTN_F32, p(ws), nb, None)
        bwd = lambda: lib.attn_head_distill_bwd(  # noqa: E731
            p(x), p(wt), p(ids), p(tl), w.cfg.tau, p(lse), p(dloss), p(dlse), p(dx), p(dw), N, V, C, K,
            A.ATTN_F32, A.ATTN_BF16, p(ws), nb, None)
        lists = teacher_lists(w.t_idx, w.t_logit, V, w.cfg.tau)
    else:
        tg = dev(w.target, torch.int32)
        fwd = lambda: lib.attn_head_ce(  # noqa: E731
            p(x), p(wt), p(tg), p(loss), p(lse), N, V, C, p(ws), nb, None)
        bwd = lambda: lib.attn_head_ce_bwd(  # noqa: E731
            p(x), p(wt), p(tg), p(lse), p(dloss), p(dlse), p(dx), p(dw), N, V, C, A.ATTN_BF16, p(ws),
            nb, None)
        lists = target_lists(w.target, V)
    assert fwd() == A.ATTN_OK
    assert lib.attn_get_status(None) == A.ATTN_OK
    assert lib.attn_debug_withhold(what) == A.ATTN_OK
    try:
        assert bwd() == A.ATTN_OK  # the launch itself is fine
        assert lib.attn_get_status(None) == A.ATTN_ETIMEOUT
    finally:
        assert lib.attn_debug_withhold(0) == A.ATTN_OK
    assert bwd() == A.ATTN_OK
    assert lib.attn_get_status(None) == A.ATTN_OK
    torch.cuda.synchronize()
    rdx, rdw = head_loss_backward(w.x, w.w, *lists, w.dloss, w.dlse, w.cfg.tau)
    f = lambda t: t.to(torch.float64).cpu().numpy()  # noqa: E731
    assert rel_fro(f(dx), rdx) <= 1e-2 and rel_fro(f(dw), rdw) <= 1e-2
