"""Pins of the head-loss oracle (CPU only): float64 PyTorch's cross-entropy
and KL divergence with their autograd, closed forms, and central finite
differences of L = sum(dloss loss + dlse lse)."""

import numpy as np
import pytest
import torch

from oracle import head_dz, head_loss, head_loss_backward, target_lists, teacher_lists
from workloads import HEAD_CONFIGS, head_config_by_name, make_head_workload


def _rand(seed, N=5, V=11, C=4):
    rng = np.random.default_rng(seed)
    return rng, rng.standard_normal((N, C)), rng.standard_normal((V, C))


def test_cross_entropy_matches_torch():
    rng, x, w = _rand(0)
    target = np.array([3, -100, 0, 10, -1])
    dloss, dlse = rng.standard_normal(5), rng.standard_normal(5)
    tx, tw = (torch.tensor(a, requires_grad=True) for a in (x, w))
    z = tx @ tw.T
    t = torch.tensor(np.where(target < 0, -100, target))
    loss = torch.nn.functional.cross_entropy(z, t, reduction="none", ignore_index=-100)
    lse = torch.logsumexp(z, dim=1) * (t >= 0)
    ((loss + 0) * torch.tensor(dloss) + lse * torch.tensor(dlse)).sum().backward()
    ids, q = target_lists(target, 11)
    got_loss, got_lse = head_loss(x, w, ids, q)
    dx, dw = head_loss_backward(x, w, ids, q, dloss, dlse)
    for got, ref in ((got_loss, loss), (got_lse, lse), (dx, tx.grad), (dw, tw.grad)):
        np.testing.assert_allclose(got, ref.detach().numpy(), rtol=1e-12, atol=1e-13)


def test_distillation_matches_torch_kl():
    rng, x, w = _rand(1)
    tau, V = 1.7, 11
    t_idx = np.array([[0, 4, 9], [10, -1, -1], [-1, -1, -1], [2, 2, 7], [5, -1, 1]])
    t_logit = rng.standard_normal((5, 3))
    t_logit[4, 2] = -np.inf
    dloss = rng.standard_normal(5)
    ids, q = teacher_lists(t_idx, t_logit, V, tau)
    tx, tw = (torch.tensor(a, requires_grad=True) for a in (x, w))
    logp = torch.log_softmax(tx @ tw.T / tau, dim=1)
    total = 0.0
    losses = np.zeros(5)
    for n in (0, 1, 3, 4):
        here = t_idx[n] >= 0
        qn = torch.softmax(torch.tensor(t_logit[n][here]) / tau, dim=0)
        # an id named twice keeps its two entries
        ln = (torch.xlogy(qn, qn) - qn * logp[n][torch.tensor(t_idx[n][here])]).sum()
        losses[n] = ln.item()
        total = total + dloss[n] * ln
    total.backward()
    loss, lse = head_loss(x, w, ids, q, tau)
    dx, dw = head_loss_backward(x, w, ids, q, dloss, None, tau)
    np.testing.assert_allclose(loss, losses, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(dx, tx.grad.numpy(), rtol=1e-11, atol=1e-13)
    np.testing.assert_allclose(dw, tw.grad.numpy(), rtol=1e-11, atol=1e-13)
    assert lse[2] == 0 and loss[2] == 0 and not dx[2].any()


def test_closed_forms():
    # equal logits: p = 1 / V; one token: loss 0
    ids, q = target_lists([2, 0], 8)
    loss, lse = head_loss(np.zeros((2, 3)), np.ones((8, 3)), ids, q)
    np.testing.assert_allclose(loss, np.log(8), rtol=1e-15)
    np.testing.assert_allclose(lse, np.log(8), rtol=1e-15)
    ids, q = target_lists([0], 1)
    assert abs(head_loss(np.ones((1, 3)), np.ones((1, 3)), ids, q)[0][0]) < 1e-15
    # a teacher with one entry is a target
    _, x, w = _rand(2)
    t = np.array([[1], [3], [-1], [7], [0]])
    a = head_loss(x, w, *teacher_lists(t, np.zeros((5, 1)), 11, 1.0))
    b = head_loss(x, w, *target_lists(t[:, 0], 11))
    np.testing.assert_allclose(a, b, rtol=1e-14)
    # the gradient of the logits sums to dlse / tau over the vocabulary
    dl = np.arange(1.0, 6.0)
    dz = head_dz(x, w, *target_lists(t[:, 0], 11), dl, dl / 3, 2.0)
    np.testing.assert_allclose(dz.sum(axis=1), np.where(t[:, 0] >= 0, dl / 6, 0), atol=1e-14)


def test_gradients_match_finite_differences():
    rng, x, w = _rand(3)
    t_idx = np.array([[0, 4, 9], [10, -1, 3], [-1, -1, -1], [2, 2, 7], [5, 6, 1]])
    t_logit = rng.standard_normal((5, 3))
    dloss, dlse = rng.standard_normal(5), rng.standard_normal(5)
    for tau in (1.0, 2.5):
        ids, q = teacher_lists(t_idx, t_logit, 11, tau)

        def total(a, b):
            loss, lse = head_loss(a, b, ids, q, tau)
            return (dloss * loss + dlse * lse).sum()

        dx, dw = head_loss_backward(x, w, ids, q, dloss, dlse, tau)
        h = 1e-6
        for arr, grad, at in ((x, dx, "x"), (w, dw, "w")):
            for i in np.ndindex(arr.shape):
                up, down = arr.copy(), arr.copy()
                up[i] += h
                down[i] -= h
                num = (total(up, w) - total(down, w) if at == "x"
                       else total(x, up) - total(x, down)) / (2 * h)
                assert grad[i] == pytest.approx(num, rel=1e-6, abs=1e-8), (at, i)


def test_left_out_rows_reach_nothing():
    rng, x, w = _rand(4)
    target = np.array([1, -1, 2, 11, 4])  # 11 is past the vocabulary
    dloss = np.array([1.0, 1.0, 0.0, 1.0, 2.0])
    ids, q = target_lists(target, 11)
    clean = head_loss_backward(x, w, ids, q, dloss)
    x[[1, 2, 3]] = np.nan
    dx, dw = head_loss_backward(x, w, ids, q, dloss)
    np.testing.assert_array_equal(dx, clean[0])
    np.testing.assert_array_equal(dw, clean[1])
    assert not dx[[1, 2, 3]].any()


def test_workloads_are_seeded_and_named():
    assert len({c.name for c in HEAD_CONFIGS}) == len(HEAD_CONFIGS)
    for name in ("head_small", "head_distill_small"):
        a, b = (make_head_workload(head_config_by_name(name)) for _ in range(2))
        np.testing.assert_array_equal(a.x, b.x)
        kept = (a.target >= 0) if a.cfg.K == 0 else (a.t_idx >= 0).any(axis=1)
        assert kept.sum() == 300 - 60
        assert a.flops()["bwd"] == 3 * a.flops()["fwd"]
    with pytest.raises(KeyError):
        head_config_by_name("nothing")
