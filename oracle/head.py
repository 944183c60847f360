"""Float64 oracle of the losses of the output head.

TEST INFRASTRUCTURE (see the package docstring): never imported by the
library.

The training decoders on the pages end in an LM head and a cross-entropy
through a stable log-sum-exp (ARK README, the training pipeline; Forge README,
"Architecture"). With x ``[N, C]`` the last hidden states and W ``[V, C]`` the
output embedding, z = x W^T / tau and p = softmax over the vocabulary of z:

  * lse_n = log sum_v exp z[n, v];
  * the target of a row is a distribution q over the vocabulary: one at the
    target id (cross-entropy), or the softmax over a teacher's K entries of
    t / tau, placed at their ids (an id named twice gets both shares);
  * loss_n = sum q log q - sum q log p, summed over the entries;
  * for L = sum_n (dloss_n loss_n + dlse_n lse_n):
    dz = ((dloss + dlse) p - dloss q) / tau, dx = dz W, dW = dz^T x.

A row without a target (negative or >= V), or without a teacher's entry above
-inf, is left out: loss, lse and its gradients are zero and its x is not used.
A row whose dloss and dlse are both zero has no gradients.
"""

from typing import Optional, Tuple

import numpy as np


def _f64(a):
    return np.asarray(a, dtype=np.float64)


def target_lists(target, V: int) -> Tuple[np.ndarray, np.ndarray]:
    """(ids [N, 1], q [N, 1]) of single targets; id -1 where there is none."""
    t = np.asarray(target, dtype=np.int64).reshape(-1, 1)
    ids = np.where((t >= 0) & (t < V), t, -1)
    return ids, (ids >= 0).astype(np.float64)


def teacher_lists(t_idx, t_logit, V: int, tau: float) -> Tuple[np.ndarray, np.ndarray]:
    """(ids, q) of a teacher's entries; id -1 and q 0 where there is none, and
    in the whole row when no entry is above -inf."""
    t_idx = np.asarray(t_idx, dtype=np.int64)
    here = (t_idx >= 0) & (t_idx < V)
    t = np.where(here, _f64(t_logit) / tau, -np.inf)
    top = t.max(axis=1, keepdims=True)
    some = top > -np.inf
    e = np.where(here & some, np.exp(t - np.where(some, top, 0.0)), 0.0)
    q = e / np.where(some, e.sum(axis=1, keepdims=True), 1.0)
    return np.where(here & some, t_idx, -1), q


def _logits(x, w, tau, kept):
    z = np.zeros((x.shape[0], w.shape[0]))
    z[kept] = x[kept] @ w.T / tau
    return z


def head_loss(x, w, ids, q, tau: float = 1.0) -> Tuple[np.ndarray, np.ndarray]:
    """(loss, lse) per row for target distributions given as lists."""
    x, w = _f64(x), _f64(w)
    kept = (ids >= 0).any(axis=1)
    z = _logits(x, w, tau, kept)
    top = z.max(axis=1, keepdims=True)
    lse = np.log(np.exp(z - top).sum(axis=1)) + top[:, 0]
    at = np.take_along_axis(z, np.maximum(ids, 0), axis=1)
    use = q > 0
    terms = q * (np.log(np.where(use, q, 1.0)) - at + lse[:, None])
    loss = np.where(use, terms, 0.0).sum(axis=1)
    return np.where(kept, loss, 0.0), np.where(kept, lse, 0.0)


def head_dz(x, w, ids, q, dloss, dlse=None, tau: float = 1.0) -> np.ndarray:
    """The gradient of the logits x W^T ([N, V]; zero rows where left out)."""
    x, w, dloss = _f64(x), _f64(w), _f64(dloss)
    dlse = np.zeros_like(dloss) if dlse is None else _f64(dlse)
    kept = (ids >= 0).any(axis=1) & ((dloss != 0) | (dlse != 0))
    z = _logits(x, w, tau, kept)
    z -= z.max(axis=1, keepdims=True)
    p = np.exp(z)
    p /= p.sum(axis=1, keepdims=True)
    dz = (dloss + dlse)[:, None] * p
    rows = np.broadcast_to(np.arange(len(ids))[:, None], ids.shape)
    np.subtract.at(dz, (rows, np.maximum(ids, 0)), np.where(ids >= 0, q, 0.0) * dloss[:, None])
    return np.where(kept[:, None], dz, 0.0) / tau


def head_loss_backward(x, w, ids, q, dloss, dlse: Optional[np.ndarray] = None,
                       tau: float = 1.0) -> Tuple[np.ndarray, np.ndarray]:
    """(dx, dW)."""
    dz = head_dz(x, w, ids, q, dloss, dlse, tau)
    used = dz.any(axis=1)
    return dz @ _f64(w), dz[used].T @ _f64(x)[used]
