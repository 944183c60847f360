"""Seeded workloads for the losses of the output head (no loss arithmetic
lives here: only random draws).

Draw order from ``numpy.random.default_rng(seed)``: W [V, C], float32 standard
normals / sqrt(C); target ids floor(V u^3), u uniform (token frequencies that
fall off with the id); x [N, C] = standard normals + 6 W[target] (hidden
states that lean towards their target); the rows left out, a random
``int(left_out N)`` of them; for a teacher (K > 0) per row K ids floor(V u^3)
(an id may come twice) with logits 4 x standard normal, and, when ragged, a
number of entries present uniform in [1, K]; dloss (0.5 + uniform) / N and
dlse 0.1 uniform / N. x and W are rounded to bf16 (RNE).
"""

from __future__ import annotations

from dataclasses import dataclass, replace
from typing import Optional

import numpy as np

from .generate import round_to_bf16


@dataclass(frozen=True)
class HeadConfig:
    name: str
    N: int          # token rows
    V: int          # vocabulary
    C: int          # model width
    K: int          # teacher entries per row (0: a single target)
    tau: float
    left_out: float
    ragged: bool
    seed: int


HEAD_CONFIGS = [
    # the 237M decoder of the ARK README's parameter table (width 768, its
    # tokenizer's 32,063 tokens), 8 sequences of 1024
    HeadConfig("head_237m", 8192, 32063, 768, 0, 1.0, 0.0, False, 50),
    # one 8K sequence at width 2048
    HeadConfig("head_8k", 8192, 32063, 2048, 0, 1.0, 0.0, False, 51),
    # the same rows learning from a teacher's 64 best logits
    HeadConfig("head_distill_8k", 8192, 32063, 2048, 64, 2.0, 0.0, False, 52),
    # small cases with ragged sizes
    HeadConfig("head_small", 300, 1000, 200, 0, 1.0, 0.2, False, 53),
    HeadConfig("head_distill_small", 300, 1000, 200, 7, 1.5, 0.2, True, 54),
]


def head_config_by_name(name: str) -> HeadConfig:
    for c in HEAD_CONFIGS:
        if c.name == name:
            return c
    raise KeyError(f"unknown head workload {name!r}; known: {[c.name for c in HEAD_CONFIGS]}")


@dataclass
class HeadWorkload:
    cfg: HeadConfig
    x: np.ndarray
    w: np.ndarray
    target: Optional[np.ndarray]    # int32 [N] (K = 0)
    t_idx: Optional[np.ndarray]     # int32 [N, K]
    t_logit: Optional[np.ndarray]   # float32 [N, K]
    dloss: np.ndarray
    dlse: np.ndarray

    def flops(self) -> dict:
        """Multiply-add flops of the products, for the rows that are kept:
        the logits in the forward; the logits again, dz W and dz^T x in the
        backward."""
        c = self.cfg
        kept = c.N - int(c.left_out * c.N)
        return {"fwd": 2.0 * kept * c.V * c.C, "bwd": 6.0 * kept * c.V * c.C}


def make_head_workload(cfg: HeadConfig, **changes) -> HeadWorkload:
    cfg = replace(cfg, **changes)
    rng = np.random.default_rng(cfg.seed)
    f32 = np.float32
    N, V, C, K = cfg.N, cfg.V, cfg.C, cfg.K
    w = rng.standard_normal((V, C), dtype=f32) * f32(1.0 / np.sqrt(C))
    ids = lambda *s: np.minimum((V * rng.random(s) ** 3).astype(np.int64), V - 1)  # noqa: E731
    target = ids(N)
    x = rng.standard_normal((N, C), dtype=f32) + f32(6.0) * w[target]
    left = rng.permutation(N)[:int(cfg.left_out * N)]
    t_idx = t_logit = None
    if K:
        t_idx = ids(N, K).astype(np.int32)
        t_logit = f32(4.0) * rng.standard_normal((N, K), dtype=f32)
        if cfg.ragged:
            t_idx[np.arange(K)[None, :] >= rng.integers(1, K + 1, (N, 1))] = -1
        t_idx[left] = -1
        target = None
    else:
        target = target.astype(np.int32)
        target[left] = -100
    dloss = ((0.5 + rng.random(N)) / N).astype(f32)
    dlse = (0.1 * rng.random(N) / N).astype(f32)
    return HeadWorkload(cfg, round_to_bf16(x), round_to_bf16(w), target, t_idx, t_logit, dloss, dlse)
