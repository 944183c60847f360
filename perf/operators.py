"""The language-model head losses: their cases, their plain form and the library's calls.

Both losses are taken on logits z = x W^T that are never stored: x [N, C] is
the final hidden state of N tokens, W [V, C] the output embedding, both bf16.

  ce       loss_n = lse_n - z[n, target_n], lse_n = log sum_v exp z[n, v];
           a negative target leaves the row out (loss 0, lse 0, no gradient).
  distill  a teacher's K best logits t with their vocabulary ids per row (a
           negative id is an absent entry; a row of absent entries is left
           out): q = softmax over the row's entries of t / tau,
           p = softmax over the vocabulary of z / tau,
           loss_n = sum_k q_k (log q_k - log p[id_k]), lse_n = log sum_v exp(z/tau).

The backward takes the upstream gradients of loss (and of lse, where a case
has them) and gives dx [N, C] and dW [V, C] in bf16:
  dz = ((dloss + dlse) p - dloss q) / tau,  dx = dz W,  dW = dz^T x.
"""

import math

import torch

own = False

# C, V and N come from the decoder shapes this repository measures: width 768
# with 8 x 1024 tokens (the 237M decoder layer), width 2048 with one sequence
# of 8192; vocabularies of 32063 and 24576 tokens.
_CASES = [
    # one token scored: launch latency and one pass over W
    dict(name="ce_score_one", op="ce", mode="fwd", N=1, C=768, V=32063, left_out=0.0),
    # one ragged evaluation batch, prompt rows left out
    dict(name="ce_eval_ragged", op="ce", mode="fwd", N=777, C=768, V=32063, left_out=0.25),
    # the loss of one micro-batch of the 237M decoder
    dict(name="ce_fwd_237m", op="ce", mode="fwd", N=8192, C=768, V=32063, left_out=0.0),
    # a short packed batch's gradients: W and dW dominate
    dict(name="ce_bwd_short", op="ce", mode="bwd", N=100, C=768, V=24576, left_out=0.0, dlse=True),
    # the gradients of that micro-batch, padding left out
    dict(name="ce_bwd_237m", op="ce", mode="bwd", N=8192, C=768, V=32063, left_out=0.1),
    # instruction tuning: most rows are prompt and carry no loss
    dict(name="ce_step_tuning", op="ce", mode="step", N=8192, C=2048, V=32063, left_out=0.7),
    # one whole long-context step, the largest call
    dict(name="ce_step_8k", op="ce", mode="step", N=8192, C=2048, V=32063, left_out=0.0, dlse=True),
    # distillation: a few rows, a short list of teacher logits
    dict(name="distill_fwd_few", op="distill", mode="fwd", N=33, C=768, V=24576, K=8, tau=1.0,
         left_out=0.0, ragged=False, t_bf16=False),
    # the forward at the long-context width
    dict(name="distill_fwd_8k", op="distill", mode="fwd", N=8192, C=2048, V=32063, K=64, tau=2.0,
         left_out=0.0, ragged=False, t_bf16=False),
    # ragged lists (a top-p cut) stored in bf16
    dict(name="distill_bwd_237m", op="distill", mode="bwd", N=8192, C=768, V=32063, K=64, tau=1.0,
         left_out=0.1, ragged=True, t_bf16=True),
    # an odd batch, a long list
    dict(name="distill_step_odd", op="distill", mode="step", N=4001, C=2048, V=24576, K=100,
         tau=1.5, left_out=0.2, ragged=True, t_bf16=True),
]
_MOST = 8 * 8192 * 32063 * 2048


def listed():
    return [dict(c) for c in _CASES]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = dict(op=rng.choice(["ce", "distill"]), mode=rng.choice(["fwd", "bwd", "step"]),
                 N=_spread(rng, 1, 8192), C=8 * _spread(rng, 8, 256), V=_spread(rng, 500, 50000),
                 left_out=rng.choice([0.0, 0.1, round(rng.uniform(0.0, 0.9), 2)]))
        if c["mode"] != "fwd":
            c["dlse"] = rng.random() < 0.3
        if c["op"] == "distill":
            c.update(K=_spread(rng, 1, 128), tau=rng.choice([1.0, round(rng.uniform(0.7, 4.0), 2)]),
                     ragged=rng.random() < 0.5, t_bf16=rng.random() < 0.5)
        if _products(c) * c["N"] * c["V"] * c["C"] * 2 <= _MOST:
            return c


def _kept(case):
    return case["N"] - int(case["left_out"] * case["N"])


def _products(case):
    # the logits once in the forward; in the backward the logits again (they
    # are not kept), dz W and dz^T x
    return {"fwd": 1, "bwd": 3, "step": 4}[case["mode"]]


def work(case):
    N, C, V, K = _kept(case), case["C"], case["V"], case.get("K", 0)
    rows = 2 * N * C + (4 * N if not K else N * K * (6 if case["t_bf16"] else 8))
    out = 8 * case["N"]
    if case["mode"] != "fwd":
        rows += (8 if not case.get("dlse") else 12) * N
        out = (out if case["mode"] == "step" else 0) + 2 * case["N"] * C + 2 * V * C
    return {"bytes": rows + 2 * V * C + out, "flops": 2.0 * _products(case) * N * V * C}


def prepare(case, seed):
    N, C, V, K = case["N"], case["C"], case["V"], case.get("K", 0)
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    uniform = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    w = normal(V, C) / math.sqrt(C)
    # token frequencies fall off as a power of the id
    target = (V * uniform(N) ** 3).long().clamp_(max=V - 1)
    # hidden states of a partly trained model: they lean towards the target's embedding
    x = normal(N, C) + 6.0 * w[target]
    left = torch.zeros(N, dtype=torch.bool, device="cuda")
    left[torch.randperm(N, generator=g, device="cuda")[:N - _kept(case)]] = True
    s = {"op": case["op"], "mode": case["mode"], "N": N, "C": C, "V": V, "K": K,
         "x": x.bfloat16(), "w": w.bfloat16(), "tau": case.get("tau", 1.0)}
    if not K:
        s["target"] = target.masked_fill(left, -100).int()
    else:
        # the teacher's best: without replacement from the same falling frequencies
        ids, vals = [], []
        fall = -torch.log1p(torch.arange(V, device="cuda", dtype=torch.float32))
        for r in range(0, N, 2048):
            noise = -torch.log(-torch.log(uniform(min(2048, N - r), V).clamp_(1e-7, 1 - 1e-6)))
            v, i = torch.topk(fall + noise, min(K, V), dim=1)
            ids.append(i)
            vals.append(v)
        ids, vals = torch.cat(ids), torch.cat(vals)
        if case["ragged"]:
            ids[torch.arange(K, device="cuda") >= 1 + (K * uniform(N, 1)).long()] = -1
        ids[left] = -1
        s["t_idx"] = ids.int().contiguous()
        s["t_logit"] = vals.to(torch.bfloat16 if case["t_bf16"] else torch.float32).contiguous()
    if case["mode"] != "fwd":
        # the mean over the rows that count, unevenly weighted in part
        s["dloss"] = (0.5 + uniform(N)) / max(1, _kept(case))
        s["dlse"] = 1e-3 * uniform(N) / max(1, _kept(case)) if case.get("dlse") else None
    if case["mode"] == "bwd":  # what the forward left behind
        s["lse"] = _forward(s)[1]
    if own:
        # what a training program keeps: the library's workspace
        import bwd_causal_sdpa_b200 as A
        s["ws_bytes"] = max(A.attn_head_workspace_bytes(N, V, C, K, int(b))
                            for b in {"fwd": (0,), "bwd": (1,), "step": (0, 1)}[case["mode"]])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device="cuda")
    return s


def _teacher(s):
    """(present, q, log q) of the teacher's entries in 32 bits."""
    present = s["t_idx"] >= 0
    t = (s["t_logit"].float() / s["tau"]).masked_fill(~present, -math.inf)
    some = present.any(dim=1, keepdim=True)
    t = t - torch.where(some, t.amax(dim=1, keepdim=True), 0.0)
    total = torch.exp(t).sum(dim=1, keepdim=True)
    logq = t - torch.log(torch.where(some, total, 1.0))
    return present, torch.exp(logq), logq


def _counts(s):
    return s["target"] >= 0 if not s["K"] else (s["t_idx"] >= 0).any(dim=1)


def _forward(s):
    z = s["x"].float() @ s["w"].float().T / s["tau"]
    top = z.amax(dim=1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(dim=1))
    if not s["K"]:
        loss = lse - z.gather(1, s["target"].long().clamp(min=0)[:, None])[:, 0]
    else:
        present, q, logq = _teacher(s)
        zk = z.gather(1, s["t_idx"].long().clamp(min=0))
        loss = torch.where(present, q * (logq - zk + lse[:, None]), 0.0).sum(dim=1)
    counts = _counts(s)
    return torch.where(counts, loss, 0.0), torch.where(counts, lse, 0.0)


def _backward(s, lse):
    x, w = s["x"].float(), s["w"].float()
    counts = _counts(s)
    dloss = torch.where(counts, s["dloss"], 0.0)
    dlse = torch.where(counts, s["dlse"], 0.0) if s["dlse"] is not None else 0.0
    dz = torch.exp(x @ w.T / s["tau"] - lse[:, None]) * (dloss + dlse)[:, None]
    if not s["K"]:
        at, share = s["target"].long().clamp(min=0)[:, None], dloss[:, None]
    else:
        present, q, _ = _teacher(s)
        at, share = s["t_idx"].long().clamp(min=0), torch.where(present, q, 0.0) * dloss[:, None]
    dz.scatter_add_(1, at, -share)
    dz = torch.where(counts[:, None], dz, 0.0) / s["tau"]
    return (dz @ w).bfloat16(), (dz.T @ x).bfloat16()


def _own_forward(s):
    import bwd_causal_sdpa_b200 as A
    loss = torch.empty(s["N"], dtype=torch.float32, device="cuda")
    lse = torch.empty_like(loss)
    stream = torch.cuda.current_stream()
    if not s["K"]:
        A.check(A.attn_head_ce(s["x"], s["w"], s["target"], loss, lse, s["N"], s["V"], s["C"],
                               s["ws"], s["ws_bytes"], stream), "attn_head_ce")
    else:
        t_dtype = A.ATTN_BF16 if s["t_logit"].dtype == torch.bfloat16 else A.ATTN_F32
        A.check(A.attn_head_distill(s["x"], s["w"], s["t_idx"], s["t_logit"], s["tau"], loss, lse,
                                    s["N"], s["V"], s["C"], s["K"], t_dtype, s["ws"],
                                    s["ws_bytes"], stream), "attn_head_distill")
    return loss, lse


def _own_backward(s, lse):
    import bwd_causal_sdpa_b200 as A
    dx, dw = torch.empty_like(s["x"]), torch.empty_like(s["w"])
    stream = torch.cuda.current_stream()
    if not s["K"]:
        A.check(A.attn_head_ce_bwd(s["x"], s["w"], s["target"], lse, s["dloss"], s["dlse"], dx, dw,
                                   s["N"], s["V"], s["C"], A.ATTN_BF16, s["ws"], s["ws_bytes"],
                                   stream), "attn_head_ce_bwd")
    else:
        t_dtype = A.ATTN_BF16 if s["t_logit"].dtype == torch.bfloat16 else A.ATTN_F32
        A.check(A.attn_head_distill_bwd(s["x"], s["w"], s["t_idx"], s["t_logit"], s["tau"], lse,
                                        s["dloss"], s["dlse"], dx, dw, s["N"], s["V"], s["C"],
                                        s["K"], t_dtype, A.ATTN_BF16, s["ws"], s["ws_bytes"],
                                        stream), "attn_head_distill_bwd")
    return dx, dw


def run(state):
    forward, backward = (_own_forward, _own_backward) if own else (_forward, _backward)
    out = {}
    if state["mode"] != "bwd":
        out["loss"], out["lse"] = forward(state)
    if state["mode"] != "fwd":
        out["dx"], out["dw"] = backward(state, state["lse"] if state["mode"] == "bwd" else out["lse"])
    return out


def exact(case, seed):
    """From the definition in 64 bits, a block of rows at a time."""
    s = prepare(case, seed)
    f64 = dict(dtype=torch.float64, device="cuda")
    w, tau = s["w"].double(), s["tau"]
    N, V, C = s["N"], s["V"], s["C"]
    loss, lse = torch.zeros(N, **f64), torch.zeros(N, **f64)
    dx, dw = torch.zeros(N, C, **f64), torch.zeros(V, C, **f64)
    for r in range(0, N, 1024):
        at = slice(r, min(N, r + 1024))
        x = s["x"][at].double()
        # the distribution that the student is held to, over the whole vocabulary
        want = torch.zeros(x.shape[0], V, **f64)
        if s["K"]:
            ids = s["t_idx"][at].long()
            e = torch.where(ids >= 0, torch.exp(s["t_logit"][at].double() / tau), 0.0)
            want.scatter_add_(1, ids.clamp(min=0), e)
            counts = (ids >= 0).sum(dim=1) > 0
            want = want / want.sum(dim=1, keepdim=True).clamp(min=1e-300)
        else:
            counts = s["target"][at] >= 0
            want[counts.nonzero()[:, 0], s["target"][at].long()[counts]] = 1.0
        z = x @ w.T / tau
        total = torch.logsumexp(z, dim=1)
        logp = z - total[:, None]
        lse[at] = total * counts
        entropy = torch.where(want > 0, want * torch.log(want.clamp(min=1e-300)), 0.0).sum(dim=1)
        loss[at] = (entropy - (want * logp).sum(dim=1)) * counts
        if s["mode"] != "fwd":
            a = s["dloss"][at].double() * counts
            b = s["dlse"][at].double() * counts if s["dlse"] is not None else 0.0 * a
            dz = ((a + b)[:, None] * torch.exp(logp) - a[:, None] * want) / tau
            dx[at] = dz @ w
            dw += dz.T @ x
    out = {"loss": loss, "lse": lse} if s["mode"] != "bwd" else {}
    if s["mode"] != "fwd":
        out.update(dx=dx, dw=dw)
    return out
