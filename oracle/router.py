"""Router of the MoE layer (float64, numpy).  Test infrastructure only.

The pages show the routing weights only where the per-expert loop consumes
them ("Efficient MoE Training for Biological Foundation Models", Challenge 1:
each expert's output is scaled by routing_weights[token, slot] before the
index_add back to token order); they do not print the router.  Reading taken,
the plainest one consistent with the Mixtral model the pages benchmark:

* probabilities = softmax of the token's E router logits;
* the k experts with the largest probabilities are kept, in descending
  order, ties going to the lower expert id;
* the kept probabilities are renormalised to sum to one.

Because the renormalisation divides out the softmax denominator, the kept
probabilities equal a softmax over the k kept logits, and the selection only
compares logits (softmax is strictly increasing).  A NaN logit ranks below
every number (as -inf).  A row whose kept logits include +inf, or are all
-inf, has no defined probabilities (NaN).  This module follows the definition
step by step (softmax first); the tests pin it against the reduced forms.
"""
from __future__ import annotations

import numpy as np


def route_topk(logits: np.ndarray, k: int):
    """logits [T, E] -> (topk_idx int32 [T, k], topk_prob float64 [T, k])."""
    lg = np.asarray(logits, dtype=np.float64)
    T, E = lg.shape
    if not 1 <= k <= E:
        raise ValueError("need 1 <= k <= E")
    key = np.where(np.isnan(lg), -np.inf, lg)
    # softmax over all experts, shifted by the row maximum
    with np.errstate(invalid="ignore"):
        m = key.max(axis=1, keepdims=True)
        p = np.exp(key - m)
        p = p / p.sum(axis=1, keepdims=True)
    # k largest, descending, ties to the lower id: a stable sort of -key
    # (ranking the logits ranks the probabilities, and keeps ties exact)
    order = np.argsort(-key, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(p, order, axis=1)
    with np.errstate(invalid="ignore"):
        top = top / top.sum(axis=1, keepdims=True)
    return order.astype(np.int32), top


def route_losses(logits: np.ndarray, k: int, mask=None):
    """The router's training outputs, from the definitions: ids and
    probabilities of route_topk (probabilities 0 for masked tokens), tokens
    per expert, sums of the softmax over all experts, the load-balance loss
    E * sum_e (count_e / (n k)) * mean_t s_te and the z-loss
    mean_t (log sum_e exp z_te)^2, over the n unmasked tokens (0 for none)."""
    z = np.asarray(logits, np.float64)
    T, E = z.shape
    live = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    idx, prob = route_topk(z, k)
    prob = np.where(live[:, None], prob, 0.0)
    n = int(live.sum())
    counts = np.zeros(E, np.int64)
    np.add.at(counts, idx[live].reshape(-1), 1)
    zl = z[live]
    with np.errstate(invalid="ignore"):
        top = zl.max(axis=1, keepdims=True) if n else np.zeros((0, 1))
        ex = np.exp(zl - top)
        s = ex / ex.sum(axis=1, keepdims=True)
        lse = (top + np.log(ex.sum(axis=1, keepdims=True)))[:, 0]
    sums = s.sum(axis=0)
    balance = E * float(np.sum(counts / (n * k) * (sums / n))) if n else 0.0
    zloss = float(np.mean(lse ** 2)) if n else 0.0
    full_s, full_l = np.zeros((T, E)), np.zeros(T)
    full_s[live], full_l[live] = s, lse
    return dict(idx=idx, prob=prob, counts=counts, sums=sums, n=n, losses=np.array([balance, zloss]), s=full_s,
                lse=full_l, live=live, k=k)


def route_backward(fwd: dict, dprob=None, dlosses=None):
    """Gradient of the logits from those of the probabilities and the two
    losses; the counts are constants."""
    s, lse, live, k = fwd["s"], fwd["lse"], fwd["live"], fwd["k"]
    T, E = s.shape
    n = max(1, fwd["n"])
    d = np.zeros((T, E))
    if dlosses is not None:
        f = fwd["counts"] / (n * k)
        ds = np.broadcast_to(float(dlosses[0]) * E / n * f, (T, E))       # d balance / d s
        d += s * (ds - np.sum(ds * s, axis=1, keepdims=True))             # softmax Jacobian
        d += float(dlosses[1]) * 2.0 / n * lse[:, None] * s               # d lse / d z = s
    if dprob is not None:
        p, dp = fwd["prob"], np.asarray(dprob, np.float64)
        inner = p * (dp - np.sum(p * dp, axis=1, keepdims=True))
        np.add.at(d, (np.arange(T)[:, None], fwd["idx"]), inner)
    return np.where(live[:, None], d, 0.0)
