"""Sampling, sampled verification and grouped routing in 64 bits, written from
their definitions, one row at a time."""
from __future__ import annotations

import math

import numpy as np

LEAST = 64.0 * math.log(2.0)   # weights under 2^-64 of the largest count as zero


def distribution(l, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """[V] fp64 kept weights of one logits row (not normalised; all 0 for a row without any logit)."""
    l = np.where(np.isnan(l), -np.inf, np.asarray(l, np.float64))
    V = l.size
    w = np.zeros(V)
    top = l.max()
    if top == -np.inf:
        return w
    if not temperature > 0:
        w[int(l.argmax())] = 1.0
        return w
    temperature = min(max(temperature, 1e-30), float(np.finfo(np.float32).max))
    with np.errstate(invalid="ignore"):
        d = np.where(l == top, 0.0, l - top)
    w = np.exp(d / temperature)
    w[(d < -LEAST * temperature) | (l == -np.inf)] = 0.0
    if min_p > 0:
        w[d < temperature * math.log(min(min_p, 1.0))] = 0.0
    order = np.argsort(-l, kind="stable")
    if 0 < top_k < V:
        w[order[top_k:]] = 0.0
    if top_p < 1:
        c = np.cumsum(w[order])
        n = 1 + int(np.count_nonzero(c[:-1] < top_p * c[-1]))   # the shortest prefix that reaches it
        w[order[max(n, 1):]] = 0.0
    return w


def pick(w, u):
    """First index whose cumulative weight exceeds u times the total; -1 where nothing has weight."""
    c = np.cumsum(w)
    return int(np.count_nonzero(c <= u * c[-1])) if c[-1] > 0 else -1


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """(token [T], probs [T, V] fp64)."""
    rows = [distribution(l, *_row(r, temperature, top_k, top_p, min_p)) for r, l in enumerate(logits)]
    tok = np.array([pick(w, float(x)) for w, x in zip(rows, u)], np.int32)
    return tok, np.stack([w / w.sum() if w.sum() > 0 else w for w in rows])


def _row(r, temperature, top_k, top_p, min_p):
    at = lambda a, default: default if a is None else a[r].item()   # noqa: E731
    return at(temperature, 1.0), at(top_k, 0), at(top_p, 1.0), at(min_p, 0.0)


def verify(logits, draft, u, draft_probs=None, temperature=None, top_k=None, top_p=None, min_p=None):
    """(committed [B, K+1] (-1 padded), n_committed [B])."""
    B, K1, V = logits.shape
    K = K1 - 1
    committed, count = np.full((B, K1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        for j in range(K1):
            w = distribution(logits[b, j], *_row(b, temperature, top_k, top_p, min_p))
            if j < K and w.sum() > 0:
                x = int(draft[b, j])
                p = w / w.sum()
                q = np.zeros(V)
                if draft_probs is not None:
                    q = draft_probs[b, j].astype(np.float64)
                elif 0 <= x < V:
                    q[x] = 1.0
                if 0 <= x < V and float(u[b, j]) * q[x] < p[x]:
                    committed[b, j] = x
                    count[b] += 1
                    continue
                left = np.where(q >= 1.0, 0.0, w) if draft_probs is None else np.maximum(p - q, 0.0)
                w = left if left.sum() > 0 else w
            committed[b, j] = pick(w, float(u[b, K]))
            count[b] += committed[b, j] >= 0
            break
    return committed, count


def route(logits, k, score="softmax", bias=None, n_groups=1, topk_groups=None, group_top=1, renormalize=False,
          scale=1.0):
    """(idx [T, k], w [T, k] fp64)."""
    T, E = logits.shape
    gs = E // n_groups
    idx, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        z = np.asarray(logits[t], np.float64)
        on = z > -np.inf   # false for NaN
        s = np.zeros(E)
        with np.errstate(over="ignore"):
            if score == "sigmoid":
                s[on] = 1.0 / (1.0 + np.exp(-z[on]))
            elif on.any():
                top = z[on].max()
                s[on] = np.where(z[on] == top, 1.0, np.exp(z[on] - top if np.isfinite(top) else np.full(on.sum(), -np.inf)))
                s /= s.sum()
        c = s + (0.0 if bias is None else np.asarray(bias, np.float64))
        c[~on | np.isnan(c)] = -np.inf   # a NaN bias ranks its expert as a masked one
        ranks = []
        for g in range(n_groups):
            best = sorted((c[e] for e in range(g * gs, (g + 1) * gs) if c[e] > -np.inf), reverse=True)[:group_top]
            ranks.append((-sum(best) if best else np.inf, g))
        groups = {g for _, g in sorted(ranks)[: topk_groups or n_groups]}
        open_ = [e for e in range(E) if e // gs in groups]
        chosen = sorted(open_, key=lambda e: (-c[e], e))[:k]
        idx[t] = chosen
        w[t] = s[chosen]
        if renormalize:
            w[t] = w[t] / w[t].sum() if w[t].sum() > 0 else 0.0
    return idx, w * scale
