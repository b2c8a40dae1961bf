"""The sampling and routing operators' measured cases: inputs, plain forms, exact values.

Three operators of the verify step that choose by score rather than by a
plain maximum:
  sample   one token per logits row by temperature, min-p, top-k and top-p,
           from a given uniform number (optionally with the distribution that
           it was drawn from, which a sampled draft hands to its verification)
  verify   speculative verification that keeps that distribution: each draft
           is accepted with probability min(1, p / q), the first rejected one
           is replaced by a draw from the positive part of p - q
  route    expert choice by softmax or sigmoid scores with a balance bias,
           expert groups, top-k and renormalised, scaled weights

`own` selects the framework's kernels; otherwise `run` is the plain form in
elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

V_LM = 129280        # vocabulary of the verify head
T_PREFILL = 36992    # tokens of the prefill workload
LN2_64 = 64.0 * math.log(2.0)   # weights under 2^-64 of the row's largest count as zero


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one sequence's next token with every filter set as a chat server sets them: latency
        dict(name="sample_b1", op="sample", rows=1, V=V_LM, dtype="bf16", filters="all", probs=False),
        # a serving batch drawn by top-p alone from fp32 logits: the sum over the whole vocabulary counts
        dict(name="sample_topp_b32_f32", op="sample", rows=32, V=V_LM, dtype="f32", filters="topp", probs=False),
        # a sampled draft: temperature only, the distribution written out for the verification
        dict(name="sample_probs_b64", op="sample", rows=64, V=V_LM, dtype="bf16", filters="temp", probs=True),
        # the largest batch of rows, each with parameters of its own (greedy rows, wide and narrow filters)
        dict(name="sample_mixed_b512", op="sample", rows=512, V=V_LM, dtype="bf16", filters="mixed", probs=False),
        # one sequence's verification, K = 3 greedy drafts, top-k and top-p: latency
        dict(name="verify_b1_k3", op="verify", B=1, K=3, V=V_LM, dtype="bf16", filters="topkp", q=False),
        # the concurrency-32 verification batch of greedy drafts
        dict(name="verify_b32_k3", op="verify", B=32, K=3, V=V_LM, dtype="bf16", filters="topp", q=False),
        # sampled drafts with their distributions, temperature only: the residual runs over the whole vocabulary
        dict(name="verify_q_b32_k3", op="verify", B=32, K=3, V=V_LM, dtype="bf16", filters="temp", q=True),
        # an odd vocabulary and a deep draft, fp32 logits, per-sequence parameters: ragged rows, unaligned starts
        dict(name="verify_odd_b7_k5_f32", op="verify", B=7, K=5, V=32003, dtype="f32", filters="mixed", q=True),
        # the verify layer's tokens at concurrency 32, 64 experts, top-6 by sigmoid with a balance bias: latency
        dict(name="route_t128_e64", op="route", T=128, E=64, dtype="f32", score="sigmoid", bias=True, groups=1,
             topk_groups=1, group_top=1, k=6, renorm=True, scale=1.0),
        # the prefill workload's tokens over 64 experts in 8 groups, softmax scores
        dict(name="route_prefill_e64", op="route", T=T_PREFILL, E=64, dtype="f32", score="softmax", bias=False,
             groups=8, topk_groups=3, group_top=1, k=6, renorm=False, scale=16.0),
        # many experts, groups ranked by their two best, ragged token count
        dict(name="route_t8191_e256", op="route", T=8191, E=256, dtype="f32", score="sigmoid", bias=True, groups=8,
             topk_groups=4, group_top=2, k=8, renorm=True, scale=2.5),
        # the prefill workload's tokens over 256 experts
        dict(name="route_prefill_e256", op="route", T=T_PREFILL, E=256, dtype="bf16", score="sigmoid", bias=True,
             groups=8, topk_groups=4, group_top=2, k=8, renorm=True, scale=2.5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "verify", "verify", "route"])
    dtype = rng.choice(["bf16", "f32"])
    filters = rng.choice(["temp", "topk", "topp", "minp", "topkp", "all", "mixed"])
    cap = 512 * V_LM // (2 if dtype == "f32" else 1)
    if op == "route":
        E = rng.choice([8, 16, 24, 40, 64, 96, 128, 160, 256])
        groups = rng.choice([g for g in (1, 2, 4, 8) if E % g == 0])
        topk_groups = rng.randint(1, groups)
        return dict(op="route", T=_log_int(rng, 1, T_PREFILL), E=E, dtype=dtype,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, groups=groups,
                    topk_groups=topk_groups, group_top=rng.randint(1, 2),
                    k=rng.randint(1, min(8, topk_groups * (E // groups))), renorm=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5, 16.0]))
    V = _log_int(rng, 500, 200000)
    if op == "sample":
        probs = rng.random() < 0.3
        rows = _log_int(rng, 1, max(1, min(512, cap // V // (3 if probs else 1))))
        return dict(op="sample", rows=rows, V=V, dtype=dtype, filters=filters, probs=probs)
    K = rng.randint(0, 8)
    q = K > 0 and rng.random() < 0.5
    B = _log_int(rng, 1, max(1, min(128, cap // V // (K + 1) // (3 if q else 1))))
    return dict(op="verify", B=B, K=K, V=V, dtype=dtype, filters=filters, q=q)


# ---------------------------------------------------------------- inputs

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _pick(g, n, values, dtype):
    at = torch.randint(0, len(values), (n,), generator=g, device="cuda")
    return torch.tensor(values, dtype=dtype, device="cuda")[at]


def _params(g, n, filters):
    """Per-row (or per-sequence) sampling parameters; None where the filter is not used."""
    f32, i32 = torch.float32, torch.int32
    p = dict(temperature=None, top_k=None, top_p=None, min_p=None)
    if filters == "mixed":   # requests of one batch that each chose for themselves, greedy ones among them
        p["temperature"] = _pick(g, n, [0.0, 0.3, 0.7, 0.9, 1.0, 1.3], f32)
        p["top_k"] = _pick(g, n, [0, 0, 1, 20, 50, 1000], i32)
        p["top_p"] = _pick(g, n, [1.0, 1.0, 0.5, 0.9, 0.95], f32)
        p["min_p"] = _pick(g, n, [0.0, 0.0, 0.05, 0.1], f32)
        return p
    p["temperature"] = _pick(g, n, [0.6, 0.7, 0.8, 1.0], f32)
    if filters in ("topk", "topkp", "all"):
        p["top_k"] = _pick(g, n, [20, 40, 50, 64], i32)
    if filters in ("topp", "topkp", "all"):
        p["top_p"] = _pick(g, n, [0.8, 0.9, 0.95], f32)
    if filters in ("minp", "all"):
        p["min_p"] = _pick(g, n, [0.02, 0.05, 0.1], f32)
    return p


def _logits(g, rows, V, dtype):
    """Language-model-like rows: a power law of the rank whose steepness differs from row to row (confident and
    undecided positions), with noise."""
    steep = 0.9 + 0.9 * torch.rand(rows, 1, generator=g, device="cuda")
    z = torch.empty(rows, V, device="cuda").exponential_(generator=g) * steep
    z += 0.7 * torch.randn(rows, V, generator=g, device="cuda")
    return (z - 2.0).to(_DTYPES[dtype])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "route":
        s["logits"] = torch.randn(case["T"], case["E"], generator=g, device="cuda").to(_DTYPES[case["dtype"]])
        s["balance"] = 0.1 * torch.randn(case["E"], generator=g, device="cuda") if case["bias"] else None
        return s
    if case["op"] == "sample":
        rows, V = case["rows"], case["V"]
        s["logits"] = _logits(g, rows, V, case["dtype"])
        s["params"] = _params(g, rows, case["filters"])
        s["u"] = torch.rand(rows, generator=g, device="cuda")
        return s
    B, K, V = case["B"], case["K"], case["V"]
    s["logits"] = _logits(g, B * (K + 1), V, case["dtype"]).view(B, K + 1, V)
    s["params"] = _params(g, B, case["filters"])
    s["u"] = torch.rand(B, K + 1, generator=g, device="cuda")
    # the drafter's scores: the verifier's with an error of its own
    z = s["logits"][:, :K].float() + 0.5 * torch.randn(B, K, V, generator=g, device="cuda")
    if case["q"]:
        s["draft_probs"] = torch.softmax(z, -1)
        race = torch.empty(B, K, V, device="cuda").exponential_(generator=g)
        s["draft"] = (s["draft_probs"] / race).argmax(-1).to(torch.int32)
    else:
        s["draft_probs"] = None
        s["draft"] = z.argmax(-1).to(torch.int32)
    return s


# ---------------------------------------------------------------- plain forms

def _kept_weights(logits, temperature, top_k, top_p, min_p):
    """[R, V] fp64 weights exp((l - max) / T) of the tokens that the filters keep, 0 elsewhere."""
    R, V = logits.shape
    dev = logits.device
    z = torch.where(torch.isnan(logits), -torch.inf, logits).float()
    t = torch.ones(R, dtype=torch.float64, device=dev) if temperature is None else temperature.double()
    greedy = ~(t > 0)
    t = torch.where(greedy, 1.0, t)[:, None]
    k = torch.zeros(R, dtype=torch.int64, device=dev) if top_k is None else top_k.long()
    k = torch.where((k <= 0) | (k > V), V, k)[:, None]
    p = torch.ones(R, dtype=torch.float64, device=dev) if top_p is None else top_p.double()
    p = torch.where(p < 1, p, torch.inf)[:, None]
    m = torch.zeros(R, dtype=torch.float64, device=dev) if min_p is None else min_p.double()
    m = torch.where(m > 0, m.clamp(max=1.0), 0.0)[:, None]
    sorts = top_k is not None or top_p is not None
    order = torch.sort(z, dim=-1, descending=True, stable=True)[1] if sorts else None
    best = z.argmax(-1, keepdim=True)
    z = z.double()
    top = z.amax(-1, keepdim=True)
    d = torch.where(z == top, 0.0, z - top)
    w = torch.exp(d / t)
    w = torch.where((d >= torch.maximum(t * torch.log(m), -LN2_64 * t)) & (z > -torch.inf), w, 0.0)
    w = torch.where(greedy[:, None] & (torch.arange(V, device=dev)[None, :] != best), 0.0, w)
    if order is None:
        return w
    ws = w.gather(1, order)
    ws = torch.where(torch.arange(V, device=dev)[None, :] < k, ws, 0.0)
    total = ws.cumsum(-1)
    before = torch.cat([torch.zeros_like(total[:, :1]), total[:, :-1]], 1)
    first = torch.arange(V, device=dev)[None, :] == 0
    ws = torch.where((before < p * total[:, -1:]) | first, ws, 0.0)
    return torch.zeros_like(w).scatter_(1, order, ws)


def _pick_token(w, u):
    """The first index whose cumulative weight exceeds u times the total; -1 where nothing has weight."""
    c = w.cumsum(-1)
    at = (c <= u.double()[:, None] * c[:, -1:]).sum(-1)
    return torch.where(c[:, -1] > 0, at, -1).to(torch.int32)


def _plain_sample(s):
    w = _kept_weights(s["logits"], **s["params"])
    token = _pick_token(w, s["u"])
    if not s["probs"]:
        return token
    return token, (w / w.sum(-1, keepdim=True)).nan_to_num(nan=0.0).float()


def _plain_verify(s):
    B, K, V = s["B"], s["K"], s["V"]
    dev = s["u"].device
    params = {n: None if v is None else v.repeat_interleave(K + 1) for n, v in s["params"].items()}
    w = _kept_weights(s["logits"].reshape(B * (K + 1), V), **params).view(B, K + 1, V)
    total = w.sum(-1)
    x = s["draft"].long()
    wx = w[:, :K].gather(2, x[..., None])[..., 0]
    q = s["draft_probs"]
    qx = 1.0 if q is None else q.gather(2, x[..., None])[..., 0].double()
    ok = s["u"][:, :K].double() * qx * total[:, :K] < wx
    n = ok.to(torch.int64).cumprod(-1).sum(-1)
    b = torch.arange(B, device=dev)
    row, S = w[b, n], total[b, n][:, None]
    if K > 0:
        at = n.clamp(max=K - 1)
        if q is None:
            left = row.scatter(1, x[b, at][:, None], 0.0)
        else:
            left = (row - q[b, at].double() * S).clamp(min=0.0)
        left = torch.where(left.sum(-1, keepdim=True) > 0, left, row)
        row = torch.where((n < K)[:, None], left, row)
    token = _pick_token(row, s["u"][:, K])
    j = torch.arange(K + 1, device=dev)[None, :]
    draft = torch.cat([s["draft"], torch.full((B, 1), -1, dtype=torch.int32, device=dev)], 1)
    committed = torch.where(j < n[:, None], draft, torch.where(j == n[:, None], token[:, None], -1))
    return committed.to(torch.int32), (n + (token >= 0)).to(torch.int32)


def _plain_route(s):
    T, E, G = s["T"], s["E"], s["groups"]
    z = s["logits"].double()
    off = torch.isnan(z) | (z == -torch.inf)
    if s["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-z))
    else:
        z = torch.where(off, -torch.inf, z)
        top = z.amax(-1, keepdim=True)
        e = torch.where(off, 0.0, torch.exp(torch.where(z == top, 0.0, z - top)))
        score = (e / e.sum(-1, keepdim=True)).nan_to_num(nan=0.0)
    score = torch.where(off, 0.0, score)
    sel = score if s["balance"] is None else score + s["balance"].double()
    sel = torch.where(off, -torch.inf, sel)
    by_group = torch.sort(sel.view(T, G, E // G), dim=-1, descending=True)[0]
    best = by_group[..., : s["group_top"]]
    group = torch.where(best[..., 0] == -torch.inf, -torch.inf, torch.where(best == -torch.inf, 0.0, best).sum(-1))
    ranked = torch.sort(group, dim=-1, descending=True, stable=True)[1]
    chosen = torch.zeros(T, G, dtype=torch.bool, device=z.device).scatter_(1, ranked[:, : s["topk_groups"]], True)
    # experts of the groups left out rank behind masked experts of the chosen ones
    sel = torch.where(sel == -torch.inf, -1e300, sel)
    sel = torch.where(chosen.repeat_interleave(E // G, dim=1), sel, -torch.inf)
    idx = torch.sort(sel, dim=-1, descending=True, stable=True)[1][:, : s["k"]]
    w = score.gather(1, idx)
    if s["renorm"]:
        w = (w / w.sum(-1, keepdim=True)).nan_to_num(nan=0.0)
    return idx.to(torch.int32), (w * s["scale"]).float()


def _own_run(s):
    from speculative_decoding_verification_router_b200 import moespec as ms
    if s["op"] == "sample":
        return ms.sample(s["logits"], s["u"], **s["params"], return_probs=s["probs"])
    if s["op"] == "verify":
        return ms.verify_sample(s["logits"], s["draft"], s["u"], draft_probs=s["draft_probs"], **s["params"])
    return ms.route_grouped(s["logits"], s["k"], score=s["score"], bias=s["balance"], n_groups=s["groups"],
                            topk_groups=s["topk_groups"], group_top=s["group_top"], renormalize=s["renorm"],
                            scale=s["scale"])


def run(state):
    if own:
        return _own_run(state)
    return {"sample": _plain_sample, "verify": _plain_verify, "route": _plain_route}[state["op"]](state)


def work(case):
    eb = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * eb + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": 4 * T * E}
    if case["op"] == "sample":
        rows, V = case["rows"], case["V"]
        return {"bytes": rows * V * (eb + (4 if case["probs"] else 0)) + 24 * rows, "flops": 4 * rows * V}
    B, K, V = case["B"], case["K"], case["V"]
    # a residual draw without filters needs its whole row of draft probabilities, one row per sequence at most
    q = B * V * 4 if case["q"] and case["filters"] == "temp" else B * K * 4 if case["q"] else 0
    return {"bytes": B * (K + 1) * (V * eb + 12) + q + 20 * B, "flops": 4 * B * (K + 1) * V}


# ---------------------------------------------------------------- exact values, in 64 bits and more on the host

def _host(x):
    return None if x is None else x.float().cpu().numpy() if x.is_floating_point() else x.cpu().numpy()


def _row_distribution(l, t, k, p, m):
    """(indices in ascending order, weights in extended precision) of the tokens kept in one row."""
    l = np.where(np.isnan(l), -np.inf, l)
    top = float(l.max())
    if top == -np.inf:
        return np.zeros(0, np.int64), np.zeros(0, np.longdouble)
    if not t > 0:
        return np.array([int(l.argmax())]), np.ones(1, np.longdouble)
    gap = np.zeros(l.shape) if top == np.inf else l.astype(np.float64) - top
    gap = np.where(l == top, 0.0, -np.inf) if top == np.inf else gap
    least = -LN2_64 * t
    if m > 0:
        least = max(least, t * math.log(min(m, 1.0)))
    at = np.flatnonzero(gap >= least)
    w = np.exp(gap[at].astype(np.longdouble) / np.longdouble(t))
    if 0 < k < at.size or p < 1:
        by = np.argsort(-l[at].astype(np.float64), kind="stable")
        if 0 < k < at.size:
            by = by[:k]
        if p < 1:
            c = np.cumsum(w[by])
            by = by[: max(1, int(np.searchsorted(c, np.longdouble(p) * c[-1], side="left")) + 1)]
        by = np.sort(by)
        at, w = at[by], w[by]
    return at, w


def _row_pick(at, w, u):
    c = np.cumsum(w)
    return int(at[min(int(np.searchsorted(c, np.longdouble(u) * c[-1], side="right")), at.size - 1)]) if at.size else -1


def _exact_rows(s, rows):
    z = _host(s["logits"].reshape(rows, s["V"]))
    par = {n: _host(v) for n, v in s["params"].items()}
    per = rows // (s["B"] if s["op"] == "verify" else rows)
    get = lambda n, r, default: default if par[n] is None else par[n][r // per].item()   # noqa: E731
    return lambda r: _row_distribution(z[r], get("temperature", r, 1.0), get("top_k", r, 0), get("top_p", r, 1.0),
                                       get("min_p", r, 0.0))


def _exact_sample(s):
    rows, u = s["rows"], _host(s["u"])
    dist = _exact_rows(s, rows)
    tokens = np.empty(rows, np.int32)
    probs = np.zeros((rows, s["V"])) if s["probs"] else None
    for r in range(rows):
        at, w = dist(r)
        tokens[r] = _row_pick(at, w, float(u[r]))
        if probs is not None and at.size:
            probs[r, at] = (w / w.sum()).astype(np.float64)
    return tokens if probs is None else (tokens, probs)


def _exact_verify(s):
    B, K = s["B"], s["K"]
    u, draft, q = _host(s["u"]), _host(s["draft"]), s["draft_probs"]
    dist = _exact_rows(s, B * (K + 1))
    committed, count = np.full((B, K + 1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        for j in range(K + 1):
            at, w = dist(b * (K + 1) + j)
            if j < K:
                x, qj = int(draft[b, j]), None if q is None else _host(q[b, j]).astype(np.longdouble)
                px = w[at == x].sum() / w.sum()
                if np.longdouble(u[b, j]) * (1 if qj is None else qj[x]) < px:
                    committed[b, j] = x
                    count[b] += 1
                    continue
                left = np.where(at == x, 0, w) if qj is None else np.maximum(w / w.sum() - qj[at], 0)
                w = left if left.sum() > 0 else w
            committed[b, j] = _row_pick(at, w, float(u[b, K]))
            count[b] += committed[b, j] >= 0
            break
    return committed, count


def _exact_route(s):
    T, E, G, k = s["T"], s["E"], s["groups"], s["k"]
    z = s["logits"].float().cpu().numpy().astype(np.float64)
    if s["score"] == "sigmoid":
        score = np.exp(-np.logaddexp(0.0, -z))
    else:
        score = np.exp(z - np.log(np.exp(z - z.max(1, keepdims=True)).sum(1, keepdims=True)) - z.max(1, keepdims=True))
    sel = score + (0.0 if s["balance"] is None else s["balance"].cpu().numpy().astype(np.float64))
    group = -np.sort(-sel.reshape(T, G, E // G), axis=2)[:, :, : s["group_top"]]
    best = np.argsort(-group.sum(2), axis=1, kind="stable")[:, : s["topk_groups"]]
    open_ = np.zeros((T, G), bool)
    np.put_along_axis(open_, best, True, 1)
    sel = np.where(np.repeat(open_, E // G, axis=1), sel, -np.inf)
    idx = np.argsort(-sel, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(score, idx, 1)
    if s["renorm"]:
        w = w / w.sum(1, keepdims=True)
    return idx.astype(np.int32), w * s["scale"]


def exact(case, seed):
    return {"sample": _exact_sample, "verify": _exact_verify, "route": _exact_route}[case["op"]](prepare(case, seed))
