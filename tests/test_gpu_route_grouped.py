"""GPU parity of moe_route_grouped against the 64-bit oracle: the chosen experts
exactly; the gate weights to fp32 evaluation, 16 x 2^-24 relative (an exp within
2 ulp, a tree sum of at most 256 positive terms, two divisions, the scale)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import sampling as sp
from speculative_decoding_verification_router_b200 import synth
from tests.gpu_util import assert_close, dev, host
from tests.inputs import routed_layer_inputs

pytestmark = pytest.mark.gpu

REL = 16 * 2.0 ** -24
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ms():
    from speculative_decoding_verification_router_b200 import moespec
    return moespec


def _logits(g, T, E):
    z = 2 * g.standard_normal((T, E))
    special = [np.zeros(E), np.full(E, -np.inf), np.full(E, np.nan), np.full(E, -1e38), 50 + g.standard_normal(E),
               -50 - g.standard_normal(E), np.round(g.standard_normal(E)),
               np.where(g.random(E) < 0.9, -np.inf, g.standard_normal(E)),
               np.where(g.random(E) < 0.5, np.nan, g.standard_normal(E)),
               np.where(g.random(E) < 0.2, np.inf, g.standard_normal(E))]
    z[: len(special)] = special[: T]
    return z.astype(np.float32)


def _check(ms, z, k, dtype, **kw):
    t = torch.from_numpy(z).to(DTYPES[dtype])
    bias = kw.pop("bias")
    idx, w = ms.route_grouped(t.cuda(), k, bias=None if bias is None else dev(bias), **kw)
    torch.cuda.synchronize()
    ri, rw = sp.route(t.float().numpy(), k, bias=bias, **kw)
    np.testing.assert_array_equal(host(idx), ri)
    assert np.all(np.abs(host(w).astype(np.float64) - rw) <= REL * rw + 1e-37)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(1, 1), (2, 1), (8, 2), (40, 4), (64, 8), (96, 1), (160, 4), (256, 8), (256, 32)])
def test_route_grouped_matches_the_oracle(ms, E, groups, score, dtype):
    g = np.random.default_rng(E + groups)
    z = _logits(g, 67, E)
    for tg in sorted({1, (groups + 1) // 2, groups}):
        for top, renorm in ((1, False), (2, True)):
            k = int(g.integers(1, min(32, tg * (E // groups)) + 1))
            bias = (0.1 * g.standard_normal(E)).astype(np.float32) if top == 2 else None
            _check(ms, z, k, dtype, bias=bias, score=score, n_groups=groups, topk_groups=tg, group_top=top,
                   renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(9, 3), (96, 3), (90, 5), (150, 6), (96, 12), (48, 16), (124, 31), (200, 25), (32, 32)])
def test_group_counts_that_are_no_power_of_two(ms, E, groups, score):
    g = np.random.default_rng(E)
    z = _logits(g, 41, E)
    for tg in sorted({1, 2, groups - 1}):
        for top in (1, 2):
            k = min(32, tg * (E // groups))
            bias = (0.1 * g.standard_normal(E)).astype(np.float32) if top == 1 else None
            _check(ms, z, k, "f32", bias=bias, score=score, n_groups=groups, topk_groups=tg, group_top=top,
                   renormalize=True, scale=1.5)


@pytest.mark.parametrize("T", [1, 7, 9, 36992])
def test_route_grouped_token_counts(ms, T):
    g = np.random.default_rng(T)
    z = 2 * g.standard_normal((T, 64)).astype(np.float32)
    bias = (0.1 * g.standard_normal(64)).astype(np.float32)
    kw = dict(score="sigmoid", n_groups=8, topk_groups=3, group_top=2, renormalize=True)
    idx, w = ms.route_grouped(dev(z), 6, bias=dev(bias), **kw)
    at = np.unique(np.r_[0, T - 1, g.integers(0, T, 200)])
    ri, rw = sp.route(z[at], 6, bias=bias, **kw)
    np.testing.assert_array_equal(host(idx)[at], ri)
    assert np.all(np.abs(host(w)[at] - rw) <= REL * rw)


def test_close_scores_are_told_apart(ms):
    # neighbours in fp32 around 0 give sigmoid scores a quarter of a step apart: equal in fp32, not in truth
    E = 64
    z = np.full((1, E), -1.0, np.float32)
    z[0, 10:20] = np.float32(0.4) + np.arange(10, dtype=np.float32) * np.float32(2.0 ** -25)
    _check(ms, z, 6, "f32", bias=None, score="sigmoid")
    bias = np.zeros(E, np.float32)
    bias[10:20] = 0.25
    _check(ms, z, 6, "f32", bias=bias, score="sigmoid")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,tg,k", [(64, 1, 1, 6), (64, 1, 1, 1), (64, 8, 3, 8), (256, 8, 4, 8), (60, 4, 2, 12)])
@pytest.mark.parametrize("values", [[np.inf], [-np.inf], [np.nan], [np.inf, -np.inf, np.nan, 0.0]])
def test_infinite_and_nan_bias(ms, values, E, groups, tg, k, score):
    g = np.random.default_rng(E + k)
    z = 2 * g.standard_normal((33, E)).astype(np.float32)
    for share in (0.02, 0.3, 0.97):
        bias = (0.1 * g.standard_normal(E)).astype(np.float32)
        at = g.random(E) < share
        at[5] = True
        bias[at] = g.choice(np.array(values, np.float32), int(at.sum()))
        _check(ms, z, k, "f32", bias=bias, score=score, n_groups=groups, topk_groups=tg, group_top=2, renormalize=True)


def _route_many(z, k, score, bias, groups, tg, top):
    """The definition over whole tensors, in fp64, for finite logits: (idx, renormalised w, whether every decision is
    by more than 1e-13, ten times the error of a score, or a tie of equal logits)."""
    T, E = z.shape
    z = z.double()
    s = torch.softmax(z, -1) if score == "softmax" else 1.0 / (1.0 + torch.exp(-z))
    c = s if bias is None else s + bias.double()
    best = c.view(T, groups, E // groups).sort(-1, descending=True).values[..., :top].sum(-1)
    keep = torch.zeros(T, groups, dtype=torch.bool, device=z.device)
    ranked = best.sort(dim=-1, descending=True, stable=True)
    keep.scatter_(1, ranked.indices[:, :tg], True)
    c = c.masked_fill(~keep.repeat_interleave(E // groups, 1), -float("inf"))
    order = c.sort(dim=-1, descending=True, stable=True)
    idx = order.indices[:, :k]
    w = s.gather(1, idx)
    clear = lambda hi, lo: (hi - lo > 1e-13) | ((hi == lo) if bias is None else hi > hi)   # noqa: E731
    sure = clear(order.values[:, :k], order.values[:, 1: k + 1] if k < E else
                 torch.cat([order.values[:, 1:], torch.full_like(c[:, :1], -1.0)], 1)).all(1)
    if tg < groups:
        sure &= clear(ranked.values[:, tg - 1], ranked.values[:, tg])
    return idx.int(), w / w.sum(-1, keepdim=True), sure


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(8, 8), (40, 4), (64, 1), (64, 8), (96, 2), (160, 4), (256, 1), (256, 8)])
def test_many_tokens_with_close_scores(ms, E, groups, score, dtype):
    """Enough tokens that coarse scores often fail to tell experts or groups apart: random logits, rounded ones (ties),
    logits within 2^-14 of each other, and wider ones."""
    T = 20000
    g = torch.Generator(device="cuda").manual_seed(E + groups)
    z = 1.5 * torch.randn(T, E, generator=g, device="cuda")
    z[: T // 4] = torch.round(z[: T // 4] * 8) / 8 + 0.046875
    near = z[T // 4: T // 2]
    near.copy_(0.25 + torch.rand(near.shape, generator=g, device="cuda") * 2.0 ** -14)
    z[-500:] *= 4
    z = z.to(DTYPES[dtype])
    tg = max(1, groups // 2)
    for bias in (None, 0.1 * torch.randn(E, generator=g, device="cuda")):
        for top in (1, 2):
            k = min(8, tg * (E // groups))
            idx, w = ms.route_grouped(z, k, score=score, bias=bias, n_groups=groups, topk_groups=tg, group_top=top,
                                      renormalize=True)
            ri, rw, sure = _route_many(z, k, score, bias, groups, tg, top)
            wrong = sure & (idx != ri).any(1)
            assert int(wrong.sum()) == 0, (top, bias is not None, wrong.nonzero()[:3].tolist())
            assert int(sure.sum()) > 0.98 * T
            assert bool(((w.double() - rw).abs() <= REL * rw + 1e-37)[sure].all())


@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(8, 2), (8, 4), (40, 2), (64, 2), (64, 4), (120, 4), (256, 2), (256, 4)])
def test_nan_bias_in_groups_of_several_lanes(ms, E, groups, score, group_top):
    g = np.random.default_rng(E + groups)
    z = 2 * g.standard_normal((65, E)).astype(np.float32)
    for n in (1, 2, E // 4):
        for values in ([np.nan], [-np.nan], [np.nan, np.inf, -np.inf]):
            bias = (0.1 * g.standard_normal(E)).astype(np.float32)
            bias[g.choice(E, n, replace=False)] = g.choice(np.array(values, np.float32), n)
            for tg in {1, groups // 2, groups - 1}:
                _check(ms, z, min(6, tg * (E // groups)), "f32", bias=bias, score=score, n_groups=groups, topk_groups=tg,
                       group_top=group_top, renormalize=True)


def _logit(s):
    return np.log(s / (1 - s)).astype(np.float32)


@pytest.mark.parametrize("bias", [0.0, 2.0 ** -30, None])
def test_a_groups_best_behind_a_lower_expert_of_the_same_coarse_score(ms, bias):
    """Scores of one step of 16 bits come to the lower expert first, the smaller one here."""
    E, step = 64, 2.0 ** -16                 # of scores in [1/2, 1)
    base = np.floor(0.6 / step) * step
    b = None if bias is None else np.full(E, bias, np.float32)
    kw = dict(bias=b, score="sigmoid")
    z = np.tile(-1 - 0.01 * np.arange(E, dtype=np.float32), (1, 1))
    z[0, [0, 1, 8]] = _logit(base + step * np.array([0.1, 0.9, 0.5]))
    _check(ms, z, 3, "f32", n_groups=8, topk_groups=1, group_top=1, **kw)
    z[0, [1, 6, 2, 9]] = [-1, *_logit(base + step * np.array([0.9, 0.1, 0.5]))]   # in another lane's group
    _check(ms, z, 3, "f32", n_groups=8, topk_groups=1, group_top=1, **kw)
    # groups of two lanes, each of which has its two best the wrong way round
    z = np.tile(-1 - 0.01 * np.arange(E, dtype=np.float32), (1, 1))
    z[0, [0, 1, 8, 9, 16, 17]] = _logit(base + step * np.array([0.46, 0.69, 0.23, 0.92, 0.76, 0.76]))
    _check(ms, z, 4, "f32", n_groups=4, topk_groups=1, group_top=2, **kw)
    _check(ms, z, 4, "f32", n_groups=2, topk_groups=1, group_top=2, **kw)


def _close_fours(E, base, low, high, between, rest):
    """Two experts at base + low, two behind them at base + high, and two of the second group in between."""
    v = np.full((1, E), rest, np.float32)
    v[0, [0, 1]], v[0, [2, 3]], v[0, [E // 8, E // 8 + 1]] = np.float32(base + low), np.float32(base + high), np.float32(base + between)
    return v


def test_four_close_scores_in_one_lane(ms):
    """Four experts of one group within one step of the coarse scores, the two larger behind: both of the group's best
    are short by up to a step, and the second group lies between."""
    E = 256
    kw = dict(n_groups=8, topk_groups=1, group_top=2)
    # by the bias alone (scores 1/2)
    bias = _close_fours(E, 0.0, 0.5, 0.50003, 0.500028, -0.4)[0]
    _check(ms, np.zeros((1, E), np.float32), 2, "f32", bias=bias, score="sigmoid", **kw)
    # by the logits: steps of 2^-15 relative
    for d in (245, 249, 251, 253):
        z = _close_fours(E, 1.0, 0.0, 255 * 2.0 ** -23, d * 2.0 ** -23, -2.0)
        _check(ms, z, 2, "f32", bias=None, score="sigmoid", **kw)
    for b in (4.0, 8.0, 64.0, 16384.0):
        z = _close_fours(E, b, 0.0, b * 255 * 2.0 ** -23, b * 230 * 2.0 ** -23, b - 8)
        _check(ms, z, 2, "f32", bias=None, score="softmax", **kw)
        bias = np.zeros(E, np.float32)
        _check(ms, z, 2, "f32", bias=bias, score="softmax", **kw)


@pytest.mark.parametrize("E", [60, 64, 256])
@pytest.mark.parametrize("groups,group_top", [(1, 1), (4, 1), (4, 2)])
def test_large_logits_whose_scores_are_equal(ms, E, groups, group_top):
    """Neighbouring fp32 logits from about 24 up have equal sigmoid scores in 64 bits: the lower expert comes first."""
    T = 400
    g = np.random.default_rng(E)
    z = (g.standard_normal((T, E)) - 3).astype(np.float32)
    x = np.linspace(18, 30, T).astype(np.float32)
    at = np.stack([g.choice(E, 4, replace=False) for _ in range(T)])
    r = np.arange(T)
    z[r, at[:, 0]] = x
    z[r, at[:, 1]] = np.nextafter(x, np.float32(100))
    z[r, at[:, 2]] = np.nextafter(x, np.float32(0))
    z[::2][r[: T // 2], at[::2, 3]] = x[::2]
    for k in (1, 2, 6):
        for tg in {1, (groups + 1) // 2}:
            _check(ms, z, k, "f32", bias=None, score="sigmoid", n_groups=groups, topk_groups=tg, group_top=group_top,
                   renormalize=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [60, 64, 256])
@pytest.mark.parametrize("groups,group_top", [(1, 1), (4, 1), (4, 2)])
def test_tiny_logits_whose_scores_are_equal(ms, groups, group_top, E, score, dtype):
    """Logits around zero that differ by less than 64-bit scores do: the lower expert comes first."""
    T = 200
    g = np.random.default_rng(E + groups)
    kinds = np.array([0.0, -0.0, 1e-20, -1e-20, 1e-30, -1e-30, 1e-44, 3e-18, -2e-18])
    z = kinds[g.integers(0, len(kinds), (T, E))]
    z[:50, ::5] = g.standard_normal((50, len(range(0, E, 5))))          # some far from zero
    z[50:100][g.random((50, E)) < 0.95] = -1.0                            # a few tiny ones among the best
    z[100:150] = np.where(g.random((50, E)) < 0.7, 0.0, -1e-30)           # the border among zeros
    z = z.astype(np.float32)
    for k in (1, 2, 6):
        for tg in {1, (groups + 1) // 2}:
            _check(ms, z, k, dtype, bias=None, score=score, n_groups=groups, topk_groups=tg, group_top=group_top,
                   renormalize=True)


def test_softmax_sum_that_rounds_one_way(ms):
    """31 weights of a little over half a step each are rounded up one by one in the fp32 sum, 1.8e-6 in all: a
    neighbour whose score is its bias must not pass the largest by that."""
    E = 256
    z = np.full((1, E), -40.0, np.float32)
    z[0, :32] = np.float32(np.log(6.05e-8))
    z[0, 0] = 0.0
    for n in (32, 33, 34, 35, 36):
        bias = np.zeros(E, np.float32)
        bias[100] = np.float32(1 - n * 2.0 ** -24)
        _check(ms, z, 2, "f32", bias=bias, score="softmax")


def test_softmax_sum_that_rounds_one_way_in_a_group(ms):
    """The same row: the largest score, nearly taken back by its bias, is its group's best by less than the sum's error
    and comes third by its key; another group's two lie in between."""
    E = 256
    z = np.full((1, E), -40.0, np.float32)
    z[0, :32] = np.float32(np.log(6.05e-8))
    z[0, 2] = 0.0
    s = 1 / np.exp(z[0].astype(np.float64)).sum()
    for over in (1.0e-6, 1.3e-6, 1.6e-6):
        for between in (0.6, 0.75, 0.9):
            bias = np.float32(-1e-3) - np.float32(2e-5) * np.arange(E, dtype=np.float32)   # (no other close scores)
            bias[[0, 1]] = 1e-3
            bias[2] = 1e-3 + over - s
            bias[[32, 33]] = 1e-3 + between * over / 2
            _check(ms, z, 2, "f32", bias=bias, score="softmax", n_groups=8, topk_groups=1, group_top=2)


def test_softmax_without_groups_is_route_topk(ms):
    g = np.random.default_rng(1)
    H, E, T = 256, 64, 50
    x = ms.rmsnorm(dev(g.standard_normal((T, H)).astype(np.float32)))
    eye = torch.zeros(E, H, device="cuda")
    eye[:, :E] = torch.eye(E, device="cuda")        # the logits are the first E activations, exactly
    idx, w = ms.route_topk(x, eye, k=6, renormalize=True)
    gi, gw = ms.route_grouped(x[:, :E].contiguous(), 6, renormalize=True)
    assert torch.equal(idx, gi)
    torch.testing.assert_close(w, gw, rtol=2 * REL, atol=0)


def test_routed_layer_with_grouped_experts(ms):
    """rmsnorm -> router logits -> moe_route_grouped -> permute -> experts -> combine, against the oracle's experts
    under the oracle's routing."""
    shp = synth.MoEShape("grouped", B=8, K=3, H=256, E=16, I=128, k=4, S=1, V=256, router_std=0.2)
    a, lw, _ = routed_layer_inputs(shp, 0)
    x = ms.rmsnorm(dev(a))
    z = x.float() @ dev(lw.w_router).t()
    bias = (0.05 * np.random.default_rng(4).standard_normal(shp.E)).astype(np.float32)
    kw = dict(score="sigmoid", n_groups=4, topk_groups=2, group_top=2, renormalize=True, scale=2.0)
    idx, w = ms.route_grouped(z, shp.k, bias=dev(bias), **kw)
    off, perm, slot = ms.permute(idx, shp.E)
    pk = lambda t: ms.pack_weights(dev(t))   # noqa: E731
    y, ysh = ms.expert_ffn(x, off, perm, pk(lw.w_gate_up), pk(lw.w_down), pk(lw.ws_gate_up), pk(lw.ws_down), shp.k)
    out = ms.combine(y, ysh, slot, w, dev(a))
    torch.cuda.synchronize()
    xh = host(x)
    ri, rw = sp.route(host(z), shp.k, bias=bias, **kw)
    ro, rp, rs = oracle.permute(ri, shp.E)
    ry = oracle.expert_ffn_routed(xh, lw.w_gate_up, lw.w_down, ro, rp, shp.k)
    rsh = oracle.expert_ffn_shared(xh, lw.ws_gate_up, lw.ws_down)
    np.testing.assert_array_equal(host(idx), ri)
    assert_close(host(out), oracle.combine(ry, rsh, rs, rw.astype(np.float32), a), what="layer")
