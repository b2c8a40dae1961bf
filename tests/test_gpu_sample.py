"""GPU parity of spec_sample and spec_verify_sample against the 64-bit oracle.

Tokens are compared exactly: the kernels decide in more than fp32, so that a
draw differs from the oracle's only where u times the total lies within about
1e-12 of a border of the cumulative sum.  probs is the fp64 quotient rounded to
fp32 once: half a step, 2^-24 relative, and 1e-11 for the weights themselves."""
import numpy as np
import pytest
import torch

from oracle import sampling as sp
from speculative_decoding_verification_router_b200 import synth
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu

REL = 2.0 ** -24 + 1e-11
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ms():
    from speculative_decoding_verification_router_b200 import moespec
    return moespec


def _row(g, kind, V):
    """One logits row of a kind that a filter can go wrong on."""
    if kind == "peaked":
        return 1.5 * g.exponential(size=V) + 0.5 * g.standard_normal(V)
    if kind == "zeros":
        return np.zeros(V)
    if kind == "tiny":                      # all weights nearly equal, keys spread over many exponents
        return g.standard_normal(V) * 1e-5
    if kind == "two":                       # two values only: ties at every border
        return g.integers(0, 2, V).astype(float)
    if kind == "lowest":
        return np.full(V, float(np.finfo(np.float32).min))
    if kind == "huge":
        return g.standard_normal(V) * 1e30
    if kind == "one":                       # a single token far above the rest
        x = g.standard_normal(V) - 20
        x[g.integers(V)] = 10
        return x
    x = g.standard_normal(V) * 3
    if kind == "masked":
        x[g.random(V) < 0.9] = -np.inf
    elif kind == "nan":
        x[g.random(V) < 0.3] = np.nan
    elif kind == "inf":
        x[g.random(V) < 0.1] = np.inf
    elif kind == "empty":
        x[:] = -np.inf
        x[:: 2] = np.nan
    return x


KINDS = ["normal", "peaked", "zeros", "tiny", "two", "lowest", "huge", "one", "masked", "nan", "inf", "empty"]


def _params(g, n, V):
    at = lambda v: np.array([v[g.integers(len(v))] for _ in range(n)])   # noqa: E731
    return dict(temperature=at([1.0, 0.7, 0.0, -1.0, 2.0, 1e-3, 100.0, 1.0]).astype(np.float32),
                top_k=at([0, 0, 1, 5, 40, V, V - 1, V + 5, max(1, V // 2), 600, 2500]).astype(np.int32),
                top_p=at([1.0, 1.0, 0.5, 0.9, 0.99, 0.0, -1.0, 1e-6, 2.0]).astype(np.float32),
                min_p=at([0.0, 0.0, 0.1, 1.0, 2.0, 1e-9]).astype(np.float32))


def _logits(g, V, per_kind, dtype):
    z = np.stack([_row(g, k, V) for k in KINDS for _ in range(per_kind)])
    with np.errstate(over="ignore"):
        t = torch.from_numpy(z.astype(np.float32)).to(DTYPES[dtype])
    return t.cuda(), t.float().numpy()


def _uniform(g, shape):
    u = (g.integers(0, 1 << 24, shape) * 2.0 ** -24).astype(np.float32)
    u[g.random(shape) < 0.1] = 0.0
    u[g.random(shape) < 0.1] = 1.0 - 2.0 ** -24
    return u


def _on(p):
    return {n: None if v is None else dev(v) for n, v in p.items()}


def _assert_probs(got, want):
    assert np.all(np.abs(got.astype(np.float64) - want) <= REL * want), np.abs(got - want).max()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 33, 1000, 1025, 4099, 20001])
def test_sample_matches_the_oracle(ms, V, dtype):
    g = np.random.default_rng(V)
    z, zh = _logits(g, V, 4, dtype)
    par = _params(g, len(zh), V)
    u = _uniform(g, len(zh))
    tok, probs = ms.sample(z, dev(u), **_on(par), return_probs=True)
    only = ms.sample(z, dev(u), **_on(par))
    torch.cuda.synchronize()
    want, wp = sp.sample(zh, u, **par)
    np.testing.assert_array_equal(host(tok), want)
    np.testing.assert_array_equal(host(only), want)
    _assert_probs(host(probs), wp)


FILTERS = {
    "temperature": dict(temperature=0.8), "nothing": dict(), "greedy": dict(temperature=0.0),
    "top_k": dict(top_k=50), "wide_top_k": dict(temperature=1.1, top_k=5000), "top_p": dict(top_p=0.9),
    "wide_top_p": dict(temperature=1.5, top_p=0.98), "min_p": dict(min_p=0.05),
    "all": dict(temperature=0.7, top_k=40, top_p=0.95, min_p=0.02),
    "wide_both": dict(temperature=1.5, top_k=20000, top_p=0.9)}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(FILTERS))
def test_sample_full_vocabulary(ms, name, dtype):
    V, R = 129280, 6
    g = np.random.default_rng(7)
    z = torch.from_numpy((g.exponential(size=(R, V)) * np.linspace(0.7, 1.8, R)[:, None] - 2).astype(np.float32))
    z = z.to(DTYPES[dtype])
    u = _uniform(g, R)
    par = {n: np.full(R, v, np.int32 if n == "top_k" else np.float32) for n, v in FILTERS[name].items()}
    tok, probs = ms.sample(z.cuda(), dev(u), **_on(par), return_probs=True)
    torch.cuda.synchronize()
    want, wp = sp.sample(z.float().numpy(), u, **par)
    np.testing.assert_array_equal(host(tok), want)
    _assert_probs(host(probs), wp)


@pytest.mark.parametrize("V", [262144, 200001])
def test_sample_largest_vocabulary(ms, V):
    g = np.random.default_rng(9)
    z = torch.from_numpy(g.standard_normal((2, V)).astype(np.float32))
    u = _uniform(g, 2)
    par = dict(temperature=np.array([1.0, 3.0], np.float32), top_p=np.array([1.0, 0.97], np.float32))
    tok = ms.sample(z.cuda(), dev(u), **_on(par))
    np.testing.assert_array_equal(host(tok), sp.sample(z.numpy(), u, **par)[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [16896, 16897, 32768, 32769, 33792, 33793, 65537, 66310, 67585, 131073, 135169])
def test_vocabularies_around_the_parts_of_a_cluster(ms, V, dtype):
    """Full batches (clusters no wider than the rows need) on both sides of the sizes at which a row takes another CTA."""
    R = 160
    g = torch.Generator(device="cuda").manual_seed(V)
    z = (2 * torch.randn(R, V, generator=g, device="cuda")).to(DTYPES[dtype])
    u = torch.rand(R, generator=g, device="cuda")
    par = dict(temperature=torch.full((R,), 0.9, device="cuda"),
               top_p=torch.tensor([1.0, 0.9, 0.5, 1.0] * (R // 4), device="cuda"),
               top_k=torch.tensor([0, 0, 0, 50] * (R // 4), dtype=torch.int32, device="cuda"))
    tok, probs = ms.sample(z, u, **par, return_probs=True)
    at = [0, 1, 2, 3, R - 4, R - 3, R - 2, R - 1]
    want, wp = sp.sample(host(z[at].float()), host(u[at]), **{k: host(v[at]) for k, v in par.items()})
    np.testing.assert_array_equal(host(tok[at]), want)
    _assert_probs(host(probs[at]), wp)
    for r in range(4, R - 4, 13):   # alone, a row takes a wider cluster
        t, p = ms.sample(z[r:r + 1], u[r:r + 1], **{k: v[r:r + 1] for k, v in par.items()}, return_probs=True)
        assert torch.equal(t, tok[r:r + 1])
        assert bool(((p - probs[r:r + 1]).abs() <= 2.0 ** -23 * p).all())   # both round sums that agree to 1e-15


def test_equal_weights_are_split_exactly(ms):
    # the border cases that rounding would decide: 2n equal weights, top_p 0.5 keeps n, u = i / 2n draws token i
    for n in (4, 512, 4096):
        V = 2 * n
        z = torch.full((V, V), 0.3, device="cuda")
        u = torch.arange(V, device="cuda", dtype=torch.float32) / V
        tok = ms.sample(z, u)
        assert torch.equal(tok, torch.arange(V, device="cuda", dtype=torch.int32))
        half = torch.full((V,), 0.5, device="cuda")
        _, p = ms.sample(z, u, top_p=half, return_probs=True)
        assert torch.equal((p > 0).sum(1), torch.full((V,), n, device="cuda"))
        assert bool((p[:, :n] > 0).all())


def test_sample_does_not_depend_on_the_batch_or_the_run(ms):
    g = np.random.default_rng(2)
    z, _ = _logits(g, 5003, 8, "bf16")
    n = z.shape[0]
    par, u = _on(_params(g, n, 5003)), dev(_uniform(g, n))
    a = ms.sample(z, u, **par, return_probs=True)
    b = ms.sample(z, u, **par, return_probs=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for r in range(0, n, 5):
        t, p = ms.sample(z[r:r + 1], u[r:r + 1], **{k: v[r:r + 1] for k, v in par.items()}, return_probs=True)
        assert torch.equal(t, a[0][r:r + 1]) and torch.equal(p, a[1][r:r + 1])


def test_sample_writes_only_its_rows(ms):
    V = 777
    z = torch.randn(3, V, device="cuda")
    probs = torch.full((5, V), 7.0, device="cuda")
    tok = torch.full((5,), 7, dtype=torch.int32, device="cuda")
    ms.sample(z, torch.rand(3, device="cuda"), return_probs=True, out=(tok[1:4], probs[1:4]))
    assert bool((probs[[0, 4]] == 7).all()) and bool((tok[[0, 4]] == 7).all())


def test_sample_on_another_stream_and_captured(ms):
    V, R = 20000, 5
    z = torch.randn(R, V, device="cuda") * 3
    u, tok = torch.rand(R, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda")
    top_p = torch.full((R,), 0.9, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ms.sample(z, u, top_p=top_p, out=tok, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(tok, ms.sample(z, u, top_p=top_p))
    graph = ms.CapturedStep(lambda: ms.sample(z, u, top_p=top_p, out=tok))
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        z.normal_(generator=g).mul_(3)
        u.uniform_(generator=g)
        torch.cuda.synchronize()
        graph()
        torch.cuda.synchronize()
        assert torch.equal(tok, ms.sample(z, u, top_p=top_p))


def test_extreme_temperatures(ms):
    V, ts = 5000, [1e-38, 1e-30, 1e-20, 1e20, 1e38, np.inf]
    g = np.random.default_rng(3)
    for dtype in DTYPES:
        for kinds in (["normal", "tiny", "two", "masked", "huge", "lowest"], ["inf", "nan", "zeros", "peaked", "one", "empty"]):
            for ps in (dict(), dict(top_p=0.9), dict(top_k=3000, top_p=0.5), dict(min_p=0.3)):
                z = np.stack([_row(g, k, V) for k in kinds for _ in ts]).astype(np.float32)
                t = torch.from_numpy(z).to(DTYPES[dtype])
                n, u = len(z), _uniform(g, len(z))
                par = {k: np.full(n, v, np.int32 if k == "top_k" else np.float32) for k, v in ps.items()}
                par["temperature"] = np.array(ts * len(kinds), np.float32)
                tok, probs = ms.sample(t.cuda(), dev(u), **_on(par), return_probs=True)
                with np.errstate(all="ignore"):
                    want, wp = sp.sample(t.float().numpy(), u, **par)
                np.testing.assert_array_equal(host(tok), want)
                _assert_probs(host(probs), wp)


def test_parameters_that_leave_their_filter_out(ms):
    R, V = 8, 6000
    g = np.random.default_rng(12)
    t = torch.from_numpy((2 * g.standard_normal((R, V))).astype(np.float32))
    u = _uniform(g, R)
    nan = np.float32(np.nan)
    par = dict(temperature=np.array([nan, 1, 1, 1, nan, 0.5, 1, -np.inf], np.float32),
               top_k=np.array([0, -5, -2 ** 31, 2 ** 31 - 1, 3, 40, V, 1], np.int32),
               top_p=np.array([nan, nan, 0.5, np.inf, 0.5, nan, -np.inf, 0.5], np.float32),
               min_p=np.array([nan, nan, -1, nan, 0.5, nan, 0, np.inf], np.float32))
    for dtype in DTYPES:
        z = t.to(DTYPES[dtype])
        tok, probs = ms.sample(z.cuda(), dev(u), **_on(par), return_probs=True)
        want, wp = sp.sample(z.float().numpy(), u, **par)
        np.testing.assert_array_equal(host(tok), want)
        _assert_probs(host(probs), wp)


def test_random_numbers_outside_their_range_are_clamped(ms):
    z = torch.randn(4, 9000, device="cuda")
    top_k = torch.tensor([0, 50, 0, 50], dtype=torch.int32, device="cuda")
    a = ms.sample(z, torch.tensor([-1.0, -1.0, 7.0, float("nan")], device="cuda"), top_k=top_k)
    b = ms.sample(z, torch.tensor([0.0, 0.0, 1 - 2.0 ** -24, 1 - 2.0 ** -24], device="cuda"), top_k=top_k)
    assert torch.equal(a, b)


def _around_zero(g, R, V):
    """Rows whose kept sets end among very many small values: |l| far under the range between the maximum and the
    last value with weight, ties among them, both signs of zero."""
    z = g.standard_normal((R, V)) * np.logspace(-6, -1, R)[:, None]
    z[:, ::7] = np.round(z[:, ::7] * 64) / 64
    z[:, ::11] = -0.0
    z[np.arange(R), g.integers(0, V, R)] = 30.0
    z[:, ::5] = -g.exponential(size=z[:, ::5].shape) * 500
    return z.astype(np.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("par", [dict(top_p=0.6), dict(top_k=9000), dict(top_k=9000, top_p=0.9), dict(top_k=2500)],
                         ids=["p", "k", "kp", "k2"])
def test_borders_among_small_values(ms, par, dtype):
    R, V = 12, 20003
    g = np.random.default_rng(5)
    t = torch.from_numpy(_around_zero(g, R, V)).to(DTYPES[dtype])
    u = _uniform(g, R)
    par = {k: np.full(R, v, np.int32 if k == "top_k" else np.float32) for k, v in par.items()}
    par["temperature"] = np.repeat(np.array([50, 8, 500], np.float32), R // 3)
    tok, probs = ms.sample(t.cuda(), dev(u), **_on(par), return_probs=True)
    want, wp = sp.sample(t.float().numpy(), u, **par)
    np.testing.assert_array_equal(host(tok), want)
    _assert_probs(host(probs), wp)
    # as verification: drafts among the small values, certain and with their distributions
    B, K = R // 3, 2
    z = t.view(B, K + 1, V)
    zh = z.float().numpy()
    d = g.integers(0, V, (B, K)).astype(np.int32)
    uv = _uniform(g, (B, K + 1)) * np.float32(1e-3)
    pv = {k: v[:: 3].copy() for k, v in par.items()}
    q = np.full((B, K, V), 1.0 / V, np.float32)
    for qq in (None, q):
        cm, n = ms.verify_sample(z.cuda(), dev(d), dev(uv), draft_probs=None if qq is None else dev(qq), **_on(pv))
        wcm, wn = sp.verify(zh, d, uv, qq, **pv)
        np.testing.assert_array_equal(host(cm), wcm)
        np.testing.assert_array_equal(host(n), wn)


@pytest.mark.parametrize("temperature,k", [(0.05, 2500), (0.3, 20000), (0.3, 49999)], ids=["fewer", "last", "all"])
@pytest.mark.parametrize("R", [5, 48])
def test_wide_top_k_whose_kth_token_is_not_counted(ms, R, temperature, k):
    """fp32 rows whose k-th token lies in the uncounted last interval, or that hold fewer than k tokens above the cut;
    50,000 fp32 are 3,126 vectors a CTA of 4 in warp segments of 224, so that the last two warps have none."""
    V = 50000
    g = np.random.default_rng(k)
    z = (g.standard_normal((R, V)) * (1.0 if k == 2500 else 3.0)).astype(np.float32)
    u = _uniform(g, R)
    for top_p in (None, 0.95):
        par = dict(temperature=np.full(R, temperature, np.float32), top_k=np.full(R, k, np.int32))
        if top_p:
            par["top_p"] = np.full(R, top_p, np.float32)
        tok, probs = ms.sample(dev(z), dev(u), **_on(par), return_probs=True)
        want, wp = sp.sample(z, u, **par)
        np.testing.assert_array_equal(host(tok), want)
        _assert_probs(host(probs), wp)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sample_from_any_element_offset(ms, dtype):
    """Rows and outputs that start at any element, filters that take every path."""
    R, V = 6, 10007
    g = torch.Generator(device="cuda").manual_seed(4)
    z = (3 * torch.randn(R, V, generator=g, device="cuda")).to(DTYPES[dtype])
    u = torch.rand(R, generator=g, device="cuda")
    par = dict(temperature=torch.tensor([1, 1, 2, 2, 3, 1.0], device="cuda"),
               top_k=torch.tensor([0, 30, 0, 4000, 0, 0], dtype=torch.int32, device="cuda"),
               top_p=torch.tensor([1, 1, 0.95, 0.9, 0.999, 1], device="cuda"),
               min_p=torch.tensor([0, 0, 0, 0, 0, 0.01], device="cuda"))
    tok, probs = ms.sample(z, u, **par, return_probs=True)
    for shift in range(1, 8):
        zs = torch.empty(R * V + 8, dtype=z.dtype, device="cuda")[shift: shift + R * V].view(R, V).copy_(z)
        out = torch.full((R * V + 16,), 7.0, device="cuda")
        t = torch.empty(R, dtype=torch.int32, device="cuda")
        ms.sample(zs, u, **par, return_probs=True, out=(t, out[shift: shift + R * V].view(R, V)))
        assert torch.equal(t, tok) and torch.equal(out[shift: shift + R * V].view(R, V), probs)
        assert bool((out[:shift] == 7).all()) and bool((out[shift + R * V:] == 7).all())


def test_offsets_beyond_32_bits(ms):
    R, V = 8250, 262144            # 2.16e9 logits and probabilities
    g = torch.Generator(device="cuda").manual_seed(6)
    z = torch.zeros(R, V, dtype=torch.bfloat16, device="cuda")
    z[-40:].normal_(generator=g).mul_(2)
    u = torch.rand(R, generator=g, device="cuda")
    top_k = torch.tensor([0, 20, 5000, 0] * (R // 4) + [20, 20], dtype=torch.int32, device="cuda")
    tok, probs = ms.sample(z, u, top_k=top_k, return_probs=True)
    t, p = ms.sample(z[-40:].clone(), u[-40:], top_k=top_k[-40:], return_probs=True)
    assert torch.equal(tok[-40:], t) and torch.equal(probs[-40:], p)
    want, _ = sp.sample(host(z[-2:].float()), host(u[-2:]), top_k=host(top_k[-2:]))
    np.testing.assert_array_equal(host(t[-2:]), want)
    del z, probs


def test_two_streams_at_once(ms):
    R, V = 64, 50000
    z = [torch.randn(R, V, device="cuda") * (1 + i) for i in range(2)]
    u = torch.rand(R, device="cuda")
    top_p = torch.full((R,), 0.95, device="cuda")
    want = [ms.sample(x, u, top_p=top_p, return_probs=True) for x in z]
    streams = [torch.cuda.Stream() for _ in z]
    out = [(torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, V, device="cuda")) for _ in z]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, s, o in zip(z, streams, out):
            ms.sample(x, u, top_p=top_p, return_probs=True, out=o, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(out, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def test_outputs_belong_to_the_stream_that_writes_them(ms):
    """Memory freed on the current stream may still be in use there: a call on another stream must not be given it."""
    R, V, E, s = 640, 64, 64, torch.cuda.Stream()
    z, u = torch.randn(R, V, device="cuda"), torch.rand(R, device="cuda")
    zv, uv = z.view(R // 4, 4, V), u.view(R // 4, 4)
    d = torch.zeros(R // 4, 3, dtype=torch.int32, device="cuda")
    calls = [lambda: ms.sample(z, u, return_probs=True, stream=s), lambda: ms.verify_sample(zv, d, uv, stream=s),
             lambda: ms.route_grouped(z, 1, stream=s)]
    want = [ms.sample(z, u, return_probs=True), ms.verify_sample(zv, d, uv), ms.route_grouped(z, 1)]
    torch.cuda.synchronize()
    for call, w in zip(calls, want):
        freed = [torch.empty_like(x) for x in w for _ in range(3)]
        at = {x.data_ptr() for x in freed}
        del freed
        out = call()
        torch.cuda.synchronize()
        assert not any(x.data_ptr() in at for x in out)
        assert all(torch.equal(x, y) for x, y in zip(out, w))


# ---------------------------------------------------------------- verification

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("with_q", [False, True])
@pytest.mark.parametrize("V,K", [(1, 1), (5, 2), (129, 1), (1003, 3), (4099, 8), (20001, 3)])
def test_verify_sample_matches_the_oracle(ms, V, K, with_q, dtype):
    g = np.random.default_rng(V + K)
    z, zh = _logits(g, V, K + 1, dtype)
    g.shuffle(perm := np.arange(len(zh)))
    B = len(zh) // (K + 1)
    z = z[torch.from_numpy(perm[: B * (K + 1)]).cuda()].view(B, K + 1, V).contiguous()
    zh = zh[perm[: B * (K + 1)]].reshape(B, K + 1, V)
    par, u = _params(g, B, V), _uniform(g, (B, K + 1))
    best = np.nan_to_num(zh[:, :K], nan=-np.inf).argmax(-1)
    d = np.where(g.random((B, K)) < 0.6, best, g.integers(-2, V + 2, (B, K))).astype(np.int32)
    q = None
    if with_q:
        q = g.random((B, K, V)) ** 8
        q = (q / q.sum(-1, keepdims=True)).astype(np.float32)
    cm, n = ms.verify_sample(z, dev(d), dev(u), draft_probs=None if q is None else dev(q), **_on(par))
    torch.cuda.synchronize()
    wcm, wn = sp.verify(zh, d, u, q, **par)
    np.testing.assert_array_equal(host(cm), wcm)
    np.testing.assert_array_equal(host(n), wn)


@pytest.mark.parametrize("par", [dict(temperature=0.8), dict(temperature=1.2, top_p=0.95), dict(top_k=50, top_p=0.9)],
                         ids=["temperature", "top_p", "top_k_p"])
@pytest.mark.parametrize("with_q", [False, True])
def test_verify_sample_full_vocabulary(ms, par, with_q):
    B, K, V = 3, 3, 129280
    g = np.random.default_rng(11)
    z = torch.from_numpy((g.exponential(size=(B, K + 1, V)) * 1.2).astype(np.float32)).bfloat16()
    zh = z.float().numpy()
    par = {n: np.full(B, v, np.int32 if n == "top_k" else np.float32) for n, v in par.items()}
    u = _uniform(g, (B, K + 1))
    d = zh[:, :K].argmax(-1).astype(np.int32)
    q = None
    if with_q:
        q = np.exp(zh[:, :K] + g.standard_normal((B, K, V)))
        q = (q / q.sum(-1, keepdims=True)).astype(np.float32)
    cm, n = ms.verify_sample(z.cuda(), dev(d), dev(u), draft_probs=None if q is None else dev(q), **_on(par))
    wcm, wn = sp.verify(zh, d, u, q, **par)
    np.testing.assert_array_equal(host(cm), wcm)
    np.testing.assert_array_equal(host(n), wn)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("par", [dict(temperature=1.5), dict(top_k=50), dict(temperature=1.5, top_p=0.97), dict(top_k=4000)],
                         ids=["row", "list", "p", "k"])
def test_draft_probs_that_are_infinite_or_nan(ms, par, dtype):
    """They reject their draft and leave nothing of their tokens, whatever the sign of a NaN and the way of the row."""
    B, K, V = 24, 2, 20011
    g = np.random.default_rng(13)
    z = torch.from_numpy((2 * g.standard_normal((B, K + 1, V))).astype(np.float32)).to(DTYPES[dtype])
    zh = z.float().numpy()
    q = np.exp(zh[:, :K] + g.standard_normal((B, K, V)))
    q = (q / q.sum(-1, keepdims=True)).astype(np.float32)
    d = zh[:, :K].argmax(-1).astype(np.int32)
    bad = np.array([0x7fc00000, 0xffc00000, 0xffffffff, 0x7f800001, 0xff800001, 0x7f800000], np.uint32).view(np.float32)
    best = np.argsort(-zh[:, :K], axis=-1)[..., :12]
    for r in range(0, B, 2):
        for j in range(K):
            for i in range(1 if r % 4 else 0, 12):   # every other time the draft's own among them
                q[r, j, best[r, j, i]] = bad[(r + i) % len(bad)]
    q[1::2, :, ::97] = bad[g.integers(0, len(bad), q[1::2, :, ::97].shape)]
    par = {n: np.full(B, v, np.int32 if n == "top_k" else np.float32) for n, v in par.items()}
    u = _uniform(g, (B, K + 1))
    cm, n = ms.verify_sample(z.cuda(), dev(d), dev(u), draft_probs=dev(q), **_on(par))
    torch.cuda.synchronize()
    # a u of 0 times an infinite probability is NaN: no acceptance either
    with np.errstate(invalid="ignore"):
        wcm, wn = sp.verify(zh, d, u, np.where(np.isfinite(q), q, np.inf).astype(np.float32), **par)
    np.testing.assert_array_equal(host(cm), wcm)
    np.testing.assert_array_equal(host(n), wn)


def test_greedy_rows_verify_as_spec_verify_greedy(ms):
    B, K, V = 16, 3, 4096
    z = torch.randn(B, K + 1, V, device="cuda").bfloat16()
    d = z[:, :K].float().argmax(-1).int()
    d[::3, 1] += 1
    d.clamp_(max=V - 1)
    zero = torch.zeros(B, device="cuda")
    cm, n = ms.verify_sample(z, d, torch.rand(B, K + 1, device="cuda"), temperature=zero)
    _, gcm, gn = ms.verify_greedy(z, d)
    assert torch.equal(cm, gcm) and torch.equal(n, gn)


def test_no_drafts_is_plain_sampling(ms):
    B, V = 40, 3001
    z, u = torch.randn(B, 1, V, device="cuda"), torch.rand(B, 1, device="cuda")
    t = torch.full((B,), 0.9, device="cuda")
    cm, n = ms.verify_sample(z, torch.empty((B, 0), dtype=torch.int32, device="cuda"), u, temperature=t)
    assert torch.equal(cm[:, 0], ms.sample(z[:, 0], u[:, 0], temperature=t)) and bool((n == 1).all())


@pytest.mark.parametrize("certain", [False, True])
def test_committed_tokens_follow_the_sampled_distribution(ms, certain):
    """Draft with spec_sample, verify with spec_verify_sample, B times on the same rows: the first committed
    token's counts are binomial with p_0, so each lies within 6 standard deviations (two in 10^9 a token)."""
    V, B, K = 24, 60000, 2
    g = torch.Generator(device="cuda").manual_seed(5)
    z1 = 1.5 * torch.randn(1, K + 1, V, generator=g, device="cuda")
    zd = z1[:, :K] + torch.randn(1, K, V, generator=g, device="cuda")
    z = z1.expand(B, K + 1, V).contiguous()
    top_p, t = torch.full((B,), 0.9, device="cuda"), torch.full((B,), 0.8, device="cuda")
    if certain:
        d, q = zd.argmax(-1).int().expand(B, K).contiguous(), None
    else:
        d, q = ms.sample(zd.expand(B, K, V).reshape(B * K, V), torch.rand(B * K, generator=g, device="cuda"),
                         return_probs=True)
        d, q = d.view(B, K), q.view(B, K, V)
    cm, n = ms.verify_sample(z, d, torch.rand(B, K + 1, generator=g, device="cuda"), temperature=t, top_p=top_p,
                             draft_probs=q)
    p = sp.distribution(host(z1)[0, 0], 0.800000011920929, 0, 0.8999999761581421)
    p /= p.sum()
    got = np.bincount(host(cm)[:, 0], minlength=V) / B
    assert np.all(np.abs(got - p) <= 6 * np.sqrt(p * (1 - p) / B) + 1e-12), (got, p)
    assert 1 < float(n.float().mean()) < K + 1


def test_verify_sample_captured(ms):
    B, K, V = 4, 3, 30011
    z, u = torch.empty(B, K + 1, V, device="cuda"), torch.empty(B, K + 1, device="cuda")
    d = torch.zeros(B, K, dtype=torch.int32, device="cuda")
    k = torch.full((B,), 20, dtype=torch.int32, device="cuda")
    out = (torch.empty(B, K + 1, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda"))
    z.normal_()
    u.uniform_()
    graph = ms.CapturedStep(lambda: ms.verify_sample(z, d, u, top_k=k, out=out))
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        z.normal_(generator=g).mul_(2)
        u.uniform_(generator=g)
        d.copy_(z[:, :K].argmax(-1))
        torch.cuda.synchronize()
        graph()
        torch.cuda.synchronize()
        cm, n = ms.verify_sample(z, d, u, top_k=k)
        assert torch.equal(out[0], cm) and torch.equal(out[1], n)


def test_draft_probs_beyond_32_bits(ms):
    B, K, V = 1040, 8, 262144      # 2.18e9 draft probabilities, 2.45e9 logits
    z = torch.zeros(B, K + 1, V, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(B, K, V, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    z[-2:].normal_(generator=g).mul_(3)
    d = z[:, :K].argmax(-1).int()
    q[-2:] = torch.softmax(z[-2:, :K].float() + 0.5 * torch.randn(2, K, V, generator=g, device="cuda"), -1)
    u = 0.7 * torch.rand(B, K + 1, generator=g, device="cuda")
    top_p = torch.full((B,), 0.9, device="cuda")
    cm, n = ms.verify_sample(z, d, u, top_p=top_p, draft_probs=q)
    want = ms.verify_sample(z[-2:].clone(), d[-2:], u[-2:], top_p=top_p[-2:], draft_probs=q[-2:].clone())
    assert torch.equal(cm[-2:], want[0]) and torch.equal(n[-2:], want[1])
    wcm, wn = sp.verify(host(z[-1:].float()), host(d[-1:]), host(u[-1:]), host(q[-1:]), top_p=host(top_p[-1:]))
    np.testing.assert_array_equal(host(cm[-1:]), wcm)
    np.testing.assert_array_equal(host(n[-1:]), wn)


def test_verify_two_graphs_with_draft_probs(ms):
    """Two captured graphs of the same inputs, replayed at once, each on its own stream."""
    B, K, V = 6, 2, 20011
    z = 2 * torch.randn(B, K + 1, V, device="cuda")
    q = torch.softmax(z[:, :K] + torch.randn(B, K, V, device="cuda"), -1)
    u, d = torch.rand(B, K + 1, device="cuda"), z[:, :K].argmax(-1).int()
    outs = [(torch.empty(B, K + 1, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda"))
            for _ in range(2)]
    graphs = [ms.CapturedStep(lambda o=o: ms.verify_sample(z, d, u, draft_probs=q, out=o)) for o in outs]
    for seed in range(4):
        u.uniform_(generator=torch.Generator(device="cuda").manual_seed(seed))
        torch.cuda.synchronize()
        for graph in graphs:
            graph()
        torch.cuda.synchronize()
        cm, n = ms.verify_sample(z, d, u, draft_probs=q)
        for o in outs:
            assert torch.equal(o[0], cm) and torch.equal(o[1], n)


def test_draft_head_sampled_verify_chain(ms):
    """A speculative step of sampled decoding through the library: FastMTP drafts (certain), the vocabulary head
    over the verify rows, sampled verification of its logits."""
    B, H, I, V, K = 4, 256, 128, 1024, 3
    n = lambda name, shape, std: dev(synth.normal_bf16(3, name, shape, std))   # noqa: E731
    pk = ms.pack_weights
    emb, w_lm = n("e", (V, H), 1.0), pk(n("lm", (V, H), 0.2))
    drafts, h = ms.fastmtp_draft(torch.randn(B, H, device="cuda"), torch.arange(B, dtype=torch.int32, device="cuda"),
                                 emb, pk(n("p", (H, 2 * H), 0.05)), pk(n("gu", (2 * I, H), 0.05)),
                                 pk(n("d", (H, I), 0.05)), w_lm, K)
    x = ms.rmsnorm(torch.randn(B * (K + 1), H, device="cuda"))
    logits = ms.lm_head(x, w_lm).view(B, K + 1, V)
    u = torch.rand(B, K + 1, device="cuda")
    par = dict(temperature=np.full(B, 0.9, np.float32), top_p=np.full(B, 0.95, np.float32))
    cm, cnt = ms.verify_sample(logits, drafts, u, **_on(par))
    torch.cuda.synchronize()
    wcm, wn = sp.verify(host(logits), host(drafts), host(u), None, **par)
    np.testing.assert_array_equal(host(cm), wcm)
    np.testing.assert_array_equal(host(cnt), wn)


def test_binding_refusals(ms):
    z, u = torch.zeros(4, 16, device="cuda"), torch.zeros(4, device="cuda")
    i = torch.zeros(4, 3, dtype=torch.int32, device="cuda")
    for bad in (lambda: ms.sample(z.half(), u), lambda: ms.sample(z[:, ::2], u), lambda: ms.sample(z, u[:3]),
                lambda: ms.sample(z, u.double()), lambda: ms.sample(z[0], u), lambda: ms.sample(z, u.cpu()),
                lambda: ms.sample(z, u, top_k=u), lambda: ms.sample(z, u, temperature=u[:2]),
                lambda: ms.sample(z, u, out=torch.zeros(4, device="cuda")),
                lambda: ms.verify_sample(z.view(1, 4, 16), i, u.view(1, 4)),
                lambda: ms.verify_sample(z.view(1, 4, 16), i[:1], u.view(1, 4), draft_probs=z[None])):
        with pytest.raises(ValueError):
            bad()
