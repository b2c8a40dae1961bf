"""The sampling and grouped-routing calls refuse bad arguments on the host,
before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from speculative_decoding_verification_router_b200 import build

P = ctypes.c_void_p
FAKE = P(4096)   # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def ms():
    build.build()
    from speculative_decoding_verification_router_b200 import moespec
    return moespec


@pytest.mark.parametrize("change,code", [
    (dict(logits=None), -1), (dict(u=None), -1), (dict(token=None), -1), (dict(T=0), -1), (dict(V=0), -1),
    (dict(T=-3), -1), (dict(dt=2), -1), (dict(logits=P(4097)), -1), (dict(V=262145), -2), (dict(T=(1 << 24) + 1), -2)])
def test_sample_refusals(ms, change, code):
    a = dict(logits=FAKE, dt=1, T=4, V=1000, u=FAKE, token=FAKE)
    a.update(change)
    assert ms.lib().spec_sample(a["logits"], a["dt"], a["T"], a["V"], None, None, None, None, a["u"], a["token"], None,
                                None) == code


@pytest.mark.parametrize("change,code", [
    (dict(logits=None), -1), (dict(draft=None), -1), (dict(u=None), -1), (dict(cm=None), -1), (dict(n=None), -1),
    (dict(B=0), -1), (dict(K=-1), -1), (dict(V=0), -1), (dict(dt=5), -1), (dict(K=9), -2), (dict(V=262145), -2),
    (dict(logits=P(4098)), -1)])
def test_verify_sample_refusals(ms, change, code):
    a = dict(logits=FAKE, dt=0, draft=FAKE, u=FAKE, B=2, K=3, V=1000, cm=FAKE, n=FAKE)
    a.update(change)
    assert ms.lib().spec_verify_sample(a["logits"], a["dt"], a["draft"], None, None, None, None, None, a["u"], a["B"],
                                       a["K"], a["V"], a["cm"], a["n"], None) == code


@pytest.mark.parametrize("change,code", [
    (dict(z=None), -1), (dict(idx=None), -1), (dict(w=None), -1), (dict(T=0), -1), (dict(E=0), -1), (dict(dt=3), -1),
    (dict(score=2), -1), (dict(G=0), -1), (dict(G=7), -1), (dict(tg=0), -1), (dict(tg=9), -1), (dict(gt=0), -1),
    (dict(gt=3), -1), (dict(k=0), -1), (dict(k=33), -1), (dict(z=P(4098)), -1), (dict(E=512, k=4), -2),
    (dict(E=128, G=64, tg=64, k=4), -2), (dict(G=1, tg=1, k=40), -2)])
def test_route_grouped_refusals(ms, change, code):
    a = dict(z=FAKE, dt=0, T=4, E=64, score=1, G=8, tg=4, gt=2, k=6, idx=FAKE, w=FAKE)
    a.update(change)
    assert ms.lib().moe_route_grouped(a["z"], a["dt"], None, a["T"], a["E"], a["score"], a["G"], a["tg"], a["gt"],
                                      a["k"], 1, 1.0, a["idx"], a["w"], None) == code


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("at", range(7))
def test_sample_refuses_pointers_between_elements(ms, at, off):
    p = [P(4096)] * 7   # temperature, top_k, top_p, min_p, u, token, probs
    p[at] = P(4096 + off)
    assert ms.lib().spec_sample(FAKE, 1, 4, 1000, *p, None) == -1


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("at", range(9))
def test_verify_sample_refuses_pointers_between_elements(ms, at, off):
    p = [P(4096)] * 9   # draft, draft_probs, temperature, top_k, top_p, min_p, u, committed, n_committed
    p[at] = P(4096 + off)
    assert ms.lib().spec_verify_sample(FAKE, 0, *p[:7], 2, 3, 1000, *p[7:], None) == -1


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("at", range(3))
def test_route_grouped_refuses_pointers_between_elements(ms, at, off):
    p = [P(4096)] * 3   # bias, topk_idx, topk_w
    p[at] = P(4096 + off)
    assert ms.lib().moe_route_grouped(FAKE, 0, p[0], 4, 64, 1, 8, 4, 2, 6, 1, 1.0, p[1], p[2], None) == -1


def test_binding_refuses_tensors_it_cannot_take(ms):
    z = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        ms.sample(z, torch.zeros(2))                       # not on a GPU
    with pytest.raises(ValueError):
        ms.verify_sample(z.view(1, 2, 8), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2))
    with pytest.raises(ValueError):
        ms.route_grouped(z, 2)
