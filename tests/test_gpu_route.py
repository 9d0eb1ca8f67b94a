"""Routing and the weighted sum against the formulas in 64 bits.

Weights are computed in 64 bits and rounded to fp32: 2^-24 of themselves, and as much
again for the scale.  The weighted sum of k terms in fp32 is off by at most
(k + 1) 2^-24 of the sum of magnitudes, its result's rounding to bf16 by 2^-8."""
import math

import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


def scores(l, kind):
    if kind == "sigmoid":
        return torch.special.expit(l)
    top = l.amax(dim=1, keepdim=True)
    e = torch.where(l == -math.inf, torch.zeros_like(l), torch.exp(l - torch.where(top == -math.inf, torch.zeros_like(top), top)))
    return e / e.sum(dim=1, keepdim=True).clamp(min=1e-300)


def reference(logits, k, bias=None, score="softmax", renorm=True, scale=1.0, groups=1, top_groups=1):
    """(w, ids) on the CPU, token by token and expert by expert."""
    l = logits.cpu().double()
    l = torch.where(torch.isnan(l), torch.full_like(l, -math.inf), l.clamp(max=3.4028234663852886e38))
    T, E = l.shape
    s = scores(l, score)
    c = s if bias is None else s + bias.cpu().double()
    w, ids = torch.zeros(T, k, dtype=torch.float64), torch.full((T, k), -1, dtype=torch.int32)
    size = E // groups
    for t in range(T):
        choice = [-math.inf if l[t, e] == -math.inf or math.isnan(c[t, e]) else c[t, e].item() for e in range(E)]
        kept = range(groups)
        if top_groups < groups:
            best = [sum(sorted(choice[g * size:(g + 1) * size])[-2:]) for g in range(groups)]
            kept = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
        rank = choice if bias is not None else l[t].tolist()
        left = [e for e in range(E) if e // size in kept and choice[e] > -math.inf]
        chosen = sorted(left, key=lambda e: (-rank[e], e))[:k]
        v = s[t, chosen]
        if score == "softmax" and renorm and chosen:
            v = torch.exp(l[t, chosen] - l[t, chosen].max())
        if renorm and chosen:
            v = v / v.sum() if v.sum() > 0 else torch.zeros_like(v)
        ids[t, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
        w[t, :len(chosen)] = v * scale
    return w, ids


def check(logits, k, **how):
    w, ids = any4.route(logits, k, **how)
    want, want_ids = reference(logits, k, **how)
    assert w.dtype == torch.float32 and ids.dtype == torch.int32
    assert torch.equal(ids.cpu(), want_ids)
    assert ((w.cpu().double() - want).abs() <= 2.0 ** -22 * want.abs() + 2.0 ** -149).all()
    return w, ids


def logits_of(T, E, seed=1, dtype=torch.float32, std=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * std).to(dtype).to(gu.DEV)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (5, 7, 7), (33, 64, 6), (9, 65, 1), (6, 200, 8), (3, 513, 64), (5, 1024, 9)])
def test_choice_and_weights(dtype, score, T, E, k):
    l = logits_of(T, E, dtype=dtype)
    bias = logits_of(1, E, seed=2)[0] * 0.1
    for renorm in (True, False):
        check(l, k, score=score, renorm=renorm, scale=2.5)
        check(l, k, score=score, renorm=renorm, bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,k", [(8, 4, 2, 4), (6, 6, 3, 2), (64, 8, 3, 8), (256, 8, 4, 8), (320, 64, 9, 5), (90, 3, 1, 30)])
def test_groups(score, E, groups, top, k):
    l = logits_of(20, E)
    bias = logits_of(1, E, seed=2)[0] * 0.1
    check(l, k, score=score, groups=groups, top_groups=top)
    check(l, k, score=score, groups=groups, top_groups=top, bias=bias, renorm=False, scale=0.5)


def test_ties_go_to_the_lowest_index():
    l = torch.zeros(3, 100, device=gu.DEV)
    l[1, 70:] = 1.0
    l[2] = torch.arange(100, device=gu.DEV) % 3
    for score in ("softmax", "sigmoid"):
        check(l, 8, score=score)
        check(l, 8, score=score, bias=torch.zeros(100, device=gu.DEV))
        check(l, 8, score=score, groups=10, top_groups=4)


def test_experts_that_are_out():
    inf, nan = math.inf, math.nan
    l = logits_of(8, 20)
    l[0] = -inf
    l[1, 2:] = -inf
    l[2, 5] = nan
    l[3] = nan
    l[4, 3] = inf
    l[5, [1, 7]] = inf
    l[6, :10] = -inf
    l[7] = torch.finfo(torch.float32).min
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            check(l, 4, score=score, renorm=renorm)
            check(l, 4, score=score, renorm=renorm, bias=torch.linspace(-0.1, 0.1, 20, device=gu.DEV))
            check(l, 4, score=score, renorm=renorm, groups=2, top_groups=1)
    b = torch.zeros(20, device=gu.DEV)
    b[3], b[4], b[5] = nan, -inf, inf
    w, ids = any4.route(l, 4, bias=b, renorm=False)
    assert not ((ids == 3) | (ids == 4)).any()
    assert (ids[[4, 5, 7], 0] == 5).all()         # a bias of +inf comes first, where its expert is not out
    assert not (ids[[2, 6]] == 5).any() and (ids[[0, 3]] == -1).all() and (w[[0, 3]] == 0).all()


def test_far_logits():
    """Scores that vanish beside the largest: the weights of the chosen stay."""
    l = torch.full((2, 6), -2000.0, device=gu.DEV)
    l[0, 0] = 300.0
    l[1] = torch.tensor([-300.0, -301.0, -302.0, -900.0, -900.0, -900.0])
    bias = torch.tensor([-5.0, 0, 0, 0, 0, 0], device=gu.DEV)
    check(l, 2, bias=bias)
    check(l, 3, score="sigmoid")
    check(l, 3)


def differences(dw, logits, ids, **how):
    """d sum(dw w) / d logits by central differences in 64 bits, the choice constant."""
    score, renorm, scale = how.get("score", "softmax"), how.get("renorm", True), how.get("scale", 1.0)
    l, ids = logits.cpu().double(), ids.cpu().long()
    live = (ids >= 0) & (ids < l.shape[1])

    def value(l):
        v = scores(l, score).gather(1, ids.clamp(0, l.shape[1] - 1)) * live
        if renorm:
            v = v / v.sum(dim=1, keepdim=True)
        return (v * scale * dw.cpu().double() * live).sum(dim=1)
    out, h = torch.zeros_like(l), 2.0 ** -17
    for e in range(l.shape[1]):
        up, down = l.clone(), l.clone()
        up[:, e] += h
        down[:, e] -= h
        out[:, e] = (value(up) - value(down)) / (2 * h)
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 2, 2), (7, 8, 2), (5, 65, 6), (3, 300, 8), (2, 1000, 16)])
def test_route_backward(dtype, score, renorm, T, E, k):
    l = logits_of(T, E, dtype=dtype)
    how = dict(score=score, renorm=renorm, scale=1.5)
    _, ids = any4.route(l, k, **how)
    dw = logits_of(T, k, seed=3)
    got = any4.route_backward(dw, l, ids, **how)
    want = differences(dw, l, ids, **how).to(gu.DEV)
    assert got.dtype == dtype
    # differences: h^2 / 6 times a third derivative below 16 |dw|, and 2^-52 / h of values of up to 10 |dw|
    e = 2.0 ** -31 * dw.abs().sum(dim=1, keepdim=True) + (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23) * want.abs()
    assert ((got.double() - want).abs() <= e).all()


def test_route_backward_of_missing_and_repeated_experts():
    l = logits_of(4, 10)
    l[1, 3] = -math.inf
    ids = torch.tensor([[1, -1, 2], [4, 5, 10], [-1, -1, -1], [7, 8, 9]], dtype=torch.int32, device=gu.DEV)
    dw = logits_of(4, 3, seed=4)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = any4.route_backward(dw, l, ids, score=score, renorm=renorm)
            want = differences(dw, l.clamp(min=-600), ids, score=score, renorm=renorm).to(gu.DEV)
            want[2] = 0
            assert ((got.double() - want).abs() <= 2.0 ** -31 * dw.abs().sum(dim=1, keepdim=True) + 2.0 ** -23 * want.abs()).all()
            assert (got[2] == 0).all()
    twice = torch.tensor([[3, 3]], dtype=torch.int32, device=gu.DEV)
    got = any4.route_backward(dw[:1, :2].contiguous(), l[:1], twice, renorm=False)
    once = any4.route_backward(dw[:1, :2].sum(dim=1, keepdim=True), l[:1], twice[:, :1].contiguous(), renorm=False)
    assert torch.allclose(got, once, rtol=1e-6, atol=0)


def sixteen(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16).to(gu.DEV)


@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 2, 512), (5, 3, 37), (33, 8, 130), (7, 9, 2056), (3, 20, 4099), (200, 2, 256)])
def test_combine(T, k, N):
    y, r, w = sixteen(1, T, k, N), sixteen(2, T, N), logits_of(T, k, seed=5)
    for weights in (w, None):
        for residual in (r, None):
            v = y.double() * (1.0 if weights is None else weights.double()[:, :, None])
            want = v.sum(dim=1) + (0 if residual is None else residual.double())
            mag = v.abs().sum(dim=1) + (0 if residual is None else residual.double().abs())
            e = (k + 1) * 2.0 ** -24 * mag
            out = any4.combine(y, weights, residual=residual)
            assert ((out.double() - want).abs() <= e + 2.0 ** -8 * (want.abs() + e)).all()
    place = r.clone()
    assert any4.combine(y, w, residual=place, out=place) is place
    assert torch.equal(place, any4.combine(y, w, residual=r))


@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 2, 512), (5, 3, 37), (33, 8, 130), (7, 9, 2056), (3, 20, 4099), (200, 2, 256)])
def test_combine_backward(T, k, N):
    y, dout, w = sixteen(1, T, k, N), sixteen(2, T, N), logits_of(T, k, seed=5)
    dy, dw = any4.combine_backward(dout, y, w)
    want = w.double()[:, :, None] * dout.double()[:, None]
    assert ((dy.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -23) * want.abs()).all()
    terms = dout.double()[:, None] * y.double()
    assert ((dw.double() - terms.sum(dim=2)).abs() <= (N + 16) * 2.0 ** -24 * terms.abs().sum(dim=2)).all()
    copy = y.clone()
    again, dw2 = any4.combine_backward(dout, copy, w, dy=copy)
    assert torch.equal(again, dy) and torch.equal(dw2, dw)


def test_empty_calls():
    w, ids = any4.route(logits_of(0, 8), 2)
    assert w.shape == ids.shape == (0, 2)
    assert any4.combine(sixteen(1, 0, 2, 16), w).shape == (0, 16)
    dy, dw = any4.combine_backward(sixteen(1, 3, 0), sixteen(1, 3, 2, 0), logits_of(3, 2))
    assert dy.shape == (3, 2, 0) and (dw == 0).all()
