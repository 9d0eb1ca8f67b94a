"""Low-rank adapters of many requests (lora, lora_plan, lora_backward) against
the formulas in 64 bits.

Tolerances.  Products of bf16 values, and of bf16 values with an fp32 factor
held in three bf16 parts, are exact, so a sum of n terms is off by at most
about n units in the last place of fp32 times the sum of the terms'
magnitudes.  With one further bit for sums that are cut rather than rounded,
    e = 2 * (terms + 16) * 2^-24 * sum of magnitudes,
where the 16 covers the few roundings of factors (a scale, an 8-bit unit).
A bf16 result is rounded once more, by at most 2^-8 of itself."""
import numpy as np
import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


def make(M, K, N, r, L, kind, seed=0):
    g = torch.Generator().manual_seed(seed * 7919 + M * 31 + K + N + r + L)

    def n(*s, std=1.0):
        return (torch.randn(*s, generator=g) * std).to(torch.bfloat16).to(gu.DEV)

    if kind == "runs":
        ids = torch.sort(torch.randint(0, L, (M,), generator=g)).values
    elif kind == "distinct":
        ids = torch.randperm(L, generator=g)[:M]
    else:
        ids = torch.randint(-1, L + 1, (M,), generator=g)     # -1 and L: no adapter
    return {"x": n(M, K), "A": n(L, r, K, std=K ** -0.5), "B": n(L, r, N, std=0.3), "y": n(M, N),
            "scale": (0.5 + torch.rand(L, generator=g)).to(gu.DEV), "ids": ids.to(torch.int32).to(gu.DEV),
            "dy": n(M, N), "dx": n(M, K)}


def gathered(t, ids, L):
    """t[ids] in 64 bits, zeros for rows without an adapter."""
    live = (ids >= 0) & (ids < L)
    out = t.double()[ids.long().clamp(0, L - 1)]
    return torch.where(live.view(-1, *[1] * (out.dim() - 1)), out, torch.zeros((), dtype=torch.float64, device=t.device))


def rows_times(x, W, ids, L, turn):
    """sum over d of x[m][d] W_a[j][d] (or over j with turn), values and magnitudes."""
    out = torch.zeros(x.shape[0], W.shape[2 if turn else 1], dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    for a in range(L):
        at = torch.nonzero(ids == a).flatten()
        if len(at):
            w = W[a].double() if turn else W[a].double().t()
            out[at] = x[at] @ w
            mag[at] = x[at].abs() @ w.abs()
    return out, mag


def forward_ref(t):
    x, ids, L = t["x"].double(), t["ids"], t["A"].shape[0]
    K, r = x.shape[1], t["A"].shape[1]
    h, hmag = rows_times(x, t["A"], ids, L, False)
    s = gathered(t["scale"], ids, L)[:, None]
    d, _ = rows_times(h, t["B"], ids, L, True)
    dmag = rows_times(hmag, t["B"], ids, L, True)[1]
    y = t["y"].double()
    out = y + s * d
    e = 2 * (K + r + 16) * U * (y.abs() + s.abs() * dmag)
    return out, e, h, 2 * (K + 16) * U * hmag


def grads_ref(t, x, h):
    """dx', dA, dB and their tolerances (before a rounding to bf16) from x and h in 64 bits."""
    ids, L, r = t["ids"], t["A"].shape[0], t["A"].shape[1]
    dy = t["dy"].double()
    N, K, M = dy.shape[1], x.shape[1], x.shape[0]
    s = gathered(t["scale"], ids, L)[:, None]
    dh, mag = rows_times(dy, t["B"], ids, L, False)
    dh, mag = dh * s, mag * s.abs()
    part, _ = rows_times(dh, t["A"], ids, L, True)
    dx = t["dx"].double() + part
    edx = 2 * (N + r + 16) * U * (t["dx"].double().abs() + rows_times(mag, t["A"], ids, L, True)[1])
    dA = torch.zeros(t["A"].shape, dtype=torch.float64, device=x.device)
    dB = torch.zeros(t["B"].shape, dtype=torch.float64, device=x.device)
    eA, eB = torch.zeros_like(dA), torch.zeros_like(dB)
    for a in range(L):
        at = torch.nonzero(ids == a).flatten()
        if len(at):
            sa = t["scale"][a].double()
            dA[a] = dh[at].t() @ x[at]
            eA[a] = 2 * (N + M + 16) * U * (mag[at].t() @ x[at].abs())
            dB[a] = sa * (h[at].t() @ dy[at])
            eB[a] = 2 * (M + 16) * U * sa * (h[at].abs().t() @ dy[at].abs())
    return (dx, edx), (dA, eA), (dB, eB)


def assert_near(got, ref, e, what):
    tol = e + (2.0 ** -8) * (ref.abs() + e) if got.dtype == torch.bfloat16 else e + U * ref.abs()
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got.double() - ref).abs() / tol.clamp_min(1e-300)).max()):.3g} of the tolerance"


SHAPES = [
    (1, 128, 1, 1, 1, "runs"), (1, 4096, 4096, 16, 8, "distinct"), (3, 640, 17, 128, 2, "mixed"),
    (16, 128, 33, 8, 32, "distinct"), (17, 256, 130, 3, 4, "mixed"), (64, 512, 512, 8, 1, "runs"),
    (64, 256, 64, 20, 64, "distinct"), (65, 384, 257, 17, 5, "mixed"), (130, 256, 1000, 33, 3, "runs"),
    (200, 128, 64, 128, 2, "mixed"), (513, 256, 129, 16, 1, "runs"), (1100, 128, 520, 64, 4, "mixed"),
    (1537, 384, 200, 65, 2, "runs"), (100, 256, 72, 5, 700, "mixed"), (90, 128, 16, 4, 4096, "distinct"),
    (20000, 128, 24, 4, 3, "mixed"), (17000, 128, 8, 2, 600, "runs"), (256, 256, 40, 16, 1, "runs"),
    (255, 128, 33, 8, 300, "mixed"), (257, 384, 72, 24, 4, "mixed"), (300, 128, 40, 8, 4096, "distinct"),
    (400, 256, 136, 100, 2, "runs"), (500, 128, 24, 4, 63, "mixed"), (500, 128, 24, 4, 64, "mixed"),
    (1500, 128, 27, 4, 65, "runs"), (3300, 256, 30, 40, 2, "mixed"), (5000, 128, 129, 65, 1, "runs"),
    (2, 640, 1100, 113, 60, "distinct"), (64, 1024, 1025, 64, 64, "mixed"), (635, 1152, 1300, 39, 200, "mixed"),
    (3000, 640, 2200, 17, 90, "runs"), (5000, 1024, 4099, 33, 20, "mixed"), (200, 512, 4099, 16, 200, "distinct"),
    (20000, 2048, 2050, 65, 5, "runs"),
]


@pytest.mark.parametrize("M,K,N,r,L,kind", SHAPES)
def test_forward_and_gradients(M, K, N, r, L, kind):
    t = make(M, K, N, r, L, kind)
    h = torch.full((M, r), float("nan"), device=gu.DEV)
    act = any4.act8_empty(t["x"])
    out = any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"], h=h, act=act)
    ref, e, href, he = forward_ref(t)
    assert_near(h, href, he, "h")
    assert_near(out, ref, e, "out")
    none = (t["ids"] < 0) | (t["ids"] >= L)
    assert torch.equal(out[none], t["y"][none])
    assert torch.count_nonzero(h[none]) == 0
    q, qs = any4.act8_save(t["x"])                      # the same codes as the call of its own
    assert torch.equal(q, act[0]) and torch.equal(qs, act[1])

    (dx, edx), (dA, eA), (dB, eB) = grads_ref(t, t["x"].double(), h.double())
    got = any4.lora_backward(t["dy"], t["x"], h, t["A"], t["B"], t["scale"], t["ids"], dx=t["dx"])
    assert_near(got[0], dx, edx, "dx")
    assert torch.equal(got[0][none], t["dx"][none])
    assert_near(got[1], dA, eA, "dA")
    assert_near(got[2], dB, eB, "dB")
    x8 = (q.double().view(M, K // 128, 128) * qs.double()[:, :, None]).view(M, K)
    (_, _), (dA, eA), _ = grads_ref(t, x8, h.double())
    got8 = any4.lora_backward(t["dy"], q, h, t["A"], t["B"], t["scale"], t["ids"], x_scale=qs, need_dx=False)
    assert got8[0] is None
    assert_near(got8[1], dA, eA, "dA from 8 bits")
    assert torch.equal(got8[2], got[2])


@pytest.mark.parametrize("M,L,kind", [(70, 3, "mixed"), (270, 9, "mixed"), (1300, 4, "runs"), (600, 700, "mixed"), (17000, 5, "mixed")])
def test_kept_plan_same_bits(M, L, kind):
    t = make(M, 128, 40, 8, L, kind)
    plan = any4.lora_plan(t["ids"], L)
    h = [torch.empty((M, 8), device=gu.DEV) for _ in range(2)]
    a = any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"], h=h[0])
    b = any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"], h=h[1], plan=plan)
    assert torch.equal(a, b) and torch.equal(h[0], h[1])
    ga = any4.lora_backward(t["dy"], t["x"], h[0], t["A"], t["B"], t["scale"], t["ids"])
    gb = any4.lora_backward(t["dy"], t["x"], h[0], t["A"], t["B"], t["scale"], t["ids"], plan=plan)
    assert all(torch.equal(p, q) for p, q in zip(ga, gb))


@pytest.mark.parametrize("N", [72, 37])
@pytest.mark.parametrize("M", [5, 200, 400])
def test_masked_and_non_finite_values(M, N):
    """A row's NaN or infinity stays in its row; rows without an adapter pass
    y through bit for bit whatever x holds; an unused adapter's weights are
    not read into anything; the gradients of other adapters stay clean."""
    t = make(M, 256, N, 8, 4, "mixed")
    t["ids"] = torch.arange(M, device=gu.DEV, dtype=torch.int32) % 3      # adapter 3 unused
    t["ids"][2] = -1
    clean = any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"])
    t["A"][3] = float("nan")
    t["B"][3] = float("inf")
    t["x"][0, 5] = float("nan")
    t["x"][1, 7] = float("inf")
    t["x"][2] = float("nan")
    t["y"][2, 3] = float("-inf")
    t["y"][2, 4] = float("nan")
    h = torch.empty((M, 8), device=gu.DEV)
    out = any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"], h=h)
    assert torch.isnan(out[0]).all() and not torch.isfinite(out[1]).any()
    assert torch.equal(out[2].view(torch.int16), t["y"][2].view(torch.int16))
    assert torch.count_nonzero(h[2]) == 0
    assert torch.equal(out[3:], clean[3:])
    dx, dA, dB = any4.lora_backward(t["dy"], t["x"], h, t["A"], t["B"], t["scale"], t["ids"], dx=t["dx"])
    assert torch.isfinite(dx).all()                      # dx does not depend on x
    assert torch.isnan(dA[0, :, 5]).all() and torch.isfinite(dA[0, :, 6:]).all()
    assert torch.isfinite(dA[2]).all() and torch.isfinite(dB[2]).all()
    assert torch.count_nonzero(dA[3]) == 0 and torch.count_nonzero(dB[3]) == 0
    # a row of dy reaches its own dx and its adapter's gradients, no neighbour's
    base = any4.lora_backward(t["dy"], t["x"], torch.zeros_like(h), t["A"], t["B"], t["scale"], t["ids"], dx=t["dx"])
    t["dy"][3] = float("nan")            # adapter 0
    got = any4.lora_backward(t["dy"], t["x"], torch.zeros_like(h), t["A"], t["B"], t["scale"], t["ids"], dx=t["dx"])
    keep = torch.arange(M, device=gu.DEV) != 3
    assert torch.isnan(got[0][3]).all() and torch.equal(got[0][keep], base[0][keep])
    assert torch.equal(got[1][2], base[1][2]) and torch.equal(got[2][1:], base[2][1:])


@pytest.mark.parametrize("M", [9, 150, 350])
def test_no_row_has_an_adapter(M):
    t = make(M, 128, 50, 4, 2, "mixed")
    t["ids"].fill_(-1)
    h = torch.full((M, 4), float("nan"), device=gu.DEV)
    out = any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"], h=h)
    assert torch.equal(out, t["y"]) and torch.count_nonzero(h) == 0
    dx, dA, dB = any4.lora_backward(t["dy"], t["x"], h, t["A"], t["B"], t["scale"], t["ids"])
    assert not dx.any() and not dA.any() and not dB.any()


@pytest.mark.parametrize("M", [1, 48, 300])
def test_in_place_and_buffers_of_the_caller(M):
    t = make(M, 256, 100, 12, 3, "mixed")
    ref = any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"])
    y = t["y"].clone()
    ws = torch.full((any4.lora_workspace_size(M, 100, 256, 12, 3),), 255, dtype=torch.uint8, device=gu.DEV)
    assert any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], y, out=y, workspace=ws) is y
    assert torch.equal(y, ref)
    h = torch.randn((M, 12), device=gu.DEV)
    a = any4.lora_backward(t["dy"], t["x"], h, t["A"], t["B"], t["scale"], t["ids"], dx=t["dx"])
    dx, dA, dB = t["dx"].clone(), torch.full_like(a[1], 7), torch.full_like(a[2], 7)
    ws = torch.full((any4.lora_backward_workspace_size(M, 100, 256, 12, 3),), 255, dtype=torch.uint8, device=gu.DEV)
    b = any4.lora_backward(t["dy"], t["x"], h, t["A"], t["B"], t["scale"], t["ids"], dx=dx, out=dx, dA=dA, dB=dB, workspace=ws)
    assert b[0] is dx and all(torch.equal(p, q) for p, q in zip(a, b))


def test_unaligned_and_odd_rows():
    """y, out, dy and B at addresses that only their elements align."""
    M, K, N, r, L = 70, 128, 37, 6, 3
    t = make(M, K, N, r, L, "mixed")
    ref = any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"])

    def shifted(v):
        room = torch.zeros(v.numel() + 9, dtype=v.dtype, device=v.device)
        room[1:1 + v.numel()] = v.flatten()
        return room, room[1:1 + v.numel()].view(v.shape)

    _, B = shifted(t["B"])
    _, y = shifted(t["y"])
    room, out = shifted(torch.zeros_like(t["y"]))
    any4.lora(t["x"], t["A"], B, t["scale"], t["ids"], y, out=out)
    assert torch.equal(out, ref)
    assert not room[0].any() and not room[1 + M * N:].any()      # nothing written around it


def test_empty_batch_and_no_outputs():
    t = make(4, 128, 16, 2, 1, "runs")
    e = torch.empty((0, 128), dtype=torch.bfloat16, device=gu.DEV)
    out = any4.lora(e, t["A"], t["B"], t["scale"], t["ids"][:0], torch.empty((0, 16), dtype=torch.bfloat16, device=gu.DEV))
    assert out.shape == (0, 16)
    dx, dA, dB = any4.lora_backward(t["dy"][:0], e, torch.empty((0, 2), device=gu.DEV), t["A"], t["B"], t["scale"], t["ids"][:0],
                                    dA=torch.full((1, 2, 128), 3.0, device=gu.DEV))
    assert dx.shape == (0, 128) and not dA.any() and not dB.any()
    for M in (4, 80):
        t = make(M, 128, 16, 2, 1, "runs")
        h, act = torch.empty((M, 2), device=gu.DEV), any4.act8_empty(t["x"])
        any4.lora(t["x"], t["A"], t["B"][:, :, :0].contiguous(), t["scale"], t["ids"],
                  torch.empty((M, 0), dtype=torch.bfloat16, device=gu.DEV), h=h, act=act)
        _, _, href, he = forward_ref(t)
        assert_near(h, href, he, "h")
        assert torch.equal(act[0], any4.act8_save(t["x"])[0])


@pytest.mark.parametrize("M,L", [(20, 4), (700, 3)])
def test_gradients_against_differences(M, L):
    """<gradient, direction> against central differences of the loss
    sum(dy * out) in 64 bits; the loss is linear in A, in B and in x alone, so
    the differences are exact but for their own rounding."""
    t = make(M, 256, 90, 8, L, "mixed")
    h = torch.empty((M, 8), device=gu.DEV)
    any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"], h=h)
    dx, dA, dB = any4.lora_backward(t["dy"], t["x"], h, t["A"], t["B"], t["scale"], t["ids"])
    ids = t["ids"]

    def loss(x, A, B):
        hh, _ = rows_times(x, A, ids, L, False)
        d, _ = rows_times(hh * gathered(t["scale"], ids, L)[:, None], B, ids, L, True)
        return float((t["dy"].double() * (t["y"].double() + d)).sum())

    at = [t["x"].double(), t["A"].double(), t["B"].double()]
    g = torch.Generator(device=gu.DEV).manual_seed(3)
    for i, grad in enumerate((dx, dA, dB)):
        v = torch.randn(at[i].shape, generator=g, device=gu.DEV, dtype=torch.float64)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + 0.5 * v, at[i] - 0.5 * v
        # each term of the sum is off by at most 2^-8 (bf16) or the fp32 bound of
        # the other tests, taken here as 2^-13 of the sum of magnitudes
        rel = 2.0 ** -8 if grad.dtype == torch.bfloat16 else 2.0 ** -13
        tol = rel * float((grad.double() * v).abs().sum()) + 1e-6
        assert abs(loss(*up) - loss(*down) - float((grad.double() * v).sum())) <= tol


@pytest.mark.parametrize("M", [7, 300])
def test_captured_and_replayed(M):
    """A training pass in a graph, two graphs of it replayed on two streams at
    once, eager passes between the replays: every result is the eager one."""
    L, r, K, N = 3, 8, 256, 136
    t = make(M, K, N, r, L, "mixed")
    t2 = make(M, K, N, r, L, "mixed", seed=1)

    def step(t):
        h, act = torch.empty((M, r), device=gu.DEV), any4.act8_empty(t["x"])
        out = any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"], h=h, act=act)
        return (out, h) + any4.lora_backward(t["dy"], act[0], h, t["A"], t["B"], t["scale"], t["ids"], dx=t["dx"],
                                             x_scale=act[1])

    refs = [[v.clone() for v in step(t)], [v.clone() for v in step(t2)]]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for tt, s in zip((t, t2), streams):
        s.wait_stream(torch.cuda.current_stream())
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            outs.append(step(tt))
        graphs.append(gr)
    torch.cuda.synchronize()
    for _ in range(3):
        for o in outs:
            for v in o:
                v.fill_(float("nan"))
        torch.cuda.synchronize()
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        eager = step(t2)
        torch.cuda.synchronize()
        for ref, o in zip(refs, outs):
            assert all(torch.equal(a, b) for a, b in zip(ref, o))
        assert all(torch.equal(a, b) for a, b in zip(refs[1], eager))


def test_on_another_stream():
    t = make(300, 256, 136, 8, 3, "mixed")
    ref = any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"], stream=v)
            for v in (s, s.cuda_stream, torch.cuda.default_stream(), 0)]
    torch.cuda.synchronize()
    assert all(torch.equal(ref, o) for o in outs)


def test_refusals():
    t = make(8, 128, 16, 4, 2, "mixed")
    a = dict(x=t["x"], A=t["A"], B=t["B"], scale=t["scale"], ids=t["ids"], y=t["y"])

    def refused(kind, **change):
        with pytest.raises(kind):
            any4.lora(**{**a, **change})

    refused(TypeError, x=t["x"].float())
    refused(TypeError, ids=t["ids"].long())
    refused(TypeError, scale=t["scale"].double())
    refused(ValueError, x=t["x"].cpu())
    refused(ValueError, y=t["y"].t().contiguous().t())
    refused(ValueError, A=t["A"][0])
    refused(ValueError, A=t["A"][:, :3].contiguous())
    refused(ValueError, ids=t["ids"][:7])
    refused(ValueError, h=torch.empty((8, 5), device=gu.DEV))
    refused(ValueError, workspace=torch.empty(64, dtype=torch.uint8))
    more = {k: v for k, v in make(80, 128, 16, 4, 2, "mixed").items() if k in a}
    refused(RuntimeError, workspace=torch.empty(64, dtype=torch.uint8, device=gu.DEV), **more)
    refused(TypeError, plan=torch.empty(64, dtype=torch.int32, device=gu.DEV))
    refused(ValueError, plan=any4.lora_plan(t["ids"], 3))
    refused(RuntimeError, x=t["x"][:, :64].contiguous(), A=t["A"][:, :, :64].contiguous())   # K % 128
    wide = torch.zeros((2, 129, 128), dtype=torch.bfloat16, device=gu.DEV)
    refused(RuntimeError, A=wide, B=torch.zeros((2, 129, 16), dtype=torch.bfloat16, device=gu.DEV))   # r > 128
    h = torch.empty((8, 4), device=gu.DEV)
    with pytest.raises(TypeError):
        any4.lora_backward(t["dy"], t["x"], h, t["A"], t["B"], t["scale"], t["ids"], x_scale=torch.ones((8, 1), device=gu.DEV))
    with pytest.raises(ValueError):
        any4.lora_backward(t["dy"], t["x"][:4], h, t["A"], t["B"], t["scale"], t["ids"])
