"""Infinite and NaN values of the data in the adapter calls: h, out and dx hold
what the formulas give for them, in every form of the kernels, also where the
rank is not a whole number of blocks.

The formulas are evaluated in 64 bits on the CPU, product by product, so that
nothing but the terms of a sum enters it.  Which results are NaN and which are
infinite (and of which sign) has to agree; the finite ones are held to the
bounds of the other adapter tests."""
import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu
from tests.test_gpu_lora import assert_near, forward_ref, grads_ref, make

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


def same_kind(got, ref, what):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN elsewhere"
    wild = torch.isinf(got) | torch.isinf(ref)
    assert torch.equal(got[wild], ref[wild]), f"{what}: infinities differ"


def products(x, W, s=None):
    """sum over d of x[d] W[j][d] for one row, one product at a time."""
    p = (x[None, :] * W).sum(dim=1)
    return p if s is None else p * s


# (M, K, r, L): one launch; two launches of few rows (ranks above 64, long rows);
# ballots beyond 64 rows; planned, with one tile and more an adapter; chunks
FORMS = [(5, 256, 1, 2), (20, 256, 40, 3), (40, 256, 100, 3), (33, 128 * 41, 13, 3), (150, 384, 1, 3), (150, 384, 20, 3),
         (100, 256, 1, 12), (300, 256, 5, 9), (300, 256, 17, 3), (300, 256, 33, 3), (300, 128, 127, 3), (700, 128, 1, 1)]


@pytest.mark.parametrize("N", [72, 37])
@pytest.mark.parametrize("M,K,r,L", FORMS)
def test_infinite_data(M, K, r, L, N):
    t = make(M, K, N, r, L, "mixed")
    t["ids"] = torch.arange(M, device=gu.DEV, dtype=torch.int32) % L
    bad = {0: INF, 1: -INF, 2: float("nan"), M - 1: INF}
    for i, (m, v) in enumerate(bad.items()):
        t["x"][m, (7 + 50 * i) % K] = v
        t["dy"][m, (5 + 9 * i) % N] = v
    h = torch.empty((M, r), device=gu.DEV)
    out = any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"], h=h)
    dx = any4.lora_backward(t["dy"], t["x"], h, t["A"], t["B"], t["scale"], t["ids"], dx=t["dx"])[0]

    c = {k: v.cpu().double() for k, v in t.items() if k != "ids"}
    some_infinite = 0
    for m in bad:
        a = m % L
        hm = products(c["x"][m], c["A"][a])
        same_kind(h[m], hm, f"h of row {m}")
        ym = c["y"][m] + c["scale"][a] * products(hm, c["B"][a].t())
        same_kind(out[m], ym, f"out of row {m}")
        dh = products(c["dy"][m], c["B"][a], c["scale"][a])
        dm = c["dx"][m] + products(dh, c["A"][a].t())
        same_kind(dx[m], dm, f"dx of row {m}")
        some_infinite += int(torch.isinf(ym).sum() + torch.isinf(dm).sum())
    if r == 1:
        assert some_infinite == 3 * (N + K)        # all of the three rows with an infinity

    # the other rows are as if there were no such values
    good = torch.ones(M, dtype=torch.bool, device=gu.DEV)
    good[list(bad)] = False
    for m in bad:
        t["x"][m] = 0
        t["dy"][m] = 0
    ref, e, href, he = forward_ref(t)
    assert_near(h[good], href[good], he[good], "h")
    assert_near(out[good], ref[good], e[good], "out")
    (rdx, edx), _, _ = grads_ref(t, t["x"].double(), href)
    assert_near(dx[good], rdx[good], edx[good], "dx")


@pytest.mark.parametrize("M,K,r,L", [(5, 256, 3, 2), (40, 256, 100, 2), (300, 256, 5, 3)])
def test_infinite_scale(M, K, r, L):
    """Positive weights and data, an infinite scale: infinities throughout, also
    where ranks behind the last stand beside the others."""
    t = make(M, K, 40, r, L, "runs")
    for k in ("x", "A", "B", "dy", "scale"):
        t[k] = t[k].abs() + 0.125
    t["scale"][0] = INF
    t["ids"][0] = 0
    h = torch.empty((M, r), device=gu.DEV)
    out = any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"], h=h)
    dx = any4.lora_backward(t["dy"], t["x"], h, t["A"], t["B"], t["scale"], t["ids"], dx=t["dx"])[0]
    hit = t["ids"] == 0
    assert torch.isfinite(h).all()
    assert (out[hit] == INF).all() and (dx[hit] == INF).all()
    assert torch.isfinite(out[~hit]).all() and torch.isfinite(dx[~hit]).all()
