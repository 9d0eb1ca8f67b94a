"""The erf GELU and its slope keep their relative accuracy for negative arguments, where
1 + erf cancels.

Bounds, with t = -z / sqrt(2): t is off by 2^-23 of itself (a rounded constant, a rounded product),
which erfc passes on as at most (2 t + 1 / t) t = 2 t^2 + 1 times as much; erfc itself is off by at most
16 steps of 2^-23, its product with z / 2 by 2^-23.  exp(-z^2 / 2) is off by 2^-24 z^2 / 2 for its rounded
argument and a few steps, 2^-20 with the factors."""
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


def tail():
    z = torch.linspace(-9, -3, 3000).to(torch.bfloat16).unique().to(gu.DEV)
    d = z.double()
    p = torch.special.ndtr(d)
    assert (p * 2 - torch.special.erfc(-d / math.sqrt(2))).abs().max() < 1e-15
    p = 0.5 * torch.special.erfc(-d / math.sqrt(2))
    return z, d, p, p * (2.0 ** -23 * (d * d + 1) + 2.0 ** -19 + 2.0 ** -22)


def identity():
    """W [16, 128]: all ones, so that z is a row's one value."""
    one = lambda v: torch.full((16, 1), v, dtype=torch.bfloat16, device=gu.DEV)      # noqa: E731
    packed = any4.pack(torch.zeros((16, 128), dtype=torch.uint8, device=gu.DEV))
    return packed, torch.ones((16, 16), dtype=torch.bfloat16, device=gu.DEV), one(1.0), one(0.0)


def test_forward():
    z, d, p, ep = tail()
    x = torch.zeros((z.numel(), 128), dtype=torch.bfloat16, device=gu.DEV)
    x[:, 5] = z
    want = d * p
    for rows in (slice(0, 7), slice(None)):         # few rows, tiles
        out = torch.empty(x[rows].shape[0], 16, device=gu.DEV)
        any4.gemm_act(x[rows].contiguous(), *identity(), 128, act="gelu", out=out)
        err = (out.double() - want[rows, None]).abs()
        assert (err <= (d.abs() * ep)[rows, None]).all(), (err / want[rows, None].abs()).max().item()
    half = any4.gemm_act(x, *identity(), 128, act="gelu")
    assert ((half.double() - want[:, None]).abs() <= (2.0 ** -8 * want.abs() + 1.01 * d.abs() * ep)[:, None]).all()


def test_gated_forward_and_backward():
    z, d, p, ep = tail()
    n = z.numel()
    gated = torch.cat([z, torch.full_like(z, 0.5)]).view(1, 2 * n)
    dy = torch.ones(1, n, dtype=torch.bfloat16, device=gu.DEV)
    _, dbias = any4.act_backward(dy, gated, "gelu", gate=True)       # one row: dz before it is rounded
    phi = torch.exp(-d * d / 2) / math.sqrt(2 * math.pi)
    slope, e = p + d * phi, ep + (d * phi).abs() * (2.0 ** -25 * d * d + 2.0 ** -20)
    assert ((dbias[:n].double() - 0.5 * slope).abs() <= 0.5 * e + 2.0 ** -23 * slope.abs()).all()
    assert ((dbias[n:].double() - d * p).abs() <= d.abs() * ep + 2.0 ** -23 * (d * p).abs()).all()


def test_backward():
    z, d, p, ep = tail()
    _, dbias = any4.act_backward(torch.ones_like(z)[None], z[None], "gelu")
    phi = torch.exp(-d * d / 2) / math.sqrt(2 * math.pi)
    slope, e = p + d * phi, ep + (d * phi).abs() * (2.0 ** -25 * d * d + 2.0 ** -20)
    assert ((dbias.double() - slope).abs() <= e + 2.0 ** -23 * slope.abs()).all()


def test_positive_and_far_arguments():
    """The right side is that of before; beyond the tail 0, never NaN."""
    z = torch.tensor([0.0, 0.5, 3.0, 9.0, 30.0, 3e38, -14.0, -30.0, -1e4, -3e38], device=gu.DEV).to(torch.bfloat16)
    x = torch.zeros((z.numel(), 128), dtype=torch.bfloat16, device=gu.DEV)
    x[:, 5] = z
    out = torch.empty(z.numel(), 16, device=gu.DEV)
    any4.gemm_act(x, *identity(), 128, act="gelu", out=out)
    want = z.double() * 0.5 * torch.special.erfc(-z.double() / math.sqrt(2))
    assert ((out.double() - want[:, None]).abs() <= 2.0 ** -21 * want.abs()[:, None] + 2.0 ** -120).all()
    _, dbias = any4.act_backward(torch.ones_like(z)[None], z[None], "gelu")
    assert torch.isfinite(dbias).all() and (dbias[-3:].abs() < 1e-30).all() and (dbias[4:6] == 1).all()
