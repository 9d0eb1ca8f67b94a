"""The adapter, 8-bit activation and input-gradient calls at the ends of the
ranges that their documentation gives: the most rows, the widest rows, tensors
just below 2 GiB.

All values are whole numbers of small magnitude (and a scale of one half), so
that every product and every partial sum in any order is exact in fp32: the
sums of n random signs stay far below 2^23 halves.  Results are compared bit
for bit, after the one rounding to bf16 where there is one."""
import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


def signs(gen, *shape):
    return torch.randint(-1, 2, shape, generator=gen, device=gu.DEV, dtype=torch.int8).to(torch.bfloat16)


def times(x, w):
    """x w in 64 bits, a block of rows at a time."""
    w = w.double()
    return torch.cat([b.double() @ w for b in x.split(max(1, 2 ** 28 // max(x.shape[1], 1)))])


def turned_times(x, z):
    """x^T z in 64 bits, summed over blocks of rows."""
    step = max(1, 2 ** 28 // max(x.shape[1], z.shape[1]))
    return sum(a.double().t() @ b.double() for a, b in zip(x.split(step), z.split(step)))


@pytest.mark.parametrize("M,K,N,r,L", [
    (2 ** 20, 128, 8, 1, 4096),         # the most rows and adapters
    (2 ** 20, 896, 72, 128, 3),         # and the highest rank
    (262143, 4096, 40, 8, 5),           # x just below 2 GiB
    (262143, 128, 4095, 8, 5),          # y too, in odd rows
    (3, 128, 2 ** 24, 1, 1),            # the widest rows, in one launch
    (100, 128, 2 ** 23 + 1, 2, 3),      # wide odd rows
    (60, 2 ** 24, 8, 1, 1),
    (70, 2 ** 23, 8, 2, 2),
])
def test_adapters(M, K, N, r, L):
    gen = torch.Generator(gu.DEV).manual_seed(M + K + N)
    x, A, B, y = signs(gen, M, K), signs(gen, L, r, K), signs(gen, L, r, N), signs(gen, M, N)
    dy, dx = signs(gen, M, N), signs(gen, M, K)
    scale = torch.full((L,), 0.5, device=gu.DEV)
    ids = torch.randint(-1, L, (M,), generator=gen, device=gu.DEV, dtype=torch.int32)
    h = torch.empty((M, r), device=gu.DEV)
    act = any4.act8_empty(x)
    out = any4.lora(x, A, B, scale, ids, y, h=h, act=act)
    got = any4.lora_backward(dy, x, h, A, B, scale, ids, dx=dx)
    some = range(L) if L < 10 else (0, 1, L // 2, L - 1)      # (all rows are checked below 10 adapters)
    for a in some:
        at = torch.nonzero(ids == a).flatten()
        xa, dya = x[at], dy[at]
        ha = times(xa, A[a].t())
        assert torch.equal(h[at].double(), ha)
        dha = times(dya, B[a].t()) * 0.5
        assert torch.equal(got[1][a].double(), turned_times(dha, xa))
        assert torch.equal(got[2][a].double(), turned_times(ha, dya) * 0.5)
        for rows in torch.arange(len(at), device=gu.DEV).split(max(1, 2 ** 28 // max(K, N))):
            o = y[at[rows]].double() + 0.5 * (ha[rows] @ B[a].double())
            assert torch.equal(out[at[rows]], o.to(torch.bfloat16))
            o = dx[at[rows]].double() + dha[rows] @ A[a].double()
            assert torch.equal(got[0][at[rows]], o.to(torch.bfloat16))
    none = torch.nonzero(ids < 0).flatten()
    assert torch.equal(out[none], y[none]) and torch.equal(got[0][none], dx[none])
    # every group of 128 channels of a row holds a 1 or -1, bar one in 3^128
    assert torch.equal(act[0], x.to(torch.int8) * 127)
    assert (act[1] == torch.tensor(1 / 127, dtype=torch.float64).float().item()).all()


@pytest.mark.parametrize("M,K", [(262143, 4096), (65535 * 64, 128), (1, 2 ** 29)])
def test_act8(M, K):
    gen = torch.Generator(gu.DEV).manual_seed(M)
    x = torch.randn((M, K), generator=gen, device=gu.DEV, dtype=torch.bfloat16)
    q, qs = any4.act8_save(x)
    back = any4.act8_load(q, qs)
    groups = x.view(-1, 128)[-5000:].contiguous()         # the last ones as a call of their own
    q1, qs1 = any4.act8_save(groups)
    assert torch.equal(q.view(-1, 128)[-5000:], q1) and torch.equal(qs.view(-1, 1)[-5000:], qs1)
    assert torch.equal(back.view(-1, 128)[-5000:], any4.act8_load(q1, qs1))
    # and all of it: off by half a step and the roundings of the scale, the code and the value
    for b, v, s in zip(x.view(-1, 128).split(2 ** 21), back.view(-1, 128).split(2 ** 21), qs.view(-1, 1).split(2 ** 21)):
        e = s * (0.5 + 127 * 4 * 2.0 ** -24)
        assert ((b.float() - v.float()).abs() <= e + 2.0 ** -8 * (b.float().abs() + e)).all()


@pytest.mark.parametrize("M,N,K,g", [
    (3, 2 ** 21, 128, 128), (200, 2 ** 21 - 3, 128, 128), (300, 2 ** 21 - 3, 128, 128),      # the longest sums
    (262143, 64, 4096, 4096),                                  # dx just below 2 GiB
    (262143, 4095, 256, 128),                                  # dy, through its padded copy
    (1, 5, 2 ** 27, 256), (129, 1, 2 ** 22, 2 ** 22), (257, 1, 2 ** 21, 2 ** 21),          # the widest rows
    (65535 * 64, 17, 128, 128),                                # the most rows
])
def test_input_gradient(M, N, K, g):
    gen = torch.Generator(gu.DEV).manual_seed(M + N)
    packed = torch.randint(0, 256, (any4.packed_bytes(N, K),), generator=gen, device=gu.DEV, dtype=torch.uint8)
    lut = torch.randint(-2, 3, (N, 16), generator=gen, device=gu.DEV).to(torch.bfloat16)
    alpha = torch.ones((N, K // g), device=gu.DEV, dtype=torch.bfloat16)
    beta = torch.zeros_like(alpha)
    dy = signs(gen, M, N)
    dx = any4.gemm_dx(dy, packed, lut, alpha, beta, g)
    w = any4.dequant(packed, lut, alpha, beta, g)
    for rows in torch.arange(M, device=gu.DEV).split(max(1, 2 ** 28 // max(K, N))):
        assert torch.equal(dx[rows], (dy[rows].double() @ w.double()).to(torch.bfloat16))
