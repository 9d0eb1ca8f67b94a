"""The gradient of a quantised layer's input against the product in 64 bits
with the oracle's weights.

Products of bf16 values are exact; the fp32 sum of N terms is off by at most
2 * (N + 16) * 2^-24 of the sum of magnitudes (one bit for sums that are cut
rather than rounded), the result's rounding to bf16 by 2^-8 of itself."""
import numpy as np
import pytest
import torch

import gemm_any4_amd as any4
import oracle
import workloads
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


def layer(fmt, N, K, g, seed=5):
    """(call, weights in 64 bits on the GPU) of a layer in a format."""
    inp = workloads.generic(seed, 1, N, K, g)
    al, be, lut = gu.dev_b16(inp.alpha), gu.dev_b16(inp.beta), gu.dev_b16(inp.lut)
    if fmt == "any2":
        codes = (inp.idx & 3).astype(np.uint8)
        packed = gu.dev_u8(oracle.tile2(oracle.pack2(codes)))
    elif fmt == "any3":
        codes = (inp.idx & 7).astype(np.uint8)
        packed = gu.dev_u8(oracle.tile3(codes))
    else:
        codes = inp.idx
        packed = gu.dev_u8(oracle.tile(oracle.pack(codes)))
    table = inp.lut
    if fmt == "int4":
        table = np.broadcast_to(oracle.f32_to_bf16(np.arange(16, dtype=np.float32)), (N, 16)).copy()
    w = oracle.dequant(oracle.pack(codes), table, inp.alpha, inp.beta, g)
    w = gu.dev_b16(w).double()
    if fmt == "int4":
        return lambda dy, **k: any4.gemm_int4_dx(dy, packed, al, be, g, **k), w
    call = {"any4": any4.gemm_dx, "any2": any4.any2_gemm_dx, "any3": any4.any3_gemm_dx}[fmt]
    return lambda dy, **k: call(dy, packed, lut, al, be, g, **k), w


def grad(M, N, seed=1):
    g = torch.Generator().manual_seed(seed * 1000 + M + N)
    return torch.randn((M, N), generator=g).to(torch.bfloat16).to(gu.DEV)


def check(dx, dy, w):
    d = dy.double()
    ref, mag = d @ w, d.abs() @ w.abs()
    e = 2 * (w.shape[0] + 16) * 2.0 ** -24 * mag
    bad = ~((dx.double() - ref).abs() <= e + 2.0 ** -8 * (ref.abs() + e))
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off"


@pytest.mark.parametrize("fmt", ["any4", "int4", "any2", "any3"])
@pytest.mark.parametrize("M,N,K,g", [(1, 1, 128, 128), (1, 64, 256, 256), (5, 37, 384, 128), (64, 128, 256, 128),
                                     (16, 1000, 256, 128), (100, 333, 384, 384), (129, 200, 512, 512),
                                     (300, 1000, 128, 128), (290, 200, 512, 512), (257, 1, 128, 128)])
def test_formats_and_odd_sizes(fmt, M, N, K, g):
    call, w = layer(fmt, N, K, g)
    dy = grad(M, N)
    check(call(dy), dy, w)


@pytest.mark.parametrize("M,N,K,g", [(16, 4096, 4096, 128), (64, 4099, 1024, 1024), (1000, 2048, 1152, 128),
                                     (513, 1024, 4096, 512), (1, 14336, 512, 128), (3001, 200, 4096, 128),
                                     (2999, 333, 4352, 256), (128, 4100, 2048, 256), (17, 1000, 14336, 1024),
                                     (2000, 8200, 2048, 256), (129, 4096, 1024, 128),
                                     (193, 4099, 4096, 128), (256, 14336, 512, 128), (260, 4096, 1024, 128),
                                     (600, 14336, 2048, 128), (1500, 4100, 4096, 4096), (2500, 8192, 2304, 256)])
def test_larger_sizes(M, N, K, g):
    """Sums split over workgroups, ragged last tiles, padded copies of dy, both
    tile sizes and the form for few rows."""
    call, w = layer("any4", N, K, g)
    dy = grad(M, N)
    check(call(dy), dy, w)


@pytest.mark.parametrize("fmt", ["any4", "int4", "any2", "any3"])
@pytest.mark.parametrize("N", [100, 190, 300])
def test_one_hot_rows_give_the_weights(fmt, N):
    """dy = unit vectors: dx is W itself, bit for bit."""
    call, w = layer(fmt, N, 256, 128)
    dy = torch.eye(N, dtype=torch.bfloat16, device=gu.DEV)
    assert torch.equal(call(dy).double(), w)


@pytest.mark.parametrize("M", [20, 140, 270])
@pytest.mark.parametrize("N", [64, 100])
def test_rows_do_not_touch_each_other(M, N):
    """NaN and infinities in one row of dy, also behind an odd row's end."""
    call, w = layer("any4", N, 256, 128)
    dy = grad(M, N)
    clean = call(dy)
    dy[7] = float("nan")
    dy[M - 1, 3] = float("inf")
    got = call(dy)
    keep = torch.ones(M, dtype=torch.bool, device=gu.DEV)
    keep[7] = keep[M - 1] = False
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[7]).all() and not torch.isfinite(got[M - 1]).any()


@pytest.mark.parametrize("fmt", ["any4", "any2", "any3"])
@pytest.mark.parametrize("M", [3, 150, 300])
def test_table_values_of_every_kind(fmt, M):
    """Negative zeros, subnormals, infinities and NaN in a row's table come out
    as any4_dequant writes them."""
    call, w = layer(fmt, 48, 256, 128)
    inp = workloads.generic(5, 1, 48, 256, 128)
    lut = gu.dev_b16(inp.lut)
    lut[0, :4] = torch.tensor([-0.0, 1e-40, float("inf"), float("nan")], device=gu.DEV)
    al, be = gu.dev_b16(inp.alpha), gu.dev_b16(inp.beta)
    be[0] = 0
    if fmt == "any4":
        packed = gu.dev_u8(oracle.tile(oracle.pack(inp.idx)))
        ref, got = any4.dequant(packed, lut, al, be, 128), None
        run = lambda dy: any4.gemm_dx(dy, packed, lut, al, be, 128)  # noqa: E731
    else:
        codes = (inp.idx & (3 if fmt == "any2" else 7)).astype(np.uint8)
        packed = gu.dev_u8(oracle.tile2(oracle.pack2(codes)) if fmt == "any2" else oracle.tile3(codes))
        ref = (any4.any2_dequant if fmt == "any2" else any4.any3_dequant)(packed, lut, al, be, 128)
        run = lambda dy: (any4.any2_gemm_dx if fmt == "any2" else any4.any3_gemm_dx)(dy, packed, lut, al, be, 128)  # noqa: E731
    dy = torch.zeros((M, 48), dtype=torch.bfloat16, device=gu.DEV)
    dy[0, 0] = 1.0
    dy[1:, 1] = 1.0
    got = run(dy)
    want = ref[0].float() + 0.0             # a sum with zeros: -0 becomes 0
    same = (got[0].float() == want) | (torch.isnan(got[0]) & torch.isnan(want))
    # a zero times an infinity or NaN of row 0 reaches the other rows' sums
    assert same.all() and torch.isfinite(got[1:, torch.isfinite(ref[0])]).all()


@pytest.mark.parametrize("M", [70, 300])
def test_unaligned_rows_and_caller_buffers(M):
    call, w = layer("any4", 128, 256, 128)
    dy = grad(M, 128)
    ref = call(dy)
    room = torch.zeros(M * 128 + 8, dtype=torch.bfloat16, device=gu.DEV)
    room[1:1 + M * 128] = dy.flatten()
    out = torch.empty_like(ref)
    ws = torch.full((any4.gemm_dx_workspace_size(M, 128, 256, 128),), 255, dtype=torch.uint8, device=gu.DEV)
    assert call(room[1:1 + M * 128].view(M, 128), out=out, workspace=ws) is out
    assert torch.equal(out, ref)


def test_empty_sizes():
    call, _ = layer("any4", 64, 256, 128)
    assert call(grad(1, 64)[:0]).shape == (0, 256)
    e = torch.empty((0, 2), dtype=torch.bfloat16, device=gu.DEV)
    dx = any4.gemm_dx(torch.empty((3, 0), dtype=torch.bfloat16, device=gu.DEV),
                      torch.empty(0, dtype=torch.uint8, device=gu.DEV),
                      torch.empty((0, 16), dtype=torch.bfloat16, device=gu.DEV), e, e, 128)
    assert dx.shape == (3, 256) and not dx.any()


@pytest.mark.parametrize("M,N", [(40, 192), (40, 100), (300, 192), (300, 100)])
def test_captured_and_replayed(M, N):
    call, _ = layer("any4", N, 512, 128)
    dy = grad(M, N)
    ref = call(dy).clone()
    torch.cuda.synchronize()
    s, gr = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(gr, stream=s):
        out = call(dy)
    torch.cuda.synchronize()
    for _ in range(3):
        out.fill_(float("nan"))
        eager = call(dy)
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(eager, ref)


def test_refusals():
    inp = workloads.generic(5, 1, 64, 256, 128)
    a = [grad(4, 64), gu.dev_u8(oracle.tile(oracle.pack(inp.idx))), gu.dev_b16(inp.lut), gu.dev_b16(inp.alpha),
         gu.dev_b16(inp.beta), 128]

    def refused(kind, at, v):
        with pytest.raises(kind):
            any4.gemm_dx(*a[:at], v, *a[at + 1:])

    refused(TypeError, 0, a[0].float())
    refused(ValueError, 0, a[0].cpu())
    refused(ValueError, 0, grad(4, 63))
    refused(ValueError, 1, a[1][:-1].contiguous())
    refused(ValueError, 3, a[3][:, :1].contiguous())
    refused(ValueError, 5, 0)
    refused(ValueError, 5, 64)           # another K than the packed tiles'
    with pytest.raises(RuntimeError):
        any4.gemm_dx(*a, workspace=torch.empty(16, dtype=torch.uint8, device=gu.DEV))
