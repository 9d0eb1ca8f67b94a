"""Rows of the experts' products in two bf16 parts: the results of one product as the
next one takes them, for any number of pairs; against the formulas in 64 bits with the
oracle's weights.

Tolerances are those of test_gpu_ffn.py.  A row in parts is the sum of two bf16 rows, so that a
sum over K has 2 K terms: twice the bound.  Parts are the value but for 2^-16 of it: what is
left of a value in [2^e, 2^(e+1)) once it is cut to 8 bits is below 2^(e-7), and half a step of
bf16 there is 2^(e-16)."""
import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu
from tests.test_gpu_ffn import call_of, choose, close, each_expert, expect, layers, normal
from tests.test_gpu_ffn_block import Block, empty, near

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


def in_parts(v):
    """fp32 values as [2, ..]: cut to bf16, and the rounded rest."""
    hi = (v.contiguous().view(torch.int32) & -65536).view(F32)
    rest = torch.where(torch.isinf(v), torch.zeros_like(v), v - hi)
    return torch.stack([hi.to(BF16), rest.to(BF16)])


def whole(p):
    return p[0].double() + p[1].double()


def rows(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(gu.DEV)


# few rows and tiles of three heights, with split sums and without
SIZES = [(1, 1, 1, 1, 128), (1, 2, 8, 96, 384), (6, 3, 5, 50, 256), (2, 2, 4, 66, 8192), (33, 2, 16, 72, 128),
         (20, 5, 5, 514, 8192), (50, 2, 2, 98, 4096), (65, 2, 2, 98, 128), (65, 2, 2, 97, 1024), (650, 2, 2, 1538, 128),
         (165, 2, 2, 1538, 2048), (500, 2, 2, 2050, 384), (2050, 2, 2, 258, 2048), (650, 2, 2, 8193, 128),
         (650, 2, 2, 1538, 4096), (200, 1, 3, 300, 1152)]


@pytest.mark.parametrize("fmt", ["any4", "int4", "any2", "any3"])
@pytest.mark.parametrize("T,k,E,N,K", SIZES)
def test_rows_in_parts(fmt, T, k, E, N, K):
    packed, tables, w = layers(fmt, E, N, K, 128)
    ids, v = choose(T, k, E), rows(T, T, k, K)
    x, out, z = in_parts(v), empty(T, k, N), empty(T, k, N)
    assert call_of(fmt, "experts")(x, packed, *tables, 128, ids, out=out, z=z) is out
    want, e = each_expert(whole(x), w, ids)
    near(out, want, 2 * e)
    assert torch.equal(z, out)
    exact, e = each_expert(v.double(), w, ids)
    near(out, exact, 2 * e + 2.0 ** -16 * each_expert(v.double().abs(), w.abs(), ids)[0])


@pytest.mark.parametrize("T,k,E,N,K", [(3, 2, 4, 98, 256), (40, 4, 30, 98, 256), (100, 2, 2, 1026, 128), (600, 2, 2, 2050, 256),
                                       (650, 2, 2, 8194, 128), (50, 2, 2, 98, 4096)])
def test_epilogues_of_rows_in_parts(T, k, E, N, K):
    packed, tables, w = layers("any4", E, N, K, 128)
    ids, x, b = choose(T, k, E), in_parts(rows(T, T, k, K)), normal(8, E, N)
    ref, e = each_expert(whole(x), w, ids, bias=b)
    live = ((ids >= 0) & (ids < E))[:, :, None]
    for act, gate in (("silu", True), ("relu", False)):
        for plan in (None, any4.experts_plan(ids, E)):
            out = any4.experts_gemm(x, packed, *tables, 128, ids, bias=b, act=act, gate=gate, plan=plan)
            want, eo = expect(ref, 2 * e, act, gate)
            close(out, torch.where(live, want, torch.zeros_like(want)), eo)
            assert not (out * ~live).any()


@pytest.mark.parametrize("fmt", ["any4", "int4", "any2", "any3"])
@pytest.mark.parametrize("T,k", [(2, 2), (16, 3), (70, 2), (300, 2)])
def test_one_hot_parts_give_the_weights(fmt, T, k):
    """hi or lo of a row is a unit vector: its weights bit for bit; both: the sum of two, rounded (or cut) once."""
    packed, tables, w = layers(fmt, 2, 70, 256, 128)
    ids = torch.tensor([0, 1, 1], dtype=torch.int32, device=gu.DEV)[:k].repeat(T, 1)
    at = torch.arange(T * k, device=gu.DEV).view(T, k)
    x = torch.zeros(2, T, k, 256, dtype=BF16, device=gu.DEV)
    for part, step in ((0, 3), (1, 7)):
        x[part].scatter_(2, (step * at % 256)[:, :, None], 1.0)
    for only in (0, 1, None):
        y = x.clone()
        if only is not None:
            y[1 - only] = 0
        out = call_of(fmt, "experts")(y, packed, *tables, 128, ids, out=empty(T, k, 70))
        want = sum(w[ids.long()].gather(3, (step * at % 256)[:, :, None, None].expand(T, k, 70, 1))[..., 0]
                   for part, step in ((0, 3), (1, 7)) if only in (None, part))
        if only is None:
            near(out, want, 2.0 ** -24 * want.abs())
        else:
            assert torch.equal(out, want.float())


@pytest.mark.parametrize("T,k,E,N,K", [(1, 2, 8, 96, 384), (6, 3, 5, 51, 256), (2, 2, 4, 66, 8192), (50, 2, 2, 98, 4096),
                                       (65, 2, 2, 99, 128), (70, 2, 2, 1538, 128), (650, 2, 2, 8193, 128)])
@pytest.mark.parametrize("gate", [False, True])
def test_results_in_parts(T, k, E, N, K, gate):
    """The parts of what the same call gives in fp32, zeros where there is no expert, for rows in bf16 and
    in parts."""
    N -= N % 2 if gate else 0
    packed, tables, _ = layers("any4", E, N, K, 128)
    ids, No = choose(T, k, E), N // 2 if gate else N
    for x in (normal(7, T, K), in_parts(rows(T, T, k, K))):
        how = dict(act="gelu_tanh", gate=gate)
        wide = any4.experts_gemm(x, packed, *tables, 128, ids, out=empty(T, k, No), **how)
        room = torch.full((2 * T * k * No + 2,), 7.0, dtype=BF16, device=gu.DEV)
        out = room[1:-1].view(2, T, k, No)
        assert any4.experts_gemm(x, packed, *tables, 128, ids, out=out, **how) is out
        assert torch.equal(out, in_parts(wide)) and room[0] == 7 and room[-1] == 7
        assert ((whole(out) - wide.double()).abs() <= 2.0 ** -16 * wide.double().abs()).all()


@pytest.mark.parametrize("T", [5, 60])
def test_values_that_are_not_finite(T):
    packed, tables, w = layers("any4", 2, 40, 256, 128)
    ids = torch.tensor([[0, 1]] * T, dtype=torch.int32, device=gu.DEV)
    v = rows(1, T, 2, 256)
    v[1, :, 7], v[2, :, 9], v[3, :, 200], v[4] = float("inf"), float("-inf"), float("nan"), 0.0
    v[4, :, 3] = torch.finfo(F32).max
    out = any4.experts_gemm(in_parts(v), packed, *tables, 128, ids, out=empty(T, 2, 40))
    parts = any4.experts_gemm(in_parts(v), packed, *tables, 128, ids, out=empty(2, T, 2, 40, dtype=BF16))
    for j in range(2):
        for t, k in ((1, 7), (2, 9)):
            assert torch.equal(out[t, j], (v[t, j, k].double() * w[j, :, k]).float())
            assert torch.equal(parts[0, t, j].float(), out[t, j]) and not parts[1, t, j].any()
    assert torch.isnan(out[3]).all() and torch.isnan(whole(parts)[3]).all()
    keep = torch.tensor([t not in (1, 2, 3, 4) for t in range(T)], device=gu.DEV)
    assert torch.isfinite(out[keep]).all() and torch.isfinite(parts[:, keep]).all()
    want = v[4, :, 3].double()[:, None] * w[:, :, 3]
    small = want.abs() < 3e38
    assert small.any() and ((out[4].double() - want).abs()[small] <= 2.0 ** -15 * want.abs()[small]).all()


@pytest.mark.parametrize("T,k,E", [(7, 3, 8), (32, 2, 8), (33, 2, 8), (200, 2, 4), (700, 2, 3)])
def test_the_second_product_keeps_what_the_first_computed(T, k, E):
    """A block's result is as exact on either side of 64 pairs: h costs it 2^-16, not a bf16's 2^-8."""
    b = Block(T, 256, 384, E, k)
    ids = choose(T, k, E)
    (w1, t1, up), (w2, t2, down) = b.up, b.down
    plan = any4.experts_plan(ids, E)
    h = torch.empty(2, T, k, 384, dtype=BF16, device=gu.DEV)
    any4.experts_gemm(b.x, w1, *t1, 128, ids, act="silu", gate=True, plan=plan, out=h)
    y = any4.experts_gemm(h, w2, *t2, 128, ids, plan=plan, out=empty(T, k, 256))
    z, ez = each_expert(b.x.double()[:, None].expand(T, k, 256), up, ids)
    h64, eh = expect(z, ez, "silu", True)
    want, e = each_expert(h64, down, ids)
    eh = eh + 2.0 ** -16 * (h64.abs() + eh)
    near(y, want, 2 * e * 1.01 + each_expert(eh, down.abs(), ids)[0] * 1.01)


@pytest.mark.parametrize("T", [9, 150])
def test_captured_and_replayed(T):
    E, k = 6, 3
    b = Block(T, 256, 128, E, k)
    (w1, t1, _), (w2, t2, _) = b.up, b.down
    ids, x = choose(T, k, E), b.x.clone()

    def run():
        h = torch.empty(2, T, k, 128, dtype=BF16, device=gu.DEV)
        any4.experts_gemm(x, w1, *t1, 128, ids, act="silu", gate=True, out=h)
        return any4.experts_gemm(h, w2, *t2, 128, ids, out=torch.empty(T, k, 256, device=gu.DEV))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run()
    for i in range(4):
        x.copy_(normal(50 + i, T, 256, std=0.05))
        ids.copy_(choose(T, k, E, seed=i + 2))
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, want)


@pytest.mark.parametrize("T,N,K", [(50, 98, 4096), (165, 1538, 2048)])
def test_a_workspace_of_the_caller(T, N, K):
    packed, tables, _ = layers("any4", 2, N, K, 128)
    ids, x = choose(T, 2, 2), in_parts(rows(T, T, 2, K))
    need = any4.experts_parts_workspace_size(T, 2, 2, N, K, 128)
    want = any4.experts_gemm(x, packed, *tables, 128, ids)
    room = torch.full((need + 256,), 77, dtype=torch.uint8, device=gu.DEV)
    assert torch.equal(any4.experts_gemm(x, packed, *tables, 128, ids, workspace=room[:need]), want) and (room[need:] == 77).all()
    with pytest.raises(any4.Any4Error):
        any4.experts_gemm(x, packed, *tables, 128, ids, workspace=room[:need - 256])


def test_rows_do_not_touch_each_other():
    packed, tables, _ = layers("any4", 3, 100, 256, 128)
    ids, v = choose(60, 2, 3, empty=False), rows(1, 60, 2, 256)
    clean = any4.experts_gemm(in_parts(v), packed, *tables, 128, ids)
    v[4, 1], v[50, 0, 3] = float("nan"), float("inf")
    got = any4.experts_gemm(in_parts(v), packed, *tables, 128, ids)
    keep = torch.ones(60, 2, dtype=torch.bool, device=gu.DEV)
    keep[4, 1] = keep[50, 0] = False
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[4, 1]).all() and not torch.isfinite(got[50, 0]).any()


def test_refusals():
    packed, tables, _ = layers("any4", 2, 40, 256, 128)
    ids, x = choose(40, 2, 2), in_parts(rows(1, 40, 2, 256))
    for bad in (x.float(), x[:1], x[:, :39], x[..., :128], torch.cat([x, x[:1]])):
        with pytest.raises((TypeError, ValueError)):
            any4.experts_gemm(bad.contiguous(), packed, *tables, 128, ids)
    with pytest.raises(ValueError):
        any4.experts_gemm(x.transpose(1, 2), packed, *tables, 128, ids)
    for out in (empty(2, 40, 2, 40), empty(2, 40, 2, 41, dtype=BF16), empty(1, 40, 2, 40, dtype=BF16)):
        with pytest.raises((TypeError, ValueError)):
            any4.experts_gemm(x, packed, *tables, 128, ids, out=out)
