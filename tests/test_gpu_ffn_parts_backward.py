"""The backward pass of experts' products with what lies between its calls in two bf16
parts: act_backward's dz, and experts_gemm_dx of it.  Tolerances as in test_gpu_ffn_parts.py."""
import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu
from tests.test_gpu_ffn import ACTS, call_of, choose, close, each_expert, expect, f64, layers, normal
from tests.test_gpu_ffn_block import Block, empty, near
from tests.test_gpu_ffn_parts import BF16, F32, in_parts, rows, whole

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


def backward64(d, z, act, gate):
    """(dz, the magnitudes that its fp32 steps are off in)."""
    No = d.shape[-1]
    a, u = z[..., :No], z[..., No:] if gate else torch.ones_like(d)
    f, slope = f64(act, a)
    want, scale = d * u * slope, (d * u).abs() * (1 + a.abs())
    if gate:
        want, scale = torch.cat([want, d * f], -1), torch.cat([scale, d.abs() * (1 + a.abs())], -1)
    return want, scale


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("M,N", [(1, 2), (33, 1030), (64, 512), (129, 98), (1000, 130)])
@pytest.mark.parametrize("kind", [F32, BF16])
def test_act_backward_in_parts(act, gate, M, N, kind):
    No = N // 2 if gate else N
    z, dy = rows(1, M, N).mul(2).to(kind), rows(2, M, No).to(kind)
    room = torch.full((2 * M * N + 2,), 7.0, dtype=BF16, device=gu.DEV)
    dz, dbias = any4.act_backward(dy, z, act, gate=gate, dz=room[1:-1].view(2, M, N))
    rounded, want_bias = any4.act_backward(dy, z, act, gate=gate)
    assert torch.equal(dbias, want_bias) and room[0] == 7 and room[-1] == 7
    want, scale = backward64(dy.double(), z.double(), act, gate)
    e = 2.0 ** -19 * scale          # as in test_gpu_ffn.py
    v = whole(dz)
    assert ((v - want).abs() <= e + 2.0 ** -16 * (want.abs() + e)).all()
    assert ((rounded.double() - v).abs() <= (2.0 ** -8 + 2.0 ** -15) * v.abs()).all()
    # hi is cut, lo what is left (rounded, up to a whole step of hi: the sum need not have the same parts)
    assert (dz[0].double().abs() <= v.abs()).all() and (dz[1].double().abs() <= 2.0 ** -7 * dz[0].double().abs()).all()
    if act == "none" and not gate:
        assert torch.equal(dz, in_parts(dy.float()))
    again, none = any4.act_backward(dy, z, act, gate=gate, dz=torch.empty(2, M, N, dtype=BF16, device=gu.DEV), need_bias=False)
    assert none is None and torch.equal(again, dz)


# tiles of two heights, with split sums and without; rows that are padded, and not
SIZES = [(1, 1, 1, 1, 128), (1, 2, 8, 96, 256), (5, 3, 7, 50, 384), (33, 2, 16, 72, 128), (50, 2, 2, 1021, 128), (1025, 2, 2, 93, 1024),
         (66, 5, 5, 1536, 2048), (350, 2, 2, 96, 8192), (165, 2, 2, 2043, 4096), (1025, 2, 2, 96, 2048), (650, 2, 2, 4091, 384)]


@pytest.mark.parametrize("fmt", ["any4", "int4", "any2", "any3"])
@pytest.mark.parametrize("T,k,E,N,K", SIZES)
def test_dx_of_parts(fmt, T, k, E, N, K):
    packed, tables, w = layers(fmt, E, N, K, 128)
    ids, dy = choose(T, k, E), in_parts(rows(T, T, k, N))
    want, e = each_expert(whole(dy), w, ids, back=True)
    for plan in (None, any4.experts_plan(ids, E)):
        out = empty(T, k, K)
        assert call_of(fmt, "dx")(dy, packed, *tables, 128, ids, plan=plan, out=out) is out
        near(out, want, 2 * e)
    close(call_of(fmt, "dx")(dy, packed, *tables, 128, ids), want, 2 * e)


@pytest.mark.parametrize("fmt", ["any4", "int4", "any2", "any3"])
@pytest.mark.parametrize("N", [96, 100])
def test_dx_of_one_hot_parts_gives_the_weights(fmt, N):
    packed, tables, w = layers(fmt, 2, N, 256, 128)
    ids = torch.tensor([[0, 1]], dtype=torch.int32, device=gu.DEV).repeat(N, 1)
    one = torch.eye(N, dtype=BF16, device=gu.DEV)[:, None].repeat(1, 2, 1)
    for dy in (torch.stack([one, torch.zeros_like(one)]), torch.stack([torch.zeros_like(one), one])):
        assert torch.equal(call_of(fmt, "dx")(dy, packed, *tables, 128, ids).double(), w.transpose(0, 1))


def test_dy_at_any_place_and_rows_that_do_not_touch():
    packed, tables, _ = layers("any4", 3, 104, 256, 128)
    ids = choose(60, 2, 3, empty=False)
    room = torch.zeros(2 * 60 * 2 * 104 + 3, dtype=BF16, device=gu.DEV)
    dy = room[3:].view(2, 60, 2, 104)           # not 16-byte aligned: through the padded copy
    dy.copy_(in_parts(rows(9, 60, 2, 104)))
    clean = any4.experts_gemm_dx(dy.clone(), packed, *tables, 128, ids)
    assert torch.equal(any4.experts_gemm_dx(dy, packed, *tables, 128, ids), clean)
    dy[1, 4, 1] = float("nan")
    dy[0, 50, 0] = float("nan")
    got = any4.experts_gemm_dx(dy, packed, *tables, 128, ids)
    keep = torch.ones(60, 2, dtype=torch.bool, device=gu.DEV)
    keep[4, 1] = keep[50, 0] = False
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[4, 1]).all() and torch.isnan(got[50, 0]).all()


def run(b, ids, plan=None):
    """The gradient of b's rows, from dout of each pair, and what it goes through."""
    (w1, t1, _), (w2, t2, _) = b.up, b.down
    T, k, F, H = b.T, b.k, b.F, b.H
    z, dh, dx = (torch.empty(T, k, n, device=gu.DEV) for n in (2 * F, F, H))
    any4.experts_gemm(b.x, w1, *t1, 128, ids, act="silu", gate=True, z=z, plan=plan)
    dy = b.dout[:, None].expand(T, k, H).contiguous()
    any4.experts_gemm_dx(dy, w2, *t2, 128, ids, plan=plan, out=dh)
    dz, _ = any4.act_backward(dh, z, "silu", gate=True, need_bias=False, dz=torch.empty(2, T, k, 2 * F, dtype=BF16, device=gu.DEV))
    return any4.experts_gemm_dx(dz, w1, *t1, 128, ids, plan=plan, out=dx)


@pytest.mark.parametrize("T,H,F,E,k", [(7, 256, 128, 8, 3), (33, 256, 384, 5, 2), (600, 128, 256, 3, 2)])
def test_the_rows_gradient_keeps_what_the_epilogues_computed(T, H, F, E, k):
    """The input's gradient through a block: dz costs it 2^-16, not a bf16's 2^-8."""
    b = Block(T, H, F, E, k)
    ids = choose(T, k, E)
    got = run(b, ids, any4.experts_plan(ids, E))
    z, ez = each_expert(b.x.double()[:, None].expand(T, k, H), b.up[2], ids)
    dh, edh = each_expert(b.dout.double()[:, None].expand(T, k, H), b.down[2], ids, back=True)
    ez, edh = ez + 2.0 ** -24 * (z.abs() + ez), edh + 2.0 ** -24 * (dh.abs() + edh)
    a, u, ea, eu = z[..., :F], z[..., F:], ez[..., :F], ez[..., F:]
    f, slope = f64("silu", a)
    da, du = dh * u * slope, dh * f
    # silu'' is at most 1/2, silu' 1.1
    eda = (dh.abs() + edh) * (u.abs() + eu) * (slope.abs() + ea / 2) - da.abs() + 2.0 ** -18 * (dh * u).abs() * (1 + a.abs())
    edu = (dh.abs() + edh) * (f.abs() + 1.2 * ea) - du.abs() + 2.0 ** -18 * dh.abs() * (1 + a.abs())
    dz, edz = torch.cat([da, du], 2), torch.cat([eda, edu], 2)
    edz = edz + 2.0 ** -16 * (dz.abs() + edz)
    want, e = each_expert(dz, b.up[2], ids, back=True)
    near(got, want, 1.01 * 2 * e + 1.01 * each_expert(edz, b.up[2].abs(), ids, back=True)[0])


@pytest.mark.parametrize("T", [9, 150])
def test_captured_and_replayed(T):
    E, k = 6, 3
    b = Block(T, 256, 128, E, k)
    ids = choose(T, k, E)
    b.x = b.x.clone()
    run(b, ids)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run(b, ids)
    for i in range(4):
        b.x.copy_(normal(50 + i, T, 256, std=0.05))
        ids.copy_(choose(T, k, E, seed=i + 2))
        want = run(b, ids)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, want)


@pytest.mark.parametrize("T,N,K", [(50, 98, 4096), (350, 96, 8192)])
def test_a_workspace_of_the_caller(T, N, K):
    packed, tables, _ = layers("any4", 2, N, K, 128)
    ids, dy = choose(T, 2, 2), in_parts(rows(T, T, 2, N))
    need = any4.experts_dx_parts_workspace_size(T, 2, 2, N, K, 128)
    want = any4.experts_gemm_dx(dy, packed, *tables, 128, ids)
    room = torch.full((need + 256,), 77, dtype=torch.uint8, device=gu.DEV)
    assert torch.equal(any4.experts_gemm_dx(dy, packed, *tables, 128, ids, workspace=room[:need]), want) and (room[need:] == 77).all()
    with pytest.raises(any4.Any4Error):
        any4.experts_gemm_dx(dy, packed, *tables, 128, ids, workspace=room[:need - 1])


def test_refusals():
    packed, tables, _ = layers("any4", 2, 40, 256, 128)
    ids, dy = choose(40, 2, 2), in_parts(rows(1, 40, 2, 40))
    for bad in (dy.float(), dy[:1], dy[:, :39], dy[..., :32]):
        with pytest.raises((TypeError, ValueError)):
            any4.experts_gemm_dx(bad.contiguous(), packed, *tables, 128, ids)
    z, d = rows(1, 5, 40), rows(2, 5, 40)
    for bad in (empty(2, 5, 40), empty(2, 5, 41, dtype=BF16), empty(1, 5, 40, dtype=BF16)):
        with pytest.raises((TypeError, ValueError)):
            any4.act_backward(d, z, "silu", dz=bad)
    T = 0
    got = any4.experts_gemm_dx(dy[:, :T].contiguous(), packed, *tables, 128, ids[:T])
    assert got.shape == (0, 2, 256)
