"""The gradient of the experts' bias against the formula in 64 bits, expert by expert, and
against differences.  Tolerances as for act_backward's dbias in test_gpu_ffn.py, over an expert's own pairs."""
import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu
from tests.test_gpu_ffn import ACTS, choose, f64, layers, normal
from tests.test_gpu_ffn_parts import rows
from tests.test_gpu_ffn_parts_backward import backward64

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


def check(got, dy, z, ids, E, act, gate):
    assert got.dtype == F32 and got.shape == (E, z.shape[2])
    want, scale = backward64(dy.double(), z.double(), act, gate)
    for e in range(E):
        own = ids == e
        w, s = want[own], scale[own]
        bound = 2.0 ** -19 * s.sum(0) + (int(own.sum()) + 16) * 2.0 ** -24 * w.abs().sum(0)
        assert ((got[e].double() - w.sum(0)).abs() <= bound).all(), e


# experts of one chunk of 512 pairs and of several, without a pair, all pairs of one
SIZES = [(1, 1, 1, 2), (1, 2, 8, 96), (5, 3, 7, 50), (33, 2, 16, 72), (256, 2, 1, 66), (257, 2, 1, 66), (300, 2, 2, 1030),
         (2000, 4, 3, 98), (700, 2, 300, 34), (3000, 2, 2, 2)]


@pytest.mark.parametrize("T,k,E,N", SIZES)
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("kinds", [(F32, F32), (BF16, BF16), (F32, BF16)])
def test_sums_by_expert(T, k, E, N, gate, kinds):
    ids, z, dy = choose(T, k, E), rows(1, T, k, N).mul(2).to(kinds[1]), rows(2, T, k, N // 2 if gate else N).to(kinds[0])
    none = (ids < 0) | (ids >= E)
    z[none], dy[none] = float("nan"), float("inf")          # left out
    for plan in (None, any4.experts_plan(ids, E)):
        out = torch.full((E, N), 7.0, device=gu.DEV)
        assert any4.experts_bias_backward(dy, z, ids, E, "silu", gate=gate, plan=plan, out=out) is out
        check(out, dy, z, ids, E, "silu", gate)
    assert torch.equal(any4.experts_bias_backward(dy, z, ids, E, "silu", gate=gate), out)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gate", [False, True])
def test_activations(act, gate):
    T, k, E, N = 40, 3, 5, 38
    ids, z, dy = choose(T, k, E), normal(1, T, k, N, std=2.0), normal(2, T, k, N // 2 if gate else N)
    got = any4.experts_bias_backward(dy, z, ids, E, act, gate=gate)
    check(got, dy, z, ids, E, act, gate)
    # one expert for all: act_backward's own sum
    one = torch.zeros_like(ids)
    alone = any4.experts_bias_backward(dy, z, one, 1, act, gate=gate)[0]
    whole = any4.act_backward(dy, z, act, gate=gate)[1]
    want, scale = backward64(dy.double(), z.double(), act, gate)
    assert ((alone - whole).abs() <= 2.0 ** -18 * scale.sum((0, 1)) + 2 * (T * k + 16) * 2.0 ** -24 * want.abs().sum((0, 1))).all()


def test_experts_without_pairs_and_empty_batches():
    ids = torch.tensor([[4], [-1], [4], [9]], dtype=torch.int32, device=gu.DEV)
    z, dy = rows(1, 4, 1, 16), rows(2, 4, 1, 16)
    got = any4.experts_bias_backward(dy, z, ids, 9, "none", out=torch.full((9, 16), 7.0, device=gu.DEV))
    assert torch.equal(got[4], dy[0, 0] + dy[2, 0]) and not got[[0, 1, 2, 3, 5, 6, 7, 8]].any()
    nobody = torch.full_like(ids, -1)
    assert not any4.experts_bias_backward(dy, z, nobody, 9, "none", out=torch.full((9, 16), 7.0, device=gu.DEV)).any()
    for plan in (None, any4.experts_plan(ids[:0], 9)):
        out = torch.full((9, 16), 7.0, device=gu.DEV)
        assert not any4.experts_bias_backward(dy[:0], z[:0], ids[:0], 9, "none", plan=plan, out=out).any()


@pytest.mark.parametrize("T,k,E,gate", [(30, 2, 3, True), (300, 2, 4, False)])
def test_with_the_product_and_against_differences(T, k, E, gate):
    N, K, act = 72, 256, "gelu_tanh"
    packed, tables, w = layers("any4", E, N, K, 128)
    ids, x, b = choose(T, k, E), normal(7, T, K, std=0.05), normal(8, E, N)
    z = torch.empty(T, k, N, device=gu.DEV)
    out = any4.experts_gemm(x, packed, *tables, 128, ids, bias=b, act=act, gate=gate, z=z)
    dy = rows(2, *out.shape)
    got = any4.experts_bias_backward(dy, z, ids, E, act, gate=gate)
    check(got, dy, z, ids, E, act, gate)
    live = (ids >= 0) & (ids < E)
    at = torch.where(live, ids, 0).long()
    base = z.double() - b.double()[at]

    def loss(bias):
        v = base + bias[at]
        o = f64(act, v[..., :N // 2])[0] * v[..., N // 2:] if gate else f64(act, v)[0]
        return (o * dy.double() * live[:, :, None]).sum()
    v, h = rows(3, E, N).double(), 1e-5
    slope = (loss(b.double() + h * v) - loss(b.double() - h * v)) / (2 * h)
    # h^2 times third derivatives and 2^-52 / h of the sums: far below 1e-6 of the magnitudes, as is the kernel's own error
    scale = (backward64(dy.double(), z.double(), act, gate)[1] * v[at].abs() * live[:, :, None]).sum()
    assert (slope - (got.double() * v).sum()).abs() <= 1e-6 * scale + 2.0 ** -18 * scale


def test_captured_and_replayed():
    T, k, E, N = 400, 2, 3, 130
    ids, z, dy = choose(T, k, E), rows(1, T, k, N), rows(2, T, k, N)
    any4.experts_bias_backward(dy, z, ids, E, "silu")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = any4.experts_bias_backward(dy, z, ids, E, "silu")
    for i in range(4):
        dy.copy_(rows(10 + i, T, k, N))
        ids.copy_(choose(T, k, E, seed=i + 2))
        want = any4.experts_bias_backward(dy, z, ids, E, "silu")
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, want)


def test_workspaces_and_plans():
    T, k, E, N = 400, 2, 1, 130
    ids, z, dy = choose(T, k, E, empty=False), rows(1, T, k, N), rows(2, T, k, N)
    want, need = any4.experts_bias_backward(dy, z, ids, E, "silu"), any4.experts_bias_workspace_size(T, k, E, N)
    room = torch.full((need + 256,), 77, dtype=torch.uint8, device=gu.DEV)
    assert torch.equal(any4.experts_bias_backward(dy, z, ids, E, "silu", workspace=room[:need]), want) and (room[need:] == 77).all()
    with pytest.raises(any4.Any4Error):
        any4.experts_bias_backward(dy, z, ids, E, "silu", workspace=room[:need - 256])
    plan = any4.experts_plan(ids, E)
    less = need - any4.lora_plan_bytes(T * k, E)
    assert torch.equal(any4.experts_bias_backward(dy, z, ids, E, "silu", plan=plan, workspace=room[:less]), want)
    with pytest.raises(any4.Any4Error):
        any4.experts_bias_backward(dy, z, ids, E, "silu", plan=plan, workspace=room[:less - 256])
    with pytest.raises(ValueError):
        any4.experts_bias_backward(dy, z, ids, E + 1, "silu", plan=plan)
    with pytest.raises(ValueError):
        any4.experts_bias_backward(dy[:, :1], z, ids, E, "silu")
    # a plan of other sizes leaves the result
    wrong, out = any4.experts_plan(ids[:-1], E), torch.full((E, N), 7.0, device=gu.DEV)
    assert any4.experts_bias_backward_raw(dy.data_ptr(), z.data_ptr(), ids.data_ptr(), wrong.words.data_ptr(), out.data_ptr(), 2, 0, T, k,
                                          E, N, room.data_ptr(), need, dy_f32=1, z_f32=1) == 0
    assert (out == 7).all()
