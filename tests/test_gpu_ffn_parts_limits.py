"""Rows in two bf16 parts at the limits, and a training pass of experts in a row: on other streams, captured, its
bias's gradient with it."""
import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu
from tests.test_gpu_ffn import choose, layers, normal
from tests.test_gpu_ffn_block import near
from tests.test_gpu_ffn_parts import BF16, F32, whole
from tests.test_gpu_ffn_parts_backward import backward64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


def big(seed, *shape):
    """Parts of random values: any hi and lo will do."""
    gen = torch.Generator(device=gu.DEV).manual_seed(seed)
    x = torch.randn(2, *shape, generator=gen, device=gu.DEV, dtype=BF16)
    x[1] *= 2.0 ** -8
    return x


def pair_of(x, w, e):
    """(the product, its error) of one pair's row, two terms for each column."""
    want, mag = w[e] @ x, w[e].abs() @ x.abs()
    return want, 4 * (x.numel() + 16) * 2.0 ** -24 * mag


def test_most_rows():
    T, k, E, N, K = 130944, 8, 4, 32, 1024
    assert T * k * K < 1 << 30 <= (T + 128) * k * K + (1 << 20)
    packed, tables, w = layers("any4", E, N, K, 128)
    gen = torch.Generator(device=gu.DEV).manual_seed(3)
    ids = torch.randint(-1, E, (T, k), generator=gen, device=gu.DEV, dtype=torch.int32)
    x = big(1, T, k, K)
    out = any4.experts_gemm(x, packed, *tables, 128, ids, out=torch.empty(T, k, N, device=gu.DEV))
    for t in (0, 1, T // 2, T - 2, T - 1):
        for j in range(k):
            e = int(ids[t, j])
            if e < 0:
                assert not out[t, j].any()
            else:
                near(out[t, j], *pair_of(whole(x[:, t, j]), w, e))


def test_most_results_and_rows_back():
    T, k, E, N, K = 130944, 8, 4, 1024, 128
    packed, tables, w = layers("any4", E, N, K, 128)
    gen = torch.Generator(device=gu.DEV).manual_seed(3)
    ids = torch.randint(-1, E, (T, k), generator=gen, device=gu.DEV, dtype=torch.int32)
    x = normal(7, T, K)
    h = any4.experts_gemm(x, packed, *tables, 128, ids, out=torch.empty(2, T, k, N, dtype=BF16, device=gu.DEV))
    dx = any4.experts_gemm_dx(h, packed, *tables, 128, ids, out=torch.empty(T, k, K, device=gu.DEV))
    for t in (0, 1, T // 2, T - 2, T - 1):
        for j in range(k):
            e = int(ids[t, j])
            if e < 0:
                assert not h[:, t, j].any() and not dx[t, j].any()
                continue
            want, err = pair_of(x[t].double(), w, e)
            v = whole(h[:, t, j])
            assert ((v - want).abs() <= err + 2.0 ** -16 * (want.abs() + err)).all()
            near(dx[t, j], *pair_of(v, w.transpose(1, 2), e))


def test_most_rows_of_an_epilogue():
    M, N = (1 << 20) - 64, 1022
    assert M * N < 1 << 30
    gen = torch.Generator(device=gu.DEV).manual_seed(3)
    z = torch.randn(M, N, generator=gen, device=gu.DEV)
    dy = torch.randn(M, N // 2, generator=gen, device=gu.DEV)
    dz, _ = any4.act_backward(dy, z, "silu", gate=True, need_bias=False, dz=torch.empty(2, M, N, dtype=BF16, device=gu.DEV))
    for rows in (slice(0, 3), slice(M // 2, M // 2 + 3), slice(M - 3, M)):
        want, scale = backward64(dy[rows].double(), z[rows].double(), "silu", True)
        e = 2.0 ** -19 * scale
        assert ((whole(dz[:, rows]) - want).abs() <= e + 2.0 ** -16 * (want.abs() + e)).all()


class Pass:
    """x -> y = sum_j w_j (W2_e h + b2_e), h = silu(gate) up of W1_e x + b1_e; and back."""

    def __init__(self, T, H, F, E, k):
        self.sizes = (T, H, F, E, k)
        self.up, self.down = layers("any4", E, 2 * F, H, 128), layers("any4", E, H, F, 128, 105)
        self.x, self.dout, self.b1, self.b2 = normal(3, T, H, std=0.05), normal(4, T, H), normal(5, E, 2 * F), normal(6, E, H)
        self.logits, self.ids = normal(7, T, E).float(), choose(T, k, E)

    def run(self, **how):
        T, H, F, E, k = self.sizes
        (w1, t1, _), (w2, t2, _) = self.up, self.down
        ids = self.ids
        stream = how.get("stream")

        def empty(*shape, dtype=F32):
            with torch.cuda.stream(stream):             # None: the current one
                return torch.empty(shape, dtype=dtype, device=gu.DEV)
        w, _ = any4.route(self.logits, k, **how)
        plan = any4.experts_plan(ids, E, **how)
        h, dz = empty(2, T, k, F, dtype=BF16), empty(2, T, k, 2 * F, dtype=BF16)
        z, y, dh, dx = (empty(T, k, n) for n in (2 * F, H, F, H))
        any4.experts_gemm(self.x, w1, *t1, 128, ids, bias=self.b1, act="silu", gate=True, z=z, plan=plan, out=h, **how)
        any4.experts_gemm(h, w2, *t2, 128, ids, bias=self.b2, plan=plan, out=y, **how)
        out = any4.combine(y, w, **how)
        dy, dw = any4.combine_backward(self.dout, y, w, **how)
        db2 = any4.experts_bias_backward(dy, y, ids, E, "none", plan=plan, **how)
        any4.experts_gemm_dx(dy, w2, *t2, 128, ids, plan=plan, out=dh, **how)
        any4.act_backward(dh, z, "silu", gate=True, need_bias=False, dz=dz, **how)
        db1 = any4.experts_bias_backward(dh, z, ids, E, "silu", gate=True, plan=plan, **how)
        any4.experts_gemm_dx(dz, w1, *t1, 128, ids, plan=plan, out=dx, **how)
        return dict(out=out, dw=dw, db1=db1, db2=db2, dx=any4.combine(dx, **how))


@pytest.mark.parametrize("T", [20, 300])
def test_on_other_streams(T):
    p = Pass(T, 256, 128, 6, 3)
    want = p.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(6):              # two passes at a time
        with torch.cuda.stream(streams[i % 2]):
            got.append(p.run())
    torch.cuda.synchronize()
    got.append(p.run(stream=streams[0]))
    torch.cuda.synchronize()
    for g in got:
        for name in want:
            assert torch.equal(g[name], want[name]), name


@pytest.mark.parametrize("T", [20, 300])
def test_captured_and_replayed(T):
    p = Pass(T, 256, 128, 6, 3)
    p.x = p.x.clone()
    p.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = p.run()
    for i in range(4):
        p.x.copy_(normal(50 + i, T, 256, std=0.05))
        p.ids.copy_(choose(T, 3, 6, seed=i + 2))
        want = p.run()
        graph.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(kept[name], want[name]), (i, name)
