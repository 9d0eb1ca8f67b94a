"""A training step through two stacked any4 layers with adapters, as a program
runs it: gemm_lora forward with the inputs kept in 8 bits, then gemm_dx and
lora_backward from the top.  Each result is checked against the formulas in 64
bits from the values that the step itself handed on."""
import pytest
import torch

import gemm_any4_amd as any4
import oracle
import workloads
from tests import gpu_util as gu
from tests.test_gpu_lora import assert_near, forward_ref, grads_ref, make

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


class Layer:
    def __init__(self, M, N, K, L, r, seed):
        inp = workloads.generic(seed, 1, N, K, 128)
        packed = oracle.pack(inp.idx)
        self.frozen = (gu.dev_u8(oracle.tile(packed)), gu.dev_b16(inp.lut), gu.dev_b16(inp.alpha),
                       gu.dev_b16(inp.beta), 128)
        self.w = gu.dev_b16(oracle.dequant(packed, inp.lut, inp.alpha, inp.beta, 128)).double()
        t = make(M, K, N, r, L, "mixed", seed)
        self.adapters = (t["A"], t["B"], t["scale"])

    def forward(self, x, ids, plan):
        M, r = x.shape[0], self.adapters[0].shape[1]
        self.x, self.h, self.act = x, torch.empty((M, r), device=gu.DEV), any4.act8_empty(x)
        self.y = any4.gemm(x, *self.frozen)          # for the check only
        return any4.gemm_lora(x, *self.frozen, *self.adapters, ids, h=self.h, act=self.act, plan=plan)

    def backward(self, dy, ids, plan):
        dx = any4.gemm_dx(dy, *self.frozen)
        self.base = dx.clone()
        q, qs = self.act
        return any4.lora_backward(dy, q, self.h, *self.adapters, ids, dx=dx, out=dx, x_scale=qs, plan=plan)


@pytest.mark.parametrize("M,L,r", [(1, 2, 8), (33, 3, 16), (257, 2, 24), (700, 1, 8)])
def test_step_through_two_layers(M, L, r):
    dims = [384, 512, 136]
    ids = (torch.arange(M, device=gu.DEV, dtype=torch.int32) * 7 // 3) % (L + 1)       # L: no adapter
    layers = [Layer(M, dims[1], dims[0], L, r, 1), Layer(M, dims[2], dims[1], L, r, 2)]
    plan = any4.lora_plan(ids, L)
    x = torch.randn((M, dims[0]), generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).to(gu.DEV)
    outs = []
    for layer in layers:
        x = layer.forward(x, ids, plan)
        outs.append(x)
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(10)).to(torch.bfloat16).to(gu.DEV)
    for layer, out in zip(reversed(layers), reversed(outs)):
        A, B, scale = layer.adapters
        t = {"x": layer.x, "A": A, "B": B, "scale": scale, "ids": ids, "y": layer.y, "dy": dy}
        dx, dA, dB = layer.backward(dy, ids, plan)
        ref, e, href, he = forward_ref(t)
        assert_near(out, ref, e, "out")
        assert_near(layer.h, href, he, "h")
        d = dy.double()
        base, mag = d @ layer.w, d.abs() @ layer.w.abs()
        assert_near(layer.base, base, 2 * (layer.w.shape[0] + 16) * U * mag, "projection's dx")
        t["dx"] = layer.base
        q, qs = layer.act
        x8 = (q.double().view(M, -1, 128) * qs.double()[:, :, None]).view(M, -1)
        (rdx, edx), (rA, eA), (rB, eB) = grads_ref(t, x8, layer.h.double())
        assert_near(dx, rdx, edx, "dx")
        assert_near(dA, rA, eA, "dA")
        assert_near(dB, rB, eB, "dB")
        dy = dx


@pytest.mark.parametrize("M", [3, 200])
def test_layer_with_adapters_in_two_graphs(M):
    """gemm_lora captured twice from one stream and replayed on two at once:
    each graph has its own workspaces (M = 200: a whole dequantised layer)."""
    L, r, K, N = 2, 8, 512, 264
    layer = Layer(M, N, K, L, r, 4)
    ids = torch.arange(M, device=gu.DEV, dtype=torch.int32) % L
    xs = [torch.randn((M, K), generator=torch.Generator().manual_seed(s)).to(torch.bfloat16).to(gu.DEV) for s in (1, 2)]
    refs = [any4.gemm_lora(x, *layer.frozen, *layer.adapters, ids).clone() for x in xs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(any4.gemm_lora(x, *layer.frozen, *layer.adapters, ids))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, t in zip(graphs, streams):
            with torch.cuda.stream(t):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, refs))
