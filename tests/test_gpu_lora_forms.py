"""Forms of the adapter calls that depend on more than the batch's size: weight
gradients where each wave has 128 columns of its own, at every rank and with
odd rows; a backward pass of which only some results are wanted; buffers at
addresses that only their elements align."""
import itertools

import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu
from tests import test_gpu_lora as base

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


@pytest.mark.parametrize("N", [2048, 2051])
@pytest.mark.parametrize("r", [16, 17, 20, 32, 33, 64, 65, 128])
@pytest.mark.parametrize("M,L,kind", [
    (64, 64, "distinct"), (50, 64, "mixed"),          # few rows: the batch's ids are searched
    (200, 64, "mixed"),                               # planned
    (1100, 64, "mixed"),                              # and in chunks
])
def test_weight_gradients_of_many_adapters(M, L, kind, r, N):
    """256 workgroups of eight waves and more: a wave has columns of its own."""
    base.test_forward_and_gradients(M, 2048, N, r, L, kind)


@pytest.mark.parametrize("M,K,N,r,L", [(64, 4096, 4096, 64, 64), (64, 4096, 4099, 64, 64), (3000, 1024, 2051, 24, 64)])
def test_uneven_adapters(M, K, N, r, L):
    """Nine tenths of the rows with one adapter of many."""
    t = base.make(M, K, N, r, L, "mixed")
    t["ids"][torch.rand(M, generator=torch.Generator().manual_seed(2)) < 0.9] = 5
    h = torch.empty((M, r), device=gu.DEV)
    out = any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"], h=h)
    ref, e, href, he = base.forward_ref(t)
    base.assert_near(h, href, he, "h")
    base.assert_near(out, ref, e, "out")
    got = any4.lora_backward(t["dy"], t["x"], h, t["A"], t["B"], t["scale"], t["ids"], dx=t["dx"])
    for g, (want, tol), what in zip(got, base.grads_ref(t, t["x"].double(), h.double()), ("dx", "dA", "dB")):
        base.assert_near(g, want, tol, what)


def ptr(t):
    return None if t is None else t.data_ptr()


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("M,K,N,r,L", [
    (40, 256, 136, 24, 3), (40, 256, 136, 100, 3),     # one launch, two
    (300, 256, 37, 24, 3), (1300, 256, 136, 24, 3),    # planned; in chunks
    (64, 2048, 2051, 20, 64), (600, 1024, 1032, 40, 200),      # a wave's own columns
])
def test_some_results_only(M, K, N, r, L, eight):
    """Every choice of dx_out, dA and dB: those asked for are the bits of the full
    call; x and h are not given where they are not read."""
    t = base.make(M, K, N, r, L, "mixed")
    h = torch.empty((M, r), device=gu.DEV)
    act = any4.act8_empty(t["x"])
    any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"], h=h, act=act)
    x, qs = act if eight else (t["x"], None)
    full = any4.lora_backward(t["dy"], x, h, t["A"], t["B"], t["scale"], t["ids"], dx=t["dx"], x_scale=qs)
    need = any4.lora_backward_workspace_size(M, N, K, r, L)
    s = torch.cuda.current_stream().cuda_stream
    for wanted in itertools.product((False, True), repeat=3):
        ws = torch.full((need,), 255, dtype=torch.uint8, device=gu.DEV)        # NaN of every kind of value
        o = [torch.full_like(f, 7) if w else None for w, f in zip(wanted, full)]
        use_x, use_h = (x if wanted[1] else None), (h if wanted[2] else None)
        x16, q, scales = (None, use_x, qs if wanted[1] else None) if eight else (use_x, None, None)
        assert any4.lora_backward_raw(ptr(t["dy"]), ptr(x16), ptr(q), ptr(scales), ptr(use_h), ptr(t["A"]), ptr(t["B"]),
                                      ptr(t["scale"]), ptr(t["ids"]), None, ptr(t["dx"]) if wanted[0] else None, *map(ptr, o),
                                      M, N, K, r, L, ptr(ws), need, stream=s) == 0
        for got, f in zip(o, full):
            assert got is None or torch.equal(got, f), wanted


class Shifted:
    """A copy of v one element behind an aligned address, 5s around it."""

    def __init__(self, v):
        self.room = torch.full((v.numel() + 9,), 5, dtype=v.dtype, device=v.device)
        self.t = self.room[1:1 + v.numel()].view(v.shape)
        self.t.copy_(v)

    def untouched(self):
        return bool((self.room[:1] == 5).all() and (self.room[1 + self.t.numel():] == 5).all())


@pytest.mark.parametrize("N", [37, 128])
@pytest.mark.parametrize("M,r", [(20, 6), (33, 100), (70, 6), (400, 6), (400, 40), (1300, 6), (1300, 65)])
def test_addresses_that_only_elements_align(M, r, N):
    """y, out, dy and B in the middle of a dword, dA, dB and h off 16 bytes: the bits
    of the aligned call, and nothing around them written."""
    K, L = 256, 3
    t = base.make(M, K, N, r, L, "mixed")
    h = torch.empty((M, r), device=gu.DEV)
    out = any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"], h=h)
    grads = any4.lora_backward(t["dy"], t["x"], h, t["A"], t["B"], t["scale"], t["ids"], dx=t["dx"])
    s = {k: Shifted(v) for k, v in (("y", t["y"]), ("B", t["B"]), ("dy", t["dy"]), ("out", torch.zeros_like(out)),
                                    ("h", torch.zeros_like(h)), ("dA", torch.zeros_like(grads[1])),
                                    ("dB", torch.zeros_like(grads[2])))}
    any4.lora(t["x"], t["A"], s["B"].t, t["scale"], t["ids"], s["y"].t, out=s["out"].t, h=s["h"].t)
    assert torch.equal(s["out"].t, out) and torch.equal(s["h"].t, h)
    any4.lora(t["x"], t["A"], s["B"].t, t["scale"], t["ids"], s["y"].t, out=s["y"].t)          # in place
    assert torch.equal(s["y"].t, out)
    dx, dA, dB = any4.lora_backward(s["dy"].t, t["x"], s["h"].t, t["A"], s["B"].t, t["scale"], t["ids"], dx=t["dx"],
                                    dA=s["dA"].t, dB=s["dB"].t)
    assert torch.equal(dx, grads[0]) and torch.equal(dA, grads[1]) and torch.equal(dB, grads[2])
    # each alone, beside aligned others
    for k in ("dy", "dA", "dB"):
        given = {"dA": torch.full_like(dA, 7), "dB": torch.full_like(dB, 7)}
        if k != "dy":
            s[k].t.fill_(7)
            given[k] = s[k].t
        got = any4.lora_backward(s["dy"].t if k == "dy" else t["dy"], t["x"], h, t["A"], t["B"], t["scale"], t["ids"],
                                 dx=t["dx"], **given)
        assert all(torch.equal(a, b) for a, b in zip(got, grads)), k
    assert all(v.untouched() for v in s.values())
