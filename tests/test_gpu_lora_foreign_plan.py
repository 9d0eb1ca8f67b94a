"""A plan of other sizes, as a caller of the C interface may hand in: the call
succeeds and writes nothing, whether that plan is larger or smaller than the
one it takes, and a fitting plan works as before.  (The binding refuses such a
plan by itself.)  The plans have buffers of exactly their size."""
import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu
from tests.test_gpu_lora import make

pytestmark = pytest.mark.gpu
K, N, r = 256, 136, 24


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


def outputs(t, M, L, value):
    dev = gu.DEV
    o = {"out": t["y"], "h": torch.empty((M, r), device=dev), "q": torch.empty((M, K), dtype=torch.int8, device=dev),
         "qs": torch.empty((M, K // 128), device=dev), "dx": t["dx"], "dA": torch.empty((L, r, K), device=dev),
         "dB": torch.empty((L, r, N), device=dev)}
    return {k: torch.full_like(v, value) for k, v in o.items()}


def call(t, M, L, plan, o, h):
    def p(k):
        return t[k].data_ptr()

    s = torch.cuda.current_stream().cuda_stream
    need = max(any4.lora_workspace_size(M, N, K, r, L), any4.lora_backward_workspace_size(M, N, K, r, L))
    ws = torch.empty(need, dtype=torch.uint8, device=gu.DEV)
    assert any4.lora_raw(p("x"), p("A"), p("B"), p("scale"), p("ids"), plan.words.data_ptr(), p("y"), o["out"].data_ptr(),
                         o["h"].data_ptr(), o["q"].data_ptr(), o["qs"].data_ptr(), M, N, K, r, L, ws.data_ptr(), need,
                         stream=s) == 0
    assert any4.lora_backward_raw(p("dy"), p("x"), None, None, h.data_ptr(), p("A"), p("B"), p("scale"), p("ids"),
                                  plan.words.data_ptr(), p("dx"), o["dx"].data_ptr(), o["dA"].data_ptr(), o["dB"].data_ptr(),
                                  M, N, K, r, L, ws.data_ptr(), need, stream=s) == 0


# sizes of the call and of the plan
@pytest.mark.parametrize("M,L,M2,L2", [
    (300, 9, 1, 1), (1300, 4, 100, 2), (20000, 700, 100, 2),         # smaller plans: unchunked, chunked, large tables
    (300, 9, 1300, 9), (300, 9, 300, 10), (300, 9, 20000, 4000),     # larger ones
    (1300, 4, 1300, 3), (1300, 4, 1301, 4), (600, 600, 300, 9),      # all but the same; an adapter a wave
])
def test_nothing_is_written(M, L, M2, L2):
    t = make(M, K, N, r, L, "mixed")
    ids2 = torch.arange(M2, device=gu.DEV, dtype=torch.int32) % L2
    other, own = any4.lora_plan(ids2, L2), any4.lora_plan(t["ids"], L)
    h = torch.randn((M, r), device=gu.DEV)
    o = outputs(t, M, L, 77)
    call(t, M, L, other, o, h)
    assert all((v == 77).all() for v in o.values())
    call(t, M, L, own, o, h)
    want_h = torch.empty_like(o["h"])
    out = any4.lora(t["x"], t["A"], t["B"], t["scale"], t["ids"], t["y"], h=want_h)
    dx, dA, dB = any4.lora_backward(t["dy"], t["x"], h, t["A"], t["B"], t["scale"], t["ids"], dx=t["dx"])
    q, qs = any4.act8_save(t["x"])
    want = {"out": out, "h": want_h, "q": q, "qs": qs, "dx": dx, "dA": dA, "dB": dB}
    assert all(torch.equal(o[k], v) for k, v in want.items())
