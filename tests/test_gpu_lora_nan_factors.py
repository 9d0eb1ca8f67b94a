"""A NaN of the fp32 factors that a caller hands in (h) is a NaN of the
gradient that it reaches, whatever its payload."""
import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu
from tests.test_gpu_lora import make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


# quiet, quiet with a payload in the low half, signalling with its payload in the
# high half, in the low half, negative
NANS = [0x7FC00000, 0x7FC00001, 0x7F810000, 0x7F800001, 0x7F80FFFF, 0xFF800001]


@pytest.mark.parametrize("bits", NANS)
@pytest.mark.parametrize("M,r", [(1, 1), (20, 5), (300, 5), (1300, 40)])
def test_nan_of_h(M, r, bits):
    t = make(M, 128, 40, r, 2, "runs")
    t["ids"] = torch.arange(M, device=gu.DEV, dtype=torch.int32) % 2
    h = torch.randn((M, r), generator=torch.Generator().manual_seed(1)).to(gu.DEV)
    clean = any4.lora_backward(t["dy"], t["x"], h, t["A"], t["B"], t["scale"], t["ids"])
    m, j = M // 2, r - 1
    h.view(torch.int32)[m, j] = bits - (1 << 32) if bits >> 31 else bits
    dx, dA, dB = any4.lora_backward(t["dy"], t["x"], h, t["A"], t["B"], t["scale"], t["ids"])
    assert torch.isnan(dB[m % 2, j]).all()
    assert torch.equal(dx, clean[0]) and torch.equal(dA, clean[1])      # these do not depend on h
    dB[m % 2, j] = clean[2][m % 2, j]
    assert torch.equal(dB, clean[2])
