"""Long batches whose pairs' rows would be beyond what a call takes, were they not shared."""
import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu
from tests.test_gpu_ffn import close, layers, product

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


def test_shared_rows_of_a_long_batch():
    T, k, E, N, K = 1 << 15, 8, 8, 16, 4096
    packed, tables, w = layers("any4", E, N, K, 128)
    gen = torch.Generator(device=gu.DEV).manual_seed(1)
    x = torch.randn(T, K, generator=gen, device=gu.DEV).to(torch.bfloat16)
    ids = torch.rand(T, E, generator=gen, device=gu.DEV).argsort(dim=1).to(torch.int32)
    ids[5, 3] = -1
    out = any4.experts_gemm(x, packed, *tables, 128, ids)
    for t in (0, 5, 1000, T - 1):
        for j in range(k):
            e = int(ids[t, j])
            if e < 0:
                assert not out[t, j].any()
            else:
                close(out[t, j][None], *product(x[t:t + 1].double(), w[e]))
