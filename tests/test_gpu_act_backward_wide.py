"""The activation's backward pass at the widest rows it takes, with the bias's gradient."""
import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


@pytest.mark.parametrize("N,gate", [(1 << 29, False), ((1 << 29) - 63, False), ((1 << 28) + 1, False), (1 << 28, False), (1 << 29, True)])
def test_widest_rows(N, gate):
    """One row: dbias is dz before it is rounded.  dy and z of few bits: all products are exact."""
    No = N // 2 if gate else N
    z = torch.empty(1, N, dtype=torch.bfloat16, device=gu.DEV)
    z[0] = (torch.arange(N, device=gu.DEV, dtype=torch.int32) % 7 - 3).to(torch.bfloat16)
    dy = torch.empty(1, No, dtype=torch.bfloat16, device=gu.DEV)
    dy[0] = (torch.arange(No, device=gu.DEV, dtype=torch.int32) % 5 + 1).to(torch.bfloat16)
    dz, dbias = any4.act_backward(dy, z, "relu", gate=gate)
    if gate:
        a, u = z[0, :No], z[0, No:]
        assert torch.equal(dz[0, :No], torch.where(a > 0, dy[0] * u, 0)) and torch.equal(dz[0, No:], dy[0] * a.clamp(min=0))
    else:
        assert torch.equal(dz[0], torch.where(z[0] > 0, dy[0], 0))
    for at in range(0, N, 1 << 26):
        assert torch.equal(dbias[at:at + (1 << 26)], dz[0, at:at + (1 << 26)].float())
    plain, none = any4.act_backward(dy, z, "relu", gate=gate, need_bias=False)
    assert none is None and torch.equal(plain, dz)
