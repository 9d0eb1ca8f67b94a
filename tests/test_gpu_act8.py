"""Activations in 8 bits: codes, scales and values bit for bit against numpy's
fp32 arithmetic (each step of the definition is one IEEE operation)."""
import numpy as np
import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


def reference(x):
    """(q, qs) of x, a CPU bf16 tensor of finite values."""
    v = x.float().numpy().reshape(x.shape[0], -1, 128)
    amax = np.abs(v).max(axis=2, keepdims=True)
    live = amax >= np.float32(2.0 ** -100)
    safe = np.where(live, amax, np.float32(1))
    inv = np.where(live, np.float32(127) / safe, np.float32(0))
    qs = np.where(live, amax / np.float32(127), np.float32(0))
    return np.rint(v * inv).astype(np.int8).reshape(x.shape), qs[:, :, 0]


@pytest.mark.parametrize("M,K", [(1, 128), (3, 384), (16, 4096), (257, 1152), (1000, 128)])
@pytest.mark.parametrize("kind", ["normal", "outliers", "tiny", "wide"])
def test_codes_and_values(M, K, kind):
    g = torch.Generator().manual_seed(M * 131 + K)
    x = torch.randn((M, K), generator=g)
    if kind == "outliers":
        x[:, ::97] *= 40
    elif kind == "tiny":
        x *= torch.exp2(torch.randint(-130, -90, (M, K // 128), generator=g).float()).repeat_interleave(128, 1)
    elif kind == "wide":
        x *= torch.exp2(torch.randint(-60, 120, (M, K // 128), generator=g).float()).repeat_interleave(128, 1)
        x[0, :128] = 0
    x = x.to(torch.bfloat16)
    q, qs = any4.act8_save(x.to(gu.DEV))
    rq, rs = reference(x)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(qs.cpu().numpy(), rs)
    values = (rq.astype(np.float32).reshape(M, -1, 128) * rs[:, :, None]).reshape(M, K)
    assert torch.equal(any4.act8_load(q, qs).cpu(), torch.from_numpy(values).to(torch.bfloat16))


def test_every_bf16_magnitude_as_the_largest():
    """A group led by each finite bf16 value, the others spread below it."""
    bits = torch.arange(0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = bits[:, None].float() * torch.linspace(-1, 1, 128)[None, :]
    x = x.to(torch.bfloat16)
    q, qs = any4.act8_save(x.to(gu.DEV))
    rq, rs = reference(x)
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(qs.cpu().numpy(), rs)


def test_non_finite_groups_read_back_non_finite():
    x = torch.randn((4, 384)).to(torch.bfloat16)
    x[1, 200] = float("inf")
    x[2, 5] = float("nan")
    x[3, 383] = float("-inf")
    got = any4.act8_load(*any4.act8_save(x.to(gu.DEV))).cpu().view(4, 3, 128)
    bad = ~torch.isfinite(got)
    want = torch.zeros((4, 3), dtype=torch.bool)
    want[1, 1] = want[2, 0] = want[3, 2] = True
    assert torch.equal(bad.any(dim=2), want) and torch.equal(bad.all(dim=2), want)


def test_caller_buffers_streams_and_refusals():
    x = torch.randn((5, 256), device=gu.DEV).to(torch.bfloat16)
    act = any4.act8_empty(x)
    assert any4.act8_save(x, act=act)[0] is act[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = any4.act8_load(*any4.act8_save(x, stream=s), stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, any4.act8_load(*act))
    empty = any4.act8_load(*any4.act8_save(x[:0]))
    assert empty.shape == (0, 256)
    for bad in (x.float(), ):
        with pytest.raises(TypeError):
            any4.act8_save(bad)
    for bad in (x.cpu(), x[:, ::2], x[:, :100].contiguous(), x[0]):
        with pytest.raises(ValueError):
            any4.act8_save(bad)
    with pytest.raises(TypeError):
        any4.act8_load(act[0].view(torch.uint8), act[1])
    with pytest.raises(ValueError):
        any4.act8_load(act[0], act[1][:, :1].contiguous())
