"""Adapter, 8-bit activation and input-gradient calls reject bad arguments
before touching the GPU, and their size queries (CPU only)."""
import pytest
import torch

import gemm_any4_amd as any4

A = 1 << 20          # a 16-byte aligned fake address (never dereferenced)
BIG = 1 << 40        # a workspace size that is always enough


def lora(x=A, a=A, b=A, scale=A, ids=A, plan=None, y=A, out=A, h=None, q=None, qs=None, M=4, N=16,
         K=128, r=8, L=2, ws=A, ws_bytes=BIG):
    return any4.lora_raw(x, a, b, scale, ids, plan, y, out, h, q, qs, M, N, K, r, L, ws, ws_bytes, stream=0)


def backward(dy=A, x=A, q=None, qs=None, h=A, a=A, b=A, scale=A, ids=A, plan=None, dx=None, dx_out=A, dA=A, dB=A, M=4,
             N=16, K=128, r=8, L=2, ws=A, ws_bytes=BIG):
    return any4.lora_backward_raw(dy, x, q, qs, h, a, b, scale, ids, plan, dx, dx_out, dA, dB, M, N, K, r, L, ws,
                                  ws_bytes, stream=0)


SHAPES = [dict(M=-1), dict(M=(1 << 20) + 1), dict(N=-1), dict(K=0), dict(K=64), dict(K=192), dict(K=-128), dict(M=1, N=(1 << 24) + 1), dict(M=1, K=(1 << 24) + 128), dict(r=0),
          dict(r=129), dict(L=0), dict(L=4097), dict(M=1 << 20, K=1024), dict(M=1 << 20, N=1024),
          dict(L=4096, r=128, K=2048), dict(L=4096, r=128, N=2048)]


@pytest.mark.parametrize("bad", SHAPES)
def test_lora_shape_errors(bad):
    assert lora(**bad) == 2
    assert backward(**bad) == 2
    sizes = dict(M=4, N=16, K=128, r=8, L=2) | bad
    assert any4.lora_workspace_size(**sizes) == 0
    assert any4.lora_backward_workspace_size(**sizes) == 0


def test_backward_needs_outputs():
    assert backward(N=0) == 2
    assert backward(*[None] * 14, M=0, ws=None, ws_bytes=0) == 0       # nothing to write either
    assert backward(M=0, dA=A + 2) == 3
    assert any4.lora_backward_workspace_size(0, 16, 128, 8, 2) == 0


@pytest.mark.parametrize("name", ["x", "a", "b", "scale", "ids", "y", "out", "ws"])
def test_lora_null_errors(name):
    assert lora(**{name: None}, M=65) == 1
    if name != "ws":                     # a few rows of a small layer need no workspace
        assert lora(**{name: None}) == 1


def test_lora_codes_need_their_scales():
    assert lora(q=A) == 1 and lora(qs=A) == 1


@pytest.mark.parametrize("name", ["dy", "x", "h", "a", "b", "scale", "ids", "ws"])
def test_backward_null_errors(name):
    assert backward(**{name: None}) == 1
    assert backward(x=None, q=A) == 1


@pytest.mark.parametrize("name,off", [("x", 8), ("a", 8), ("b", 1), ("scale", 2), ("ids", 2), ("plan", 8), ("y", 1),
                                      ("out", 1), ("h", 2), ("ws", 8)])
def test_lora_alignment_errors(name, off):
    assert lora(**{name: A + off}) == 3
    assert lora(q=A + 8, qs=A) == 3 and lora(q=A, qs=A + 2) == 3


@pytest.mark.parametrize("name,off", [("dy", 1), ("x", 8), ("h", 2), ("a", 8), ("b", 1), ("scale", 2), ("ids", 2),
                                      ("plan", 8), ("dx", 8), ("dx_out", 8), ("dA", 2), ("dB", 2), ("ws", 8)])
def test_backward_alignment_errors(name, off):
    assert backward(**{name: A + off}) == 3


@pytest.mark.parametrize("M", [1, 64, 65, 5000, 40000])
def test_workspace_errors(M):
    need = any4.lora_workspace_size(M, 16, 128, 128, 2)
    assert need > 0 and lora(M=M, r=128, ws_bytes=need - 1) == 4
    need = any4.lora_backward_workspace_size(M, 16, 128, 8, 2)
    assert need > 0 and backward(M=M, ws_bytes=need - 1) == 4


def test_empty_batch_is_a_no_op():
    assert lora(None, None, None, None, None, None, None, None, M=0, ws=None, ws_bytes=0) == 0
    assert any4.lora_workspace_size(0, 16, 128, 8, 2) == 0


def test_plan_errors_and_sizes():
    assert any4.lora_plan_bytes(0, 4) == 0 and any4.lora_plan_bytes(4, 0) == 0
    assert any4.lora_plan_bytes(4, 4097) == 0 and any4.lora_plan_bytes((1 << 20) + 1, 1) == 0
    need = any4.lora_plan_bytes(1000, 4)
    assert need >= 4 * 1000
    assert any4.lora_plan_raw(A, A, need - 1, 1000, 4, stream=0) == 4
    assert any4.lora_plan_raw(None, A, need, 1000, 4, stream=0) == 1
    assert any4.lora_plan_raw(A, None, need, 1000, 4, stream=0) == 1
    assert any4.lora_plan_raw(A + 2, A, need, 1000, 4, stream=0) == 3
    assert any4.lora_plan_raw(A, A + 4, need, 1000, 4, stream=0) == 3
    assert any4.lora_plan_raw(A, A, need, -1, 4, stream=0) == 2
    assert any4.lora_plan_raw(A, A, need, 1000, 0, stream=0) == 2
    assert any4.lora_plan_raw(None, None, 0, 0, 4, stream=0) == 0


def test_act8_errors():
    for call in (any4.act8_save_raw, any4.act8_load_raw):
        assert call(A, A, A, 4, 100, stream=0) == 2
        assert call(A, A, A, -1, 128, stream=0) == 2
        assert call(A, A, A, 1 << 20, 1024, stream=0) == 2
        assert call(A, A, None, 4, 128, stream=0) == 1
        assert call(None, A, A, 4, 128, stream=0) == 1
        assert call(A + 8, A, A, 4, 128, stream=0) == 3
        assert call(None, None, None, 0, 128, stream=0) == 0
        assert call(None, None, None, 4, 0, stream=0) == 0
    assert any4.act8_save_raw(A, A, A + 2, 4, 128, stream=0) == 3
    assert any4.act8_load_raw(A, A + 2, A, 4, 128, stream=0) == 3


CALLS = ["any4_gemm_dx", "any2_gemm_dx", "any3_gemm_dx", "int4"]


def dx(call, dy=A, packed=A, lut=A, alpha=A, beta=A, out=A, M=4, N=64, K=256, g=128, ws=A, ws_bytes=BIG):
    if call == "int4":
        return any4.gemm_int4_dx_raw(dy, packed, alpha, beta, out, M, N, K, g, ws, ws_bytes, stream=0)
    return any4.gemm_dx_raw(dy, packed, lut, alpha, beta, out, M, N, K, g, ws, ws_bytes, stream=0, call=call)


@pytest.mark.parametrize("call", CALLS)
def test_gemm_dx_errors(call):
    for bad in (dict(M=-1), dict(N=-1), dict(K=-128), dict(g=0), dict(g=64), dict(K=384, g=256), dict(M=65535 * 64 + 1),
                dict(M=1 << 20, K=1024), dict(M=1 << 20, N=1024), dict(N=(1 << 21) + 1), dict(N=1 << 20, K=4096, g=128)):
        assert dx(call, **bad) == 2, bad
        assert any4.gemm_dx_workspace_size(**(dict(M=4, N=64, K=256, g=128) | bad)) == 0
    for name in ("dy", "packed", "alpha", "beta", "out", "ws"):
        assert dx(call, **{name: None}) == 1
    if call != "int4":
        assert dx(call, lut=None) == 1 and dx(call, lut=A + 1) == 3
    for name, off in (("dy", 1), ("packed", 8), ("alpha", 1), ("beta", 1), ("out", 8), ("ws", 8)):
        assert dx(call, **{name: A + off}) == 3
    for M in (4, 300):
        need = any4.gemm_dx_workspace_size(M, 64, 256, 128)
        assert need > 0 and dx(call, M=M, ws_bytes=need - 1) == 4
    assert need >= 64 * 256 * 2          # beyond a few rows: the layer in bf16
    assert dx(call, None, None, None, None, None, None, M=0, ws=None) == 0
    assert dx(call, None, None, None, None, None, None, K=0, ws=None) == 0


def test_cpu_tensors_are_refused():
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    w = torch.zeros((1, 4, 128), dtype=torch.bfloat16)
    ids, scale = torch.zeros(2, dtype=torch.int32), torch.ones(1)
    with pytest.raises(ValueError):
        any4.lora(x, w, w, scale, ids, x)
    with pytest.raises(ValueError):
        any4.lora_backward(x, x, torch.zeros((2, 4)), w, w, scale, ids)
    with pytest.raises(ValueError):
        any4.lora_plan(ids, 1)
    with pytest.raises(ValueError):
        any4.act8_save(x)
