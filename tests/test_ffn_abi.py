"""Feed-forward calls reject bad arguments before touching the GPU, and their size
queries (CPU only)."""
import pytest
import torch

import gemm_any4_amd as any4

A = 1 << 20          # a 16-byte aligned fake address (never dereferenced)
BIG = 1 << 40        # a workspace size that is always enough


def act(fmt=0, x=A, packed=A, lut=A, alpha=A, beta=A, bias=None, residual=None, z=None, out=A, act=2, gate=0, M=4, N=16,
        K=128, g=128, ws=A, ws_bytes=BIG):
    return any4.gemm_act_raw(fmt, x, packed, lut, alpha, beta, bias, residual, z, out, act, gate, M, N, K, g, ws, ws_bytes,
                             stream=0)


def experts(fmt=0, x=A, per_pair=0, packed=A, lut=A, alpha=A, beta=A, bias=None, ids=A, plan=None, z=None, out=A, act=2,
            gate=0, T=100, k=2, E=4, N=16, K=128, g=128, ws=A, ws_bytes=BIG):
    return any4.experts_gemm_raw(fmt, x, per_pair, packed, lut, alpha, beta, bias, ids, plan, z, out, act, gate, T, k, E, N,
                                 K, g, ws, ws_bytes, stream=0)


def dx(fmt=0, dy=A, packed=A, lut=A, alpha=A, beta=A, ids=A, plan=None, out=A, T=100, k=2, E=4, N=16, K=128, g=128, ws=A,
       ws_bytes=BIG):
    return any4.experts_gemm_dx_raw(fmt, dy, packed, lut, alpha, beta, ids, plan, out, T, k, E, N, K, g, ws, ws_bytes,
                                    stream=0)


SHAPES = [dict(N=-1), dict(K=0), dict(K=64), dict(K=192), dict(K=-128), dict(g=0), dict(g=64), dict(K=384, g=256),
          dict(N=1 << 20, K=4096), dict(fmt=-1), dict(fmt=4), dict(N=1 << 30), dict(K=1 << 31)]


@pytest.mark.parametrize("bad", SHAPES + [dict(M=-1), dict(M=(1 << 20) + 1), dict(M=1 << 20, N=1024), dict(M=1 << 20, K=1024),
                                          dict(act=5), dict(act=-1), dict(gate=1, N=15)])
def test_gemm_act_shapes(bad):
    assert act(**bad) == 2
    if "fmt" not in bad and "act" not in bad and "gate" not in bad:
        assert any4.gemm_act_workspace_size(**(dict(M=4, N=16, K=128, g=128) | bad)) == 0


@pytest.mark.parametrize("bad", SHAPES + [dict(T=-1), dict(k=0), dict(T=1 << 20), dict(T=1 << 62, k=4), dict(k=1 << 62), dict(E=0),
                                          dict(E=1025), dict(T=1 << 19, N=1024)])
def test_experts_shapes(bad):
    assert experts(**bad) == 2 and dx(**bad) == 2
    if "fmt" not in bad:
        sizes = dict(T=100, k=2, E=4, N=16, K=128, g=128) | bad
        assert any4.experts_workspace_size(**sizes) == 0 and any4.experts_dx_workspace_size(**sizes) == 0


def test_experts_more_shapes():
    assert experts(act=5) == 2 and experts(gate=1, N=15) == 2 and experts(T=1 << 19, k=1, K=2048) == 2
    assert experts(T=1 << 19, k=2, K=1024, per_pair=1) == 2
    assert dx(N=0) == 2 and dx(T=700000, k=1, N=1533) == 2


@pytest.mark.parametrize("name", ["x", "packed", "lut", "alpha", "beta", "out"])
def test_null_pointers(name):
    assert act(**{name: None}) == 1 and experts(**{name: None}) == 1
    assert dx(**{{"x": "dy"}.get(name, name): None}) == 1
    if name == "lut":
        assert act(fmt=1, lut=None, ws=A + 8) == 3         # plain int4 has none


def test_more_null_pointers():
    assert experts(ids=None) == 1 and dx(ids=None) == 1 and dx(ws=None) == 1
    assert experts(ws=None) == 1                            # its own plan
    assert any4.gemm_act_workspace_size(1, 64, 8192, 128) > 0
    assert act(M=1, N=64, K=8192, ws=None) == 1             # a split sum


@pytest.mark.parametrize("name,off", [("x", 8), ("packed", 8), ("lut", 1), ("alpha", 1), ("beta", 1), ("bias", 1), ("z", 1),
                                      ("out", 1), ("ws", 8)])
def test_alignment(name, off):
    assert act(**{name: A + off}) == 3 and experts(**{name: A + off}) == 3
    if name not in ("bias", "z"):
        assert dx(**{{"x": "dy"}.get(name, name): A + (1 if name == "x" else off)}) == 3


def test_more_alignment():
    assert act(residual=A + 1) == 3
    for call in (experts, dx):
        assert call(ids=A + 2) == 3 and call(plan=A + 8) == 3


def test_workspace():
    need = any4.gemm_act_workspace_size(1, 64, 8192, 128)
    assert act(M=1, N=64, K=8192, ws_bytes=need - 1) == 4
    need = any4.experts_workspace_size(100, 2, 4, 16, 128, 128)
    assert need >= any4.lora_plan_bytes(200, 4) and experts(ws_bytes=any4.lora_plan_bytes(200, 4) - 1) == 4
    assert experts(T=2, N=64, K=8192, ws_bytes=any4.experts_workspace_size(2, 2, 4, 64, 8192, 128) - 1) == 4
    need = any4.experts_dx_workspace_size(100, 2, 4, 16, 128, 128)
    assert need > 0 and dx(ws_bytes=need - 1) == 4
    assert any4.experts_dx_workspace_size(1, 1, 1, 16, 128, 128) > 0


def test_empty_calls_are_no_ops():
    none = dict(x=None, packed=None, lut=None, alpha=None, beta=None, out=None, ws=None, ws_bytes=0)
    assert act(**none, M=0) == 0 and act(**none, N=0) == 0
    assert experts(**none, ids=None, T=0) == 0 and experts(**none, ids=None, N=0) == 0
    none["dy"] = none.pop("x")
    assert dx(**none, ids=None, T=0) == 0


def test_act_backward_errors():
    def call(dy=A, z=A, dz=A, dbias=A, act=2, gate=0, M=129, N=16, ws=A, ws_bytes=BIG):
        return any4.act_backward_raw(dy, z, dz, dbias, act, gate, M, N, ws, ws_bytes, stream=0)
    for bad in (dict(M=-1), dict(N=-1), dict(M=(1 << 20) + 1), dict(M=1 << 20, N=1024), dict(N=1 << 31), dict(act=5),
                dict(act=-1), dict(gate=1, N=15)):
        assert call(**bad) == 2, bad
    for name in ("dy", "z", "dz", "ws"):
        assert call(**{name: None}) == 1
    for name, off in (("dy", 1), ("z", 1), ("dz", 1), ("dbias", 2), ("ws", 8)):
        assert call(**{name: A + off}) == 3
    need = any4.act_backward_workspace_size(129, 16, 0)
    assert need > 0 and call(ws_bytes=need - 1) == 4 and any4.act_backward_workspace_size(128, 16, 0) == 0
    assert call(None, None, None, None, N=0, ws=None) == 0 and call(None, None, None, None, M=0, ws=None) == 0


def test_route_errors():
    def call(logits=A, bf16=0, bias=None, w=A, ids=A, score=0, T=4, E=8, k=2, groups=1, top=1):
        return any4.route_raw(logits, bf16, bias, w, ids, score, 1, 1.0, T, E, k, groups, top, stream=0)

    def back(dw=A, logits=A, bf16=0, ids=A, out=A, score=0, T=4, E=8, k=2):
        return any4.route_backward_raw(dw, logits, bf16, ids, out, score, 1, 1.0, T, E, k, stream=0)
    both = [dict(T=-1), dict(T=(1 << 20) + 1), dict(E=0), dict(E=1025), dict(k=0), dict(k=65, E=100), dict(k=9), dict(score=2),
            dict(score=-1), dict(T=1 << 20, k=2)]
    for bad in both:
        assert call(**bad) == 2 and back(**bad) == 2, bad
    for bad in (dict(groups=0), dict(groups=3), dict(groups=65, E=130), dict(groups=4, top=0), dict(groups=4, top=5),
                dict(groups=4, top=1, k=3)):
        assert call(**bad) == 2, bad
    for name in ("logits", "w", "ids"):
        assert call(**{name: None}) == 1
    for name in ("dw", "logits", "ids", "out"):
        assert back(**{name: None}) == 1
    for name in ("logits", "bias", "w", "ids"):
        assert call(**{name: A + 2}) == 3
    for name in ("dw", "logits", "ids", "out"):
        assert back(**{name: A + 2}) == 3
    assert call(logits=A + 1, bf16=1) == 3 and back(logits=A + 1, bf16=1) == 3 and back(out=A + 1, bf16=1) == 3
    assert call(None, w=None, ids=None, T=0) == 0 and back(None, None, ids=None, out=None, T=0) == 0


def test_combine_errors():
    def call(y=A, w=A, residual=A, out=A, T=4, k=2, N=16):
        return any4.combine_raw(y, w, residual, out, T, k, N, stream=0)

    def back(dout=A, y=A, w=A, dy=A, dw=A, T=4, k=2, N=16):
        return any4.combine_backward_raw(dout, y, w, dy, dw, T, k, N, stream=0)
    for f in (call, back):
        for bad in (dict(T=-1), dict(k=0), dict(N=-1), dict(T=1 << 20), dict(k=1 << 62), dict(T=1 << 19, N=1024), dict(N=1 << 30)):
            assert f(**bad) == 2, bad
        assert f(None, None, None, None, T=0) == 0
    assert call(y=None) == 1 and call(out=None) == 1 and call(None, None, None, None, N=0) == 0
    for name in ("dout", "y", "w"):
        assert back(**{name: None}) == 1
    assert back(None, None, None, None, None) == 0
    for name, off in (("y", 1), ("w", 2), ("residual", 1), ("out", 1)):
        assert call(**{name: A + off}) == 3
    for name, off in (("dout", 1), ("y", 1), ("w", 2), ("dy", 1), ("dw", 2)):
        assert back(**{name: A + off}) == 3


def test_the_binding_refuses():
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    table = torch.zeros((16, 1), dtype=torch.bfloat16)
    packed, lut = torch.zeros(16 * 64, dtype=torch.uint8), torch.zeros((16, 16), dtype=torch.bfloat16)
    ids = torch.zeros((2, 1), dtype=torch.int32)
    with pytest.raises(ValueError):
        any4.gemm_act(x, packed, lut, table, table, 128)
    with pytest.raises(ValueError):
        any4.experts_gemm(x, packed, lut[None], table[None], table[None], 128, ids)
    with pytest.raises(ValueError):
        any4.experts_gemm_dx(x[:, None, :16], packed, lut[None], table[None], table[None], 128, ids)
    with pytest.raises(ValueError):
        any4.experts_plan(ids, 1)
    with pytest.raises(ValueError):
        any4.act_backward(x, x, "silu")
    with pytest.raises(ValueError):
        any4.route(x, 2)
    with pytest.raises(ValueError):
        any4.combine(x[:, None])
    with pytest.raises(ValueError):
        any4.combine_backward(x, x[:, None], torch.ones(2, 1))


def test_fp32_results_and_inputs_need_four_bytes():
    for name, flag in (("z", "z_f32"), ("out", "out_f32")):
        args = dict(fmt=0, x_ptr=A, packed_ptr=A, lut_ptr=A, alpha_ptr=A, beta_ptr=A, bias_ptr=None, z_ptr=A, out_ptr=A, act=2, gate=0,
                    N=16, K=128, g=128, ws_ptr=A, ws_bytes=BIG, stream=0) | {name + "_ptr": A + 2, flag: 1}
        assert any4.gemm_act_raw(**args, residual_ptr=None, M=4) == 3
        assert any4.experts_gemm_raw(**args, per_pair=0, ids_ptr=A, plan_ptr=None, T=100, k=2, E=4) == 3
    assert any4.experts_gemm_dx_raw(0, A, A, A, A, A, A, None, A + 2, 100, 2, 4, 16, 128, 128, A, BIG, stream=0, dx_f32=1) == 3
    assert any4.act_backward_raw(A + 2, A, A, A, 2, 0, 4, 16, A, BIG, stream=0, dy_f32=1) == 3
    assert any4.act_backward_raw(A, A + 2, A, A, 2, 0, 4, 16, A, BIG, stream=0, z_f32=1) == 3
    assert any4.combine_raw(A + 2, A, None, A, 4, 2, 16, stream=0, y_f32=1) == 3
    assert any4.combine_backward_raw(A, A + 2, A, A, A, 4, 2, 16, stream=0, y_f32=1) == 3


def test_sizes_whose_packed_layers_or_grids_would_be_too_large():
    """A layer is packed in groups of 16 rows, whatever its N."""
    assert act(M=1, N=1, K=1 << 29, g=1 << 20) == 2 and any4.gemm_act_workspace_size(1, 1, 1 << 29, 1 << 20) == 0
    assert experts(T=1, k=1, N=1, K=1 << 28, g=1 << 20) == 2 and dx(T=1, k=1, N=1, K=1 << 28, g=1 << 20) == 2
    assert any4.act_backward_raw(A, A, A, A, 0, 0, 1, (1 << 29) + 2, A, BIG, stream=0) == 2
    assert any4.act_backward_workspace_size(1, (1 << 29) + 2, 0) == 0


def test_fp32_rows_for_few_pairs():
    args = (0, A, 0, A, A, A, A, None, A, None, None, A, 2, 0)
    assert any4.experts_gemm_raw(*args, 65, 1, 4, 16, 128, 128, A, BIG, stream=0, x_f32=1) == 2
    assert any4.experts_gemm_raw(0, A + 4, *args[2:], 8, 8, 4, 16, 128, 128, A, BIG, stream=0, x_f32=1) == 3
