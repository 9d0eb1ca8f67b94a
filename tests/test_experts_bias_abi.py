"""any4_experts_bias_backward refuses bad arguments before touching the GPU (CPU only)."""
import gemm_any4_amd as any4
from tests.test_ffn_abi import A, BIG


def call(dy=A, z=A, ids=A, plan=None, dbias=A, act=2, gate=0, T=400, k=2, E=4, N=16, ws=A, ws_bytes=BIG, dy_f32=0, z_f32=0):
    return any4.experts_bias_backward_raw(dy, z, ids, plan, dbias, act, gate, T, k, E, N, ws, ws_bytes, stream=0, dy_f32=dy_f32,
                                          z_f32=z_f32)


def test_shapes():
    for bad in (dict(T=-1), dict(k=0), dict(T=1 << 20), dict(T=1 << 62, k=4), dict(k=1 << 62), dict(E=0), dict(E=1025), dict(N=-1),
                dict(N=(1 << 28) + 1, T=1, k=1), dict(T=1 << 19, N=1024), dict(act=5), dict(act=-1), dict(gate=1, N=15)):
        assert call(**bad) == 2, bad
        if "act" not in bad and "gate" not in bad:
            assert any4.experts_bias_workspace_size(**(dict(T=400, k=2, E=4, N=16) | bad)) == 0


def test_pointers():
    for name in ("dy", "z", "ids", "dbias", "ws"):
        assert call(**{name: None}) == 1
    for name, off in (("dy", 1), ("z", 1), ("ids", 2), ("dbias", 2), ("ws", 8), ("plan", 8)):
        assert call(**{name: A + off}) == 3
    assert call(dy=A + 2, dy_f32=1) == 3 and call(z=A + 2, z_f32=1) == 3
    assert call(None, None, None, None, None, N=0) == 0 and call(None, None, None, dbias=None, T=0) == 1


def test_workspaces():
    need = any4.experts_bias_workspace_size(400, 2, 4, 16)
    plan = any4.lora_plan_bytes(800, 4)
    assert need > plan and call(ws_bytes=need - 1) == 4 and call(plan=A, ws_bytes=need - plan - 1) == 4
    assert any4.experts_bias_workspace_size(256, 2, 4, 16) == any4.lora_plan_bytes(512, 4)
