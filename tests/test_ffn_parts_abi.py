"""Rows and results in two bf16 parts: refusals and size queries of the C calls (CPU only)."""
import gemm_any4_amd as any4
from tests.test_ffn_abi import A, BIG

PARTS = any4.ANY4_PARTS


def experts(x=A, per_pair=1, z=None, out=A, T=100, k=2, E=4, N=16, K=128, ws=A, ws_bytes=BIG, x_f32=PARTS, out_f32=0, ids=A):
    return any4.experts_gemm_raw(0, x, per_pair, A, A, A, A, None, ids, None, z, out, 0, 0, T, k, E, N, K, 128, ws, ws_bytes,
                                 stream=0, x_f32=x_f32, out_f32=out_f32)


def test_rows_in_parts_are_those_of_pairs():
    assert experts(per_pair=0) == 2 and experts(per_pair=0, T=3) == 2
    assert experts(T=1 << 19, K=1024) == 2 and experts(T=0) == 0 and experts(N=0) == 0
    assert experts(T=33, x_f32=1) == 2 and experts(T=33, x_f32=2) == 2         # other values say fp32: up to 64 pairs


def test_pointers():
    assert experts(x=None) == 1 and experts(out=None) == 1 and experts(ids=None) == 1 and experts(ws=None) == 1
    assert experts(x=A + 8) == 3 and experts(out=A + 1, out_f32=PARTS) == 3 and experts(out=A + 2, out_f32=1) == 3
    assert experts(out=A + 2, out_f32=PARTS, x=None) == 1


def test_workspaces():
    for sizes in ((100, 2, 4, 16, 128), (2, 2, 4, 64, 8192), (165, 2, 2, 1538, 2048)):
        T, k, E, N, K = sizes
        need = any4.experts_parts_workspace_size(*sizes, 128)
        assert need > 0 and experts(T=T, k=k, E=E, N=N, K=K, ws_bytes=need - 1) == 4
    for bad in ((-1, 2, 4, 16, 128, 128), (100, 0, 4, 16, 128, 128), (100, 2, 0, 16, 128, 128), (100, 2, 4, 16, 64, 64),
                (1 << 20, 2, 4, 16, 128, 128), (100, 2, 4, 1 << 30, 128, 128)):
        assert any4.experts_parts_workspace_size(*bad) == 0


def dx(dy=A, out=A, T=100, k=2, E=4, N=16, K=128, ws=A, ws_bytes=BIG, dx_f32=0, ids=A, plan=None):
    return any4.experts_gemm_dx_raw(0, dy, A, A, A, A, ids, plan, out, T, k, E, N, K, 128, ws, ws_bytes, stream=0, dx_f32=dx_f32,
                                    call="any4_experts_gemm_dx_parts")


def test_dx_of_parts():
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(N=0), dict(K=64), dict(T=1 << 20), dict(T=700000, k=1, N=1533)):
        assert dx(**bad) == 2, bad
        sizes = dict(T=100, k=2, E=4, N=16, K=128, g=128) | bad
        assert any4.experts_dx_parts_workspace_size(**sizes) == 0
    for name in ("dy", "out", "ids", "ws"):
        assert dx(**{name: None}) == 1
    assert dx(dy=A + 1) == 3 and dx(plan=A + 8) == 3 and dx(ws=A + 8) == 3 and dx(out=A + 2, dx_f32=1) == 3
    for N in (16, 17):
        need = any4.experts_dx_parts_workspace_size(100, 2, 4, N, 128, 128)
        assert need > any4.experts_dx_workspace_size(100, 2, 4, N, 128, 128) and dx(N=N, ws_bytes=need - 1) == 4
    assert dx(None, None, T=0, ws=None, ws_bytes=0, ids=None) == 0


def test_act_backward_in_parts():
    def call(dy=A, z=A, dz=A, dbias=A, act=2, gate=0, M=129, N=16, ws=A, ws_bytes=BIG):
        return any4.act_backward_raw(dy, z, dz, dbias, act, gate, M, N, ws, ws_bytes, stream=0, call="any4_act_backward_parts")
    for bad in (dict(M=-1), dict(N=-1), dict(M=(1 << 20) + 1), dict(M=1 << 20, N=1024), dict(act=5), dict(gate=1, N=15)):
        assert call(**bad) == 2, bad
    for name in ("dy", "z", "dz", "ws"):
        assert call(**{name: None}) == 1
    for name, off in (("dy", 1), ("z", 1), ("dz", 1), ("dbias", 2), ("ws", 8)):
        assert call(**{name: A + off}) == 3
    assert call(ws_bytes=any4.act_backward_workspace_size(129, 16, 0) - 1) == 4
    assert call(None, None, None, None, M=0, ws=None) == 0
