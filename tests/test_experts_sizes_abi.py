"""Rows of x that the pairs of a token share count once (CPU only)."""
import gemm_any4_amd as any4
from tests.test_ffn_abi import A, BIG, experts

LONG = dict(T=1 << 15, k=8, E=8, N=16, K=4096, g=128)       # T K = 2^27, T k K = 2^30


def test_the_size_query_knows_what_the_call_takes():
    need = any4.experts_workspace_size(**LONG)
    assert need >= any4.lora_plan_bytes(1 << 18, 8)
    assert experts(**LONG, ws_bytes=need - 1) == 4 and experts(**LONG, ws=None) == 1
    assert experts(**LONG, per_pair=1) == 2 and any4.experts_parts_workspace_size(**LONG) == 0
    more = LONG | dict(T=1 << 16, K=16384)
    assert any4.experts_workspace_size(**more) == 0 and experts(**more, ws_bytes=BIG, x=A) == 2
