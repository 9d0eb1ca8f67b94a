"""Every form of the feed-forward products in every format: the sizes of test_ffn_forms.py, which
asserts the form that each reaches.  Tolerances as in test_gpu_ffn.py; rows in parts as in test_gpu_ffn_parts.py."""
import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu
from tests.test_ffn_forms import ACT, DX, DX_PARTS, EXPERTS, PARTS, even
from tests.test_gpu_ffn import FORMATS, call_of, choose, close, each_expert, expect, layers, normal, product
from tests.test_gpu_ffn_block import empty, near
from tests.test_gpu_ffn_parts import in_parts, rows, whole

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


@pytest.mark.parametrize("size", ACT)
@pytest.mark.parametrize("fmt", FORMATS)
def test_one_layer(fmt, size):
    M, N, K = size
    N = even(N)                     # the layer of both calls; without a gate its first size[1] rows
    packed, tables, w = layers(fmt, 1, N, K, 128)
    n = size[1]
    assert (n + 15) // 16 == (N + 15) // 16
    x, b, r = normal(M + N, M, K), normal(3, N), normal(4, M, N // 2)
    ref, e = product(x.double(), w[0], b)
    cut = [t[0, :n].contiguous() for t in tables]
    z, out = empty(M, n), empty(M, n)
    call_of(fmt, "act")(x, packed, *cut, 128, bias=b[:n].contiguous(), act="relu", z=z, out=out)
    near(z, ref[:, :n], e[:, :n], "z")
    near(out, *expect(ref[:, :n], e[:, :n], "relu", False), "out")
    z = empty(M, N, dtype=torch.bfloat16)
    out = call_of(fmt, "act")(x, packed, *[t[0] for t in tables], 128, bias=b, act="silu", gate=True, residual=r, z=z)
    near(z, ref, e, "gated z")
    near(out, *expect(ref, e, "silu", True, r), "gated out")


@pytest.mark.parametrize("parts,size", [(False, s) for s in EXPERTS] + [(True, s) for s in PARTS])
@pytest.mark.parametrize("fmt", FORMATS)
def test_experts(fmt, parts, size):
    T, k, E, N, K = size
    packed, tables, w = layers(fmt, E, N, K, 128)
    ids, b = choose(T, k, E), normal(8, E, N)
    x = in_parts(rows(7, T, k, K)) if parts else normal(7, T, K)
    wide = whole(x) if parts else x.double()[:, None].expand(T, k, K)
    ref, e = each_expert(wide, w, ids, bias=b)
    e = 2 * e if parts else e
    z, out = empty(T, k, N), empty(T, k, N)
    call_of(fmt, "experts")(x, packed, *tables, 128, ids, bias=b, act="relu", z=z, out=out)
    live = ((ids >= 0) & (ids < E))[:, :, None]
    near(z, ref, e, "z")
    want, eo = expect(ref, e, "relu", False)
    near(out, torch.where(live, want, torch.zeros_like(want)), eo, "out")
    assert not (out * ~live).any()


@pytest.mark.parametrize("parts,size", [(False, s) for s in EXPERTS] + [(True, s) for s in PARTS])
@pytest.mark.parametrize("fmt", FORMATS)
def test_experts_gated(fmt, parts, size):
    T, k, E, N, K = size
    N = even(N)
    packed, tables, w = layers(fmt, E, N, K, 128)
    ids = choose(T, k, E)
    x = in_parts(rows(7, T, k, K)) if parts else normal(7, T, K)
    wide = whole(x) if parts else x.double()[:, None].expand(T, k, K)
    ref, e = each_expert(wide, w, ids)
    e = 2 * e if parts else e
    out = call_of(fmt, "experts")(x, packed, *tables, 128, ids, act="silu", gate=True, plan=any4.experts_plan(ids, E))
    live = ((ids >= 0) & (ids < E))[:, :, None]
    want, eo = expect(ref, e, "silu", True)
    close(out, torch.where(live, want, torch.zeros_like(want)), eo)


@pytest.mark.parametrize("parts,size", [(False, s) for s in DX] + [(True, s) for s in DX_PARTS])
@pytest.mark.parametrize("fmt", FORMATS)
def test_dx(fmt, parts, size):
    T, k, E, N, K = size
    packed, tables, w = layers(fmt, E, N, K, 128)
    ids = choose(T, k, E)
    dy = in_parts(rows(9, T, k, N)) if parts else normal(9, T, k, N)
    want, e = each_expert(whole(dy) if parts else dy.double(), w, ids, back=True)
    for kind in (torch.float32, torch.bfloat16):
        out = empty(T, k, K, dtype=kind)
        call_of(fmt, "dx")(dy, packed, *tables, 128, ids, out=out)
        near(out, want, 2 * e if parts else e)
