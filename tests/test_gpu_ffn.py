"""Products with an epilogue, one layer or many experts', against the formulas
in 64 bits with the oracle's weights.

Tolerances.  Products of bf16 values are exact; the fp32 sum of n terms is off by
at most 2 (n + 16) 2^-24 of the sum of magnitudes (one bit for sums that are cut
rather than rounded), bias and residual are two more terms.  An activation passes
an error e of z on as at most 1.2 e (the largest slope of the five is 1.13) and adds
its own, at most 2^-20 (1 + |z|): a few rounded fp32 steps, each of 2^-24, in values of up
to 1 + |z|.  A gate multiplies both.  A bf16 result is off by another 2^-8 of itself."""
import functools
import math

import numpy as np
import pytest
import torch

import gemm_any4_amd as any4
import oracle
import workloads
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

FORMATS = ["any4", "int4", "any2", "any3"]
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


@functools.lru_cache(maxsize=8)
def layers(fmt, E, N, K, g, seed=5):
    """(packed bytes, tables, weights [E, N, K] in 64 bits) of E layers of a format."""
    packed, lut, alpha, beta, ws = [], [], [], [], []
    for e in range(E):
        inp = workloads.generic(seed + 17 * e, 1, N, K, g)
        codes = {"any2": inp.idx & 3, "any3": inp.idx & 7}.get(fmt, inp.idx).astype(np.uint8)
        pack = {"any2": lambda c: oracle.tile2(oracle.pack2(c)), "any3": oracle.tile3}.get(
            fmt, lambda c: oracle.tile(oracle.pack(c)))
        packed.append(gu.dev_u8(pack(codes)).reshape(-1))
        table = inp.lut
        if fmt == "int4":
            table = np.broadcast_to(oracle.f32_to_bf16(np.arange(16, dtype=np.float32)), (N, 16)).copy()
        ws.append(gu.dev_b16(oracle.dequant(oracle.pack(codes), table, inp.alpha, inp.beta, g)).double())
        lut.append(gu.dev_b16(inp.lut))
        alpha.append(gu.dev_b16(inp.alpha))
        beta.append(gu.dev_b16(inp.beta))
    tables = ((torch.stack(lut),) if fmt != "int4" else ()) + (torch.stack(alpha), torch.stack(beta))
    return torch.cat(packed), tables, torch.stack(ws)


def normal(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).to(gu.DEV)


def f64(act, z):
    """(act(z), act'(z)) in 64 bits."""
    one = torch.ones_like(z)
    if act == "none":
        return z, one
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        p = torch.special.expit(z)
        return z * p, p * (1 + z * (1 - p))
    if act == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c, d = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(c * (z + d * z ** 3))
    return z * (1 + t) / 2, (1 + t) / 2 + z / 2 * (1 - t * t) * c * (1 + 3 * d * z * z)


def expect(z, ez, act, gate, residual=None):
    """(out, its error before rounding) for z with errors ez."""
    if gate:
        F = z.shape[-1] // 2
        a, u, ea, eu = z[..., :F], z[..., F:], ez[..., :F], ez[..., F:]
    else:
        a, u, ea, eu = z, torch.ones_like(z), ez, torch.zeros_like(z)
    f = f64(act, a)[0]
    ef = 1.2 * ea + (0 if act in ("none", "relu") else 2.0 ** -20 * (1 + a.abs()))
    out, e = f * u, ef * (u.abs() + eu) + f.abs() * eu
    if gate:
        e = e + 2.0 ** -23 * out.abs()
    if residual is not None:
        out = out + residual.double()
        e = e + 2.0 ** -23 * (out.abs() + residual.double().abs())
    return out, e


def product(x, w, bias=None):
    """(z, its error) of x [M, K] and w [N, K] in 64 bits."""
    z, mag = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    return z, 2 * (w.shape[1] + 16) * 2.0 ** -24 * mag


def close(got, want, e, what=""):
    assert got.dtype == torch.bfloat16 and got.shape == want.shape
    bad = ~((got.double() - want).abs() <= e + 2.0 ** -8 * (want.abs() + e))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}"


def call_of(fmt, kind):
    names = {"act": ["gemm_act", "gemm_int4_act", "any2_gemm_act", "any3_gemm_act"],
             "experts": ["experts_gemm", "experts_gemm_int4", "any2_experts_gemm", "any3_experts_gemm"],
             "dx": ["experts_gemm_dx", "experts_gemm_int4_dx", "any2_experts_gemm_dx", "any3_experts_gemm_dx"]}[kind]
    return getattr(any4, names[FORMATS.index(fmt)])


def run_act(fmt, M, N, K, g, act, gate, bias, residual, keep):
    packed, tables, w = layers(fmt, 1, N, K, g)
    x = normal(M + N, M, K)
    No = N // 2 if gate else N
    b = normal(3, N) if bias else None
    r = normal(4, M, No, std=4.0) if residual else None
    z = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=gu.DEV) if keep else None
    out = call_of(fmt, "act")(x, packed, *[t[0] for t in tables], g, bias=b, act=act, gate=gate, residual=r, z=z)
    ref, e = product(x.double(), w[0], b)
    if keep:
        close(z, ref, e, "z")
    close(out, *expect(ref, e, act, gate, r), "out")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K,g", [(1, 1, 128, 128), (1, 64, 256, 256), (3, 100, 384, 128), (5, 37, 256, 128),
                                     (16, 130, 512, 512), (17, 64, 128, 128), (33, 200, 384, 384), (65, 77, 256, 128),
                                     (129, 1030, 256, 128), (300, 1100, 384, 128), (257, 1024, 128, 128)])
def test_formats_and_odd_sizes(fmt, M, N, K, g):
    """Every tile size, last rows and columns that are not whole, one split and several."""
    run_act(fmt, M, N, K, g, "none", False, True, False, True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("M,N", [(1, 98), (9, 96), (40, 1154), (300, 2050)])
def test_epilogues(act, gate, M, N):
    run_act("any4", M, N, 256, 128, act, gate, False, True, True)
    run_act("any4", M, N, 256, 128, act, gate, True, False, False)


@pytest.mark.parametrize("M,N,K,g", [(1, 4096, 4096, 128), (16, 4096, 14336, 1024), (4, 512, 8192, 128), (20, 96, 8192, 256),
                                     (100, 640, 4096, 128), (1, 14336, 512, 128), (1030, 2048, 1024, 256)])
def test_larger_sizes(M, N, K, g):
    """Sums split over workgroups and joined."""
    run_act("any4", M, N, K, g, "silu", True, True, True, True)
    run_act("any4", M, N - 1, K, g, "gelu", False, True, True, True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 4, 16, 32, 128])
def test_one_hot_rows_give_the_weights(fmt, M):
    """Unit vectors: z is W itself, bit for bit."""
    packed, tables, w = layers(fmt, 1, 70, 256, 128)
    call = call_of(fmt, "act")
    for k0 in range(0, 256, M):
        x = torch.zeros((M, 256), dtype=torch.bfloat16, device=gu.DEV)
        n = min(M, 256 - k0)
        x[torch.arange(n), k0 + torch.arange(n)] = 1.0
        assert torch.equal(call(x, packed, *[t[0] for t in tables], 128)[:n].double(), w[0, :, k0:k0 + n].t())


@pytest.mark.parametrize("M", [3, 16, 40, 300])
def test_rows_do_not_touch_each_other(M):
    packed, tables, _ = layers("any4", 1, 100, 256, 128)
    tables = [t[0] for t in tables]
    x = normal(1, M, 256)
    clean = any4.gemm_act(x, packed, *tables, 128, act="silu")
    x[1] = float("nan")
    x[M - 1, 3] = float("inf")
    got = any4.gemm_act(x, packed, *tables, 128, act="silu")
    keep = torch.ones(M, dtype=torch.bool, device=gu.DEV)
    keep[1] = keep[M - 1] = False
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[M - 1]).all()


def test_residual_in_place_and_unaligned_outputs():
    packed, tables, _ = layers("any4", 1, 96, 256, 128)
    tables = [t[0] for t in tables]
    for M in (2, 50):
        x, r = normal(1, M, 256), normal(2, M, 96)
        want = any4.gemm_act(x, packed, *tables, 128, act="relu", residual=r)
        room = torch.zeros(M * 96 + 3, dtype=torch.bfloat16, device=gu.DEV)
        out = room[1:1 + M * 96].view(M, 96)
        out.copy_(r)
        got = any4.gemm_act(x, packed, *tables, 128, act="relu", residual=out, out=out)
        assert got is out and torch.equal(out, want)
        assert room[0] == 0 and (room[-2:] == 0).all()


def test_empty_calls():
    packed, tables, _ = layers("any4", 1, 96, 256, 128)
    tables = [t[0] for t in tables]
    x = normal(1, 0, 256)
    assert any4.gemm_act(x, packed, *tables, 128, gate=True).shape == (0, 48)
    dz, dbias = any4.act_backward(normal(1, 0, 48), normal(1, 0, 96), "silu", gate=True)
    assert dz.shape == (0, 96) and torch.equal(dbias, torch.zeros(96, device=gu.DEV))


# ---------------------------------------------------------------------------
# the activation's backward pass
# ---------------------------------------------------------------------------
def check_backward(M, N, act, gate):
    No = N // 2 if gate else N
    z, dy = normal(5, M, N, std=2.0), normal(6, M, No)
    dz, dbias = any4.act_backward(dy, z, act, gate=gate)
    zd, d = z.double(), dy.double()
    if gate:
        a, u = zd[:, :No], zd[:, No:]
        f, slope = f64(act, a)
        want = torch.cat([d * u * slope, d * f], dim=1)
        scale = torch.cat([(d * u).abs(), d.abs()], dim=1) * (1 + zd[:, :No].abs().repeat(1, 2))
    else:
        want = d * f64(act, zd)[1]
        scale = d.abs() * (1 + zd.abs())
    # a few rounded fp32 steps in values of up to 1.2 (1 + |z|) beside the factors
    e = 2.0 ** -19 * scale
    close(dz, want, e, "dz")
    err = (dbias.double() - want.sum(dim=0)).abs()
    assert (err <= e.sum(dim=0) + (M + 16) * 2.0 ** -24 * want.abs().sum(dim=0)).all()
    none, nothing = any4.act_backward(dy, z, act, gate=gate, need_bias=False)
    assert nothing is None and torch.equal(none, dz)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("M,N", [(1, 2), (5, 34), (64, 512), (33, 1030), (128, 98), (129, 98), (257, 2050), (1000, 130)])
def test_act_backward(act, gate, M, N):
    check_backward(M, N, act, gate)


def test_act_backward_long():
    check_backward(5000, 4100, "silu", True)
    check_backward(3, 30001, "gelu", False)


def test_act_backward_in_place_and_shapes():
    z, dy = normal(5, 6, 3, 64), normal(6, 6, 3, 32)
    want, wb = any4.act_backward(dy, z, "gelu_tanh", gate=True)
    copy = z.clone()
    got, gb = any4.act_backward(dy, copy, "gelu_tanh", gate=True, dz=copy)
    assert got is copy and torch.equal(copy, want) and torch.equal(gb, wb)


@pytest.mark.parametrize("act", ACTS[1:])
def test_slopes_against_differences(act):
    """dz for dy = 1 against differences of the formula in 64 bits."""
    z = torch.linspace(-8, 8, 4096).to(torch.bfloat16).to(gu.DEV).view(1, -1)
    z = z[:, z[0].double().abs() > 2.0 ** -9]
    dz, _ = any4.act_backward(torch.ones_like(z), z, act)
    h = 2.0 ** -16
    want = (f64(act, z.double() + h)[0] - f64(act, z.double() - h)[0]) / (2 * h)
    # h^2 / 6 times a third derivative below 4, and the rounding to bf16
    close(dz, want, torch.full_like(want, h * h + 2.0 ** -17))


@pytest.mark.parametrize("act", ACTS)
def test_values_far_out(act):
    """Up to the largest finite ones an activation and its slope are those of z or of 0.
    At |z| = 30 silu and its slope are off by |z| e^-|z| < 30 * 9.4e-14 < 2^-38, the others
    and values farther out by less; all factors here are at most 1."""
    same = lambda got, want: bool(((got - want).abs() <= 2.0 ** -38).all())      # noqa: E731
    z = torch.tensor([[s * v for v in (30.0, 1e4, 1e13, 1e19, 3e19, 1e30, 3e38) for s in (1, -1)]], dtype=torch.bfloat16, device=gu.DEV)
    up = act == "none"
    dz, dbias = any4.act_backward(torch.ones_like(z), z, act)
    want = ((z > 0) | up).float()
    assert same(dz.float(), want) and same(dbias, want[0])
    gated = torch.cat([z, torch.full_like(z, 0.5)], dim=1)
    dz = any4.act_backward(torch.full_like(z, 2.0 ** -8), gated, act, gate=True)[0].float()
    assert same(dz[:, :14], want * 2.0 ** -9) and same(dz[:, 14:], want * z.float() * 2.0 ** -8)
    # an identity layer: forward
    one = lambda v: torch.full((16, 1), v, dtype=torch.bfloat16, device=gu.DEV)      # noqa: E731
    packed = any4.pack(torch.zeros((16, 128), dtype=torch.uint8, device=gu.DEV))
    lut = torch.ones((16, 16), dtype=torch.bfloat16, device=gu.DEV)
    x = torch.zeros((14, 128), dtype=torch.bfloat16, device=gu.DEV)
    x[:, 5] = z[0]
    assert same(any4.gemm_act(x, packed, lut, one(1.0), one(0.0), 128, act=act)[:, 3].float(), (want * z.float())[0])


# ---------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------
def choose(T, k, E, seed=1, empty=True):
    """ids: mostly distinct experts, some pairs without one, one expert named twice."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(max(E, k), generator=g)[:k] % E for _ in range(T)]).to(torch.int32)
    if empty and T > 2:
        ids[torch.rand(T, k, generator=g) < 0.1] = -1
        ids[1, 0] = E
        if k > 1:
            ids[2] = ids[2, 0]
    return ids.to(gu.DEV)


def each_expert(x, w, ids, back=False, bias=None):
    """(z, its error) [T, k, .] of x [T, k, .] in 64 bits; zeros where there is no expert."""
    T, k = ids.shape
    flat, x = ids.reshape(-1).long(), x.reshape(T * k, -1)
    z = torch.zeros((T * k, w.shape[2] if back else w.shape[1]), dtype=torch.float64, device=gu.DEV)
    e = torch.zeros_like(z)
    for i in range(w.shape[0]):
        rows = (flat == i).nonzero().flatten()
        z[rows], e[rows] = product(x[rows], w[i].t() if back else w[i], None if bias is None else bias[i])
    return z.view(T, k, -1), e.view(T, k, -1)


def check_experts(fmt, T, k, E, N, K, g, act="none", gate=False, per_pair=False, bias=False, keep=False, plan=False, ids=None):
    packed, tables, w = layers(fmt, E, N, K, g)
    ids = choose(T, k, E) if ids is None else ids
    x = normal(7, T, k, K) if per_pair else normal(7, T, K)
    b = normal(8, E, N) if bias else None
    z = torch.full((T, k, N), 7.0, dtype=torch.bfloat16, device=gu.DEV) if keep else None
    out = call_of(fmt, "experts")(x, packed, *tables, g, ids, bias=b, act=act, gate=gate, z=z,
                                  plan=any4.experts_plan(ids, E) if plan else None)
    wide = x.double() if per_pair else x.double()[:, None].expand(T, k, K)
    ref, e = each_expert(wide, w, ids, bias=b)
    if keep:
        close(z, ref, e, "z")
    want, eo = expect(ref, e, act, gate)
    live = (ids >= 0) & (ids < E)
    close(out, torch.where(live[:, :, None], want, torch.zeros_like(want)), eo, "out")
    assert (out[~live] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,k,E,N,K,g", [(1, 1, 1, 1, 128, 128), (1, 2, 8, 96, 256, 128), (5, 3, 7, 50, 384, 128),
                                         (30, 2, 4, 64, 256, 256), (33, 2, 16, 72, 128, 128), (70, 4, 3, 130, 256, 128),
                                         (150, 2, 5, 40, 256, 128), (400, 2, 3, 1030, 128, 128)])
def test_experts(fmt, T, k, E, N, K, g):
    check_experts(fmt, T, k, E, N, K, g, bias=True, keep=True)


@pytest.mark.parametrize("T,k,E,N,K", [(3, 2, 4, 98, 256), (40, 4, 30, 98, 256), (100, 2, 2, 1026, 128), (600, 2, 2, 2050, 256)])
@pytest.mark.parametrize("plan", [False, True])
def test_experts_gated(T, k, E, N, K, plan):
    check_experts("any4", T, k, E, N, K, 128, act="silu", gate=True, keep=True, plan=plan)
    check_experts("any4", T, k, E, N, K, 128, act="gelu", per_pair=True, bias=True, plan=plan)


def test_experts_with_one_expert_for_all_and_none():
    for T in (8, 64, 300):
        check_experts("any4", T, 2, 70, 64, 128, 128, ids=torch.full((T, 2), 69, dtype=torch.int32, device=gu.DEV))
        check_experts("any4", T, 2, 70, 64, 128, 128, ids=torch.full((T, 2), -1, dtype=torch.int32, device=gu.DEV))


def test_many_experts():
    check_experts("any4", 200, 2, 300, 32, 128, 128)
    check_experts("any4", 2000, 4, 300, 32, 128, 128, plan=True)


def test_experts_split_sums():
    check_experts("any4", 2, 2, 4, 66, 8192, 128, act="silu", gate=True, keep=True)
    check_experts("any4", 200, 1, 2, 130, 4096, 256, bias=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,k,E,N,K,g", [(1, 1, 1, 1, 128, 128), (1, 2, 8, 96, 256, 128), (5, 3, 7, 50, 384, 128),
                                         (33, 2, 16, 72, 128, 128), (70, 4, 3, 131, 256, 128), (400, 2, 2, 200, 1152, 128)])
def test_experts_dx(fmt, T, k, E, N, K, g):
    packed, tables, w = layers(fmt, E, N, K, g)
    ids, dy = choose(T, k, E), normal(9, T, k, N)
    want, e = each_expert(dy.double(), w, ids, back=True)
    for plan in (None, any4.experts_plan(ids, E)):
        close(call_of(fmt, "dx")(dy, packed, *tables, g, ids, plan=plan), want, e)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("N", [96, 100])
def test_experts_dx_gives_the_weights(fmt, N):
    packed, tables, w = layers(fmt, 2, N, 256, 128)
    ids = torch.tensor([[0, 1]], dtype=torch.int32, device=gu.DEV).repeat(N, 1)
    dy = torch.eye(N, dtype=torch.bfloat16, device=gu.DEV)[:, None].repeat(1, 2, 1)
    got = call_of(fmt, "dx")(dy, packed, *tables, 128, ids)
    assert torch.equal(got.double(), w.transpose(0, 1))


def test_experts_dx_rows_do_not_touch_each_other():
    packed, tables, _ = layers("any4", 3, 100, 256, 128)
    ids = choose(60, 2, 3, empty=False)
    dy = normal(9, 60, 2, 100)
    clean = any4.experts_gemm_dx(dy, packed, *tables, 128, ids)
    dy[4, 1] = float("nan")
    got = any4.experts_gemm_dx(dy, packed, *tables, 128, ids)
    keep = torch.ones(60, 2, dtype=torch.bool, device=gu.DEV)
    keep[4, 1] = False
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[4, 1]).all()
