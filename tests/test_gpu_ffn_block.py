"""The feed-forward calls at the sizes of every form of their products, with results
kept in fp32, in a row as a block runs them, captured, on other streams and at
their limits; against the formulas in 64 bits with the oracle's weights.

Tolerances are those of test_gpu_ffn.py; an fp32 result is off by another 2^-24 of
itself instead of a bf16 one's 2^-8.  What a block's run adds up to is worked out
beside its formulas: every stage passes the errors of its inputs on."""
import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu
from tests.test_gpu_ffn import call_of, choose, close, each_expert, expect, f64, layers, normal, product

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


def near(got, want, e, what=""):
    if got.dtype is torch.bfloat16:
        return close(got, want, e, what)
    assert got.dtype is F32 and got.shape == want.shape
    bad = ~((got.double() - want).abs() <= e + 2.0 ** -24 * (want.abs() + e))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}"


def empty(*shape, dtype=F32):
    return torch.full(shape, 7.0, dtype=dtype, device=gu.DEV)


# ---------------------------------------------------------------------------
# every form: few rows and tiles of four sizes, laid out first or not, with split sums
# and without
# ---------------------------------------------------------------------------
def check_act(M, N, K, act="none", gate=False, kind=F32, fmt="any4"):
    packed, tables, w = layers(fmt, 1, N, K, 128)
    x, b = normal(M + N, M, K), normal(3, N)
    No = N // 2 if gate else N
    z, out = empty(M, N, dtype=kind), empty(M, No, dtype=kind)
    call_of(fmt, "act")(x, packed, *[t[0] for t in tables], 128, bias=b, act=act, gate=gate, z=z, out=out)
    ref, e = product(x.double(), w[0], b)
    near(z, ref, e, "z")
    near(out, *expect(ref, e, act, gate), "out")


@pytest.mark.parametrize("M,N,K", [(100, 98, 256), (520, 98, 8192), (700, 258, 4096), (100, 98, 4096), (100, 97, 128),
                                   (520, 97, 4096), (1300, 1538, 128), (330, 1538, 2048), (1300, 4098, 128), (4100, 258, 2048),
                                   (1300, 8194, 128), (130, 8194, 4096), (2050, 98, 128), (2050, 97, 4096)])
def test_forms(M, N, K):
    check_act(M, N, K)
    if N % 2 == 0:
        check_act(M, N, K, "silu", True, kind=torch.bfloat16)


@pytest.mark.parametrize("fmt", ["any4", "int4", "any2", "any3"])
@pytest.mark.parametrize("M,N,K", [(4100, 6147, 1024), (4100, 515, 8192)])
def test_layers_laid_out_first(fmt, M, N, K):
    assert any4.gemm_act_workspace_size(M, N, K, 128) >= 2 * N * K
    check_act(M, N, K, "gelu_tanh", kind=F32 if fmt == "any4" else torch.bfloat16, fmt=fmt)


def check_experts(T, k, E, N, K, act="none", gate=False, kind=F32):
    packed, tables, w = layers("any4", E, N, K, 128)
    ids, x, b = choose(T, k, E), normal(7, T, K), normal(8, E, N)
    z, out = empty(T, k, N, dtype=kind), empty(T, k, N // 2 if gate else N, dtype=kind)
    any4.experts_gemm(x, packed, *tables, 128, ids, bias=b, act=act, gate=gate, z=z, out=out)
    ref, e = each_expert(x.double()[:, None].expand(T, k, K), w, ids, bias=b)
    near(z, ref, e, "z")
    live = ((ids >= 0) & (ids < E))[:, :, None]
    want, eo = expect(ref, e, act, gate)
    near(out, torch.where(live, want, torch.zeros_like(want)), eo, "out")
    assert not (out * ~live).any()


@pytest.mark.parametrize("T,k,E,N,K", [(50, 2, 2, 98, 256), (20, 5, 5, 514, 8192), (20, 5, 5, 1538, 4096), (50, 2, 2, 98, 4096),
                                       (50, 2, 2, 98, 128), (65, 2, 2, 98, 1024), (650, 2, 2, 1538, 128), (165, 2, 2, 1538, 2048),
                                       (650, 2, 2, 4098, 128), (2050, 2, 2, 258, 2048), (650, 2, 2, 8194, 128),
                                       (650, 2, 2, 1538, 4096), (65, 2, 2, 98, 128), (40, 5, 5, 8194, 128),
                                       (820, 5, 5, 98, 2048)])
def test_forms_of_experts(T, k, E, N, K):
    check_experts(T, k, E, N, K)
    check_experts(T, k, E, N, K, "silu", True, kind=torch.bfloat16)


@pytest.mark.parametrize("T,k,E,N,K", [(50, 2, 2, 96, 128), (50, 2, 2, 1021, 128), (1025, 2, 2, 93, 1024), (66, 5, 5, 1536, 2048),
                                       (350, 2, 2, 96, 8192), (165, 2, 2, 2043, 4096),
                                       (1025, 2, 2, 96, 2048), (650, 2, 2, 4091, 384)])
@pytest.mark.parametrize("fmt", ["any4", "any3"])
def test_forms_of_dx(fmt, T, k, E, N, K):
    packed, tables, w = layers(fmt, E, N, K, 128)
    ids, dy = choose(T, k, E), normal(9, T, k, N)
    want, e = each_expert(dy.double(), w, ids, back=True)
    for kind in (F32, torch.bfloat16):
        out = empty(T, k, K, dtype=kind)
        assert call_of(fmt, "dx")(dy, packed, *tables, 128, ids, out=out) is out
        near(out, want, e)


@pytest.mark.parametrize("fmt", ["any4", "int4", "any2", "any3"])
@pytest.mark.parametrize("T,k,E,N,K", [(1, 1, 1, 1, 128), (1, 2, 8, 96, 384), (6, 3, 5, 50, 256), (32, 2, 3, 130, 4096), (64, 1, 1, 33, 256),
                                       (2, 2, 4, 66, 8192), (16, 4, 20, 2050, 512)])
def test_fp32_rows(fmt, T, k, E, N, K):
    """At least 16 bits of a value enter: 2^-16 of its magnitude is left out."""
    packed, tables, w = layers(fmt, E, N, K, 128)
    ids = choose(T, k, E)
    gen = torch.Generator().manual_seed(T)
    for shape in ((T, K), (T, k, K)):
        x = torch.randn(*shape, generator=gen).to(gu.DEV)
        out = empty(T, k, N)
        call_of(fmt, "experts")(x, packed, *tables, 128, ids, out=out)
        wide = x.double() if len(shape) == 3 else x.double()[:, None].expand(T, k, K)
        want, e = each_expert(wide, w, ids)
        # twice as many terms as the bound of a bf16 row's
        near(out, want, 2 * e + 2.0 ** -16 * each_expert(wide.abs(), w.abs(), ids)[0])


def test_fp32_rows_that_are_not_finite():
    """The formulas' infinities and NaN, and values beyond bf16's largest."""
    packed, tables, w = layers("any4", 2, 40, 256, 128)
    ids, x = torch.tensor([[0, 1]] * 5, dtype=torch.int32, device=gu.DEV), torch.randn(5, 256, device=gu.DEV)
    x[1, 7], x[2, 9], x[3, 200], x[4] = float("inf"), float("-inf"), float("nan"), 0.0
    x[4, 3] = torch.finfo(F32).max
    out = empty(5, 2, 40)
    any4.experts_gemm(x, packed, *tables, 128, ids, out=out)
    for j in range(2):
        for t, k in ((1, 7), (2, 9)):
            assert torch.equal(out[t, j], (x[t, k].double() * w[j, :, k]).float())
    assert torch.isnan(out[3]).all() and torch.isfinite(out[0]).all()
    want = x[4, 3].double() * torch.stack([w[j, :, 3] for j in range(2)])
    small = want.abs() < 3e38
    assert small.any() and ((out[4].double() - want).abs()[small] <= 2.0 ** -15 * want.abs()[small]).all()
    with pytest.raises(ValueError):
        any4.experts_gemm(x.repeat(7, 1), packed, *tables, 128, ids.repeat(7, 1))


def test_fp32_results_at_odd_places():
    """fp32 rows that start 4 bytes off a piece of 16."""
    packed, tables, w = layers("any4", 1, 75, 256, 128)
    tables = [t[0] for t in tables]
    for M in (2, 50):
        room = empty(M * 75 + 2)
        out = room[1:-1].view(M, 75)
        x = normal(1, M, 256)
        any4.gemm_act(x, packed, *tables, 128, out=out)
        near(out, *product(x.double(), w[0]))
        assert room[0] == 7 and room[-1] == 7


# ---------------------------------------------------------------------------
# what the others read and write in fp32
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("kinds", [(F32, F32), (F32, torch.bfloat16), (torch.bfloat16, F32)])
@pytest.mark.parametrize("M,N", [(1, 2), (33, 1030), (40, 1024), (3, 4112)])
def test_act_backward_of_fp32(M, N, kinds, gate):
    No = N // 2 if gate else N
    gen = torch.Generator().manual_seed(M)
    dy = torch.randn(M, No, generator=gen).to(gu.DEV).to(kinds[0])
    z = (2 * torch.randn(M, N, generator=gen)).to(gu.DEV).to(kinds[1])
    dz, dbias = any4.act_backward(dy, z, "silu", gate=gate)
    d, a = dy.double(), z.double()[:, :No]
    f, slope = f64("silu", a)
    u = z.double()[:, No:] if gate else torch.ones_like(a)
    want, scale = d * u * slope, (d * u).abs() * (1 + a.abs())
    if gate:
        want, scale = torch.cat([want, d * f], 1), torch.cat([scale, d.abs() * (1 + a.abs())], 1)
    e = 2.0 ** -19 * scale          # as in test_gpu_ffn.py
    close(dz, want, e)
    assert ((dbias.double() - want.sum(0)).abs() <= e.sum(0) + (M + 16) * 2.0 ** -24 * want.abs().sum(0)).all()


@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (5, 3, 37), (9, 2, 2048), (33, 8, 130), (7, 9, 2056)])
def test_weighted_sums_of_fp32(T, k, N):
    gen = torch.Generator().manual_seed(T)
    y, w = torch.randn(T, k, N, generator=gen).to(gu.DEV), torch.rand(T, k, generator=gen).to(gu.DEV)
    r, dout = normal(2, T, N), normal(3, T, N)
    for weights in (w, None):
        p = y.double() * (1 if weights is None else w.double()[:, :, None])
        mag = p.abs().sum(1) + r.double().abs()
        close(any4.combine(y, weights, residual=r), p.sum(1) + r.double(), (k + 1) * 2.0 ** -24 * mag)
    dy, dw = any4.combine_backward(dout, y, w)
    close(dy, w.double()[:, :, None] * dout.double()[:, None], torch.zeros(T, k, N, device=gu.DEV))
    p = dout.double()[:, None] * y.double()
    assert ((dw.double() - p.sum(2)).abs() <= (N + 16) * 2.0 ** -24 * p.abs().sum(2)).all()


# ---------------------------------------------------------------------------
# a block of experts as a layer of a model runs it, forward and back
# ---------------------------------------------------------------------------
class Block:
    """x and logits -> x + sum_j w_j W2_e (silu(gate) up), e the j-th expert of a token."""

    def __init__(self, T, H, F, E, k, seed=3):
        self.T, self.H, self.F, self.E, self.k = T, H, F, E, k
        self.up, self.down = layers("any4", E, 2 * F, H, 128), layers("any4", E, H, F, 128, seed + 100)
        # tables and scales of O(1): weights of a size that keeps z of O(1)
        self.x, self.dout = normal(seed, T, H, std=0.05), normal(seed + 1, T, H)
        g = torch.Generator().manual_seed(seed)
        self.logits = torch.randn(T, E, generator=g).to(gu.DEV)
        self.bias = (0.1 * torch.randn(E, generator=g)).to(gu.DEV)

    def run(self, x, logits, **how):
        (w1, t1, _), (w2, t2, _) = self.up, self.down
        T, k = self.T, self.k
        w, ids = any4.route(logits, k, bias=self.bias, score="sigmoid", scale=2.5, **how)
        plan = any4.experts_plan(ids, self.E, **how)
        z, y, dh, dxp = (empty(T, k, n) for n in (2 * self.F, self.H, self.F, self.H))
        h = any4.experts_gemm(x, w1, *t1, 128, ids, act="silu", gate=True, z=z, plan=plan, **how)
        any4.experts_gemm(h, w2, *t2, 128, ids, plan=plan, out=y, **how)
        out = any4.combine(y, w, residual=x, **how)
        dy, dw = any4.combine_backward(self.dout, y, w, **how)
        any4.experts_gemm_dx(dy, w2, *t2, 128, ids, plan=plan, out=dh, **how)
        dz, dbias = any4.act_backward(dh, z, "silu", gate=True, **how)
        any4.experts_gemm_dx(dz, w1, *t1, 128, ids, plan=plan, out=dxp, **how)
        dx = any4.combine(dxp, residual=self.dout, **how)
        return dict(out=out, dx=dx, dlogits=any4.route_backward(dw, logits, ids, score="sigmoid", scale=2.5, **how),
                    dbias=dbias, w=w, ids=ids)


def weights64(logits, ids):
    s = torch.special.expit(logits.double()).gather(1, ids.long())
    return 2.5 * s / s.sum(1, keepdim=True), s


def forward64(b, x, logits, ids):
    w = weights64(logits, ids)[0]
    wide = x[:, None].expand(b.T, b.k, b.H)
    z = each_expert(wide, b.up[2], ids)[0]
    h = f64("silu", z[..., :b.F])[0] * z[..., b.F:]
    return x + (w[..., None] * each_expert(h, b.down[2], ids)[0]).sum(1)


@pytest.mark.parametrize("T,H,F,E,k", [(1, 128, 128, 4, 2), (7, 256, 128, 8, 3), (70, 256, 384, 5, 2), (600, 128, 256, 3, 2)])
def test_a_block_forward_and_back(T, H, F, E, k):
    b = Block(T, H, F, E, k)
    got = b.run(b.x, b.logits)
    ids = got["ids"]
    score = torch.special.expit(b.logits.double()) + b.bias.double()
    assert torch.equal(ids.long(), score.topk(k, dim=1)[1])
    x, dout, (w, s) = b.x.double(), b.dout.double(), weights64(b.logits, ids)
    ew = 2.0 ** -22 * w
    assert ((got["w"].double() - w).abs() <= ew).all()

    def experts(v, ev, layer, back=False):
        """A product and its error where the input has an error of its own."""
        r, e = each_expert(v, layer[2], ids, back=back)
        passed = each_expert(ev, layer[2].abs(), ids, back=back)[0]
        return r, 1.01 * e + 1.01 * passed      # the rounding of the sum is of v + ev
    z, ez = experts(x[:, None].expand(T, k, H), torch.zeros(T, k, H, dtype=torch.float64, device=gu.DEV), b.up)
    ez = ez + 2.0 ** -24 * z.abs()
    h, eh = expect(z, ez, "silu", True)
    eh = eh + 2.0 ** -8 * (h.abs() + eh)
    y, ey = experts(h, eh, b.down)
    ey = ey + 2.0 ** -24 * y.abs()
    p, ep = w[..., None] * y, (w + ew)[..., None] * ey + ew[..., None] * y.abs()
    mag = x.abs() + (p.abs() + ep).sum(1)
    close(got["out"], x + p.sum(1), ep.sum(1) + (k + 1) * 2.0 ** -24 * mag, "out")
    # back
    dy, edy = w[..., None] * dout[:, None], ew[..., None] * dout.abs()[:, None]
    edy = edy + 2.0 ** -8 * (dy.abs() + edy)
    dw = (dout[:, None] * y).sum(2)
    edw = (dout.abs()[:, None] * (ey + (H + 16) * 2.0 ** -24 * (y.abs() + ey))).sum(2)
    dh, edh = experts(dy, edy, b.down, back=True)
    edh = edh + 2.0 ** -24 * dh.abs()
    a, u, ea, eu = z[..., :F], z[..., F:], ez[..., :F], ez[..., F:]
    f, slope = f64("silu", a)
    da, du = dh * u * slope, dh * f
    # silu'' is at most 1/2, silu' 1.1
    eda = (dh.abs() + edh) * (u.abs() + eu) * (slope.abs() + ea / 2) - da.abs() + 2.0 ** -18 * (dh * u).abs() * (1 + a.abs())
    edu = (dh.abs() + edh) * (f.abs() + 1.2 * ea) - du.abs() + 2.0 ** -18 * dh.abs() * (1 + a.abs())
    dz, edz = torch.cat([da, du], 2), torch.cat([eda, edu], 2)
    wide, ewide = dz.reshape(T * k, -1), edz.reshape(T * k, -1)
    assert ((got["dbias"].double() - wide.sum(0)).abs()
            <= ewide.sum(0) + (T * k + 16) * 2.0 ** -24 * (wide.abs() + ewide).sum(0)).all()
    edz = edz + 2.0 ** -8 * (dz.abs() + edz)
    dxp, edxp = experts(dz, edz, b.up, back=True)
    edxp = edxp + 2.0 ** -24 * dxp.abs()
    dx = dout + dxp.sum(1)
    close(got["dx"], dx, edxp.sum(1) + (k + 1) * 2.0 ** -24 * ((dxp.abs() + edxp).sum(1) + dout.abs()), "dx")
    S = s.sum(1)[:, None, None]
    J = 2.5 * (torch.diag_embed(s * (1 - s)) / S - s[:, :, None] * (s * (1 - s))[:, None, :] / S ** 2)     # d w_j / d l_i
    dl, edl = torch.zeros(T, E, dtype=torch.float64, device=gu.DEV), torch.zeros(T, E, dtype=torch.float64, device=gu.DEV)
    dl.scatter_(1, ids.long(), (dw[:, None] @ J)[:, 0])
    edl.scatter_(1, ids.long(), ((edw + 2.0 ** -22 * dw.abs())[:, None] @ J.abs())[:, 0])
    near(got["dlogits"], dl, edl, "dlogits")
    # the formulas against differences of the forward pass: central ones of steps h = 1e-5 are off by
    # h^2 times third derivatives and 2^-52 / h of the values, both far below 1e-6 of the magnitudes
    gen = torch.Generator().manual_seed(9)
    vx, vl = torch.randn(T, H, generator=gen).double().to(gu.DEV), torch.randn(T, E, generator=gen).double().to(gu.DEV)
    step = 1e-5
    up, down = (forward64(b, x + t * vx, b.logits.double() + t * vl, ids) for t in (step, -step))
    slope = ((up - down) / (2 * step) * dout).sum()
    want = (dx * vx).sum() + (dl * vl).sum()
    assert (slope - want).abs() <= 1e-6 * ((dx * vx).abs().sum() + (dl * vl).abs().sum())


@pytest.mark.parametrize("T", [9, 150])
def test_a_block_captured_and_replayed(T):
    """Every replay gives the eager run's bits, with other work between them."""
    b = Block(T, 256, 128, 6, 3)
    x, logits = b.x.clone(), b.logits.clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    b.run(x, logits)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        kept = b.run(x, logits)
    for i in range(4):
        x.copy_(normal(50 + i, T, 256, std=0.05))
        logits.copy_(b.logits.roll(i, dims=1))
        want = b.run(x, logits)
        graph.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(kept[name], want[name]), (i, name)


def test_a_block_on_other_streams():
    b = Block(40, 256, 128, 6, 3)
    want = b.run(b.x, b.logits)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(6):              # two blocks at a time
        with torch.cuda.stream(streams[i % 2]):
            got.append(b.run(b.x, b.logits))
    torch.cuda.synchronize()
    got.append(b.run(b.x, b.logits, stream=streams[0]))
    torch.cuda.synchronize()
    for g in got:
        for name in want:
            assert torch.equal(g[name], want[name]), name


# ---------------------------------------------------------------------------
# plans, workspaces
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,k,N,K", [(50, 2, 98, 256), (50, 2, 98, 4096), (50, 2, 98, 128), (65, 2, 98, 1024)])
def test_a_plan_of_other_sizes_leaves_the_results(T, k, N, K):
    """Few rows and tiles, with split sums and without."""
    E = 2
    packed, (lut, alpha, beta), _ = layers("any4", E, N, K, 128)
    ids, x, dy = choose(T, k, E), normal(7, T, K), normal(9, T, k, N)
    wrong = [any4.experts_plan(choose(T + 1, k, E), E), any4.experts_plan(ids, E + 1), any4.experts_plan(ids[:3], E)]
    with pytest.raises(ValueError):
        any4.experts_gemm(x, packed, lut, alpha, beta, 128, ids, plan=wrong[0])
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=gu.DEV)
    for plan in wrong:
        z, out, dx = empty(T, k, N), empty(T, k, N), empty(T, k, K)
        p = plan.words.data_ptr()
        layer = [t.data_ptr() for t in (packed, lut, alpha, beta)]
        sizes = (T, k, E, N, K, 128, ws.data_ptr(), ws.numel())
        assert any4.experts_gemm_raw(0, x.data_ptr(), 0, *layer, None, ids.data_ptr(), p, z.data_ptr(), out.data_ptr(), 0, 0,
                                     *sizes, z_f32=1, out_f32=1) == 0
        assert any4.experts_gemm_dx_raw(0, dy.data_ptr(), *layer, ids.data_ptr(), p, dx.data_ptr(), *sizes, dx_f32=1) == 0
        for t in (z, out, dx):
            assert (t == 7).all()


def test_workspaces_of_the_callers():
    """Exactly as large as asked for, with others' bytes behind; and too small."""
    packed, tables, _ = layers("any4", 2, 98, 4096, 128)
    ids, x, dy, z = choose(50, 2, 2), normal(7, 50, 4096), normal(9, 50, 2, 98), normal(5, 150, 98)
    calls = [(any4.gemm_act_workspace_size(50, 98, 4096, 128),
              lambda ws: any4.gemm_act(x, packed[:packed.numel() // 2], *[t[0] for t in tables], 128, workspace=ws)),
             (any4.experts_workspace_size(50, 2, 2, 98, 4096, 128),
              lambda ws: any4.experts_gemm(x, packed, *tables, 128, ids, workspace=ws)),
             (any4.experts_dx_workspace_size(50, 2, 2, 98, 4096, 128),
              lambda ws: any4.experts_gemm_dx(dy, packed, *tables, 128, ids, workspace=ws)),
             (any4.act_backward_workspace_size(150, 98, True),
              lambda ws: torch.cat([t.flatten().float() for t in any4.act_backward(normal(10, 150, 49), z, "silu", gate=True,
                                                                                   workspace=ws)]))]
    for need, call in calls:
        assert need > 0
        room = torch.full((need + 256,), 77, dtype=torch.uint8, device=gu.DEV)
        want = call(None)
        for _ in range(2):
            assert torch.equal(call(room[:need]), want) and (room[need:] == 77).all()
        with pytest.raises((any4.Any4Error, ValueError)):
            call(room[:need - 256])


# ---------------------------------------------------------------------------
# limits
# ---------------------------------------------------------------------------
def test_most_experts_of_a_token():
    """1024 experts, 64 of them a token."""
    E, k, T = 1024, 64, 3
    packed, (lut, alpha, beta), w = layers("any4", 4, 16, 128, 128)
    packed, lut, alpha, beta, w = (t.repeat(*([E // 4] + [1] * (t.dim() - 1))) for t in (packed, lut, alpha, beta, w))
    w8, ids = any4.route(torch.randn(T, E, generator=torch.Generator().manual_seed(1)).to(gu.DEV), k)
    x, dy = normal(1, T, 128), normal(2, T, k, 16)
    close(any4.experts_gemm(x, packed, lut, alpha, beta, 128, ids), *each_expert(x.double()[:, None].expand(T, k, 128), w, ids))
    close(any4.experts_gemm_dx(dy, packed, lut, alpha, beta, 128, ids), *each_expert(dy.double(), w, ids, back=True))


def test_stacked_layers_beyond_four_gib():
    """One-hot rows give the last experts' weights, bit for bit."""
    E, N, K = 560, 4096, 4096
    gen = torch.Generator(device=gu.DEV).manual_seed(1)
    packed = torch.randint(0, 256, (E * N * K // 2,), dtype=torch.uint8, generator=gen, device=gu.DEV)
    assert packed.numel() > 1 << 32
    lut = torch.randn(E, N, 16, generator=gen, device=gu.DEV, dtype=torch.bfloat16)
    alpha, beta = (torch.randn(E, N, K // 128, generator=gen, device=gu.DEV, dtype=torch.bfloat16) for _ in range(2))
    for T in (16, 100):             # few rows, tiles
        for e in (E - 1, 513, 1):
            w = any4.dequant(packed[e * N * K // 2:(e + 1) * N * K // 2], lut[e], alpha[e], beta[e], 128)
            ids = torch.full((T, 1), e, dtype=torch.int32, device=gu.DEV)
            x = torch.eye(K, dtype=torch.bfloat16, device=gu.DEV)[-T:].contiguous()
            assert torch.equal(any4.experts_gemm(x, packed, lut, alpha, beta, 128, ids)[:, 0], w.view(N, K)[:, -T:].t())
            dy = torch.eye(N, dtype=torch.bfloat16, device=gu.DEV)[-T:, None].contiguous()
            assert torch.equal(any4.experts_gemm_dx(dy, packed, lut, alpha, beta, 128, ids)[:, 0], w.view(N, K)[-T:])


def test_results_beyond_four_gib():
    M, N = 16300, 65800
    assert M * N < 1 << 30 and M * N * 4 > (1 << 32) - (1 << 25)
    packed, tables, w = layers("any4", 1, N, 128, 128)
    x = normal(1, M, 128)
    z, out = torch.empty(M, N, device=gu.DEV), torch.empty(M, N, device=gu.DEV)
    any4.gemm_act(x, packed, *[t[0] for t in tables], 128, act="relu", z=z, out=out)
    for rows in (slice(0, 40), slice(M - 40, M)):
        ref, e = product(x[rows].double(), w[0])
        near(z[rows], ref, e)
        near(out[rows], *expect(ref, e, "relu", False))
    dz, dbias = any4.act_backward(out, z, "relu")
    assert torch.equal(dz[-40:], out[-40:].bfloat16()) and torch.equal(dz[:40], out[:40].bfloat16())
    total = sum(out[r:r + 1000].double().sum(0) for r in range(0, M, 1000))      # out > 0 only where the slope is 1
    assert ((dbias.double() - total).abs() <= (M + 16) * 2.0 ** -24 * total).all()


def test_weighted_sums_beyond_four_gib():
    T, k, N = 131072, 8, 1023
    assert T * k * N < 1 << 30
    y = torch.randn(T, k, N, generator=torch.Generator(device=gu.DEV).manual_seed(1), device=gu.DEV)
    w = torch.rand(T, k, generator=torch.Generator(device=gu.DEV).manual_seed(2), device=gu.DEV)
    out, dout = any4.combine(y, w), normal(3, T, N)
    dy, dw = any4.combine_backward(dout, y, w)
    for rows in (slice(0, 3), slice(T - 3, T)):
        p = y[rows].double() * w[rows].double()[:, :, None]
        close(out[rows], p.sum(1), (k + 1) * 2.0 ** -24 * p.abs().sum(1))
        close(dy[rows], w[rows].double()[:, :, None] * dout[rows].double()[:, None], torch.zeros(3, k, N, device=gu.DEV))
        p = y[rows].double() * dout[rows].double()[:, None]
        assert ((dw[rows].double() - p.sum(2)).abs() <= (N + 16) * 2.0 ** -24 * p.abs().sum(2)).all()


def test_empty_batches():
    b = Block(1, 128, 128, 4, 2)
    b.T, b.dout = 0, b.dout[:0]
    got = b.run(b.x[:0], b.logits[:0])
    assert got["out"].shape == (0, 128) and got["dx"].shape == (0, 128) and got["dlogits"].shape == (0, 4)
    assert torch.equal(got["dbias"], torch.zeros(256, device=gu.DEV))
