"""Sizes that reach every form of the feed-forward products, by the library's own choice
(CPU only); test_gpu_ffn_forms.py runs them in every format.  A size that moves to another form fails here."""
import pytest

import gemm_any4_amd as any4

# one layer: (M, N, K): rows of a tile (0: few rows), waves, split sums, laid out first
ACT = {(3, 97, 384): (0, 4, False, False), (3, 97, 4096): (0, 8, False, False), (16, 4096, 14336): (0, 8, True, False),
       (820, 257, 128): (32, 4, False, False), (1030, 515, 1152): (32, 4, True, False), (1300, 1537, 384): (64, 4, False, False),
       (1030, 515, 2048): (64, 4, True, False), (1300, 4101, 384): (128, 4, False, False), (1300, 1025, 2176): (128, 4, True, False),
       (2050, 6147, 384): (256, 8, False, False), (4100, 1025, 2176): (256, 8, True, False),
       (3000, 3333, 2048): (256, 8, False, True), (4100, 1541, 4096): (256, 8, True, True)}
# (T, k, E, N, K)
EXPERTS = {(3, 2, 4, 97, 384): (0, 4, False), (5, 2, 3, 97, 4096): (0, 8, False), (2, 2, 3, 35, 8192): (0, 8, True),
           (65, 2, 2, 33, 384): (32, 4, False), (65, 2, 2, 35, 1152): (32, 4, True), (650, 2, 2, 1537, 384): (64, 4, False),
           (1025, 2, 2, 129, 2176): (64, 4, True), (650, 2, 2, 4099, 384): (128, 4, False), (650, 2, 2, 1025, 2176): (128, 4, True),
           (650, 2, 2, 8193, 384): (256, 8, False), (2050, 2, 2, 1025, 2176): (256, 8, True)}
PARTS = {(3, 2, 4, 97, 384): (0, 4, False), (5, 2, 3, 97, 4096): (0, 8, False), (2, 2, 3, 35, 8192): (0, 8, True),
         (65, 2, 2, 33, 384): (64, 4, False), (65, 2, 2, 35, 1152): (64, 4, True), (2050, 2, 2, 515, 384): (128, 4, False),
         (1025, 2, 2, 259, 2176): (128, 4, True), (650, 2, 2, 4099, 384): (256, 8, False), (650, 2, 2, 1025, 2176): (256, 8, True)}
DX = {(3, 2, 3, 37, 384): (32, 4, False), (3, 2, 2, 1026, 128): (32, 4, True), (100, 2, 2, 33, 8192): (64, 4, False),
      (650, 2, 2, 1027, 640): (64, 4, True), (500, 2, 2, 33, 4096): (128, 4, False), (1025, 2, 2, 1539, 640): (128, 4, True)}
DX_PARTS = {(3, 2, 3, 37, 384): (64, 4, False), (3, 2, 2, 1026, 128): (64, 4, True), (100, 2, 2, 33, 8192): (128, 4, False),
            (500, 2, 2, 1541, 640): (128, 4, True)}


def short(f):
    return (f.tile, f.waves, f.splits > 1)


def even(N):
    return N + N % 2


@pytest.mark.parametrize("size", ACT)
def test_one_layer(size):
    M, N, K = size
    for n in (N, even(N)):          # without a gate, and with one
        f = any4.ffn_form(M, 0, n, K)
        assert short(f) + (f.laid_out,) == ACT[size]


@pytest.mark.parametrize("back,parts,sizes", [(False, False, EXPERTS), (False, True, PARTS), (True, False, DX), (True, True, DX_PARTS)])
def test_experts(back, parts, sizes):
    for (T, k, E, N, K), want in sizes.items():
        for n in ((N,) if back else (N, even(N))):
            f = any4.ffn_form(T * k, E, n, K, back=back, parts=parts)
            assert short(f) == want and not f.laid_out, (T, k, E, n, K, f)


def test_every_form_is_reached():
    few = {(0, 4, False), (0, 8, False), (0, 8, True)}
    tiles = lambda *rows: {(r, 8 if r == 256 else 4, s) for r in rows for s in (False, True)}       # noqa: E731
    assert {v[:3] for v in ACT.values() if not v[3]} == set(EXPERTS.values()) == few | tiles(32, 64, 128, 256)
    assert {v[:3] for v in ACT.values() if v[3]} == tiles(256)
    assert set(PARTS.values()) == few | tiles(64, 128, 256)
    assert set(DX.values()) == tiles(32, 64, 128) and set(DX_PARTS.values()) == tiles(64, 128)


def test_errors():
    for bad in (dict(P=0), dict(P=-1), dict(N=0), dict(K=64), dict(E=-1), dict(E=1025), dict(E=0, back=True), dict(E=0, parts=True),
                dict(P=(1 << 20) + 1), dict(P=1 << 20, K=1024)):
        with pytest.raises(any4.Any4Error) as e:
            any4.ffn_form(**(dict(P=4, E=2, N=16, K=128) | bad))
        assert e.value.status == 2
    assert any4.lib().any4_ffn_form(4, 2, 16, 128, 0, 0, None) == 1
