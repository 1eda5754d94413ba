"""The 4-bit operators and the mixture-of-experts layer without a GPU: the
oracle's functions against hand-worked values and plain loops, and the host's
checks of arguments (nothing is enqueued, so the codes come back without a
device)."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

import oracle
import top_activation_sparse_b200 as qs
import workloads
from top_activation_sparse_b200 import build as qs_build


@pytest.fixture(scope="module")
def L():
    qs_build.build()
    return qs.lib()


# ---- oracle ------------------------------------------------------------------------------

def loop_e2m1(v):
    """Code of the nearest magnitude in exact arithmetic, by trying all eight
    (on a tie the even code)."""
    grid = [Fraction(x) for x in ("0", "1/2", "1", "3/2", "2", "3", "4", "6")]
    m = abs(v)
    best = min(range(8), key=lambda c: (abs(grid[c] - m), c % 2))
    return best + (8 if v < 0 else 0)


def test_e2m1_rounding_golden_hand():
    """Midpoints go to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2,
    2.5 -> 2, 3.5 -> 4, 5 -> 4; beyond 6 saturates."""
    row = np.zeros((1, 32), dtype=np.float32)
    row[0, :12] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.5, -0.2, 7.5, -7.9]
    # amax 7.9: floor(log2) = 2, the scale 2^0
    r = oracle.fp4_quantize(row, "mx")
    assert r["scale_codes"].tolist() == [[127]]
    assert r["codes"][0, :12].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 15, 8, 7, 15]
    assert r["values"][0, :12].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -6, 0, 6, -6]


def test_e4m3_grid_golden_hand():
    g = oracle.e4m3_grid()
    assert g.size == 127 and g[0] == 0 and g[1] == 2.0 ** -9 and g[7] == 7 * 2.0 ** -9
    assert g[8] == 2.0 ** -6 and g[56] == 1.0 and g[57] == 1.125 and g[126] == 448.0
    assert np.all(np.diff(g) > 0)


@pytest.mark.parametrize("seed", range(4))
def test_mx_quantize_bruteforce(seed):
    g = workloads.rng(seed)
    x = (workloads.normal_f32(g, (5, 64)) * np.exp2(g.integers(-30, 30, size=(5, 1)))).astype(np.float32)
    x[1, 3] = 0.0
    x[4] = 0.0
    r = oracle.fp4_quantize(x, "mx")
    for t in range(5):
        for b in range(2):
            blk = [Fraction(float(v)) for v in x[t, 32 * b: 32 * b + 32]]
            amax = max(abs(v) for v in blk)
            e = -127 if amax == 0 else math.floor(math.log2(float(amax))) - 2
            assert r["scale_codes"][t, b] == e + 127
            s = Fraction(2) ** e
            for i, v in enumerate(blk):
                c = loop_e2m1(v / s)
                if v != 0:
                    assert r["codes"][t, 32 * b + i] == c
                assert r["values"][t, 32 * b + i] == float((-1 if c & 8 else 1) * Fraction(float(oracle.E2M1[c & 7])) * s)


def test_nv_quantize_golden_hand():
    """amax 6 g: the scale is 1 and codes round x / g.  A block with amax g / 2:
    amax / 6 / g = 1/12 lies in [1/16, 1/8), where e4m3 has steps of 1/128:
    1/12 = 10.67/128 -> 11/128, and x / (11/128 g) = 5.8 -> 6."""
    g = 0.25
    x = np.zeros((1, 32), dtype=np.float32)
    x[0, :4] = [6 * g, 1.5 * g, -3.4 * g, 0.2 * g]
    x[0, 16] = 0.5 * g
    r = oracle.fp4_quantize(x, "nv", g)
    grid = oracle.e4m3_grid()
    assert grid[r["scale_codes"][0]].tolist() == [1.0, 11 / 128]
    assert r["codes"][0, :4].tolist() == [7, 3, 13, 0]
    assert r["values"][0, :4].tolist() == [1.5, 0.375, -0.75, 0.0]
    assert r["codes"][0, 16] == 7 and r["values"][0, 16] == float(np.float32(6 * 11 / 128 * g))


def test_non_finite_blocks_stand_for_nan():
    x = np.ones((2, 64), dtype=np.float32)
    x[0, 5], x[1, 40] = np.inf, np.nan
    for fmt, byte, block in (("mx", 255, 32), ("nv", 127, 16)):
        r = oracle.fp4_quantize(x, fmt)
        bad = np.zeros((2, 64), dtype=bool)
        bad[0, :block] = True
        bad[1, 40 // block * block: (40 // block + 1) * block] = True
        assert np.array_equal(np.isnan(r["values"]), bad)
        assert np.all(r["codes"][bad] == 0)
        assert (r["scale_codes"] == byte).sum() == 2


def test_pack_and_tiles_golden_hand():
    assert oracle.fp4_pack(np.array([[1, 2, 15, 8]])).tolist() == [[0x21, 0x8F]]
    sc = np.arange(1, 131 * 5 + 1).reshape(131, 5) % 251
    t = oracle.fp4_tile_scales(sc)
    assert t.size == 2 * 2 * 512
    assert t[0] == sc[0, 0] and t[1] == sc[0, 1] and t[4] == sc[32, 0] and t[16] == sc[1, 0]
    assert t[512] == sc[0, 4] and t[513] == 0                 # block 4 opens the row's second tile
    assert t[1024] == sc[128, 0] and t[1024 + 16 * 3] == 0    # row 131 is not there
    assert int((t != 0).sum()) == int((sc != 0).sum())


def test_fp4_sparse_linear_golden_hand():
    """x = (6, 1, -3, 0.5, 0...), k = 3 drops 0.5; amax 6 keeps the scale 1:
    y = 6 w0 + w1 - 3 w2."""
    x = np.zeros((1, 32), dtype=np.float32)
    x[0, :4] = [6, 1, -3, 0.5]
    w = np.zeros((2, 32))
    w[0, :4], w[1, :4] = [1, 2, 4, 100], [-0.5, 3, 1, 100]
    r = oracle.fp4_sparse_linear(x, w, 3, "mx")
    assert r["y"].tolist() == [[6 + 2 - 12, -3 + 3 - 3]]
    assert r["mag"].tolist() == [[20, 9]]


@pytest.mark.parametrize("act", ["drelu", "relu2_glu"])
@pytest.mark.parametrize("seed", [0, 1])
def test_moe_ffn_bruteforce(act, seed):
    g = workloads.rng(seed)
    T, dm, dff, E, K = 4, 6, 5, 7, 3
    n = lambda *s: workloads.normal_f32(g, s).astype(np.float64)  # noqa: E731
    x, wr, wg, wu, wd, bg, bu = n(T, dm), n(E, dm), n(E, dff, dm), n(E, dff, dm), n(E, dff, dm), n(E, dff), n(E, dff)
    biased = act == "drelu"
    r = oracle.moe_ffn(x, wr, wg, wu, wd, K, act, bg if biased else None, bu if biased else None)
    for t in range(T):
        logit = [sum(x[t, i] * wr[e, i] for i in range(dm)) for e in range(E)]
        chosen = sorted(range(E), key=lambda e: (-logit[e], e))[:K]
        z = [math.exp(logit[e] - logit[chosen[0]]) for e in chosen]
        p = [v / sum(z) for v in z]
        y = [0.0] * dm
        for e, share in zip(chosen, p):
            for j in range(dff):
                gate = sum(x[t, i] * wg[e, j, i] for i in range(dm))
                up = sum(x[t, i] * wu[e, j, i] for i in range(dm))
                if biased:
                    h = max(gate + bg[e, j], 0.0) * max(up + bu[e, j], 0.0)
                else:
                    h = max(up, 0.0) ** 2 * gate
                for i in range(dm):
                    y[i] += share * h * wd[e, j, i]
        assert r["experts"][t].tolist() == chosen
        np.testing.assert_allclose(r["weights"][t], p, rtol=1e-13)
        np.testing.assert_allclose(r["y"][t], y, rtol=1e-11, atol=1e-12)


def test_moe_ffn_equal_logits_and_one_expert():
    x = np.array([[1.0, 2.0]])
    wr = np.ones((4, 2))
    w = np.arange(4 * 1 * 2, dtype=np.float64).reshape(4, 1, 2) + 1
    r = oracle.moe_ffn(x, wr, w, w, w, 2, "relu2_glu")
    assert r["experts"].tolist() == [[0, 1]] and r["weights"].tolist() == [[0.5, 0.5]]
    # h = u^3, u = x.w: (1 + 4)^3 = 125 and (3 + 8)^3 = 1331
    assert r["y"].tolist() == [[0.5 * (125 * 1 + 1331 * 3), 0.5 * (125 * 2 + 1331 * 4)]]
    one = oracle.moe_ffn(x, wr[:1], w[:1], w[:1], w[:1], 1, "relu2_glu")
    assert one["weights"].tolist() == [[1.0]] and one["y"].tolist() == [[125.0, 250.0]]


# ---- the host's checks -------------------------------------------------------------------

FAKE = 0x10000      # 16-byte aligned, never dereferenced: validation fails first
BIG = 1 << 34


def _p(v):
    return ctypes.c_void_p(v)


def _call(f, args, **change):
    a = dict(args)
    assert set(change) <= set(a)
    a.update(change)
    return f(*a.values())


def test_fp4_scale_bytes():
    assert qs.qs_fp4_scale_bytes(3, 64, "mx", "rows") == 6
    assert qs.qs_fp4_scale_bytes(3, 64, "nv", "rows") == 12
    assert qs.qs_fp4_scale_bytes(3, 64, "mx", "tiled") == 512
    assert qs.qs_fp4_scale_bytes(129, 160, "mx", "tiled") == 2 * 2 * 512
    assert qs.qs_fp4_scale_bytes(1 << 33, 32, "mx", "rows") == 1 << 33
    for R, d, fmt, lay in ((0, 64, 0, 0), (1, 0, 0, 0), (1, 40, 0, 0), (1, 64, 2, 0), (1, 64, 0, 2), (-1, 64, 1, 1)):
        assert qs.qs_fp4_scale_bytes(R, d, fmt, lay) == 0


def test_fp4_quantize_refusals(L):
    ok = dict(x=_p(FAKE), dtype=1, R=4, d=64, format=0, g=None, layout=0, codes=_p(FAKE), scales=_p(FAKE),
              values=_p(FAKE), stream=None)
    for change in (dict(x=None), dict(dtype=2), dict(dtype=-1), dict(R=0), dict(R=-5), dict(d=0), dict(format=2),
                   dict(format=-1), dict(layout=2), dict(codes=None, scales=None, values=None)):
        assert _call(L.qs_fp4_quantize, ok, **change) == qs.QS_ERR_INVALID_ARG, change
    for change in (dict(d=48), dict(d=1), dict(x=_p(FAKE + 8)), dict(codes=_p(FAKE + 4)), dict(scales=_p(FAKE + 1)),
                   dict(values=_p(FAKE + 2)), dict(g=_p(FAKE + 2))):
        assert _call(L.qs_fp4_quantize, ok, **change) == qs.QS_ERR_ALIGNMENT, change


def test_fp4_sparse_linear_refusals(L):
    ok = dict(x=_p(FAKE), dtype=1, T=2, d_in=64, d_out=16, k=8, format=1, xs=None, wc=_p(FAKE), wsc=_p(FAKE), wg=None,
              y=_p(FAKE), y_dtype=0, events=None, ws=_p(FAKE), ws_bytes=BIG, stream=None)
    for change in (dict(x=None), dict(wc=None), dict(wsc=None), dict(y=None), dict(dtype=3), dict(y_dtype=2), dict(T=0),
                   dict(d_in=0), dict(d_out=0), dict(k=-1), dict(k=65), dict(format=2)):
        assert _call(L.qs_fp4_sparse_linear, ok, **change) == qs.QS_ERR_INVALID_ARG, change
    for change in (dict(d_in=72), dict(d_out=12), dict(x=_p(FAKE + 8)), dict(wc=_p(FAKE + 8)), dict(wsc=_p(FAKE + 4)),
                   dict(y=_p(FAKE + 4)), dict(xs=_p(FAKE + 1)), dict(wg=_p(FAKE + 2))):
        assert _call(L.qs_fp4_sparse_linear, ok, **change) == qs.QS_ERR_ALIGNMENT, change
    for change in (dict(d_in=qs.QS_MAX_ROW + 32), dict(d_out=qs.QS_MAX_ROW + 8)):
        assert _call(L.qs_fp4_sparse_linear, ok, **change) == qs.QS_ERR_UNSUPPORTED, change
    need = qs.qs_workspace_size(qs.QS_OP_FP4_SPARSE_LINEAR, 2, 64, 16, 8)
    for change in (dict(ws=None), dict(ws_bytes=need - 1), dict(ws_bytes=0)):
        assert _call(L.qs_fp4_sparse_linear, ok, **change) == qs.QS_ERR_WORKSPACE, change


def test_moe_ffn_refusals(L):
    ok = dict(x=_p(FAKE), T=2, d_model=64, d_ff=16, E=8, top_k=2, act=1, router=_p(FAKE), gate=_p(FAKE), up=_p(FAKE),
              down=_p(FAKE), s_gate=None, s_up=None, s_down=None, b_gate=None, b_up=None, y=_p(FAKE), y_dtype=1,
              experts=None, weights=None, ws=_p(FAKE), ws_bytes=BIG, stream=None)
    for change in (dict(x=None), dict(router=None), dict(gate=None), dict(up=None), dict(down=None), dict(y=None),
                   dict(y_dtype=2), dict(T=0), dict(d_model=0), dict(d_ff=0), dict(E=0), dict(top_k=0), dict(top_k=9),
                   dict(act=2), dict(s_gate=_p(FAKE)), dict(s_up=_p(FAKE)), dict(s_gate=_p(FAKE), s_up=_p(FAKE)),
                   dict(s_down=_p(FAKE))):
        assert _call(L.qs_moe_ffn, ok, **change) == qs.QS_ERR_INVALID_ARG, change
    for change in (dict(d_model=qs.QS_MOE_MAX_MODEL + 32), dict(d_ff=qs.QS_MAX_ROW + 8), dict(E=qs.QS_MOE_MAX_EXPERTS + 1),
                   dict(E=32, top_k=qs.QS_MOE_MAX_TOP_K + 1)):
        assert _call(L.qs_moe_ffn, ok, **change) == qs.QS_ERR_UNSUPPORTED, change
    for change in (dict(d_model=72), dict(d_ff=20), dict(x=_p(FAKE + 8)), dict(router=_p(FAKE + 2)), dict(down=_p(FAKE + 8)),
                   dict(b_gate=_p(FAKE + 4)), dict(y=_p(FAKE + 2)), dict(experts=_p(FAKE + 4)), dict(weights=_p(FAKE + 4))):
        assert _call(L.qs_moe_ffn, ok, **change) == qs.QS_ERR_ALIGNMENT, change
    need = qs.qs_workspace_size(qs.QS_OP_MOE_FFN, 2, 64, 16, 2)
    for change in (dict(ws=None), dict(ws_bytes=need - 1)):
        assert _call(L.qs_moe_ffn, ok, **change) == qs.QS_ERR_WORKSPACE, change


def test_workspace_sizes(L):
    f = qs.qs_workspace_size
    lin, moe = qs.QS_OP_FP4_SPARSE_LINEAR, qs.QS_OP_MOE_FFN
    assert 0 < f(lin, 1, 4096, 11008, 2867) < f(lin, 300, 4096, 11008, 2867)
    assert f(lin, 8, 4096, 11008, 0) == f(lin, 8, 4096, 11008, 4096) == f(lin, 8, 4096, 4096, 9)
    for bad in ((0, 64, 8, 1), (1, 48, 8, 1), (1, 64, 12, 1), (1, 64, 8, 65), (1, 64, 8, -1),
                (1, qs.QS_MAX_ROW + 32, 8, 1), (1, 64, qs.QS_MAX_ROW + 8, 1)):
        assert f(lin, *bad) == 0, bad
    # more than one launch's tokens do not grow the layer's buffers
    assert 0 < f(moe, 1, 4096, 14336, 2) < f(moe, 64, 4096, 14336, 2) == f(moe, 1000, 4096, 14336, 2)
    for bad in ((0, 64, 8, 1), (1, 48, 8, 1), (1, 64, 12, 1), (1, 64, 8, 0), (1, 64, 8, qs.QS_MOE_MAX_TOP_K + 1),
                (1, qs.QS_MOE_MAX_MODEL + 32, 8, 1), (1, 64, qs.QS_MAX_ROW + 8, 1)):
        assert f(moe, *bad) == 0, bad


def test_binding_refuses_what_it_can_see(L):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    u8 = torch.zeros(16, 32, dtype=torch.uint8)
    with pytest.raises(ValueError):
        qs.qs_fp4_quantize(x)                                     # a CPU tensor
    with pytest.raises(ValueError):
        qs.qs_fp4_sparse_linear(x, u8, u8, 8)
    w = torch.zeros(4, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        qs.qs_moe_ffn(x, torch.zeros(4, 64, dtype=torch.bfloat16), w, w, w, 2, "drelu")
