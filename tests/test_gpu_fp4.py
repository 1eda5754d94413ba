"""The 4-bit operators (qs_fp4_quantize, qs_fp4_sparse_linear) on the GPU
against the oracle.

Quantisation is defined by float32 steps, so codes, scales and values are
compared bit for bit.  The projection's products and block sums are exact;
each of its d_in / 32 scaled block sums (at most) enters a float32 sum with a
relative error of 2^-23 of the magnitudes added so far, hence
|y - ref| <= (d_in / 32 + 8) 2^-23 |X|.|W|^T, and half a step of the output
type."""
import numpy as np
import pytest
import torch

import oracle
import top_activation_sparse_b200 as qs
import workloads
from gpu_common import check_status, need_gpu, to_dev, to_np

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rows(seed, R, d, dtype):
    """Normal rows with outliers, zeros, tiny and huge blocks, and values on the borders."""
    g = workloads.rng(seed)
    x = workloads.normal_f32(g, (R, d))
    x[:, g.choice(d, size=max(1, d // 100), replace=False)] *= np.float32(20)
    for r in range(R):
        kind = r % 7
        at = 32 * int(g.integers(0, d // 32))
        if kind == 1:
            x[r, at:at + 32] = 0
            x[r, at:at + 32:2] = np.float32(-0.0)
        elif kind == 2:     # borders of e2m1 for a block whose largest value is 6 or 4
            x[r, at:at + 32] = np.resize(np.array([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -5],
                                                  dtype=np.float32), 32)
        elif kind == 3:
            x[r, at:at + 32] *= np.float32(2.0 ** -30)
        elif kind == 4:
            x[r, at:at + 32] *= np.float32(2.0 ** 60)
        elif kind == 5:
            x[r, at:at + 32] = np.float32(2.0 ** -130) * g.integers(-3, 4, size=32).astype(np.float32)
        elif kind == 6:     # just below and at a power of two
            x[r, at:at + 32] = np.float32(0.5)
            x[r, at] = np.nextafter(np.float32(8), np.float32(0))
    return workloads.round_to_dtype(x, dtype)


def _check_quant(x, dtype, fmt, layout, g=1.0):
    xt = to_dev(x, dtype)
    ts = torch.tensor([g], device="cuda") if g != 1.0 else None
    r = qs.qs_fp4_quantize(xt, fmt, layout, ts, values=True)
    ref = oracle.fp4_quantize(x, fmt, g)
    sc = r.scales.cpu().numpy()
    if layout == "rows":
        np.testing.assert_array_equal(sc, ref["scale_codes"])
    else:
        np.testing.assert_array_equal(sc, oracle.fp4_tile_scales(ref["scale_codes"]))
    np.testing.assert_array_equal(r.codes.cpu().numpy(), oracle.fp4_pack(ref["codes"]))
    want = torch.from_numpy(ref["values"].astype(np.float32)).to(DT[dtype]).float().numpy()
    np.testing.assert_array_equal(to_np(r.values), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("layout", ["rows", "tiled"])
@pytest.mark.parametrize("R,d", [(1, 32), (1, 4096), (3, 96), (7, 4160), (130, 160), (129, 256), (40, 11008)])
def test_quantize_is_bit_exact(R, d, layout, fmt, dtype):
    need_gpu()
    _check_quant(_rows(R * 7919 + d, R, d, dtype), dtype, fmt, layout)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("g", [2.0 ** -9, 0.00137, 3.7])
def test_quantize_nv_tensor_scale(g, dtype):
    need_gpu()
    _check_quant(_rows(11, 14, 512, dtype), dtype, "nv", "tiled", float(np.float32(g)))


def test_quantize_many_rows_takes_the_unrolled_kernel():
    need_gpu()
    _check_quant(_rows(5, 600, 4128, "bf16"), "bf16", "mx", "rows")


@pytest.mark.parametrize("fmt,block,nan", [("mx", 32, 255), ("nv", 16, 127)])
def test_quantize_non_finite_blocks_stand_for_nan(fmt, block, nan):
    need_gpu()
    x = np.ones((3, 128), dtype=np.float32)
    x[0, 5], x[1, 40], x[2, 127] = np.inf, np.nan, -np.inf
    r = qs.qs_fp4_quantize(to_dev(x, "f32"), fmt, "rows", values=True)
    v, s = to_np(r.values), r.scales.cpu().numpy()
    bad = np.zeros((3, 128 // block), dtype=bool)
    bad[0, 5 // block] = bad[1, 40 // block] = bad[2, 127 // block] = True
    np.testing.assert_array_equal(s == nan, bad)
    np.testing.assert_array_equal(np.isnan(v), np.repeat(bad, block, axis=1))
    # a block of ones: exact in mx; nv's scale e4m3(1/6) is 0.171875, and 1 / 0.171875 = 5.82 becomes 6
    assert np.all(v[~np.repeat(bad, block, axis=1)] == (1.0 if fmt == "mx" else 6 * 0.171875))


def test_quantize_outputs_are_optional_and_leading_dimensions_kept():
    need_gpu()
    x = to_dev(_rows(3, 12, 64, "bf16"), "bf16").reshape(3, 4, 64)
    full = qs.qs_fp4_quantize(x, "mx", "rows", values=True)
    assert full.codes.shape == (3, 4, 32) and full.scales.shape == (3, 4, 2) and full.values.shape == (3, 4, 64)
    only = qs.qs_fp4_quantize(x, "mx", "rows", codes=None, scales=None, values=True)
    assert only.codes is None and only.scales is None
    assert torch.equal(only.values, full.values)


# ---- projection -------------------------------------------------------------------------

def _weight(seed, d_out, d_in, fmt):
    g = workloads.rng(seed)
    w = workloads.normal_f32(g, (d_out, d_in), d_in ** -0.5)
    ws = float(np.float32(np.abs(w).max() / 2688)) if fmt == "nv" else 1.0
    r = qs.qs_fp4_quantize(to_dev(w, "f32"), fmt, "tiled", torch.tensor([ws], device="cuda"))
    return r, oracle.fp4_quantize(w, fmt, ws)["values"], ws


def _check_linear(x, k, fmt, dtype, y_dtype, w, values, ws_scale, xs_scale=1.0, ws=None):
    xt = to_dev(x, dtype)
    T, d_in = x.shape
    one = lambda v: None if v == 1.0 else torch.tensor([v], device="cuda")  # noqa: E731
    y = qs.qs_fp4_sparse_linear(xt, w.codes, w.scales, k, fmt, one(xs_scale), one(ws_scale), y_dtype=DT[y_dtype], ws=ws)
    ref = oracle.fp4_sparse_linear(x, values, k, fmt, xs_scale)
    # the tensor scales enter as one float32 product: two more roundings, and
    # values rounds their product with a scale once more
    tol = (d_in / 32 + 8) * 2.0 ** -23 * ref["mag"] + (2.0 ** -8 if y_dtype == "bf16" else 2.0 ** -24) * np.abs(ref["y"])
    err = np.abs(to_np(y).astype(np.float64) - ref["y"])
    assert np.all(err <= tol + 1e-300), (float(err.max()), float((err / np.maximum(tol, 1e-300)).max()))
    return y


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T,d_in,d_out", [(1, 32, 8), (1, 256, 128), (1, 4096, 264), (2, 64, 136), (3, 96, 1000),
                                          (8, 1024, 1152), (9, 544, 128), (17, 2080, 640), (33, 4160, 1000),
                                          (64, 1056, 72), (65, 512, 520), (128, 768, 256), (129, 320, 264)])
def test_linear_sizes(T, d_in, d_out, fmt):
    need_gpu()
    x = workloads.round_to_dtype(workloads.normal_f32(workloads.rng(T + d_in), (T, d_in)), "bf16")
    w, values, s = _weight(d_out, d_out, d_in, fmt)
    for k in sorted({d_in, d_in // 2 + 1, 0}):
        y = _check_linear(x, k, fmt, "bf16", "f32", w, values, s)
        if k == 0:
            assert torch.count_nonzero(y).item() == 0


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype,y_dtype", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
def test_linear_types(dtype, y_dtype, fmt):
    need_gpu()
    x = workloads.round_to_dtype(workloads.normal_f32(workloads.rng(8), (5, 640), 3.0), dtype)
    w, values, s = _weight(77, 384, 640, fmt)
    _check_linear(x, 448, fmt, dtype, y_dtype, w, values, s, xs_scale=0.0123 if fmt == "nv" else 1.0)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T", [1, 8, 32])
def test_linear_llama_shapes(T, fmt):
    """4096 -> 11008 with 70% kept, and 11008 -> 4096 dense."""
    need_gpu()
    wl = workloads.WORKLOADS["ffn_relu2_llama7b"]
    x = workloads.activations(wl, 8)
    x = np.resize(x, (T, x.shape[1]))
    w, values, s = _weight(1, 11008, 4096, fmt)
    _check_linear(x, wl.k, fmt, "bf16", "bf16", w, values, s)
    x = workloads.round_to_dtype(workloads.normal_f32(workloads.rng(T), (T, 11008)), "bf16")
    w, values, s = _weight(2, 4096, 11008, fmt)
    _check_linear(x, 11008, fmt, "bf16", "f32", w, values, s)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T,d_in,d_out", [(640, 512, 6400), (515, 96, 6408)])
def test_linear_many_tokens_takes_the_wide_tiles(T, d_in, d_out, fmt):
    """150 and 153 tiles of 128 x 256: the tokens' last tile is full, half full, nearly empty."""
    need_gpu()
    x = workloads.round_to_dtype(workloads.normal_f32(workloads.rng(T), (T, d_in)), "bf16")
    w, values, s = _weight(d_out, d_out, d_in, fmt)
    _check_linear(x, d_in, fmt, "bf16", "f32", w, values, s)
    _check_linear(x, d_in // 3, fmt, "bf16", "bf16", w, values, s)


def test_linear_is_the_same_bits_each_time_and_leaves_the_workspace_ready():
    need_gpu()
    x = workloads.round_to_dtype(workloads.normal_f32(workloads.rng(4), (6, 4096)), "bf16")
    w, values, s = _weight(3, 1024, 4096, "mx")
    ws = qs.new_workspace(qs.QS_OP_FP4_SPARSE_LINEAR, 6, 4096, 1024, 4096, "cuda")
    first = _check_linear(x, 4096, "mx", "bf16", "f32", w, values, s, ws=ws)
    for _ in range(5):
        assert torch.equal(first, _check_linear(x, 4096, "mx", "bf16", "f32", w, values, s, ws=ws))
    check_status(ws)
    assert int(ws[256:256 + 65536].count_nonzero()) == 0


def test_linear_rows_of_one_scale_select_the_right_scales():
    """Blocks whose scales all differ: a scale taken from a neighbouring row or block shows."""
    need_gpu()
    for fmt in ("mx", "nv"):
        g = workloads.rng(17)
        T, d_in, d_out = 130, 512, 136
        x = workloads.normal_f32(g, (T, d_in)) * np.exp2(g.integers(-3, 4, size=(T, d_in // 16))).repeat(16, 1)
        x = workloads.round_to_dtype(x.astype(np.float32), "bf16")
        w = (workloads.normal_f32(g, (d_out, d_in)) * np.exp2(g.integers(-3, 4, size=(d_out, d_in // 16))).repeat(16, 1)).astype(np.float32)
        r = qs.qs_fp4_quantize(to_dev(w, "f32"), fmt, "tiled")
        _check_linear(x, d_in, fmt, "bf16", "f32", r, oracle.fp4_quantize(w, fmt)["values"], 1.0)


def test_linear_nan_block_stays_in_its_rows():
    need_gpu()
    g = workloads.rng(6)
    x = workloads.round_to_dtype(workloads.normal_f32(g, (3, 256)), "bf16")
    w = workloads.normal_f32(g, (136, 256), 0.06)
    clean = qs.qs_fp4_quantize(to_dev(w, "f32"), "mx")
    w[5, 40] = np.inf
    r = qs.qs_fp4_quantize(to_dev(w, "f32"), "mx")
    y0 = qs.qs_fp4_sparse_linear(to_dev(x, "bf16"), clean.codes, clean.scales, 256, y_dtype=torch.float32)
    y = qs.qs_fp4_sparse_linear(to_dev(x, "bf16"), r.codes, r.scales, 256, y_dtype=torch.float32)
    assert torch.isnan(y[:, 5]).all()
    keep = [j for j in range(136) if j != 5]
    assert torch.equal(y[:, keep], y0[:, keep])


# ---- the selection that feeds the projection ---------------------------------------------

def _kept_through_identity(x, k, fmt, dtype):
    """What the projection multiplies, read back through a weight that is the
    identity on blocks of columns (exact in 4 bits: 1 = code 2, scale 1)."""
    T, d = x.shape
    eye = np.zeros((d, d), dtype=np.float32)
    np.fill_diagonal(eye, 1.0)
    w = qs.qs_fp4_quantize(to_dev(eye, "f32"), fmt, "tiled")
    values = oracle.fp4_quantize(eye, fmt)["values"]
    assert np.abs(values - eye).max() <= 2.0 ** -5
    return _check_linear(x, k, fmt, dtype, "f32", w, values, 1.0)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_ties_are_kept_in_index_order(dtype, fmt):
    """Rows of few distinct magnitudes (more equal values than are kept), of one,
    of zeros, and with both signs of zero."""
    need_gpu()
    g = workloads.rng(12)
    d = 512
    x = g.integers(-2, 3, size=(6, d)).astype(np.float32)
    x[1] = 1.5
    x[2] = 0.0
    x[3, ::2] = -0.0
    x[4] = 0.0
    x[4, 100:140] = -3.0
    x[5, :] = np.where(np.arange(d) % 3 == 0, 2.0, -2.0)
    for k in (1, 7, 33, 100, 255, 511):
        y = _kept_through_identity(x, k, fmt, dtype)
        kept = to_np(y)[1] != 0
        assert kept[:k].all() and not kept[k:].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(2, 1024), (2, 1056), (3, 2048), (2, 2080), (300, 2080), (297, 4096), (5, 4096),
                                 (2, 4128), (2, 8192), (2, 8224), (1, 16384), (2, 16416), (1, 49152)])
def test_linear_rows_of_every_length(T, d, dtype):
    need_gpu()
    g = workloads.rng(T + d)
    x = workloads.normal_f32(g, (T, d))
    if T > 1:
        x[-1] = np.round(x[-1] * 2) / 2            # many ties
    x = workloads.round_to_dtype(x, dtype)
    fmt = "nv" if (d // 32) % 2 else "mx"
    w, values, s = _weight(d, 72, d, fmt)
    for k in (1, d // 3, d - 1):
        _check_linear(x, k, fmt, dtype, "f32", w, values, s)


def test_linear_equal_values_spread_over_the_row():
    """Ties in more places than a short list of them holds, at every length class."""
    need_gpu()
    for d in (1024, 2048, 4096, 8192, 16384):
        x = np.tile(np.array([1.0, -2.0, 0.5, 2.0], dtype=np.float32), (2, d // 4))
        w, values, s = _weight(d, 40, d, "mx")
        for k in (d // 4 + 3, d // 2, d // 2 + 1, d - 5):
            _check_linear(x, k, "mx", "bf16", "f32", w, values, s)


def test_linear_captured_and_replayed():
    need_gpu()
    g = workloads.rng(40)
    x = to_dev(workloads.normal_f32(g, (9, 512)), "bf16")
    w, values, s = _weight(41, 264, 512, "nv")
    sc = torch.tensor([s], device="cuda")
    call = lambda x: qs.qs_fp4_sparse_linear(x, w.codes, w.scales, 300, "nv", None, sc)  # noqa: E731
    eager = call(x)
    static = torch.zeros_like(x)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q = qs.qs_fp4_quantize(static, "nv", "rows", values=True)
            y = call(static)
        graphs.append((graph, y, q))
    static.copy_(x)
    want = qs.qs_fp4_quantize(x, "nv", "rows", values=True)
    for _ in range(3):
        for graph, y, q in graphs:
            graph.replay()
            assert torch.equal(y, eager) and torch.equal(q.codes, want.codes) and torch.equal(q.values, want.values)
    assert torch.equal(call(x), eager)


def test_linear_on_two_streams_at_once():
    need_gpu()
    g = workloads.rng(42)
    xs = [to_dev(workloads.normal_f32(g, (T, 1024)), "bf16") for T in (3, 40, 700)]
    w, values, s = _weight(43, 6400, 1024, "mx")
    want = [qs.qs_fp4_sparse_linear(x, w.codes, w.scales, 700) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for i, x in enumerate(xs):
            got += [(i, qs.qs_fp4_sparse_linear(x, w.codes, w.scales, 700, stream=st)) for st in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i, y in got)


def test_linear_rows_behind_the_last_are_left_as_they_were():
    need_gpu()
    g = workloads.rng(44)
    for T, d_out in ((5, 136), (130, 264), (600, 6408)):
        x = to_dev(workloads.normal_f32(g, (T, 96)), "bf16")
        w, _, _ = _weight(d_out, d_out, 96, "mx")
        buf = torch.full((T + 60, d_out), 7.0, device="cuda")
        y = qs.qs_fp4_sparse_linear(x, w.codes, w.scales, 96, y=buf[:T])
        assert bool((buf[T:] == 7.0).all())
        assert torch.equal(y, qs.qs_fp4_sparse_linear(x, w.codes, w.scales, 96, y_dtype=torch.float32))


def test_quantize_leaves_what_lies_behind_its_outputs():
    need_gpu()
    x = torch.randn(5, 96, device="cuda")
    codes = torch.full((7, 48), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((512 + 64,), 9, dtype=torch.uint8, device="cuda")
    values = torch.full((7, 96), 9.0, device="cuda")
    qs.qs_fp4_quantize(x, "mx", "tiled", codes=codes[:5], scales=scales[:512], values=values[:5])
    assert bool((codes[5:] == 9).all()) and bool((scales[512:] == 9).all()) and bool((values[5:] == 9).all())


def test_refusals_on_the_device():
    need_gpu()
    x = torch.randn(3, 64, device="cuda")
    w = qs.qs_fp4_quantize(torch.randn(16, 64, device="cuda"))
    lin = qs.qs_fp4_sparse_linear
    with pytest.raises(qs.QSError):
        lin(x, w.codes, w.scales, 65)
    with pytest.raises(qs.QSError):
        lin(x, w.codes, w.scales, 8, ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(qs.QSError):
        lin(x[:0], w.codes, w.scales, 8)
    for bad in (lambda: lin(x, w.codes[:, :16].contiguous(), w.scales, 8), lambda: lin(x, w.codes, w.scales[:-16], 8),
                lambda: lin(x.t(), w.codes, w.scales, 8), lambda: lin(x, w.codes, w.scales, 8, w_scale=torch.ones(2, device="cuda")),
                lambda: lin(x, w.codes.cpu(), w.scales, 8), lambda: qs.qs_fp4_quantize(x.t()),
                lambda: qs.qs_fp4_quantize(x, tensor_scale=torch.ones(1, device="cuda", dtype=torch.float64))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: qs.qs_fp4_quantize(x[:, :40].contiguous()), lambda: qs.qs_fp4_quantize(x[:0]),
                lambda: qs.qs_fp4_quantize(x, codes=None, scales=None)):
        with pytest.raises(qs.QSError):
            bad()
