"""GPU parity of the norm with the residual's addition, microscaled quantisation and the product, against the
definitions in 64 bits (step_ref.py).  Tolerances follow from the stated roundings."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import step_ref as R  # noqa: E402
from sparse_activation_ffn_amd import binding as pb  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
NP = {"f16": np.float16, "f32": np.float32}
FMT = {"fp8": pb.PI_MXFP8, "fp4": pb.PI_MXFP4}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    return t.detach().cpu().numpy()


def strided(a, pad, fill, off=0):
    """A device copy of a [rows][...][d] with `pad` more elements after each innermost row and `off` elements before the
    first; the tensor, and a function that says whether the rest still holds `fill`."""
    a = np.ascontiguousarray(a)
    rows = int(np.prod(a.shape[:-1]))
    wide = torch.full((off + rows * (a.shape[-1] + pad),), fill, dtype=torch.from_numpy(a).dtype, device=DEV)
    view = wide[off:].view(*a.shape[:-1], a.shape[-1] + pad)[..., :a.shape[-1]]
    view.copy_(dev(a))

    def untouched():
        rest = wide[off:].view(rows, -1)[:, a.shape[-1]:]
        return bool((rest == fill).all()) and bool((wide[:off] == fill).all())
    return view, untouched


def check_y(got, y, f16):
    """One rounding to the type (2^-11 or 2^-24 of the value, and of the smallest subnormal half a step), and 2^-22 before."""
    got = got.astype(np.float64)
    tol = np.abs(y) * (2.0 ** -11 + 2.0 ** -22) + 2.0 ** -25 if f16 else np.abs(y) * 2.0 ** -22 + 2.0 ** -149
    with np.errstate(over="ignore"):
        y = y.astype(np.float16).astype(np.float64) if f16 else y
    fine = np.isfinite(y)
    assert (np.isnan(got) == np.isnan(y)).all() and (got[np.isinf(y)] == y[np.isinf(y)]).all()
    assert (np.abs(got[fine] - y[fine]) <= 2 * tol[fine]).all() if f16 else (np.abs(got[fine] - y[fine]) <= tol[fine]).all()


def check_mx(codes, scales, y, form, rel=2.0 ** -22):
    """Microscaled values of y, where y itself was known within rel: the scale is the definition's for some value in that
    range, and every element the nearest for some value in it."""
    lo, hi = R.scales(y * (1 - rel), form), R.scales(y * (1 + rel), form)
    assert ((scales == lo) | (scales == hi)).all()
    top = R.GRIDS[form][1][-1]
    fine = np.repeat(scales != 255, 32, axis=-1)
    with np.errstate(invalid="ignore"):
        want = np.ldexp(R.blocks(y), -(scales.astype(np.int64) - 127)[..., None]).reshape(y.shape)
    want, got = want[fine], R.elements(R.unpacked(codes, form), form)[fine]
    m = np.minimum(np.abs(want), top)
    grid = R.GRIDS[form][1]
    near = np.abs(grid[np.clip(np.searchsorted(grid, m), 0, len(grid) - 1)] - m)
    below = np.abs(grid[np.clip(np.searchsorted(grid, m) - 1, 0, len(grid) - 1)] - m)
    assert (np.abs(np.abs(got) - m) <= np.minimum(near, below) + 2 * rel * m).all()
    assert (np.signbit(got) == np.signbit(want)).all()


NORMS = [  # dtype, tokens, heads, d, delta, weight, eps
    ("f16", 1, 1, 7168, "f32", "f16", 1e-5), ("f16", 3, 1, 8192, "f16", "f32", 1e-6), ("f32", 2, 1, 12288, "f32", "f32", 1e-5),
    ("f32", 5, 1, 1024, "f16", "f16", 1e-5), ("f16", 7, 5, 64, None, "f16", 1e-5), ("f16", 33, 3, 128, "f16", None, 1e-5),
    ("f32", 9, 2, 96, "f32", "f32", 1e-5), ("f16", 4, 2, 256, None, "f32", 0.0), ("f32", 6, 1, 512, None, None, 1e-5),
    ("f16", 2, 1, 2048, "f32", "f16", 1e-5), ("f16", 2, 1, 4096, "f16", "f16", 1e-5), ("f32", 1, 1, 16384, "f32", "f32", 1e-5),
    ("f16", 2, 1, 16416, "f16", "f16", 1e-5), ("f32", 1, 1, 40000, "f16", "f32", 1e-5), ("f16", 70, 1, 32, None, "f16", 1e-5),
    ("f16", 3, 1, 1, "f16", "f16", 1e-5), ("f32", 3, 2, 7, "f32", "f32", 1e-5), ("f16", 2, 1, 1001, "f32", "f16", 1e-5),
    ("f32", 2, 1, 5003, None, "f16", 1e-5)]


def norm_case(dtype, tokens, heads, d, delta, weight, seed=0, size=1.0):
    rng = np.random.default_rng([seed, tokens, heads, d])
    x = (size * rng.standard_normal((tokens, heads, d)) * np.where(rng.random(d) < 0.02, 20, 1)).astype(NP[dtype])
    dl = None if delta is None else rng.standard_normal((tokens, heads, d)).astype(NP[delta])
    w = None if weight is None else (1 + 0.1 * rng.standard_normal(d)).astype(NP[weight])
    return x, dl, w


@pytest.mark.parametrize("case", NORMS)
@pytest.mark.parametrize("pad,off", [(0, 0), (8, 0), (3, 1)])
def test_norm(case, pad, off):
    dtype, tokens, heads, d, delta, weight, eps = case
    x, dl, w = norm_case(*case[:6])
    tx, _ = strided(x, pad, float("nan"), off)
    td = None if dl is None else strided(dl, pad, float("nan"), off)[0]
    ty, y_rest = strided(np.zeros_like(x), pad, 7.0, off)
    ts, s_rest = strided(np.zeros_like(x), pad, 7.0, off)
    norm = pb.make_norm(None if w is None else dev(w), eps, d)
    forms = ("fp8", "fp4") if d % 32 == 0 else (None,)
    for form in forms:
        mx = None if form is None else pb.empty_mx(tokens, heads * d, FMT[form])
        ty.zero_(), ts.zero_()
        pb.pi_rms_norm(norm, tx, delta=td, sum_out=None if dl is None else ts, y=ty, mx=mx)
        torch.cuda.synchronize()
        s = x if dl is None else R.sums(x, dl)
        assert np.array_equal(host(ts), np.zeros_like(s) if dl is None else s)
        y = R.norm(s, w, eps)
        check_y(host(ty), y, dtype == "f16")
        if mx is not None:
            check_mx(host(mx._keep[0]), host(mx._keep[1]), y.reshape(tokens, heads * d), form)
    assert y_rest() and s_rest()


@pytest.mark.parametrize("d", [128, 7168, 1001, 20000])
@pytest.mark.parametrize("sum_to,y_to", [("x", None), ("delta", "x"), ("x", "delta"), (None, "x"), (None, "delta"), ("x", "new")])
def test_norm_in_place(d, sum_to, y_to):
    x, dl, w = norm_case("f16", 5, 1, d, "f16", "f16", 1)
    x, dl = x[:, 0], dl[:, 0]
    t = {"x": dev(x), "delta": dev(dl), "new": torch.empty((5, d), dtype=torch.float16, device=DEV), None: None}
    mx = pb.empty_mx(5, d, pb.PI_MXFP8) if y_to is None and d % 32 == 0 else None
    pb.pi_rms_norm(pb.make_norm(dev(w)), t["x"], delta=t["delta"], sum_out=t[sum_to], y=t[y_to], mx=mx)
    torch.cuda.synchronize()
    s = R.sums(x, dl)
    if sum_to:
        assert np.array_equal(host(t[sum_to]), s)
    if y_to:
        check_y(host(t[y_to]), R.norm(s, w, 1e-5), True)
    for name, before in (("x", x), ("delta", dl)):
        if name not in (sum_to, y_to):
            assert np.array_equal(host(t[name]), before)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("d", [96, 2048, 1001])
def test_norm_of_extreme_rows(dtype, d):
    """Zeros, the largest and the smallest values, infinities and NaN, each row by itself."""
    x, _, w = norm_case(dtype, 8, 1, d, None, dtype, 2)
    x = x[:, 0]
    info = np.finfo(NP[dtype])
    x[0], x[1], x[2] = 0, info.max, info.smallest_subnormal
    x[3, d // 2], x[4, 3], x[5, 0], x[5, d - 1] = np.inf, np.nan, np.inf, -np.inf
    x[6] = np.where(np.arange(d) % 2, info.max, -info.max)
    y = torch.empty((8, d), dtype=dev(x).dtype, device=DEV)
    mx = pb.empty_mx(8, d, pb.PI_MXFP8) if d % 32 == 0 else None
    pb.pi_rms_norm(pb.make_norm(dev(w), 1e-30), dev(x), y=y, mx=mx)
    torch.cuda.synchronize()
    want = R.norm(x, w, 1e-30)
    check_y(host(y), want, dtype == "f16")
    if mx is not None:
        s = host(mx._keep[1])
        assert (s[3].reshape(-1)[d // 2 // 32] == 255) and (s[4] == 255).all() and (s[0] == 0).all()
        check_mx(host(mx._keep[0])[[1, 2, 6, 7]], s[[1, 2, 6, 7]], want[[1, 2, 6, 7]], "fp8")


def wild(rng, rows, cols, dtype):
    """Every exponent of the type, zeros and signs of zeros among them."""
    if dtype == "f16":
        x = rng.integers(0, 1 << 16, (rows, cols)).astype(np.uint16).view(np.float16)
    else:
        x = rng.integers(0, 1 << 32, (rows, cols), dtype=np.uint64).astype(np.uint32).view(np.float32)
    # blocks of one size and blocks of all
    near = np.repeat(rng.random((rows, cols // 32)) < 0.7, 32, axis=1)
    with np.errstate(over="ignore"):
        alike = (rng.standard_normal((rows, cols)) * np.repeat(2.0 ** rng.integers(-20, 15, (rows, cols // 32)), 32, axis=1)).astype(x.dtype)
    x = np.where(near, alike, x)
    return np.where(np.isfinite(x), x, np.where(rng.random(x.shape) < 0.5, 0.0, -0.0).astype(x.dtype)).astype(x.dtype)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("form", ["fp8", "fp4"])
@pytest.mark.parametrize("rows,cols,pad,off", [(1, 32, 0, 0), (3, 64, 0, 0), (17, 96, 5, 1), (5, 7168, 8, 0), (130, 2080, 0, 0),
                                               (2, 12288, 1, 3), (1, 1 << 20, 0, 0), (70000, 32, 0, 0)])
def test_quantize_and_back(dtype, form, rows, cols, pad, off):
    rng = np.random.default_rng([rows, cols])
    x = wild(rng, rows, cols, dtype)
    x[0, :32] = 0
    if rows > 2:
        x[1, 0], x[2, 31] = np.inf, np.nan
    tx, _ = strided(x, pad, float("nan"), off)
    mx = pb.empty_mx(rows, cols, FMT[form])
    pb.pi_mx_quantize(tx, mx)
    out, rest = strided(np.zeros_like(x), pad, 7.0, off)
    pb.pi_mx_dequantize(mx, out)
    torch.cuda.synchronize()
    codes, scales = (host(t) for t in mx._keep)
    want = R.scales(x, form)
    assert np.array_equal(scales, want)
    fine = np.repeat(want != 255, 32, axis=1)
    got = R.unpacked(codes, form)
    assert np.array_equal(got[fine], R.codes(np.where(fine, x, 0), form)[fine])
    with np.errstate(over="ignore"):
        assert np.array_equal(host(out), R.values(codes, scales, form).astype(x.dtype), equal_nan=True)
    assert rest()


def test_every_tie():
    """Values half between two codes, next to them, and past the largest: in f32, with the block's scale at 1."""
    for form in ("fp8", "fp4"):
        grid = R.GRIDS[form][1]
        mid = np.append((grid[1:] + grid[:-1]) / 2, [grid[-1] * 1.0625, grid[-1] * 1.125]).astype(np.float32)
        v = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9)), grid.astype(np.float32)])
        v = np.concatenate([v, -v])
        v = np.append(v, np.zeros(-len(v) % 31, np.float32)).reshape(-1, 31)
        # the last element of a block holds the scale
        x = np.concatenate([v, np.full((len(v), 1), grid[-1], np.float32)], axis=1)
        mx = pb.empty_mx(len(x), 32, FMT[form])
        pb.pi_mx_quantize(dev(x), mx)
        torch.cuda.synchronize()
        assert (host(mx._keep[1]) == 127).all()
        assert np.array_equal(host(mx._keep[0]), R.packed(R.codes(x, form), form))


def random_mx(rng, rows, cols, form, spread=6):
    """Random codes (no NaN) with scales around 1."""
    c = rng.integers(0, 256 if form == "fp8" else 16, (rows, cols)).astype(np.uint8)
    if form == "fp8":
        c = np.where(c % 128 == 127, 0, c).astype(np.uint8)
    return R.packed(c, form), rng.integers(127 - spread, 127 + spread, (rows, cols // 32)).astype(np.uint8)


def run_product(a, w, fa, bias=None, out="f32", pad=0, ws=None, off=0):
    am, wm = pb.make_mx(dev(a[0]), dev(a[1]), FMT[fa]), pb.make_mx(dev(w[0]), dev(w[1]), pb.PI_MXFP4)
    m, n, k = am.rows, wm.rows, am.cols
    o, rest = strided(np.zeros((m, n), NP[out]), pad, 7.0, off)
    need = pb.pi_mx_product_workspace_bytes(m, n, k)
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device=DEV)
    pb.pi_mx_product(am, wm, o, bias=None if bias is None else dev(bias), ws=ws)
    torch.cuda.synchronize()
    assert rest()
    return host(o)


def check_product(a, w, fa, got, bias=None):
    va, vw = R.values(*a, fa), R.values(*w, "fp4")
    want, tol = R.product(va, vw, bias, cut=fa == "fp8" and got.dtype == np.float16)
    if got.dtype == np.float16:
        # from half a step past the largest value on (65520), f16 has infinities
        past, short = np.abs(want) - tol >= 65520, np.abs(want) + tol < 65520
        assert (np.isinf(got) & (np.sign(got) == np.sign(want)))[past].all() and np.isfinite(got[short]).all()
        tol = tol + 2.0 ** -11 * (np.abs(want) + tol) + 2.0 ** -25
        got, want, tol = got[short], want[short], tol[short]
    else:
        tol = tol + 2.0 ** -24 * np.abs(want)
    assert (np.abs(got.astype(np.float64) - want) <= tol).all()


PRODUCTS = [(1, 64, 32), (1, 1, 32), (1, 100, 1024), (2, 33, 96), (3, 7168, 160), (15, 200, 512), (16, 1024, 1024), (17, 17, 544),
            (33, 130, 7168), (48, 500, 2048), (64, 256, 8192), (65, 257, 1056), (100, 129, 480), (129, 1000, 640), (200, 300, 288),
            (256, 256, 256), (257, 513, 384), (300, 1025, 1536), (513, 260, 128), (1, 4099, 12288), (1000, 700, 64),
            (5, 8300, 1056), (16, 8192, 512), (20, 400, 2080), (200, 300, 4128), (130, 257, 3584)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
@pytest.mark.parametrize("fa", ["fp8", "fp4"])
def test_product(m, n, k, fa):
    rng = np.random.default_rng([m, n, k])
    a, w = random_mx(rng, m, k, fa), random_mx(rng, n, k, "fp4")
    bias = rng.standard_normal(n).astype(np.float32) * 100
    check_product(a, w, fa, run_product(a, w, fa))
    check_product(a, w, fa, run_product(a, w, fa, bias, pad=5), bias.astype(np.float64))
    # inside f16's range
    a16 = (a[0], (a[1] - 12).astype(np.uint8)) if fa == "fp8" else a
    check_product(a16, w, fa, run_product(a16, w, fa, out="f16", pad=(-n) % 8), None)
    check_product(a16, w, fa, run_product(a16, w, fa, bias, out="f16", pad=3, off=1), bias.astype(np.float64))


@pytest.mark.parametrize("fa", ["fp8", "fp4"])
def test_product_of_many_tiles(fa):
    """Outputs in hundreds of tiles, odd sizes: some rows of them."""
    m, n, k = 2177, 4001, 672
    rng = np.random.default_rng(9)
    a, w = random_mx(rng, m, k, fa), random_mx(rng, n, k, "fp4")
    if fa == "fp8":
        a = (a[0], (a[1] - 12).astype(np.uint8))
    bias = rng.standard_normal(n).astype(np.float32) * 100
    rows = np.unique(np.concatenate([[0, 15, 16, 63, 64, 127, 128, 129, 2047, 2048, 2175, m - 1], rng.integers(0, m, 20)]))
    some = (a[0][rows], a[1][rows])
    check_product(some, w, fa, run_product(a, w, fa, bias, pad=3)[rows], bias.astype(np.float64))
    check_product(some, w, fa, run_product(a, w, fa, out="f16", pad=7)[rows])


@pytest.mark.parametrize("m,n,k", [(1, 40, 160), (20, 40, 544), (150, 280, 1056)])
@pytest.mark.parametrize("fa", ["fp8", "fp4"])
def test_product_nan_rows_and_far_scales(m, n, k, fa):
    """A NaN reaches its row or column and nothing else; scales at the ends of their range multiply as they should."""
    rng = np.random.default_rng([m, n, k, 1])
    a, w = random_mx(rng, m, k, fa), random_mx(rng, n, k, "fp4")
    a, w = (a[0].copy(), a[1].copy()), (w[0].copy(), w[1].copy())
    w[1][n // 2, -1] = 255
    if m > 1:
        a[1][m - 1, 0] = 255
        if fa == "fp8":
            a[0][m // 2, k - 1] = 0x7f
    a[1][0], w[1][1] = 0, 220
    got = run_product(a, w, fa)
    nan = np.zeros((m, n), bool)
    nan[:, n // 2] = True
    if m > 1:
        nan[m - 1] = True
        nan[m // 2] |= fa == "fp8"
    assert (np.isnan(got) == nan).all()
    va, vw = np.nan_to_num(R.values(*a, fa)), np.nan_to_num(R.values(*w, "fp4"))
    want, tol = R.product(va, vw, None)
    # products below float32's smallest numbers are lost (at most half of 2^-149 for each), and in the form by bfloat16 either
    # factor is off by up to half of 2^-133, its smallest step
    tol = tol + 2.0 ** -24 * np.abs(want) + k * 2.0 ** -149
    if fa == "fp8":
        tol = tol + 2.0 ** -134 * (np.abs(va).sum(1)[:, None] + np.abs(vw).sum(1)[None])
    assert (np.abs(got.astype(np.float64) - want) <= tol)[~nan].all()


def test_products_repeat_and_calls_share_nothing():
    """The same product again, on another stream, and next to another one: bit for bit the same."""
    rng = np.random.default_rng(5)
    for m, n, k in ((1, 1024, 8192), (48, 520, 7168), (300, 700, 2048)):
        a, w, a2 = random_mx(rng, m, k, "fp8"), random_mx(rng, n, k, "fp4"), random_mx(rng, m, k, "fp8")
        first = run_product(a, w, "fp8")
        am, am2 = (pb.make_mx(dev(x[0]), dev(x[1]), pb.PI_MXFP8) for x in (a, a2))
        wm = pb.make_mx(dev(w[0]), dev(w[1]), pb.PI_MXFP4)
        outs = [torch.empty((m, n), device=DEV) for _ in range(2)]
        need = max(1, pb.pi_mx_product_workspace_bytes(m, n, k))
        ws = [torch.empty(need, dtype=torch.uint8, device=DEV) for _ in range(2)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(5):
            for x, o, s, b in zip((am, am2), outs, streams, ws):
                pb.pi_mx_product(x, wm, o, ws=b, stream=s)
        torch.cuda.synchronize()
        assert np.array_equal(host(outs[0]), first)
        assert np.array_equal(host(outs[1]), run_product(a2, w, "fp8"))


def test_nothing_to_do_and_wrong_tensors():
    mx = pb.empty_mx(0, 64, pb.PI_MXFP8)
    pb.pi_mx_quantize(torch.empty((0, 64), device=DEV), mx)
    pb.pi_mx_dequantize(mx, torch.empty((0, 64), device=DEV))
    w = pb.empty_mx(10, 64, pb.PI_MXFP4)
    pb.pi_mx_product(mx, w, torch.empty((0, 10), device=DEV))
    pb.pi_rms_norm(pb.make_norm(torch.ones(64, device=DEV)), torch.empty((0, 64), device=DEV), y=torch.empty((0, 64), device=DEV))
    with pytest.raises(ValueError):
        pb.pi_mx_quantize(torch.zeros((4, 64)), pb.empty_mx(4, 64, pb.PI_MXFP8))      # in host memory
    with pytest.raises(ValueError):
        pb.pi_rms_norm(pb.make_norm(torch.ones(64)), torch.zeros((4, 64), device=DEV), y=torch.zeros((4, 64), device=DEV))
