"""Products of microscaled matrices in the forms that real widths take: K a multiple of 512 in several stages, scales at the
ends of their range and NaN through the f16 form, and how exact that form is on the whole."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import step_ref as R  # noqa: E402
from sparse_activation_ffn_amd import binding as pb  # noqa: E402
from test_gpu_norm_mx import NP, check_product, random_mx, run_product  # noqa: E402

pytestmark = pytest.mark.gpu


def form(m, n):
    """The widest tile of the library that this size fills, as its rule has it: rows of a, of w, or "waves" without tiles."""
    if m <= 16:
        return "waves" if (n + 63) // 64 < 128 else "16x64"
    if m <= 64:
        return "32x64" if m <= 32 else "64x128"
    return "128x256" if (m + 127) // 128 * ((n + 255) // 256) > 256 else "128x128"


def splits(m, n, k):
    """Whether K is split: such a product has a join's launch."""
    pb.pi_kernel_timer_start(pb.PI_K_MX_JOIN, 8)
    rng = np.random.default_rng(0)
    run_product(random_mx(rng, m, k, "fp4"), random_mx(rng, n, k, "fp4"), "fp4")
    return pb.pi_kernel_timer_stop(pb.PI_K_MX_JOIN)[1] > 0


# sizes whose K is a multiple of 512 (scales by direct loads), two stages of it at least: name of the form, and whether K is split
ALIGNED = [(1, 1000, 2048, "waves", False), (13, 130, 8192, "waves", False), (1, 8300, 4096, "16x64", False),
           (16, 8197, 1536, "16x64", False), (9, 8193, 512 * 5, "16x64", False), (20, 400, 2048, "32x64", True),
           (32, 7168, 1024, "32x64", False), (29, 203, 8192, "32x64", True), (33, 1000, 1024, "64x128", False),
           (47, 1001, 7168, "64x128", True), (64, 1300, 1024, "64x128", False), (100, 1000, 1536, "128x128", False),
           (130, 150, 4096, "128x128", True)]


def cases(m, n, k, fa):
    """Random matrices, the left one inside what f16 holds of the product."""
    rng = np.random.default_rng([m, n, k, 7])
    a, w = random_mx(rng, m, k, fa), random_mx(rng, n, k, "fp4")
    a = (a[0], (a[1] - (14 if fa == "fp8" else 6)).astype(np.uint8))
    return a, w, (rng.standard_normal(n) * 10).astype(np.float32)


@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("fa", ["fp8", "fp4"])
@pytest.mark.parametrize("m,n,k,name,split", ALIGNED)
def test_aligned_forms(m, n, k, name, split, fa, out):
    assert form(m, n) == name and k % 512 == 0
    a, w, bias = cases(m, n, k, fa)
    check_product(a, w, fa, run_product(a, w, fa, out=out, pad=-n % 8))
    check_product(a, w, fa, run_product(a, w, fa, bias, out=out, pad=3, off=1), bias.astype(np.float64))


@pytest.mark.parametrize("m,n,k,name,split", ALIGNED)
def test_aligned_forms_split_as_named(m, n, k, name, split):
    assert splits(m, n, k) == split


@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("fa", ["fp8", "fp4"])
def test_aligned_form_of_many_tiles(fa, out):
    """Tiles of 128 x 256, twelve stages, odd sizes: some rows of the output."""
    m, n, k = 2177, 4001, 1536
    assert form(m, n) == "128x256"
    a, w, bias = cases(m, n, k, fa)
    rng = np.random.default_rng(1)
    rows = np.unique(np.concatenate([[0, 15, 16, 63, 64, 127, 128, 129, 2047, 2048, 2175, m - 1], rng.integers(0, m, 12)]))
    some = (a[0][rows], a[1][rows])
    check_product(some, w, fa, run_product(a, w, fa, bias, out=out, pad=3)[rows], bias.astype(np.float64))
    check_product(some, w, fa, run_product(a, w, fa, out=out, pad=-n % 8)[rows])


@pytest.mark.parametrize("m,n,k", [(1, 10240, 4096), (16, 8197, 1536), (40, 3000, 7168), (130, 1000, 4096), (2177, 4001, 1536),
                                   (300, 1000, 2080)])
def test_f16_form_on_the_whole(m, n, k):
    """MXFP8 to f16 of ordinary values, over all outputs.  With q what rounding the exact output to f16 leaves, and c the cut
    of the instruction (2^-16 of the outputs' root mean square; twice that is allowed): the squares of the errors add up to
    those of q and c, and no part of the output itself is in the error: <error, out> / <out, out> is c's 2^-16 at most but for
    noise.  The noise: of n independent errors of at most 2^-11, q's squares spread by less than 2^-22 / sqrt(n), and the part by
    2^-11 / sqrt(n); six times these."""
    rng = np.random.default_rng([m, n, k, 3])
    x, v = rng.standard_normal((m, k)), rng.standard_normal((n, k)) / np.sqrt(k)
    a, w = ((R.packed(R.codes(t, f), f), R.scales(t, f)) for t, f in ((x, "fp8"), (v, "fp4")))
    rows = np.unique(np.concatenate([[0, m - 1], rng.integers(0, m, 60)])) if m > 200 else np.arange(m)
    got = run_product(a, w, "fp8", out="f16")[rows].astype(np.float64)
    want = R.values(*a, "fp8")[rows] @ R.values(*w, "fp4").T
    size, count = (want * want).mean(), want.size
    e, q = got - want, want.astype(np.float16).astype(np.float64) - want
    assert (e * e).mean() <= (q * q).mean() + (2.0 ** -30 + 6 * 2.0 ** -22 / np.sqrt(count)) * size
    assert abs((e * want).mean()) <= (2.0 ** -16 + 6 * 2.0 ** -11 / np.sqrt(count)) * size


FAR = [(1, 40, 160), (20, 40, 544), (150, 280, 1056), (7, 900, 1024), (5, 8300, 1024), (32, 400, 2048), (50, 300, 1024),
       (150, 280, 1536), (2100, 4100, 512)]


@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("fa", ["fp8", "fp4"])
@pytest.mark.parametrize("m,n,k", FAR)
def test_nan_and_far_scales(m, n, k, fa, out):
    """A NaN, as an element or as a block's scale, reaches its row or column and nothing else; the smallest scale times the
    largest is 1.  (f32 out of MXFP8: the factors of 2^127 are values below bfloat16's largest.)"""
    rng = np.random.default_rng([m, n, k, 2])
    a, w = random_mx(rng, m, k, fa), random_mx(rng, n, k, "fp4")
    a = (a[0].copy(), (a[1] - (14 if fa == "fp8" else 6)).astype(np.uint8))
    w = (w[0].copy(), w[1].copy())
    w[1][n // 2, -1] = 255
    w[1][1] = 254
    if fa == "fp8" and out == "f32":
        w[0][1] &= 0xBB                                             # (magnitudes of up to 1.5: 2^128 is past bfloat16)
    a[1][0] = 0
    if m > 1:
        a[1][m - 1, 0] = 255
        if fa == "fp8":
            a[0][m // 2, k - 1] = 0x7f
            a[0][m // 4 + 1, 0] = 0xff
    rows = np.unique(np.concatenate([[0, 1, m // 4 + 1, m // 2, m - 1], rng.integers(0, m, 40)]) % m)
    got = run_product(a, w, fa, out=out)[rows].astype(np.float64)
    nan = np.zeros((len(rows), n), bool)
    nan[:, n // 2] = True
    if m > 1:
        nan[rows == m - 1] = True
        if fa == "fp8":
            nan[(rows == m // 2) | (rows == m // 4 + 1)] = True
    # column 1 of the other rows is past float32 or beside it, in whatever order it is summed
    known = np.ones((len(rows), n), bool)
    known[1:, 1] = False
    assert (np.isnan(got) == nan)[known].all()
    va, vw = np.nan_to_num(R.values(a[0][rows], a[1][rows], fa)), np.nan_to_num(R.values(*w, "fp4"))
    want, tol = R.product(va, vw, None, cut=fa == "fp8" and out == "f16")
    tol = tol + 2.0 ** -24 * np.abs(want) + k * 2.0 ** -149
    if fa == "fp8" and out == "f32":
        tol = tol + 2.0 ** -134 * (np.abs(va).sum(1)[:, None] + np.abs(vw).sum(1)[None])
    if out == "f16":
        tol = tol + 2.0 ** -11 * (np.abs(want) + tol) + 2.0 ** -25
    fine = known & ~nan
    assert (np.abs(want[fine]) < 60000).all()
    assert np.abs(want[0, 1]) > 0.01 and (np.abs(got - want) <= tol)[fine].all()


@pytest.mark.parametrize("m,n", [(1, 70), (5, 8200), (20, 70), (40, 70), (70, 70), (2100, 4100)])
def test_values_at_float32s_end(m, n):
    """MXFP8 to float32 goes through bfloat16: exact up to the largest values that quantisation gives (448 and 6 times 2^119
    and 2^125), infinite from 2^128 on.  The f16 form has no such end."""
    k = 1024

    def product(code, scale, w_code, w_scale, out):
        a, w = np.zeros((m, k), np.uint8), np.zeros((n, k // 2), np.uint8)
        sa, sw = np.full((m, k // 32), 127, np.uint8), np.full((n, k // 32), 127, np.uint8)
        a[:, 515], w[:, 257], sa[:, 16], sw[:, 16] = code, w_code << 4, scale, w_scale
        got = run_product((a, sa), (w, sw), "fp8", out=out)
        assert (got == got[0, 0]).all() or np.isnan(got).all()
        return float(got[0, 0])
    top, one, two, six, zero = 0x7e, 0x38, 4, 7, 0                       # (448, 1; 2, 6, 0)
    for out in ("f32", "f16"):
        assert product(top, 246, two, 5, out) == 448 * 2 * 2.0 ** -3
        assert product(one, 254, two, 0, out) == 2
        assert product(one, 7, six, 252, out) == 6 * 2.0 ** 5
    assert product(top, 247, two, 4, "f32") == product(one, 0, six, 253, "f32") == np.inf
    assert np.isnan(product(top, 254, zero, 127, "f32")) and np.isnan(product(0, 127, six, 254, "f32"))
    assert product(top, 247, two, 4, "f16") == 448 * 2 * 2.0 ** -3 and product(one, 0, six, 253, "f16") == 6 * 2.0 ** -1
    assert product(top, 254, zero, 127, "f16") == product(0, 127, six, 254, "f16") == 0
