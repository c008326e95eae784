"""The 8-bit oracle against library casts, its definition and differences."""
import ml_dtypes
import numpy as np
import pytest

from oracle import fp8

LIB = {"e4m3": ml_dtypes.float8_e4m3fn, "e5m2": ml_dtypes.float8_e5m2}


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_decode_every_code(fmt):
    codes = np.arange(256, dtype=np.uint8)
    want = codes.view(LIB[fmt]).astype(np.float64)
    got = fp8.decode(codes, fmt)
    assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(np.signbit(got[~np.isnan(got)]), np.signbit(want[~np.isnan(want)]))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_encode_matches_library_cast(fmt):
    g = np.random.default_rng(5)
    v = np.concatenate([g.uniform(-1, 1, 20000) * fp8.FMAX[fmt], g.standard_normal(20000) * 2.0 ** g.integers(-20, 8, 20000)])
    grid = fp8.decode(np.arange(0, 256), fmt)
    grid = grid[np.isfinite(grid)]
    mid = (np.unique(grid)[1:] + np.unique(grid)[:-1]) / 2                  # every tie
    v = np.clip(np.concatenate([v, grid, mid, [0.0, -0.0]]), -fp8.FMAX[fmt], fp8.FMAX[fmt])
    v32 = v.astype(np.float32).astype(np.float64)
    want = v32.astype(np.float32).astype(LIB[fmt]).view(np.uint8)
    assert np.array_equal(fp8.encode(v32, fmt), want)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_scale_is_the_least_power_of_two_that_fits(fmt):
    g = np.random.default_rng(6)
    amax = np.concatenate([np.exp2(g.uniform(-110, 120, 500)), fp8.FMAX[fmt] * np.exp2(np.arange(-40.0, 40.0)),
                           np.nextafter(fp8.FMAX[fmt] * np.exp2(np.arange(-40.0, 40.0)), np.inf)])
    e = fp8.scale_exponent(amax, fmt)
    assert np.all(amax <= fp8.FMAX[fmt] * np.exp2(e.astype(float)))
    assert np.all(amax > fp8.FMAX[fmt] * np.exp2(e - 1.0))


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_half_step_and_special_blocks(fmt, tile):
    g = np.random.default_rng(7)
    x = g.standard_normal((150, 300)) * np.exp2(g.integers(-30, 30, (150, 1)))
    x[3] = 0.0
    codes, byte = fp8.quantize(x, fmt, tile)
    d = fp8.dequantize(codes, byte, fmt)
    scale = np.repeat(np.ldexp(1.0, byte.astype(int) - 127), 128, axis=1)[:, :300]
    m, low = (3, -6) if fmt == "e4m3" else (2, -14)
    assert np.all(np.abs(d - x) <= np.maximum(np.abs(x) * 2.0 ** -(m + 1), scale * 2.0 ** (low - m - 1)))
    x[5, 130] = np.inf
    x[149, 0] = np.nan
    codes, byte = fp8.quantize(x, fmt, tile)
    assert byte[5, 1] == 255 and byte[149, 0] == 255 and np.all(np.isnan(fp8.decode(codes[5, 128:256], fmt)))
    assert byte[140, 0] == (255 if tile else byte[140, 0]) and byte[3, 0] == 0 or tile


def test_transposed_tiles_have_the_same_values():
    x = np.random.default_rng(8).standard_normal((200, 264))
    a, b = fp8.quantize(x, "e4m3", True), fp8.quantize(x.T, "e4m3", True)
    assert np.array_equal(a[0], b[0].T)
    assert np.array_equal(a[1][::128], b[1][::128].T)


@pytest.mark.parametrize("cols", [8, 136])
def test_norm_gradient_against_differences(cols):
    g = np.random.default_rng(9)
    h, w, dy = g.standard_normal((3, cols)), 1 + 0.1 * g.standard_normal(cols), g.standard_normal((3, cols))
    eps = 1e-3

    def loss(h_, w_):
        return float((fp8.rmsnorm(h_, w_, eps)[0] * dy).sum())

    dh, dw = fp8.rmsnorm_backward(dy, h, w, fp8.rmsnorm(h, w, eps)[1])
    step = 1e-5                                     # central differences: error ~ step^2 + 2^-52 / step
    for i in range(3):
        for j in range(0, cols, 7):
            d = np.zeros_like(h)
            d[i, j] = step
            assert abs((loss(h + d, w) - loss(h - d, w)) / (2 * step) - dh[i, j]) < 1e-7
    for j in range(0, cols, 5):
        d = np.zeros_like(w)
        d[j] = step
        assert abs((loss(h, w + d) - loss(h, w - d)) / (2 * step) - dw[j]) < 1e-7


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_non_finite_elements_reach_their_block_only(fmt, bad):
    """Byte 255 and NaN codes in the element's whole 128 x 128 tile, or in its row's 1 x 128 block, and nowhere else."""
    x = np.random.default_rng(10).standard_normal((150, 300))
    x[3] = 0.0
    x[5, 130], x[149, 0] = bad, bad
    for tile in (True, False):
        codes, byte = fp8.quantize(x, fmt, tile)
        want = np.zeros(byte.shape, bool)
        if tile:
            want[:128, 1] = want[128:, 0] = True
        else:
            want[5, 1] = want[149, 0] = True
            assert np.all(byte[3] == 0)
        assert np.array_equal(byte == 255, want)
        assert np.array_equal(np.isnan(fp8.decode(codes, fmt)), np.repeat(want, 128, axis=1)[:, :300])
        assert np.array_equal(np.isnan(fp8.dequantize(codes, byte, fmt)), np.repeat(want, 128, axis=1)[:, :300])
