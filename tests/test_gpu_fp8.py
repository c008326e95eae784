"""8-bit quantizers and products on the GPU against the 64-bit oracle."""
import numpy as np
import pytest
import torch

import microscaling_fp4_quantization_mxfp4_b200 as fp
from oracle import fp8, sf_from_mma

pytestmark = pytest.mark.gpu


def _input(rows, cols, seed, ld=None):
    """bf16 [rows, cols] in rows of `ld` with changing magnitudes, a zero block, -0 and subnormal elements."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-40, 40, (rows, 1), generator=g).float())
    x[0, :128] = 0.0
    x[rows // 2, : min(cols, 24)] = -0.0
    x[rows - 1, cols // 2:] = 1e-39
    buf = torch.full((rows, ld or cols), float("nan"), dtype=torch.bfloat16)
    buf[:, :cols] = x.to(torch.bfloat16)
    return buf.cuda()[:, :cols]


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _check(q, x64, fmt, tile, sf):
    """Codes and scales bit for bit, the layout's padding included."""
    codes, byte = fp8.quantize(x64, fmt, tile)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    s = q.scales.cpu().numpy()
    assert np.array_equal(s, byte if sf == "rowmajor" else fp8.mma(byte))


SHAPES = [(1, 8), (1, 128), (3, 120), (2, 136), (5, 384), (127, 1000), (128, 512), (129, 640), (300, 264), (1030, 520)]


@pytest.mark.parametrize("sf", ["rowmajor", "mma"])
@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows, cols", SHAPES)
def test_quantize(rows, cols, fmt, axis, sf):
    x = _input(rows, cols, rows + cols, cols + (24 if rows % 2 else 0))
    q = fp.fp4_fp8_quantize(x, fmt, axis, sf)
    _check(q, _f64(x) if axis == 1 else _f64(x).T, fmt, False, sf)


@pytest.mark.parametrize("sf", ["rowmajor", "mma"])
@pytest.mark.parametrize("transposed", [True, False])
@pytest.mark.parametrize("rows, cols", SHAPES)
def test_quantize_2d(rows, cols, transposed, sf):
    x = _input(rows, cols, rows * cols, cols + (8 if rows % 2 else 0))
    for fmt in ("e4m3", "e5m2"):
        q, t = fp.fp4_fp8_quantize_2d(x, fmt, sf, transposed)
        _check(q, _f64(x), fmt, True, sf)
        assert (t is not None) == transposed
        if transposed:
            _check(t, _f64(x).T, fmt, True, sf)


@pytest.mark.parametrize("axis", [1, 0, 2])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_non_finite_blocks_are_nan(bad, axis):
    x = _input(200, 264, 3)
    x[70, 100], x[199, 263] = bad, bad
    if axis == 2:
        q = fp.fp4_fp8_quantize_2d(x)[0]
        _check(q, _f64(x), "e4m3", True, "rowmajor")
    else:
        q = fp.fp4_fp8_quantize(x, axis=axis)
        _check(q, _f64(x) if axis == 1 else _f64(x).T, "e4m3", False, "rowmajor")
    d = fp.fp4_fp8_dequantize(q.codes, q.scales)
    assert torch.isnan(d).sum() == (q.scales.repeat_interleave(128, 1)[:, : d.shape[1]] == 255).sum() > 0


def test_bytes_past_the_rows_are_left_alone():
    for axis, (rows, cols) in ((1, (37, 72)), (0, (37, 72))):
        orows, length = (rows, cols) if axis == 1 else (cols, rows)
        buf = torch.full((orows, 112), 0xA5, dtype=torch.uint8, device="cuda")
        fp.fp4_fp8_quantize(_input(rows, cols, 1), axis=axis, codes=buf[:, :length])
        assert torch.all(buf[:, length:] == 0xA5)
    buf, buf_t = (torch.full((n, 112), 0xA5, dtype=torch.uint8, device="cuda") for n in (37, 72))
    fp.fp4_fp8_quantize_2d(_input(37, 72, 1), codes=buf[:, :72], codes_t=buf_t[:, :37])
    assert torch.all(buf[:, 72:] == 0xA5) and torch.all(buf_t[:, 37:] == 0xA5)


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sf", ["rowmajor", "mma"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows, cols", [(1, 1), (3, 127), (130, 136), (64, 1001)])
def test_dequantize(rows, cols, fmt, sf, out_dtype):
    g = np.random.default_rng(rows + cols)
    codes = g.integers(0, 256, (rows, (cols + 15) // 16 * 16), dtype=np.uint8)
    byte = g.integers(64, 190, (rows, -(-cols // 128)), dtype=np.uint8)
    byte[0, 0] = 255
    byte[rows - 1, -1] = 0
    want = fp8.dequantize(codes[:, :cols], byte, fmt)
    c = torch.from_numpy(codes).cuda()[:, :cols]
    s = torch.from_numpy(byte if sf == "rowmajor" else fp8.mma(byte)).cuda()
    got = fp.fp4_fp8_dequantize(c, s, fmt, sf, out_dtype)
    want = torch.from_numpy(want).float() if out_dtype == "f32" else torch.from_numpy(want).float().to(torch.bfloat16)
    assert torch.equal(torch.nan_to_num(got.cpu(), 7.0), torch.nan_to_num(want, 7.0))


# ---------------------------------------------------------------- products --
def _operand(rows, k, fmt, seed, tile=False):
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, k)) * np.exp2(g.integers(-6, 7, (rows, 1)))
    codes, byte = fp8.quantize(x, fmt, tile)
    c = torch.full((rows, (k + 15) // 16 * 16 + 16), 0x7F, dtype=torch.uint8)      # NaN past the row's end
    c[:, :k] = torch.from_numpy(codes)
    return c.cuda()[:, :k], torch.from_numpy(fp8.mma(byte)).cuda(), fp8.dequantize(codes, byte, fmt)


def _bound(k, absum):
    # products are exact in fp32 (8 significant bits at most, power-of-two scales); k of them are added in
    # fp32 in some order, each addition off by at most one unit of the last place (2^-23; the tensor core need not
    # round to nearest), so the sum is off by at most k * 2^-23 * sum |a b|, to first order
    return (k + 8) * 2.0 ** -23 * absum


def _check_gemm(M, N, K, a_fmt="e4m3", b_fmt="e4m3", seed=0, ldy=None):
    a, sa, av = _operand(M, K, a_fmt, seed)
    b, sb, bv = _operand(N, K, b_fmt, seed + 1, tile=True)
    want, absum = fp8.gemm(av, bv)
    for dtype in (torch.float32, torch.bfloat16):
        buf = torch.full((M + 1, (ldy or N)), 77.0, dtype=dtype, device="cuda")
        y = fp.fp4_fp8_gemm(a, sa, b, sb, a_fmt, b_fmt, out=buf[:M, :N])
        fp.fp4_check_device_errors()
        tol = _bound(K, absum) + (0 if dtype == torch.float32 else 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8))
        err = np.abs(_f64(y) - want)
        assert np.all(err <= tol), (M, N, K, dtype, float((err / np.maximum(tol, 1e-300)).max()))
        assert torch.all(buf[M:] == 77.0) and torch.all(buf[:, N:] == 77.0)


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 100, 128, 129, 257])
@pytest.mark.parametrize("N, K", [(1, 1), (128, 128), (136, 31), (300, 640), (257, 1000), (16, 4104)])
def test_gemm(M, N, K):
    _check_gemm(M, N, K, seed=M + N + K)


@pytest.mark.parametrize("K", [16, 127, 129, 511, 512, 513, 1024, 1025, 2047, 5000])
def test_gemm_lengths(K):
    _check_gemm(40, 200, K, seed=K)


@pytest.mark.parametrize("M", [1, 20, 64, 65])
@pytest.mark.parametrize("K", [256, 300, 500, 640, 700, 800, 1100])
def test_gemm_slices(M, K):
    """K over 2 to 8 CTAs: slices of 64 columns down to 16, those of 3, 5, 6 and 7 CTAs cut unevenly, on a short last tile."""
    _check_gemm(M, 202, K, seed=9, ldy=203)


@pytest.mark.parametrize("a_fmt, b_fmt", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("M, N, K", [(1, 130, 300), (70, 260, 999), (600, 520, 1032)])
def test_gemm_types(M, N, K, a_fmt, b_fmt):
    _check_gemm(M, N, K, a_fmt, b_fmt, seed=5)


@pytest.mark.parametrize("M, N, K, ldy", [(3, 33, 256, 40), (3, 33, 256, 33), (200, 130, 256, 131), (700, 300, 640, 304)])
def test_gemm_row_strides(M, N, K, ldy):
    _check_gemm(M, N, K, seed=6, ldy=ldy)


@pytest.mark.parametrize("M, N, K", [(2048, 2304, 768), (4096, 4096, 1024), (2500, 2700, 2200), (1000, 4096, 1500)])
def test_gemm_large(M, N, K):
    _check_gemm(M, N, K, seed=7)


@pytest.mark.parametrize("M, N, K, ldy", [
    (130, 300, 5000, 304), (300, 513, 4100, 513),        # few tiles, long K: K over clusters, more than 128 rows
    (2048, 2304, 768, 2304), (1500, 2000, 300, 2001),    # 256 x 256 tiles
    (513, 1000, 1016, 1008), (257, 200, 1600, 201),      # 256 x 192 tiles, rows of codes 16 bytes off a sector
    (96, 9600, 256, 9600), (128, 9501, 520, 9501),       # 65 to 128 rows against many weights
    (40, 9600, 300, 9600), (16, 20000, 264, 20000)])     # one CTA a tile, more tiles than SMs
def test_gemm_kernels(M, N, K, ldy):
    _check_gemm(M, N, K, "e5m2", "e4m3", seed=8, ldy=ldy)


@pytest.mark.parametrize("M", [1, 40, 700])
def test_gemm_nan_blocks_reach_their_rows_only(M):
    a, sa, av = _operand(M, 300, "e4m3", 1)
    b, sb, bv = _operand(260, 300, "e4m3", 2)
    byte = sf_from_mma(sa.cpu().numpy(), M, 3)
    byte[M - 1, 1] = 255
    a[M - 1, 128:256] = 0x7F
    y = fp.fp4_fp8_gemm(a, torch.from_numpy(fp8.mma(byte)).cuda(), b, sb)
    nan = torch.isnan(y)
    assert torch.all(nan[M - 1]) and not torch.any(nan[: M - 1])


@pytest.mark.parametrize("M, N, K", [(1, 512, 512), (300, 512, 1024), (2048, 2048, 2048)])
def test_gemm_repeats_bit_for_bit(M, N, K):
    a, sa, _ = _operand(M, K, "e4m3", 1)
    b, sb, _ = _operand(N, K, "e4m3", 2)
    first = fp.fp4_fp8_gemm(a, sa, b, sb, out_dtype="f32")
    for _ in range(3):
        assert torch.equal(fp.fp4_fp8_gemm(a, sa, b, sb, out_dtype="f32"), first)


def test_offsets_past_32_bits():
    """2.4e9 elements: the last rows (and columns, along axis 0) are those of the same rows on their own."""
    rows, cols = 600_040, 4096
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(0, rows, 65536):
        x[i:i + 65536] = torch.randn(min(65536, rows - i), cols, generator=g, device="cuda").to(torch.bfloat16)
    last = (rows - 1) // 128 * 128 - 128                            # a whole and a partial block of 128 rows
    part = x[last:].clone()
    q = fp.fp4_fp8_quantize(x, sf_layout="mma")
    p = fp.fp4_fp8_quantize(part, sf_layout="mma")
    assert torch.equal(q.codes[last:], p.codes) and torch.equal(q.scales[-p.scales.numel():], p.scales)
    w = torch.randn(24, cols, generator=g, device="cuda").to(torch.bfloat16)
    wq = fp.fp4_fp8_quantize(w, sf_layout="mma")
    y = fp.fp4_fp8_gemm(q.codes, q.scales, wq.codes, wq.scales, out_dtype="f32")
    z = fp.fp4_fp8_gemm(wq.codes, wq.scales, q.codes, q.scales, out_dtype="f32")
    a = fp.fp4_fp8_dequantize(p.codes, p.scales, "e4m3", "mma").double()
    b = fp.fp4_fp8_dequantize(wq.codes, wq.scales, "e4m3", "mma").double()
    tol = _bound(cols, (a.abs() @ b.abs().t()).cpu().numpy())
    assert np.all((y[last:].double() - a @ b.t()).abs().cpu().numpy() <= tol)
    assert np.all((z[:, last:].t().double() - a @ b.t()).abs().cpu().numpy() <= tol)
    del q, y, z
    q, p = fp.fp4_fp8_quantize(x, axis=0), fp.fp4_fp8_quantize(part, axis=0)
    assert torch.equal(q.codes[:, last:], p.codes) and torch.equal(q.scales[:, -2:], p.scales)
    del q
    n, m = fp.fp4_rmsnorm_fp8_quantize(x, w[0], x), fp.fp4_rmsnorm_fp8_quantize(part, w[0], part)
    assert torch.equal(n.codes[last:], m.codes) and torch.equal(n.residual_out[last:], m.residual_out)
    assert torch.equal(n.rstd[last:], m.rstd)
    dx = fp.fp4_rmsnorm_backward(x, n.residual_out, w[0], n.rstd, x, dx=n.residual_out)[0]
    assert torch.equal(dx[last:], fp.fp4_rmsnorm_backward(part, m.residual_out, w[0], m.rstd, part)[0])


def test_streams_and_graphs():
    """Two streams at once, and the calls captured and replayed on new inputs, give the plain calls' bits."""
    x = [torch.randn(300, 640, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    w = torch.randn(512, 640, device="cuda", dtype=torch.bfloat16)
    wq = fp.fp4_fp8_quantize_2d(w, sf_layout="mma", transposed=False)[0]

    def linear(t, stream=None):
        q = fp.fp4_fp8_quantize(t, sf_layout="mma", stream=stream)
        return fp.fp4_fp8_gemm(q.codes, q.scales, wq.codes, wq.scales, stream=stream)

    want = [linear(t) for t in x]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [linear(t, s) for t, s in zip(x, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    static = x[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = linear(static)
    for t, expect in ((x[1], want[1]), (x[0], want[0])):
        static.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, expect)


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    q = fp.fp4_fp8_quantize(x, sf_layout="mma")
    row = fp.fp4_fp8_quantize(x)
    for call in (lambda: fp.fp4_fp8_quantize(x.float()), lambda: fp.fp4_fp8_quantize(x.t()),
                 lambda: fp.fp4_fp8_quantize(x, codes=torch.empty(4, 48, dtype=torch.uint8, device="cuda")),
                 lambda: fp.fp4_fp8_quantize(x, scales=torch.empty(4, 2, dtype=torch.uint8, device="cuda")),
                 lambda: fp.fp4_fp8_quantize(x, codes=torch.empty(4, 64, dtype=torch.uint8)),
                 lambda: fp.fp4_fp8_gemm(q.codes, row.scales, q.codes, q.scales),
                 lambda: fp.fp4_fp8_gemm(q.codes, q.scales, q.codes[:, :48], q.scales),
                 lambda: fp.fp4_fp8_gemm(q.codes, q.scales, q.codes, q.scales.cpu()),
                 lambda: fp.fp4_fp8_gemm(q.codes, q.scales, q.codes, q.scales, out=torch.empty(4, 5, device="cuda")),
                 lambda: fp.fp4_fp8_gemm(q.codes.float(), q.scales, q.codes, q.scales),
                 lambda: fp.fp4_fp8_dequantize(q.codes, q.scales)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fp.Fp4Error):
        fp.fp4_fp8_quantize(torch.zeros(4, 60, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(fp.Fp4Error):
        fp.fp4_fp8_quantize(x[:0])
    with pytest.raises(KeyError):
        fp.fp4_fp8_quantize(x, "e3m4")


def test_types_of_codes_and_scales():
    """Codes may have their format's own type, scales E8M0's; another format's type is refused, not read as this one's."""
    x = torch.randn(4, 128, device="cuda", dtype=torch.bfloat16)
    q = fp.fp4_fp8_quantize(x, "e5m2", sf_layout="mma")
    c, s = q.codes.view(torch.float8_e5m2), q.scales.view(torch.float8_e8m0fnu)
    assert torch.equal(fp.fp4_fp8_gemm(c, s, c, s, "e5m2", "e5m2"),
                       fp.fp4_fp8_gemm(q.codes, q.scales, q.codes, q.scales, "e5m2", "e5m2"))
    assert torch.equal(fp.fp4_fp8_dequantize(c, s, "e5m2", "mma"), fp.fp4_fp8_dequantize(q.codes, q.scales, "e5m2", "mma"))
    for call in (lambda: fp.fp4_fp8_gemm(c, s, c, s), lambda: fp.fp4_fp8_gemm(c, s, c, s, "e5m2"),
                 lambda: fp.fp4_fp8_dequantize(c, s, sf_layout="mma"), lambda: fp.fp4_fp8_quantize(x, codes=c),
                 lambda: fp.fp4_fp8_dequantize(c, q.scales.view(torch.float8_e5m2), "e5m2", "mma"),
                 lambda: fp.fp4_fp8_quantize_2d(x, transposed=False, codes_t=q.codes)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("M, N, K", [(3, 40, 130), (100, 130, 300), (300, 260, 31), (600, 520, 2200)])
def test_gemm_reads_nothing_past_its_operands(M, N, K):
    """NaN codes past K in the rows, and NaN scales in the layout's padding, change no bit of the product."""
    def operand(rows, seed):
        g = torch.Generator().manual_seed(seed)
        L = (K + 7) // 8 * 8
        x = torch.randn(rows, L, generator=g).to(torch.bfloat16).cuda()
        q = fp.fp4_fp8_quantize(x, sf_layout="mma")
        wide = torch.full((rows, (K + 15) // 16 * 16 + 32), 0x7F, dtype=torch.uint8, device="cuda")
        wide[:, :K] = q.codes[:, :K]
        groups = (K + 127) // 128
        byte = np.full(((rows + 127) // 128 * 128, (groups + 3) // 4 * 4), 255, np.uint8)
        scales = fp.fp4_fp8_quantize(x).scales.cpu().numpy()[:, :groups]
        byte[:rows, :groups] = scales
        plain = np.zeros_like(byte)
        plain[:rows, :groups] = scales
        return (q.codes[:, :K], torch.from_numpy(fp8.mma(plain)).cuda(), wide[:, :K], torch.from_numpy(fp8.mma(byte)).cuda())

    a, b = operand(M, 1), operand(N, 2)
    want = fp.fp4_fp8_gemm(a[0], a[1], b[0], b[1], out_dtype="f32")
    assert torch.all(torch.isfinite(want))
    assert torch.equal(fp.fp4_fp8_gemm(a[2], a[3], b[2], b[3], out_dtype="f32"), want)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_another_device_than_the_current_one():
    """Each device runs every kernel on its own: what was set up for the first is not taken for the second."""
    def run(dev):
        g = torch.Generator().manual_seed(1)
        out = []
        for M, N, K in ((1, 256, 512), (100, 256, 512), (400, 512, 2048)):
            a, b = (torch.randn(n, K, generator=g).to(torch.bfloat16).to(dev) for n in (M, N))
            w = torch.ones(K, device=dev)
            q, wq = fp.fp4_rmsnorm_fp8_quantize(a, w, a, sf_layout="mma"), fp.fp4_fp8_quantize(b, sf_layout="mma")
            out += [fp.fp4_fp8_gemm(q.codes, q.scales, wq.codes, wq.scales),
                    *fp.fp4_rmsnorm_backward(a, q.residual_out, w, q.rstd, a)]
        torch.cuda.synchronize(dev)
        return [t.cpu() for t in out]

    assert all(torch.equal(a, b) for a, b in zip(run("cuda:0"), run("cuda:1")))


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("length", [1, 2, 3, 4, 5, 6, 7, 8, 9, 13, 127, 129, 1003])
def test_dequantize_of_rows_that_end_with_their_codes(length, out_dtype):
    """A row without padding, and a matrix whose last row ends with its last code."""
    pitch = (length + 15) // 16 * 16
    for rows in (1, 3):
        g = np.random.default_rng(length + rows)
        flat = g.integers(0, 256, ((rows - 1) * pitch + length,), dtype=np.uint8)
        codes = torch.from_numpy(flat).cuda().as_strided((rows, length), (pitch if rows > 1 else length, 1))
        byte = g.integers(100, 150, (rows, -(-length // 128)), dtype=np.uint8)
        got = fp.fp4_fp8_dequantize(codes, torch.from_numpy(byte).cuda(), out_dtype=out_dtype)
        want = torch.from_numpy(fp8.dequantize(codes.cpu().numpy(), byte)).float().to(got.dtype)
        assert torch.equal(torch.nan_to_num(got.cpu(), 7.0), torch.nan_to_num(want, 7.0))


def _operand_in_rows(rows, k, fmt, seed, pitch, tile=False):
    """As _operand, rows `pitch` bytes apart and the values on the GPU."""
    g = np.random.default_rng(seed)
    codes, byte = fp8.quantize(g.standard_normal((rows, k)) * np.exp2(g.integers(-6, 7, (rows, 1))), fmt, tile)
    c = torch.full((rows, pitch), 0x7F, dtype=torch.uint8)
    c[:, :k] = torch.from_numpy(codes)
    return c.cuda()[:, :k], torch.from_numpy(fp8.mma(byte)).cuda(), torch.from_numpy(fp8.dequantize(codes, byte, fmt)).cuda()


@pytest.mark.parametrize("M, N, K, pitch, a_fmt, b_fmt", [
    (4096, 4096, 2048, 2048, "e4m3", "e4m3"),      # 5 waves of 192 columns against 4 of 256, rows on sector borders
    (4001, 4001, 2008, 2016, "e5m2", "e4m3"),      # the same, ragged
    (2500, 5000, 1600, 1600, "e4m3", "e5m2"),      # 4 against 3
    (4096, 5111, 520, 528, "e4m3", "e4m3")])       # 6 against 5 with a short K, rows off sector borders
def test_gemm_waves_of_192_columns(M, N, K, pitch, a_fmt, b_fmt):
    """The second accumulator and its reuse, with tiles whose scales start in the middle of an atom: every element."""
    a, sa, av = _operand_in_rows(M, K, a_fmt, M + K, pitch)
    b, sb, bv = _operand_in_rows(N, K, b_fmt, N + K, pitch, tile=True)
    want, absum = av @ bv.t(), av.abs() @ bv.abs().t()
    for dtype in (torch.float32, torch.bfloat16):
        y = fp.fp4_fp8_gemm(a, sa, b, sb, a_fmt, b_fmt, out_dtype="f32" if dtype == torch.float32 else "bf16")
        fp.fp4_check_device_errors()
        assert y.dtype == dtype
        tol = _bound(K, absum) + (0 if dtype == torch.float32 else 2.0 ** -8 * want.abs() * (1 + 2.0 ** -8))
        assert bool(torch.all((y.double() - want).abs() <= tol))


def test_more_blocks_than_threads_in_32_bits():
    """Past 2^30 blocks (rows of 8 elements) a thread's number passes 32 bits: the last rows are those of the same rows alone."""
    rows, n = (1 << 30) + 1000, 2000
    x = torch.zeros(rows, 8, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(1)
    for part in (x[:n], x[-n:]):
        part.copy_(torch.randn(n, 8, generator=g) * torch.exp2(torch.randint(-9, 9, (n, 1), generator=g).float()))
    codes = torch.full((rows, 16), 0xA5, dtype=torch.uint8, device="cuda")[:, :8]
    scales = torch.full((rows, 1), 0xA5, dtype=torch.uint8, device="cuda")
    q = fp.fp4_fp8_quantize(x, codes=codes, scales=scales)
    for part in (slice(0, n), slice(rows - n, rows)):
        alone = fp.fp4_fp8_quantize(x[part].clone())
        assert torch.equal(q.codes[part], alone.codes) and torch.equal(q.scales[part], alone.scales)
    assert torch.all(q.codes[1 << 29:(1 << 29) + n] == 0) and torch.all(q.scales[1 << 29:(1 << 29) + n] == 0)
