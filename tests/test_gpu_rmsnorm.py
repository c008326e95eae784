"""RMS norm with residual and 8-bit output, and its backward pass, against 64 bits; a training step of both."""
import numpy as np
import pytest
import torch

import microscaling_fp4_quantization_mxfp4_b200 as fp
from oracle import fp8, sf_from_mma

pytestmark = pytest.mark.gpu
U = 2.0 ** -24                    # half a step of fp32, relative


def _rand(rows, cols, seed, std=1.0, ld=None):
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((rows, ld or cols), float("nan"), dtype=torch.bfloat16)
    buf[:, :cols] = (torch.randn(rows, cols, generator=g) * std).to(torch.bfloat16)
    return buf.cuda()[:, :cols]


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _check_quantized(codes, byte, y, fmt, rel):
    """Codes and scale bytes of values known to a relative error `rel`: the scale is that of a maximum within
    `rel` of the true one, and each code is the nearest to a value within `rel` of the true one."""
    rows, cols = y.shape
    pad = np.zeros((rows, -(-cols // 128) * 128))
    pad[:, :cols] = np.abs(y)
    amax = pad.reshape(rows, -1, 128).max(axis=2)
    lo = np.where(amax == 0, 0, fp8.scale_exponent(amax * (1 - rel), fmt) + 127)
    hi = np.where(amax == 0, 0, fp8.scale_exponent(amax * (1 + rel), fmt) + 127)
    assert np.all((lo <= byte) & (byte <= hi))
    d = fp8.dequantize(codes, byte, fmt)
    scale = np.repeat(np.ldexp(1.0, byte.astype(int) - 127), 128, axis=1)[:, :cols]
    m, low = (3, -6) if fmt == "e4m3" else (2, -14)
    tol = np.maximum(np.abs(y) * (1 + rel) * 2.0 ** -(m + 1), scale * 2.0 ** (low - m - 1)) + np.abs(y) * rel
    assert np.all(np.abs(d - y) <= tol)


def _norm_case(rows, cols, residual=True, wf32=False, fmt="e4m3", sf="mma", seed=0, eps=1e-6, ld=None, norm_out=True):
    x, r = _rand(rows, cols, seed, 1.0, ld), (_rand(rows, cols, seed + 1, 2.0, ld) if residual else None)
    w = (1 + 0.1 * torch.randn(cols, generator=torch.Generator().manual_seed(seed + 2)))
    w = w.cuda() if wf32 else w.to(torch.bfloat16).cuda()
    yo = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda") if norm_out else None
    q = fp.fp4_rmsnorm_fp8_quantize(x, w, r, eps, fmt, sf, norm_out=yo)
    h = x
    if residual:
        h = (x.float() + r.float()).to(torch.bfloat16)
        assert torch.equal(q.residual_out, h)
    else:
        assert q.residual_out is None
    y, rstd = fp8.rmsnorm(_f64(h), w.double().cpu().numpy(), eps)
    # sum of squares: cols non-negative terms, every partial sum off by at most (cols + 1) U; the square root
    # halves that; the division, the addition of eps, the reciprocal root and two products add 5 U
    rel = ((cols + 1) / 2 + 3) * U
    assert np.all(np.abs(q.rstd.double().cpu().numpy() - rstd) <= rel * rstd)
    rel += 2 * U
    g = -(-cols // 128)
    s = q.scales.cpu().numpy()
    if sf == "mma":
        byte = sf_from_mma(s, rows, g)
        assert np.array_equal(fp8.mma(byte), s)                  # padding bytes are zero
    else:
        byte = s
    _check_quantized(q.codes.cpu().numpy(), byte, y, fmt, rel)
    if norm_out:
        assert np.all(np.abs(_f64(yo) - y) <= (2.0 ** -8 * (1 + rel) + rel) * np.abs(y))


@pytest.mark.parametrize("rows", [1, 2, 127, 129, 300])
@pytest.mark.parametrize("cols", [8, 64, 128, 136, 768, 1000, 2056, 4096, 11008, 16384])
def test_norm(rows, cols):
    _norm_case(rows, cols, seed=rows + cols)


@pytest.mark.parametrize("residual, wf32, fmt, sf, norm_out, ld", [
    (False, False, "e4m3", "mma", True, None), (False, True, "e4m3", "rowmajor", False, 1040),
    (True, True, "e5m2", "mma", False, 1040), (True, False, "e5m2", "rowmajor", True, None)])
@pytest.mark.parametrize("rows", [3, 200])
def test_norm_forms(rows, residual, wf32, fmt, sf, norm_out, ld):
    _norm_case(rows, 1000, residual, wf32, fmt, sf, 11, 1e-5, ld, norm_out)


def test_norm_zero_rows_and_non_finite_rows():
    x = _rand(6, 264, 1)
    x[1] = 0.0
    x[3, 200] = float("inf")
    x[4, 7] = float("nan")
    w = torch.ones(264, dtype=torch.bfloat16, device="cuda")
    q = fp.fp4_rmsnorm_fp8_quantize(x, w, eps=1e-6)
    assert torch.all(q.codes[1] & 0x7F == 0) and torch.all(q.scales[1] == 0)
    assert abs(float(q.rstd[1]) - 1e3) <= 1e3 * 4 * U + 1e3 * 2.0 ** -24        # eps itself is rounded to fp32
    d = fp.fp4_fp8_dequantize(q.codes, q.scales)
    assert torch.all(torch.isnan(d[4])) and torch.all(q.scales[4] == 255)
    assert float(q.rstd[3]) == 0.0 and q.scales[3, 1] == 255 and torch.all(d[3, :128] == 0)
    for i in (0, 2, 5):                                              # their neighbours keep their values
        _check_quantized(q.codes[i:i + 1].cpu().numpy(), q.scales[i:i + 1].cpu().numpy(),
                         fp8.rmsnorm(_f64(x[i:i + 1]), np.ones(264), 1e-6)[0], "e4m3", 300 * U)


def test_norm_in_place_residual():
    x, r = _rand(50, 512, 1), _rand(50, 512, 2)
    w = torch.ones(512, device="cuda")
    want = fp.fp4_rmsnorm_fp8_quantize(x, w, r)
    r2 = r.clone()
    got = fp.fp4_rmsnorm_fp8_quantize(x, w, r2, residual_out=r2)
    assert got.residual_out is r2 and torch.equal(r2, want.residual_out) and torch.equal(got.codes, want.codes)
    x2 = x.clone()
    got = fp.fp4_rmsnorm_fp8_quantize(x2, w, r, residual_out=x2)
    assert torch.equal(x2, want.residual_out) and torch.equal(got.codes, want.codes)


def _backward_case(rows, cols, dres=True, wf32=False, seed=0, ld=None):
    h, dy = _rand(rows, cols, seed, 3.0, ld), _rand(rows, cols, seed + 1, 0.1, ld)
    dr = _rand(rows, cols, seed + 2, 0.1, ld) if dres else None
    w = 1 + 0.1 * torch.randn(cols, generator=torch.Generator().manual_seed(seed + 3))
    w = w.cuda() if wf32 else w.to(torch.bfloat16).cuda()
    w64 = w.double().cpu().numpy()
    rstd = torch.from_numpy(fp8.rmsnorm(_f64(h), w64, 1e-6)[1]).float().cuda()
    dx, dw = fp.fp4_rmsnorm_backward(dy, h, w, rstd, dr)
    r64 = rstd.double().cpu().numpy()
    want, wantw = fp8.rmsnorm_backward(_f64(dy), _f64(h), w64, r64, None if dr is None else _f64(dr))
    # mean(g * xh): each term off by 3 U, sums of cols terms by cols * U of the sum of magnitudes;
    # dx: g and xh 1 U each, their combination and the final sum a few more; then the rounding to bf16
    g, xh, r = np.abs(_f64(dy) * w64), np.abs(_f64(h) * r64[:, None]), r64[:, None]
    cerr = (cols + 5) * U * (g * xh).mean(axis=1, keepdims=True)
    cabs = np.abs((_f64(dy) * w64 * _f64(h) * r).mean(axis=1, keepdims=True))
    err = r * (g * 4 * U + xh * (cabs * 6 * U + cerr)) + 4 * U * (np.abs(want) + (0 if dr is None else np.abs(_f64(dr))))
    assert np.all(np.abs(_f64(dx) - want) <= err + 2.0 ** -8 * (np.abs(want) + err))
    terms = np.abs(_f64(dy)) * xh
    assert np.all(np.abs(dw.double().cpu().numpy() - wantw) <= (rows + 4) * U * terms.sum(axis=0))


@pytest.mark.parametrize("rows", [1, 3, 129, 1100])
@pytest.mark.parametrize("cols", [8, 136, 768, 1000, 2056, 4096, 11008, 16384])
def test_backward(rows, cols):
    _backward_case(rows, cols, seed=rows + cols)


@pytest.mark.parametrize("dres, wf32, ld", [(False, False, None), (False, True, 1040), (True, True, 1040)])
@pytest.mark.parametrize("rows", [5, 700])
def test_backward_forms(rows, dres, wf32, ld):
    _backward_case(rows, 1000, dres, wf32, 4, ld)


def test_backward_repeats_and_runs_on_two_streams_at_once():
    h, dy = _rand(3000, 1024, 1), _rand(3000, 1024, 2)
    w = torch.ones(1024, device="cuda")
    rstd = torch.rand(3000, device="cuda")
    want = fp.fp4_rmsnorm_backward(dy, h, w, rstd)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        got = [fp.fp4_rmsnorm_backward(dy, h, w, rstd, stream=s) for s in streams]
        torch.cuda.synchronize()
        for dx, dw in got:
            assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def test_backward_in_place():
    h, dy, dr = _rand(70, 256, 1), _rand(70, 256, 2), _rand(70, 256, 3)
    w = torch.ones(256, device="cuda")
    rstd = torch.rand(70, device="cuda")
    want = fp.fp4_rmsnorm_backward(dy, h, w, rstd, dr)[0]
    for i in range(3):
        t = [dy.clone(), h.clone(), dr.clone()]
        assert torch.equal(fp.fp4_rmsnorm_backward(t[0], t[1], w, rstd, t[2], dx=t[i])[0], want)


def test_backward_of_tiny_rows():
    """eps = 0 and rows near 1e-20: rstd squared is past fp32, dx is not."""
    h, dy = _rand(3, 264, 1, 1e-20), _rand(3, 264, 2, 1e-3)
    rstd = torch.from_numpy(fp8.rmsnorm(_f64(h), np.ones(264), 0.0)[1]).float().cuda()
    dx, dw = fp.fp4_rmsnorm_backward(dy, h, torch.ones(264, device="cuda"), rstd)
    want, wantw = fp8.rmsnorm_backward(_f64(dy), _f64(h), np.ones(264), rstd.double().cpu().numpy())
    r = rstd.double().cpu().numpy()[:, None]
    g, xh = np.abs(_f64(dy)), np.abs(_f64(h) * r)
    err = (264 + 16) * U * r * (g + xh * (g * xh).mean(axis=1, keepdims=True))
    assert np.all(np.abs(_f64(dx) - want) <= err + 2.0 ** -8 * (np.abs(want) + err))
    assert np.all(np.abs(dw.double().cpu().numpy() - wantw) <= 7 * U * (g * xh).sum(axis=0))


def test_two_graphs_share_nothing():
    """Norm and backward captured twice and replayed in turn on new inputs give the plain calls' bits."""
    w = torch.ones(1032, device="cuda")

    def step(x, r, dy):
        q = fp.fp4_rmsnorm_fp8_quantize(x, w, r, sf_layout="mma")
        return (q.codes, q.scales, q.residual_out, q.rstd, *fp.fp4_rmsnorm_backward(dy, q.residual_out, w, q.rstd, r))

    data = [[_rand(300, 1032, 10 * i + j) for j in range(3)] for i in range(2)]
    want = [[t.clone() for t in step(*d)] for d in data]
    graphs, statics, outs = [], [], []
    for i in range(2):
        static = [t.clone() for t in data[i]]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(*static)
        graphs.append(graph), statics.append(static), outs.append(out)
    for turn in range(4):
        for i in range(2):
            for s, d in zip(statics[i], data[(i + turn) % 2]):
                s.copy_(d)
        graphs[0].replay(), graphs[1].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want[(i + turn) % 2]))


def test_backward_workspace_is_checked():
    h = _rand(70, 256, 1)
    w, rstd = torch.ones(256, device="cuda"), torch.rand(70, device="cuda")
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(fp.Fp4Error):
        fp.fp4_rmsnorm_backward(h, h, w, rstd, workspace=small)
    with pytest.raises(fp.Fp4Error):
        fp.fp4_rmsnorm_backward(h[:, :252].contiguous(), h[:, :252].contiguous(), w[:252], rstd)


def test_binding_refusals():
    x = _rand(4, 64, 1)
    w = torch.ones(64, device="cuda")
    q = fp.fp4_rmsnorm_fp8_quantize(x, w, x)
    for call in (lambda: fp.fp4_rmsnorm_fp8_quantize(x, w[:32]), lambda: fp.fp4_rmsnorm_fp8_quantize(x, w.half()),
                 lambda: fp.fp4_rmsnorm_fp8_quantize(x, w, x[:2]), lambda: fp.fp4_rmsnorm_fp8_quantize(x, w, residual_out=x),
                 lambda: fp.fp4_rmsnorm_fp8_quantize(x, w, rstd=torch.empty(3, device="cuda")),
                 lambda: fp.fp4_rmsnorm_fp8_quantize(x.cpu(), w), lambda: fp.fp4_rmsnorm_fp8_quantize(x, w.cpu()),
                 lambda: fp.fp4_rmsnorm_backward(x, x, w, q.rstd[:2]), lambda: fp.fp4_rmsnorm_backward(x, x[:3], w, q.rstd),
                 lambda: fp.fp4_rmsnorm_backward(x, x, w, q.rstd, dx=torch.empty(4, 64, device="cuda"))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("tokens", [1, 333])
def test_training_step(tokens):
    """Norm -> linear and back: y = Q(norm(x + r)) . Q(W)^T, dgrad through W^T's codes, wgrad along the tokens, the
    norm's backward -- each against 64-bit products of the operands' own values."""
    cols, n = 384, 520
    x, r, w = _rand(tokens, cols, 1), _rand(tokens, cols, 2), torch.ones(cols, device="cuda")
    W, dY = _rand(n, cols, 3, 0.05), _rand(tokens, n, 4, 1e-3)
    yn = torch.empty(tokens, cols, dtype=torch.bfloat16, device="cuda")
    q = fp.fp4_rmsnorm_fp8_quantize(x, w, r, sf_layout="mma", norm_out=yn)
    wq, wt = fp.fp4_fp8_quantize_2d(W, sf_layout="mma")
    Y = fp.fp4_fp8_gemm(q.codes, q.scales, wq.codes, wq.scales, out_dtype="f32")
    g1 = fp.fp4_fp8_quantize(dY, "e5m2", 1, "mma")
    dx = fp.fp4_fp8_gemm(g1.codes, g1.scales, wt.codes, wt.scales, "e5m2", "e4m3")
    gt, xt = fp.fp4_fp8_quantize(dY, "e5m2", 0, "mma"), fp.fp4_fp8_quantize(yn, "e4m3", 0, "mma")
    dW = fp.fp4_fp8_gemm(gt.codes, gt.scales, xt.codes, xt.scales, "e5m2", "e4m3", "f32")
    dh, dw = fp.fp4_rmsnorm_backward(dx, q.residual_out, w, q.rstd, r)

    def val(t, fmt):
        return fp.fp4_fp8_dequantize(t.codes, t.scales, fmt, "mma").double().cpu().numpy()

    def close(got, a, b, k, bits):
        want, absum = fp8.gemm(a, b)
        tol = (k + 8) * 2.0 ** -23 * absum
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol + bits * (np.abs(want) + tol))

    close(Y, val(q, "e4m3"), val(wq, "e4m3"), cols, 0)
    close(dx, val(g1, "e5m2"), val(wt, "e4m3"), n, 2.0 ** -8)
    close(dW, val(gt, "e5m2"), val(xt, "e4m3"), tokens, 0)
    # and against the unquantized step: every operand is within half a code step of its value (2^-4 E4M3, 2^-3 E5M2)
    yn64, W64, dY64 = _f64(yn), _f64(W), _f64(dY)
    want, absum = np.abs(yn64 @ W64.T - Y.double().cpu().numpy()), np.abs(yn64) @ np.abs(W64).T
    amax = np.abs(yn64).max() * np.abs(W64).max() * cols            # codes near zero: absolute steps, 2^-18 of the maxima
    assert np.all(want <= (2 * 2.0 ** -4 + 2.0 ** -8 + 2.0 ** -7) * absum + 2.0 ** -16 * amax)
    # the norm's backward of what it was given: dh rounds to bf16 (2^-8) after fp32 sums of cols terms, dw sums `tokens`
    h64, r64 = _f64(q.residual_out), q.rstd.double().cpu().numpy()
    want64, wantw = fp8.rmsnorm_backward(_f64(dx), h64, np.ones(cols), r64, _f64(r))
    g, xh = np.abs(_f64(dx)), np.abs(h64 * r64[:, None])
    err = (cols + 16) * U * r64[:, None] * (g + xh * (g * xh).mean(axis=1, keepdims=True)) + 8 * U * np.abs(_f64(r))
    assert np.all(np.abs(_f64(dh) - want64) <= err + 2.0 ** -8 * (np.abs(want64) + err))
    assert np.all(np.abs(dw.double().cpu().numpy() - wantw) <= (tokens + 4) * U * (g * xh).sum(axis=0))


def _check_rstd(rstd, want):
    # the mean of squares and its root are taken in fp64 (squares of bf16 are exact there; 16384 additions are off by
    # 2^-39 at most, in any order), so rstd is off by its rounding to fp32: U, or half the subnormals' step 2^-149
    assert np.all(np.abs(rstd.double().cpu().numpy() - want) <= U * want * (1 + 2.0 ** -10) + 2.0 ** -150)


@pytest.mark.parametrize("rows", [1, 300])
@pytest.mark.parametrize("cols", [8, 136, 1000, 2056, 4096, 11008, 16384])
def test_norm_rstd_is_rounded_once(rows, cols):
    x = _rand(rows, cols, rows * cols, 3.0)
    eps = float(np.float32(1e-5))
    q = fp.fp4_rmsnorm_fp8_quantize(x, torch.ones(cols, device="cuda"), eps=eps)
    _check_rstd(q.rstd, fp8.rmsnorm(_f64(x), np.ones(cols), eps)[1])


@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("cols", [8, 264, 2056, 4096])
def test_norm_over_the_range_of_bf16(cols, few):
    """Rows of any finite magnitude keep their values, with eps = 0 too: squares neither overflow nor vanish."""
    g = torch.Generator().manual_seed(cols)
    rows = [torch.full((cols,), 1.5 * 2.0 ** 62), torch.randn(cols, generator=g) * 1e37, torch.randn(cols, generator=g) * 1e-23,
            torch.randn(cols, generator=g) * 1e-30, torch.full((cols,), 3.3e38), torch.full((cols,), 1e-37),
            torch.randn(cols, generator=g), torch.where(torch.arange(cols) == cols - 3, 1.5 * 2.0 ** 63, 0.0),
            torch.where(torch.arange(cols) % 8 < 3, 1e30, 1e-30), torch.where(torch.arange(cols) < 8, 1e-25, 0.0)]
    x = torch.stack(rows).to(torch.bfloat16)
    x = (x if few else x.repeat(30, 1)).cuda()
    w = torch.ones(cols, device="cuda")
    q = fp.fp4_rmsnorm_fp8_quantize(x, w, eps=0.0)
    y, rstd = fp8.rmsnorm(_f64(x), np.ones(cols), 0.0)
    _check_rstd(q.rstd, rstd)
    # y: rstd's rounding (half the subnormals' step, 2^-150, of at least 2^-128: 2^-22) and two products, U each
    _check_quantized(q.codes.cpu().numpy(), q.scales.cpu().numpy(), y, "e4m3", 2.0 ** -22 + 3 * U)


def test_norm_past_the_range_of_rstd():
    """eps = 0: rows whose root mean square is below 2^-128, zeros among them, have an infinite rstd and NaN codes."""
    x = torch.zeros(3, 264, dtype=torch.bfloat16, device="cuda")
    x[1], x[2] = 1e-40, 1.0
    q = fp.fp4_rmsnorm_fp8_quantize(x, torch.ones(264, device="cuda"), eps=0.0)
    assert torch.all(torch.isinf(q.rstd[:2])) and float(q.rstd[2]) == 1.0
    assert torch.all(q.scales[:2] == 255) and torch.all(fp.fp4_fp8_dequantize(q.codes, q.scales)[2] == 1.0)
