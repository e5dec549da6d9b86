"""GPU tier: the RMS norm with residual addition, in every output form, against the fp64 oracle.

Tolerances.  The sum of squares is a chain of at most 8 * (vectors per lane) fused adds and about 22
more (lanes, waves): below 64 roundings of 2^-24 for the widths here, half of that in 1 / sqrt; forming
h, the division, the root and two products add 6 more.  So y is within 2^-18 of the exact value
relatively before its rounding to 16 bits (half a step: eps / 2, or half the smallest subnormal)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import w4_groupwise_gemm_amd as w4
from test_gpu_mx_quant import DTYPES, device_codes, exact64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
REL = 2.0 ** -18
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def inputs(T, K, dtype, residual=True, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed * 1000 + T + K)
    x = (torch.randn(T, K, generator=g) * scale).to(dtype)
    r = (torch.randn(T, K, generator=g) * scale).to(dtype) if residual else None
    w = (1 + 0.2 * torch.randn(K, generator=g)).to(dtype)
    return x.to(DEV), None if r is None else r.to(DEV), w.to(DEV)


def reference(x, r, w, eps):
    return oracle.rmsnorm(exact64(x), exact64(w), eps, None if r is None else exact64(r))


def check_rounded(got, want, dtype, rel):
    tol = np.abs(want) * (torch.finfo(dtype).eps / 2 * (1 + rel) + rel) + TINY[dtype]
    bad = np.abs(exact64(got) - want) > tol
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4])


def check_a8(ws, T, K, y):
    """Codes within half a step (and the fp32 error) of y, scales within it, of each group."""
    raw = ws.cpu().numpy()
    q = raw[:T * K].view(np.int8).reshape(T, K // 8, 8)
    codes = np.empty_like(q)
    codes[:, :, [0, 4, 1, 5, 2, 6, 3, 7]] = q
    codes = codes.reshape(T, K).astype(np.float64)
    off, KB = (T * K + 15) // 16 * 16, (K + 127) // 128
    s = raw[off:off + KB * T * 8].view(np.float32).reshape(KB, T, 2).transpose(1, 0, 2).reshape(T, 2 * KB)
    assert not s[:, K // 64:].any()
    s = s[:, :K // 64].astype(np.float64)
    want = np.abs(y).reshape(T, -1, 64).max(2) / 127
    assert np.all(np.abs(s - want) <= want * 2 * REL + 2.0 ** -149)
    s = np.repeat(s, 64, 1)
    assert np.all(np.abs(codes * s - y) <= s * (0.5 + 127 * 4 * REL)), np.max(np.abs(codes * s - y) / s)


def check_mx(q, y):
    """Scale bytes those of y moved by less than the fp32 error; codes the nearest to such a y."""
    lo, hi = y * (1 - REL), y * (1 + REL)
    bl, bh = oracle.quantize_mx(lo, q.fmt)[1], oracle.quantize_mx(hi, q.fmt)[1]
    b = q.scales.cpu().numpy()
    assert np.all((b >= bl) & (b <= bh))
    unit = np.repeat(np.ldexp(1.0, b.astype(np.int64) - 127), 32, 1)
    half = 8 if q.fmt == 4 else 128
    c = device_codes(q)
    assert np.all((c >= half) == np.signbit(y))
    mag = c % half
    assert np.all(mag >= oracle.nearest_code(np.abs(lo) / unit, q.fmt))
    assert np.all(mag <= oracle.nearest_code(np.abs(hi) / unit, q.fmt))


SHAPES = [(1, 1), (1, 7), (3, 64), (2, 65), (5, 511), (4, 5119), (7, 5120), (130, 512), (2, 8193), (3, 17408),
          (2, 32768), (2, 32769), (1, 40001)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,K", SHAPES)
def test_16_bit_output(T, K, dtype):
    dt = DTYPES[dtype]
    for residual in (True, False):
        x, r, w = inputs(T, K, dt, residual)
        y, h = w4.rmsnorm(x, w, eps=1e-5, residual=r)
        wy, wh = reference(x, r, w, 1e-5)
        check_rounded(y, wy, dt, REL)
        if residual:
            check_rounded(h, wh, dt, 2.0 ** -24)
        else:
            assert h is None


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,K", [(1, 64), (3, 192), (5, 704), (9, 5120), (2, 17408), (1, 33024)])
def test_a8_output(T, K, dtype):
    x, r, w = inputs(T, K, DTYPES[dtype])
    ws, h = w4.rmsnorm_a8(x, w, eps=1e-6, residual=r)
    wy, wh = reference(x, r, w, 1e-6)
    check_a8(ws, T, K, wy)
    check_rounded(h, wh, DTYPES[dtype], 2.0 ** -24)


@pytest.mark.parametrize("fmt", [4, 8])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,K", [(1, 32), (3, 96), (5, 544), (17, 5120), (2, 17408), (1, 33024)])
def test_mx_output(T, K, dtype, fmt):
    x, r, w = inputs(T, K, DTYPES[dtype])
    q, h = w4.rmsnorm_mx(x, w, fmt=fmt, eps=1e-6, residual=r)
    wy, wh = reference(x, r, w, 1e-6)
    check_mx(q, wy)
    check_rounded(h, wh, DTYPES[dtype], 2.0 ** -24)
    off, stride = T * K * fmt // 8, (K + 511) // 512 * 16
    rows = q.workspace[off:off + T * stride].view(T, stride).cpu().numpy()
    assert not rows[:, K // 32:].any()


def test_many_rows():
    x, r, w = inputs(4099, 128, torch.bfloat16)
    y, h = w4.rmsnorm(x, w, residual=r)
    wy, wh = reference(x, r, w, 1e-6)
    check_rounded(y, wy, torch.bfloat16, REL)
    check_rounded(h, wh, torch.bfloat16, 2.0 ** -24)


def test_more_rows_than_a_grid_dimension():
    T, K = 70001, 64
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(T, K, device=DEV, generator=g).half()
    w = torch.ones(K, device=DEV).half()
    y, _ = w4.rmsnorm(x, w)
    q, _ = w4.rmsnorm_mx(x, w)
    d = w4.dequantize_mx(q)
    rows = torch.tensor([0, 1, 65535, 65536, 65537, T - 1], device=DEV)
    y6, _ = w4.rmsnorm(x[rows], w)
    q6, _ = w4.rmsnorm_mx(x[rows], w)
    assert torch.equal(y[rows], y6) and torch.equal(q.codes[rows], q6.codes) and torch.equal(q.scales[rows], q6.scales)
    assert torch.equal(d[rows], w4.dequantize_mx(q6))
    assert torch.equal(w4.quantize_mx(x).codes[rows], w4.quantize_mx(x[rows]).codes)
    ws, _ = w4.rmsnorm_a8(x, w)
    ws6, _ = w4.rmsnorm_a8(x[rows], w)
    assert torch.equal(w4.dequantize_a8(ws, T, K)[rows], w4.dequantize_a8(ws6, 6, K))


def test_on_another_stream():
    x, r, w = inputs(33, 5120, torch.float16)
    want = [w4.rmsnorm(x, w, residual=r), w4.rmsnorm_mx(x, w, residual=r), w4.rmsnorm_a8(x, w, residual=r)]
    wq = w4.quantize_mx(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y, h = w4.rmsnorm(x, w, residual=r, stream=s)
    q, _ = w4.rmsnorm_mx(x, w, residual=r, stream=s)
    ws, _ = w4.rmsnorm_a8(x, w, residual=r, stream=s)
    xq = w4.quantize_mx(x, stream=s)
    d = w4.dequantize_mx(xq, stream=s)
    e = w4.dequantize_a8(ws, 33, 5120, stream=s)
    s.synchronize()
    assert torch.equal(y, want[0][0]) and torch.equal(h, want[0][1])
    assert torch.equal(q.codes, want[1][0].codes) and torch.equal(q.scales, want[1][0].scales)
    assert torch.equal(xq.codes, wq.codes) and torch.equal(d, w4.dequantize_mx(wq))
    assert torch.equal(e, w4.dequantize_a8(want[2][0], 33, 5120))


@pytest.mark.parametrize("K,stride,off", [(288, 1024, 256), (257, 1001, 8), (256, 259, 0)])
def test_strided_rows(K, stride, off):
    g = torch.Generator().manual_seed(K)
    wide = torch.randn(6, stride, generator=g).half().to(DEV)
    x = wide[:, off:off + K]
    _, r, w = inputs(6, K, torch.float16)
    y, h = w4.rmsnorm(x, w, residual=r)
    y2, h2 = w4.rmsnorm(x.contiguous(), w, residual=r)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    check_rounded(y, reference(x, r, w, 1e-6)[0], torch.float16, REL)


@pytest.mark.parametrize("K", [200, 5120, 33000])
def test_in_place_forms(K):
    x, r, w = inputs(5, K, torch.float16)
    y, h = w4.rmsnorm(x, w, residual=r)
    r2 = r.clone()
    y2, h2 = w4.rmsnorm(x, w, residual=r2, residual_out=r2)   # the residual stream updated in place
    assert h2 is r2 and torch.equal(y2, y) and torch.equal(h2, h)
    x2, r2 = x.clone(), r.clone()
    w4.rmsnorm(x2, w, residual=r2, residual_out=r2, out=x2)   # and y over x
    assert torch.equal(x2, y) and torch.equal(r2, h)
    x2, r2 = x.clone(), r.clone()
    w4.rmsnorm(x2, w, residual=r2, residual_out=x2, out=r2)
    assert torch.equal(x2, h) and torch.equal(r2, y)
    x2 = x.clone()
    y3, _ = w4.rmsnorm(x, w)
    w4.rmsnorm(x2, w, out=x2)
    assert torch.equal(x2, y3)


def test_zero_rows_extremes_and_guard_rows():
    x, _, w = inputs(6, 512, torch.float16, False)
    x[1] = 0
    x[2] = 65504.0
    x[3] = 6e-8
    out = torch.full((8, 512), 3.0, dtype=torch.float16, device=DEV)
    w4.rmsnorm(x, w, out=out[:6])
    wy, _ = reference(x, None, w, 1e-6)
    check_rounded(out[:6], wy, torch.float16, REL)
    assert (out[6:] == 3).all() and (out[1] == 0).all()
    for fmt in (4, 8):  # a row of zeros: scale bytes 0, codes 0 (with the sign of the weight's product)
        q, _ = w4.rmsnorm_mx(x, w, fmt=fmt)
        assert not q.scales[1].any()
        assert (w4.dequantize_mx(q)[1] == 0).all()
    ws, _ = w4.rmsnorm_a8(x, w)
    assert (w4.dequantize_a8(ws, 6, 512)[1] == 0).all()


def test_infinities_and_nans_stay_in_their_rows():
    x, _, w = inputs(4, 256, torch.bfloat16, False)
    x[1, 70] = float("inf")
    x[2, 3] = float("nan")
    y, _ = w4.rmsnorm(x, w)
    assert y[0].isfinite().all() and y[3].isfinite().all() and y[2].isnan().all()
    assert y[1, 70].isnan() and (y[1, :70] == 0).all()  # inf * 0, and finite * 0
    q, _ = w4.rmsnorm_mx(x, w)
    d = w4.dequantize_mx(q, dtype=torch.bfloat16)
    assert d[0].isfinite().all() and d[3].isfinite().all() and d[2].isnan().all() and d[1, 64:96].isnan().all()
    ws, _ = w4.rmsnorm_a8(x, w)
    d = w4.dequantize_a8(ws, 4, 256, dtype=torch.bfloat16)
    assert d[0].isfinite().all() and d[3].isfinite().all() and d[2].isnan().all() and d[1, 64:128].isnan().all()


def test_binding_refusals():
    x, r, w = inputs(4, 96, torch.float16)
    with pytest.raises(ValueError):
        w4.rmsnorm(x, w.bfloat16())
    with pytest.raises(ValueError):
        w4.rmsnorm(x, w[:64])
    with pytest.raises(ValueError):
        w4.rmsnorm(x.float(), w)
    with pytest.raises(ValueError):
        w4.rmsnorm(x, w, residual=r[:2])
    with pytest.raises(ValueError):
        w4.rmsnorm(x, w, residual_out=r)
    with pytest.raises(ValueError):
        w4.rmsnorm_a8(x, w)  # 96 is no multiple of 64
    with pytest.raises(ValueError):
        w4.rmsnorm_mx(x[:, :48].contiguous(), w[:48])
    with pytest.raises(ValueError):
        w4.rmsnorm(x[:, ::2], w[:48])
    with pytest.raises(ValueError):
        w4.rmsnorm(x[:1].expand(4, 96), w)
    with pytest.raises(w4.W4Error):
        w4.rmsnorm(x, w, eps=-1.0)
    y, h = w4.rmsnorm(x[:0], w, residual=r[:0])
    assert y.shape == (0, 96) and h.shape == (0, 96)
