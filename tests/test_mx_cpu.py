"""CPU tier of the MX formats and the RMS norm: the oracle against values fixed by the formats and
worked by hand, the host repacker against an independent model of the layout, and the refusals of
the C ABI and the binding (which touch no device)."""
from __future__ import annotations

import fractions
import re

import numpy as np
import pytest
import torch

import oracle
import w4_groupwise_gemm_amd as w4

F = fractions.Fraction


# ---- oracle

def test_element_tables():
    assert oracle.mx_elements(4).tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    v = oracle.mx_elements(8)
    # fixed points of E4M3: smallest subnormal and normal, one, largest
    assert len(v) == 127 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1.0 and v[126] == 448.0
    assert np.all(np.diff(v) > 0)


def test_rounding_by_hand():
    # midpoints go to the even code; beyond the largest value the largest
    a = np.array([0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 7.99, 1e9])
    assert oracle.nearest_code(a, 4).tolist() == [0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 7]
    a = np.array([2.0 ** -10, 2.0 ** -10 * 1.01, 3 * 2.0 ** -10, 17 / 16, 19 / 16, 432, 480, 1e9])
    # 2^-10 is half the smallest subnormal; 17/16 and 19/16 lie between 1, 9/8 and 10/8; 432 between 416 and 448
    assert oracle.nearest_code(a, 8).tolist() == [0, 1, 2, 0x38, 0x3A, 0x7E, 0x7E, 0x7E]


@pytest.mark.parametrize("fmt", [4, 8])
def test_nearest_code_against_rationals(fmt):
    vals = [F(float(v)) for v in oracle.mx_elements(fmt)]
    pts = []
    for lo, hi in zip(vals, vals[1:]):
        mid, q = (lo + hi) / 2, (hi - lo) / 64
        pts += [lo, lo + q, mid - q, mid, mid + q, hi - q]
    pts.append(vals[-1] * 2)
    got = oracle.nearest_code(np.array([float(p) for p in pts]), fmt)
    for p, c in zip(pts, got):
        d = [abs(p - v) for v in vals]
        best = [i for i, e in enumerate(d) if e == min(d)]
        want = best[0] if len(best) == 1 else next(i for i in best if i % 2 == 0)
        assert c == want, (float(p), c, want)


def test_block_scales_by_hand():
    x = np.zeros((6, 32))
    x[0, 5] = 6.0                    # E2M1: exponent 2 - 2 = 0; E4M3: 2 - 8 = -6
    x[1, 0], x[1, 1] = -7.5, 1.0     # saturates at -6
    x[2, 3] = 2.0 ** -130            # below the scales' range: byte 0
    x[3, 2], x[3, 4] = np.inf, 1.0
    x[4, 2], x[4, 4] = np.nan, 1.0
    x[5, 1] = -0.0
    c, b = oracle.quantize_mx(x, 4)
    assert b[:, 0].tolist() == [127, 127, 0, 255, 255, 0]
    assert c[0, 5] == 7 and c[1, 0] == 15 and c[1, 1] == 2 and c[2, 3] == 0 and c[5, 1] == 8
    assert not c[3].any() and not c[4].any()
    c, b = oracle.quantize_mx(x, 8)
    assert b[:, 0].tolist() == [121, 121, 0, 255, 255, 0]
    assert oracle.mx_elements(8)[c[0, 5]] == 384.0
    # 7.5 * 2^6 = 480 saturates at 448
    assert c[1, 0] == 128 + 126
    v = oracle.mx_value(c, b, 8)
    assert v[0, 5] == 6.0 and v[1, 0] == -7.0 and np.isnan(v[3]).all() and np.isnan(v[4]).all()


def test_values_that_quantise_to_themselves():
    rng = np.random.default_rng(3)
    for fmt in (4, 8):
        codes = rng.integers(0, 8 if fmt == 4 else 127, (5, 64)).astype(np.uint8)
        codes[:, ::32] = 7 if fmt == 4 else 126  # the largest element fixes the scale
        codes |= (rng.integers(0, 2, codes.shape) << (3 if fmt == 4 else 7)).astype(np.uint8)
        bytes_ = rng.integers(100, 140, (5, 2)).astype(np.uint8)
        c, b = oracle.quantize_mx(oracle.mx_value(codes, bytes_, fmt), fmt)
        assert np.array_equal(c, codes) and np.array_equal(b, bytes_)


def test_linear_mx_against_rationals():
    rng = np.random.default_rng(5)
    wc, wb = rng.integers(0, 16, (3, 64)).astype(np.uint8), rng.integers(120, 130, (3, 2)).astype(np.uint8)
    x = rng.standard_normal((2, 64)).astype(np.float16).astype(np.float64)
    y = oracle.linear_mx(x, wc, wb, 4)
    q, e = oracle.quantize_mx(x, 4)
    tab = [F(0), F(1, 2), F(1), F(3, 2), F(2), F(3), F(4), F(6)]
    val = lambda c: tab[c % 8] * (-1 if c >= 8 else 1)  # noqa: E731
    two = lambda n: F(2) ** int(n)                      # noqa: E731
    for t in range(2):
        for n in range(3):
            want = sum(val(q[t, k]) * val(wc[n, k]) * two(int(e[t, k // 32]) + int(wb[n, k // 32]) - 254) for k in range(64))
            assert abs(y[t, n] - float(want)) <= 1e-12 * (1 + abs(float(want)))


def test_rmsnorm_by_hand():
    y, h = oracle.rmsnorm([[3.0, 4.0]], [1.0, 2.0], 0.0)
    assert np.allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]], rtol=1e-15)
    y, h = oracle.rmsnorm([[1.0, 0.0]], [1.0, 1.0], 1.5, [[1.0, 0.0]])
    assert h.tolist() == [[2.0, 0.0]] and np.allclose(y, [[2 / np.sqrt(3.5), 0.0]], rtol=1e-15)


# ---- repacker

def _spec_pack(tiles, K):
    """Packed bytes of a list of (codes [16, K/2], scales [16, K/32]) row tiles, from the header."""
    KB = -(-K // 128)
    w = np.zeros((len(tiles), KB, 64, 16), np.uint8)
    s = np.zeros((len(tiles), KB, 16, 4), np.uint8)
    for i, (c, e) in enumerate(tiles):
        for kb in range(KB):
            for lane in range(64):
                k = 128 * kb + 32 * (lane // 16)
                if k < K:
                    w[i, kb, lane] = c[lane % 16, k // 2:k // 2 + 16]
                    s[i, kb, lane % 16, lane // 16] = e[lane % 16, k // 32]
    return w.reshape(-1), s.reshape(-1)


@pytest.mark.parametrize("N,K", [(16, 32), (32, 160), (48, 512), (16, 5152)])
def test_repack_matches_the_layout(N, K):
    rng = np.random.default_rng(N + K)
    mk = lambda: (rng.integers(0, 256, (N, K // 2)).astype(np.uint8), rng.integers(0, 256, (N, K // 32)).astype(np.uint8))  # noqa: E731
    g, u = mk(), mk()
    tiles = lambda m: [(m[0][i:i + 16], m[1][i:i + 16]) for i in range(0, N, 16)]  # noqa: E731
    w, s = w4.repack_mx(*g)
    rw, rs = _spec_pack(tiles(g), K)
    assert np.array_equal(w, rw) and np.array_equal(s, rs)
    w, s = w4.repack_mx_pair(g, u)
    rw, rs = _spec_pack([t for p in zip(tiles(g), tiles(u)) for t in p], K)
    assert np.array_equal(w, rw) and np.array_equal(s, rs)


# ---- C ABI refusals: fake addresses are fine because nothing touches the device

X, W, S, R, O, WS, H = (0x100000000 * i for i in range(1, 8))
BIG = 1 << 31


def _lin(fn="w4_linear_mx", x=X, w=W, s=S, r=R, T=4, N=64, K=256, fmt=8, dtype=0, out=O, ws=WS, nb=BIG):
    res = (r,) if fn == "w4_linear_add_mx" else ()
    return getattr(w4.lib(), fn)(x, w, s, *res, T, N, K, fmt, dtype, out, ws, nb, None)


@pytest.mark.parametrize("fn", ["w4_linear_mx", "w4_linear_swiglu_mx", "w4_linear_add_mx"])
def test_linear_mx_refusals(fn):
    assert _lin(fn, fmt=6) == -2 and _lin(fn, dtype=2) == -2
    for bad in (dict(T=-1), dict(N=0), dict(N=40), dict(K=0), dict(K=48), dict(w=None), dict(s=None), dict(out=None),
                dict(ws=None, x=None), dict(nb=w4.mx_workspace_bytes(4, 256, 8) - 1, x=None), dict(N=1 << 25), dict(K=1 << 25),
                dict(T=40, ws=None), dict(T=40, nb=w4.mx_workspace_bytes(40, 256, 8) - 1)):
        assert _lin(fn, **bad) == -1, bad
    for bad in (dict(x=X + 8), dict(w=W + 4), dict(s=S + 1), dict(out=O + 2), dict(T=40, ws=WS + 8), dict(x=None, ws=WS + 8)):
        assert _lin(fn, **bad) == -3, bad
    for bad in (dict(out=X), dict(out=W), dict(out=S), dict(T=40, ws=X), dict(T=40, ws=O), dict(x=None, ws=W), dict(out=X + 16)):
        assert _lin(fn, **bad) == -4, bad
    assert _lin(fn, T=0, x=None, w=None, s=None, out=None, ws=None) == 0
    assert _lin(fn, T=1 << 20, K=1024) == -2  # 2 GiB of activations
    if fn == "w4_linear_add_mx":
        assert _lin(fn, r=None) == -1 and _lin(fn, r=R + 8) == -3 and _lin(fn, r=O + 16) == -4 and _lin(fn, T=40, ws=R) == -4


def test_quantize_and_dequantize_refusals():
    L = w4.lib()
    q = lambda x=X, ldx=256, T=4, K=256, fmt=4, dtype=0, ws=WS, nb=BIG: L.w4_quantize_mx(x, ldx, T, K, fmt, dtype, ws, nb, None)  # noqa: E731
    assert q(fmt=5) == -2 and q(dtype=3) == -2
    for bad in (dict(T=-1), dict(K=0), dict(K=40), dict(ldx=248), dict(ldx=260), dict(x=None), dict(ws=None), dict(nb=8)):
        assert q(**bad) == -1, bad
    assert q(x=X + 2) == -3 and q(ws=WS + 8) == -3 and q(ws=X) == -4 and q(T=0, x=None, ws=None) == 0
    assert q(ws=X + (3 * 512 + 255) * 2, ldx=512) in (-3, -4)
    d = lambda ws=WS, nb=BIG, T=4, K=256, fmt=4, dtype=0, out=O: L.w4_dequantize_mx(ws, nb, T, K, fmt, dtype, out, None)  # noqa: E731
    assert d(fmt=0) == -2 and d(dtype=-1) == -2 and d(K=16) == -1 and d(out=None) == -1 and d(ws=None) == -1
    assert d(nb=100) == -1 and d(out=O + 8) == -3 and d(out=WS) == -4 and d(T=0, out=None) == 0
    e = lambda ws=WS, nb=BIG, T=4, K=256, dtype=0, out=O: L.w4_dequantize_a8(ws, nb, T, K, dtype, out, None)  # noqa: E731
    assert e(dtype=2) == -2 and e(K=96) == -1 and e(out=None) == -1 and e(ws=None) == -1 and e(nb=16) == -1
    assert e(out=O + 4) == -3 and e(out=WS) == -4 and e(T=0) == 0
    assert w4.mx_workspace_bytes(3, 160, 4) == 3 * (80 + 16) and w4.mx_workspace_bytes(2, 544, 8) == 2 * (544 + 32)
    assert w4.mx_workspace_bytes(3, 48, 4) == 0 and w4.mx_workspace_bytes(3, 64, 5) == 0
    assert w4.mx_packed_bytes(16, 160) == 2048 and w4.mx_packed_scale_bytes(16, 160) == 128
    assert w4.mx_packed_bytes(8, 160) == 0 and w4.mx_packed_scale_bytes(16, 100) == 0


def _norm(kind="", x=X, ldx=256, r=R, w=W, eps=1e-6, T=4, K=256, fmt=8, dtype=0, h=H, out=O, ws=WS, nb=BIG):
    L = w4.lib()
    if kind == "":
        return L.w4_rmsnorm(x, ldx, r, w, eps, T, K, dtype, h, out, None)
    if kind == "a8":
        return L.w4_rmsnorm_a8(x, ldx, r, w, eps, T, K, dtype, h, ws, nb, None)
    return L.w4_rmsnorm_mx(x, ldx, r, w, eps, T, K, fmt, dtype, h, ws, nb, None)


@pytest.mark.parametrize("kind", ["", "a8", "mx"])
def test_rmsnorm_refusals(kind):
    assert _norm(kind, dtype=7) == -2
    for bad in (dict(T=-1), dict(K=0), dict(ldx=255), dict(x=None), dict(w=None), dict(r=None), dict(h=None),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert _norm(kind, **bad) == -1, bad
    for bad in (dict(x=X + 2), dict(r=R + 8), dict(w=W + 4), dict(h=H + 2)):
        assert _norm(kind, **bad) == -3, bad
    for bad in (dict(h=X + 16), dict(h=R + 16), dict(h=W), dict(h=X, ldx=512)):
        assert _norm(kind, **bad) == -4, bad
    assert _norm(kind, T=0, x=None, r=None, h=None, w=None, out=None, ws=None) == 0
    if kind == "":
        assert _norm(kind, out=None) == -1 and _norm(kind, out=O + 2) == -3
        assert _norm(kind, out=H) == -4 and _norm(kind, out=W) == -4 and _norm(kind, out=X + 32) == -4
    else:
        assert _norm(kind, ws=None) == -1 and _norm(kind, nb=64) == -1 and _norm(kind, ws=WS + 4) == -3
        assert _norm(kind, ws=X) == -4 and _norm(kind, ws=R) == -4 and _norm(kind, ws=H) == -4 and _norm(kind, ws=W) == -4
        assert _norm(kind, K=80, ldx=80) == -1
    if kind == "mx":
        assert _norm(kind, fmt=16) == -2


# ---- binding refusals

def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros((2, 128), dtype=torch.float16)
    pw = w4.PackedMX(torch.zeros(w4.mx_packed_bytes(32, 128), dtype=torch.uint8),
                     torch.zeros(w4.mx_packed_scale_bytes(32, 128), dtype=torch.uint8), 32, 128)
    pair = w4.PackedMX(pw.w, pw.scales, 16, 128, True)
    q = w4.MXTensor(torch.zeros(4096, dtype=torch.uint8), 2, 128, 4)
    wt = torch.ones(128, dtype=torch.float16)
    for call in (lambda: w4.linear_mx(x, pw), lambda: w4.linear_mx(q, pw), lambda: w4.linear_add_mx(x, pw, x),
                 lambda: w4.quantize_mx(x), lambda: w4.dequantize_mx(q), lambda: w4.dequantize_a8(q.workspace, 2, 128),
                 lambda: w4.rmsnorm(x, wt), lambda: w4.rmsnorm_a8(x, wt), lambda: w4.rmsnorm_mx(x, wt),
                 lambda: w4.linear_mx(x, pair), lambda: w4.linear_swiglu_mx(x, pw)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError, match="fmt"):
        w4.rmsnorm_mx(x, wt, fmt=6)
    for codes, scales in ((np.zeros((16, 16), np.int8), np.zeros((16, 1), np.uint8)),
                          (np.zeros((16, 16), np.uint8), np.zeros((16, 2), np.uint8)),
                          (np.zeros((16, 16), np.uint8), np.zeros((32, 1), np.uint8)),
                          (np.zeros(16, np.uint8), np.zeros(1, np.uint8))):
        with pytest.raises(ValueError):
            w4.repack_mx(codes, scales)
    with pytest.raises(w4.W4Error):
        w4.repack_mx(np.zeros((8, 16), np.uint8), np.zeros((8, 1), np.uint8))  # 8 rows


def test_mx_tensor_views():
    q = w4.MXTensor(torch.arange(3 * (80 + 16), dtype=torch.uint8), 3, 160, 4)
    assert q.codes.shape == (3, 80) and q.scales.shape == (3, 5)
    assert q.codes[1, 0] == 80 and q.scales[1].tolist() == [(240 + 16 + i) % 256 for i in range(5)]


def test_routes_and_workspace_of_every_shape():
    """Every shape has a kernel; a workspace is asked for exactly where that is not the streaming one."""
    for op in (0, 1, 2):
        for fmt in (4, 8):
            for K in (32, 512, 5120, 5152, 17408, 65536, 1 << 20):
                for N in (16, 256, 5120, 12288):
                    for T in (1, 2, 4, 5, 8, 16, 17, 32, 33, 64, 65, 100, 256, 1000, 4096):
                        name, need = w4.mx_route_name(op, T, N, K, fmt), w4.linear_mx_workspace_bytes(op, T, N, K, fmt)
                        assert need == (0 if name.startswith("mx_stream") else w4.mx_workspace_bytes(T, K, fmt))
                        if op == 1:
                            assert not re.match(r"mx_(stream|ring)_r[135](_|$)", name)
                        if fmt == 8:
                            assert name != "mx_wide_320x256"
                        if name.startswith("mx_ring") and T <= 64:
                            assert int(name.rsplit("t", 1)[1]) == (16 if T <= 16 else 32 if T <= 32 else 64)
    for bad in ((3, 1, 16, 32, 4), (0, 1, 24, 32, 4), (0, 1, 16, 48, 4), (0, -1, 16, 32, 4), (0, 1, 16, 32, 5)):
        assert w4.mx_route_name(*bad) is None and w4.linear_mx_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("op,T,N,K,fmt,route", [
    (0, 1, 12288, 5120, 8, "mx_stream_r3"), (0, 8, 12288, 5120, 8, "mx_stream_r3"), (0, 16, 12288, 5120, 8, "mx_ring_r3_t16"),
    (1, 4, 17408, 5120, 8, "mx_stream_r10"), (1, 16, 17408, 5120, 8, "mx_ring_r10_t16"), (0, 4, 17408, 5120, 8, "mx_stream_r5"),
    (1, 64, 17408, 5120, 8, "mx_ring_r10_t64"), (2, 2, 5120, 17408, 4, "mx_stream_r2"),
    (2, 8, 5120, 17408, 4, "mx_ring_r2_t16"), (0, 64, 12288, 5120, 8, "mx_ring_r3_t64"), (0, 128, 12288, 5120, 8, "mx_wide_128x64"),
    (2, 4096, 5120, 6144, 4, "mx_wide_320x256"), (1, 1024, 17408, 5120, 4, "mx_wide_320x256"), (0, 4096, 10240, 5120, 8, "mx_wide_256x128")])
def test_route_choice_follows_the_measured_times(op, T, N, K, fmt, route):
    assert w4.mx_route_name(op, T, N, K, fmt) == route
