"""GPU tier: every kernel of the MX products at shapes that select it, ragged at its tiles' edges, against
the fp64 oracle on a sample of tokens and columns (tile edges among them), with the tolerances derived
in test_gpu_mx_linear.py; nothing outside the output is written and every output is."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import w4_groupwise_gemm_amd as w4
from test_gpu_mx_linear import OPS, TINY
from test_gpu_mx_quant import DTYPES, exact64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# (operation, T, N, K, format, kernel)
CASES = [
    ("linear", 1, 16, 32, 8, "mx_stream_r1"), ("add", 3, 1040, 2080, 4, "mx_stream_r1"), ("add", 16, 48, 1056, 8, "mx_stream_r1"),
    ("linear", 2, 4112, 2080, 8, "mx_stream_r2"), ("swiglu", 5, 1040, 1184, 4, "mx_stream_r2"), ("swiglu", 13, 16, 160, 8, "mx_stream_r2"),
    ("linear", 1, 8208, 5152, 8, "mx_stream_r3"), ("add", 7, 8208, 1184, 4, "mx_stream_r3"),
    ("linear", 2, 12304, 672, 4, "mx_stream_r4"), ("swiglu", 3, 4112, 2080, 8, "mx_stream_r4"),
    ("add", 3, 17424, 672, 8, "mx_stream_r5"), ("swiglu", 6, 8208, 672, 4, "mx_stream_r6"),
    ("swiglu", 9, 12304, 160, 8, "mx_stream_r8"), ("swiglu", 2, 17424, 1184, 4, "mx_stream_r10"), ("swiglu", 7, 17424, 416, 8, "mx_stream_r10"),
    ("add", 16, 48, 8224, 4, "mx_ring_r1_t16"), ("linear", 9, 528, 33024, 8, "mx_ring_r1_t16"),
    ("linear", 16, 4112, 5152, 8, "mx_ring_r2_t16"), ("swiglu", 12, 80, 8224, 4, "mx_ring_r2_t16"),
    ("add", 16, 8208, 5152, 8, "mx_ring_r3_t16"), ("linear", 16, 12304, 5152, 4, "mx_ring_r4_t16"), ("swiglu", 16, 4112, 5152, 8, "mx_ring_r4_t16"),
    ("linear", 12, 17424, 5152, 4, "mx_ring_r5_t16"), ("swiglu", 12, 8208, 5152, 8, "mx_ring_r6_t16"),
    ("swiglu", 15, 12304, 5152, 4, "mx_ring_r8_t16"), ("swiglu", 13, 17424, 5152, 8, "mx_ring_r10_t16"),
    ("swiglu", 16, 17424, 5152, 4, "mx_ring_r10_t16"),
    ("add", 21, 17424, 1184, 8, "mx_ring_r5_t32"), ("swiglu", 32, 8208, 2080, 4, "mx_ring_r6_t32"),
    ("swiglu", 18, 12304, 672, 4, "mx_ring_r8_t32"), ("swiglu", 31, 17424, 1184, 8, "mx_ring_r10_t32"),
    ("swiglu", 24, 17424, 672, 4, "mx_ring_r10_t32"),
    ("linear", 63, 17424, 1184, 4, "mx_ring_r5_t64"), ("swiglu", 45, 8208, 1184, 8, "mx_ring_r6_t64"),
    ("swiglu", 64, 12304, 672, 8, "mx_ring_r8_t64"), ("swiglu", 49, 17424, 2080, 4, "mx_ring_r10_t64"),
    ("swiglu", 60, 17424, 1184, 8, "mx_ring_r10_t64"),
    ("linear", 17, 16, 160, 8, "mx_ring_r1_t32"), ("add", 30, 528, 5152, 4, "mx_ring_r1_t32"),
    ("linear", 32, 4112, 2080, 4, "mx_ring_r2_t32"), ("swiglu", 25, 272, 1184, 8, "mx_ring_r2_t32"),
    ("add", 31, 8208, 1184, 8, "mx_ring_r3_t32"), ("linear", 19, 12304, 672, 4, "mx_ring_r4_t32"), ("swiglu", 28, 4112, 672, 8, "mx_ring_r4_t32"),
    ("add", 33, 48, 160, 4, "mx_ring_r1_t64"), ("linear", 64, 528, 8224, 8, "mx_ring_r1_t64"),
    ("linear", 63, 4112, 1184, 8, "mx_ring_r2_t64"), ("swiglu", 40, 1040, 2080, 4, "mx_ring_r2_t64"), ("add", 65, 2064, 672, 8, "mx_ring_r2_t64"),
    ("add", 64, 8208, 2080, 4, "mx_ring_r3_t64"), ("linear", 50, 12304, 672, 8, "mx_ring_r4_t64"), ("swiglu", 37, 4112, 1184, 8, "mx_ring_r4_t64"),
    ("linear", 65, 4112, 1184, 8, "mx_wide_64x64"), ("swiglu", 70, 2064, 160, 4, "mx_wide_64x64"), ("add", 90, 4112, 2080, 4, "mx_wide_64x64"),
    ("add", 65, 8208, 672, 8, "mx_ring_r5_t64"), ("linear", 128, 12304, 416, 8, "mx_wide_128x64"), ("swiglu", 65, 4112, 544, 4, "mx_wide_128x64"),
    ("linear", 200, 12304, 416, 4, "mx_wide_128x128"), ("swiglu", 65, 12304, 288, 8, "mx_wide_128x128"), ("add", 200, 12304, 1184, 8, "mx_wide_128x128"),
    ("add", 500, 12304, 288, 8, "mx_wide_256x128"), ("linear", 1000, 12304, 160, 4, "mx_wide_256x128"), ("swiglu", 257, 17424, 672, 4, "mx_wide_256x128"),
    ("add", 4100, 4112, 160, 4, "mx_wide_320x256"), ("swiglu", 1000, 8208, 416, 4, "mx_wide_320x256"), ("linear", 4100, 4112, 1184, 4, "mx_wide_320x256"),
    ("add", 1, 1040, 51200, 8, "mx_stream_r1"),  # over 64 KB of LDS
    ("linear", 40, 48, 131072, 8, "mx_wide_64x64"), ("linear", 5, 32, 524288, 4, "mx_wide_64x64"),  # rows too long for the ring's LDS
]


def _edges(n, step, count, rng):
    e = {0, 1, 15, 16, 31, 32, 63, 64, n - 1, n - 2, n - 16, n - 17, n // step * step, n // step * step - 1}
    e |= set(rng.integers(0, n, count).tolist())
    return np.array(sorted(i for i in e if 0 <= i < n))


@pytest.mark.parametrize("op,T,N,K,fmt,route", CASES)
def test_kernel(op, T, N, K, fmt, route):
    assert w4.mx_route_name(OPS.index(op), T, N, K, fmt) == route
    for dtype in (("fp16", "bf16")[T % 2],):
        dt = DTYPES[dtype]
        g = torch.Generator(device=DEV).manual_seed(T + N + K)
        rng = np.random.default_rng(T + N + K)
        ws = [(torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=g),
               torch.randint(117, 122, (N, K // 32), dtype=torch.uint8, device=DEV, generator=g)) for _ in range(2 if op == "swiglu" else 1)]
        x = torch.randn(T, K, device=DEV, generator=g) * (0.5 if op == "swiglu" else 1) * min(1.0, 40 / K ** 0.5)
        x[:, torch.randint(0, K, (max(1, K // 640),), device=DEV, generator=g)] *= 10
        x = x.to(dt)
        r = torch.randn(T, N, device=DEV, generator=g).to(dt)
        pw = w4.pack_mx_pair(*ws, device=DEV) if op == "swiglu" else w4.pack_mx(*ws[0], device=DEV)
        buf = torch.full((T + 2, N), float("nan"), dtype=dt, device=DEV)
        buf[0] = buf[-1] = 3
        out = buf[1:-1]
        kw = dict(fmt=fmt, out=out)
        if op == "add":
            w4.linear_add_mx(x, pw, r, **kw)
        elif op == "swiglu":
            w4.linear_swiglu_mx(x, pw, **kw)
        else:
            w4.linear_mx(x, pw, **kw)
        assert (buf[0] == 3).all() and (buf[-1] == 3).all() and out.isfinite().all()

        rows, cols = _edges(T, 256, 24, rng), _edges(N, 320, 200, rng)
        a = oracle.mx_value(*oracle.quantize_mx(exact64(x[torch.from_numpy(rows).to(DEV)]), fmt), fmt)
        ci = torch.from_numpy(cols).to(DEV)
        wv = [oracle.mx_value(oracle.unpack_fp4(c[ci].cpu().numpy()), e[ci].cpu().numpy(), 4) for c, e in ws]
        p = [a @ w.T for w in wv]
        rel = (-(-K // 128) + 16) * 2.0 ** -24 + (2.0 ** -12 if fmt == 8 else 0)
        d = [np.abs(a) @ np.abs(w).T * rel for w in wv]
        if op == "swiglu":
            s = oracle.silu(p[0])
            y = s * p[1]
            tol = np.abs(p[1]) * 1.1 * d[0] + np.abs(s) * d[1] + 1.1 * d[0] * d[1] + np.abs(y) * 2.0 ** -20
        else:
            y = p[0] + (exact64(r)[np.ix_(rows, cols)] if op == "add" else 0)
            tol = d[0] + np.abs(y) * 2.0 ** -24
        tol = tol + (np.abs(y) + tol) * torch.finfo(dt).eps / 2 + TINY[dt]
        got = exact64(out)[np.ix_(rows, cols)]
        bad = ~(np.abs(got - y) <= tol)
        assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], got[bad][:4], y[bad][:4], tol[bad][:4])
