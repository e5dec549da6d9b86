"""GPU tier: MX quantisation and reading back, and the A8 workspace read back, against the fp64
oracle.  Dividing by a power of two and choosing the nearest element are exact decisions, so codes,
scale bytes and (after one rounding) values are compared bit for bit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import w4_groupwise_gemm_amd as w4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def exact64(t):
    return t.detach().cpu().double().numpy()


def device_codes(q):
    c = q.codes.cpu().numpy()
    return oracle.unpack_fp4(c) if q.fmt == 4 else c


def check_quantised(q, x):
    codes, bytes_ = oracle.quantize_mx(exact64(x), q.fmt)
    assert np.array_equal(q.scales.cpu().numpy(), bytes_)
    assert np.array_equal(device_codes(q), codes)
    # the bytes past K / 32 of each row of scales
    off, stride = q.T * q.K * q.fmt // 8, (q.K + 511) // 512 * 16
    rows = q.workspace[off:off + q.T * stride].view(q.T, stride).cpu().numpy()
    assert not rows[:, q.K // 32:].any()


def check_dequantised(q, dtype):
    y = w4.dequantize_mx(q, dtype=dtype)
    want = torch.from_numpy(oracle.mx_value(device_codes(q), q.scales.cpu().numpy(), q.fmt)).float().to(dtype)
    # (the values are exact in fp32: at most 4 significant bits, exponents from 2^-136)
    torch.testing.assert_close(y.cpu(), want, rtol=0, atol=0, equal_nan=True)
    assert torch.equal(torch.signbit(y.cpu())[~want.isnan()], torch.signbit(want)[~want.isnan()])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("fmt", [4, 8])
def test_every_16_bit_value(dtype, fmt):
    """Each bit pattern as the largest of its block, next to smaller ones, and as one of many."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    alone = torch.zeros((4096, 512), dtype=torch.int16)
    alone.view(-1, 32)[:, 7] = bits  # one value to a block
    mixed = bits[torch.randperm(65536, generator=torch.Generator().manual_seed(1))].view(128, 512)
    for raw in (alone, mixed, bits.view(128, 512)):
        x = raw.view(DTYPES[dtype]).to(DEV)
        q = w4.quantize_mx(x, fmt=fmt)
        check_quantised(q, x)
        for out in DTYPES.values():
            check_dequantised(q, out)


@pytest.mark.parametrize("T,K", [(1, 32), (1, 512), (3, 160), (17, 5152), (300, 96), (2, 17408), (1030, 544)])
@pytest.mark.parametrize("dtype,fmt", [("fp16", 4), ("bf16", 8), ("fp16", 8), ("bf16", 4)])
def test_shapes(T, K, dtype, fmt):
    g = torch.Generator().manual_seed(T + K)
    x = torch.randn(T, K, generator=g)
    x *= torch.exp2(torch.randint(-20, 12, (T, K // 32), generator=g).float()).repeat_interleave(32, 1)
    x[0, :32] = 0
    x = x.to(DTYPES[dtype]).to(DEV)
    q = w4.quantize_mx(x, fmt=fmt)
    check_quantised(q, x)
    check_dequantised(q, DTYPES[dtype])


def test_strided_rows_and_given_buffers():
    wide = torch.randn(9, 1024, device=DEV).half()
    x = wide[:, 256:256 + 288]
    need = w4.mx_workspace_bytes(9, 288, 4)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    q = w4.quantize_mx(x, fmt=4, workspace=ws)
    check_quantised(q, x)
    assert (ws[need:] == 0xA5).all()  # nothing behind the last row
    out = torch.full((10, 288), 7.0, dtype=torch.float16, device=DEV)
    w4.dequantize_mx(q, out=out[:9])
    assert torch.equal(out[:9], w4.dequantize_mx(q)) and (out[9] == 7).all()
    with pytest.raises(w4.W4Error):
        w4.quantize_mx(wide[:, 4:4 + 288])  # not 16-byte aligned
    with pytest.raises(ValueError):
        w4.quantize_mx(wide[:, ::2])
    with pytest.raises(ValueError):
        w4.quantize_mx(wide[:, :40])
    with pytest.raises(ValueError):
        w4.quantize_mx(x, workspace=ws[:need - 1])


def test_empty():
    q = w4.quantize_mx(torch.empty((0, 64), dtype=torch.float16, device=DEV))
    assert q.codes.shape == (0, 32) and q.scales.shape == (0, 2) and w4.dequantize_mx(q).shape == (0, 64)


def test_scale_bytes_of_any_origin():
    """Reading back codes and scales that no quantisation here wrote: every code with every byte."""
    for fmt in (4, 8):
        n = 16 if fmt == 4 else 256
        codes = (np.arange(256 * 256).reshape(256, 256) % n).astype(np.uint8)
        bytes_ = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, 1)
        raw = np.zeros((256, 16), np.uint8)
        raw[:, :8] = bytes_
        ws = np.concatenate([(oracle.pack_fp4(codes) if fmt == 4 else codes).reshape(-1), raw.reshape(-1)])
        q = w4.MXTensor(torch.from_numpy(ws).to(DEV), 256, 256, fmt)
        for dtype in DTYPES.values():
            check_dequantised(q, dtype)


@pytest.mark.parametrize("T,K", [(1, 64), (5, 704), (33, 6144)])
def test_a8_read_back(T, K):
    rng = np.random.default_rng(K)
    x = (rng.standard_normal((T, K)) * 3).astype(np.float16)
    x[0, :64] = 0
    ws = w4.quantize_a8(torch.from_numpy(x).to(DEV))
    q, s = oracle.quantize_a8(x)
    want = torch.from_numpy(q.astype(np.float32) * np.repeat(s, 64, 1))  # the kernel's own fp32 product
    for dtype in DTYPES.values():
        y = w4.dequantize_a8(ws, T, K, dtype=dtype)
        assert torch.equal(y.cpu(), want.to(dtype))
