// 16-bit activations (or weights) to MXFP4 / MXFP8 and back, and the A8 workspace back to 16 bits.
//
// Quantisation, block of 32 columns with largest magnitude m: E = floor(log2 m) - emax (emax = 2
// for E2M1, 8 for E4M3, E not below -127), code = the element nearest to v * 2^-E (ties to even),
// saturated at 6 / 448 -- the conversion of the OCP MX specification, v1.0, section 6.3.  Dividing
// by a power of two is exact, so the rounding to the element type is the only one.
//
// Both directions are bound by memory.  One lane owns one block: its 64 bytes arrive as four
// 16-byte loads whose lines the wave shares, the maximum needs no other lane, and a wave's codes
// leave as one contiguous 1 KB store (2 KB for E4M3).
#include "mx.h"

namespace w4 {
namespace {

using namespace w4mx;

constexpr int kThreads = 256;

// Row and block of this thread among T rows of nblk blocks (rows taken one after another); false
// past the last.  The quotient of the workgroup's first block is 64-bit and uniform.
__device__ __forceinline__ bool locate(int T, int nblk, int& t, int& b) {
  const uint64_t first = (uint64_t)blockIdx.x * kThreads;
  const uint64_t t0 = first / (uint32_t)nblk;
  const uint32_t i = (uint32_t)(first - t0 * (uint32_t)nblk) + threadIdx.x;
  const uint32_t dt = i / (uint32_t)nblk;
  b = (int)(i - dt * (uint32_t)nblk);
  if (t0 + dt >= (uint64_t)T) return false;
  t = (int)(t0 + dt);
  return true;
}

template <int FMT, bool BF>
__global__ __launch_bounds__(kThreads) void mx_quant_kernel(const uint16_t* x, int64_t ldx, int T, int nblk,
                                                            uint8_t* codes, uint8_t* scales, int sstride) {
  int t, b;
  if (!locate(T, nblk, t, b)) return;
  const u32x4* src = reinterpret_cast<const u32x4*>(x + t * ldx + (int64_t)b * 32);
  uint32_t p[16], code[FMT];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u32x4 v = src[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) p[4 * i + j] = v[j];
  }
  const uint32_t byte = quantize_block<FMT, BF>(p, code);
  u32x4* dst = reinterpret_cast<u32x4*>(codes + ((size_t)t * nblk + b) * (4 * FMT));
#pragma unroll
  for (int i = 0; i < FMT / 4; ++i) dst[i] = u32x4{code[4 * i], code[4 * i + 1], code[4 * i + 2], code[4 * i + 3]};
  uint8_t* srow = scales + (size_t)t * sstride;
  srow[b] = (uint8_t)byte;
  if (b == nblk - 1)  // the rest of the row's last 16 bytes
    for (int i = nblk; i < sstride; ++i) srow[i] = 0;
}

// v * s, kept apart from the rounding to 16 bits that follows: fused into one instruction, the
// product has +0 added and loses the sign of -0.
__device__ __forceinline__ float scaled(float v, float s) {
  float y = v * s;
  asm("" : "+v"(y));
  return y;
}

// 8 columns of codes (fmt / 4 dwords) -> 16-bit pairs.  E2M1 / E4M3 to floats with scale 1, then the product
// with 2^E (exact in fp32, subnormals included), then one rounding.
template <int FMT, bool BF>
__device__ __forceinline__ u32x4 values8(const uint32_t* c, float s) {
  u32x4 o;
  if constexpr (FMT == 4) {
    const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[0], 1.0f, 0);
    const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[0], 1.0f, 1);
    const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[0], 1.0f, 2);
    const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[0], 1.0f, 3);
    o[0] = pack16<BF>(scaled(v0[0], s), scaled(v0[1], s));
    o[1] = pack16<BF>(scaled(v1[0], s), scaled(v1[1], s));
    o[2] = pack16<BF>(scaled(v2[0], s), scaled(v2[1], s));
    o[3] = pack16<BF>(scaled(v3[0], s), scaled(v3[1], s));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[i], 1.0f, false);
      const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[i], 1.0f, true);
      o[2 * i] = pack16<BF>(scaled(v0[0], s), scaled(v0[1], s));
      o[2 * i + 1] = pack16<BF>(scaled(v1[0], s), scaled(v1[1], s));
    }
  }
  return o;
}

// Reading back: a lane per 8 columns, so that a wave's stores are one contiguous kilobyte (a lane per
// block of 32 stores 16 bytes every 64: 52.6 us for 4096 x 17408 from E2M1); kSteps rounds of a
// workgroup's lanes are loaded before the first is stored.
constexpr int kSteps = 4;

template <int FMT, bool BF>
__global__ __launch_bounds__(kThreads) void mx_dequant_kernel(const uint8_t* codes, const uint8_t* scales, int T,
                                                              int nblk, int sstride, uint16_t* out) {
  const uint64_t total = (uint64_t)T * nblk * 4, first = (uint64_t)blockIdx.x * (kThreads * kSteps);
  const uint64_t b0 = first / 4, t0 = b0 / (uint32_t)nblk;
  const uint32_t r0 = (uint32_t)(b0 - t0 * (uint32_t)nblk);
  uint32_t c[kSteps][FMT / 4], byte[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const uint32_t in = i * kThreads + threadIdx.x;
    const uint32_t b = r0 + in / 4, dt = b / (uint32_t)nblk;
    byte[i] = 0;
#pragma unroll
    for (int j = 0; j < FMT / 4; ++j) c[i][j] = 0;
    if (first + in < total) {
      const uint32_t* src = reinterpret_cast<const uint32_t*>(codes) + (first + in) * (FMT / 4);
#pragma unroll
      for (int j = 0; j < FMT / 4; ++j) c[i][j] = src[j];
      byte[i] = scales[(size_t)(t0 + dt) * sstride + (b - dt * (uint32_t)nblk)];
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const uint32_t in = i * kThreads + threadIdx.x;
    const float s = __builtin_bit_cast(float, byte[i] == 255 ? 0x7FC00000u : byte[i] == 0 ? 0x00400000u : byte[i] << 23);
    if (first + in < total) reinterpret_cast<u32x4*>(out)[first + in] = values8<FMT, BF>(c[i], s);
  }
}

// A8 workspace (int8 codes, each 8-column run stored as columns 0 4 1 5 2 6 3 7; fp32 scales
// [ceil(K / 128)][T][2]) to 16 bits, laid out likewise.
template <bool BF>
__global__ __launch_bounds__(kThreads) void a8_dequant_kernel(const int8_t* codes, const float* scales, int T,
                                                              int nblk, uint16_t* out) {
  const uint64_t total = (uint64_t)T * nblk * 4, first = (uint64_t)blockIdx.x * (kThreads * kSteps);
  const uint64_t b0 = first / 4, t0 = b0 / (uint32_t)nblk;
  const uint32_t r0 = (uint32_t)(b0 - t0 * (uint32_t)nblk);
  u32x2 c[kSteps];
  float s[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const uint32_t in = i * kThreads + threadIdx.x;
    const uint32_t b = r0 + in / 4, dt = b / (uint32_t)nblk;
    c[i] = u32x2{0, 0};
    s[i] = 0.f;
    if (first + in < total) {
      const uint32_t g = (b - dt * (uint32_t)nblk) >> 1;
      c[i] = reinterpret_cast<const u32x2*>(codes)[first + in];
      s[i] = scales[((size_t)(g >> 1) * T + t0 + dt) * 2 + (g & 1)];
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const uint32_t in = i * kThreads + threadIdx.x;
    auto v = [&](int col) {
      const int pos = 2 * (col & 3) + (col >> 2);
      return (float)(int8_t)(c[i][pos >> 2] >> (8 * (pos & 3))) * s[i];
    };
    if (first + in < total)
      reinterpret_cast<u32x4*>(out)[first + in] =
          u32x4{pack16<BF>(v(0), v(1)), pack16<BF>(v(2), v(3)), pack16<BF>(v(4), v(5)), pack16<BF>(v(6), v(7))};
  }
}

dim3 grid_for(uint64_t items, int per_group) { return dim3((uint32_t)((items + per_group - 1) / per_group)); }

}  // namespace

hipError_t launch_mx_quant(const uint16_t* x, int64_t ldx, int T, int K, bool bf16, int fmt, uint8_t* codes,
                           uint8_t* scales, hipStream_t stream) {
  const int nblk = K / kMxBlock, ss = (int)mx_scale_stride(K);
  auto k = fmt == 4 ? (bf16 ? &mx_quant_kernel<4, true> : &mx_quant_kernel<4, false>)
                    : (bf16 ? &mx_quant_kernel<8, true> : &mx_quant_kernel<8, false>);
  return launch_kernel(k, grid_for((uint64_t)T * nblk, kThreads), dim3(kThreads), 0, stream, x, ldx, T, nblk, codes, scales, ss);
}

hipError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int T, int K, bool bf16, int fmt,
                             uint16_t* out, hipStream_t stream) {
  const int nblk = K / kMxBlock, ss = (int)mx_scale_stride(K);
  auto k = fmt == 4 ? (bf16 ? &mx_dequant_kernel<4, true> : &mx_dequant_kernel<4, false>)
                    : (bf16 ? &mx_dequant_kernel<8, true> : &mx_dequant_kernel<8, false>);
  return launch_kernel(k, grid_for((uint64_t)T * nblk * 4, kThreads * kSteps), dim3(kThreads), 0, stream, codes, scales, T, nblk, ss, out);
}

hipError_t launch_a8_dequant(const int8_t* codes, const float* scales, int T, int K, bool bf16, uint16_t* out,
                             hipStream_t stream) {
  const int nblk = K / 32;
  auto k = bf16 ? &a8_dequant_kernel<true> : &a8_dequant_kernel<false>;
  return launch_kernel(k, grid_for((uint64_t)T * nblk * 4, kThreads * kSteps), dim3(kThreads), 0, stream, codes, scales, T, nblk, out);
}

}  // namespace w4
