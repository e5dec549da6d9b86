// Root-mean-square norm of each token row, with the residual's addition in front of it and the
// output in 16 bits, in the A8 route's int8 form or in MX form.
//
//   h = x + r,   y = h * (1 / sqrt(mean(h^2) + eps)) * weight
//
// h is formed in fp32 and y from the unrounded h, so each output is rounded once: residual_out
// to 16 bits, y to 16 bits or straight to its 8- or 4-bit codes.
//
// Bound by memory: every tensor is touched once.  One workgroup owns a row and keeps it in
// registers, 8 columns per lane and vector, between the sum and the scaling; the sum is a wave
// reduction and one exchange through LDS.  An A8 group (64 columns) is 8 neighbouring lanes, an MX
// block (32 columns) 4, so their maxima are lane exchanges too.
#include "mx.h"

namespace w4 {
namespace {

using namespace w4mx;

constexpr int kMaxWaves = 16;

// The 8 columns at c of one row, or those of them below K (the others 0).  Rows of odd length or
// stride start at any 2-byte address: memory access need not be aligned.
template <bool BF>
__device__ __forceinline__ void load8(const uint16_t* row, int c, int K, float (&f)[8]) {
  if (c + 8 <= K) {
    u32x4 v;
    __builtin_memcpy(&v, row + c, 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = lo16<BF>(v[i]);
      f[2 * i + 1] = hi16<BF>(v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < K ? lo16<BF>(row[c + i]) : 0.f;
  }
}

template <bool BF>
__device__ __forceinline__ void store8(uint16_t* row, int c, int K, const float (&f)[8]) {
  if (c + 8 <= K) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack16<BF>(f[2 * i], f[2 * i + 1]);
    __builtin_memcpy(row + c, &v, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < K) row[c + i] = round16<BF>(f[i]);
  }
}

template <bool BF>
__device__ __forceinline__ void load_h(const NormArgs& a, int t, int c, float (&h)[8]) {
  load8<BF>(a.x + t * a.ldx, c, a.K, h);
  if (a.res) {
    float r[8];
    load8<BF>(a.res + (size_t)t * a.K, c, a.K, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] += r[i];
  }
}

// 1 / sqrt(mean + eps) from every thread's share of the sum of squares.  Two slots of partial sums
// alternate between rows, so one barrier a row is enough.
__device__ __forceinline__ float row_rstd(float ss, float (*part)[kMaxWaves], int slot, const NormArgs& a) {
#pragma unroll
  for (int o = 32; o; o >>= 1) ss += __shfl_xor(ss, o);
  const int waves = blockDim.x >> 6;
  if (waves > 1) {
    if ((threadIdx.x & 63) == 0) part[slot][threadIdx.x >> 6] = ss;
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < waves; ++i) ss += part[slot][i];
  }
  return 1.0f / sqrtf(ss / (float)a.K + a.eps);
}

// y of the 8 columns at c, written in the output's form.  Every lane of the wave calls this (the
// group maxima cross lanes); c >= K writes nothing.
template <int KIND, bool BF>
__device__ __forceinline__ void put8(const NormArgs& a, int t, int c, const float (&h)[8], float rstd) {
  float y[8];
  if (c < a.K) {
    load8<BF>(a.weight, c, a.K, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] *= h[i] * rstd;
    if (a.res) store8<BF>(a.res_out + (size_t)t * a.K, c, a.K, h);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = 0.f;
  }
  if constexpr (KIND == NORM_16) {
    if (c < a.K) store8<BF>(a.out + (size_t)t * a.K, c, a.K, y);
    return;
  }
  // largest magnitude as its bits: infinity and NaN above every finite value
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __builtin_bit_cast(uint32_t, y[i]) & 0x7FFFFFFFu);
  m = max(m, (uint32_t)__shfl_xor((int)m, 1));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2));
  if constexpr (KIND == NORM_A8) {
    m = max(m, (uint32_t)__shfl_xor((int)m, 4));
    if (c >= a.K) return;
    // s = max / 127, q = rint(y / s), as the A8 route's own quantisation.  A group with an infinity
    // or NaN has that as its scale, and codes of 1 where a 0 code would lose it.
    const float s = __builtin_bit_cast(float, m) / 127.0f;
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = s > 0.f ? rintf(y[i] / s) : 0.f;
      v = m >= 0x7F800000u ? 1.f : fminf(fmaxf(v, -127.f), 127.f);
      q[i] = (uint32_t)(int)v & 0xFFu;
    }
    int8_t* dst = static_cast<int8_t*>(a.codes) + (size_t)t * a.K + c;
    *reinterpret_cast<u32x2*>(dst) = u32x2{q[0] | (q[4] << 8) | (q[1] << 16) | (q[5] << 24),
                                           q[2] | (q[6] << 8) | (q[3] << 16) | (q[7] << 24)};
    if ((c & 63) == 0) {
      const int g = c >> 6;
      float* sx = static_cast<float*>(a.scales);
      sx[((size_t)(g >> 1) * a.T + t) * 2 + (g & 1)] = s;
      if ((g & 1) == 0 && c + 64 == a.K) sx[((size_t)(g >> 1) * a.T + t) * 2 + 1] = 0.f;
    }
  } else {
    if (c >= a.K) return;
    constexpr int FMT = KIND == NORM_MX4 ? 4 : 8;
    const uint32_t byte = scale_byte<FMT>(m);
    const float s = scale_float(byte);
    uint8_t* dst = static_cast<uint8_t*>(a.codes) + (size_t)t * mx_code_stride(a.K, FMT) + (size_t)c * FMT / 8;
    if constexpr (FMT == 4) {
      *reinterpret_cast<uint32_t*>(dst) = byte == 255 ? 0u : fp4x8(y, s);
    } else {
      const float top = fp8_top(byte);
      const uint32_t lo = byte == 255 ? 0u : fp8x4(y[0], y[1], y[2], y[3], s, top);
      const uint32_t hi = byte == 255 ? 0u : fp8x4(y[4], y[5], y[6], y[7], s, top);
      *reinterpret_cast<u32x2*>(dst) = u32x2{lo, hi};
    }
    if ((c & 31) == 0) {
      const int ss = (int)mx_scale_stride(a.K);
      uint8_t* srow = static_cast<uint8_t*>(a.scales) + (size_t)t * ss;
      srow[c >> 5] = (uint8_t)byte;
      if (c + 32 == a.K)  // the rest of the row's last 16 bytes
        for (int i = (c >> 5) + 1; i < ss; ++i) srow[i] = 0;
    }
  }
}

// VPT vectors of 8 columns per lane in registers.
template <int KIND, bool BF, int VPT>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a) {
  __shared__ float part[2][kMaxWaves];
  int slot = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, slot ^= 1) {
    float h[VPT][8];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * 8;
      if (c < a.K) {
        load_h<BF>(a, t, c, h[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[v][i], h[v][i], ss);
      }
    }
    const float rstd = row_rstd(ss, part, slot, a);
#pragma unroll
    for (int v = 0; v < VPT; ++v) put8<KIND, BF>(a, t, (v * blockDim.x + threadIdx.x) * 8, h[v], rstd);
  }
}

// Rows too long for registers: h is formed again for the second pass (each lane reads its columns
// before it writes them, so the outputs may still be the inputs).
template <int KIND, bool BF>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormArgs a) {
  __shared__ float part[2][kMaxWaves];
  int slot = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, slot ^= 1) {
    float ss = 0.f;
    for (int c = threadIdx.x * 8; c < a.K; c += blockDim.x * 8) {
      float h[8];
      load_h<BF>(a, t, c, h);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(h[i], h[i], ss);
    }
    const float rstd = row_rstd(ss, part, slot, a);
    for (int c0 = 0; c0 < a.K; c0 += blockDim.x * 8) {
      const int c = c0 + threadIdx.x * 8;
      float h[8] = {};
      if (c < a.K) load_h<BF>(a, t, c, h);
      put8<KIND, BF>(a, t, c, h, rstd);
    }
  }
}

constexpr int kMaxGrid = 1 << 20;  // workgroups; further rows are taken in turn

template <int KIND, bool BF>
hipError_t run_norm(const NormArgs& a, hipStream_t stream) {
  const dim3 grid(a.T < kMaxGrid ? a.T : kMaxGrid);
  const int64_t nvec = ((int64_t)a.K + 7) / 8;
  const int vpt = nvec <= 1024 ? 1 : nvec <= 2048 ? 2 : 4;
  if (nvec > 4 * 1024) return launch_kernel(&norm_long_kernel<KIND, BF>, grid, dim3(1024), 0, stream, a);
  const int threads = (int)(((nvec + vpt - 1) / vpt + 63) / 64 * 64);
  auto k = vpt == 1 ? &norm_kernel<KIND, BF, 1> : vpt == 2 ? &norm_kernel<KIND, BF, 2> : &norm_kernel<KIND, BF, 4>;
  return launch_kernel(k, grid, dim3(threads), 0, stream, a);
}

}  // namespace

hipError_t launch_norm(int kind, bool bf16, const NormArgs& a, hipStream_t stream) {
  switch (kind) {
    case NORM_16: return bf16 ? run_norm<NORM_16, true>(a, stream) : run_norm<NORM_16, false>(a, stream);
    case NORM_A8: return bf16 ? run_norm<NORM_A8, true>(a, stream) : run_norm<NORM_A8, false>(a, stream);
    case NORM_MX4: return bf16 ? run_norm<NORM_MX4, true>(a, stream) : run_norm<NORM_MX4, false>(a, stream);
    case NORM_MX8: return bf16 ? run_norm<NORM_MX8, true>(a, stream) : run_norm<NORM_MX8, false>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace w4
