// MX product over quantised activations, any number of tokens: one workgroup per group of row
// tiles and block of 64 tokens, its waves splitting K.
//
//   Y[t][n] = sum over blocks b of 2^(ex[t][b] + ew[n][b]) * sum over k in b of cx[t][k] cw[n][k]
//
// One scaled matrix-core step covers 16 rows x 16 tokens x 128 columns, four scale blocks, and
// applies both scales itself.
#include "mx.h"

namespace w4 {
namespace {

using namespace w4mx;

constexpr int kWaves = 4;
constexpr int kTT = 4;  // token tiles of 16 per workgroup

// Activation operand of token t, k-block kb: codes and scale byte of this lane.  Columns at or past
// K are zeros.
template <int FMT>
__device__ __forceinline__ uint32_t load_x(const MxArgs& a, int t, int kb, int g, uint32_t (&x)[FMT]) {
#pragma unroll
  for (int i = 0; i < FMT; ++i) x[i] = 0;
  uint32_t s = 0;
  if (t < a.T) {
    const uint8_t* row = a.xq + (size_t)t * mx_code_stride(a.K, FMT);
    if constexpr (FMT == 4) {
      if (kb * 128 + g * 32 < a.K) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(row + kb * 64 + g * 16);
        x[0] = v[0]; x[1] = v[1]; x[2] = v[2]; x[3] = v[3];
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = kb * 128 + h * 64 + g * 16;
        if (c < a.K) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(row + c);
          x[4 * h] = v[0]; x[4 * h + 1] = v[1]; x[4 * h + 2] = v[2]; x[4 * h + 3] = v[3];
        }
      }
    }
    s = a.xs[(size_t)t * mx_scale_stride(a.K) + kb * 4 + g];  // (rows are padded past K with zeros)
  }
  return s;
}

// RT: row tiles of 16 (a gate tile and its up tile for the SwiGLU pair).
template <int EPI, bool BF, int FMT, int RT>
__global__ __launch_bounds__(64 * kWaves) void mx_stream_kernel(MxArgs a) {
  __shared__ f32x4 red[kWaves][RT][kTT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, r = lane & 15;
  const int groups = a.rows / 16 / RT;  // of row tiles
  const int rt0 = blockIdx.x % groups * RT, tok0 = blockIdx.x / groups * 16 * kTT;
  const int ntt = min(kTT, (a.T - tok0 + 15) / 16);
  f32x4 acc[RT][kTT] = {};
  for (int kb = wave; kb < a.KB; kb += kWaves) {
    u32x4 w[RT];
    uint32_t sw[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const size_t blk = (size_t)(rt0 + i) * a.KB + kb;
      w[i] = *reinterpret_cast<const u32x4*>(a.w + blk * 1024 + lane * 16);
      sw[i] = a.ws[blk * 64 + lane];
    }
#pragma unroll
    for (int j = 0; j < kTT; ++j) {
      if (j < ntt) {
        uint32_t x[FMT];
        const uint32_t sx = load_x<FMT>(a, tok0 + 16 * j + r, kb, g, x);
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i][j] = mfma_mx16<FMT>(w[i], sw[i], x, sx, acc[i][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < kTT; ++j) red[wave][i][j][lane] = acc[i][j];
  __syncthreads();
  // the waves' sums in wave order; wave w finishes token tile w
  const int j = wave, t = tok0 + 16 * j + r;
  if (t >= a.T) return;
  f32x4 y[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    y[i] = red[0][i][j][lane];
#pragma unroll
    for (int v = 1; v < kWaves; ++v) y[i] += red[v][i][j][lane];
  }
  if constexpr (EPI == EPI_SWIGLU) {
    store_quad_mx<EPI, BF>(a, t, 8 * rt0 + 4 * g, y[0], y[1]);
  } else {
#pragma unroll
    for (int i = 0; i < RT; ++i) store_quad_mx<EPI, BF>(a, t, 16 * (rt0 + i) + 4 * g, y[i], y[i]);
  }
}

template <int EPI, bool BF, int FMT>
hipError_t run(const MxArgs& a, hipStream_t stream) {
  constexpr int RT = EPI == EPI_SWIGLU ? 2 : 1;
  return launch_kernel(&mx_stream_kernel<EPI, BF, FMT, RT>, 
                       dim3(a.rows / 16 / RT * ((a.T + 16 * kTT - 1) / (16 * kTT))), dim3(64 * kWaves), 0, stream, a);
}

template <int EPI>
hipError_t run_epi(bool bf16, int fmt, const MxArgs& a, hipStream_t stream) {
  if (fmt == 4) return bf16 ? run<EPI, true, 4>(a, stream) : run<EPI, false, 4>(a, stream);
  return bf16 ? run<EPI, true, 8>(a, stream) : run<EPI, false, 8>(a, stream);
}

}  // namespace

hipError_t launch_mx_stream(int epi, bool bf16, int fmt, const MxArgs& a, hipStream_t stream) {
  if (epi == EPI_SWIGLU) return run_epi<EPI_SWIGLU>(bf16, fmt, a, stream);
  if (epi == EPI_ADD) return run_epi<EPI_ADD>(bf16, fmt, a, stream);
  return run_epi<EPI_STORE>(bf16, fmt, a, stream);
}

}  // namespace w4
