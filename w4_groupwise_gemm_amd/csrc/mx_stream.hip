// MX product at decode and verification widths (up to 64 tokens): the weights streamed once from
// memory into registers, K split over the waves of a workgroup.
#include "mx.h"
#include "tile32.h"

namespace w4 {
namespace {

using namespace w4mx;
using t32::rsrc;

constexpr int kOut = (int)0x80000000u;  // past every resource's end: reads as zero

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, int voff, int soff) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
}

// The 16 packed pairs of block b (32 columns) of token t.
__device__ __forceinline__ void load_block(__amdgpu_buffer_rsrc_t r, int off, uint32_t (&p)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u32x4 v = load16(r, off + 16 * i, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) p[4 * i + j] = v[j];
  }
}

// The waves' sums in wave order, then the epilogue: wave w finishes tiles (or gate / up pairs) w,
// w + NW, ..
template <int RT, int TT, int NW>
__device__ __forceinline__ void finish(const MxArgs& a, f32x4 (*red)[RT][TT][64], f32x4 (&acc)[RT][TT], int rt0,
                                       int tok0, int wave, int lane) {
  const int g = lane >> 4, r = lane & 15;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) red[wave][i][j][lane] = acc[i][j];
  __syncthreads();
  auto total = [&](int i, int j) {
    f32x4 y = red[0][i][j][lane];
#pragma unroll
    for (int v = 1; v < NW; ++v) y += red[v][i][j][lane];
    return y;
  };
  const bool pair = a.epi == EPI_SWIGLU;
  const int per = pair ? 2 : 1;
  for (int e = wave; e < RT / per * TT; e += NW) {
    const int i = e / TT * per, j = e % TT;
    const int t = tok0 + 16 * j + r;
    if (t >= a.T || rt0 + i >= a.rows / 16) continue;
    const f32x4 y = total(i, j), up = pair ? total(i + 1, j) : y;
    store_quad_mx(a, t, (pair ? 8 : 16) * (rt0 + i) + 4 * g, y, up);
  }
}

// Weights of RT row tiles and one k-block.
template <int RT>
struct WLoad {
  u32x4 c[RT];
  uint32_t s[RT];
};
template <int RT>
struct WSource {
  __amdgpu_buffer_rsrc_t w, s;
  int KB, woff, soff;
  __device__ __forceinline__ WSource(const MxArgs& a, int rt0, int lane) : KB(a.KB) {
    const int ntiles = a.rows / 16;
    w = rsrc(a.w, (uint32_t)((size_t)ntiles * a.KB * 1024));
    s = rsrc(a.ws, (uint32_t)((size_t)ntiles * a.KB * 64));
    woff = rt0 * a.KB * 1024 + lane * 16;
    soff = rt0 * a.KB * 64 + (lane & 15) * 4 + (lane >> 4);
  }
  // (row tiles past the last, and k-blocks at or past KB, are zeros)
  __device__ __forceinline__ void load(int kb, WLoad<RT>& o) const {
    const bool on = kb < KB;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      o.c[i] = load16(w, on ? woff + i * KB * 1024 : kOut, kb * 1024);
      o.s[i] = __builtin_amdgcn_raw_buffer_load_b8(s, on ? soff + i * KB * 64 : kOut, kb * 64, 0);
    }
  }
};

// Bytes of LDS per token and k-block: codes, and one scale byte per block.
constexpr int x_lds(int fmt) { return 16 * fmt + 4; }

// Up to TP <= 16 tokens, held in LDS for all of K.  RT row tiles per workgroup of NW waves; wave w
// takes k-blocks w, w + NW, .., DW of them in flight.  FUSED: the activations come in 16 bits and are
// quantised on their way into LDS.
template <int FMT, int RT, bool FUSED, int NW, int DW, bool BF>
__global__ __launch_bounds__(64 * NW) void mx_stream_kernel(MxArgs a, int tp_log) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ f32x4 red[NW][RT][1][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int rt0 = blockIdx.x * RT, nblk = a.K / 32, tp = 1 << tp_log;
  uint8_t* xsc = reinterpret_cast<uint8_t*>(smem) + (size_t)a.KB * tp * 16 * FMT;  // scales [KB][4][tp]

  // activations: [KB][FMT chunks of 16 bytes][tp]; tokens past T repeat none (their outputs are not
  // stored), blocks past K are zeros
  const int xstride = FUSED ? a.K * 2 : (int)mx_code_stride(a.K, FMT), sstride = (int)mx_scale_stride(a.K);
  const auto rx = rsrc(FUSED ? (const void*)a.x : a.xq, (uint32_t)((size_t)a.T * xstride));
  const auto rxs = rsrc(a.xs, (uint32_t)((size_t)a.T * sstride));
  const WSource<RT> src(a, rt0, lane);
  WLoad<RT> w[DW];
  const int items = a.KB * 4 << tp_log;  // blocks, tokens fastest
  auto put = [&](int it, const uint32_t (&c)[FMT], uint32_t byte) {
    const int t = it & (tp - 1), b = it >> tp_log;
    u32x4* dst = reinterpret_cast<u32x4*>(smem) + (((b >> 2) * FMT) << tp_log);
#pragma unroll
    for (int i = 0; i < FMT / 4; ++i)
      dst[(((b & 3) * (FMT / 4) + i) << tp_log) + t] = u32x4{c[4 * i], c[4 * i + 1], c[4 * i + 2], c[4 * i + 3]};
    xsc[it] = (uint8_t)byte;
  };
  // the first block's loads ahead of the weights', the rest after them
  uint32_t p[16], c[FMT], byte;
  auto fetch = [&](int it) {
    const int t = it & (tp - 1), b = it >> tp_log;
    const bool on = it < items && t < a.T && b < nblk;
    if constexpr (FUSED) {
      load_block(rx, on ? t * xstride + b * 64 : kOut, p);
    } else {
#pragma unroll
      for (int i = 0; i < FMT / 4; ++i) {
        const u32x4 v = load16(rx, on ? t * xstride + b * 4 * FMT + 16 * i : kOut, 0);
        c[4 * i] = v[0]; c[4 * i + 1] = v[1]; c[4 * i + 2] = v[2]; c[4 * i + 3] = v[3];
      }
      byte = __builtin_amdgcn_raw_buffer_load_b8(rxs, on ? t * sstride + b : kOut, 0, 0);
    }
  };
  fetch(threadIdx.x);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int d = 0; d < DW; ++d) src.load(wave + NW * d, w[d]);
  __builtin_amdgcn_sched_barrier(0);
  for (int it = threadIdx.x; it < items; it += 64 * NW) {
    if (it != (int)threadIdx.x) fetch(it);
    if constexpr (FUSED) byte = quantize_block<FMT, BF>(p, c);
    put(it, c, byte);
  }
  arrive_wait();

  f32x4 acc[RT][1] = {};
  const int rr = r & (tp - 1);
  for (int kb = wave; kb < a.KB; kb += NW * DW) {
#pragma unroll
    for (int d = 0; d < DW; ++d) {
      const int k = kb + NW * d, kx = min(k, a.KB - 1);  // (past the end the weights are zeros)
      const u32x4* xp = reinterpret_cast<const u32x4*>(smem) + ((kx * FMT) << tp_log) + rr;
      uint32_t x[FMT];
#pragma unroll
      for (int e = 0; e < FMT / 4; ++e) {
        const u32x4 v = xp[(4 * e + g) << tp_log];  // E4M3: columns 64 e + 16 g .. + 15
        x[4 * e] = v[0]; x[4 * e + 1] = v[1]; x[4 * e + 2] = v[2]; x[4 * e + 3] = v[3];
      }
      const uint32_t sx = xsc[((kx * 4 + g) << tp_log) + rr];
#pragma unroll
      for (int i = 0; i < RT; ++i) acc[i][0] = mfma_mx16<FMT>(w[d].c[i], w[d].s[i], x, sx, acc[i][0]);
      src.load(k + NW * DW, w[d]);
    }
  }
  finish<RT, 1, NW>(a, red, acc, rt0, 0, wave, lane);
}

// Any number of tokens, TT tiles of 16 per workgroup, quantised activations straight from memory (L2) to
// registers beside the weights, D k-blocks of both in flight: one in-order load counter serves
// both, so neither may run ahead of the other.
template <int FMT, int RT, int TT, int NW, int D>
__global__ __launch_bounds__(64 * NW) void mx_direct_kernel(MxArgs a, int groups) {
  __shared__ f32x4 red[NW][RT][TT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int grp = blockIdx.x % groups, tok0 = blockIdx.x / groups * 16 * TT;
  const int rt0 = grp * RT;
  const WSource<RT> src(a, rt0, lane);
  const int xstride = (int)mx_code_stride(a.K, FMT), sstride = (int)mx_scale_stride(a.K);
  const auto rx = rsrc(a.xq, (uint32_t)((size_t)a.T * xstride));
  const auto rxs = rsrc(a.xs, (uint32_t)((size_t)a.T * sstride));
  struct X {
    uint32_t c[TT][FMT], s[TT];
  };
  auto load_x = [&](int kb, X& o) {
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const int t = tok0 + 16 * j + r;
#pragma unroll
      for (int e = 0; e < FMT / 4; ++e) {
        // E2M1: block g; E4M3: columns 64 e + 16 g .. + 15
        const bool on = FMT == 4 ? kb * 128 + g * 32 < a.K : kb * 128 + 64 * e + 16 * g < a.K;
        const u32x4 v = load16(rx, on ? t * xstride + 64 * e + 16 * g : kOut, kb * 16 * FMT);
        o.c[j][4 * e] = v[0]; o.c[j][4 * e + 1] = v[1]; o.c[j][4 * e + 2] = v[2]; o.c[j][4 * e + 3] = v[3];
      }
      o.s[j] = __builtin_amdgcn_raw_buffer_load_b8(rxs, kb < a.KB ? t * sstride + g : kOut, kb * 4, 0);
    }
  };
  f32x4 acc[RT][TT] = {};
  WLoad<RT> w[D];
  X x[D];
#pragma unroll
  for (int d = 0; d < D; ++d) {
    load_x(wave + NW * d, x[d]);
    src.load(wave + NW * d, w[d]);
  }
  for (int kb = wave; kb < a.KB; kb += NW * D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int k = kb + NW * (d + D);
#pragma unroll
      for (int j = 0; j < TT; ++j)
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i][j] = mfma_mx16<FMT>(w[d].c[i], w[d].s[i], x[d].c[j], x[d].s[j], acc[i][j]);
      load_x(k, x[d]);
      src.load(k, w[d]);
    }
  }
  finish<RT, TT, NW>(a, red, acc, rt0, tok0, wave, lane);
}

template <int FMT, int RT, int NW, int DW>
hipError_t run_stream(const MxArgs& a, hipStream_t stream) {
  const dim3 grid((a.rows / 16 + RT - 1) / RT);
  int tp_log = 0;
  while ((1 << tp_log) < a.T) ++tp_log;
  const size_t lds = (size_t)(a.KB << tp_log) * x_lds(FMT);
  auto k = !a.x ? &mx_stream_kernel<FMT, RT, false, NW, DW, false>
                : a.bf16 ? &mx_stream_kernel<FMT, RT, true, NW, DW, true> : &mx_stream_kernel<FMT, RT, true, NW, DW, false>;
  return launch_kernel(k, grid, dim3(64 * NW), lds, stream, a, tp_log);
}

template <int FMT, int RT, int TT, int NW, int D>
hipError_t run_direct(const MxArgs& a, hipStream_t stream) {
  const int groups = (a.rows / 16 + RT - 1) / RT;
  return launch_kernel(&mx_direct_kernel<FMT, RT, TT, NW, D>, dim3(groups * ((a.T + 16 * TT - 1) / (16 * TT))),
                       dim3(64 * NW), 0, stream, a, groups);
}

template <int FMT>
hipError_t pick(const MxArgs& a, hipStream_t stream) {
  if (mx_stream_fits(a.T, a.K, FMT)) return run_stream<FMT, 2, 8, 4>(a, stream);
  if (a.T <= 16) return run_direct<FMT, 2, 1, 8, 4>(a, stream);
  if (a.T <= 32) return run_direct<FMT, 2, 2, 8, 3>(a, stream);
  return run_direct<FMT, 2, 4, 8, 2>(a, stream);
}

}  // namespace

bool mx_stream_fits(int T, int K, int fmt) {
  int tp = 1;
  while (tp < T) tp *= 2;
  return T <= 16 && (size_t)w4layout::num_kblocks(K) * tp * x_lds(fmt) <= 96 * 1024;
}

hipError_t launch_mx_stream(int fmt, const MxArgs& a, hipStream_t stream) {
  return fmt == 4 ? pick<4>(a, stream) : pick<8>(a, stream);
}

}  // namespace w4
