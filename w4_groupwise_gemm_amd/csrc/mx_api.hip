// C ABI of the MX formats and the RMS norm: argument validation and launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "../../include/w4gemm.h"
#include "mx.h"

namespace {

constexpr int kMaxDim = 1 << 24;
constexpr size_t kLimit = (size_t)1 << 31;  // tensors of the products stay below 2 GiB

struct Range {
  uintptr_t lo, hi;
};
Range span(const void* p, size_t n) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return {b, b + (p ? n : 0)};
}
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool dims_ok(int T, int K) { return T >= 0 && K > 0 && T <= kMaxDim && K <= kMaxDim; }
bool mx_dims_ok(int T, int K) { return dims_ok(T, K) && K % w4::kMxBlock == 0; }
bool fmt_ok(int fmt) { return fmt == W4_MXFP4 || fmt == W4_MXFP8; }
bool dtype_ok(int dtype) { return dtype == W4_FP16 || dtype == W4_BF16; }
// kernels with one thread per 32 columns: the launch's thread count is 32 bits
bool grid_ok(int T, int K) { return (uint64_t)T * (K / 32) < 0xFFFFFF00u; }

size_t a8_bytes(int T, int K) {
  return ((size_t)T * K + 15) / 16 * 16 + (size_t)w4layout::num_kblocks(K) * T * 2 * sizeof(float);
}

// Bytes from the first element of row 0 to the end of row T - 1, rows ldx elements apart.
size_t strided_bytes(int T, int K, int64_t ldx) { return ((size_t)(T - 1) * ldx + K) * 2; }

// A workspace: present, aligned, large enough, overlapping none of `others`.
int check_ws(const void* ws, size_t bytes, size_t need, std::initializer_list<Range> others) {
  if (!ws) return W4_ERR_INVALID_ARG;
  if (!aligned16(ws)) return W4_ERR_MISALIGNED;
  if (bytes < need) return W4_ERR_INVALID_ARG;
  for (const Range& r : others)
    if (overlap(span(ws, need), r)) return W4_ERR_ALIAS;
  return W4_OK;
}

int launched(hipError_t e) { return e == hipSuccess ? W4_OK : W4_ERR_LAUNCH; }

// ---- routes of the product
enum RouteKind { STREAM, RING, WIDE };
struct Route {
  RouteKind kind;
  int rt, tt;  // row tiles and token tiles per workgroup (wide: rt is the index in kMxWide)
};

// Microseconds per 128 columns of a launch whose fullest compute unit runs m workgroups: c0 + c1 * m,
// fitted to launches of 128 to 2560 workgroups at K = 5120 (every kernel within 12 % of its fit).
struct Cost {
  double c0, c1;
};
double cost(Cost c, int64_t workgroups) { return c.c0 + c.c1 * (double)((workgroups + 255) / 256); }
const Cost kWideCost[2][5] = {
    {{0.125, 0.16}, {0.12, 0.28}, {0.25, 0.37}, {0.45, 0.57}, {0, 1.62}},  // MXFP4 activations
    {{0.135, 0.184}, {0.18, 0.295}, {0.2, 0.5}, {0.3, 0.86}, {0, 1e9}},    // MXFP8
};

// The cheapest kernel for the shape.  Few activations (up to 16 tokens): the streaming kernel, which
// saves the launch for the quantisation (about 2.3 us) but quantises in every workgroup, m of them one
// after another on a compute unit.  Measured at 12288 x 5120: 8 tokens 10.9 us against the ring's 11.4, 16
// tokens 13.7 against 11.9; at the 2 x 17408 x 5120 pair: 8 tokens 22.1 against 22.6; at 5120 x 17408: 2
// tokens 12.6 against 14.5, 4 tokens 15.7 against 15.4.  Otherwise whichever of the ring (blocks of up to
// 64 tokens) and the wide tiles the fits above name.  Both take as many row tiles per workgroup as spare
// the compute units a second round: the pair at 64 tokens 27.4 us with ten (one round), 38.4 with
// four (three), 41.0 with two (five).
constexpr double kStreamWork = 65536;  // T * K * (1 + m / 4)
Route pick(int op, int T, int rows, int K, int fmt) {
  const int n = rows / 16, step = op == W4_OP_SWIGLU ? 2 : 1;
  Route best = {WIDE, 0, 0};
  double least = 1e30;
  if (T <= 16) {
    for (int rt : w4::kMxRows) {
      if (rt % step) continue;
      if (w4::mx_stream_lds(T, K, fmt, rt) > w4::kMxLds) continue;
      const double c = cost({0, 0.3 + rt}, (n + rt - 1) / rt);
      if (c < least) least = c, best = {STREAM, rt, 0};
    }
    const double m = best.kind == STREAM ? ((n + best.rt - 1) / best.rt + 255) / 256 : 0;
    if (best.kind == STREAM && (double)T * K * (1 + m / 4) <= kStreamWork) return best;
    least = 1e30;
  }
  const int tt = T <= 16 ? 1 : T <= 32 ? 2 : 4;
  for (int rt : w4::kMxRows) {
    if (rt % step) continue;
    if (w4::mx_ring_lds(K, fmt, rt, tt) > w4::kMxLds) continue;
    const Cost c = fmt == 4 ? Cost{0.12, 0.01 * tt + 0.047 * rt} : Cost{0.14, 0.0125 * tt + 0.056 * rt};
    const double v = cost(c, (int64_t)((n + rt - 1) / rt) * ((T + 16 * tt - 1) / (16 * tt)));
    if (v < least) least = v, best = {RING, rt, tt};
  }
  if (T <= 64 && best.kind == RING) return best;
  for (int i = 0; i < 5; ++i) {
    const w4::MxTile t = w4::kMxWide[i];
    const double v = cost(kWideCost[fmt == 8][i], (int64_t)((rows + t.rows - 1) / t.rows) * ((T + t.tokens - 1) / t.tokens));
    if (v < least) least = v, best = {WIDE, i, 0};
  }
  return best;
}

bool product_ok(int op, int T, int N, int K, int fmt) {
  return (op == W4_OP_LINEAR || op == W4_OP_SWIGLU || op == W4_OP_ADD) && fmt_ok(fmt) && mx_dims_ok(T, K) && N > 0 &&
         N <= kMaxDim && N % w4layout::kRowTile == 0;
}

int run_linear_mx(int op, const uint16_t* x, const void* w, const uint8_t* scales, const uint16_t* res, int T, int N,
                  int K, int fmt, int dtype, uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
  if (!fmt_ok(fmt) || !dtype_ok(dtype)) return W4_ERR_UNSUPPORTED;
  if (!mx_dims_ok(T, K) || N <= 0 || N > kMaxDim || N % w4layout::kRowTile) return W4_ERR_INVALID_ARG;
  if (T == 0) return W4_OK;
  if (!w || !scales || !out || (op == W4_OP_ADD && !res)) return W4_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(scales) || !aligned16(out) || !aligned16(res))
    return W4_ERR_MISALIGNED;
  const int rows = op == W4_OP_SWIGLU ? 2 * N : N;
  const size_t wb = w4_mx_packed_bytes(rows, K), sb = w4_mx_packed_scale_bytes(rows, K);
  const size_t xb = (size_t)T * K * 2, ob = (size_t)T * N * 2;
  if (xb >= kLimit || ob >= kLimit || wb >= kLimit) return W4_ERR_UNSUPPORTED;
  const Range ro = span(out, ob), rr = span(res, ob);
  if (overlap(ro, span(x, xb)) || overlap(ro, span(w, wb)) || overlap(ro, span(scales, sb)) ||
      (res != out && overlap(ro, rr)))
    return W4_ERR_ALIAS;
  const Route route = pick(op, T, rows, K, fmt);
  const bool fused = x && route.kind == STREAM;
  int st = fused ? W4_OK : check_ws(ws, ws_bytes, w4::mx_workspace_bytes(T, K, fmt),
                                    {span(x, xb), ro, rr, span(w, wb), span(scales, sb)});
  if (st != W4_OK) return st;
  st = w4::device_status();
  if (st != W4_OK) return st;
  const hipStream_t hs = static_cast<hipStream_t>(stream);
  uint8_t* codes = static_cast<uint8_t*>(ws);
  uint8_t* xs = codes ? codes + w4::mx_scale_offset(T, K, fmt) : nullptr;
  const bool bf16 = dtype == W4_BF16;
  if (x && !fused && w4::launch_mx_quant(x, K, T, K, bf16, fmt, codes, xs, hs) != hipSuccess) return W4_ERR_LAUNCH;
  w4::MxArgs a;
  a.xq = codes;
  a.xs = xs;
  a.x = fused ? x : nullptr;
  a.w = static_cast<const uint8_t*>(w);
  a.ws = scales;
  a.res = res;
  a.out = out;
  a.T = T;
  a.rows = rows;
  a.K = K;
  a.KB = w4layout::num_kblocks(K);
  a.ldo = N;
  a.epi = op == W4_OP_SWIGLU ? w4dev::EPI_SWIGLU : op == W4_OP_ADD ? w4dev::EPI_ADD : w4dev::EPI_STORE;
  a.bf16 = bf16;
  return launched(route.kind == STREAM ? w4::launch_mx_stream(fmt, route.rt, a, hs)
                  : route.kind == RING ? w4::launch_mx_ring(fmt, route.rt, route.tt, a, hs)
                                       : w4::launch_mx_wide(fmt, route.rt, a, hs));
}

// kind: one of w4::NORM_*.  need: bytes of the workspace (0: the 16-bit output `out` instead).
int run_rmsnorm(int kind, const uint16_t* x, int64_t ldx, const uint16_t* res, const uint16_t* weight, float eps,
                int T, int K, int k_multiple, int dtype, uint16_t* res_out, uint16_t* out, void* ws, size_t ws_bytes,
                size_t need, size_t scale_offset, void* stream) {
  if (!dtype_ok(dtype)) return W4_ERR_UNSUPPORTED;
  if (!dims_ok(T, K) || K % k_multiple || ldx < K || ldx > ((int64_t)1 << 40)) return W4_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || std::isinf(eps)) return W4_ERR_INVALID_ARG;
  if ((res == nullptr) != (res_out == nullptr)) return W4_ERR_INVALID_ARG;
  if (T == 0) return W4_OK;
  if (!x || !weight || (need == 0 && !out)) return W4_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(res) || !aligned16(weight) || !aligned16(res_out) || !aligned16(out))
    return W4_ERR_MISALIGNED;
  const size_t nb = (size_t)T * K * 2;
  const Range rx = span(x, strided_bytes(T, K, ldx)), rr = span(res, nb), rw = span(weight, (size_t)K * 2);
  const Range rh = span(res_out, nb), ro = span(out, nb);
  // an output may be one of the row inputs exactly: every element is read before it is written
  auto clash = [&](const void* p, Range r) {
    return (overlap(r, rx) && !(p == x && ldx == K)) || (overlap(r, rr) && p != res) || overlap(r, rw);
  };
  if (clash(res_out, rh) || clash(out, ro) || overlap(rh, ro)) return W4_ERR_ALIAS;
  if (need) {
    const int st = check_ws(ws, ws_bytes, need, {rx, rr, rw, rh});
    if (st != W4_OK) return st;
  }
  const int st = w4::device_status();
  if (st != W4_OK) return st;
  w4::NormArgs a;
  a.x = x;
  a.res = res;
  a.weight = weight;
  a.res_out = res_out;
  a.out = out;
  a.codes = ws;
  a.scales = need ? static_cast<char*>(ws) + scale_offset : nullptr;
  a.ldx = ldx;
  a.inv_k = 1.0 / K;
  a.eps = eps;
  a.T = T;
  a.K = K;
  return launched(w4::launch_norm(kind, dtype == W4_BF16, a, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" size_t w4_mx_workspace_bytes(int T, int K, int fmt) {
  return mx_dims_ok(T, K) && fmt_ok(fmt) ? w4::mx_workspace_bytes(T, K, fmt) : 0;
}

extern "C" size_t w4_linear_mx_workspace_bytes(int op, int T, int N, int K, int fmt) {
  if (!product_ok(op, T, N, K, fmt) || T == 0) return 0;
  return pick(op, T, op == W4_OP_SWIGLU ? 2 * N : N, K, fmt).kind == STREAM ? 0 : w4::mx_workspace_bytes(T, K, fmt);
}

extern "C" const char* w4_mx_route_name(int op, int T, int N, int K, int fmt) {
  if (!product_ok(op, T, N, K, fmt)) return nullptr;
  static const char* const kStream[] = {"mx_stream_r1", "mx_stream_r2", "mx_stream_r3", "mx_stream_r4",
                                        "mx_stream_r5", "mx_stream_r6", "mx_stream_r8", "mx_stream_r10"};
#define RING_NAMES(t)                                                                                   \
  {"mx_ring_r1_" t, "mx_ring_r2_" t, "mx_ring_r3_" t, "mx_ring_r4_" t, "mx_ring_r5_" t, "mx_ring_r6_" t, \
   "mx_ring_r8_" t, "mx_ring_r10_" t}
  static const char* const kRing[][8] = {RING_NAMES("t16"), RING_NAMES("t32"), RING_NAMES("t64")};
#undef RING_NAMES
  static const char* const kWide[] = {"mx_wide_64x64", "mx_wide_128x64", "mx_wide_128x128", "mx_wide_256x128",
                                      "mx_wide_320x256"};
  const Route r = pick(op, T < 1 ? 1 : T, op == W4_OP_SWIGLU ? 2 * N : N, K, fmt);
  const int row = (int)(std::find(w4::kMxRows, w4::kMxRows + 8, r.rt) - w4::kMxRows);
  return r.kind == STREAM ? kStream[row] : r.kind == RING ? kRing[r.tt == 4 ? 2 : r.tt - 1][row] : kWide[r.rt];
}

extern "C" int w4_quantize_mx(const uint16_t* x, int64_t ldx, int T, int K, int fmt, int dtype, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (!fmt_ok(fmt) || !dtype_ok(dtype)) return W4_ERR_UNSUPPORTED;
  if (!mx_dims_ok(T, K) || ldx < K || ldx % 8 || ldx > ((int64_t)1 << 40)) return W4_ERR_INVALID_ARG;
  if (T == 0) return W4_OK;
  if (!grid_ok(T, K)) return W4_ERR_UNSUPPORTED;
  if (!x) return W4_ERR_INVALID_ARG;
  if (!aligned16(x)) return W4_ERR_MISALIGNED;
  int st = check_ws(workspace, workspace_bytes, w4::mx_workspace_bytes(T, K, fmt), {span(x, strided_bytes(T, K, ldx))});
  if (st != W4_OK) return st;
  st = w4::device_status();
  if (st != W4_OK) return st;
  uint8_t* codes = static_cast<uint8_t*>(workspace);
  return launched(w4::launch_mx_quant(x, ldx, T, K, dtype == W4_BF16, fmt, codes,
                                      codes + w4::mx_scale_offset(T, K, fmt), static_cast<hipStream_t>(stream)));
}

extern "C" int w4_dequantize_mx(const void* workspace, size_t workspace_bytes, int T, int K, int fmt, int dtype,
                                uint16_t* out, void* stream) {
  if (!fmt_ok(fmt) || !dtype_ok(dtype)) return W4_ERR_UNSUPPORTED;
  if (!mx_dims_ok(T, K)) return W4_ERR_INVALID_ARG;
  if (T == 0) return W4_OK;
  if (!grid_ok(T, K)) return W4_ERR_UNSUPPORTED;
  if (!out) return W4_ERR_INVALID_ARG;
  if (!aligned16(out)) return W4_ERR_MISALIGNED;
  int st = check_ws(workspace, workspace_bytes, w4::mx_workspace_bytes(T, K, fmt), {span(out, (size_t)T * K * 2)});
  if (st != W4_OK) return st;
  st = w4::device_status();
  if (st != W4_OK) return st;
  const uint8_t* codes = static_cast<const uint8_t*>(workspace);
  return launched(w4::launch_mx_dequant(codes, codes + w4::mx_scale_offset(T, K, fmt), T, K, dtype == W4_BF16, fmt,
                                        out, static_cast<hipStream_t>(stream)));
}

extern "C" int w4_dequantize_a8(const void* workspace, size_t workspace_bytes, int T, int K, int dtype, uint16_t* out,
                                void* stream) {
  if (!dtype_ok(dtype)) return W4_ERR_UNSUPPORTED;
  if (!dims_ok(T, K) || K % 64) return W4_ERR_INVALID_ARG;
  if (T == 0) return W4_OK;
  if (!grid_ok(T, K)) return W4_ERR_UNSUPPORTED;
  if (!out) return W4_ERR_INVALID_ARG;
  if (!aligned16(out)) return W4_ERR_MISALIGNED;
  int st = check_ws(workspace, workspace_bytes, a8_bytes(T, K), {span(out, (size_t)T * K * 2)});
  if (st != W4_OK) return st;
  st = w4::device_status();
  if (st != W4_OK) return st;
  const char* ws = static_cast<const char*>(workspace);
  return launched(w4::launch_a8_dequant(reinterpret_cast<const int8_t*>(ws),
                                        reinterpret_cast<const float*>(ws + ((size_t)T * K + 15) / 16 * 16), T, K,
                                        dtype == W4_BF16, out, static_cast<hipStream_t>(stream)));
}

extern "C" int w4_linear_mx(const uint16_t* x, const void* w, const uint8_t* scales, int T, int N, int K, int fmt,
                            int dtype, uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  return run_linear_mx(W4_OP_LINEAR, x, w, scales, nullptr, T, N, K, fmt, dtype, out, workspace, workspace_bytes,
                       stream);
}

extern "C" int w4_linear_swiglu_mx(const uint16_t* x, const void* w_pair, const uint8_t* scales_pair, int T, int N,
                                   int K, int fmt, int dtype, uint16_t* out, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  return run_linear_mx(W4_OP_SWIGLU, x, w_pair, scales_pair, nullptr, T, N, K, fmt, dtype, out, workspace,
                       workspace_bytes, stream);
}

extern "C" int w4_linear_add_mx(const uint16_t* x, const void* w, const uint8_t* scales, const uint16_t* residual,
                                int T, int N, int K, int fmt, int dtype, uint16_t* out, void* workspace,
                                size_t workspace_bytes, void* stream) {
  return run_linear_mx(W4_OP_ADD, x, w, scales, residual, T, N, K, fmt, dtype, out, workspace, workspace_bytes,
                       stream);
}

extern "C" int w4_rmsnorm(const uint16_t* x, int64_t ldx, const uint16_t* residual, const uint16_t* weight, float eps,
                          int T, int K, int dtype, uint16_t* residual_out, uint16_t* out, void* stream) {
  return run_rmsnorm(w4::NORM_16, x, ldx, residual, weight, eps, T, K, 1, dtype, residual_out, out, nullptr, 0, 0, 0,
                     stream);
}

extern "C" int w4_rmsnorm_a8(const uint16_t* x, int64_t ldx, const uint16_t* residual, const uint16_t* weight,
                             float eps, int T, int K, int dtype, uint16_t* residual_out, void* workspace,
                             size_t workspace_bytes, void* stream) {
  return run_rmsnorm(w4::NORM_A8, x, ldx, residual, weight, eps, T, K, 64, dtype, residual_out, nullptr, workspace,
                     workspace_bytes, dims_ok(T, K) ? a8_bytes(T, K) : 1, ((size_t)T * K + 15) / 16 * 16, stream);
}

extern "C" int w4_rmsnorm_mx(const uint16_t* x, int64_t ldx, const uint16_t* residual, const uint16_t* weight,
                             float eps, int T, int K, int fmt, int dtype, uint16_t* residual_out, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (!fmt_ok(fmt)) return W4_ERR_UNSUPPORTED;
  return run_rmsnorm(fmt == W4_MXFP4 ? w4::NORM_MX4 : w4::NORM_MX8, x, ldx, residual, weight, eps, T, K,
                     w4::kMxBlock, dtype, residual_out, nullptr, workspace, workspace_bytes,
                     dims_ok(T, K) ? w4::mx_workspace_bytes(T, K, fmt) : 1, w4::mx_scale_offset(T, K, fmt), stream);
}
