// Host-side repacker of MXFP4 weights: canonical codes and scales -> the layout the MX kernels
// read.  A row's 32 columns of one scale block are 16 consecutive bytes in both layouts (the bytes
// one lane of a matrix-core step holds), so packing moves whole 16-byte blocks: a permutation
// plus zero padding of the last 128 columns, bit-exact.
#include <cstring>

#include "../../include/w4gemm.h"
#include "layout.h"

namespace {

using namespace w4layout;

bool shape_ok(int N, int K) { return N > 0 && K > 0 && N % kRowTile == 0 && K % 32 == 0; }

void pack_tile(const uint8_t* codes, const uint8_t* scales, int K, int src, size_t dst, uint8_t* w_out,
               uint8_t* s_out) {
  const int KB = num_kblocks(K), blocks = K / 32;
  for (int kb = 0; kb < KB; ++kb) {
    uint8_t* w = w_out + (dst * KB + kb) * 1024;
    uint8_t* s = s_out + (dst * KB + kb) * 64;
    for (int lane = 0; lane < 64; ++lane) {
      const size_t n = (size_t)src * kRowTile + lane % 16;
      const int b = kb * 4 + lane / 16;
      if (b < blocks) {
        std::memcpy(w + lane * 16, codes + n * (K / 2) + (size_t)b * 16, 16);
        s[lane % 16 * 4 + lane / 16] = scales[n * blocks + b];
      } else {
        std::memset(w + lane * 16, 0, 16);
        s[lane % 16 * 4 + lane / 16] = 0;
      }
    }
  }
}

}  // namespace

extern "C" size_t w4_mx_packed_bytes(int N, int K) {
  return shape_ok(N, K) ? (size_t)(N / kRowTile) * num_kblocks(K) * 1024 : 0;
}

extern "C" size_t w4_mx_packed_scale_bytes(int N, int K) {
  return shape_ok(N, K) ? (size_t)(N / kRowTile) * num_kblocks(K) * 64 : 0;
}

extern "C" int w4_mx_repack(const uint8_t* codes, const uint8_t* scales, int N, int K, void* w_out,
                            uint8_t* scales_out) {
  if (!shape_ok(N, K) || !codes || !scales || !w_out || !scales_out) return W4_ERR_INVALID_ARG;
  for (int rt = 0; rt < N / kRowTile; ++rt)
    pack_tile(codes, scales, K, rt, rt, static_cast<uint8_t*>(w_out), scales_out);
  return W4_OK;
}

extern "C" int w4_mx_repack_pair(const uint8_t* gate_codes, const uint8_t* gate_scales, const uint8_t* up_codes,
                                 const uint8_t* up_scales, int N, int K, void* w_pair_out,
                                 uint8_t* scales_pair_out) {
  if (!shape_ok(N, K) || !gate_codes || !gate_scales || !up_codes || !up_scales || !w_pair_out || !scales_pair_out)
    return W4_ERR_INVALID_ARG;
  for (int rt = 0; rt < N / kRowTile; ++rt) {
    pack_tile(gate_codes, gate_scales, K, rt, 2 * (size_t)rt, static_cast<uint8_t*>(w_pair_out), scales_pair_out);
    pack_tile(up_codes, up_scales, K, rt, 2 * (size_t)rt + 1, static_cast<uint8_t*>(w_pair_out), scales_pair_out);
  }
  return W4_OK;
}
