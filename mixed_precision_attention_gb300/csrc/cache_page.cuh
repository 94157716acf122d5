// cache_page.cuh -- the page layout of the 4-bit K/V cache (include/apa.h) and
// the element types of its entry points.
//
// A page of 64 keys holds, per KV head, four blocks of 16 keys, 18*d bytes each:
// K codes, V codes, K scales, V scales.  A block is what one warp of the decode
// attention takes per product step, contiguous, so one bulk copy brings it in.
// K rows are in channel order: lane (g, c) of an m16n8k16 product reads a quarter
// of a key's codes as one vector.  V is stored as the products' A fragments of
// V^T: lane (g, c) needs channels g and g + 8 of a 16-channel tile for the keys
// 4c .. 4c+3, which is one word (a byte per key, two channels in it), and four
// tiles make the lane's 16-byte vector.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "apa_internal.h"

namespace apa {

constexpr int kBlkKeys = 16;  // keys per block of a page

__host__ __device__ constexpr int page_head_bytes(int d) { return 72 * d; }
__host__ __device__ constexpr int blk_bytes(int d) { return 18 * d; }
__host__ __device__ constexpr int blk_v(int d) { return 8 * d; }
__host__ __device__ constexpr int blk_ks(int d) { return 16 * d; }
__host__ __device__ constexpr int blk_vs(int d) { return 17 * d; }
// V code byte of (key i, channels 16t + g and 16t + 8 + g), and the scale bytes of (key i, channels 16t ..)
__host__ __device__ constexpr int v_byte(int d, int i, int t, int g) {
  return blk_v(d) + 512 * (t >> 2) + 16 * (4 * g + (i >> 2)) + 4 * (t & 3) + (i & 3);
}
__host__ __device__ constexpr int ks_byte(int d, int i, int t) { return blk_ks(d) + i * (d / 16) + t; }
__host__ __device__ constexpr int vs_byte(int d, int i, int t) {
  return blk_vs(d) + 4 * ((i >> 2) * (d / 16) + t) + (i & 3);
}

// Two 16-bit elements <-> FP32.
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (F16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace apa
