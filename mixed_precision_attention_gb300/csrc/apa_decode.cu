// apa_decode.cu -- attention of a few query rows per sequence over the 4-bit K/V
// cache, with an optional sliding window and sinks.
#include <cmath>

#include "../../include/apa.h"
#include "apa_internal.h"
#include "cache_page.cuh"
#include "quant_tile.cuh"
#include "tc.cuh"

namespace apa {
namespace {

constexpr int kMaxSeqs = 8192;

struct DecodeParams {
  const uint16_t* q;
  long long qs_b, qs_h, qs_r;
  const uint8_t* pages;
  int num_pages;
  const int32_t* table;
  int max_pages;
  const int32_t* lens;
  const float *k_scale, *v_scale;
  int B, Hq, Hkv, Nq, window, sinks;
  uint16_t* out;
  float* lse;
  int* err;
};

// One CTA of D threads per query row: 32 keys at a time, a warp per key in turn
// for the scores, a thread per channel for the values.
template <int D, bool F16>
__global__ void __launch_bounds__(D) decode_kernel(const DecodeParams p) {
  __shared__ float q[D], score[32];
  const int row = blockIdx.x, i = row % p.Nq, hq = row / p.Nq % p.Hq, b = row / p.Nq / p.Hq;
  const int h = hq / (p.Hq / p.Hkv), c = threadIdx.x, lane = c & 31, warp = c >> 5;
  int len = p.lens[b];
  if (len < 0 || len > (long long)p.max_pages * kTile) {
    if (c == 0 && p.err) atomicCAS(p.err, 0, APA_DEVERR_BOUNDS);
    len = len < 0 ? 0 : p.max_pages * kTile;
  }
  const uint16_t* src = p.q + b * p.qs_b + hq * p.qs_h + i * p.qs_r;
  q[c] = unpack2<F16>(src[c]).x;
  __syncthreads();
  const int pos = len - p.Nq + i;
  const int lo = p.window ? max(0, pos - p.window + 1) : 0;
  float m = -INFINITY, l = 0.f, o = 0.f;
  const float sc = p.k_scale[h] * kLog2e * rsqrtf((float)D);
  for (int j0 = 0; j0 <= pos; j0 += 32) {
    if (j0 + 32 <= lo && j0 >= p.sinks) {
      j0 = (lo / 32) * 32 - 32;
      continue;
    }
    int page = p.table[(size_t)b * p.max_pages + j0 / kTile];
    if (page < 0 || page >= p.num_pages) {
      if (c == 0 && p.err) atomicCAS(p.err, 0, APA_DEVERR_BOUNDS);
      page = 0;
    }
    const uint8_t* pg = p.pages + ((size_t)page * p.Hkv + h) * page_head_bytes(D);
    for (int x = warp; x < 32; x += D / 32) {
      const int j = j0 + x, ki = j % 16;
      const uint8_t* blk = pg + j % kTile / 16 * blk_bytes(D);
      float s = 0.f;
      for (int e = lane; e < D; e += 32) {
        const uint32_t code = blk[ki * (D / 2) + e / 2] >> (4 * (e & 1)) & 15u;
        s += q[e] * (e2m1_value(code) * ue4m3_value(blk[ks_byte(D, ki, e / 16)]));
      }
      for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
      const bool see = j <= pos && (j >= lo || j < p.sinks);
      if (lane == 0) score[x] = see ? s * sc : -INFINITY;
    }
    __syncthreads();
    float mx = m;
    for (int x = 0; x < 32; ++x) mx = fmaxf(mx, score[x]);
    const float f = mx == -INFINITY ? 1.f : exp2f(m - mx);
    o *= f;
    l *= f;
    for (int x = 0; x < 32; ++x) {
      if (score[x] == -INFINITY) continue;
      const int j = j0 + x, ki = j % 16;
      const uint8_t* blk = pg + j % kTile / 16 * blk_bytes(D);
      const float w = exp2f(score[x] - mx);
      const uint32_t code = blk[v_byte(D, ki, c / 16, c % 8)] >> (c % 16 / 8 * 4) & 15u;
      o += w * (e2m1_value(code) * ue4m3_value(blk[vs_byte(D, ki, c / 16)]));
      l += w;
    }
    m = mx;
    __syncthreads();
  }
  const size_t at = ((size_t)b * p.Hq + hq) * p.Nq + i;
  p.out[at * D + c] = (uint16_t)pack2<F16>(l > 0.f ? o * p.v_scale[h] / l : 0.f, 0.f);
  if (c == 0 && p.lse) p.lse[at] = l > 0.f ? 0.6931471805599453f * (m + log2f(l)) : -INFINITY;
}

}  // namespace
}  // namespace apa

using namespace apa;

extern "C" {

size_t apa_attention_cache_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d) {
  return 0;
}

int apa_attention_cache(const void* q, int dtype, long long q_batch_stride, long long q_head_stride,
                        long long q_row_stride, const uint8_t* pages, int num_pages, const int32_t* block_table,
                        int max_pages, const int32_t* lens, const float* k_scale, const float* v_scale, int B, int Hq,
                        int Hkv, int Nq, int d, int window, int sinks, void* out, float* lse, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
  if (!q || !pages || !block_table || !lens || !k_scale || !v_scale || !out) return APA_ERR_NULL;
  if (B < 1 || B > kMaxSeqs || Hq < 1 || Hkv < 1 || Hq % Hkv || Hkv > (1 << 16) || Nq < 1 ||
      (long long)(Hq / Hkv) * Nq > (1 << 20) || (long long)B * Hq * Nq > 0x7FFFFFFF || num_pages < 1 ||
      num_pages >= (1 << 25) || max_pages < 1 || max_pages >= (1 << 25))
    return APA_ERR_SHAPE;
  if (d != 64 && d != 128 && d != 256) return APA_ERR_HEAD_DIM;
  if (dtype != APA_DTYPE_BF16 && dtype != APA_DTYPE_F16) return APA_ERR_DTYPE;
  if (window < 0 || sinks < 0) return APA_ERR_WINDOW;
  if ((((uintptr_t)q | (uintptr_t)pages | (uintptr_t)out) & 15) || ((q_batch_stride | q_head_stride | q_row_stride) & 7))
    return APA_ERR_ALIGN;
  DecodeParams prm{(const uint16_t*)q, q_batch_stride, q_head_stride, q_row_stride, pages,  num_pages,
                   block_table,        max_pages,      lens,          k_scale,      v_scale, B,
                   Hq,                 Hkv,            Nq,            window,       sinks,  (uint16_t*)out,
                   lse,                device_error_word()};
  const bool f16 = dtype == APA_DTYPE_F16;
  auto go = [&](auto kern) { kern<<<B * Hq * Nq, d, 0, stream>>>(prm); };
  switch (d) {
    case 64: f16 ? go(decode_kernel<64, true>) : go(decode_kernel<64, false>); break;
    case 128: f16 ? go(decode_kernel<128, true>) : go(decode_kernel<128, false>); break;
    case 256: f16 ? go(decode_kernel<256, true>) : go(decode_kernel<256, false>); break;
  }
  return cudaGetLastError() == cudaSuccess ? APA_OK : APA_ERR_CUDA;
}

}  // extern "C"
