// apa_tree.cu -- attention of a tree of drafted tokens over the 4-bit paged K/V cache.
//
// out = softmax(q K^T / sqrt(d)) V, row i (a drafted token, or node) over the context's keys and
// the drafted keys whose bits it has, under an optional window and sinks, by positions: a
// context key stands at its index, node n at base + depth(n).
//
// Trees have tens of nodes, and G rows for each, so the products run on tcgen05 tiles of 128 rows
// (rows.cuh) and what bounds it is turning codes into FP16 operands in shared memory: 2 x 64 x d
// values per page and KV head, once for up to 256 rows.  One warp brings pages in (a bulk copy
// each: a page's part of a head is contiguous), two turn K's codes and two V's.  E2M1 * UE4M3 has
// 6 significant bits and lies in 2^-10 .. 2688, so K and V are exact in FP16; Q's rows are
// scaled by a power of two to 2^14 .. 2^16 as in the decode kernel (apa_decode.cu).  A V code byte
// holds channels g and 8 + g of 16, one FP16 pair: the pairs are stored side by side (kPairedV),
// and the epilogue puts O's columns in order again, which costs no instruction.
//
// Trees of up to 64 nodes, G = 4, over 4 contexts to 131072 keys: 194 us (the products alone 90 at
// the measured rate, the pages' bytes 31); of up to 32 nodes, G = 3, over 32 contexts to 8192 keys 100 us.
// A page of a head takes the K and V warps 1160 and 1100 cycles in the first case, 1410 and 1900 in the second (some
// 200 instructions of each of the four warps, 5 to 9 cycles apart: fixed latencies, instruction fetch and the softmax
// warps' slots), and the SM twice the issue slots of the softmax of one block.  Eight such warps in two teams were slower
// (155 us for 145 at the time), and so were deeper rings.
#include "rows.cuh"

namespace apa {
namespace {

// Eight E2M1 codes -> four FP16 pairs.
__device__ __forceinline__ void tree_e2m1x8(uint32_t w, uint32_t* h) {
  asm("{\n.reg .b8 b0, b1, b2, b3;\n"
      "mov.b32 {b0, b1, b2, b3}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t tree_e4m3x2(uint32_t w) {  // two scale codes -> an FP16 pair
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
  return r;
}
__device__ __forceinline__ uint32_t tree_hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// kTwo: items of up to two blocks, else of one.
template <int D, bool kTwo>
struct TreePick;
template <>
struct TreePick<64, false> { using Cfg = RowCfg<64, 64, 1, 2, true, 3, 3, true>; static constexpr int kRaw = 8; };
template <>
struct TreePick<128, true> { using Cfg = RowCfg<128, 64, 2, 2, false, 2, 4, true>; static constexpr int kRaw = 4; };
template <>
struct TreePick<128, false> { using Cfg = RowCfg<128, 64, 1, 1, true, 2, 2, true>; static constexpr int kRaw = 3; };
template <>
struct TreePick<256, false> { using Cfg = RowCfg<256, 64, 1, 2, true, 2, 2, true>; static constexpr int kRaw = 4; };

template <int D, bool F16, bool kTwo>
struct TreeSrc {
  using Cfg = typename TreePick<D, kTwo>::Cfg;
  static constexpr int KT = Cfg::KT, kRaw = TreePick<D, kTwo>::kRaw;
  static_assert(KT == kTile, "a tile is a page");
  static constexpr int kPageBytes = page_head_bytes(D);
  static constexpr int kKWarps = 2, kVWarps = 2, kSrcWarps = 1 + kKWarps + kVWarps;
  static constexpr int kThreads = (Cfg::kSrcWarp + kSrcWarps) * 32;
  static constexpr int kKArrivals = kKWarps, kVArrivals = kVWarps;
  static constexpr bool kVFirst = false;
  static constexpr int kBars = 2 * kRaw;  // pages there, pages read
  static __device__ __forceinline__ uint32_t bar_count(int i) { return i < kRaw ? 1 : kKWarps + kVWarps; }
  static constexpr bool kPairedV = true, kOutF16 = F16, kScaledQ = true, kMasked = true;
  static constexpr int kItemCost = Cfg::kItemCost;
  static constexpr int kSoftUnroll = 1;  // (the teams' code wants room in the instruction caches: 2 here, 221 us for 207)
  static constexpr int kSmem = Cfg::kSrcOff + kRaw * kPageBytes + 1024;
  static_assert(Cfg::kCtasPerSm * (kSmem + (Cfg::NG == 2 ? 4096 : 2048) + 1024) <= 233472, "shared memory");

  static __device__ __forceinline__ float largest(uint4 v) {  // magnitude of eight values
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float a = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = unpack2<F16>(w[k]);
      a = fmaxf(a, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
    return a;
  }

  struct Params {
    RowParams r;
    const uint8_t* pages;
    int num_pages;
    const int32_t* table;
    int max_pages;
    const int32_t* lens;
    const int32_t* nodes;  // or null: Nq for all
    const uint32_t* mask;  // [B][Nq][words], sequences mask_stride apart
    long long mask_stride;
    int words;
    const int32_t* depths;  // [B][Nq], sequences depth_stride apart; or null (no window)
    long long depth_stride;
    const float *k_scale, *v_scale;
    int window, sinks;
  };
  // Keys len, of which the last `nodes` are the drafted ones; tiles: pages that hold sinks, then those from lo on.
  // len is at most 2^31 - 64 (tables have fewer than 2^25 entries), and so is a context key's position; a node's, base +
  // depth, may pass 2^31: what compares it does so from base.
  struct Seq {
    int blocks, tiles, len, base, nodes, n_sink, lo;
    Seq() = default;
    __device__ __forceinline__ Seq(const Params& p, int b) {
      len = max(0, min(p.lens[b], p.max_pages * kTile));
      nodes = max(0, min(p.nodes ? p.nodes[b] : p.r.Nq, min(p.r.Nq, len)));
      base = len - nodes;
      blocks = (p.r.G() * nodes + kBlockRows - 1) / kBlockRows;
      lo = p.window ? max(0, base - p.window + 1) / kTile : 0;
      n_sink = p.window ? min((p.sinks + kTile - 1) / kTile, lo) : 0;
      tiles = nodes ? n_sink + (len + kTile - 1) / kTile - lo : 0;
    }
    __device__ __forceinline__ void report(const Params& p, int b) const {
      if (blockIdx.x == 0 && p.r.err && (p.lens[b] != len || (p.nodes ? p.nodes[b] : p.r.Nq) != nodes))
        atomicCAS(p.r.err, 0, APA_DEVERR_BOUNDS);
    }
    __device__ __forceinline__ int page(int tile) const { return tile < n_sink ? tile : lo + tile - n_sink; }
  };

  struct Row {
    bool valid;
    int out_row, pos, depth;
    float c2, v_scale;
    __device__ __forceinline__ void set(const Params& p, const Seq& s, int b, int h, int P) {
      const int G = p.r.G();
      pos = P / G;
      valid = pos < s.nodes;
      out_row = pos < p.r.Nq ? (b * p.r.Hq + h * G + P % G) * p.r.Nq + pos : -1;
      c2 = p.k_scale[h] * kLog2e * rsqrtf((float)D);
      v_scale = p.v_scale[h];
      depth = valid && p.window ? max(0, min(p.depths[b * p.depth_stride + pos], p.r.Nq - 1)) : 0;
    }
    // The row's factors; returns the power of two that brings its largest magnitude to 2^14 .. 2^16.
    __device__ __forceinline__ float scale(float amax) {
      int e = (int)((__float_as_uint(amax) >> 23) & 255) - 127;
      e = max(-100, min(126, e));
      const float down = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
      // (a positive finite number, so that a masked score stays -inf and a key of zeros 0)
      const float f = down * c2;
      c2 = f < FLT_MIN ? FLT_MIN : f > FLT_MAX ? FLT_MAX : f;
      return __uint_as_float((uint32_t)(127 + 14 - e) << 23);
    }
    __device__ __forceinline__ uint32_t convert(uint32_t w, float up) const {
      const float2 f = unpack2<F16>(w);
      return pack2<true>(f.x * up, f.y * up);
    }
    // which of the keys j .. j + 31 of sequence b the row sees (out of line: few tiles need it)
    static __device__ __forceinline__ uint32_t sees(const Params& p, const Seq& s, int b, int pos, int depth, int j) {
      auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
      uint32_t ctx = below(s.base - j), drafted = 0u;
      const int at = j - s.base;  // node of key j
      if (at > -32 && at < s.nodes) {
        const uint32_t* bits = p.mask + b * p.mask_stride + (long long)pos * p.words;
        const int w = at >> 5, sh = at & 31;  // (at = -1: word -1, shifted by 31)
        const uint32_t lo = w >= 0 ? bits[w] : 0u, hi = w + 1 < p.words ? bits[w + 1] : 0u;
        drafted = __funnelshift_r(lo, hi, sh) & below(s.nodes - at) & ~ctx;
      }
      if (p.window) {
        // The window's first position is base - back; all of the context is before it if that is past base.  (Where j is past
        // base there is no context, and the difference may wrap.)
        const int back = p.window - 1 - depth;
        ctx &= ~below((int)((unsigned)(s.base - j) - (unsigned)max(back, 0))) | below(p.sinks - j);
        if (p.window < p.r.Nq)  // only then may a drafted key lie behind it
          for (uint32_t x = drafted; x; x &= x - 1) {
            const int k = __ffs(x) - 1;
            const int dk = max(0, min(p.depths[b * p.depth_stride + at + k], p.r.Nq - 1));
            if (dk < -back && dk >= p.sinks - s.base) drafted &= ~(1u << k);
          }
      }
      return ctx | drafted;
    }
    // which of a tile's keys the row sees, in words of 32
    template <int N>
    __device__ __forceinline__ void mask(const Params& p, const RowWalk<TreeSrc>& walk, int tile, uint32_t* vis) const {
      const Seq& s = walk.seq;
      const int j0 = s.page(walk.g.t0 + tile) * kTile;
#pragma unroll 1
      for (int c = 0; c < N; ++c) {
        const uint32_t v = valid ? sees(p, s, walk.g.b, pos, depth, j0 + 32 * c) : 0u;
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (k == c) vis[k] = v;
      }
    }
  };
  // Pages of the context alone, behind the sinks' and past the last position that a window may begin at.
  static __device__ __forceinline__ void plain(const Params& p, const RowWalk<TreeSrc>& walk, int& lo, int& hi) {
    const Seq& s = walk.seq;
    const int off = s.n_sink - s.lo - walk.g.t0;  // from a page to the segment's tile
    const long long first = (long long)s.base + p.r.Nq - 1 - p.window;  // (a key at or before it may be hidden)
    lo = max(s.lo, p.window && first >= 0 ? (int)(first / kTile) + 1 : 0) + off;
    hi = s.base / kTile + off;
  }

  template <class Bars>
  static __device__ __forceinline__ void produce(const Params& p, RowWalk<TreeSrc>& walk, uint8_t* smem, uint32_t sbase,
                                                 const Bars& bars, int warp, int lane) {
    using C = Cfg;
    auto raw_full = [&](int T) { return bars.at(Bars::kNum + T % kRaw); };
    auto raw_empty = [&](int T) { return bars.at(Bars::kNum + kRaw + T % kRaw); };
    const RowSeg& g = walk.g;
    int T = 0;
    bool ok = true;
    if (warp == 0) {
      // ---- pages come in
      while (ok && walk.next(p, lane)) {
        const uint8_t* head = p.pages + (size_t)g.h * kPageBytes;
        const int32_t* table = p.table + (size_t)g.b * p.max_pages;
        const int held = (walk.seq.len + kTile - 1) / kTile;
        int tbase = -64, entry = 0;  // entry: this lane's of the 32 table entries from tbase
        for (int t = g.t0; t < g.t1; ++t, ++T) {
          const int e = walk.seq.page(t);
          if ((unsigned)(e - tbase) >= 32u) {
            tbase = e;
            entry = e + lane < held ? table[e + lane] : 0;
          }
          int page = __shfl_sync(0xffffffffu, entry, e - tbase);
          if (T >= kRaw && !(ok = bars.warp_wait(raw_empty(T), ((T / kRaw) & 1) ^ 1))) break;
          if (lane == 0) {
            if ((unsigned)page >= (unsigned)p.num_pages) {  // reads page 0, and is reported
              if (p.r.err) atomicCAS(p.r.err, 0, APA_DEVERR_BOUNDS);
              page = 0;
            }
            mbar_arrive_expect_tx(raw_full(T), kPageBytes);
            bulk_g2s(sbase + C::kSrcOff + T % kRaw * kPageBytes, head + (size_t)page * p.r.Hkv * kPageBytes, kPageBytes,
                     raw_full(T));
          }
          __syncwarp();
        }
      }
      // every copy issued lands before the CTA exits, also when another warp gave up
      if (lane == 0)
        for (int x = max(0, T - kRaw); x < T; ++x) rows_wait_in_flight(raw_full(x), (x / kRaw) & 1, p.r.err);
      __syncwarp();
      return;
    }
    const bool of_k = warp <= kKWarps;
    const int w = of_k ? warp - 1 : warp - 1 - kKWarps;
    while (ok && walk.next(p, lane)) {
      for (int t = g.t0; t < g.t1; ++t, ++T) {
        const uint8_t* raw = smem + C::kSrcOff + T % kRaw * kPageBytes;
        if (!(ok = bars.warp_wait(raw_full(T), (T / kRaw) & 1))) break;
        if (of_k) {
          if (T >= C::NK && !(ok = bars.warp_wait(bars.k_empty(T), Bars::k_par(T) ^ 1))) break;
          uint8_t* dst = smem + C::kKOff + T % C::NK * C::kTileBytes;
          // A lane takes 32 channels (16 code bytes, two scales) of a key.  Eight neighbouring lanes store to four
          // keys and both halves of 64 channels: all banks once.
          constexpr int kQuarters = D / 32 < 4 ? D / 32 : 4, kUnits = kTile * D / 1024;
#pragma unroll 1
          for (int u = 0; u < kUnits / kKWarps; ++u) {
            const int unit = u * kKWarps + w;
            int key, q;
            if constexpr (D == 64) {
              key = 16 * unit + (lane & 3) + 4 * (lane >> 3);
              q = (lane >> 2) & 1;
            } else {
              key = 8 * (unit / (D / 128)) + (lane & 3) + 4 * ((lane >> 3) & 1);
              q = ((lane >> 2) & 1) + 2 * (lane >> 4) + 4 * (unit % (D / 128));
            }
            static_assert(kQuarters >= 2, "channels");
            const uint8_t* blk = raw + key / kBlkKeys * blk_bytes(D);
            const uint4 code = *reinterpret_cast<const uint4*>(blk + key % kBlkKeys * (D / 2) + 16 * q);
            const uint32_t sc = tree_e4m3x2(*reinterpret_cast<const uint16_t*>(blk + ks_byte(D, key % kBlkKeys, 2 * q)));
            const uint32_t f[2] = {__byte_perm(sc, 0, 0x1010), __byte_perm(sc, 0, 0x3232)};
            const uint32_t cw[4] = {code.x, code.y, code.z, code.w};
            uint8_t* row = dst + (q >> 1) * (KT * 128) + key * 128;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t h[4];
              tree_e2m1x8(cw[k], h);
#pragma unroll
              for (int e = 0; e < 4; ++e) h[e] = tree_hmul2(h[e], f[k >> 1]);
              *reinterpret_cast<uint4*>(row + ((((q & 1) * 4 + k) ^ (key & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(raw_empty(T));
            mbar_arrive(bars.k_full(T));
          }
        } else {
          if (T >= C::NV && !(ok = bars.warp_wait(bars.v_empty(T), Bars::v_par(T) ^ 1))) break;
          uint8_t* dst = smem + C::kVOff + T % C::NV * C::kTileBytes;
          const Seq& s = walk.seq;
          const int j0 = s.page(t) * kTile;
          // keys past the end, and before every window, count as 0 whatever the page holds there: a weight of 0 does not
          // hide a NaN
          const int gap = p.window ? s.base - p.window : -1;  // the last key before every row's window
          const bool edge = j0 + kTile > s.len || (j0 <= gap && j0 + kTile > p.sinks);
          // A lane takes four keys and four of the eight byte rows (channels g, g + 8) of 64 channels.
          const int q = lane & 3, gh = (lane >> 2) & 1, mb = lane >> 3;
          const uint8_t* blk = raw + mb * blk_bytes(D);
#pragma unroll
          for (int u = 0; u < D / 64; ++u) {
            if (D == 64 ? (T & 1) != w : u % kVWarps != w) continue;
            uint4 code[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              code[j] = *reinterpret_cast<const uint4*>(blk + blk_v(D) + 512 * u + 64 * (4 * gh + j) + 16 * q);
            const uint4 sc4 = *reinterpret_cast<const uint4*>(blk + blk_vs(D) + 4 * (q * (D / 16) + 4 * u));
            const uint32_t sc[4] = {sc4.x, sc4.y, sc4.z, sc4.w};
            uint32_t keep = ~0u;
            if (edge)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int j = j0 + 16 * mb + 4 * q + k;
                if (j >= s.len || (j <= gap && j >= p.sinks)) keep &= ~(255u << (8 * k));
              }
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) {
              const uint32_t b = sc[tt] & keep, f01 = tree_e4m3x2(b & 0xFFFFu), f23 = tree_e4m3x2(b >> 16);
              const uint32_t f[4] = {__byte_perm(f01, 0, 0x1010), __byte_perm(f01, 0, 0x3232), __byte_perm(f23, 0, 0x1010),
                                     __byte_perm(f23, 0, 0x3232)};
              uint32_t h[4][4];  // [byte row][key]
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t cw[4] = {code[j].x, code[j].y, code[j].z, code[j].w};
                tree_e2m1x8(cw[tt], h[j]);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int key = 16 * mb + 4 * q + k;
                *reinterpret_cast<uint4*>(dst + u * (KT * 128) + key * 128 + (((2 * tt + gh) ^ (key & 7)) << 4)) =
                    make_uint4(tree_hmul2(h[0][k], f[k]), tree_hmul2(h[1][k], f[k]), tree_hmul2(h[2][k], f[k]),
                               tree_hmul2(h[3][k], f[k]));
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(raw_empty(T));
            mbar_arrive(bars.v_full(T));
          }
        }
      }
    }
  }
};

}  // namespace
}  // namespace apa

using namespace apa;

extern "C" {

size_t apa_attention_tree_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d) {
  if (rows_bad_heads(B, Hq, Hkv, Nq) || Nq > APA_TREE_MAX_NODES || (d != 64 && d != 128 && d != 256)) return 0;
  return rows_workspace(Hq / Hkv * Nq, d);
}

int apa_attention_tree(const void* q, int dtype, long long q_batch_stride, long long q_head_stride,
                       long long q_row_stride, const uint8_t* pages, int num_pages, const int32_t* block_table,
                       int max_pages, const int32_t* lens, const int32_t* nodes, const uint32_t* mask,
                       long long mask_stride, const int32_t* depths, long long depth_stride, const float* k_scale,
                       const float* v_scale, int B, int Hq, int Hkv, int Nq, int d, int window, int sinks, void* out,
                       float* lse, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!q || !pages || !block_table || !lens || !mask || !k_scale || !v_scale || !out || (window && !depths))
    return APA_ERR_NULL;
  if (rows_bad_heads(B, Hq, Hkv, Nq) || Nq > APA_TREE_MAX_NODES || num_pages < 1 || num_pages >= (1 << 25) ||
      max_pages < 1 || (long long)B * max_pages >= (1 << 29) || max_pages >= (1 << 25) || mask_stride < 0 || depth_stride < 0)
    return APA_ERR_SHAPE;
  if (d != 64 && d != 128 && d != 256) return APA_ERR_HEAD_DIM;
  if (dtype != APA_DTYPE_BF16 && dtype != APA_DTYPE_F16) return APA_ERR_DTYPE;
  if (window < 0 || sinks < 0) return APA_ERR_WINDOW;
  // (uses are counted in 32 bits per head, and per CTA)
  const double uses = (double)B * (max_pages + 16.0) * (((double)(Hq / Hkv) * Nq + 127) / 128 + 1);
  if (uses >= 2147483648.0 || uses * Hkv >= 137438953472.0) return APA_ERR_SHAPE;
  // (the stride of an axis of length 1 is never used: any value will do)
  if (B == 1) q_batch_stride = mask_stride = depth_stride = 0;
  if (Hq == 1) q_head_stride = 0;
  if (Nq == 1) q_row_stride = 0;
  if ((((uintptr_t)q | (uintptr_t)pages | (uintptr_t)out) & 15) || ((q_batch_stride | q_head_stride | q_row_stride) & 7))
    return APA_ERR_ALIGN;
  const size_t need = apa_attention_tree_workspace_bytes(B, Hq, Hkv, Nq, d);
  void* ws = workspace;
  if (ws && (workspace_bytes < need || ((uintptr_t)ws & 255))) return APA_ERR_NOMEM;
  // (past every position, of which none exceeds 64 * max_pages + Nq: that may pass 2^31)
  if (window > (long long)max_pages * kTile + Nq) window = 0;
  // (past every key of the largest table; whole pages of them are counted in 32 bits)
  if (sinks > 0x7FFFFFFF - (kTile - 1)) sinks = 0x7FFFFFFF - (kTile - 1);
  if (!ws && cudaMallocAsync(&ws, need, stream) != cudaSuccess) return APA_ERR_NOMEM;
  const bool f16 = dtype == APA_DTYPE_F16;
  auto go = [&](auto src) {
    using Src = decltype(src);
    typename Src::Params p{};
    p.r.B = B;
    p.r.Hq = Hq;
    p.r.Hkv = Hkv;
    p.r.Nq = Nq;
    p.r.q = (const uint16_t*)q;
    p.r.qs_b = q_batch_stride;
    p.r.qs_h = q_head_stride;
    p.r.qs_r = q_row_stride;
    p.r.out = (uint16_t*)out;
    p.r.lse = lse;
    p.r.err = device_error_word();
    p.pages = pages;
    p.num_pages = num_pages;
    p.table = block_table;
    p.max_pages = max_pages;
    p.lens = lens;
    p.nodes = nodes;
    p.mask = mask;
    p.mask_stride = mask_stride;
    p.words = (Nq + 31) / 32;
    p.depths = depths;
    p.depth_stride = depth_stride;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.window = window;
    p.sinks = sinks;
    return launch_rows<Src>(p, ws, stream);
  };
  cudaError_t e = cudaErrorInvalidValue;
  const bool two = rows_two_blocks(Hq / Hkv * Nq, d);
  switch (d) {
    case 64:
      e = f16 ? go(TreeSrc<64, true, false>{}) : go(TreeSrc<64, false, false>{});
      break;
    case 128:
      e = two ? (f16 ? go(TreeSrc<128, true, true>{}) : go(TreeSrc<128, false, true>{}))
              : (f16 ? go(TreeSrc<128, true, false>{}) : go(TreeSrc<128, false, false>{}));
      break;
    case 256: e = f16 ? go(TreeSrc<256, true, false>{}) : go(TreeSrc<256, false, false>{}); break;
  }
  int st = e == cudaSuccess ? APA_OK : APA_ERR_CUDA;
  if (!workspace && cudaFreeAsync(ws, stream) != cudaSuccess && st == APA_OK) st = APA_ERR_CUDA;
  return st;
}

}  // extern "C"
