// apa_cross.cu -- attention to an encoder's states, of a length of its own for each sequence.
//
// out = softmax(q K^T / sqrt(d)) V over the keys below lens[b]; every row sees all of them.
// K and V tiles come by TMA (any strides); keys past Nkv arrive as zeros, and where a
// sequence ends before, its last tile's values behind the end are set to zero in shared
// memory, as a weight of 0 does not hide a NaN.
// A decoding step is bound by HBM: 64 sequences of up to 4096 keys, G = 3, d = 128, 118 us, 5.7
// TB/s of the copy's 6.8.  Prompts are bound by the products and what lies between them (rows.cuh):
// 4 x 2048 rows, 24 heads on 8, to 8192 keys, 413 us, 0.67 of the measured BF16 rate; with all
// lengths 8192 597 us, 0.71 (d = 64: 485 us, 0.44; d = 256: 1243 us, 0.69).
#include "rows.cuh"

namespace apa {
namespace {

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

// kTwo: items of up to two blocks, else of one.
template <int D, bool F16, bool kTwo>
struct CrossPick;
template <bool F16>
struct CrossPick<64, F16, false> { using Cfg = RowCfg<64, 64, 1, 2, true, 5, 5, F16>; };
template <bool F16>
struct CrossPick<128, F16, true> { using Cfg = RowCfg<128, 64, 2, 2, false, 4, 4, F16>; };
template <bool F16>
struct CrossPick<128, F16, false> { using Cfg = RowCfg<128, 64, 1, 1, true, 2, 3, F16>; };
template <bool F16>
struct CrossPick<256, F16, false> { using Cfg = RowCfg<256, 64, 1, 2, true, 3, 3, F16>; };

template <int D, bool F16, bool kTwo>
struct CrossSrc {
  using Cfg = typename CrossPick<D, F16, kTwo>::Cfg;
  static constexpr int kSrcWarps = 2, kThreads = (Cfg::kSrcWarp + kSrcWarps) * 32;
  static constexpr int kKArrivals = 1, kVArrivals = 1;
  static constexpr bool kVFirst = true;  // stages of V go back before S is issued: the copies behind them are long
  static constexpr int kBars = Cfg::NV;  // per stage of V: a last tile has landed, values behind the end and all
  static __device__ __forceinline__ uint32_t bar_count(int) { return 1; }
  static constexpr bool kPairedV = false, kOutF16 = F16, kScaledQ = false, kMasked = false;
  static constexpr int kItemCost = Cfg::kItemCost;
  static constexpr int kSoftUnroll = 2;
  static constexpr int kSmem = Cfg::kSrcOff + 1024;
  static_assert(Cfg::kCtasPerSm * (kSmem + (Cfg::NG == 2 ? 4096 : 2048) + 1024) <= 233472, "shared memory");

  struct Params {
    RowParams r;
    const int32_t* lens;  // or null: Nkv for all
    int Nkv;
    int kb, kh, vb, vh;  // 0 where all sequences (heads) share K (V), else 1
    CUtensorMap kmap, vmap;
  };
  struct Seq {
    int blocks, tiles, len;
    Seq() = default;
    __device__ __forceinline__ Seq(const Params& p, int b) {
      len = p.lens ? max(0, min(p.lens[b], p.Nkv)) : p.Nkv;
      tiles = (len + Cfg::KT - 1) / Cfg::KT;
      blocks = (p.r.G() * p.r.Nq + kBlockRows - 1) / kBlockRows;
    }
    __device__ __forceinline__ void report(const Params& p, int b) const {
      if (blockIdx.x == 0 && p.lens && p.lens[b] != len && p.r.err) atomicCAS(p.r.err, 0, APA_DEVERR_BOUNDS);
    }
    // the last tile holds keys behind the end that are not zeros already
    __device__ __forceinline__ bool ragged(const Params& p) const { return len < min(p.Nkv, tiles * Cfg::KT); }
  };
  struct Row {
    bool valid;
    int out_row;
    float c2, v_scale;
    __device__ __forceinline__ void set(const Params& p, const Seq&, int b, int h, int P) {
      const int G = p.r.G();
      valid = P < G * p.r.Nq;
      out_row = valid ? (b * p.r.Hq + h * G + P % G) * p.r.Nq + P / G : -1;
      c2 = kLog2e * rsqrtf((float)D);
      v_scale = 1.f;
    }
    __device__ __forceinline__ uint32_t convert(uint32_t w, float) const { return w; }
    // which of a tile's keys the row sees, in words of 32
    template <int N>
    __device__ __forceinline__ void mask(const Params&, const RowWalk<CrossSrc>& walk, int tile, uint32_t* vis) const {
      const int left = walk.seq.len - (walk.g.t0 + tile) * Cfg::KT;
#pragma unroll
      for (int c = 0; c < N; ++c) {
        const int n = left - 32 * c;
        vis[c] = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
      }
    }
  };

  template <class Bars>
  static __device__ __forceinline__ void produce(const Params& p, RowWalk<CrossSrc>& walk, uint8_t* smem, uint32_t sbase,
                                                 const Bars& bars, int warp, int lane) {
    using C = Cfg;
    constexpr int KT = C::KT, kAtoms = D / 64;
    auto landed = [&](int T) { return bars.at(Bars::kNum + T % C::NV); };
    const RowSeg& g = walk.g;
    int T = 0;
    bool ok = true;
    if (warp == 0) {
      int issued_k = 0, issued_v = 0;
      uint32_t last = 0, last_par = 0;  // bit per stage of V: its copy counts on `landed`, and that barrier's parity
      if (lane == 0) {
        prefetch_tmap(&p.kmap);
        prefetch_tmap(&p.vmap);
      }
      while (ok && walk.next(p, lane)) {
        if (lane == 0) {
          const bool ragged = walk.seq.ragged(p);
          for (int t = g.t0; t < g.t1; ++t, ++T) {
            if (T >= C::NK && !(ok = bars.wait(bars.k_empty(T), Bars::k_par(T) ^ 1))) break;
            mbar_arrive_expect_tx(bars.k_full(T), C::kTileBytes);
#pragma unroll
            for (int a = 0; a < kAtoms; ++a)
              tma_load_4d(sbase + C::kKOff + (T % C::NK) * C::kTileBytes + a * (KT * 128), &p.kmap, a * 64, t * KT,
                          g.h * p.kh, g.b * p.kb, bars.k_full(T));
            issued_k = T + 1;
            if (T >= C::NV && !(ok = bars.wait(bars.v_empty(T), Bars::v_par(T) ^ 1))) break;
            const bool fix = ragged && t == g.n - 1;
            const uint32_t bit = 1u << (T % C::NV), bar = fix ? landed(T) : bars.v_full(T);
            if (last & bit) last_par ^= bit;
            last = fix ? last | bit : last & ~bit;
            mbar_arrive_expect_tx(bar, C::kTileBytes);
#pragma unroll
            for (int a = 0; a < kAtoms; ++a)
              tma_load_4d(sbase + C::kVOff + (T % C::NV) * C::kTileBytes + a * (KT * 128), &p.vmap, a * 64, t * KT,
                          g.h * p.vh, g.b * p.vb, bar);
            issued_v = T + 1;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      // every copy issued lands before the CTA exits, also when another warp gave up
      if (lane == 0) {
        for (int x = max(0, issued_k - C::NK); x < issued_k; ++x) rows_wait_in_flight(bars.k_full(x), Bars::k_par(x), p.r.err);
        for (int x = max(0, issued_v - C::NV); x < issued_v; ++x) {
          const uint32_t bit = 1u << (x % C::NV);
          if (last & bit)
            rows_wait_in_flight(landed(x), last_par & bit ? 1 : 0, p.r.err);
          else
            rows_wait_in_flight(bars.v_full(x), Bars::v_par(x), p.r.err);
        }
      }
      __syncwarp();
    } else {
      // the last tiles' values behind the end: zeros
      uint32_t par = 0;
      while (walk.next(p, lane)) {
        T += g.t1 - g.t0;
        if (g.t1 < g.n || !walk.seq.ragged(p)) continue;
        const int x = T - 1, st = x % C::NV;
        if (!bars.warp_wait(landed(x), (par >> st) & 1)) break;
        par ^= 1u << st;
        const int n = walk.seq.len - (g.n - 1) * KT;  // keys of the tile in use
        uint8_t* tile = smem + C::kVOff + st * C::kTileBytes;
        for (int i = lane; i < (KT - n) * (D / 8); i += 32) {  // 16 bytes each; whole 128-byte rows, so in any order
          const int key = n + i / (D / 8), c = i % (D / 8);
          *reinterpret_cast<uint4*>(tile + (c >> 3) * (KT * 128) + key * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.v_full(x));
      }
    }
  }
};

// Tensor map of K or V, [B][Hkv][Nkv][d] with the given strides (in elements), for boxes of 64 channels x
// kt keys with the 128-byte swizzle.  Axes that are shared (stride 0) or have length 1 become axes of length 1.
bool cross_map(CUtensorMap* map, const void* base, bool f16, int B, int H, int N, int d, long long sb, long long sh,
               long long st, int kt) {
  using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::atomic<EncodeFn> known{nullptr};
  EncodeFn encode = known.load();
  if (!encode) {
    cudaDriverEntryPointQueryResult found;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess || !fn)
      return false;
    known.store(encode = reinterpret_cast<EncodeFn>(fn));
  }
  const cuuint64_t row = (cuuint64_t)d * 2;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)(sh ? H : 1), (cuuint64_t)(sb ? B : 1)};
  const cuuint64_t strides[3] = {N > 1 ? (cuuint64_t)st * 2 : row, sh ? (cuuint64_t)sh * 2 : row, sb ? (cuuint64_t)sb * 2 : row};
  const cuuint32_t box[4] = {64, (cuuint32_t)kt, 1, 1}, steps[4] = {1, 1, 1, 1};
  return encode(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
                dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct CrossArgs {
  RowParams r;
  const void *k, *v;
  long long ks[3], vs[3];  // batch, head, token strides
  const int32_t* lens;
  int Nkv;
};
template <int D, bool F16, bool kTwo>
cudaError_t launch_cross_rows(const CrossArgs& a, void* ws, cudaStream_t stream) {
  using Src = CrossSrc<D, F16, kTwo>;
  typename Src::Params p{};
  p.r = a.r;
  p.lens = a.lens;
  p.Nkv = a.Nkv;
  p.kb = a.ks[0] != 0;
  p.kh = a.ks[1] != 0;
  p.vb = a.vs[0] != 0;
  p.vh = a.vs[1] != 0;
  if (!cross_map(&p.kmap, a.k, F16, a.r.B, a.r.Hkv, a.Nkv, D, a.ks[0], a.ks[1], a.ks[2], Src::Cfg::KT) ||
      !cross_map(&p.vmap, a.v, F16, a.r.B, a.r.Hkv, a.Nkv, D, a.vs[0], a.vs[1], a.vs[2], Src::Cfg::KT))
    return cudaErrorInvalidValue;
  return launch_rows<Src>(p, ws, stream);
}
template <int D, bool F16>
cudaError_t launch_cross(const CrossArgs& a, void* ws, cudaStream_t stream) {
  if constexpr (D == 128)
    if (rows_two_blocks(a.r.G() * a.r.Nq, D)) return launch_cross_rows<D, F16, true>(a, ws, stream);
  return launch_cross_rows<D, F16, false>(a, ws, stream);
}

}  // namespace
}  // namespace apa

using namespace apa;

extern "C" {

size_t apa_attention_cross_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d) {
  if (rows_bad_heads(B, Hq, Hkv, Nq) || (d != 64 && d != 128 && d != 256)) return 0;
  return rows_workspace(Hq / Hkv * Nq, d);
}

int apa_attention_cross(const void* q, int dtype, long long q_batch_stride, long long q_head_stride,
                        long long q_row_stride, const void* k, long long k_batch_stride, long long k_head_stride,
                        long long k_token_stride, const void* v, long long v_batch_stride, long long v_head_stride,
                        long long v_token_stride, const int32_t* lens, int B, int Hq, int Hkv, int Nq, int Nkv, int d,
                        void* out, float* lse, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!q || !k || !v || !out) return APA_ERR_NULL;
  if (rows_bad_heads(B, Hq, Hkv, Nq) || Nkv < 1 || Nkv > (1 << 30)) return APA_ERR_SHAPE;
  if (d != 64 && d != 128 && d != 256) return APA_ERR_HEAD_DIM;
  if (dtype != APA_DTYPE_BF16 && dtype != APA_DTYPE_F16) return APA_ERR_DTYPE;
  // (uses are counted in 32 bits per head, and per CTA)
  const double uses = (double)B * ((Nkv + 63) / 64 + 16.0) * (((double)(Hq / Hkv) * Nq + 127) / 128 + 1);
  if (uses >= 2147483648.0 || uses * Hkv >= 137438953472.0) return APA_ERR_SHAPE;
  // (the stride of an axis of length 1 is never used: any value will do)
  if (B == 1) q_batch_stride = k_batch_stride = v_batch_stride = 0;
  if (Hq == 1) q_head_stride = 0;
  if (Hkv == 1) k_head_stride = v_head_stride = 0;
  if (Nq == 1) q_row_stride = 0;
  if (Nkv == 1) k_token_stride = v_token_stride = d;
  const long long all[8] = {k_batch_stride, k_head_stride, k_token_stride, v_batch_stride,
                            v_head_stride,  v_token_stride, 0, 0};
  for (long long s : all)
    if (s < 0 || s >= (1ll << 39) || (s & 7)) return APA_ERR_ALIGN;
  if (!k_token_stride || !v_token_stride) return APA_ERR_ALIGN;
  if ((((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)out) & 15) ||
      ((q_batch_stride | q_head_stride | q_row_stride) & 7))
    return APA_ERR_ALIGN;
  const size_t need = apa_attention_cross_workspace_bytes(B, Hq, Hkv, Nq, d);
  void* ws = workspace;
  if (ws && (workspace_bytes < need || ((uintptr_t)ws & 255))) return APA_ERR_NOMEM;
  if (!ws && cudaMallocAsync(&ws, need, stream) != cudaSuccess) return APA_ERR_NOMEM;
  CrossArgs a{};
  a.r.B = B;
  a.r.Hq = Hq;
  a.r.Hkv = Hkv;
  a.r.Nq = Nq;
  a.r.q = (const uint16_t*)q;
  a.r.qs_b = q_batch_stride;
  a.r.qs_h = q_head_stride;
  a.r.qs_r = q_row_stride;
  a.r.out = (uint16_t*)out;
  a.r.lse = lse;
  a.r.err = device_error_word();
  a.k = k;
  a.v = v;
  a.ks[0] = k_batch_stride, a.ks[1] = k_head_stride, a.ks[2] = k_token_stride;
  a.vs[0] = v_batch_stride, a.vs[1] = v_head_stride, a.vs[2] = v_token_stride;
  a.lens = lens;
  a.Nkv = Nkv;
  const bool f16 = dtype == APA_DTYPE_F16;
  cudaError_t e = cudaErrorInvalidValue;
  switch (d) {
    case 64: e = f16 ? launch_cross<64, true>(a, ws, stream) : launch_cross<64, false>(a, ws, stream); break;
    case 128: e = f16 ? launch_cross<128, true>(a, ws, stream) : launch_cross<128, false>(a, ws, stream); break;
    case 256: e = f16 ? launch_cross<256, true>(a, ws, stream) : launch_cross<256, false>(a, ws, stream); break;
  }
  int st = e == cudaSuccess ? APA_OK : APA_ERR_CUDA;
  if (!workspace && cudaFreeAsync(ws, stream) != cudaSuccess && st == APA_OK) st = APA_ERR_CUDA;
  return st;
}

}  // extern "C"
