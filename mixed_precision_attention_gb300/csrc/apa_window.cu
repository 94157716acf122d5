// apa_window.cu -- exact causal prefill attention with a sliding window and sinks.
//
// out = softmax(q K^T / sqrt(d)) V over the keys j <= x with j > x - window or
// j < sinks, x the row's position.  The matrix products bound it (4 d flop per visible
// pair); what it comes to is set by the hand-overs between S, softmax and P.V of a tile,
// and, as walks are short, by what happens between two row blocks.  24 heads on 8, d = 128:
// 8192 rows, window 1024: 116 us (0.44 of the measured BF16 rate, the masked parts of
// tiles not counted); 16384 rows at the end of 122880 keys, window 4096: 663 us (0.65).
//
// One work item = 128 GQA-packed rows of one KV head (tcgen05 M = 128), which walk the
// 64-key tiles that hold sinks and those that their windows reach.  Persistent CTAs, two
// per SM at d <= 128 (256 TMEM columns and half the shared memory each), take items in
// turn, the longest walks first.  7 warps:
//   warps 0-3  softmax, one thread per row (TMEM lane = row), and the epilogue;
//   warp 4     TMA producer: K and V tiles (64 keys x d, 128-byte swizzle), a ring each;
//   warp 5     TMEM owner and S issuer: S = Q K^T (kind::f16);
//   warp 6     PV issuer: O += P V, P read from TMEM.
// TMEM: O, one S and two P.  S is free again as soon as the softmax threads hold its
// scores in registers, so the next tile's is computed while they work on this one, and
// P.V of a tile has a tile's time.
// Everything runs on over the end of an item: the producer is already loading the next
// item's tiles; the softmax threads store the next Q as soon as the last S is done and
// before they wait for the last P.V, so the next item's first S is computed under
// the epilogue; the first P.V of an item comes after it anyway, as its P does.
// P goes to the product in BF16 (2^-8 relative, the rounding of the output) against V
// itself, so there is no copy of V and no workspace; l adds the FP32 values.  The
// running maximum moves only when a score exceeds it by 8 (log2 units).
// Hidden scores are masked whatever they are.  A hidden V has the weight 0 in the product,
// which hides every finite value, but not a NaN or an infinity.
#include <atomic>

#include "apa_internal.h"
#include "apa_window.h"
#include "tc.cuh"

namespace apa {
namespace {

constexpr int kThreads = 224;
constexpr int kSms = 152;
constexpr float kTauWin = 8.0f;  // lazy rescale threshold (log2 units)

struct WinParams {
  Shape s;
  const uint16_t* q;
  int window, sinks;
  uint16_t* out;  // [B,Hq,Nq,d] bf16
  float* lse;     // [B,Hq,Nq] or null
  int* err;
};

template <int D>
struct WinCfg {
  static constexpr int kCtasPerSm = D <= 128 ? 2 : 1;
  // stages: V's products come last, so V waits longer (16384 rows, window 4096, d = 128:
  // 2 of K and 3 of V 670 us, 3 and 2 681, two stages for both together 885)
  static constexpr int NS = D == 64 ? 3 : 2, NSV = D == 256 ? 2 : 3;
  static constexpr int kAtoms = D / 64;
  static constexpr int kQBytes = 128 * D * 2;
  static constexpr int kKVBytes = 64 * D * 2;  // one of K or V per stage
  static constexpr int kKOff = kQBytes, kVOff = kKOff + NS * kKVBytes;
  static constexpr int kNumBars = 2 * NS + 2 * NSV + 9;
  static constexpr int kBarOff = kVOff + NSV * kKVBytes;
  // two CTAs of d = 128 leave no room to align the window: it must start on 1024 bytes
  static constexpr int kSlack = D == 128 ? 0 : 1024;
  static constexpr int kSmem = kBarOff + kNumBars * 8 + 16 + kSlack;
  static constexpr uint32_t kTmemCols = D + 128 <= 256 ? 256 : 512;
  static constexpr uint32_t kOCol = 0, kSCol = D, kPCol = D + 64;  // O, S, and P twice (32 columns each)
  static_assert(kCtasPerSm * (kSmem + 1024) <= 233472, "shared memory");
  static_assert(kCtasPerSm * kTmemCols <= 512, "TMEM");
};

// Work item k and its walk: entries 0 .. n_sink-1 are tiles 0 .., then tiles t_lo ..
struct WinItem {
  int bh, p0, n_sink, t_lo, n;
  __device__ __forceinline__ WinItem(const WinParams& p, int k) {
    const Shape& s = p.s;
    const int BH = s.BH(), G = s.G();
    bh = k % BH;
    p0 = (s.nblk() - 1 - k / BH) * kBlockRows;
    const int last = (min(s.R(), p0 + kBlockRows) - 1) / G + s.off();  // position of the block's last row
    t_lo = max(0, p0 / G + s.off() - p.window + 1) / kTile;
    n_sink = min((p.sinks + kTile - 1) / kTile, t_lo);
    n = n_sink + last / kTile - t_lo + 1;
  }
  __device__ __forceinline__ int tile(int i) const { return i < n_sink ? i : t_lo + i - n_sink; }
};
// The keys of tile j0 .. j0+63 that a row at position x sees: indices 0 .. nvis-1 but
// for gap_lo .. gap_hi-1.  nvis <= 0 if there is none.
struct RowKeys {
  int nvis, gap_lo, gap_hi;
  __device__ __forceinline__ RowKeys(const WinParams& p, int x, int j0, bool valid) {
    nvis = valid ? min(kTile, x + 1 - j0) : 0;
    gap_hi = min(kTile, x - p.window + 1 - j0);  // first key of the window
    gap_lo = max(0, min(kTile, p.sinks - j0));   // first key that is no sink
    if (gap_lo == 0 && gap_hi >= nvis) nvis = 0;
  }
  __device__ __forceinline__ bool all() const { return nvis == kTile && gap_lo >= gap_hi; }
  __device__ __forceinline__ bool sees(int i) const { return i < nvis && (i < gap_lo || i >= gap_hi); }
};

// P of eight consecutive keys, 2^(x*c2 + nb), as four BF16x2 words (key 2k in the low half
// of word k); the FP32 values are added into (s0, s1): even keys into s0, odd keys into
// s1.  The affine step and the sums run as packed FP32 pairs.
__device__ __forceinline__ void p8_bf16(const float* x, float c2, float nb, uint32_t* h, float& s0, float& s1) {
  uint64_t c, n, one, s, a[4];
  asm("mov.b64 %0, {%1, %1};" : "=l"(c) : "f"(c2));
  asm("mov.b64 %0, {%1, %1};" : "=l"(n) : "f"(nb));
  asm("mov.b64 %0, {%1, %1};" : "=l"(one) : "f"(1.f));
  asm("mov.b64 %0, {%1, %2};" : "=l"(s) : "f"(s0), "f"(s1));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float lo, hi;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a[k]) : "f"(x[2 * k]), "f"(x[2 * k + 1]));
    asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(a[k]) : "l"(c), "l"(n));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a[k]));
    lo = ex2_approx(lo);
    hi = ex2_approx(hi);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[k]) : "f"(hi), "f"(lo));
    asm("mov.b64 %0, {%1, %2};" : "=l"(a[k]) : "f"(lo), "f"(hi));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(s) : "l"(a[k]), "l"(one));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(s0), "=f"(s1) : "l"(s));
}

// used only while unwinding: waits for copies already in flight, ignoring the abort flag
__device__ __forceinline__ void wait_in_flight(uint32_t bar, uint32_t parity, int* err) {
  const unsigned long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > APA_WAIT_LIMIT_CYCLES) {
      if (err) atomicCAS(err, 0, APA_DEVERR_TIMEOUT);
      return;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, WinCfg<D>::kCtasPerSm)
    window_kernel(const WinParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using C = WinCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  if (C::kSlack == 0 && smem != smem_raw) {  // no room to realign: refuse loudly
    if (threadIdx.x == 0) atomicCAS(p.err, 0, APA_DEVERR_SMEM_ALIGN);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint32_t& tmem_slot = *reinterpret_cast<uint32_t*>(smem + C::kBarOff + C::kNumBars * 8);
  int& abort_flag = *reinterpret_cast<int*>(smem + C::kBarOff + C::kNumBars * 8 + 4);

  const Shape& s = p.s;
  const int G = s.G(), R = s.R(), off = s.off(), items = s.BH() * s.nblk();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = smem_u32(bars);
  // Barriers.  T counts the tiles of all of this CTA's items in turn, j its items.
  auto k_full = [&](int T) { return bar0 + 8u * (T % C::NS); };
  auto k_empty = [&](int T) { return bar0 + 8u * (C::NS + T % C::NS); };
  auto v_full = [&](int T) { return bar0 + 8u * (2 * C::NS + T % C::NSV); };
  auto v_empty = [&](int T) { return bar0 + 8u * (2 * C::NS + C::NSV + T % C::NSV); };
  constexpr int kB0 = 2 * C::NS + 2 * C::NSV;
  const uint32_t s_full = bar0 + 8u * kB0, s_free = bar0 + 8u * (kB0 + 1);  // s_free: one arrive per softmax warp
  auto p_full = [&](int T) { return bar0 + 8u * (kB0 + 2 + (T & 1)); };     // one arrive per softmax warp
  auto pv_done = [&](int T) { return bar0 + 8u * (kB0 + 4 + (T & 1)); };
  const uint32_t q_full = bar0 + 8u * (kB0 + 6);  // one arrive per softmax warp
  const uint32_t drain_s = bar0 + 8u * (kB0 + 7), drain_pv = bar0 + 8u * (kB0 + 8);
  // every lane of a softmax warp waits; the warp proceeds only if all lanes succeeded
  auto warp_wait = [&](uint32_t bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;  // already complete
    const bool okl = mbar_wait(bar, parity, &abort_flag, p.err);
    return __all_sync(0xffffffffu, okl);
  };

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < C::kNumBars; ++i) {
      const int x = i - kB0;
      mbar_init(bar0 + 8u * i, x == 1 || x == 2 || x == 3 || x == 6 ? 4u : 1u);
    }
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(&tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 4 && lane == 0) {
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp == 4) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int T = 0, issued_k = 0, issued_v = 0;
      bool ok = true;
      for (int k = blockIdx.x; ok && k < items; k += gridDim.x) {
        const WinItem it(p, k);
        for (int i = 0; i < it.n; ++i, ++T) {
          const int y = it.tile(i) * kTile;
          if (T >= C::NS && !(ok = mbar_wait(k_empty(T), ((T / C::NS) - 1) & 1, &abort_flag, p.err))) break;
          mbar_arrive_expect_tx(k_full(T), C::kKVBytes);
#pragma unroll
          for (int a = 0; a < C::kAtoms; ++a)
            tma_load_3d(sbase + C::kKOff + (T % C::NS) * C::kKVBytes + a * 8192, &kmap, a * 64, y, it.bh, k_full(T));
          issued_k = T + 1;
          if (T >= C::NSV && !(ok = mbar_wait(v_empty(T), ((T / C::NSV) - 1) & 1, &abort_flag, p.err))) break;
          mbar_arrive_expect_tx(v_full(T), C::kKVBytes);
#pragma unroll
          for (int a = 0; a < C::kAtoms; ++a)
            tma_load_3d(sbase + C::kVOff + (T % C::NSV) * C::kKVBytes + a * 8192, &vmap, a * 64, y, it.bh, v_full(T));
          issued_v = T + 1;
        }
      }
      // every copy issued lands before the CTA exits, also when another warp gave up
      // (normally they have all landed: the waits return at once)
      for (int x = max(0, issued_k - C::NS); x < issued_k; ++x) wait_in_flight(k_full(x), (x / C::NS) & 1, p.err);
      for (int x = max(0, issued_v - C::NSV); x < issued_v; ++x) wait_in_flight(v_full(x), (x / C::NSV) & 1, p.err);
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------ S issuer
    if (lane == 0) {
      const uint32_t idS = idesc_bf16(128, 64, 0);
      int T = 0, j = 0;
      bool ok = true;
      for (int k = blockIdx.x; ok && k < items; k += gridDim.x, ++j) {
        const int n = WinItem(p, k).n;
        if (!(ok = mbar_wait(q_full, j & 1, &abort_flag, p.err))) break;
        for (int i = 0; i < n; ++i, ++T) {
          if (!(ok = mbar_wait(k_full(T), (T / C::NS) & 1, &abort_flag, p.err))) break;
          // the softmax threads have taken the scores of the tile before
          if (T >= 1 && !(ok = mbar_wait(s_free, (T - 1) & 1, &abort_flag, p.err))) break;
          tc_fence_after();
          const uint32_t kaddr = sbase + C::kKOff + (T % C::NS) * C::kKVBytes;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t ad = smem_desc(sbase + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024, kSwizzle128B);
            const uint64_t bd = smem_desc(kaddr + (kk >> 2) * 8192 + (kk & 3) * 32, 16, 1024, kSwizzle128B);
            mma_bf16(tmem + C::kSCol, ad, bd, idS, kk > 0);
          }
          mma_commit(s_full);
          mma_commit(k_empty(T));  // this stage's K has been read
        }
      }
      // drain: every tcgen05 op issued by this thread has completed before TMEM is freed
      mma_commit(drain_s);
      wait_in_flight(drain_s, 0, p.err);
    }
  } else if (warp == 6) {
    // ------------------------------------------------------------ PV issuer
    if (lane == 0) {
      const uint32_t idO = idesc_bf16(128, D, 1);
      int T = 0;
      bool ok = true;
      for (int k = blockIdx.x; ok && k < items; k += gridDim.x) {
        const int n = WinItem(p, k).n;
        // (the P of an item's first tile comes after the epilogue that read the last item's O)
        for (int i = 0; i < n; ++i, ++T) {
          if (!(ok = mbar_wait(p_full(T), (T >> 1) & 1, &abort_flag, p.err))) break;
          if (!(ok = mbar_wait(v_full(T), (T / C::NSV) & 1, &abort_flag, p.err))) break;
          tc_fence_after();
          const uint32_t vaddr = sbase + C::kVOff + (T % C::NSV) * C::kKVBytes;
          const uint32_t pcol = tmem + C::kPCol + 32u * (T & 1);  // P (BF16): 16 keys per MMA
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t bd = smem_desc(vaddr + kk * 2048, 8192, 1024, kSwizzle128B);
            mma_f16_ts(tmem + C::kOCol, pcol + 8u * kk, bd, idO, (i > 0 || kk > 0) ? 1u : 0u);
          }
          mma_commit(pv_done(T));
          mma_commit(v_empty(T));  // this stage's V has been read
        }
      }
      mma_commit(drain_pv);
      wait_in_flight(drain_pv, 0, p.err);
    }
  } else {
    // ------------------------------------------------------------ softmax (one thread per row)
    const int r = threadIdx.x;  // row within the block
    const float c2 = kLog2e * rsqrtf((float)D);
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    // this thread's row of item k: its place in q and out (in rows), or -1
    auto row_of = [&](const WinItem& it, int& x) -> long long {
      const int P = it.p0 + r;
      if (P >= R) return -1;
      const int pos = P / G, b = it.bh / s.Hkv, h = it.bh % s.Hkv;
      x = pos + off;
      return ((long long)b * s.Hq + h * G + P % G) * s.Nq + pos;
    };
    // stores the row into Q's tile (128-byte swizzle, K-major), zeros behind the last row
    auto put_q = [&](long long row) {
      const uint4* src = reinterpret_cast<const uint4*>(p.q + row * D);
#pragma unroll 16
      for (int c = 0; c < D / 8; ++c) {
        const uint4 val = row >= 0 ? src[c] : make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(smem + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = val;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    };
    int T = 0, x = 0;
    bool ok = true;
    long long row = row_of(WinItem(p, blockIdx.x), x);
    put_q(row);
    for (int k = blockIdx.x; ok && k < items; k += gridDim.x) {
      const WinItem it(p, k);
      if (k + (int)gridDim.x < items) {  // the next item's Q comes nearer meanwhile
        int xn;
        const long long next = row_of(WinItem(p, k + gridDim.x), xn);
        if (next >= 0)
#pragma unroll
          for (int c = 0; c < D; c += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + next * D + c));
      }
      float m2 = -INFINITY, l2 = 0.f;
      for (int i = 0; i < it.n; ++i, ++T) {
        if (!(ok = warp_wait(s_full, T & 1))) break;
        const RowKeys rk(p, x, it.tile(i) * kTile, row >= 0);
        const uint32_t pslot = tmem + lane_base + C::kPCol + 32u * (T & 1);  // P, two keys per column
        tc_fence_after();
        if (!__any_sync(0xffffffffu, rk.nvis > 0)) {
          // no row of this warp takes part in this tile: its P rows are zero
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free);
          if (T >= 2 && !(ok = warp_wait(pv_done(T), ((T >> 1) - 1) & 1))) break;
          tc_fence_after();
          uint32_t z[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) z[c] = 0u;
          tmem_st_x16(pslot, z);
          tmem_st_x16(pslot + 16, z);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(T));
          continue;
        }
        uint32_t raw[64];
        tmem_ld_x32(tmem + lane_base + C::kSCol, raw);
        tmem_ld_x32(tmem + lane_base + C::kSCol + 32, raw + 32);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free);
        float sv[64];
#pragma unroll
        for (int c = 0; c < 64; ++c) sv[c] = __uint_as_float(raw[c]);
        // hidden keys are masked where a row sees a part of the tile; a row that sees none of it
        // keeps its scores but takes no part: its maximum and its P bias are -inf
        if (__any_sync(0xffffffffu, rk.nvis > 0 && !rk.all())) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (!rk.sees(c)) sv[c] = -INFINITY;
        }
        float g8[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
          g8[c] = max3(max3(sv[8 * c], sv[8 * c + 1], sv[8 * c + 2]), max3(sv[8 * c + 3], sv[8 * c + 4], sv[8 * c + 5]),
                       fmaxf(sv[8 * c + 6], sv[8 * c + 7]));
        const float rmax = max3(max3(g8[0], g8[1], g8[2]), max3(g8[3], g8[4], g8[5]), fmaxf(g8[6], g8[7]));
        const float top = (rk.nvis <= 0 || rmax == -INFINITY) ? -INFINITY : rmax * c2;
        float f = 1.f;
        bool rescale = false;
        if (top > m2 + kTauWin || (m2 == -INFINITY && top > -INFINITY)) {
          if (l2 > 0.f) {
            f = ex2_approx(m2 - top);
            rescale = true;
          }
          m2 = top;
        }
        const float nb = (rk.nvis <= 0 || m2 == -INFINITY) ? -INFINITY : -m2;
        // the P.V of tile T - 2 has read what this P goes over
        if (T >= 2 && !(ok = warp_wait(pv_done(T), ((T >> 1) - 1) & 1))) break;
        tc_fence_after();
        float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pk[16];
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4) {
            const int ch = 4 * hf + c4;
            p8_bf16(sv + 8 * ch, c2, nb, pk + 4 * c4, ps[ch & 1], ps[2 + (ch & 1)]);
          }
          tmem_st_x16(pslot + 16u * hf, pk);
        }
        l2 = l2 * f + ((ps[0] + ps[1]) + (ps[2] + ps[3]));
        if (__any_sync(0xffffffffu, rescale)) {
          // O must not be read before the P.V of the tile before has landed
          if (!(ok = warp_wait(pv_done(T - 1), ((T - 1) >> 1) & 1))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t o[32];
            tmem_ld_x32(tmem + lane_base + C::kOCol + c0, o);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
            tmem_st_x16(tmem + lane_base + C::kOCol + c0, o);
            tmem_st_x16(tmem + lane_base + C::kOCol + c0 + 16, o + 16);
          }
        }
        tmem_wait_st();  // P (and a rescaled O) in TMEM before P.V is issued
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(T));
      }
      if (!ok) break;
      // ---- the next item's Q (every S of this one is done), then this one's epilogue
      const long long row0 = row;
      if (k + (int)gridDim.x < items) {
        row = row_of(WinItem(p, k + gridDim.x), x);
        put_q(row);
      }
      if (!(ok = warp_wait(pv_done(T - 1), ((T - 1) >> 1) & 1))) break;
      tc_fence_after();
      const float inv = 1.f / l2;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 64) {
        uint32_t o[64];
        tmem_ld_x32(tmem + lane_base + C::kOCol + c0, o);
        tmem_ld_x32(tmem + lane_base + C::kOCol + c0 + 32, o + 32);
        tmem_wait_ld();
        if (row0 >= 0) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + row0 * D + c0);
#pragma unroll
          for (int c = 0; c < 64; c += 8) {
            uint4 w;
            uint32_t* wr = &w.x;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                  : "=r"(wr[e])
                  : "f"(__uint_as_float(o[c + 2 * e + 1]) * inv), "f"(__uint_as_float(o[c + 2 * e]) * inv));
            dst[c / 8] = w;
          }
        }
      }
      if (row0 >= 0 && p.lse) p.lse[row0] = 0.6931471805599453f * (m2 + log2f(l2));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Tensor map of a contiguous K or V [B*Hkv][Nkv][d] for boxes of 64 channels x 64 keys with the
// 128-byte swizzle; keys past Nkv come as zeros.
bool tile_map(CUtensorMap* map, const void* base, const Shape& s) {
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
  const cuuint64_t dims[3] = {(cuuint64_t)s.d, (cuuint64_t)s.Nkv, (cuuint64_t)s.BH()};
  const cuuint64_t strides[2] = {(cuuint64_t)s.d * 2, (cuuint64_t)s.Nkv * s.d * 2};
  const cuuint32_t box[3] = {64, 64, 1}, steps[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_d(const WinParams& prm, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  using C = WinCfg<D>;
  static std::atomic<uint64_t> ready{0};  // the attribute, once per device (a bit each)
  cudaError_t e;
  int dev = 0;
  if ((e = cudaGetDevice(&dev))) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || !(ready.load() & bit)) {
    if ((e = cudaFuncSetAttribute(window_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem))) return e;
    if (dev <= 63) ready.fetch_or(bit);
  }
  const long long items = (long long)prm.s.BH() * prm.s.nblk();
  if (items > 0x7FFFFFFF - kSms * C::kCtasPerSm) return cudaErrorInvalidValue;
  const int grid = items < kSms * C::kCtasPerSm ? (int)items : kSms * C::kCtasPerSm;
  window_kernel<D><<<grid, kThreads, C::kSmem, st>>>(prm, km, vm);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window(const Shape& s, const void* q, const void* k, const void* v, int window, int sinks, void* out,
                          float* lse, cudaStream_t st) {
  CUtensorMap km, vm;
  if (!tile_map(&km, k, s) || !tile_map(&vm, v, s)) return cudaErrorInvalidValue;
  const WinParams prm{s, (const uint16_t*)q, window, sinks, (uint16_t*)out, lse, device_error_word()};
  switch (s.d) {
    case 64: return launch_d<64>(prm, km, vm, st);
    case 128: return launch_d<128>(prm, km, vm, st);
    case 256: return launch_d<256>(prm, km, vm, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace apa
