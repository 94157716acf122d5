// apa_decode.cu -- attention of a few query rows per sequence over the 4-bit K/V
// cache, with an optional sliding window and sinks.
//
// out = softmax(q K^T / sqrt(d)) V per (sequence, KV head), with the G * Nq rows that
// share the head's keys taken together (position-major, as in the prefill kernels).
//
// What bounds it: a key's K and V are 9 d / 8 bytes and are used by G * Nq rows, so
// up to a few tens of rows the cache's bytes do, next to the work of turning codes into
// FP16 operands, which an SM has to do at the rate it is fed (24 bytes, or 42 values, a
// cycle).  The products' M (or N) is the handful of rows; a tcgen05 tile has 128, and
// its block-scaled form would need Q and P in FP4 too, so the products run as
// mma.sync m16n8k16 on FP16 operands made in registers, at the bandwidth's rate.
//   S^T = K Q^T: A = 16 keys x 16 channels of K, B = Q^T, 8 rows; O^T = V^T P^T: A = 16
//   channels x 16 keys of V, B = P^T.  E2M1 * UE4M3 has 6 significant bits and lies in
//   2^-10 .. 2688, so K and V are exact in FP16; a row of Q is scaled by a power of two
//   into FP16's range.  P is rounded to FP16 (2^-11), lifted by 2^6 so that weights
//   down to 2^-30 of the row's largest keep a value; l sums the FP32 weights.
//
// Split: every warp works for itself.  The units (32 keys of one KV head, one
// contiguous half page) of all sequences, heads and row blocks form one list, which is
// cut evenly over the warps of the GPU, so lengths need not be alike and no length is
// read on the host.  A warp streams its units through a ring of its own with bulk
// copies (no barrier with other warps), keeps its own running maximum and sum, and
// moves the maximum only when a score exceeds it by 8 (log2 units).  An item (sequence,
// head, row block) that one warp holds entirely is written out at once; otherwise the
// parts go to the workspace, the warps of a CTA that works on one item joined
// first, and a second kernel joins them in order, so results do not depend on timing.
#include <cmath>

#include "../../include/apa.h"
#include "apa_internal.h"
#include "cache_page.cuh"
#include "tc.cuh"

namespace apa {
namespace {

constexpr int kMaxSeqs = 8192;
constexpr int kCtas = 152;   // one per SM
constexpr int kUnit = 32;    // keys per unit
constexpr float kTauDec = 8.f;   // lazy-maximum threshold, log2 units
constexpr float kLift = 6.f;     // P is 2^(x - m + kLift): at most 2^14, within FP16
constexpr float kLn2 = 0.6931471805599453f;

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
  int nstages;
  // workspace
  int* pref;       // [B + 1] units before each sequence (of one head and row block)
  float2* part_ml; // [slots][rows] (m, l)
  float* part_o;   // [slots][rows][d]
};

// Registers set the number of warps: O takes d * NT / 4 per thread, Q's fragments
// d * NT / 8.
template <int D, int NT>
struct DecCfg {
  static constexpr int kRegs = D * NT * 3 / 8;
  static constexpr int W = kRegs <= 64 ? 16 : kRegs <= 96 ? 12 : 8;
  static constexpr int kRows = 8 * NT;
  static constexpr int kUnitBytes = 36 * D;
  static constexpr int kMaxStages = 6;
  static constexpr int kSlots = 2 * kCtas * W;
  static constexpr int kBarBytes = W * kMaxStages * 8 + 16;
  static constexpr int kMergeBytes = W * kRows * (D + 2) * 4;
  static int stages(int B) {
    const int room = 232448 - kBarBytes - (B + 1) * 4 - 256;  // (256: the static arrays)
    const int n = room / (W * kUnitBytes);
    return n > kMaxStages ? kMaxStages : n;
  }
  static int ring_bytes(int B) {
    const int r = stages(B) * W * kUnitBytes;
    return r > kMergeBytes ? r : kMergeBytes;
  }
  static int smem(int B) { return ring_bytes(B) + kBarBytes + (B + 1) * 4; }
  static size_t ws_bytes(int B) {
    return align256((size_t)(B + 1) * 4) + align256((size_t)kSlots * kRows * 8) + (size_t)kSlots * kRows * D * 4;
  }
  static size_t align256(size_t x) { return (x + 255) / 256 * 256; }
};

// The keys of a sequence that its rows see, as units: first those that hold sinks, then
// those that the windows reach.
struct SeqUnits {
  int len, n_sink, lo, n;
  __device__ __forceinline__ SeqUnits(const DecodeParams& p, int length) {
    const long long cap = (long long)p.max_pages * kTile;
    len = length < 0 ? 0 : length > cap ? (int)cap : length;
    lo = n_sink = n = 0;
    if (len == 0) return;
    if (p.window) {
      const int first = max(0, len - p.Nq);  // the first row's position
      lo = max(0, first - p.window + 1) / kUnit;
      n_sink = min((p.sinks + kUnit - 1) / kUnit, lo);
    }
    n = n_sink + (len + kUnit - 1) / kUnit - lo;
  }
  __device__ __forceinline__ int key(int u) const { return (u < n_sink ? u : lo + u - n_sink) * kUnit; }
};

// The list of units: sequence, then head, then row block, then the item's units in order.
struct Item {
  int b, h, rb;
  long long first, end;  // the item's units in the list
};
__device__ __forceinline__ long long warp_first(long long total, int w, int nwarps) { return total * w / nwarps; }
__device__ __forceinline__ Item find_item(const int* pref, int B, int heads_rb, int nrb, long long x) {
  const int y = (int)(x / heads_rb);
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pref[mid] <= y)
      lo = mid;
    else
      hi = mid;
  }
  Item it;
  it.b = lo;
  const int n = pref[lo + 1] - pref[lo];
  const long long base = (long long)pref[lo] * heads_rb;
  const int k = (int)((x - base) / n);
  it.h = k / nrb;
  it.rb = k % nrb;
  it.first = base + (long long)k * n;
  it.end = it.first + n;
  return it;
}

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Eight E2M1 codes -> four FP16 pairs.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t* h) {
  asm("{\n.reg .b8 b0, b1, b2, b3;\n"
      "mov.b32 {b0, b1, b2, b3}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2(uint32_t w) {  // two scale codes -> an FP16 pair
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

template <bool F16>
__device__ __forceinline__ void write_row(const DecodeParams& p, int D, int b, int h, int r, int ch, float v) {
  const int G = p.Hq / p.Hkv;
  const size_t row = ((size_t)b * p.Hq + h * G + r % G) * p.Nq + r / G;
  p.out[row * D + ch] = (uint16_t)pack2<F16>(v, 0.f);
}

template <int D, int NT, bool F16>
__global__ void __launch_bounds__(DecCfg<D, NT>::W * 32, 1) decode_kernel(const DecodeParams p) {
  using C = DecCfg<D, NT>;
  constexpr int W = C::W, kRows = C::kRows;
  constexpr int kHalves = D == 256 ? 2 : 1;      // 128-channel halves of a K row
  constexpr int kSteps = D / 16 / kHalves;       // products of 16 channels per half
  constexpr int kTiles = D / 16;                 // 16-channel tiles of V
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int ring = p.nstages * W * C::kUnitBytes > C::kMergeBytes ? p.nstages * W * C::kUnitBytes : C::kMergeBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + ring) + warp * C::kMaxStages;
  int* abort_flag = reinterpret_cast<int*>(smem + ring + W * C::kMaxStages * 8);
  int* pref = reinterpret_cast<int*>(smem + ring + C::kBarBytes);
  const uint32_t bar0 = smem_u32(bars), stage0 = smem_u32(smem) + warp * p.nstages * C::kUnitBytes;

  if (lane < C::kMaxStages) mbar_init(bar0 + 8 * lane, 1);
  if (tid == 0) *abort_flag = 0;
  fence_mbar_init();

  // ---- units before each sequence: every CTA scans the lengths for itself
  {
    __shared__ int wsum[W];
    __shared__ int carry;
    if (tid == 0) carry = 0;
    __syncthreads();
    for (int b0 = 0; b0 < p.B; b0 += W * 32) {
      const int b = b0 + tid;
      int n = 0;
      if (b < p.B) {
        const int len = p.lens[b];
        const SeqUnits su(p, len);
        n = su.n;
        if (su.len != len && blockIdx.x == 0 && p.err) atomicCAS(p.err, 0, APA_DEVERR_BOUNDS);
      }
      int x = n;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, s);
        if (lane >= s) x += y;
      }
      if (lane == 31) wsum[warp] = x;
      __syncthreads();
      int before = carry;
      for (int k = 0; k < warp; ++k) before += wsum[k];
      if (b < p.B) pref[b] = before + x - n;
      __syncthreads();
      if (tid == W * 32 - 1) carry = before + x;
      __syncthreads();
    }
    if (tid == 0) pref[p.B] = carry;
    __syncthreads();
    if (blockIdx.x == 0)
      for (int b = tid; b <= p.B; b += W * 32) p.pref[b] = pref[b];
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int G = p.Hq / p.Hkv, R = G * p.Nq, nrb = (R + kRows - 1) / kRows, heads_rb = p.Hkv * nrb;
  const long long total = (long long)pref[p.B] * heads_rb;
  const int nwarps = gridDim.x * W, gw = blockIdx.x * W + warp;
  const long long x0 = warp_first(total, gw, nwarps), x1 = warp_first(total, gw + 1, nwarps);
  const long long c0 = warp_first(total, blockIdx.x * W, nwarps), c1 = warp_first(total, (blockIdx.x + 1) * W, nwarps);
  // one item for the whole CTA, in more than one warp: the warps are joined here
  bool alone = c1 - c0 > 1 && x1 - x0 < c1 - c0;
  if (alone) alone = find_item(pref, p.B, heads_rb, nrb, c0).end >= c1;
  const bool joined = __syncthreads_and(alone);

  bool ok = true;
  float o[kTiles][NT][4];
  float m[NT][2], l[NT][2];

  if (x1 > x0) {
    // ---- producer cursor: unit px of the list goes into stage ps
    Item pit = find_item(pref, p.B, heads_rb, nrb, x0);
    SeqUnits psu(p, p.lens[pit.b]);
    long long px = x0;
    int ps = 0, tbase = -64, tid_page = 0;  // this lane's entry of the 32 table entries from tbase
    auto issue = [&]() {
      if (px >= pit.end) {
        pit = find_item(pref, p.B, heads_rb, nrb, px);
        psu = SeqUnits(p, p.lens[pit.b]);
        tbase = -64;
      }
      const int key = psu.key((int)(px - pit.first)), e = key / kTile;
      if (e < tbase || e >= tbase + 32) {
        tbase = e;
        const int last = (psu.len - 1) / kTile;
        tid_page = e + lane <= last ? p.table[(size_t)pit.b * p.max_pages + e + lane] : 0;
        if (tid_page < 0 || tid_page >= p.num_pages) {
          // reported only for entries of visible keys: those that are really used, below
          tid_page = -1;
        }
      }
      int page = __shfl_sync(0xffffffffu, tid_page, e - tbase);
      if (lane == 0) {
        if (page < 0) {
          if (p.err) atomicCAS(p.err, 0, APA_DEVERR_BOUNDS);
          page = 0;
        }
        const uint8_t* src = p.pages + ((size_t)page * p.Hkv + pit.h) * page_head_bytes(D) +
                             (key % kTile / kUnit) * C::kUnitBytes;
        mbar_arrive_expect_tx(bar0 + 8 * ps, C::kUnitBytes);
        bulk_g2s(stage0 + ps * C::kUnitBytes, src, C::kUnitBytes, bar0 + 8 * ps);
      }
      ++px;
      ps = ps + 1 == p.nstages ? 0 : ps + 1;
    };
    for (int i = 0; i < p.nstages && px < x1; ++i) issue();

    long long x = x0;
    int st = 0;
    uint32_t parity = 0;
    while (x < x1 && ok) {
      // ---- one segment: the units of one item that are this warp's
      const Item it = find_item(pref, p.B, heads_rb, nrb, x);
      const SeqUnits su(p, p.lens[it.b]);
      const long long seg_end = min(it.end, x1);
      const int r0 = it.rb * kRows;

      // Q rows as the B operand: lane (g, c) has row 8 nt + g, channels 128 hf + (D/4 or 32) c + 4 s ..
      uint32_t qf[NT][kHalves][kSteps][2];
      float rf[NT][2];  // score factor of rows 2c, 2c + 1: the power of two back, and k_scale log2(e) / sqrt(d)
      int pos[NT][2];   // their positions
      const float sc = p.k_scale[it.h] * kLog2e * rsqrtf((float)D);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = r0 + 8 * nt + g;
        uint2 raw[kHalves][kSteps];
        float amax = 0.f;
        const uint16_t* src =
            p.q + it.b * p.qs_b + (long long)(it.h * G + r % G) * p.qs_h + (long long)(r / G) * p.qs_r;
#pragma unroll
        for (int hf = 0; hf < kHalves; ++hf)
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            raw[hf][s] = r < R ? *reinterpret_cast<const uint2*>(src + 128 * hf + c * (4 * kSteps) + 4 * s)
                               : make_uint2(0u, 0u);
            const float2 u = unpack2<F16>(raw[hf][s].x), v = unpack2<F16>(raw[hf][s].y);
            amax = fmaxf(amax, fmaxf(fmaxf(fabsf(u.x), fabsf(u.y)), fmaxf(fabsf(v.x), fabsf(v.y))));
          }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^e <= amax < 2^(e+1) becomes 2^14 .. 2^15: e clamped so that both factors are normal numbers
        int e = (int)((__float_as_uint(amax) >> 23) & 255) - 127;
        e = max(-110, min(126, e));
        const float up = __uint_as_float((uint32_t)(127 + 14 - max(e, -100)) << 23);
        const float down = __uint_as_float((uint32_t)(127 - 14 + max(e, -100)) << 23);
#pragma unroll
        for (int hf = 0; hf < kHalves; ++hf)
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            const float2 u = unpack2<F16>(raw[hf][s].x), v = unpack2<F16>(raw[hf][s].y);
            qf[nt][hf][s][0] = pack2<true>(u.x * up, u.y * up);
            qf[nt][hf][s][1] = pack2<true>(v.x * up, v.y * up);
          }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          rf[nt][k] = __shfl_sync(0xffffffffu, down, (2 * c + k) * 4) * sc;
          const int rr = r0 + 8 * nt + 2 * c + k;
          pos[nt][k] = su.len - p.Nq + (rr < R ? rr / G : p.Nq - 1);
          m[nt][k] = -INFINITY;
          l[nt][k] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[t][nt][k] = 0.f;
      }
      const int pmin = su.len - p.Nq + r0 / G;              // positions of the block's first row
      const int pmax = su.len - p.Nq + min(r0 + kRows - 1, R - 1) / G;  // and of its last

      for (; x < seg_end; ++x) {
        if (!__all_sync(0xffffffffu, mbar_test_wait(bar0 + 8 * st, parity))) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar0 + 8 * st, parity, abort_flag, p.err));
          if (!ok) break;
        }
        const uint32_t unit = stage0 + st * C::kUnitBytes;
        const int j0 = su.key((int)(x - it.first));
        float s[2][NT][4];
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[mb][nt][k] = 0.f;
          // rows r = g and g + 8 of the product are keys 4 (g/2) + g%2 and that + 2, so that
          // a lane's four keys of V^T below are neighbours
          const uint32_t blk = unit + mb * blk_bytes(D);
          const int kg = 4 * (g >> 1) + (g & 1);
#pragma unroll
          for (int hf = 0; hf < kHalves; ++hf) {
            uint32_t wa[4], wb[4], sa, sb;
            const uint32_t ka = blk + kg * (D / 2) + 64 * hf + c * (2 * kSteps);
            if constexpr (kSteps == 8) {
              const uint4 a = lds128(ka), b = lds128(ka + D);
              wa[0] = a.x, wa[1] = a.y, wa[2] = a.z, wa[3] = a.w;
              wb[0] = b.x, wb[1] = b.y, wb[2] = b.z, wb[3] = b.w;
              const uint32_t sp = blk + blk_ks(D) + kg * (D / 16) + 8 * hf + 2 * c;
              sa = e4m3x2(lds16(sp));
              sb = e4m3x2(lds16(sp + 2 * (D / 16)));
            } else {
              const uint2 a = lds64(ka), b = lds64(ka + D);
              wa[0] = a.x, wa[1] = a.y, wb[0] = b.x, wb[1] = b.y;
              const uint32_t sp = blk + blk_ks(D) + kg * (D / 16) + c;
              sa = e4m3x2(lds8(sp));
              sb = e4m3x2(lds8(sp + 2 * (D / 16)));
            }
#pragma unroll
            for (int w = 0; w < kSteps / 2; ++w) {
              // a lane's words 0, 1 (16 codes) share its first scale, words 2, 3 the second
              const uint32_t fa = __byte_perm(sa, sa, w < 2 ? 0x1010 : 0x3232);
              const uint32_t fb = __byte_perm(sb, sb, w < 2 ? 0x1010 : 0x3232);
              uint32_t ha[4], hb[4];
              e2m1x8(wa[w], ha);
              e2m1x8(wb[w], hb);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                ha[k] = hmul2(ha[k], fa);
                hb[k] = hmul2(hb[k], fb);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_f16(s[mb][nt], ha[0], hb[0], ha[1], hb[1], qf[nt][hf][2 * w][0], qf[nt][hf][2 * w][1]);
                mma_f16(s[mb][nt], ha[2], hb[2], ha[3], hb[3], qf[nt][hf][2 * w + 1][0], qf[nt][hf][2 * w + 1][1]);
              }
            }
          }
        }
        // ---- softmax: s[mb][nt] = keys kg (0, 1) and kg + 2 (2, 3) of block mb, rows 2c and 2c + 1
        const bool edge = j0 + kUnit - 1 > pmin || (p.window && j0 <= pmax - p.window && j0 + kUnit > p.sinks);
        bool lift = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int mb = 0; mb < 2; ++mb)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float y = s[mb][nt][k] * rf[nt][k & 1];
              if (edge) {
                const int j = j0 + 16 * mb + 4 * (g >> 1) + (g & 1) + (k & 2), pr = pos[nt][k & 1];
                if (j > pr || (p.window && j <= pr - p.window && j >= p.sinks)) y = -INFINITY;
              }
              s[mb][nt][k] = y;
              lift |= y > m[nt][k & 1] + kTauDec;
            }
        if (__any_sync(0xffffffffu, lift)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float y = fmaxf(fmaxf(s[0][nt][k], s[0][nt][k + 2]), fmaxf(s[1][nt][k], s[1][nt][k + 2]));
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
              if (y > m[nt][k]) {
                const float f = ex2_approx(m[nt][k] - y);  // 0 for the first
                m[nt][k] = y;
                l[nt][k] *= f;
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                  o[t][nt][k] *= f;
                  o[t][nt][k + 2] *= f;
                }
              }
            }
        }
        uint32_t pf[2][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // a row without a visible key yet has m = -inf and scores -inf: its weights are 0
          const float b0 = m[nt][0] == -INFINITY ? 0.f : kLift - m[nt][0];
          const float b1 = m[nt][1] == -INFINITY ? 0.f : kLift - m[nt][1];
#pragma unroll
          for (int mb = 0; mb < 2; ++mb) {
            const float p0 = ex2_approx(s[mb][nt][0] + b0), p1 = ex2_approx(s[mb][nt][1] + b1);
            const float p2 = ex2_approx(s[mb][nt][2] + b0), p3 = ex2_approx(s[mb][nt][3] + b1);
            l[nt][0] += p0 + p2;
            l[nt][1] += p1 + p3;
            pf[mb][nt][0] = transpose8(pack2<true>(p0, p1));
            pf[mb][nt][1] = transpose8(pack2<true>(p2, p3));
          }
        }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
          const uint32_t blk = unit + mb * blk_bytes(D);
          // keys past the end: whatever scales the page holds there (NaN too) count as 0
          const int left = su.len - (j0 + 16 * mb + 4 * c);
          const uint32_t keep = left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
#pragma unroll
          for (int tq = 0; tq < kTiles / 4; ++tq) {
            const uint4 vw = lds128(blk + blk_v(D) + 512 * tq + 16 * lane);
            const uint4 vs = lds128(blk + blk_vs(D) + 4 * (c * kTiles + 4 * tq));
            const uint32_t w4[4] = {vw.x, vw.y, vw.z, vw.w}, s4[4] = {vs.x, vs.y, vs.z, vs.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t h[4];
              e2m1x8(w4[k], h);  // h[j]: key 4c + j, channels g (low) and g + 8
              const uint32_t sw = s4[k] & keep, f0 = e4m3x2(sw & 0xFFFFu), f1 = e4m3x2(sw >> 16);
              const uint32_t a0 = hmul2(__byte_perm(h[0], h[1], 0x5410), f0);
              const uint32_t a1 = hmul2(__byte_perm(h[0], h[1], 0x7632), f0);
              const uint32_t a2 = hmul2(__byte_perm(h[2], h[3], 0x5410), f1);
              const uint32_t a3 = hmul2(__byte_perm(h[2], h[3], 0x7632), f1);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(o[4 * tq + k][nt], a0, a1, a2, a3, pf[mb][nt][0], pf[mb][nt][1]);
            }
          }
        }
        st = st + 1 == p.nstages ? (parity ^= 1, 0) : st + 1;
        __syncwarp();
        if (px < x1) issue();
      }
      if (!ok) break;

      // ---- the segment's state: l over the lanes that share the rows
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], d);
      if (joined) break;  // (its only segment)
      const long long a = x0;
      if (it.first >= a && it.end <= x1) {
        const float vsc = p.v_scale[it.h];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int r = r0 + 8 * nt + 2 * c + k;
            if (r >= R) continue;
            const float inv = l[nt][k] == 0.f ? 0.f : vsc / l[nt][k];
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
              write_row<F16>(p, D, it.b, it.h, r, 16 * t + g, o[t][nt][k] * inv);
              write_row<F16>(p, D, it.b, it.h, r, 16 * t + 8 + g, o[t][nt][k + 2] * inv);
            }
            if (g == 0 && p.lse)
              p.lse[((size_t)it.b * p.Hq + it.h * G + r % G) * p.Nq + r / G] =
                  l[nt][k] == 0.f ? -INFINITY : kLn2 * (m[nt][k] - kLift + log2f(l[nt][k]));
          }
      } else {
        // slot 2 gw: the warp's last (or only) item; 2 gw + 1: one that began before and ends here
        const size_t slot = 2 * (size_t)gw + (it.end < x1 ? 1 : 0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const size_t row = slot * kRows + 8 * nt + 2 * c + k;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
              p.part_o[row * D + 16 * t + g] = o[t][nt][k];
              p.part_o[row * D + 16 * t + 8 + g] = o[t][nt][k + 2];
            }
            if (g == 0) p.part_ml[row] = make_float2(m[nt][k], l[nt][k]);
          }
      }
    }
    if (!ok) {
      // a wait gave up: the copies in flight land before the CTA ends (waited with a limit again)
      const unsigned long long t0 = clock64();
      for (long long y = x; y < px; ++y) {
        while (!mbar_test_wait(bar0 + 8 * st, parity) && clock64() - t0 < APA_WAIT_LIMIT_CYCLES) {
        }
        st = st + 1 == p.nstages ? (parity ^= 1, 0) : st + 1;
      }
    }
  }

  if (joined) {
    // ---- the CTA's warps, all on one item: joined in order through shared memory
    if (!__syncthreads_and(ok)) return;
    float* mo = reinterpret_cast<float*>(smem);                              // [W][rows][D]
    float2* mml = reinterpret_cast<float2*>(smem + W * kRows * D * 4);       // [W][rows]
    const bool has = x1 > x0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = warp * kRows + 8 * nt + 2 * c + k;
        if (has) {
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            mo[row * D + 16 * t + g] = o[t][nt][k];
            mo[row * D + 16 * t + 8 + g] = o[t][nt][k + 2];
          }
        }
        if (g == 0) mml[row] = has ? make_float2(m[nt][k], l[nt][k]) : make_float2(-INFINITY, 0.f);
      }
    __syncthreads();
    const Item it = find_item(pref, p.B, heads_rb, nrb, c0);
    const bool whole = it.first == c0 && it.end == c1;
    const int r0 = it.rb * kRows;
    const float vsc = p.v_scale[it.h];
    for (int i = tid; i < kRows * D; i += W * 32) {
      const int row = i / D, ch = i % D, r = r0 + row;
      float M = -INFINITY, L = 0.f, acc = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, mml[w * kRows + row].x);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float2 ml = mml[w * kRows + row];
        if (ml.y == 0.f) continue;
        const float f = ex2_approx(ml.x - M);
        L = fmaf(f, ml.y, L);
        acc = fmaf(f, mo[(w * kRows + row) * D + ch], acc);
      }
      if (whole) {
        if (r >= R) continue;
        write_row<F16>(p, D, it.b, it.h, r, ch, L == 0.f ? 0.f : acc * (vsc / L));
        if (ch == 0 && p.lse)
          p.lse[((size_t)it.b * p.Hq + it.h * G + r % G) * p.Nq + r / G] =
              L == 0.f ? -INFINITY : kLn2 * (M - kLift + log2f(L));
      } else {  // in the slot of the CTA's first warp with units
        const size_t prow = 2 * (((c0 + 1) * nwarps - 1) / total) * kRows + row;
        p.part_o[prow * D + ch] = acc;
        if (ch == 0) p.part_ml[prow] = make_float2(M, L);
      }
    }
  }
}

// Joins the parts of the items that the first kernel left in more than one: one CTA per
// query row, a thread per channel, the parts in list order.  Also writes the rows of
// sequences without keys.
constexpr int kPartChunk = 256;
template <int D, int NT, bool F16>
__global__ void __launch_bounds__(D) join_kernel(const DecodeParams p) {
  using C = DecCfg<D, NT>;
  constexpr int W = C::W, kRows = C::kRows;
  __shared__ int s_slot[kPartChunk];
  __shared__ float s_f[kPartChunk], s_l[kPartChunk];
  __shared__ float red[D / 32];
  const int G = p.Hq / p.Hkv, R = G * p.Nq, nrb = (R + kRows - 1) / kRows, heads_rb = p.Hkv * nrb;
  const int r = blockIdx.x % R, bh = blockIdx.x / R, h = bh % p.Hkv, b = bh / p.Hkv;
  const int rb = r / kRows, row = r % kRows, tid = threadIdx.x;
  const size_t orow = ((size_t)b * p.Hq + h * G + r % G) * p.Nq + r / G;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = p.pref[b + 1] - p.pref[b];
  if (n == 0) {
    p.out[orow * D + tid] = 0;
    if (tid == 0 && p.lse) p.lse[orow] = -INFINITY;
    return;
  }
  const long long total = (long long)p.pref[p.B] * heads_rb;
  const int nwarps = kCtas * W;
  const long long u0 = (long long)p.pref[b] * heads_rb + (long long)(h * nrb + rb) * n, u1 = u0 + n;
  auto warp_of = [&](long long x) { return (int)(((x + 1) * nwarps - 1) / total); };
  const int w0 = warp_of(u0), w1 = warp_of(u1 - 1);
  if (w0 == w1) return;  // one warp had all of it
  const int ca = w0 / W, cb = w1 / W;
  if (ca == cb && warp_first(total, ca * W, nwarps) == u0 && warp_first(total, (ca + 1) * W, nwarps) == u1)
    return;  // one CTA had nothing else
  // candidates: the slots of warps w0 .. w1 in order; the ones in use are kept
  float M = -INFINITY, L = 0.f, acc = 0.f;
  for (int wa = w0; wa <= w1;) {
    // a chunk of the candidates: thread i looks at warp wa + i
    const int count = min(w1 - wa + 1, kPartChunk);
    __syncthreads();
    float mx = -INFINITY;
    for (int i = tid; i < count; i += D) {
      const int w = wa + i, cta = w / W;
      const long long a = warp_first(total, w, nwarps), e = warp_first(total, w + 1, nwarps);
      const long long a0 = warp_first(total, cta * W, nwarps), e0 = warp_first(total, (cta + 1) * W, nwarps);
      int slot = -1;
      if (a0 >= u0 && e0 <= u1) {
        // a CTA with this item alone: joined in the slot of its first warp with units
        const int wf = e0 > a0 ? warp_of(a0) : -1;
        if (w == wf) slot = 2 * w;
      } else if (e > a) {
        slot = 2 * w + (a >= u0 && e > u1 ? 1 : 0);
      }
      float2 ml = make_float2(-INFINITY, 0.f);
      if (slot >= 0) ml = p.part_ml[(size_t)slot * kRows + row];
      s_slot[i] = ml.y == 0.f ? -1 : slot;  // (a NaN sum goes on to the output)
      s_f[i] = ml.x;
      s_l[i] = ml.y;
      mx = fmaxf(mx, ml.x);
    }
    // the chunk's maximum, then the weights
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    float m2 = M;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) m2 = fmaxf(m2, red[k]);
    const float fo = M == -INFINITY ? 1.f : ex2_approx(M - m2);  // (nothing summed yet: 0, or NaN)
    acc *= fo;
    L *= fo;
    M = m2;
    for (int i = tid; i < count; i += D) s_f[i] = ex2_approx(s_f[i] - M);
    __syncthreads();
#pragma unroll 8
    for (int i = 0; i < count; ++i) {
      if (s_slot[i] < 0) continue;
      acc = fmaf(s_f[i], p.part_o[((size_t)s_slot[i] * kRows + row) * D + tid], acc);
      L = fmaf(s_f[i], s_l[i], L);
    }
    wa += count;
  }
  p.out[orow * D + tid] = (uint16_t)pack2<F16>(L == 0.f ? 0.f : acc * (p.v_scale[h] / L), 0.f);
  if (tid == 0 && p.lse) p.lse[orow] = L == 0.f ? -INFINITY : kLn2 * (M - kLift + log2f(L));
}

template <int D, int NT, bool F16>
cudaError_t launch_decode(DecodeParams prm, void* ws, cudaStream_t stream) {
  using C = DecCfg<D, NT>;
  uint8_t* w = static_cast<uint8_t*>(ws);
  prm.pref = (int*)w;
  w += C::align256((size_t)(prm.B + 1) * 4);
  prm.part_ml = (float2*)w;
  w += C::align256((size_t)C::kSlots * C::kRows * 8);
  prm.part_o = (float*)w;
  prm.nstages = C::stages(prm.B);
  cudaError_t e;
  const int smem = C::smem(prm.B);
  if ((e = cudaFuncSetAttribute(decode_kernel<D, NT, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))) return e;
  decode_kernel<D, NT, F16><<<kCtas, C::W * 32, smem, stream>>>(prm);
  if ((e = cudaGetLastError())) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(prm.B * prm.Hq * prm.Nq);
  cfg.blockDim = dim3(D);
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D, NT, F16>, prm);
}

// Rows per block: as few n = 8 tiles as hold all G * Nq rows, up to what the registers
// hold (32 rows at d <= 128, 16 at d = 256); more rows go in several blocks, each of
// which reads the keys again (through L2).
int row_tiles(int d, int rows) {
  if (rows <= 8) return 1;
  if (rows <= 16 || d == 256) return 2;
  return 4;
}

bool bad_heads(int B, int Hq, int Hkv, int Nq) {
  return B < 1 || B > kMaxSeqs || Hq < 1 || Hkv < 1 || Hq % Hkv || Hkv > (1 << 16) || Nq < 1 ||
         (long long)(Hq / Hkv) * Nq > (1 << 20) || (long long)B * Hq * Nq > 0x7FFFFFFF;
}

}  // namespace
}  // namespace apa

using namespace apa;

extern "C" {

size_t apa_attention_cache_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d) {
  if (bad_heads(B, Hq, Hkv, Nq)) return 0;
  const int nt = row_tiles(d, Hq / Hkv * Nq);
  switch (d) {
    case 64: return nt == 1 ? DecCfg<64, 1>::ws_bytes(B) : nt == 2 ? DecCfg<64, 2>::ws_bytes(B) : DecCfg<64, 4>::ws_bytes(B);
    case 128:
      return nt == 1 ? DecCfg<128, 1>::ws_bytes(B) : nt == 2 ? DecCfg<128, 2>::ws_bytes(B) : DecCfg<128, 4>::ws_bytes(B);
    case 256: return nt == 1 ? DecCfg<256, 1>::ws_bytes(B) : DecCfg<256, 2>::ws_bytes(B);
  }
  return 0;
}

int apa_attention_cache(const void* q, int dtype, long long q_batch_stride, long long q_head_stride,
                        long long q_row_stride, const uint8_t* pages, int num_pages, const int32_t* block_table,
                        int max_pages, const int32_t* lens, const float* k_scale, const float* v_scale, int B, int Hq,
                        int Hkv, int Nq, int d, int window, int sinks, void* out, float* lse, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
  if (!q || !pages || !block_table || !lens || !k_scale || !v_scale || !out) return APA_ERR_NULL;
  if (bad_heads(B, Hq, Hkv, Nq) || num_pages < 1 || num_pages >= (1 << 25) || max_pages < 1 ||
      (long long)B * max_pages >= (1 << 29) || max_pages >= (1 << 25))
    return APA_ERR_SHAPE;
  if (d != 64 && d != 128 && d != 256) return APA_ERR_HEAD_DIM;
  if (dtype != APA_DTYPE_BF16 && dtype != APA_DTYPE_F16) return APA_ERR_DTYPE;
  if (window < 0 || sinks < 0) return APA_ERR_WINDOW;
  if ((((uintptr_t)q | (uintptr_t)pages | (uintptr_t)out) & 15) || ((q_batch_stride | q_head_stride | q_row_stride) & 7))
    return APA_ERR_ALIGN;
  const size_t need = apa_attention_cache_workspace_bytes(B, Hq, Hkv, Nq, d);
  void* ws = workspace;
  if (ws && (workspace_bytes < need || ((uintptr_t)ws & 255))) return APA_ERR_NOMEM;
  // (the kernels' index arithmetic stays within 32 bits: no position exceeds 64 * max_pages)
  const int most = max_pages * kTile;
  if (window > most) window = 0;
  if (sinks > most) sinks = most;
  if (!ws && cudaMallocAsync(&ws, need, stream) != cudaSuccess) return APA_ERR_NOMEM;
  DecodeParams prm{};
  prm.q = (const uint16_t*)q;
  prm.qs_b = q_batch_stride;
  prm.qs_h = q_head_stride;
  prm.qs_r = q_row_stride;
  prm.pages = pages;
  prm.num_pages = num_pages;
  prm.table = block_table;
  prm.max_pages = max_pages;
  prm.lens = lens;
  prm.k_scale = k_scale;
  prm.v_scale = v_scale;
  prm.B = B;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.Nq = Nq;
  prm.window = window;
  prm.sinks = sinks;
  prm.out = (uint16_t*)out;
  prm.lse = lse;
  prm.err = device_error_word();
  const bool f16 = dtype == APA_DTYPE_F16;
  const int nt = row_tiles(d, Hq / Hkv * Nq);
  auto go = [&](auto D_, auto NT_) {
    constexpr int D = decltype(D_)::value, NT = decltype(NT_)::value;
    return f16 ? launch_decode<D, NT, true>(prm, ws, stream) : launch_decode<D, NT, false>(prm, ws, stream);
  };
  using I64 = std::integral_constant<int, 64>;
  using I128 = std::integral_constant<int, 128>;
  using I256 = std::integral_constant<int, 256>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I4 = std::integral_constant<int, 4>;
  cudaError_t e = cudaErrorInvalidValue;
  switch (d) {
    case 64: e = nt == 1 ? go(I64{}, I1{}) : nt == 2 ? go(I64{}, I2{}) : go(I64{}, I4{}); break;
    case 128: e = nt == 1 ? go(I128{}, I1{}) : nt == 2 ? go(I128{}, I2{}) : go(I128{}, I4{}); break;
    case 256: e = nt == 1 ? go(I256{}, I1{}) : go(I256{}, I2{}); break;
  }
  int st = e == cudaSuccess ? APA_OK : APA_ERR_CUDA;
  if (!workspace && cudaFreeAsync(ws, stream) != cudaSuccess && st == APA_OK) st = APA_ERR_CUDA;
  return st;
}

}  // extern "C"
