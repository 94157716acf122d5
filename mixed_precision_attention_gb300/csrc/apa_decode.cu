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
//   to 2^14 .. 2^16: its BF16 values are exact down to 2^-31 of the largest, those below
//   are off by 2^-39 of it at most.  P is rounded to FP16 (2^-11), lifted by 2^6 so that weights
//   down to 2^-30 of the row's largest keep a value; l sums the FP32 weights.
//
// Split: the units (32 keys of one KV head, one contiguous half page) of all sequences,
// heads and row blocks form one list, cut evenly over the CTAs, one per SM, and again
// over each CTA's warps, so lengths need not be alike and no length is read on the host.
// Every warp works for itself: it streams its units through a ring of its own with bulk
// copies (no barrier with other warps), keeps its own running maximum and sum, and moves
// the maximum only when a score exceeds it by 8 (log2 units).  An item (sequence, head,
// row block) that one warp holds entirely is written out at once; then the CTA joins its
// warps' parts of the others in order, and a second kernel those that span CTAs, so
// results do not depend on timing.
#include <atomic>
#include <cfloat>
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
  int nstages, ring_off;
  // workspace
  int* pref;        // [B + 1] units before each sequence (of one head and row block)
  float2* part_ml;  // [slots][rows] (m, l): slots 2 cta + 1 and 2 cta are the CTA's part of the item
  float* part_o;    // [slots][rows][d]      that ends in it, and of the one that goes on behind it;
                    // slot 2 kCtas + warp is a warp's part of an item that ends in it
};

// kRows rows share the keys: 8 per n = 8 tile, or 4 (kQuad), which then take a tile of
// V^T P^T twice (see there).
template <int D, int ROWS>
struct DecCfg {
  static constexpr int kRows = ROWS;
  static constexpr int NT = ROWS < 8 ? 1 : ROWS / 8;
  static constexpr bool kQuad = ROWS == 4;
  static constexpr int kAcc = kQuad ? D / 32 : D / 16;   // product tiles of O^T per n tile
  // Warps: what the registers of O and Q leave room for (16 rows at d = 64: 12 warps 37 us,
  // 16 warps 39; 8 rows at d = 128: 35 and 33); at d = 256 two stages must fit.
  static constexpr int W = D == 256 ? 8 : ROWS <= 8 ? 16 : D * ROWS <= 2048 ? 12 : 8;
  static constexpr int kUnitBytes = 36 * D;
  static constexpr int kScaleBytes = kQuad ? 8 * D : 4 * D;  // a unit's V scales as FP16 pairs, per warp
  // Q's fragments in shared memory, where registers are short (32 rows at d = 128: 93 us with
  // them in registers, spilling, and 70 so)
  static constexpr bool kQShared = D * ROWS >= 2048;
  static constexpr int kQBytes = kQShared ? NT * D * 16 : 0;  // per warp
  static constexpr int kMaxStages = 6;
  static constexpr int kStaticBytes = 1536;  // room for the kernel's static arrays
  static constexpr int kSlots = kCtas * (2 + W);
  static constexpr int kBarBytes = W * kMaxStages * 8 + 16;
  static constexpr int kPitch = D + (kQuad ? 8 : 4);  // floats per row of a state in shared memory: no bank twice
  static constexpr int kMergeBytes = W * kRows * (kPitch + 2) * 4;
  // Shared memory: the barriers, the warps' scales and Q, the units before each sequence, the
  // rings (the joined states take the place of all but the barriers at the end).
  static constexpr int kScaleOff = kBarBytes, kQOff = kScaleOff + W * kScaleBytes, kPrefOff = kQOff + W * kQBytes;
  static constexpr int ring_off(int B) { return kPrefOff + ((B + 1) * 4 + 15) / 16 * 16; }
  static constexpr int stages(int B) {
    const int n = (232448 - kStaticBytes - ring_off(B)) / (W * kUnitBytes);
    return n > kMaxStages ? kMaxStages : n;
  }
  static constexpr int smem(int B) {
    const int r = ring_off(B) + W * stages(B) * kUnitBytes, m = kBarBytes + kMergeBytes;
    return r > m ? r : m;
  }
  // (two stages or more, but for 16 rows at d = 256 from 2332 sequences on: one, without overlap)
  static constexpr bool kFits = stages(D * ROWS == 4096 ? 2331 : kMaxSeqs) >= 2 && stages(kMaxSeqs) >= 1 &&
                                smem(kMaxSeqs) <= 232448 - kStaticBytes;
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
};

// The list of units: sequence, then head, then row block, then the item's units in order.
struct Item {
  int b, h, rb;
  long long first, end;  // the item's units in the list
};
// x / n for x >= 0 below 2^63; nearly always a 32-bit division.
__device__ __forceinline__ long long quotient(long long x, int n) {
  if (((unsigned long long)x >> 32) == 0) return (unsigned)x / (unsigned)n;
  return x / n;
}
// n things in k nearly equal runs, the longer ones first.
struct Cut {
  long long q;
  int r;
  __device__ __forceinline__ Cut(long long n, int k) : q(quotient(n, k)) { r = (int)(n - q * k); }
  __device__ __forceinline__ long long first(int i) const { return q * i + min(i, r); }
  __device__ __forceinline__ int of(long long x) const {  // the run that holds x < n
    const long long y = r * (q + 1);
    if (x < y) return (int)(q < 0x7FFFFFFF ? quotient(x, (int)q + 1) : x / (q + 1));
    return r + (int)(q < 0x7FFFFFFF ? quotient(x - y, (int)q) : (x - y) / q);
  }
};
__device__ __forceinline__ Item find_item(const int* pref, int B, int heads_rb, int nrb, long long x) {
  const int y = (int)quotient(x, heads_rb);
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
  const int k = (int)quotient(x - base, n);
  it.h = k / nrb;
  it.rb = k % nrb;
  it.first = base + (long long)k * n;
  it.end = it.first + n;
  return it;
}

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
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
template <typename T>
__device__ __forceinline__ T lds(const uint8_t* p) {
  return *reinterpret_cast<const T*>(p);
}

// The channel of o[t][.][2 i + k] in lane (g, c), and the row of the block (of n tile nt).
template <bool QUAD>
__device__ __forceinline__ int channel_of(int t, int i, int g, int c) {
  return QUAD ? 32 * t + 16 * i + 8 * (c >> 1) + g : 16 * t + 8 * i + g;
}
template <bool QUAD>
__device__ __forceinline__ int row_of(int nt, int c, int k) {
  return QUAD ? (2 * c + k) & 3 : 8 * nt + 2 * c + k;
}

template <bool F16>
__device__ __forceinline__ void write_row(const DecodeParams& p, int D, int b, int h, int r, int ch, float v) {
  const int G = p.Hq / p.Hkv;
  const size_t row = ((size_t)b * p.Hq + h * G + r % G) * p.Nq + r / G;
  p.out[row * D + ch] = (uint16_t)pack2<F16>(v, 0.f);
}

// acc += f * (kVec floats at src)
template <int kVec>
__device__ __forceinline__ void add_vec(float* acc, float f, const float* src) {
  if constexpr (kVec == 4) {
    const float4 y = *reinterpret_cast<const float4*>(src);
    acc[0] = fmaf(f, y.x, acc[0]);
    acc[1] = fmaf(f, y.y, acc[1]);
    acc[2] = fmaf(f, y.z, acc[2]);
    acc[3] = fmaf(f, y.w, acc[3]);
  } else {
    const float2 y = *reinterpret_cast<const float2*>(src);
    acc[0] = fmaf(f, y.x, acc[0]);
    acc[1] = fmaf(f, y.y, acc[1]);
  }
}
// A joined row (a lane's channels in acc), written to out and lse.
template <bool F16, int kVec, int kVecs>
__device__ __forceinline__ void finish_row(const DecodeParams& p, int D, int b, int h, int r, int lane,
                                           const float (*acc)[kVec], float M, float L) {
  const int G = p.Hq / p.Hkv;
  const size_t row = ((size_t)b * p.Hq + h * G + r % G) * p.Nq + r / G;
  const float inv = L == 0.f ? 0.f : p.v_scale[h] / L;
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + row * D + (32 * v + lane) * kVec);
#pragma unroll
    for (int k = 0; k < kVec; k += 2) dst[k / 2] = pack2<F16>(acc[v][k] * inv, acc[v][k + 1] * inv);
  }
  if (lane == 0 && p.lse) p.lse[row] = L == 0.f ? -INFINITY : kLn2 * (M - kLift + log2f(L));
}

struct Seg {  // an item that a warp holds units of; counted from the CTA's first unit
  int first, end, b, h, rb;
};

template <int D, int ROWS, bool F16>
__global__ void __launch_bounds__(DecCfg<D, ROWS>::W * 32, 1) decode_kernel(const DecodeParams p) {
  using C = DecCfg<D, ROWS>;
  static_assert(C::kFits, "shared memory");
  constexpr int W = C::W, kRows = C::kRows, NT = C::NT, kAcc = C::kAcc;
  constexpr bool kQuad = C::kQuad;
  constexpr int kHalves = D == 256 ? 2 : 1;      // 128-channel halves of a K row
  constexpr int kSteps = D / 16 / kHalves;       // products of 16 channels per half
  constexpr int kTiles = D / 16;                 // 16-channel tiles of V
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem) + warp * C::kMaxStages;
  int* abort_flag = reinterpret_cast<int*>(smem + W * C::kMaxStages * 8);
  uint8_t* scales = smem + C::kScaleOff + warp * C::kScaleBytes;
  uint8_t* qsh = smem + C::kQOff + warp * C::kQBytes + 8 * lane;
  int* pref = reinterpret_cast<int*>(smem + C::kPrefOff);
  const int ring = p.ring_off + warp * p.nstages * C::kUnitBytes;
  const uint32_t bar0 = smem_u32(bars), stage0 = smem_u32(smem) + ring;

  if (lane < C::kMaxStages) mbar_init(bar0 + 8 * lane, 1);
  if (tid == 0) *abort_flag = 0;
  fence_mbar_init();

  __shared__ Seg seg[W][2];  // each warp's first and last item
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
  const Cut ctas(total, kCtas);
  const long long c0 = ctas.first(blockIdx.x);
  const int cta_count = (int)(ctas.first(blockIdx.x + 1) - c0);
  if (cta_count == 0) return;
  const Cut warps(cta_count, W);
  const int w0 = (int)warps.first(warp), count = (int)warps.first(warp + 1) - w0;
  const long long x0 = c0 + w0;

  bool ok = true, waiting = false;  // waiting: the last item is in o, m, l for the CTA to join
  // o[t][.][0 .. 1] and [2 .. 3]: the columns 2c, 2c + 1 of the rows g and g + 8 of product tile t
  // (channel_of, row_of)
  float o[kAcc][NT][4];
  float m[NT][2], l[NT][2];

  if (count > 0) {
    // Units are counted from the warp's first one, x0, from here on.
    // ---- producer cursor: unit px, of an item [pfirst, pend), goes into stage ps next
    struct Entered {
      int b, h, rb, len, lo, sink, first, end;  // lo: from a unit behind the sinks to its half page
    };
    int px = 0;
    Entered pi;
    const uint8_t* head;  // the KV head's part of page 0
    auto enter = [&](int x) {
      const Item it = find_item(pref, p.B, heads_rb, nrb, x0 + x);
      const SeqUnits su(p, p.lens[it.b]);
      return Entered{it.b, it.h, it.rb, su.len, su.lo - su.n_sink, su.n_sink, (int)(it.first - x0), (int)(it.end - x0)};
    };
    pi = enter(0);
    head = p.pages + (size_t)pi.h * page_head_bytes(D);
    int ps = 0, tbase = -64, entry = 0;  // entry: this lane's of the 32 table entries from tbase
    auto issue = [&]() {
      if (px == pi.end) {
        pi = enter(px);
        head = p.pages + (size_t)pi.h * page_head_bytes(D);
        tbase = -64;
      }
      const int u = px - pi.first, half = u < pi.sink ? u : u + pi.lo, e = half / 2;
      if ((unsigned)(e - tbase) >= 32u) {
        tbase = e;
        entry = e + lane <= (pi.len - 1) / kTile ? p.table[(size_t)pi.b * p.max_pages + e + lane] : 0;
      }
      int page = __shfl_sync(0xffffffffu, entry, e - tbase);
      if (lane == 0) {
        if ((unsigned)page >= (unsigned)p.num_pages) {  // reads page 0, and is reported
          if (p.err) atomicCAS(p.err, 0, APA_DEVERR_BOUNDS);
          page = 0;
        }
        mbar_arrive_expect_tx(bar0 + 8 * ps, C::kUnitBytes);
        bulk_g2s(stage0 + ps * C::kUnitBytes,
                 head + (size_t)page * p.Hkv * page_head_bytes(D) + (half & 1) * C::kUnitBytes, C::kUnitBytes,
                 bar0 + 8 * ps);
      }
      ++px;
      ps = ps + 1 == p.nstages ? 0 : ps + 1;
    };
    for (int i = 0; i < p.nstages && px < count; ++i) issue();

    int x = 0, st = 0;
    uint32_t parity = 0;
    while (x < count) {
      // ---- one segment: the units of one item that are this warp's
      const Entered it = x >= pi.first && x < pi.end ? pi : enter(x);
      const int len = it.len, sink = it.sink, lo = it.lo, r0 = it.rb * kRows, first = it.first;
      const int seg_end = min(it.end, count);
      if (lane == 0) {
        const Seg sg{w0 + it.first, w0 + it.end, it.b, it.h, it.rb};
        if (x == 0) seg[warp][0] = sg;
        seg[warp][1] = sg;
      }

      // Q rows as the B operand: lane (g, c) has row 8 nt + g, channels 128 hf + (D/4 or 32) c + 4 s ..
      uint32_t qf[C::kQShared ? 1 : NT][kHalves][kSteps][2];
      float rf[NT][2];  // score factor of rows 2c, 2c + 1: the power of two back, and k_scale log2(e) / sqrt(d)
      const float sc = p.k_scale[it.h] * kLog2e * rsqrtf((float)D);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = r0 + (kQuad ? g & 3 : 8 * nt + g);
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
            const uint32_t q0 = pack2<true>(u.x * up, u.y * up), q1 = pack2<true>(v.x * up, v.y * up);
            if constexpr (C::kQShared) {
              *reinterpret_cast<uint2*>(qsh + 256 * ((nt * kHalves + hf) * kSteps + s)) = make_uint2(q0, q1);
            } else {
              qf[nt][hf][s][0] = q0;
              qf[nt][hf][s][1] = q1;
            }
          }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // a positive finite number: a masked score is -inf times it, a key of zeros 0 times it (without a
          // value above 2^-100 in the row the product is 0 for k_scale < 1e-10; scores are below 2^35
          // here, so that at the smallest normal number they are all 0 to FP32)
          const float f = __shfl_sync(0xffffffffu, down, (kQuad ? (2 * c + k) & 3 : 2 * c + k) * 4) * sc;
          rf[nt][k] = f < FLT_MIN ? FLT_MIN : f > FLT_MAX ? FLT_MAX : f;
          m[nt][k] = -INFINITY;
          l[nt][k] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < kAcc; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[t][nt][k] = 0.f;
      }
      const int pmin = len - p.Nq + r0 / G;                             // positions of the block's first row
      const int pmax = len - p.Nq + min(r0 + kRows - 1, R - 1) / G;  // and of its last
      // the item's units from plain0 on, plain of them, hold only keys that some row sees; the others,
      // those of the sinks among them, are looked at key by key
      const int plain0 = p.window ? max(0, max(0, pmin - p.window + kUnit) / kUnit - lo) : 0;
      const unsigned plain = max(len / kUnit - lo - plain0, 0);

      for (; x < seg_end; ++x) {
        if (!__all_sync(0xffffffffu, mbar_test_wait(bar0 + 8 * st, parity))) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar0 + 8 * st, parity, abort_flag, p.err));
          if (!ok) break;
        }
        const uint8_t* unit = smem + ring + st * C::kUnitBytes;
        const int u = x - first, j0 = (u < sink ? u : u + lo) * kUnit;
        // ---- V's scales as FP16 pairs, converted once per warp (here, so that nothing below waits):
        // word i of a block holds those of keys 4 (i / kTiles) .. + 3 for tile i % kTiles.  Keys past
        // the end, and between the sinks and the first row's window, count as 0 whatever the page holds
        // there: a weight of 0 does not hide a NaN.
        const bool edge = (unsigned)(u - plain0) >= plain;
#pragma unroll
        for (int mb = 0; mb < 2; ++mb)
#pragma unroll
          for (int i = lane; i < 4 * kTiles; i += 32) {
            const int kc = i / kTiles, j = j0 + 16 * mb + 4 * kc;
            uint32_t w = lds<uint32_t>(unit + mb * blk_bytes(D) + blk_vs(D) + 4 * i);
            if (edge)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (j + k >= len || (p.window && j + k <= pmin - p.window && j + k >= p.sinks)) w &= ~(255u << (8 * k));
            const uint32_t f0 = e4m3x2(w & 0xFFFFu), f1 = e4m3x2(w >> 16);
            uint8_t* dst = scales + mb * (C::kScaleBytes / 2) + (kQuad ? 16 : 8) * (4 * (i % kTiles) + kc);
            if constexpr (kQuad)  // (s, s) of each key
              *reinterpret_cast<uint4*>(dst) =
                  make_uint4(__byte_perm(f0, 0, 0x1010), __byte_perm(f0, 0, 0x3232), __byte_perm(f1, 0, 0x1010),
                             __byte_perm(f1, 0, 0x3232));
            else  // of two keys
              *reinterpret_cast<uint2*>(dst) = make_uint2(f0, f1);
          }
        __syncwarp();
        // ---- S^T = K Q^T.  Rows g and g + 8 of the product are keys 4 (g/2) + g%2 and that + 2, so
        // that a lane's four keys of V^T below are neighbours.  Both blocks go side by side.
        float s[2][NT][4];
#pragma unroll
        for (int mb = 0; mb < 2; ++mb)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[mb][nt][k] = 0.f;
        const int kg = 4 * (g >> 1) + (g & 1);
#pragma unroll
        for (int hf = 0; hf < kHalves; ++hf) {
          uint32_t wk[2][2][4], sk[2][2];  // [block][key kg, kg + 2]
#pragma unroll
          for (int mb = 0; mb < 2; ++mb)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint8_t* blk = unit + mb * blk_bytes(D);
              const uint8_t* ka = blk + (kg + 2 * i) * (D / 2) + 64 * hf + c * (2 * kSteps);
              const uint8_t* sp = blk + blk_ks(D) + (kg + 2 * i) * (D / 16);
              if constexpr (kSteps == 8) {
                const uint4 a = lds<uint4>(ka);
                wk[mb][i][0] = a.x, wk[mb][i][1] = a.y, wk[mb][i][2] = a.z, wk[mb][i][3] = a.w;
                sk[mb][i] = e4m3x2(lds<uint16_t>(sp + 8 * hf + 2 * c));
              } else {
                const uint2 a = lds<uint2>(ka);
                wk[mb][i][0] = a.x, wk[mb][i][1] = a.y;
                sk[mb][i] = e4m3x2(lds<uint8_t>(sp + c));
              }
            }
#pragma unroll
          for (int w = 0; w < kSteps / 2; ++w) {
            auto q_at = [&](int nt, int i) -> uint2 {  // of product 2 w + i
              if constexpr (C::kQShared) return lds<uint2>(qsh + 256 * ((nt * kHalves + hf) * kSteps + 2 * w + i));
              return make_uint2(qf[C::kQShared ? 0 : nt][hf][2 * w + i][0], qf[C::kQShared ? 0 : nt][hf][2 * w + i][1]);
            };
#pragma unroll
            for (int mb = 0; mb < 2; ++mb) {
              // a lane's words 0, 1 (16 codes) share its first scale, words 2, 3 the second
              const uint32_t fa = __byte_perm(sk[mb][0], 0, w < 2 ? 0x1010 : 0x3232);
              const uint32_t fb = __byte_perm(sk[mb][1], 0, w < 2 ? 0x1010 : 0x3232);
              uint32_t ha[4], hb[4];
              e2m1x8(wk[mb][0][w], ha);
              e2m1x8(wk[mb][1][w], hb);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                ha[k] = hmul2(ha[k], fa);
                hb[k] = hmul2(hb[k], fb);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint2 q0 = q_at(nt, 0), q1 = q_at(nt, 1);
                mma_f16(s[mb][nt], ha[0], hb[0], ha[1], hb[1], q0.x, q0.y);
                mma_f16(s[mb][nt], ha[2], hb[2], ha[3], hb[3], q1.x, q1.y);
              }
            }
          }
        }
        // ---- softmax: s[mb][nt] = keys kg (0, 1) and kg + 2 (2, 3) of block mb, rows 2c and 2c + 1,
        // still without the row's factor rf
        if (j0 + kUnit - 1 > pmin || (p.window && j0 <= pmax - p.window && j0 + kUnit > p.sinks)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            for (int k = 0; k < 4; ++k) {
              const int rr = r0 + row_of<kQuad>(nt, c, k & 1), pr = rr < R ? len - p.Nq + rr / G : pmax;
#pragma unroll
              for (int mb = 0; mb < 2; ++mb) {
                const int j = j0 + 16 * mb + 4 * (g >> 1) + (g & 1) + (k & 2);
                if (j > pr || (p.window && j <= pr - p.window && j >= p.sinks)) s[mb][nt][k] = -INFINITY;
              }
            }
        }
        float top[NT][2];  // the largest of this lane's scores (rf > 0, so of the scaled ones too)
        bool lift = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            top[nt][k] = rf[nt][k] * fmaxf(max3(s[0][nt][k], s[0][nt][k + 2], s[1][nt][k]), s[1][nt][k + 2]);
            lift |= top[nt][k] > m[nt][k] + kTauDec;
          }
        if (__any_sync(0xffffffffu, lift)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float y = top[nt][k];
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
              if (y > m[nt][k]) {
                const float f = ex2_approx(m[nt][k] - y);  // 0 for the first
                m[nt][k] = y;
                l[nt][k] *= f;
#pragma unroll
                for (int t = 0; t < kAcc; ++t)
#pragma unroll
                  for (int i = 0; i < 2; ++i) o[t][nt][2 * i + k] *= f;
              }
            }
        }
        // P^T: pf[mb][nt] = the weights of row g for keys 4c, 4c + 1 and 4c + 2, 4c + 3
        uint32_t pf[2][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // a row without a visible key yet has m = -inf and scores -inf: its weights are 0
          const float b0 = m[nt][0] == -INFINITY ? 0.f : kLift - m[nt][0];
          const float b1 = m[nt][1] == -INFINITY ? 0.f : kLift - m[nt][1];
#pragma unroll
          for (int mb = 0; mb < 2; ++mb) {
            const float p0 = ex2_approx(fmaf(s[mb][nt][0], rf[nt][0], b0));
            const float p1 = ex2_approx(fmaf(s[mb][nt][1], rf[nt][1], b1));
            const float p2 = ex2_approx(fmaf(s[mb][nt][2], rf[nt][0], b0));
            const float p3 = ex2_approx(fmaf(s[mb][nt][3], rf[nt][1], b1));
            l[nt][0] += p0 + p2;
            l[nt][1] += p1 + p3;
            pf[mb][nt][0] = transpose8(pack2<true>(p0, p1));
            pf[mb][nt][1] = transpose8(pack2<true>(p2, p3));
          }
        }
        // ---- O^T += V^T P^T.  A code byte holds channels g and 8 + g of a tile for one key, a
        // word four keys.  The products sum over pairs of keys: the FP16 pairs of two keys are
        // permuted into rows g and 8 + g.  With up to four rows the pair goes in as it is, as two
        // steps of the summed axis, against P with zeros at every other step: (P, 0) in columns
        // 0 .. 3 gives the channels g, (0, P) in columns 4 .. 7 the channels 8 + g, and rows g and
        // g + 8 are tiles t and t + 1: as many products, and no permutes, of which the integer
        // pipe would be full.
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
          const uint8_t* blk = unit + mb * blk_bytes(D);
          const uint8_t* sc_mb = scales + mb * (C::kScaleBytes / 2);
          // (four rows) lanes g < 4 take (P, 0), the others (0, P), of keys 4c, 4c + 1 and 4c + 2, 4c + 3
          uint32_t pz[2][2];
          if constexpr (kQuad) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              pz[i][0] = __byte_perm(pf[mb][0][i], 0, g < 4 ? 0x4410 : 0x1044);
              pz[i][1] = __byte_perm(pf[mb][0][i], 0, g < 4 ? 0x4432 : 0x3244);
            }
          }
#pragma unroll
          for (int tq = 0; tq < kTiles / 4; ++tq) {
            const uint4 vw = lds<uint4>(blk + blk_v(D) + 512 * tq + 16 * lane);
            const uint32_t w4[4] = {vw.x, vw.y, vw.z, vw.w};
            if constexpr (kQuad) {
#pragma unroll
              for (int k = 0; k < 4; k += 2) {
                const int t = 4 * tq + k;
                const uint4 sa = lds<uint4>(sc_mb + 16 * (4 * t + c)), sb = lds<uint4>(sc_mb + 16 * (4 * t + 4 + c));
                uint32_t ha[4], hb[4];
                e2m1x8(w4[k], ha);  // [key 4c + i]
                e2m1x8(w4[k + 1], hb);
                ha[0] = hmul2(ha[0], sa.x), ha[1] = hmul2(ha[1], sa.y), ha[2] = hmul2(ha[2], sa.z), ha[3] = hmul2(ha[3], sa.w);
                hb[0] = hmul2(hb[0], sb.x), hb[1] = hmul2(hb[1], sb.y), hb[2] = hmul2(hb[2], sb.z), hb[3] = hmul2(hb[3], sb.w);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  mma_f16(o[t / 2][0], ha[2 * i], hb[2 * i], ha[2 * i + 1], hb[2 * i + 1], pz[i][0], pz[i][1]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int t = 4 * tq + k;
                const uint2 f = lds<uint2>(sc_mb + 8 * (4 * t + c));
                uint32_t h[4];
                e2m1x8(w4[k], h);  // [key 4c + i]
                const uint32_t a0 = hmul2(__byte_perm(h[0], h[1], 0x5410), f.x);
                const uint32_t a1 = hmul2(__byte_perm(h[0], h[1], 0x7632), f.x);
                const uint32_t a2 = hmul2(__byte_perm(h[2], h[3], 0x5410), f.y);
                const uint32_t a3 = hmul2(__byte_perm(h[2], h[3], 0x7632), f.y);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(o[t][nt], a0, a1, a2, a3, pf[mb][nt][0], pf[mb][nt][1]);
              }
            }
          }
        }
        st = st + 1 == p.nstages ? (parity ^= 1, 0) : st + 1;
        __syncwarp();
        if (px < count) issue();
      }
      if (!ok) break;

      // ---- the segment's state: l over the lanes that share the rows
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], d);
      waiting = false;
      if (first >= 0 && it.end <= count) {
        // the whole item
        const float vsc = p.v_scale[it.h];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int r = r0 + row_of<kQuad>(nt, c, k);
            if (r >= R) continue;
            const float inv = l[nt][k] == 0.f ? 0.f : vsc / l[nt][k];
#pragma unroll
            for (int t = 0; t < kAcc; ++t)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                write_row<F16>(p, D, it.b, it.h, r, channel_of<kQuad>(t, i, g, c), o[t][nt][2 * i + k] * inv);
            if (g == 0 && p.lse)
              p.lse[((size_t)it.b * p.Hq + it.h * G + r % G) * p.Nq + r / G] =
                  l[nt][k] == 0.f ? -INFINITY : kLn2 * (m[nt][k] - kLift + log2f(l[nt][k]));
          }
      } else if (x < count) {
        // one that began before this warp and ends in it, while the warp goes on to others
        const size_t slot = 2 * kCtas + (size_t)blockIdx.x * W + warp;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const size_t row = slot * kRows + row_of<kQuad>(nt, c, k);
#pragma unroll
            for (int t = 0; t < kAcc; ++t)
#pragma unroll
              for (int i = 0; i < 2; ++i) p.part_o[row * D + channel_of<kQuad>(t, i, g, c)] = o[t][nt][2 * i + k];
            if (g == 0) p.part_ml[row] = make_float2(m[nt][k], l[nt][k]);
          }
      } else {
        waiting = true;
      }
    }
    if (!ok) {
      // a wait gave up: the copies in flight land before the CTA ends (waited with a limit again)
      const unsigned long long t0 = clock64();
      for (; x < px; ++x) {
        while (!mbar_test_wait(bar0 + 8 * st, parity) && clock64() - t0 < APA_WAIT_LIMIT_CYCLES) {
        }
        st = st + 1 == p.nstages ? (parity ^= 1, 0) : st + 1;
      }
    }
  }

  // ---- the items that are in several warps, or go on in other CTAs: joined in order.  A warp's last
  // item is in shared memory (the rings are idle now), one that ended in it in the workspace.
  if (!__syncthreads_and(ok)) return;
  constexpr int kPitch = C::kPitch;
  float* mo = reinterpret_cast<float*>(smem + C::kBarBytes);                 // [W][rows][pitch]
  float2* mml = reinterpret_cast<float2*>(mo + W * kRows * kPitch);          // [W][rows]
  if (waiting) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = warp * kRows + row_of<kQuad>(nt, c, k);
#pragma unroll
        for (int t = 0; t < kAcc; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) mo[row * kPitch + channel_of<kQuad>(t, i, g, c)] = o[t][nt][2 * i + k];
        if (g == 0) mml[row] = make_float2(m[nt][k], l[nt][k]);
      }
  }
  __syncthreads();
  // lane 2 w: the item that ends in warp w after beginning before it; lane 2 w + 1: the one that
  // goes on behind the CTA from its last warp w.  Each (item, row) is one warp's to join.
  const int jw = lane >> 1;
  bool mine = false;
  Seg sg{};
  bool tail_in_ws = false;
  if (jw < W) {
    const int a = (int)warps.first(jw), e = (int)warps.first(jw + 1);
    if (e > a) {
      sg = seg[jw][lane & 1];
      mine = lane & 1 ? e == cta_count && sg.end > e : sg.end <= e && sg.first < a;
      tail_in_ws = !(lane & 1) && sg.end < e;
    }
  }
  const int from_ = mine ? warps.of(max(sg.first, 0)) : 0;
  const unsigned todo = __ballot_sync(0xffffffffu, mine);
  constexpr int kVec = D / 32 < 4 ? D / 32 : 4, kVecs = D / (32 * kVec);  // a lane's channels: kVecs vectors
  for (int task = warp; task < __popc(todo) * kRows; task += W) {
    const int row = task % kRows, src = __fns(todo, 0, task / kRows + 1), to = src >> 1;
    const int from = __shfl_sync(0xffffffffu, from_, src), first = __shfl_sync(0xffffffffu, sg.first, src);
    const int end = __shfl_sync(0xffffffffu, sg.end, src), b = __shfl_sync(0xffffffffu, sg.b, src);
    const int h = __shfl_sync(0xffffffffu, sg.h, src), r = __shfl_sync(0xffffffffu, sg.rb, src) * kRows + row;
    const bool in_ws = __shfl_sync(0xffffffffu, tail_in_ws, src);
    const size_t wrow = (2 * kCtas + (size_t)blockIdx.x * W + to) * kRows + row;
    // lane i: the state of warp from + i
    float2 ml = make_float2(-INFINITY, 0.f);
    if (from + lane <= to) ml = from + lane == to && in_ws ? p.part_ml[wrow] : mml[(from + lane) * kRows + row];
    float M = ml.x;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    const float f = ml.y == 0.f ? 0.f : ex2_approx(ml.x - M);  // (a NaN sum goes on to the output)
    float L = f * ml.y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
    float acc[kVecs][kVec];
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
#pragma unroll
      for (int k = 0; k < kVec; ++k) acc[v][k] = 0.f;
#pragma unroll 4
    for (int i = 0; i <= to - from; ++i) {
      const float fi = __shfl_sync(0xffffffffu, f, i);
      const float* src = from + i == to && in_ws ? p.part_o + wrow * D : mo + ((from + i) * kRows + row) * kPitch;
#pragma unroll
      for (int v = 0; v < kVecs; ++v) add_vec<kVec>(acc[v], fi, src + (32 * v + lane) * kVec);
    }
    if (first >= 0 && end <= cta_count) {
      if (r < R) finish_row<F16, kVec, kVecs>(p, D, b, h, r, lane, acc, M, L);
    } else {
      const size_t crow = (2 * (size_t)blockIdx.x + (end <= cta_count ? 1 : 0)) * kRows + row;
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
#pragma unroll
        for (int k = 0; k < kVec; ++k) p.part_o[crow * D + (32 * v + lane) * kVec + k] = acc[v][k];
      if (lane == 0) p.part_ml[crow] = make_float2(M, L);
    }
  }
}

// Joins the parts of the items that span several CTAs of the first kernel, in order;
// also writes the rows of sequences without keys.  WPR warps per query row, a vector of
// channels per lane, and each warp takes a share of the parts with many loads in flight.
constexpr int kJoinThreads = 256;
template <int D, int ROWS, bool F16, int WPR>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const DecodeParams p) {
  using C = DecCfg<D, ROWS>;
  constexpr int kRows = C::kRows, kPer = kJoinThreads / 32 / WPR;
  constexpr int kVec = D / 32 < 4 ? D / 32 : 4, kVecs = D / (32 * kVec);  // a lane's channels: kVecs vectors
  __shared__ float s_m[WPR], s_l[WPR], s_o[WPR > 1 ? WPR : 1][WPR > 1 ? D : 1];
  const int G = p.Hq / p.Hkv, R = G * p.Nq, nrb = (R + kRows - 1) / kRows, heads_rb = p.Hkv * nrb;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % WPR;
  const int at = blockIdx.x * kPer + warp / WPR;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (at >= p.B * p.Hkv * R) return;  // (with WPR > 1 the whole CTA)
  const int r = at % R, bh = at / R, h = bh % p.Hkv, b = bh / p.Hkv, row = r % kRows;
  const int before = p.pref[b], n = p.pref[b + 1] - before;
  int ca = 0, parts = 0;
  long long u1 = 0;
  const Cut ctas((long long)p.pref[p.B] * heads_rb, kCtas);
  if (n > 0) {
    const long long u0 = (long long)before * heads_rb + (long long)(h * nrb + r / kRows) * n;
    u1 = u0 + n;
    ca = ctas.of(u0);
    parts = ctas.of(u1 - 1) - ca + 1;
    if (parts == 1) return;  // that CTA wrote it
  }
  float acc[kVecs][kVec], M = -INFINITY, L = 0.f;
#pragma unroll
  for (int v = 0; v < kVecs; ++v)
#pragma unroll
    for (int k = 0; k < kVec; ++k) acc[v][k] = 0.f;
  // 32 of this warp's parts at a time: parts sub, sub + WPR, ...
  for (int i0 = sub; i0 < parts; i0 += 32 * WPR) {
    const int mine = i0 + lane * WPR;
    float2 ml = make_float2(-INFINITY, 0.f);
    size_t prow = 0;
    if (mine < parts) {
      const int cta = ca + mine;
      prow = (2 * (size_t)cta + (u1 <= ctas.first(cta + 1) ? 1 : 0)) * kRows + row;
      ml = p.part_ml[prow];
    }
    float mx = fmaxf(M, ml.x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    const float fo = M == mx ? 1.f : ex2_approx(M - mx);
    const float f = ml.y == 0.f ? 0.f : ex2_approx(ml.x - mx);  // (a NaN sum goes on to the output)
    M = mx;
    L *= fo;
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
#pragma unroll
      for (int k = 0; k < kVec; ++k) acc[v][k] *= fo;
    const int here = min(32, (parts - i0 + WPR - 1) / WPR);  // (the loads below do not wait for the weights)
#pragma unroll 8
    for (int i = 0; i < here; ++i) {
      const float fi = __shfl_sync(0xffffffffu, f, i), li = __shfl_sync(0xffffffffu, ml.y, i);
      const float* src = p.part_o + __shfl_sync(0xffffffffu, prow, i) * D;
      L = fmaf(fi, li, L);
#pragma unroll
      for (int v = 0; v < kVecs; ++v) add_vec<kVec>(acc[v], fi, src + (32 * v + lane) * kVec);
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
#pragma unroll
      for (int k = 0; k < kVec; ++k) s_o[sub][(32 * v + lane) * kVec + k] = acc[v][k];
    if (lane == 0) {
      s_m[sub] = M;
      s_l[sub] = L;
    }
    __syncthreads();
    if (warp > 0) return;
    M = -INFINITY;
    L = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) M = fmaxf(M, s_m[w]);
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
#pragma unroll
      for (int k = 0; k < kVec; ++k) acc[v][k] = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      const float f = s_l[w] == 0.f ? 0.f : ex2_approx(s_m[w] - M);
      L = fmaf(f, s_l[w], L);
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
#pragma unroll
        for (int k = 0; k < kVec; ++k) acc[v][k] = fmaf(f, s_o[w][(32 * v + lane) * kVec + k], acc[v][k]);
    }
  }
  finish_row<F16, kVec, kVecs>(p, D, b, h, r, lane, acc, M, L);
}

template <int D, int ROWS, bool F16>
cudaError_t launch_decode(DecodeParams prm, void* ws, cudaStream_t stream) {
  using C = DecCfg<D, ROWS>;
  uint8_t* w = static_cast<uint8_t*>(ws);
  prm.pref = (int*)w;
  w += C::align256((size_t)(prm.B + 1) * 4);
  prm.part_ml = (float2*)w;
  w += C::align256((size_t)C::kSlots * C::kRows * 8);
  prm.part_o = (float*)w;
  prm.nstages = C::stages(prm.B);
  prm.ring_off = C::ring_off(prm.B);
  cudaError_t e;
  const int smem = C::smem(prm.B);
  // the largest size, once per device (a bit each)
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  if ((e = cudaGetDevice(&dev))) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || !(ready.load() & bit)) {
    if ((e = cudaFuncSetAttribute(decode_kernel<D, ROWS, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  232448 - C::kStaticBytes)))
      return e;
    if (dev <= 63) ready.fetch_or(bit);
  }
  decode_kernel<D, ROWS, F16><<<kCtas, C::W * 32, smem, stream>>>(prm);
  if ((e = cudaGetLastError())) return e;
  // few rows: all warps of a CTA on each, since an item may have up to kCtas parts; many: a
  // warp each (there are few parts per item then)
  const int rows = prm.B * prm.Hq * prm.Nq;
  const bool wide = rows <= 8 * kCtas;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(wide ? rows : (rows + 7) / 8);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return wide ? cudaLaunchKernelEx(&cfg, join_kernel<D, ROWS, F16, 8>, prm)
              : cudaLaunchKernelEx(&cfg, join_kernel<D, ROWS, F16, 1>, prm);
}

// Rows per block: the fewest of 4, 8, 16, 32 that hold all G * Nq rows, up to what the
// registers hold (32 at d <= 128, 16 at d = 256); more rows go in several blocks, each of
// which reads the keys again (through L2).
int block_rows(int d, int rows) {
  if (rows <= 4) return 4;
  if (rows <= 8) return 8;
  if (rows <= 16 || d == 256) return 16;
  return 32;
}
// f(D, ROWS) as constants
template <typename F>
auto with_config(int d, int rows, F f) {
  using std::integral_constant;
  auto with_d = [&](auto D) {
    switch (rows) {
      case 4: return f(D, integral_constant<int, 4>{});
      case 8: return f(D, integral_constant<int, 8>{});
      case 16: return f(D, integral_constant<int, 16>{});
    }
    return f(D, integral_constant<int, decltype(D)::value == 256 ? 16 : 32>{});
  };
  if (d == 64) return with_d(integral_constant<int, 64>{});
  if (d == 128) return with_d(integral_constant<int, 128>{});
  return with_d(integral_constant<int, 256>{});
}

bool bad_heads(int B, int Hq, int Hkv, int Nq) {
  return B < 1 || B > kMaxSeqs || Hq < 1 || Hkv < 1 || Hq % Hkv || Hkv > (1 << 16) || Nq < 1 ||
         (long long)(Hq / Hkv) * Nq > (1 << 20) || (long long)B * Hq * Nq > 0x7FFFFFF0;  // (rounded up to 8 it is an int)
}

}  // namespace
}  // namespace apa

using namespace apa;

extern "C" {

size_t apa_attention_cache_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d) {
  if (bad_heads(B, Hq, Hkv, Nq) || (d != 64 && d != 128 && d != 256)) return 0;
  return with_config(d, block_rows(d, Hq / Hkv * Nq),
                     [&](auto D, auto rows) { return DecCfg<decltype(D)::value, decltype(rows)::value>::ws_bytes(B); });
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
  // (the stride of an axis of length 1 is never used: any value will do)
  if (B == 1) q_batch_stride = 0;
  if (Hq == 1) q_head_stride = 0;
  if (Nq == 1) q_row_stride = 0;
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
  const cudaError_t e = with_config(d, block_rows(d, Hq / Hkv * Nq), [&](auto D, auto rows) {
    constexpr int kD = decltype(D)::value, kR = decltype(rows)::value;
    return dtype == APA_DTYPE_F16 ? launch_decode<kD, kR, true>(prm, ws, stream)
                                  : launch_decode<kD, kR, false>(prm, ws, stream);
  });
  int st = e == cudaSuccess ? APA_OK : APA_ERR_CUDA;
  if (!workspace && cudaFreeAsync(ws, stream) != cudaSuccess && st == APA_OK) st = APA_ERR_CUDA;
  return st;
}

}  // extern "C"
