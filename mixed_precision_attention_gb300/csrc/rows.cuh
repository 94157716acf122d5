// rows.cuh -- exact attention of packed query rows over tiles of 64 keys, for sources of keys
// that bring their own producers (rows_kernel), and the joining of split walks.
//
// out = softmax(q K^T c + mask) V for the G * Nq rows that share a KV head's keys, taken
// together position-major in blocks of 128 (tcgen05 M).  A source says how many blocks and
// key tiles each sequence has, fills K and V tiles in shared memory (FP16 or BF16, 128-byte
// swizzle, a key per row), and masks scores.
//
// Work: an item is one block, or two neighbouring ones, of one KV head against all its
// tiles; a use is one block against one tile.  The items of all sequences form one list in
// units of a use's time (beginning an item counts, too), cut evenly over the CTAs, so
// lengths need not be alike and no length is read on the host.  A CTA's run of tiles of one
// item is a segment.  An item that one CTA holds entirely is written out at once; the states
// (m, l, O) of the others go to the workspace and a second kernel joins them in order, so
// results do not depend on timing.
//
// A softmax group is four warps with a thread per row, and a warp that issues its products: P V
// of use i, then S of use i + NB.  Those execute in that order, so S may go over the P that
// lies in its columns, and the commit of S says that the P V before it is done.  P goes to
// the product from tensor memory; O stays there, and moves with the running maximum only
// when a score exceeds that by 8 (log2 units).
//   Items of two blocks (d = 128, more than 128 rows): one CTA per SM with two groups, both
//     blocks against the same tiles, or one block (the last of an odd number) against every
//     other tile each, whose two states are then joined over tensor memory.  Two buffers of
//     S, so that a group's next S is there when it has stored P; Q in shared memory, as tensor
//     memory is full.
//   Items of one block at d <= 128: two CTAs per SM with one group and half of tensor memory
//     each, so that one works while the other begins an item (a row of 64 sequences, G = 3, over
//     up to 4096 keys: 118 us, 129 with one CTA of two groups; d = 64, any number of rows, likewise: 4 x 2048
//     rows, 24 heads on 8, over 8192 keys 493 us, 537; now 485).  Q is an operand in tensor memory: S of 64
//     keys would otherwise read 6 KB of shared memory per 32 cycles of product, 1.5 times what it delivers.
//   d = 256: O takes half of tensor memory: one group, one CTA.
//
// What bounds it, by traces of single CTAs: at 128 channels a use's products take 512 cycles
// (640 with Q in shared memory), its 8192 exponentials some 290 of the special-function units (28.5
// a cycle and SM, measured), and it costs 770 to 850: what is left is hand-overs.  A segment's
// beginning and end cost 10 000 to 15 000, most of it latency, which is why the list counts them: once per
// item, in front of its uses, not for the later CTAs that take a part of it.  Where items have few tiles that
// leaves the work uneven: 24 of the 96 CTAs that share 8 items of 17 tiles get the beginning of one alone, and
// of 8 x 333 rows (G = 3, d = 256, to 1021 keys) the busiest CTA has 16 uses where the mean is 8.7.  Tried and not kept: one diverged
// thread as issuer (1900 cycles a use), one issuer for both groups (1140), tiles of 128 keys
// (1230 TF/s on prompts where this form has 1350, and registers spill), all 64 scores in
// registers at once where there are more than 12 warps (spills that miss the cache), register
// shares by setmaxnreg (the compiler keeps to the launch's count), two threads per row, each
// with half of a tile's keys, where a block has at most 64 rows (trees of 32 nodes 114 us for 100).
//
// The kernel is launched while the one before it ends (programmatic dependent launch): barriers
// are set up meanwhile.  Everything that another kernel may have written is read, and tensor
// memory taken, behind griddepcontrol.wait (with it, and segments found without divisions, trees
// of 32 nodes over 32 contexts went from 104 to 100 us, 64-node trees over 131072 keys from 197 to 194).
#pragma once
#include <atomic>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "../../include/apa.h"
#include "apa_internal.h"
#include "cache_page.cuh"
#include "tc.cuh"

namespace apa {
namespace {

constexpr int kRowSms = 152;
constexpr int kMaxRowSeqs = 8192;
constexpr float kTauRows = 8.f;    // lazy-maximum threshold, log2 units
constexpr float kLn2 = 0.6931471805599453f;

// x / n for x >= 0; nearly always a 32-bit division.
__device__ __forceinline__ long long rows_quotient(long long x, int n) {
  if (((unsigned long long)x >> 32) == 0) return (unsigned)x / (unsigned)n;
  return x / n;
}
// n things in k nearly equal runs, the longer ones first.
struct RowCut {
  long long q;
  int r, k;
  __device__ __forceinline__ RowCut(long long n, int k_) : k(k_) {
    q = rows_quotient(n, k);
    r = (int)(n - q * k);
  }
  __device__ __forceinline__ long long first(int i) const { return i >= k ? q * k + r : q * i + min(i, r); }
};
// How many CTAs share a list of `total` units.  A CTA takes no fewer than k, where k follows the units of an item: joining
// the parts costs in their number, and a use about a microsecond itself (8 items of 17 tiles: trees of 26 nodes over 1000
// keys 22 us with k = 1, 19 with 2, 19.6 with 4; of 24 tiles: a row over 1500 keys 20, 16.5, 16.2; of 128: over 8192 keys
// 28, 28, 25).
__device__ __forceinline__ int cut_ctas(long long total, long long items, int grid) {
  int k = 1;
  while (k < 8 && 20 * k * k * items < total) k *= 2;
  const long long n = rows_quotient(total + k - 1, k);
  return n < 1 ? 1 : n < grid ? (int)n : grid;
}

// The item that begins in a CTA and goes on behind it (n = 0: none).
struct SplitRec {
  long long first, total;  // its first use in the list; the list's length
  int b, h, rb, n, w, ctas;  // (ctas: how many share the list)
};

struct RowParams {
  int B, Hq, Hkv, Nq;
  const uint16_t* q;
  long long qs_b, qs_h, qs_r;
  uint16_t* out;  // [B][Hq][Nq][d]
  float* lse;     // [B][Hq][Nq] or null
  int* err;
  // workspace
  SplitRec* rec;    // [grid]
  // Slots 2 cta + 1 and 2 cta hold the CTA's part of the item that ends in it, and of the one that goes on behind it.
  float2* part_ml;  // [2 grid][slot rows] (m, l)
  float* part_o;    // [2 grid][d / 4][slot rows][4], so that 32 neighbouring rows' vectors are 512 bytes in a run
  int slot_rows;
  __host__ __device__ int G() const { return Hq / Hkv; }
};

template <int D_, int KT_, int NG_, int NB_, bool QT_, int NK_, int NV_, bool F16_>
struct RowCfg {
  static constexpr int D = D_, KT = KT_, NG = NG_, NB = NB_;
  static constexpr bool QT = QT_, F16 = F16_;
  static constexpr int NK = NK_, NV = NV_;
  // One group at d <= 128: two CTAs share an SM, and its tensor memory.
  static constexpr int kCtasPerSm = NG == 1 && D <= 128 ? 2 : 1, kCtas = kRowSms * kCtasPerSm;
  static constexpr uint32_t kTmemCols = 512 / kCtasPerSm;
  static constexpr int kBlocks = NG;  // row blocks of an item, at most
  static constexpr int kTileBytes = KT * D * 2;
  static constexpr int kQBytes = QT ? 0 : 128 * D * 2;  // per block
  static constexpr uint32_t kOCol = 0, kSCol = NG * D, kQCol = kSCol + NG * NB * KT;  // S: NB buffers per group
  static constexpr uint32_t kPOff = KT / 2;  // P, two keys per column, in the upper half of its S
  static constexpr int kQOff = 0, kKOff = NG * kQBytes, kVOff = kKOff + NK * kTileBytes;
  static constexpr int kStagePitch = 144, kStageOff = kVOff + NV * kTileBytes;  // Q on its way to tensor memory: 64 channels
  static constexpr int kSrcOff = kStageOff + (QT ? NG * 128 * kStagePitch : 0);  // of each row; the source's own
  static constexpr int kSoftWarps = 4 * NG, kMmaWarp = kSoftWarps, kSrcWarp = kSoftWarps + NG;
  // With one buffer (and one group) the commit of S(i + 1) says that K of that use and V of use i have been read: a lane of
  // the softmax group hands the stages back.  With two, V would wait for another use: the issuer's commits do.
  static constexpr bool kSoftRelease = NB == 1;
  static_assert(NG == 1 || NB == 2, "two groups have two buffers each");
  static constexpr float kLift = F16 ? 6.f : 0.f;  // P is 2^(x - m + kLift): at most 2^14, within FP16
  // Where |m| reaches this the roundings of m and kLift - m (an ulp of m: 1 below 2^24, 32 below 2^29) take P out of its
  // type's range: such rows are NaN.  Rounding x c2 to FP32 before m comes off has no such limit, but cost 2 to 8 % on
  // some case in each of eight forms (a branch per tile, its code in line or not): the loop is bound by its own latency.
  static constexpr float kFar = F16 ? 16777216.f : 536870912.f;
  // What beginning an item takes, in uses.  Without it (0) CTAs with many short items end last: trees of 32 nodes over 32
  // contexts to 8192 keys 127 us, 104 with 7 (106 with 10); prompts of 2048 rows 440 us, 410 with 20 (420 with 34); 333 rows
  // at d = 256 40 us, 32 with 12.
  static constexpr int kItemCost = NG == 2 ? 20 : D == 256 ? 12 : 7;
  static_assert(NG == 1 || (NK % 2 == 0 && NV % 2 == 0), "RowShare");
  static_assert(kQCol + (QT ? NG * D / 2 : 0) <= kTmemCols, "tensor memory");
};

// A CTA's run of tiles t0 .. t1-1 (of n) of one item: blocks rb .. rb+w-1 of head h of sequence b.
struct RowSeg {
  int b, h, rb, w, t0, t1, n;
};
// A group's uses of a segment with T tiles before it in the CTA: all its tiles, or (two groups, one block) those with
// the group's parity in the CTA's count.  The rings have an even number of stages then, so that such a tile's stage
// is its group's: nobody skips a phase of a barrier that it waits for within the segment.
struct RowShare {
  int first, step, uses;
  __device__ __forceinline__ RowShare(int NG, int w, int tiles, int g, int T) {
    step = NG == 2 && w == 1 ? 2 : 1;
    first = step == 2 ? (g ^ T) & 1 : 0;
    uses = (tiles - first + step - 1) / step;
  }
  __device__ __forceinline__ int tile(int i) const { return first + step * i; }  // counted from the segment's first
};
// The list in units of a use's time: an item is its uses behind kItemCost units for what beginning one takes (Q, the last
// item's epilogue, the first S).
template <class Src>
__device__ __forceinline__ long long rows_cost(const typename Src::Seq& s) {  // of one head
  const int per = (s.blocks + Src::Cfg::kBlocks - 1) / Src::Cfg::kBlocks;
  return s.tiles ? (long long)s.blocks * s.tiles + (long long)per * Src::kItemCost : 0;
}
// A warp's way through the segments of its CTA, in shared memory: what is the same for all its lanes, and
// looked up now and then, does not take every lane's registers.
template <class Src>
struct RowWalk {
  static constexpr int kBlocks = Src::Cfg::kBlocks;
  using Params = typename Src::Params;
  int b, item, pos, left;     // item of the sequence, units into it, units left
  typename Src::Seq seq;      // the source's numbers of the segment's sequence
  RowSeg g;                   // the segment
  __device__ __forceinline__ void start(const int* begin, const typename Src::Seq& first, int left_) {
    b = begin[0];
    item = begin[1];
    pos = begin[2];
    left = left_;
    seq = first;
  }
  // one lane's work
  __device__ __forceinline__ bool step(const Params& p) {
    while (left > 0) {
      int per = (seq.blocks + kBlocks - 1) / kBlocks, h = per == 1 ? item : item / per, rb = (item - h * per) * kBlocks;
      int w = min(kBlocks, seq.blocks - rb);
      if (pos == Src::kItemCost + seq.tiles * w) {  // the next item
        pos = 0;
        if (++item == per * p.r.Hkv) {
          item = 0;
          do {
            seq = typename Src::Seq(p, ++b);
          } while (seq.blocks == 0 || seq.tiles == 0);
          per = (seq.blocks + kBlocks - 1) / kBlocks;
        }
        h = per == 1 ? item : item / per;
        rb = (item - h * per) * kBlocks;
        w = min(kBlocks, seq.blocks - rb);
      }
      const int end = min(Src::kItemCost + seq.tiles * w, pos + left);
      g = RowSeg{b, h, rb, w, max(0, pos - Src::kItemCost) >> (w - 1), max(0, end - Src::kItemCost) >> (w - 1), seq.tiles};
      left -= end - pos;
      pos = end;
      if (g.t1 > g.t0) return true;  // (half a tile of two blocks is the next CTA's)
    }
    return false;
  }
  // the whole warp's
  __device__ __forceinline__ bool next(const Params& p, int lane) {
    __syncwarp();
    bool any = false;
    if (lane == 0) any = step(p);
    __syncwarp();
    return __any_sync(0xffffffffu, any);
  }
};

// One lane of a warp that is together.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n.reg .pred p;\n"
      "elect.sync _|p, 0xffffffff;\n"
      "selp.u32 %0, 1, 0, p;\n}"
      : "=r"(e));
  return e != 0;
}

// used only while unwinding: waits for copies and products already in flight, ignoring the abort flag
__device__ __forceinline__ void rows_wait_in_flight(uint32_t bar, uint32_t parity, int* err) {
  const unsigned long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > APA_WAIT_LIMIT_CYCLES) {
      if (err) atomicCAS(err, 0, APA_DEVERR_TIMEOUT);
      return;
    }
  }
}

// P of eight consecutive keys, 2^(x*c2 + nb), as four words of two 16-bit values (key 2k in the low
// half of word k); the FP32 values are added into (s0, s1): even keys into s0, odd keys into s1.
// The rounding (half a step: 2^-11 in FP16, 2^-8 in BF16) is what the product with V asks for: both its operands have one
// 16-bit type, and V comes as BF16 or is exact in FP16.  Against 64 bits the outputs' error grows by it from 0.0017, their own
// rounding's, to 0.0023 of their norm where both are BF16, from 0.00021 to 0.00029 where both are FP16, and not
// visibly where weights are FP16 and outputs BF16.  Weights in two terms would take twice the products with V.
// The affine step and the sums run as packed FP32 pairs.
template <bool F16>
__device__ __forceinline__ void rows_p8(const float* x, float c2, float nb, uint32_t* h, float& s0, float& s1) {
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
    h[k] = pack2<F16>(lo, hi);
    asm("mov.b64 %0, {%1, %2};" : "=l"(a[k]) : "f"(lo), "f"(hi));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(s) : "l"(a[k]), "l"(one));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(s0), "=f"(s1) : "l"(s));
}

// Barriers of the core (the source's follow): K and V rings, S and P per buffer, a segment's last P.V and the
// last but one per group, Q there and read, the exchange of
// two groups' states and its end, and the issuers' drains.
template <class C>
struct RowBars {
  static constexpr int kKFull = 0, kKEmpty = C::NK, kVFull = 2 * C::NK, kVEmpty = 2 * C::NK + C::NV;
  static constexpr int kBufs = C::NG * C::NB, kS = 2 * C::NK + 2 * C::NV, kP = kS + kBufs, kPV = kP + kBufs, kPV2 = kPV + C::NG, kQ = kPV2 + C::NG,
                       kQFree = kQ + 1, kX = kQ + 2, kXDone = kX + 1, kDrain = kXDone + 1, kNum = kDrain + C::NG;
  uint32_t bar0;
  volatile int* abort;
  int* err;
  __device__ __forceinline__ uint32_t at(int i) const { return bar0 + 8u * i; }
  __device__ __forceinline__ uint32_t k_full(int T) const { return at(kKFull + T % C::NK); }
  __device__ __forceinline__ uint32_t k_empty(int T) const { return at(kKEmpty + T % C::NK); }
  __device__ __forceinline__ uint32_t v_full(int T) const { return at(kVFull + T % C::NV); }
  __device__ __forceinline__ uint32_t v_empty(int T) const { return at(kVEmpty + T % C::NV); }
  static __device__ __forceinline__ uint32_t k_par(int T) { return (T / C::NK) & 1; }
  static __device__ __forceinline__ uint32_t v_par(int T) { return (T / C::NV) & 1; }
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const { return mbar_wait(bar, parity, abort, err); }
  // every lane waits; the warp proceeds only if all lanes succeeded
  __device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) const {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err));
  }
};

// What a row's O is multiplied by, and its lse: 0 and -inf where it has seen no key, NaN where its maximum is too far from 0
// (its weights, and their sum, may have become 0 there).
template <class C>
__device__ __forceinline__ float rows_inverse(float m, float l, float v_scale) {
  if (m == -INFINITY && l == 0.f) return 0.f;
  return fabsf(m) < C::kFar ? v_scale / l : __int_as_float(0x7FFFFFFF);
}
template <class C>
__device__ __forceinline__ float rows_lse(float m, float l) {
  if (m == -INFINITY && l == 0.f) return -INFINITY;
  return fabsf(m) < C::kFar ? kLn2 * (m - C::kLift + log2f(l)) : __int_as_float(0x7FFFFFFF);
}

// The column of O that holds channel c: sources may store V's channels in another order within each 16.
template <class Src>
__device__ __forceinline__ constexpr int o_column(int c) {
  return Src::kPairedV ? (c & ~15) | ((c & 7) << 1) | ((c >> 3) & 1) : c;
}

template <class Src>
__global__ void __launch_bounds__(Src::kThreads, Src::Cfg::kCtasPerSm) rows_kernel(const __grid_constant__ typename Src::Params p) {
  using C = typename Src::Cfg;
  using Bars = RowBars<C>;
  constexpr int D = C::D, KT = C::KT, NG = C::NG;
  constexpr uint32_t kTmemCols = C::kTmemCols;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t bar_mem[Bars::kNum + Src::kBars];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ float2 xml[NG == 2 ? 2 : 1][NG == 2 ? 128 : 1];  // two groups' (m, l) of a row
  __shared__ RowWalk<Src> walks[Src::kThreads / 32];
  __shared__ long long warp_sum[32];
  __shared__ int found[2];   // the last unit's sequence, and units (of a head) before it
  __shared__ int begin[3];   // the first unit's sequence, item of it, units into that
  __shared__ typename Src::Seq first_seq;
  const RowParams& r = p.r;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);
  Bars bars{smem_u32(bar_mem), &abort_flag, r.err};

  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < Bars::kNum; ++i) {
      uint32_t count = 1;
      if (i < Bars::kKEmpty) count = Src::kKArrivals;
      if (i >= Bars::kVFull && i < Bars::kVEmpty) count = Src::kVArrivals;
      if ((i >= Bars::kKEmpty && i < Bars::kVFull) || (i >= Bars::kVEmpty && i < Bars::kS)) count = NG;
      if (i >= Bars::kP && i < Bars::kPV) count = 4;
      if (i == Bars::kQFree) count = 2 * NG;  // a lane of each group, and its issuer
      if (i == Bars::kQ || i == Bars::kX || i == Bars::kXDone) count = C::kSoftWarps;
      mbar_init(bars.at(i), count);
    }
    for (int i = 0; i < Src::kBars; ++i) mbar_init(bars.at(Bars::kNum + i), Src::bar_count(i));
    fence_mbar_init();
  }
  // (launched early: what is above needs nothing that the kernel before this one writes, and takes nothing that it may still
  // want: columns of tensor memory, held here, could keep it from ending, and this CTA waits for that)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == C::kMmaWarp) {
    tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  // ---- the list's length, and this CTA's place in it: each thread sums up a run of sequences
  constexpr int kWarps = Src::kThreads / 32;
  const int run = (r.B + Src::kThreads - 1) / Src::kThreads, b_lo = min(r.B, tid * run), b_hi = min(r.B, b_lo + run);
  long long before = 0, total = 0, mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const typename Src::Seq s(p, b);
    s.report(p, b);
    mine += rows_cost<Src>(s);
  }
  {
    long long x = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, s);
      if (lane >= s) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += warp_sum[w];
      total += warp_sum[w];
    }
    before += x - mine;
  }
  total *= r.Hkv;
  const RowCut cut(total, cut_ctas(total, (long long)r.B * r.Hkv * ((r.G() * r.Nq + kBlockRows - 1) / kBlockRows), gridDim.x));
  const long long x0 = cut.first(blockIdx.x), x1 = cut.first(blockIdx.x + 1);
  // a place in the list, x, of a sequence with `sum` units (of a head) before it, as its item and units into that
  auto place = [&](const typename Src::Seq& s, long long sum, long long x, int& item, int& pos) {
    const int per = (s.blocks + C::kBlocks - 1) / C::kBlocks, head = (int)rows_cost<Src>(s);
    const int full = C::kBlocks * s.tiles + Src::kItemCost;
    const long long y = x - sum * r.Hkv;
    const int h = (int)rows_quotient(y, head), z = (int)(y - (long long)h * head), kk = z / full;
    item = h * per + kk;
    pos = z - kk * full;
  };
  auto here = [&](long long x) { return x1 > x0 && x >= before * r.Hkv && x < (before + mine) * r.Hkv; };
  if (here(x0) || here(x1 - 1)) {
    long long sum = before;
    for (int b = b_lo; b < b_hi; ++b) {
      const typename Src::Seq s(p, b);
      const long long n = rows_cost<Src>(s), end = (sum + n) * r.Hkv;
      if (x0 >= sum * r.Hkv && x0 < end) {
        begin[0] = b;
        first_seq = s;
        place(s, sum, x0, begin[1], begin[2]);
      }
      if (x1 - 1 >= sum * r.Hkv && x1 - 1 < end) {
        found[0] = b;
        found[1] = (int)sum;
      }
      sum += n;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == C::kMmaWarp && lane == 0) {  // (it waits for Q first of all)
    SplitRec rec{};
    if (x1 > x0) {
      const int b = found[0];
      const typename Src::Seq s(p, b);
      int item, pos;
      place(s, found[1], x1 - 1, item, pos);
      const int per = (s.blocks + C::kBlocks - 1) / C::kBlocks, rb = item % per * C::kBlocks;
      const int w = min(C::kBlocks, s.blocks - rb);
      const long long first = x1 - 1 - pos;
      if (first >= x0 && first + Src::kItemCost + (long long)s.tiles * w > x1) rec = SplitRec{first, total, b, item / per, rb, s.tiles, w, cut.k};
    }
    r.rec[blockIdx.x] = rec;
  }
  if (x1 > x0) {
    RowWalk<Src>& walk = walks[warp];
    if (lane == 0) walk.start(begin, first_seq, (int)(x1 - x0));
    if (warp >= C::kSrcWarp) {
      Src::produce(p, walk, smem, sbase, bars, warp - C::kSrcWarp, lane);
    } else if (warp >= C::kMmaWarp) {
      // ------------------------------------------------------------ a group's issuer
      // The warp stays together and one lane issues: what the products take is the same in all lanes and so
      // in uniform registers.
      constexpr uint32_t idS = C::F16 ? idesc_f16(128, KT, 0) : idesc_bf16(128, KT, 0);
      constexpr uint32_t idO = C::F16 ? idesc_f16(128, D, 1) : idesc_bf16(128, D, 1);
      const int g = __shfl_sync(0xffffffffu, warp, 0) - C::kMmaWarp;
      const bool elected = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), ocol = tm + C::kOCol + g * D;
      const uint64_t qd0 = smem_desc(sbase + C::kQOff, 16, 1024, kSwizzle128B);
      const uint64_t kd0 = smem_desc(sbase + C::kKOff, 16, 1024, kSwizzle128B);
      const uint64_t vd0 = smem_desc(sbase + C::kVOff, KT * 128, 1024, kSwizzle128B);
      uint32_t T = 0, n = 0, qpar = 0;  // tiles before the segment; this group's uses before it
      bool ok = true;
      while (ok && walk.next(p, lane)) {
        const int w = __shfl_sync(0xffffffffu, walk.g.w, 0), tiles = __shfl_sync(0xffffffffu, walk.g.t1 - walk.g.t0, 0);
        const RowShare mine(NG, w, tiles, g, T);
        if (!(ok = bars.warp_wait(bars.at(Bars::kQ), qpar))) break;
        qpar ^= 1;
        // (an issuer without a use in the segment has to have seen its Q, too, before the next one comes)
        if (NG == 2 && elected) mbar_arrive(bars.at(Bars::kQFree));
        const bool alone = NG == 2 && w == 1;  // (a tile that the other group has no part in counts twice)
        const uint32_t blk = w == 2 ? g : 0, qcol = tm + C::kQCol + blk * (D / 2);
        const uint64_t qd = qd0 + blk * (C::kQBytes >> 4);
        // P V of use i, then S of use i + NB, in whose columns that P lies: its commit says as well that this P V is done.
        auto give_v = [&](uint32_t t) {
          if (elected) {
            mma_commit(bars.v_empty(t));
            if (alone) mma_commit(bars.v_empty(t));
          }
          __syncwarp();
        };
        for (int i = -C::NB; i < mine.uses; ++i) {
          const int j = i + C::NB;
          const uint32_t buf = (n + j) % C::NB;
          const uint32_t scol = tm + C::kSCol + (g * C::NB + buf) * KT;
          const uint32_t tv = T + mine.tile(max(i, 0)), tk = T + mine.tile(j);
          if (i >= 0) {
            // (P first: it comes behind the end of the last segment, when all of V there has been read)
            if (!(ok = bars.warp_wait(bars.at(Bars::kP + g * C::NB + buf), ((n + i) / C::NB) & 1))) break;
            if (!(ok = bars.warp_wait(bars.v_full(tv), Bars::v_par(tv)))) break;
            tc_fence_after();
            const uint64_t vd = vd0 + tv % C::NV * (C::kTileBytes >> 4);
            if (elected) {
              mma_f16_ts(ocol, scol + C::kPOff, vd, idO, i > 0 ? 1u : 0u);  // (the first of the segment starts O anew)
#pragma unroll
              for (int kk = 1; kk < KT / 16; ++kk)
                mma_f16_ts(ocol, scol + C::kPOff + 8u * kk, vd + kk * (2048 >> 4), idO, 1u);
              if (j >= mine.uses) mma_commit(bars.at((i + 1 == mine.uses ? Bars::kPV : Bars::kPV2) + g));
            }
            __syncwarp();
            if (!C::kSoftRelease && Src::kVFirst) give_v(tv);
          }
          if (j < mine.uses) {
            if (!(ok = bars.warp_wait(bars.k_full(tk), Bars::k_par(tk)))) break;
            tc_fence_after();
            const uint64_t kd = kd0 + tk % C::NK * (C::kTileBytes >> 4);
            if (elected) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t bd = kd + (((kk >> 2) * (KT * 128) + (kk & 3) * 32) >> 4);
                if constexpr (C::QT)
                  mma_f16_ts(scol, qcol + 8u * kk, bd, idS, kk > 0);
                else
                  mma_bf16(scol, qd + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4), bd, idS, kk > 0);
              }
              mma_commit(bars.at(Bars::kS + g * C::NB + buf));
            }
            __syncwarp();
          }
          // the stages go back (a commit costs the issuing warp a hundred cycles and more, so behind all products)
          if (i >= 0 && !C::kSoftRelease && !Src::kVFirst) give_v(tv);
          if (elected && !C::kSoftRelease) {
            if (j < mine.uses) {
              mma_commit(bars.k_empty(tk));
              if (alone) mma_commit(bars.k_empty(tk));
            }
          }
          __syncwarp();
        }
        T += tiles;
        n += mine.uses;
      }
      // drain: every product issued by this thread has completed before tensor memory is freed
      if (elected) {
        mma_commit(bars.at(Bars::kDrain + g));
        rows_wait_in_flight(bars.at(Bars::kDrain + g), 0, r.err);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ softmax (one thread per row)
      const int g = warp >> 2, row = tid & 127;
      const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t tl = tmem + lane_base;
      typename Src::Row me;  // this thread's row: me.valid, me.out_row (in rows, or -1), what masks and scales it
      float m2 = -INFINITY, l2 = 0.f;
      // Q of a segment, a warp its 32 rows, so that neighbouring lanes read neighbouring channels.  Both groups share
      // the block of an item with one, a half of the channels each.
      auto put_q = [&]() {
        const RowSeg& s = walk.g;
        const int buf = s.w == 2 ? g : 0, P = (s.rb + buf) * kBlockRows + row, G = r.G();
        me.set(p, walk.seq, s.b, s.h, P);
        const uint16_t* base = r.q + s.b * r.qs_b + (long long)s.h * G * r.qs_h;
        const long long off = (P % G) * r.qs_h + (P / G) * r.qs_r;
        const unsigned used = __ballot_sync(0xffffffffu, me.valid);
        // rows kRows i + lane / kLanes of the warp, channels c + 8 (lane % kLanes) ..
        auto fetch = [&](auto lanes, int i, int c) {
          constexpr int kLanes = decltype(lanes)::value, kRows = 32 / kLanes;
          const int from = kRows * i + lane / kLanes;
          const long long o = __shfl_sync(0xffffffffu, off, from);
          return (used >> from) & 1 ? *reinterpret_cast<const uint4*>(base + o + c + 8 * (lane % kLanes))
                                    : make_uint4(0u, 0u, 0u, 0u);
        };
        float up = 1.f;
        if constexpr (Src::kScaledQ) {
          constexpr int kLanes = D / 8, kRows = 32 / kLanes;
          float amax = 0.f;
#pragma unroll 1
          for (int i0 = 0; i0 < 32 / kRows; i0 += 8) {
            uint4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fetch(std::integral_constant<int, kLanes>{}, i0 + i, 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float a = Src::largest(v[i]);
#pragma unroll
              for (int d = kLanes / 2; d > 0; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
              a = __shfl_sync(0xffffffffu, a, lane % kRows * kLanes);  // that of row kRows (i0 + i) + lane % kRows
              if (lane / kRows == i0 + i) amax = a;
            }
          }
          up = me.scale(amax);
        }
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 64) {
          if (NG == 2 && s.w == 1 && c0 / 64 != g) continue;
          uint4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = fetch(std::integral_constant<int, 8>{}, i, c0);
          if constexpr (C::QT) {
            uint8_t* stage = smem + C::kStageOff + warp * 32 * C::kStagePitch;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(stage + (4 * i + lane / 8) * C::kStagePitch + lane % 8 * 16) = v[i];
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t w[16];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint4 x = *reinterpret_cast<const uint4*>(stage + lane * C::kStagePitch + 64 * h + 16 * k);
                w[4 * k] = me.convert(x.x, up);
                w[4 * k + 1] = me.convert(x.y, up);
                w[4 * k + 2] = me.convert(x.z, up);
                w[4 * k + 3] = me.convert(x.w, up);
              }
              tmem_st_x16(tl + C::kQCol + buf * (D / 2) + c0 / 2 + 16 * h, w);
            }
            __syncwarp();
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int from = 4 * i + lane / 8, at = (warp & 3) * 32 + from;
              const float f = __shfl_sync(0xffffffffu, up, from);
              *reinterpret_cast<uint4*>(smem + C::kQOff + buf * C::kQBytes + (c0 / 64) * 16384 + at * 128 +
                                        ((lane % 8 ^ (at & 7)) << 4)) =
                  make_uint4(me.convert(v[i].x, f), me.convert(v[i].y, f), me.convert(v[i].z, f), me.convert(v[i].w, f));
            }
          }
        }
        if constexpr (C::QT) {
          tmem_wait_st();
          tc_fence_before();
        } else {
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.at(Bars::kQ));
      };
      // Parities: tiles before the segment, segments, each group's commits of P V, this group's of the last but one,
      // exchanges of two states; and this group's uses before the segment.
      constexpr uint32_t kParT = 1, kParSeg = 2, kParPV = 4, kParPV2 = 16, kParX = 32;
      uint32_t par = 0;
      int n = 0, T = 0;  // (T: tiles, only for the stages)
      bool ok = true, any = walk.next(p, lane);
      if (any) put_q();
      while (any) {
        const int tiles = walk.g.t1 - walk.g.t0, w = walk.g.w;
        const RowShare share(NG, w, tiles, g, par & kParT);
        const bool warp_idle = !__any_sync(0xffffffffu, me.valid);
        int plain_lo = 0, plain_hi = 0;  // the segment's tiles of which every row sees every key
        if constexpr (Src::kMasked) Src::plain(p, walk, plain_lo, plain_hi);
        m2 = -INFINITY;
        l2 = 0.f;
        for (int i = 0; i < share.uses; ++i) {
          const int buf = (n + i) % C::NB;
          uint32_t vis[KT / 32];
          if (Src::kMasked && share.tile(i) >= plain_lo && share.tile(i) < plain_hi) {
#pragma unroll
            for (int c = 0; c < KT / 32; ++c) vis[c] = me.valid ? ~0u : 0u;
          } else {
            me.template mask<KT / 32>(p, walk, share.tile(i), vis);
          }
          if (!(ok = bars.warp_wait(bars.at(Bars::kS + g * C::NB + buf), ((n + i) / C::NB) & 1))) break;
          const uint32_t scol = tl + C::kSCol + (g * C::NB + buf) * KT, pcol = scol + C::kPOff;
          if (C::kSoftRelease && (warp & 3) == 0 && lane == 0) {
            mbar_arrive(bars.k_empty(T + share.tile(i)));
            if (i > 0) mbar_arrive(bars.v_empty(T + share.tile(i - 1)));
          }
          if (warp_idle) {  // (rows of P that nobody uses: whatever is there)
            if (lane == 0) mbar_arrive(bars.at(Bars::kP + g * C::NB + buf));
            continue;
          }
          tc_fence_after();
          // 32 keys at a time, so that few registers are live; the first 32 are loaded again after the maximum
          float sv[32], rmax = -INFINITY;
          auto load = [&](int c) {
            uint32_t raw[32];
            tmem_ld_x32(scol + 32 * c, raw);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) sv[k] = __uint_as_float(raw[k]);
            uint32_t v = vis[0];
#pragma unroll
            for (int k = 1; k < KT / 32; ++k) v = c == k ? vis[k] : v;
            if (__any_sync(0xffffffffu, v != ~0u)) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!((v >> k) & 1u)) sv[k] = -INFINITY;
            }
          };
#pragma unroll Src::kSoftUnroll
          for (int c = 0; c < KT / 32; ++c) {
            load(c);
            float g8[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              g8[k] = max3(max3(sv[8 * k], sv[8 * k + 1], sv[8 * k + 2]), max3(sv[8 * k + 3], sv[8 * k + 4], sv[8 * k + 5]),
                           fmaxf(sv[8 * k + 6], sv[8 * k + 7]));
            rmax = fmaxf(rmax, max3(max3(g8[0], g8[1], g8[2]), g8[3], g8[3]));
          }
          const float top = __fmul_rn(rmax, me.c2);  // (c2 > 0)
          float f = 1.f;
          bool rescale = false;
          if (top - m2 > kTauRows) {  // (infinite for a row's first score; a NaN, so false, before it)
            if (l2 > 0.f) {
              f = ex2_approx(m2 - top);
              rescale = true;
            }
            m2 = top;
          }
          // a row that has seen no key yet: its scores are -inf and its weights 0
          const float nb = m2 == -INFINITY ? 0.f : C::kLift - m2;
          float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll Src::kSoftUnroll
          for (int c = KT / 32 - 1; c >= 0; --c) {
            if (Src::kSoftUnroll == 1 || c < KT / 32 - 1) load(c);
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) rows_p8<C::F16>(sv + 8 * k, me.c2, nb, pk + 4 * k, ps[k & 1], ps[2 + (k & 1)]);
            tmem_st_x16(pcol + 16u * c, pk);
          }
          l2 = l2 * f + ((ps[0] + ps[1]) + (ps[2] + ps[3]));
          if (__any_sync(0xffffffffu, rescale)) {
            // This S came behind P V of use i - NB.  With two buffers, that of use i - 1 has to land: the S behind it
            // says so, or its own commit.
            if (C::NB == 2 && i > 0) {
              if (!(ok = i + 1 < share.uses
                             ? bars.warp_wait(bars.at(Bars::kS + g * C::NB + (buf ^ 1)), ((n + i + 1) / C::NB) & 1)
                             : bars.warp_wait(bars.at(Bars::kPV2 + g), par & kParPV2 ? 1 : 0)))
                break;
            }
            tc_fence_after();
            const uint32_t ocol = tl + C::kOCol + g * D;
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t o[32];
              tmem_ld_x32(ocol + c0, o);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
              tmem_st_x16(ocol + c0, o);
              tmem_st_x16(ocol + c0 + 16, o + 16);
            }
          }
          tmem_wait_st();  // P (and a rescaled O) in tensor memory before P.V is issued
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars.at(Bars::kP + g * C::NB + buf));
        }
        if (!ok) break;
        // ---- the next segment's Q, once every S of this one is done; then this one's epilogue
        const int out_row = me.out_row;
        const float v_scale = me.v_scale;
        const bool whole = walk.g.t0 == 0 && walk.g.t1 == walk.g.n, ends = walk.g.t1 == walk.g.n;
        if (NG == 2) {
          if ((warp & 3) == 0 && lane == 0) mbar_arrive(bars.at(Bars::kQFree));
          if (!(ok = bars.warp_wait(bars.at(Bars::kQFree), par & kParSeg ? 1 : 0))) break;
        }
        any = walk.next(p, lane);
        if (any) put_q();
        const bool joint = NG == 2 && w == 1;  // the groups' states belong to the same rows
        float f0 = 1.f, f1 = 0.f;  // of this group's O, and the other's
        if (joint) {
          xml[g][row] = make_float2(m2, l2);
          __syncwarp();
          if (lane == 0) mbar_arrive(bars.at(Bars::kX));
          if (!(ok = bars.warp_wait(bars.at(Bars::kX), par & kParX ? 1 : 0))) break;
          const float2 y = xml[g ^ 1][row];
          const float M = fmaxf(m2, y.x);
          f0 = l2 == 0.f ? 0.f : ex2_approx(m2 - M);  // (a NaN sum goes on to the output)
          f1 = y.y == 0.f ? 0.f : ex2_approx(y.x - M);
          l2 = g == 0 ? f0 * l2 + f1 * y.y : f1 * y.y + f0 * l2;
          m2 = M;
        }
        bool has_own = true, has_other = false;
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          const int uses = RowShare(NG, w, tiles, k, par & kParT).uses;
          if (k == g)
            has_own = uses > 0;
          else
            has_other = joint && uses > 0;
          if (ok && uses > 0 && (joint || k == g)) ok = bars.warp_wait(bars.at(Bars::kPV + k), par & (kParPV << k) ? 1 : 0);
          if (uses > 0) par ^= kParPV << k;
        }
        if (!ok) break;
        tc_fence_after();
        if (C::kSoftRelease && (warp & 3) == 0 && lane == 0 && share.uses > 0)  // the last use's V
          mbar_arrive(bars.v_empty(T + share.tile(share.uses - 1)));
        T += tiles;
        const int slot = 2 * blockIdx.x + (ends ? 1 : 0), prow = (w == 2 ? g * kBlockRows : 0) + row;
        float* part = r.part_o + (size_t)slot * r.slot_rows * D + 4 * prow;
        const float inv = rows_inverse<C>(m2, l2, v_scale);
        const uint32_t own = tl + C::kOCol + g * D, other = tl + C::kOCol + (NG == 2 ? (g ^ 1) * D : 0);
        const int c_lo = joint ? g * (D / 2) : 0, c_hi = joint ? c_lo + D / 2 : D;
        if (__any_sync(0xffffffffu, out_row >= 0)) {
#pragma unroll 1
          for (int c0 = c_lo; c0 < c_hi; c0 += 16) {
            float o[16];
            {
              uint32_t x[16];
              if (has_own) {
                tmem_ld_x16(own + c0, x);
                tmem_wait_ld();
              }
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] = has_own && l2 != 0.f && f0 != 0.f ? __uint_as_float(x[c]) * f0 : 0.f;
              if (has_other) {
                tmem_ld_x16(other + c0, x);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 16; ++c)
                  if (f1 != 0.f) o[c] += __uint_as_float(x[c]) * f1;
              }
            }
            if (out_row >= 0) {
              if (whole) {
                uint4* dst = reinterpret_cast<uint4*>(r.out + (size_t)out_row * D + c0);
#pragma unroll
                for (int c = 0; c < 16; c += 8) {
                  uint4 y;
                  uint32_t* yw = &y.x;
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    yw[e] = pack2<Src::kOutF16>(o[o_column<Src>(c + 2 * e)] * inv, o[o_column<Src>(c + 2 * e + 1)] * inv);
                  dst[c / 8] = y;
                }
              } else {
#pragma unroll
                for (int c = 0; c < 16; c += 4)
                  *reinterpret_cast<float4*>(part + (size_t)(c0 + c) * r.slot_rows) =
                      make_float4(o[o_column<Src>(c)], o[o_column<Src>(c + 1)], o[o_column<Src>(c + 2)], o[o_column<Src>(c + 3)]);
              }
            }
          }
          if (out_row >= 0 && (!joint || g == 0)) {
            if (!whole)
              r.part_ml[(size_t)slot * r.slot_rows + prow] = make_float2(m2, l2);
            else if (r.lse)
              r.lse[out_row] = rows_lse<C>(m2, l2);
          }
        }
        if (joint) {  // no P of the next segment before both groups have read both states
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars.at(Bars::kXDone));
          if (!(ok = bars.warp_wait(bars.at(Bars::kXDone), par & kParX ? 1 : 0))) break;
          par ^= kParX;
        }
        if (C::NB == 2 && share.uses > 1) par ^= kParPV2;
        if (tiles & 1) par ^= kParT;
        par ^= kParSeg;
        n += share.uses;
      }
    }
  }

  if (warp == C::kSrcWarp) {
    // ---- rows that no item covers: zeros, every CTA's warp its share of them
    const int R = r.G() * r.Nq;
    for (int b0 = 0; b0 < r.B; b0 += 32) {
      int from = R;
      if (b0 + lane < r.B) {
        const typename Src::Seq s(p, b0 + lane);
        from = s.tiles > 0 ? min(R, s.blocks * kBlockRows) : 0;
      }
      for (unsigned todo = __ballot_sync(0xffffffffu, from < R); todo; todo &= todo - 1) {
        const int k = __ffs(todo) - 1, b = b0 + k, first = __shfl_sync(0xffffffffu, from, k);
        const long long n = (long long)(R - first) * r.Hkv * (D / 8);
        for (long long i = blockIdx.x * 32 + lane; i < n; i += gridDim.x * 32) {
          const long long y = rows_quotient(i, D / 8);
          const int c = (int)(i % (D / 8)), h = (int)rows_quotient(y, R - first), P = first + (int)(y - (long long)h * (R - first));
          const size_t row = ((size_t)b * r.Hq + h * r.G() + P % r.G()) * r.Nq + P / r.G();
          *reinterpret_cast<uint4*>(r.out + row * D + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
          if (c == 0 && r.lse) r.lse[row] = -INFINITY;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of the item that begins in CTA blockIdx.x of the first kernel and goes on behind it,
// in order: a warp takes 32 rows, one per lane, and 16 channels of them.
constexpr int kRowJoinThreads = 256;
template <class Src>
__global__ void __launch_bounds__(kRowJoinThreads) rows_join_kernel(const __grid_constant__ typename Src::Params p) {
  using C = typename Src::Cfg;
  constexpr int D = C::D, kCols = D / 16, kAhead = 4;  // parts whose loads are under way together
  const RowParams& r = p.r;
  const int lane = threadIdx.x & 31, task = blockIdx.y * (kRowJoinThreads / 32) + (threadIdx.x >> 5);
  const int row = task / kCols * 32 + lane, c0 = task % kCols * 16;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const SplitRec rec = r.rec[blockIdx.x];
  if (rec.n == 0 || task / kCols * 32 >= rec.w * kBlockRows) return;
  const RowCut cut(rec.total, rec.ctas);
  const long long uses = (long long)rec.n * rec.w;
  float acc[16], M = -INFINITY, L = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) acc[k] = 0.f;
  const long long begin = rec.first + Src::kItemCost;  // of its uses in the list
  for (int cta = blockIdx.x; cut.first(cta) - begin < uses; cta += kAhead) {
    float2 ml[kAhead];
    float4 o[kAhead][4];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      // the tiles t0 .. t1-1 of CTA cta + k
      const long long a = cut.first(cta + k) - begin, e = cut.first(cta + k + 1) - begin;
      const int t0 = a <= 0 ? 0 : (int)((a < uses ? a : uses) >> (rec.w - 1));
      const int t1 = e <= 0 ? 0 : (int)((e < uses ? e : uses) >> (rec.w - 1));
      if (t0 == 0 && t1 == rec.n) return;  // it has the item alone, and wrote it
      ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int c = 0; c < 4; ++c) o[k][c] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t1 > t0) {
        const size_t slot = 2 * (size_t)(cta + k) + (t1 == rec.n ? 1 : 0);
        ml[k] = r.part_ml[slot * r.slot_rows + row];
        const float* src = r.part_o + slot * r.slot_rows * D + 4 * row;
#pragma unroll
        for (int c = 0; c < 4; ++c) o[k][c] = *reinterpret_cast<const float4*>(src + (size_t)(c0 + 4 * c) * r.slot_rows);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const float mx = fmaxf(M, ml[k].x);
      const float fo = L == 0.f ? 0.f : ex2_approx(M - mx);
      const float f = ml[k].y == 0.f ? 0.f : ex2_approx(ml[k].x - mx);  // (a NaN sum goes on to the output)
      M = mx;
      L = fmaf(f, ml[k].y, L * fo);  // (also with f = 0: a part of scores that are no numbers has no maximum, but a NaN sum)
#pragma unroll
      for (int c = 0; c < 4; ++c) {  // (a part without weight may hold anything)
        acc[4 * c] = f == 0.f ? acc[4 * c] * fo : fmaf(f, o[k][c].x, acc[4 * c] * fo);
        acc[4 * c + 1] = f == 0.f ? acc[4 * c + 1] * fo : fmaf(f, o[k][c].y, acc[4 * c + 1] * fo);
        acc[4 * c + 2] = f == 0.f ? acc[4 * c + 2] * fo : fmaf(f, o[k][c].z, acc[4 * c + 2] * fo);
        acc[4 * c + 3] = f == 0.f ? acc[4 * c + 3] * fo : fmaf(f, o[k][c].w, acc[4 * c + 3] * fo);
      }
    }
  }
  const typename Src::Seq seq(p, rec.b);
  typename Src::Row me;
  me.set(p, seq, rec.b, rec.h, rec.rb * kBlockRows + row);
  if (me.out_row < 0) return;
  const float inv = rows_inverse<C>(M, L, me.v_scale);
  uint32_t y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) y[k] = pack2<Src::kOutF16>(acc[2 * k] * inv, acc[2 * k + 1] * inv);
  uint4* dst = reinterpret_cast<uint4*>(r.out + (size_t)me.out_row * D + c0);
  dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
  dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
  if (c0 == 0 && r.lse) r.lse[me.out_row] = rows_lse<C>(M, L);
}

__host__ inline size_t rows_align(size_t x) { return (x + 255) / 256 * 256; }
// Rows of a part's slot: those of the largest item.
__host__ inline bool rows_two_blocks(int rows, int d) { return d == 128 && rows > kBlockRows; }
// (one CTA per SM with slots of two blocks, or, d <= 128, two per SM with slots of one)
__host__ inline size_t rows_workspace(int rows, int d) {
  const size_t ctas = kRowSms * (d <= 128 && !rows_two_blocks(rows, d) ? 2 : 1);
  const size_t slots = 2 * ctas * (rows_two_blocks(rows, d) ? 2 : 1) * kBlockRows;
  return rows_align(ctas * sizeof(SplitRec)) + rows_align(slots * 8) + slots * d * 4;
}
// What the sources' entry points take alike.
__host__ inline bool rows_bad_heads(int B, int Hq, int Hkv, int Nq) {
  return B < 1 || B > kMaxRowSeqs || Hq < 1 || Hkv < 1 || Hq % Hkv || Hkv > (1 << 16) || Nq < 1 ||
         (long long)(Hq / Hkv) * Nq > (1 << 20) || (long long)B * Hq * Nq > 0x7FFFFFF0;
}

template <class Src>
cudaError_t launch_rows(typename Src::Params prm, void* ws, cudaStream_t stream) {
  RowParams& r = prm.r;
  const int rows = r.G() * r.Nq, D = Src::Cfg::D;
  constexpr int kCtas = Src::Cfg::kCtas;
  r.slot_rows = Src::Cfg::NG * kBlockRows;
  uint8_t* w = static_cast<uint8_t*>(ws);
  const size_t slots = 2 * (size_t)kCtas * r.slot_rows;
  r.rec = (SplitRec*)w;
  w += rows_align(kCtas * sizeof(SplitRec));
  r.part_ml = (float2*)w;
  w += rows_align(slots * 8);
  r.part_o = (float*)w;
  static std::atomic<uint64_t> ready{0};  // the attribute, once per device (a bit each)
  cudaError_t e;
  int dev = 0;
  if ((e = cudaGetDevice(&dev))) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || !(ready.load() & bit)) {
    if ((e = cudaFuncSetAttribute(rows_kernel<Src>, cudaFuncAttributeMaxDynamicSharedMemorySize, Src::kSmem))) return e;
    if (dev <= 63) ready.fetch_or(bit);
  }
  cudaLaunchAttribute at{};  // both kernels begin while the one before them ends, and wait for it where they read
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kCtas);
  cfg.blockDim = dim3(Src::kThreads);
  cfg.dynamicSmemBytes = Src::kSmem;
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, rows_kernel<Src>, prm))) return e;
  const int most = r.slot_rows < rows ? r.slot_rows : rows;
  cfg.gridDim = dim3(kCtas, (unsigned)((most + 31) / 32 * (D / 16) + 7) / 8);
  cfg.blockDim = dim3(kRowJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, rows_join_kernel<Src>, prm);
}

}  // namespace
}  // namespace apa
