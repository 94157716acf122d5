// apa_cache.cu -- the 4-bit K/V cache: block tables and slot maps from request
// lengths, quantizing tokens into pages, and reading them back.
#include "../../include/apa.h"
#include "apa_internal.h"
#include "cache_page.cuh"
#include "quant_tile.cuh"
#include "tc.cuh"

namespace apa {
namespace {

// ------------------------------------------------------------------ tables
// What bounds it is latency: a few dependent loads behind a launch.  One cluster (a
// single CTA for a decoding step).  Every CTA scans the B requests (tokens, pages given back, pages
// taken) for itself, then does its share of the three lists.  No CTA reads what
// another writes: a page taken is looked up in the old stack or, if a request of
// this call gave it back, in that request's table row, which no one writes; the
// entries and stack positions written are ones that nobody reads.  Only the
// stack's count can be input and output at once: it is written after a cluster
// barrier behind every CTA's read of it.  Up to kInline tokens are mapped to slots here,
// one per thread; more of them by a second kernel over the whole GPU, from the table
// and the starts (2^18 prompt tokens: 17 us in the cluster alone).
constexpr int kTabThreads = 1024;
constexpr int kMaxRequests = 8192;
constexpr int kInline = 8192;

struct TablesParams {
  const int32_t *old_lens, *new_lens;
  int B;
  int32_t* table;
  int max_pages;
  int32_t* free_pages;
  int free_capacity;
  const int32_t* free_count;
  int max_tokens;
  int32_t *slots, *positions, *starts, *free_count_out, *status;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// The last index i of [0, n) with a[i] <= x (a[0] = 0 <= x, a not falling).
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int slot_of(int page, int pos) {
  return page < 0 || page >= (1 << 25) ? -1 : page * kTile + pos % kTile;
}

__global__ void __launch_bounds__(kTabThreads) tables_kernel(const TablesParams p) {
  extern __shared__ int tab_smem[];
  int* s_tok = tab_smem;              // [B] tokens of the requests before b
  int* s_give = tab_smem + p.B;       // [B] pages given back by them
  int* s_take = tab_smem + 2 * p.B;   // [B] pages taken by them
  int* s_old = tab_smem + 3 * p.B;    // [B] the lengths
  int* s_new = tab_smem + 4 * p.B;
  __shared__ int warp_sum[3][32];
  __shared__ int carry[3];
  __shared__ unsigned long long total[3];  // in 64 bits: what the checks below go by
  __shared__ int bad;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster_rank(), ncta = (int)cluster_size();
  if (tid < 3) {
    carry[tid] = 0;
    total[tid] = 0;
  }
  if (tid == 0) bad = 0;
  __syncthreads();
  const int count = *p.free_count;
  const long long longest = (long long)p.max_pages * kTile;

  for (int b0 = 0; b0 < p.B; b0 += kTabThreads) {
    const int b = b0 + tid;
    int v[3] = {0, 0, 0};
    if (b < p.B) {
      const int o = p.old_lens[b], n = p.new_lens[b];
      s_old[b] = o;
      s_new[b] = n;
      if (o < 0 || n < 0 || o > longest || n > longest) {
        bad = 1;
      } else {
        const int ho = (int)(((long long)o + kTile - 1) / kTile), hn = (int)(((long long)n + kTile - 1) / kTile);
        v[0] = max(n - o, 0);
        v[1] = max(ho - hn, 0);
        v[2] = max(hn - ho, 0);
      }
    }
    int x[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      x[k] = v[k];
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x[k], s);
        if (lane >= s) x[k] += y;
      }
      // a warp's 32 lengths, each below 2^31, need 36 bits
      unsigned long long w = (unsigned long long)v[k];
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) w += __shfl_xor_sync(0xffffffffu, w, s);
      if (lane == 0) atomicAdd(&total[k], w);
      if (lane == 31) warp_sum[k][warp] = x[k];
    }
    __syncthreads();
    if (warp < 3) {
      int y = warp_sum[warp][lane];
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, s);
        if (lane >= s) y += z;
      }
      const int c = carry[warp];
      __syncwarp();
      const int before = __shfl_up_sync(0xffffffffu, y, 1);
      warp_sum[warp][lane] = c + (lane ? before : 0);
      if (lane == 31) carry[warp] = c + y;
    }
    __syncthreads();
    if (b < p.B) {
      s_tok[b] = warp_sum[0][warp] + x[0] - v[0];
      s_give[b] = warp_sum[1][warp] + x[1] - v[1];
      s_take[b] = warp_sum[2][warp] + x[2] - v[2];
    }
    __syncthreads();
  }

  const long long tokens = (long long)total[0], gives = (long long)total[1], takes = (long long)total[2];
  int st = 0;
  if (bad)
    st = APA_TABLES_LENGTH;
  else if (tokens > p.max_tokens)
    st = APA_TABLES_TOKENS;
  else if (count < 0 || count + gives > p.free_capacity)
    st = APA_TABLES_FREE;
  else if (takes > count + gives)
    st = APA_TABLES_PAGES;
  const int nth = ncta * kTabThreads, me = rank * kTabThreads + tid;
  const int ntok = st ? 0 : (int)tokens;

  // page number x of those taken: off the stack's top, where the pages given back lie
  auto taken = [&](int x) -> int {
    const long long at = count + gives - 1 - x;
    if (at < count) return p.free_pages[at];
    const int y = (int)(at - count);
    const int b = last_at_most(s_give, p.B, y);
    const int hn = (int)(((long long)s_new[b] + kTile - 1) / kTile);
    return p.table[(size_t)b * p.max_pages + hn + (y - s_give[b])];
  };

  if (st == 0) {
    const long long left = count + gives - takes;
    for (int x = me; x < (int)gives; x += nth) {  // given back, and not taken again
      if (count + x >= left) break;
      const int b = last_at_most(s_give, p.B, x);
      const int hn = (int)(((long long)s_new[b] + kTile - 1) / kTile);
      p.free_pages[count + x] = p.table[(size_t)b * p.max_pages + hn + (x - s_give[b])];
    }
    for (int x = me; x < (int)takes; x += nth) {
      const int b = last_at_most(s_take, p.B, x);
      const int ho = (int)(((long long)s_old[b] + kTile - 1) / kTile);
      p.table[(size_t)b * p.max_pages + ho + (x - s_take[b])] = taken(x);
    }
  }
  if (p.max_tokens <= kInline) {
    for (int t = me; t < p.max_tokens; t += nth) {
      int slot = -1, pos = 0;
      if (t < ntok) {
        const int b = last_at_most(s_tok, p.B, t), o = s_old[b];
        const int ho = (int)(((long long)o + kTile - 1) / kTile);
        pos = o + (t - s_tok[b]);
        const int e = pos / kTile;
        slot = slot_of(e < ho ? p.table[(size_t)b * p.max_pages + e] : taken(s_take[b] + (e - ho)), pos);
      }
      p.slots[t] = slot;
      p.positions[t] = pos;
    }
  }
  for (int b = me; b <= p.B; b += nth) p.starts[b] = st ? 0 : (b < p.B ? s_tok[b] : ntok);
  if (ncta > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  if (me == 0) {
    *p.free_count_out = st ? count : (int)(count + gives - takes);
    *p.status = st;
  }
}

// The slots and positions of many tokens, from what tables_kernel left: four tokens per
// thread, one search for them, and a page looked up when it changes.
__global__ void __launch_bounds__(256) slots_kernel(const TablesParams p, bool vec) {
  const int t0 = 4 * (blockIdx.x * 256 + threadIdx.x);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (t0 >= p.max_tokens) return;
  const int ntok = p.starts[p.B];  // 0 where nothing was changed
  int slot[4], pos[4], b = 0, next = 0, start = 0, o = 0, entry = -1, page = -1;
  if (t0 < ntok) {
    b = last_at_most(p.starts, p.B, t0);
    next = p.starts[b + 1];
    start = p.starts[b];
    o = p.old_lens[b];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int t = t0 + k;
    slot[k] = -1;
    pos[k] = 0;
    if (t >= ntok) continue;
    while (t >= next) {  // the next request with new tokens
      start = next;
      next = p.starts[++b + 1];
      o = p.old_lens[b];
      entry = -1;
    }
    pos[k] = o + (t - start);
    if (pos[k] / kTile != entry) {
      entry = pos[k] / kTile;
      page = p.table[(size_t)b * p.max_pages + entry];
    }
    slot[k] = slot_of(page, pos[k]);
  }
  if (vec && t0 + 3 < p.max_tokens) {
    *reinterpret_cast<int4*>(p.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
  } else {
    for (int k = 0; k < 4 && t0 + k < p.max_tokens; ++k) {
      p.slots[t0 + k] = slot[k];
      p.positions[t0 + k] = pos[k];
    }
  }
}

// ------------------------------------------------------------------ write, read
// A CTA takes kWin tokens of one head.  Four tokens in consecutive slots from a multiple
// of 4 on (as prompts have them, wherever they start) are a quad: the four keys whose V
// codes share 32-bit words.  A thread takes 16 channels of a quad's K or of its V; for V
// it transposes 4 keys x 8 code bytes in registers, and a warp's stores (or loads) are
// whole 64-byte runs.  Tokens that are in no quad (decoding: one key per sequence) go
// byte by byte.  Both move 2 + 9/16 bytes per value.  Reading is bound by HBM (40 000 tokens of
// 8 heads, d = 128: 34 us, 0.9 of the copy rate).  Writing a prompt (16 411 tokens: 23 us, 1.8 times
// its bytes' time) is bound by the phases of a CTA, which come one after the other in 2.7 waves:
// slots, sort, barrier, loads, stores.  It takes as long without its arithmetic or its stores.
constexpr int kCacheThreads = 256;
// 32 bytes in one access (sm_100 on), if the address allows
__device__ __forceinline__ void ld32(const uint16_t* p, bool wide, uint32_t* w) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
    return;
  }
  const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
  w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}
__device__ __forceinline__ void st32(uint16_t* p, bool wide, const uint32_t* w) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
    return;
  }
  reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}


struct Window {
  int quad[16], single[64];  // first token of each quad; the other tokens in use
  int quads, singles;
};
// Fills w and s_slot for n <= 64 tokens: one warp's work.  skip: leaves out tokens without
// a slot in the pool (else they are singles).
__device__ __forceinline__ void sort_window(Window& w, int* s_slot, const int32_t* slots, int n, int num_pages,
                                            bool skip, int* err) {
  const int lane = threadIdx.x & 31;
  int slot[2];
  bool quad[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = 32 * k + lane;
    slot[k] = i < n ? slots[i] : -1;
    s_slot[i] = slot[k];
    if (slot[k] >= 0 && slot[k] / kTile >= num_pages) {
      if (err) atomicCAS(err, 0, APA_DEVERR_BOUNDS);
      slot[k] = -1;
    }
  }
  __syncwarp();
  unsigned long long starts = 0, singles = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = 32 * k + lane;
    quad[k] = slot[k] >= 0 && slot[k] % 4 == 0 && i + 3 < n && s_slot[i + 1] == slot[k] + 1 &&
              s_slot[i + 2] == slot[k] + 2 && s_slot[i + 3] == slot[k] + 3;
    starts |= (unsigned long long)__ballot_sync(0xffffffffu, quad[k]) << (32 * k);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = 32 * k + lane, f = i - (slot[k] & 3);
    const bool member = slot[k] >= 0 && f >= 0 && ((starts >> f) & 1);
    const bool single = i < n && !member && (slot[k] >= 0 || !skip);
    singles |= (unsigned long long)__ballot_sync(0xffffffffu, single) << (32 * k);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = 32 * k + lane;
    const unsigned long long below = (1ull << i) - 1;
    if (quad[k]) w.quad[__popcll(starts & below)] = i;
    if ((singles >> i) & 1) w.single[__popcll(singles & below)] = i;
  }
  if (lane == 0) {
    w.quads = __popcll(starts);
    w.singles = __popcll(singles);
  }
}

// 4 x 4 bytes, transposed: byte j of out[i] is byte i of in[j].
__device__ __forceinline__ void transpose4(const uint32_t* in, uint32_t* out) {
  const uint32_t a = __byte_perm(in[0], in[1], 0x5140), b = __byte_perm(in[2], in[3], 0x5140);
  const uint32_t c = __byte_perm(in[0], in[1], 0x7362), d = __byte_perm(in[2], in[3], 0x7362);
  out[0] = __byte_perm(a, b, 0x5410);
  out[1] = __byte_perm(a, b, 0x7632);
  out[2] = __byte_perm(c, d, 0x5410);
  out[3] = __byte_perm(c, d, 0x7632);
}
// Codes of 16 channels (two words of eight nibbles) <-> the eight code bytes of V, channel
// g in the low and 8 + g in the high nibble of byte g.
__device__ __forceinline__ uint2 v_bytes(uint2 codes) {
  const uint32_t even = (codes.x & 0x0F0F0F0Fu) | ((codes.y & 0x0F0F0F0Fu) << 4);   // g = 0, 2, 4, 6
  const uint32_t odd = ((codes.x >> 4) & 0x0F0F0F0Fu) | (codes.y & 0xF0F0F0F0u);    // g = 1, 3, 5, 7
  return make_uint2(__byte_perm(even, odd, 0x5140), __byte_perm(even, odd, 0x7362));
}
__device__ __forceinline__ uint2 v_codes(uint2 bytes) {
  const uint32_t even = __byte_perm(bytes.x, bytes.y, 0x6420), odd = __byte_perm(bytes.x, bytes.y, 0x7531);
  return make_uint2((even & 0x0F0F0F0Fu) | ((odd & 0x0F0F0F0Fu) << 4),
                    ((even >> 4) & 0x0F0F0F0Fu) | (odd & 0xF0F0F0F0u));
}

struct WriteParams {
  const uint16_t *k, *v;
  long long ks_h, ks_t, vs_h, vs_t;
  int H, T, win;
  bool wide;          // every row is 32-byte aligned
  const int32_t* slots;
  uint8_t* pages;
  int num_pages;
  const float *k_scale, *v_scale;
  int* err;
};

// Eight values -> a word of E2M1 codes.
__device__ __forceinline__ uint32_t e2m1_word(const float* x) {
  uint32_t w;
  asm("{\n.reg .b8 a, b, c, d;\n"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      "mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(w)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return w;
}
// The largest of three, NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// quant16's steps on 16 values in memory.  s6 = fp32(6 s); inv[b] = fp32(1 / fp32(b s)), 0 for
// b = 0: 127 reciprocals per CTA and head instead of one per 16 values.  A group with a NaN gets
// the scale code 0x7F, which is NaN, and codes of 0, so that it reads back as NaN.
template <bool F16>
__device__ __forceinline__ uint32_t quant_row(const uint16_t* src, bool wide, float s6, const float* inv, uint2* codes) {
  uint32_t w[8];
  ld32(src, wide, w);
  float x[16];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 f = unpack2<F16>(w[e]);
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
  float a = max3_nan(fabsf(x[0]), fabsf(x[1]), fabsf(x[2]));
#pragma unroll
  for (int e = 3; e < 15; e += 2) a = max3_nan(a, fabsf(x[e]), fabsf(x[e + 1]));
  a = max3_nan(a, fabsf(x[15]), 0.f);
  const uint32_t sb = cvt_ue4m3(__fdiv_rn(a, s6)) & 127u;  // (no sign, whatever the scale)
  const float f = inv[sb];
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = __fmul_rn(x[e], f);
  const bool some = sb - 1u < 126u;  // neither 0 nor NaN
  codes->x = some ? e2m1_word(x) : 0u;
  codes->y = some ? e2m1_word(x + 8) : 0u;
  return sb;
}

template <int D, bool F16>
__global__ void __launch_bounds__(kCacheThreads, 5) write_kernel(const WriteParams p) {
  constexpr int N = D / 16;
  __shared__ Window w;
  __shared__ int s_slot[64];
  __shared__ float s_inv[2][128];
  const int h = blockIdx.x % p.H, t0 = blockIdx.x / p.H * p.win, n = min(p.win, p.T - t0);
  const uint16_t *k = p.k + h * p.ks_h + t0 * p.ks_t, *v = p.v + h * p.vs_h + t0 * p.vs_t;
  const float sk = p.k_scale[h], sv = p.v_scale[h];
  const float s6[2] = {__fmul_rn(6.f, sk), __fmul_rn(6.f, sv)};
  if (threadIdx.x < 32) {
    sort_window(w, s_slot, p.slots + t0, n, p.num_pages, true, p.err);
  } else {  // the values come nearer meanwhile, 128 bytes per thread, and the reciprocals are made
    constexpr int kLines = D / 64;
    for (int i = threadIdx.x - 32; i < n * 2 * kLines; i += kCacheThreads - 32) {
      const int line = i % kLines, tok = i / kLines % n;
      const uint16_t* a = (i < n * kLines ? k + tok * p.ks_t : v + tok * p.vs_t) + 64 * line;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a));
    }
    for (int i = threadIdx.x - 32; i < 256; i += kCacheThreads - 32)
      s_inv[i >> 7][i & 127] = i & 127 ? __frcp_rn(__fmul_rn(ue4m3_value(i & 127), i < 128 ? sk : sv)) : 0.f;
  }
  __syncthreads();
  uint8_t* head = p.pages + (size_t)h * page_head_bytes(D);
  const size_t page_bytes = (size_t)p.H * page_head_bytes(D);
  const int nq = w.quads * 2 * N, ns = w.singles * 2 * N;
  auto block = [&](int slot) { return head + slot / kTile * page_bytes + slot % kTile / kBlkKeys * blk_bytes(D); };
  for (int i = threadIdx.x; i < nq; i += kCacheThreads) {
    const int t = i % N, tok = w.quad[i / N % w.quads], slot = s_slot[tok], ki = slot % kBlkKeys;
    uint8_t* blk = block(slot);
    uint2 codes[4];
    uint32_t sb[4];
    if (i < w.quads * N) {
#pragma unroll
      for (int j = 0; j < 4; ++j) sb[j] = quant_row<F16>(k + (tok + j) * p.ks_t + 16 * t, p.wide, s6[0], s_inv[0], codes + j);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        *reinterpret_cast<uint2*>(blk + (ki + j) * (D / 2) + 8 * t) = codes[j];
        blk[ks_byte(D, ki + j, t)] = (uint8_t)sb[j];
      }
    } else {
      uint32_t lo[4], hi[4], wl[4], wh[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sb[j] = quant_row<F16>(v + (tok + j) * p.vs_t + 16 * t, p.wide, s6[1], s_inv[1], codes + j);
        const uint2 y = v_bytes(codes[j]);
        lo[j] = y.x;
        hi[j] = y.y;
      }
      transpose4(lo, wl);
      transpose4(hi, wh);
#pragma unroll
      for (int g = 0; g < 8; ++g)
        *reinterpret_cast<uint32_t*>(blk + v_byte(D, ki, t, g)) = g < 4 ? wl[g & 3] : wh[g & 3];
      *reinterpret_cast<uint32_t*>(blk + vs_byte(D, ki, t)) = sb[0] | sb[1] << 8 | sb[2] << 16 | sb[3] << 24;
    }
  }
  // (from the threads that the quads' last round left idle)
  for (int i = (threadIdx.x + kCacheThreads - nq % kCacheThreads) % kCacheThreads; i < ns; i += kCacheThreads) {
    const int t = i % N, tok = w.single[i / N % w.singles], slot = s_slot[tok], ki = slot % kBlkKeys;
    uint8_t* blk = block(slot);
    uint2 codes;
    if (i < w.singles * N) {
      const uint32_t sb = quant_row<F16>(k + tok * p.ks_t + 16 * t, p.wide, s6[0], s_inv[0], &codes);
      *reinterpret_cast<uint2*>(blk + ki * (D / 2) + 8 * t) = codes;
      blk[ks_byte(D, ki, t)] = (uint8_t)sb;
    } else {
      const uint32_t sb = quant_row<F16>(v + tok * p.vs_t + 16 * t, p.wide, s6[1], s_inv[1], &codes);
      const uint2 y = v_bytes(codes);
#pragma unroll
      for (int g = 0; g < 8; ++g) blk[v_byte(D, ki, t, g)] = (uint8_t)((g < 4 ? y.x : y.y) >> (8 * (g & 3)));
      blk[vs_byte(D, ki, t)] = (uint8_t)sb;
    }
  }
}

struct ReadParams {
  const uint8_t* pages;
  int num_pages, H, T, win;
  bool wide;
  const int32_t* slots;
  const float *k_scale, *v_scale;
  uint16_t *k, *v;
  int* err;
};

// 16 values: fp32(fp32(E2M1 * UE4M3) * s) rounded to the type.
template <bool F16>
__device__ __forceinline__ void put_row(uint16_t* dst, bool wide, uint2 codes, uint32_t sb, float s) {
  // the first product is exact in FP16 (6 bits, 2^-10 .. 2688)
  uint32_t b2, out[8];
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b2) : "h"((uint16_t)(sb | sb << 8)));
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint32_t h;
    asm("{\n.reg .b8 t;\ncvt.u8.u32 t, %1;\ncvt.rn.f16x2.e2m1x2 %0, t;\nmul.rn.f16x2 %0, %0, %2;\n}"
        : "=r"(h)
        : "r"((e < 4 ? codes.x : codes.y) >> (8 * (e & 3))), "r"(b2));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
    out[e] = pack2<F16>(__fmul_rn(x.x, s), __fmul_rn(x.y, s));
  }
  st32(dst, wide, out);
}

template <int D, bool F16>
__global__ void __launch_bounds__(kCacheThreads, 8) read_kernel(const ReadParams p) {
  constexpr int N = D / 16;
  __shared__ Window w;
  __shared__ int s_slot[64];
  const int h = blockIdx.x % p.H, t0 = blockIdx.x / p.H * p.win;
  const float sk = p.k_scale[h], sv = p.v_scale[h];
  if (threadIdx.x < 32) sort_window(w, s_slot, p.slots + t0, min(p.win, p.T - t0), p.num_pages, false, p.err);
  __syncthreads();
  const size_t row0 = (size_t)h * p.T + t0;
  const uint8_t* head = p.pages + (size_t)h * page_head_bytes(D);
  const size_t page_bytes = (size_t)p.H * page_head_bytes(D);
  const int nq = w.quads * 2 * N, ns = w.singles * 2 * N;
  auto block = [&](int slot) { return head + slot / kTile * page_bytes + slot % kTile / kBlkKeys * blk_bytes(D); };
  for (int i = threadIdx.x; i < nq; i += kCacheThreads) {
    const int t = i % N, tok = w.quad[i / N % w.quads], slot = s_slot[tok], ki = slot % kBlkKeys;
    const uint8_t* blk = block(slot);
    if (i < w.quads * N) {
      uint2 codes[4];
      uint32_t sb[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        codes[j] = *reinterpret_cast<const uint2*>(blk + (ki + j) * (D / 2) + 8 * t);
        sb[j] = blk[ks_byte(D, ki + j, t)];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) put_row<F16>(p.k + (row0 + tok + j) * D + 16 * t, p.wide, codes[j], sb[j], sk);
    } else {
      uint32_t wl[4], wh[4], lo[4], hi[4];
#pragma unroll
      for (int g = 0; g < 8; ++g) (g < 4 ? wl : wh)[g & 3] = *reinterpret_cast<const uint32_t*>(blk + v_byte(D, ki, t, g));
      const uint32_t sb = *reinterpret_cast<const uint32_t*>(blk + vs_byte(D, ki, t));
      transpose4(wl, lo);
      transpose4(wh, hi);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        put_row<F16>(p.v + (row0 + tok + j) * D + 16 * t, p.wide, v_codes(make_uint2(lo[j], hi[j])), (sb >> (8 * j)) & 255u, sv);
    }
  }
  // (from the threads that the quads' last round left idle)
  for (int i = (threadIdx.x + kCacheThreads - nq % kCacheThreads) % kCacheThreads; i < ns; i += kCacheThreads) {
    const int t = i % N, tok = w.single[i / N % w.singles], slot = s_slot[tok], ki = slot % kBlkKeys;
    const bool of_k = i < w.singles * N;
    uint2 codes = make_uint2(0u, 0u);  // without a slot in the pool: zeros
    uint32_t sb = 0;
    if (slot >= 0 && slot / kTile < p.num_pages) {
      const uint8_t* blk = block(slot);
      if (of_k) {
        codes = *reinterpret_cast<const uint2*>(blk + ki * (D / 2) + 8 * t);
        sb = blk[ks_byte(D, ki, t)];
      } else {
#pragma unroll
        for (int g = 0; g < 8; ++g) (g < 4 ? codes.x : codes.y) |= (uint32_t)blk[v_byte(D, ki, t, g)] << (8 * (g & 3));
        codes = v_codes(codes);
        sb = blk[vs_byte(D, ki, t)];
      }
    }
    put_row<F16>((of_k ? p.k : p.v) + (row0 + tok) * D + 16 * t, p.wide, codes, sb, of_k ? sk : sv);
  }
}

// Tokens per CTA: 64, so that few quads are cut at a window's end; with little work, 16, for
// more CTAs than SMs.
int window_tokens(long long T, int H) { return T * H >= 64 * 152 * 4 ? 64 : 16; }

int check_cache(int dtype, int Hkv, int T, int d, int num_pages) {
  if (Hkv < 1 || T < 0 || num_pages < 1 || num_pages >= (1 << 25) || Hkv > (1 << 16)) return APA_ERR_SHAPE;
  if (d != 64 && d != 128 && d != 256) return APA_ERR_HEAD_DIM;
  if (dtype != APA_DTYPE_BF16 && dtype != APA_DTYPE_F16) return APA_ERR_DTYPE;
  return APA_OK;
}

}  // namespace
}  // namespace apa

using namespace apa;

extern "C" {

size_t apa_cache_page_bytes(int Hkv, int d) {
  if (Hkv < 1 || (d != 64 && d != 128 && d != 256)) return 0;
  return (size_t)Hkv * page_head_bytes(d);
}

int apa_cache_tables(const int32_t* old_lens, const int32_t* new_lens, int B, int32_t* block_table, int max_pages,
                     int32_t* free_pages, int free_capacity, const int32_t* free_count, int max_tokens, int32_t* slots,
                     int32_t* positions, int32_t* starts, int32_t* free_count_out, int32_t* status,
                     cudaStream_t stream) {
  if (!old_lens || !new_lens || !block_table || !free_pages || !free_count || !starts || !free_count_out || !status)
    return APA_ERR_NULL;
  if (max_tokens > 0 && (!slots || !positions)) return APA_ERR_NULL;
  if (B < 1 || B > kMaxRequests || max_pages < 1 || max_pages >= (1 << 25) || free_capacity < 1 || max_tokens < 0 || max_tokens > (1 << 30))
    return APA_ERR_SHAPE;
  TablesParams prm{old_lens,   new_lens,   B,     block_table, max_pages, free_pages,     free_capacity,
                   free_count, max_tokens, slots, positions,   starts,    free_count_out, status};
  int ncta = 1;
  while (ncta < 8 && ncta * 4096 < max_tokens) ncta *= 2;
  const int smem = 5 * B * (int)sizeof(int);
  if (smem > 40 * 1024 &&  // (48 KB with the static arrays need no leave)
      cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 5 * kMaxRequests * 4))
    return APA_ERR_CUDA;
  if (ncta == 1) {  // (a plain launch takes the host less time)
    tables_kernel<<<1, kTabThreads, smem, stream>>>(prm);
    return cudaGetLastError() == cudaSuccess ? APA_OK : APA_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ncta);
  cfg.blockDim = dim3(kTabThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = ncta;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, tables_kernel, prm) != cudaSuccess) return APA_ERR_CUDA;
  if (max_tokens <= kInline) return APA_OK;
  // (more than kInline tokens: ncta > 1)
  cudaLaunchConfig_t cfg2{};
  cfg2.gridDim = dim3((max_tokens + 1023) / 1024);
  cfg2.blockDim = dim3(256);
  cfg2.stream = stream;
  cudaLaunchAttribute at2{};
  at2.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at2.val.programmaticStreamSerializationAllowed = 1;
  cfg2.attrs = &at2;
  cfg2.numAttrs = 1;
  const bool vec = (((uintptr_t)slots | (uintptr_t)positions) & 15) == 0;
  return cudaLaunchKernelEx(&cfg2, slots_kernel, prm, vec) == cudaSuccess ? APA_OK : APA_ERR_CUDA;
}

int apa_cache_write(const void* k, const void* v, int dtype, int Hkv, int T, int d, long long k_head_stride,
                    long long k_token_stride, long long v_head_stride, long long v_token_stride, const int32_t* slots,
                    uint8_t* pages, int num_pages, const float* k_scale, const float* v_scale, cudaStream_t stream) {
  const int st = check_cache(dtype, Hkv, T, d, num_pages);
  if (st) return st;
  if (T == 0) return APA_OK;
  if (!k || !v || !slots || !pages || !k_scale || !v_scale) return APA_ERR_NULL;
  // (the stride of an axis of length 1 is never used: any value will do)
  if (Hkv == 1) k_head_stride = v_head_stride = 0;
  if (T == 1) k_token_stride = v_token_stride = 0;
  if ((((uintptr_t)k | (uintptr_t)v | (uintptr_t)pages) & 15) ||
      ((k_head_stride | k_token_stride | v_head_stride | v_token_stride) & 7))
    return APA_ERR_ALIGN;
  const int win = window_tokens(T, Hkv);
  const bool wide = ((((uintptr_t)k | (uintptr_t)v) & 31) | ((k_head_stride | k_token_stride | v_head_stride | v_token_stride) & 15)) == 0;
  WriteParams prm{(const uint16_t*)k, (const uint16_t*)v, k_head_stride, k_token_stride, v_head_stride,
                  v_token_stride,     Hkv,                T,             win, wide,      slots,
                  pages,              num_pages,          k_scale,       v_scale,        device_error_word()};
  const long long blocks = ((long long)T + win - 1) / win * Hkv;
  if (blocks > 0x7FFFFFFFll) return APA_ERR_SHAPE;
  const bool f16 = dtype == APA_DTYPE_F16;
  auto go = [&](auto kern) { kern<<<(unsigned)blocks, kCacheThreads, 0, stream>>>(prm); };
  switch (d) {
    case 64: f16 ? go(write_kernel<64, true>) : go(write_kernel<64, false>); break;
    case 128: f16 ? go(write_kernel<128, true>) : go(write_kernel<128, false>); break;
    case 256: f16 ? go(write_kernel<256, true>) : go(write_kernel<256, false>); break;
  }
  return cudaGetLastError() == cudaSuccess ? APA_OK : APA_ERR_CUDA;
}

int apa_cache_read(const uint8_t* pages, int num_pages, int dtype, int Hkv, int T, int d, const int32_t* slots,
                   const float* k_scale, const float* v_scale, void* k, void* v, cudaStream_t stream) {
  const int st = check_cache(dtype, Hkv, T, d, num_pages);
  if (st) return st;
  if (T == 0) return APA_OK;
  if (!k || !v || !slots || !pages || !k_scale || !v_scale) return APA_ERR_NULL;
  if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)pages) & 15) return APA_ERR_ALIGN;
  const int win = window_tokens(T, Hkv);
  const bool wide = (((uintptr_t)k | (uintptr_t)v) & 31) == 0;
  ReadParams prm{pages, num_pages, Hkv, T, win, wide, slots, k_scale, v_scale, (uint16_t*)k, (uint16_t*)v, device_error_word()};
  const long long blocks = ((long long)T + win - 1) / win * Hkv;
  if (blocks > 0x7FFFFFFFll) return APA_ERR_SHAPE;
  const bool f16 = dtype == APA_DTYPE_F16;
  auto go = [&](auto kern) { kern<<<(unsigned)blocks, kCacheThreads, 0, stream>>>(prm); };
  switch (d) {
    case 64: f16 ? go(read_kernel<64, true>) : go(read_kernel<64, false>); break;
    case 128: f16 ? go(read_kernel<128, true>) : go(read_kernel<128, false>); break;
    case 256: f16 ? go(read_kernel<256, true>) : go(read_kernel<256, false>); break;
  }
  return cudaGetLastError() == cudaSuccess ? APA_OK : APA_ERR_CUDA;
}

}  // extern "C"
