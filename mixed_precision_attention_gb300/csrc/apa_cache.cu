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
// One cluster.  Every CTA scans the B requests (tokens, pages given back, pages
// taken) for itself, then does its share of the three lists.  No CTA reads what
// another writes: a page taken is looked up in the old stack or, if a request of
// this call gave it back, in that request's table row, which no one writes; the
// entries and stack positions written are ones that nobody reads.  Only the
// stack's count can be input and output at once: it is written after a cluster
// barrier behind every CTA's read of it.
constexpr int kTabThreads = 1024;
constexpr int kMaxRequests = 8192;

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

__global__ void __launch_bounds__(kTabThreads) tables_kernel(const TablesParams p) {
  extern __shared__ int tab_smem[];
  int* s_tok = tab_smem;              // [B] tokens of the requests before b
  int* s_give = tab_smem + p.B;       // [B] pages given back by them
  int* s_take = tab_smem + 2 * p.B;   // [B] pages taken by them
  __shared__ int warp_sum[3][32];
  __shared__ int carry[3];
  __shared__ unsigned long long total[3];  // in 64 bits: what the checks below go by
  __shared__ int bad;

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
    const int hn = (int)(((long long)p.new_lens[b] + kTile - 1) / kTile);
    return p.table[(size_t)b * p.max_pages + hn + (y - s_give[b])];
  };

  if (st == 0) {
    const long long left = count + gives - takes;
    for (int x = me; x < (int)gives; x += nth) {  // given back, and not taken again
      if (count + x >= left) break;
      const int b = last_at_most(s_give, p.B, x);
      const int hn = (int)(((long long)p.new_lens[b] + kTile - 1) / kTile);
      p.free_pages[count + x] = p.table[(size_t)b * p.max_pages + hn + (x - s_give[b])];
    }
    for (int x = me; x < (int)takes; x += nth) {
      const int b = last_at_most(s_take, p.B, x);
      const int ho = (int)(((long long)p.old_lens[b] + kTile - 1) / kTile);
      p.table[(size_t)b * p.max_pages + ho + (x - s_take[b])] = taken(x);
    }
  }
  for (int t = me; t < p.max_tokens; t += nth) {
    int slot = -1, pos = 0;
    if (t < ntok) {
      const int b = last_at_most(s_tok, p.B, t);
      const int o = p.old_lens[b];
      const int ho = (int)(((long long)o + kTile - 1) / kTile);
      pos = o + (t - s_tok[b]);
      const int e = pos / kTile;
      const int page = e < ho ? p.table[(size_t)b * p.max_pages + e] : taken(s_take[b] + (e - ho));
      slot = page < 0 || page >= (1 << 25) ? -1 : page * kTile + pos % kTile;
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
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

// ------------------------------------------------------------------ write
// One thread per (token, head, 16 channels, K or V).
struct WriteParams {
  const uint16_t *k, *v;
  long long ks_h, ks_t, vs_h, vs_t;
  int H, T;
  const int32_t* slots;
  uint8_t* pages;
  int num_pages;
  const float *k_scale, *v_scale;
  int* err;
};

template <int D, bool F16>
__global__ void __launch_bounds__(256) write_kernel(const WriteParams p) {
  constexpr int N = D / 16;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int t = (int)(i % N), which = (int)(i / N % 2), h = (int)(i / (2 * N) % p.H);
  const long long tok = i / (2 * N) / p.H;
  if (tok >= p.T) return;
  const int slot = p.slots[tok];
  if (slot < 0) return;
  if (slot / kTile >= p.num_pages) {
    if (p.err) atomicCAS(p.err, 0, APA_DEVERR_BOUNDS);
    return;
  }
  const uint16_t* src = which ? p.v + h * p.vs_h + tok * p.vs_t : p.k + h * p.ks_h + tok * p.ks_t;
  const uint4 a = reinterpret_cast<const uint4*>(src + 16 * t)[0], b = reinterpret_cast<const uint4*>(src + 16 * t)[1];
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float x[16];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 f = unpack2<F16>(w[e]);
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
  uint2 codes;
  const uint32_t sb = quant16(x, which ? p.v_scale[h] : p.k_scale[h], &codes);
  const int key = slot % kTile, ki = key % kBlkKeys;
  uint8_t* blk = p.pages + ((size_t)(slot / kTile) * p.H + h) * page_head_bytes(D) + key / kBlkKeys * blk_bytes(D);
  if (which == 0) {
    *reinterpret_cast<uint2*>(blk + ki * (D / 2) + 8 * t) = codes;
    blk[ks_byte(D, ki, t)] = (uint8_t)sb;
  } else {
#pragma unroll
    for (int g = 0; g < 8; ++g)
      blk[v_byte(D, ki, t, g)] = (uint8_t)(((codes.x >> (4 * g)) & 15u) | (((codes.y >> (4 * g)) & 15u) << 4));
    blk[vs_byte(D, ki, t)] = (uint8_t)sb;
  }
}

// ------------------------------------------------------------------ read
struct ReadParams {
  const uint8_t* pages;
  int num_pages, H, T;
  const int32_t* slots;
  const float *k_scale, *v_scale;
  uint16_t *k, *v;
  int* err;
};

template <int D, bool F16>
__global__ void __launch_bounds__(256) read_kernel(const ReadParams p) {
  constexpr int N = D / 16;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int t = (int)(i % N), which = (int)(i / N % 2);
  const long long row = i / (2 * N);
  if (row >= (long long)p.H * p.T) return;
  const int h = (int)(row / p.T);
  const int tok = (int)(row % p.T);
  const int slot = p.slots[tok];
  uint32_t out[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
  if (slot >= 0 && slot / kTile >= p.num_pages) {
    if (p.err) atomicCAS(p.err, 0, APA_DEVERR_BOUNDS);
  } else if (slot >= 0) {
    const int key = slot % kTile, ki = key % kBlkKeys;
    const uint8_t* blk =
        p.pages + ((size_t)(slot / kTile) * p.H + h) * page_head_bytes(D) + key / kBlkKeys * blk_bytes(D);
    uint2 codes;
    uint32_t sb;
    if (which == 0) {
      codes = *reinterpret_cast<const uint2*>(blk + ki * (D / 2) + 8 * t);
      sb = blk[ks_byte(D, ki, t)];
    } else {
      codes = make_uint2(0u, 0u);
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const uint32_t c = blk[v_byte(D, ki, t, g)];
        codes.x |= (c & 15u) << (4 * g);
        codes.y |= (c >> 4) << (4 * g);
      }
      sb = blk[vs_byte(D, ki, t)];
    }
    const float b = ue4m3_value(sb), s = which ? p.v_scale[h] : p.k_scale[h];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t c = (e < 4 ? codes.x : codes.y) >> (8 * (e & 3));
      out[e] = pack2<F16>(__fmul_rn(e2m1_value(c & 15u) * b, s), __fmul_rn(e2m1_value((c >> 4) & 15u) * b, s));
    }
  }
  uint4* dst = reinterpret_cast<uint4*>((which ? p.v : p.k) + row * D + 16 * t);
  dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
  dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

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
  const int smem = 3 * B * (int)sizeof(int);
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 3 * kMaxRequests * 4))
    return APA_ERR_CUDA;
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
  return cudaLaunchKernelEx(&cfg, tables_kernel, prm) == cudaSuccess ? APA_OK : APA_ERR_CUDA;
}

int apa_cache_write(const void* k, const void* v, int dtype, int Hkv, int T, int d, long long k_head_stride,
                    long long k_token_stride, long long v_head_stride, long long v_token_stride, const int32_t* slots,
                    uint8_t* pages, int num_pages, const float* k_scale, const float* v_scale, cudaStream_t stream) {
  const int st = check_cache(dtype, Hkv, T, d, num_pages);
  if (st) return st;
  if (T == 0) return APA_OK;
  if (!k || !v || !slots || !pages || !k_scale || !v_scale) return APA_ERR_NULL;
  if ((((uintptr_t)k | (uintptr_t)v | (uintptr_t)pages) & 15) ||
      ((k_head_stride | k_token_stride | v_head_stride | v_token_stride) & 7))
    return APA_ERR_ALIGN;
  WriteParams prm{(const uint16_t*)k, (const uint16_t*)v, k_head_stride, k_token_stride, v_head_stride,
                  v_token_stride,     Hkv,                T,             slots,          pages,
                  num_pages,          k_scale,            v_scale,       device_error_word()};
  const long long blocks = ((long long)T * Hkv * (d / 8) + 255) / 256;
  if (blocks > 0x7FFFFFFFll) return APA_ERR_SHAPE;
  const bool f16 = dtype == APA_DTYPE_F16;
  auto go = [&](auto kern) { kern<<<(unsigned)blocks, 256, 0, stream>>>(prm); };
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
  ReadParams prm{pages, num_pages, Hkv, T, slots, k_scale, v_scale, (uint16_t*)k, (uint16_t*)v, device_error_word()};
  const long long blocks = ((long long)T * Hkv * (d / 8) + 255) / 256;
  if (blocks > 0x7FFFFFFFll) return APA_ERR_SHAPE;
  const bool f16 = dtype == APA_DTYPE_F16;
  auto go = [&](auto kern) { kern<<<(unsigned)blocks, 256, 0, stream>>>(prm); };
  switch (d) {
    case 64: f16 ? go(read_kernel<64, true>) : go(read_kernel<64, false>); break;
    case 128: f16 ? go(read_kernel<128, true>) : go(read_kernel<128, false>); break;
    case 256: f16 ? go(read_kernel<256, true>) : go(read_kernel<256, false>); break;
  }
  return cudaGetLastError() == cudaSuccess ? APA_OK : APA_ERR_CUDA;
}

}  // extern "C"
