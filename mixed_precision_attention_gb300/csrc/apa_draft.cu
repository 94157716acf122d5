// apa_draft.cu -- what goes around the attention of drafted trees: which nodes each one sees,
// from their parents, and the keys of the accepted path moved behind the context.
#include "../../include/apa.h"
#include "apa_internal.h"
#include "cache_page.cuh"
#include "tc.cuh"

namespace apa {
namespace {

// ------------------------------------------------------------------ trees
// S(i) = {i} + S(parent(i)).  A CTA per sequence, a thread per node, which walks up its own
// ancestors: they come in falling order, so the words of its row are filled from the last to
// the first and each is written once.  What bounds it is latency: a launch, one load of the
// parents, and a shared-memory load per level (64 trees of 64 nodes 2.0 us, 256 of 250 2.4).
struct TreeParams {
  const int32_t *parents, *nodes;
  int Nq, words;
  uint32_t* mask;
  int32_t* depths;
  int* err;
};

__global__ void __launch_bounds__(APA_TREE_MAX_NODES) draft_tree_kernel(const TreeParams p) {
  __shared__ int16_t up[APA_TREE_MAX_NODES];
  const int b = blockIdx.x, i = threadIdx.x;
  const int given = p.nodes ? p.nodes[b] : p.Nq, n = max(0, min(given, p.Nq));
  int parent = -1;
  bool bad = i == 0 && given != n;
  if (i < n) {
    parent = p.parents[(size_t)b * p.Nq + i];
    if (parent < -1 || parent >= i) {
      bad = true;
      parent = -1;
    }
  }
  up[i] = (int16_t)parent;
  if (bad && p.err) atomicCAS(p.err, 0, APA_DEVERR_BOUNDS);
  __syncthreads();
  if (i >= p.Nq) return;
  const size_t row = (size_t)b * p.Nq + i;
  int at = i < n ? i : -1, count = 0;
  auto word = [&](int w) {
    uint32_t bits = 0;
    while (at >= 32 * w) {  // (at is in word w or before it; -1 ends every word)
      bits |= 1u << (at & 31);
      ++count;
      at = up[at];
    }
    return bits;
  };
  if (p.words % 4 == 0) {
    uint4* dst = reinterpret_cast<uint4*>(p.mask + row * p.words);
    for (int w = p.words - 4; w >= 0; w -= 4) {
      uint4 x;
      x.w = word(w + 3);
      x.z = word(w + 2);
      x.y = word(w + 1);
      x.x = word(w);
      dst[w / 4] = x;
    }
  } else {
    for (int w = p.words - 1; w >= 0; --w) p.mask[row * p.words + w] = word(w);
  }
  p.depths[row] = max(0, count - 1);
}

// ------------------------------------------------------------------ the accepted path
// A key of one KV head is d/32 vectors of K codes, a run of K scales, d/8 vectors of 16 bytes
// that hold one V code byte of it in each word, and as many of V scales: a thread takes one
// such piece of one key.  A CTA moves all keys of a sequence for a few heads of one layer, in
// rounds: all pieces are read, then, behind a barrier, written.  A path rises, so path[k] > k
// wherever something moves: no later key is read where an earlier one has been written.  A
// V code byte is alone in its 4 bytes and 16 of a key's lie in sectors of their own, so what moves is
// five times a key's bytes; 32 sequences in 28 layers of 8 heads take 16 us, 64 in one layer 4.2
// (launch, path, table entry and key, one load behind the other).
constexpr int kAcceptThreads = 256;
constexpr int kAcceptHeads = 1 << 15;  // of a CTA, at most: it counts its pieces in 32 bits
struct AcceptParams {
  uint8_t* pages;
  size_t layer_bytes;
  int num_pages, H, heads;  // heads of a CTA
  const int32_t* table;
  int max_pages;
  const int32_t *lens, *nodes, *path, *counts;
  int path_len;
  int32_t* new_lens;
  int* err;
};

template <int D>
__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const AcceptParams p) {
  constexpr int kKVec = D / 32, kVVec = D / 8, kSVec = D / 64, kPieces = kKVec + 1 + kVVec + kSVec;
  static_assert((long long)APA_TREE_MAX_NODES * kAcceptHeads * kPieces + kAcceptThreads < (1ll << 31), "pieces of a CTA");
  const int b = blockIdx.x, h0 = blockIdx.y * p.heads, heads = min(p.heads, p.H - h0);
  const int len = p.lens[b], nodes = p.nodes[b], count = p.counts[b];
  const int32_t* path = p.path + (size_t)b * p.path_len;
  const bool sizes = len >= 0 && len <= (long long)p.max_pages * kTile && nodes >= 0 && nodes <= len;
  const int base = sizes ? len - nodes : max(0, min(len, p.max_pages * kTile));
  bool good = sizes && count >= 0 && count <= min(p.path_len, nodes);
  if (good)
    for (int k = threadIdx.x; k < count; k += kAcceptThreads) {
      const int x = path[k];
      if (x >= nodes || x <= (k ? path[k - 1] : -1)) good = false;
    }
  good = __syncthreads_and(good);
  if (threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
    p.new_lens[b] = good ? base + count : base;
    if (!good && p.err) atomicCAS(p.err, 0, APA_DEVERR_BOUNDS);
  }
  if (!good) return;
  uint8_t* pool = p.pages + blockIdx.z * p.layer_bytes;
  const int32_t* table = p.table + (size_t)b * p.max_pages;
  // (a rising path: what stays in place are its first keys)
  const int per = heads * kPieces, total = count * per;
  for (int x0 = 0; x0 < total; x0 += kAcceptThreads) {
    const int x = x0 + threadIdx.x;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    uint8_t *to = nullptr, *blk_to = nullptr;
    int piece = 0, from_i = 0, to_i = 0;
    if (x < total) {
      const int k = x / per, y = x - k * per, h = h0 + y / kPieces;
      piece = y % kPieces;
      const int node = path[k];
      if (node != k) {
        const int src = base + node, dst = base + k, ps = table[src / kTile], pd = table[dst / kTile];
        if ((unsigned)ps < (unsigned)p.num_pages && (unsigned)pd < (unsigned)p.num_pages) {
          from_i = src % kBlkKeys;
          to_i = dst % kBlkKeys;
          const uint8_t* blk = pool + ((size_t)ps * p.H + h) * page_head_bytes(D) + src % kTile / kBlkKeys * blk_bytes(D);
          blk_to = pool + ((size_t)pd * p.H + h) * page_head_bytes(D) + dst % kTile / kBlkKeys * blk_bytes(D);
          if (piece < kKVec) {
            v = *reinterpret_cast<const uint4*>(blk + from_i * (D / 2) + 16 * piece);
            to = blk_to + to_i * (D / 2) + 16 * piece;
          } else if (piece == kKVec) {  // D / 16 bytes
            const uint8_t* s = blk + ks_byte(D, from_i, 0);
            to = blk_to + ks_byte(D, to_i, 0);
            if constexpr (D == 256) v = *reinterpret_cast<const uint4*>(s);
            if constexpr (D == 128) v.x = reinterpret_cast<const uint32_t*>(s)[0], v.y = reinterpret_cast<const uint32_t*>(s)[1];
            if constexpr (D == 64) v.x = *reinterpret_cast<const uint32_t*>(s);
          } else if (piece < kKVec + 1 + kVVec) {  // a byte in each word of a vector of four 16-channel tiles
            const int z = piece - kKVec - 1, t = 4 * (z / 8), g = z % 8;
            v = *reinterpret_cast<const uint4*>(blk + v_byte(D, from_i & ~3, t, g));
            to = blk_to + v_byte(D, to_i, t, g);
          } else {
            const int t = 4 * (piece - kKVec - 1 - kVVec);
            v = *reinterpret_cast<const uint4*>(blk + vs_byte(D, from_i & ~3, t));
            to = blk_to + vs_byte(D, to_i, t);
          }
        } else if (p.err) {
          atomicCAS(p.err, 0, APA_DEVERR_BOUNDS);
        }
      }
    }
    __syncthreads();
    if (to) {
      if (piece < kKVec) {
        *reinterpret_cast<uint4*>(to) = v;
      } else if (piece == kKVec) {
        if constexpr (D == 256) *reinterpret_cast<uint4*>(to) = v;
        if constexpr (D == 128) reinterpret_cast<uint32_t*>(to)[0] = v.x, reinterpret_cast<uint32_t*>(to)[1] = v.y;
        if constexpr (D == 64) *reinterpret_cast<uint32_t*>(to) = v.x;
      } else {
        const int sh = 8 * (from_i & 3);
        to[0] = (uint8_t)(v.x >> sh);
        to[4] = (uint8_t)(v.y >> sh);
        to[8] = (uint8_t)(v.z >> sh);
        to[12] = (uint8_t)(v.w >> sh);
      }
    }
  }
}

}  // namespace
}  // namespace apa

using namespace apa;

extern "C" {

int apa_draft_tree(const int32_t* parents, const int32_t* nodes, int B, int Nq, uint32_t* mask, int32_t* depths,
                   cudaStream_t stream) {
  if (!parents || !mask || !depths) return APA_ERR_NULL;
  if (B < 1 || Nq < 1 || Nq > APA_TREE_MAX_NODES) return APA_ERR_SHAPE;
  if ((uintptr_t)mask & 15) return APA_ERR_ALIGN;
  const TreeParams prm{parents, nodes, Nq, (Nq + 31) / 32, mask, depths, device_error_word()};
  draft_tree_kernel<<<B, (Nq + 31) / 32 * 32, 0, stream>>>(prm);
  return cudaGetLastError() == cudaSuccess ? APA_OK : APA_ERR_CUDA;
}

int apa_cache_accept(uint8_t* pages, int layers, int num_pages, int Hkv, int d, const int32_t* block_table, int max_pages,
                     const int32_t* lens, const int32_t* nodes, const int32_t* path, int path_len, const int32_t* counts,
                     int B, int32_t* new_lens, cudaStream_t stream) {
  if (!pages || !block_table || !lens || !nodes || !path || !counts || !new_lens) return APA_ERR_NULL;
  if (layers < 1 || layers > 65535 || num_pages < 1 || num_pages >= (1 << 25) || Hkv < 1 || Hkv > (1 << 16) || max_pages < 1 ||
      max_pages >= (1 << 25) || path_len < 1 || path_len > APA_TREE_MAX_NODES || B < 1)
    return APA_ERR_SHAPE;
  // a sequence's first CTA writes new_lens while its others may not have read theirs
  auto within = [&](const int32_t* in, long long words) {
    const uintptr_t a = (uintptr_t)in, n = (uintptr_t)new_lens;
    return n < a + 4 * (uintptr_t)words && a < n + 4 * (uintptr_t)B;
  };
  if (within(lens, B) || within(nodes, B) || within(counts, B) || within(path, (long long)B * path_len) ||
      within(block_table, (long long)B * max_pages))
    return APA_ERR_SHAPE;
  if (d != 64 && d != 128 && d != 256) return APA_ERR_HEAD_DIM;
  if ((uintptr_t)pages & 15) return APA_ERR_ALIGN;
  // one head per CTA, several where there are ten thousand CTAs anyway (28 layers x 32 sequences x 8 heads: 16 us, 21 with all heads in one)
  int heads = 1;
  while (heads < Hkv && heads < kAcceptHeads && (long long)B * layers * ((Hkv + heads - 1) / heads) > 152 * 64) heads *= 2;
  const AcceptParams prm{pages, (size_t)num_pages * Hkv * page_head_bytes(d), num_pages, Hkv, heads, block_table, max_pages,
                         lens,  nodes, path, counts, path_len, new_lens, device_error_word()};
  const dim3 grid(B, (Hkv + heads - 1) / heads, layers);
  auto go = [&](auto kern) { kern<<<grid, kAcceptThreads, 0, stream>>>(prm); };
  switch (d) {
    case 64: go(accept_kernel<64>); break;
    case 128: go(accept_kernel<128>); break;
    case 256: go(accept_kernel<256>); break;
  }
  return cudaGetLastError() == cudaSuccess ? APA_OK : APA_ERR_CUDA;
}

}  // extern "C"
