/*
 * apa.h -- C ABI of libapa.so: adaptive-precision causal attention prefill
 * with GQA packing on GB300 (sm_103a).
 *
 * The method is the one of "APA: sloppy attention, exact where it counts"
 * (rfriedmann.de blog):
 *   - pass 1 ("Pass 1: FP4 everywhere, with a hot test") computes every 64-key
 *     tile in block-scaled NVFP4 (E2M1 elements, one UE4M3 scale per 16 values,
 *     one FP32 scale per head; keys mean-centred per channel) and flags "hot"
 *     tiles, those where a row of a 16-row group has FP4 tile mass above
 *     eps times its running sum lambda;
 *   - pass 2 ("Pass 2: exact FP16 on the hot tiles") recomputes only the hot
 *     tiles exactly (here in BF16 with FP32 accumulation);
 *   - the two online-softmax states, which share one logit frame, are merged
 *     exactly by log-sum-exp ("The merge that makes it exact").
 * Shapes and masking follow SDPA (ffpa-attn.readthedocs.io, the "Note" on
 * cross-, GQA and causal attention): BHSD layout, Hq % Hkv == 0, and with
 * causal != 0 the queries are aligned to the key tail: query row i sees key j
 * iff j <= i + (Nkv - Nq), which needs Nkv >= Nq.  The softmax scale is 1/sqrt(d).
 *
 * Common conventions:
 *   - All pointer arguments of the device entry points are device memory owned
 *     by the caller; the library never frees them.  q, k, v must be 16-byte
 *     aligned.
 *   - Calls are asynchronous: they enqueue work on `stream` and return.
 *     Asynchronous kernel errors surface at the caller's next synchronisation;
 *     a device-side wait that timed out, or a page, slot or length in device
 *     memory that is out of range, is recorded in a library-wide device error
 *     word that apa_check_error() reports.
 *   - Results are deterministic: reruns with the same inputs are bitwise equal.
 *   - On a negative status nothing has been enqueued.  No C++ exception crosses
 *     the ABI.
 */
#ifndef APA_H
#define APA_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* status codes */
#define APA_OK 0
#define APA_ERR_NULL (-1)      /* a required pointer is null */
#define APA_ERR_SHAPE (-2)     /* B, Hq, Hkv, Nq, Nkv out of range, Hq % Hkv != 0, or causal with Nkv < Nq */
#define APA_ERR_EPS (-3)       /* eps < 0 or NaN */
#define APA_ERR_HEAD_DIM (-4)  /* d not in {64, 128, 256} */
#define APA_ERR_CUDA (-5)      /* a CUDA call or launch failed; cudaGetLastError() holds the cause */
#define APA_ERR_NOMEM (-6)     /* the workspace could not be allocated, or the given one is too small or misaligned */
#define APA_ERR_DEVICE (-7)    /* a kernel recorded a device-side error: a timeout, or a page, slot or length in device memory that is out of range (apa_check_error) */
#define APA_ERR_ALIGN (-8)     /* a tensor not 16-byte aligned, or a stride no multiple of 8 elements */
#define APA_ERR_SCRATCH (-9)   /* too large for the fixed scratch of apa_quantize_noalloc */
#define APA_ERR_FLAGS (-10)    /* an unknown bit in `flags` */
#define APA_ERR_DTYPE (-11)    /* an unknown element type */
#define APA_ERR_WINDOW (-12)   /* window or sinks out of range */

/* Element types of the cache entry points. */
#define APA_DTYPE_BF16 0
#define APA_DTYPE_F16 1

/* Options of the _ex entry points. */
#define APA_FLAG_Q_RESIDUAL 1u /* Q as two FP4 terms in pass 1 (see apa_attention_ex) */
#define APA_FLAG_LSE_SCALES 2u /* least-squared-error block scales for Q, K, V (see apa_attention_ex) */
#define APA_FLAG_VALUE_WEIGHTED 4u /* hot test weighted by value norm (see apa_attention_ex) */
#define APA_FLAG_ROWSUM_MMA 8u /* pass-1 tile row sums from an MMA against an E2M1 ones tile (see apa_attention_ex) */

/* Size of the fixed device scratch array behind apa_quantize_noalloc (16 MiB). */
#define APA_NOALLOC_SCRATCH_BYTES (16u * 1024u * 1024u)

/* Adaptive-precision attention, eps >= 0:
 *   q        bf16 [B, Hq, Nq, d], contiguous
 *   k, v     bf16 [B, Hkv, Nkv, d], contiguous
 *   causal   0: every key visible; else tail-aligned causal mask
 *   eps      hot-test threshold.  0 runs every visible tile exactly (the all-exact
 *            path: pass 2 only, Q K^T in BF16, P.V with P rounded once to FP16
 *            against an FP16 copy of V, FP32 accumulation); +inf makes every tile
 *            cold (all-FP4 pass 1).
 *   out      fp32 [B, Hq, Nq, d] (required)
 *   lse      fp32 [B, Hq, Nq], natural-log log-sum-exp of the scaled scores (nullable)
 *   hot_mask uint32 [B, Hkv, ceil(G*Nq/16), ceil(T/32)] with G = Hq/Hkv and
 *            T = ceil(Nkv/64): bit t%32 of word t/32 is set iff key tile t was
 *            hot for that 16-row group of GQA-packed rows (packed row p = pos*G + g
 *            holds query head h*G + g at position pos).  At eps = 0 every tile the
 *            group can see is marked.  Nullable.
 * The workspace is allocated stream-ordered on `stream` (cudaMallocAsync) and
 * released the same way.  Returns APA_OK or a negative status.
 * When the pass-1 CTAs leave at least 8 SMs free, the K/V tiles are quantized
 * inside the pass-1 launch ("What else is in the box" on the page: quantization
 * inside the launch): that kernel is then launched cooperatively with one block
 * on every SM, so it starts once the whole GPU is free and holds it while it
 * runs.  If the driver refuses that launch (fewer SMs available to the context
 * than the device has), the call falls back to the separate quantizer kernel.
 * The results are the same bits either way. */
int apa_attention(const void* q, const void* k, const void* v, int B, int Hq, int Hkv, int Nq, int Nkv, int d,
                  int causal, float eps, float* out, float* lse, uint32_t* hot_mask, cudaStream_t stream);

/* Bytes of device workspace apa_attention_ws() needs for this problem.  At
 * eps = 0 that is the FP16 copy of V ([B][Hkv][Nkv][d] FP16, V divided by a
 * power of two per head only when max |v| > 2^15, so exact for every bf16 value
 * above the FP16 subnormals) and the heads' maxima of |v|; at d = 256, when a KV
 * head has at most 4 blocks of 128 packed rows and 2048 or more key tiles, also
 * the (m, l, O) states of the parts into which each block's walk is split (one
 * part per 1024 tiles, at most 4).  At eps > 0 it holds the quantized operands,
 * the pass-1 states and the hot lists, and at d = 256, when a KV head has at most
 * 4 blocks and 1024 or more key tiles, the states of the parts of pass 2's walks
 * over the hot lists (one part per 512 tiles, at most 4). */
size_t apa_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nkv, int d, float eps);

/* apa_attention() with a caller-provided device workspace of at least
 * apa_workspace_bytes() bytes, 256-byte aligned; it allocates nothing.
 * Two calls that overlap on the GPU must not share a workspace. */
int apa_attention_ws(const void* q, const void* k, const void* v, int B, int Hq, int Hkv, int Nq, int Nkv, int d,
                     int causal, float eps, float* out, float* lse, uint32_t* hot_mask, void* workspace,
                     size_t workspace_bytes, cudaStream_t stream);

/* apa_attention() with options (APA_FLAG_*; unknown bits give APA_ERR_FLAGS):
 *   APA_FLAG_Q_RESIDUAL  Q goes to pass 1 as two FP4 terms ("Second hunt" on the
 *                        page): Q1 as before and Q2, the FP4 quantization of the
 *                        residual Q - Q1 under the same FP32 head scale (block
 *                        scales of its own; residual r = fp32(x - fp32(E2M1 *
 *                        UE4M3 * s)) per element).  Both terms accumulate into
 *                        the same S against the same K: twice the QK^T work of
 *                        pass 1, which then runs one 128-row block per CTA.
 *   APA_FLAG_LSE_SCALES  every block scale of Q, K, V (and of the residual Q
 *                        term) picked by least squared error instead of the
 *                        nearest one ("Second hunt"): among the nearest UE4M3
 *                        code and its two neighbours, tried in that order, the
 *                        one whose FP32 sum of squared errors over the 16 values
 *                        (in index order) is strictly smallest.
 *   APA_FLAG_VALUE_WEIGHTED  the hot test weighted by value norm ("Honest
 *                        limits" on the page: the plain test bounds a cold
 *                        tile's share of the softmax mass, not of the output):
 *                        tile t is hot iff some row has w_t * l_t > eps * lambda,
 *                        w_t = (largest key value norm in the tile) / (mean key
 *                        value norm of the head); norms are FP32 sums of FP32
 *                        squares in channel order with a rounded square root,
 *                        the mean follows the key mean's summation order.
 *                        lambda stays the plain running sum.  A cold tile then
 *                        moves each output row by at most eps times the mean
 *                        value norm.  Costs 8 bytes of workspace per tile.
 *   APA_FLAG_ROWSUM_MMA  the tile row sums l_t of pass 1 from one extra MMA of
 *                        the E2M1 P against an E2M1 ones tile ("Pass 1", step 3
 *                        on the page), instead of the default: each row's thread
 *                        sums its own E2M1 codes exactly in registers.  Both are
 *                        the exact sum of the quantized P; the MMA form runs one
 *                        128-row block per pass-1 CTA with the separate K/V
 *                        quantizer.  Not combinable with APA_FLAG_Q_RESIDUAL
 *                        (APA_ERR_FLAGS): both need the same TMEM columns.
 * `workspace` of at least apa_workspace_bytes_ex() bytes (256-byte aligned), or
 * null to have it allocated stream-ordered for the call. */
int apa_attention_ex(const void* q, const void* k, const void* v, int B, int Hq, int Hkv, int Nq, int Nkv, int d,
                     int causal, float eps, unsigned flags, float* out, float* lse, uint32_t* hot_mask,
                     void* workspace, size_t workspace_bytes, cudaStream_t stream);
size_t apa_workspace_bytes_ex(int B, int Hq, int Hkv, int Nq, int Nkv, int d, float eps, unsigned flags);

/* apa_attention() on a paged K/V cache.  Every (sequence, KV head) keeps its keys
 * and values in pages of 64 keys (one key tile) drawn from one pool:
 *   k_pages, v_pages  bf16 [num_pages][Hkv][64][d], contiguous, 16-byte aligned
 *   block_table       int32 [B][max_pages] in device memory: entry t of sequence b
 *                     is the page holding its keys 64t .. 64t+63;
 *                     max_pages >= ceil(Nkv/64); num_pages * Hkv * 64 < 2^31
 * (the blog, "What else is in the box": pass 2 reads through a block table; here
 * every read of K and V does).  All sequences have Nkv keys and Nq queries, as
 * in apa_attention.  Keys past Nkv in a sequence's last page are never used.  A
 * table entry outside [0, num_pages) reads page 0 and is reported by
 * apa_check_error as a bounds error (status APA_ERR_DEVICE).  The results are
 * those of apa_attention on the same keys laid out contiguously, bit for bit. */
int apa_attention_paged(const void* q, const void* k_pages, const void* v_pages, int num_pages,
                        const int32_t* block_table, int max_pages, int B, int Hq, int Hkv, int Nq, int Nkv, int d,
                        int causal, float eps, float* out, float* lse, uint32_t* hot_mask, cudaStream_t stream);

/* apa_attention() on HOST buffers (page-locked memory recommended): copies q, k,
 * v to the device, runs, copies out (and lse / hot_mask when non-null) back,
 * and synchronizes `stream` before returning.  The results equal those of
 * apa_attention().  Each (b, KV head) is an independent problem of the method,
 * so the call pipelines them: one's inputs are copied (on a library-owned copy
 * stream) while earlier ones compute (on up to 8 library-owned streams, created
 * at rising priority so that the sub-problems that arrive last are dispatched
 * first) and their results are copied back.  All of it is ordered after the work already
 * on `stream`.  The device memory is one library-owned buffer per device, grown
 * on demand and kept until the process exits; calls on the same device are
 * serialized by a lock. */
int apa_attention_host(const void* q, const void* k, const void* v, int B, int Hq, int Hkv, int Nq, int Nkv, int d,
                       int causal, float eps, float* out, float* lse, uint32_t* hot_mask, cudaStream_t stream);

/* Where, inside a caller's workspace, an eps > 0 call of apa_attention_ws() or
 * apa_attention_ex() (with these flags) leaves the pass-1 NVFP4 operands: byte
 * offsets of the K/V tile blobs, the Q blobs, the key mean and the FP32 head
 * scales, in the layouts apa_quantize() writes them.  They hold the call's
 * operands once the call has completed, until the workspace is used again; that
 * holds whether the K/V tiles were quantized by the separate kernel or inside
 * the pass-1 launch.  A measurement and testing aid, not needed to use the
 * library.  Returns APA_OK; APA_ERR_EPS for eps <= 0 (the all-exact path
 * quantizes nothing), or the argument errors of apa_attention_ex(). */
int apa_workspace_operands(int B, int Hq, int Hkv, int Nq, int Nkv, int d, float eps, unsigned flags,
                           size_t* kv_blob, size_t* q_blob, size_t* mu, size_t* s_q, size_t* s_k, size_t* s_v);

/* The pass-1 NVFP4 operands on their own (blog, "Pass 1" and "Mean-centred K"):
 *   kv_blob  uint8 [B*Hkv][T][apa_kv_blob_bytes / (B*Hkv*T)]: per 64-key tile the
 *            E2M1 codes of the centred keys and of V^T with their UE4M3 scales, in
 *            the tcgen05 shared-memory image (layout in the library's
 *            apa_internal.h; 9216 bytes per tile at d = 128)
 *   q_blob   uint8 [B*Hkv][ceil(G*Nq/128)][72*d]: E2M1 codes and UE4M3 scales of
 *            128 GQA-packed query rows per block
 *   mu       fp32 [B, Hkv, d]  per-channel key mean
 *   s_q      fp32 [B, Hq]; s_k, s_v fp32 [B, Hkv]: FP32 per-head scales
 * Temporary statistics are allocated stream-ordered on `stream`. */
int apa_quantize(const void* q, const void* k, const void* v, int B, int Hq, int Hkv, int Nq, int Nkv, int d,
                 uint8_t* kv_blob, uint8_t* q_blob, float* mu, float* s_q, float* s_k, float* s_v,
                 cudaStream_t stream);
size_t apa_kv_blob_bytes(int B, int Hkv, int Nkv, int d);
/* apa_quantize() with options: q2_blob (nullable, q_blob's layout) receives the
 * codes and scales of the FP4 residual term of Q (APA_FLAG_Q_RESIDUAL);
 * APA_FLAG_LSE_SCALES picks every block scale by least squared error.  The flag
 * APA_FLAG_Q_RESIDUAL is implied by a non-null q2_blob; APA_FLAG_VALUE_WEIGHTED
 * changes nothing here (the weights are not an operand). */
int apa_quantize_ex(const void* q, const void* k, const void* v, int B, int Hq, int Hkv, int Nq, int Nkv, int d,
                    unsigned flags, uint8_t* kv_blob, uint8_t* q_blob, uint8_t* q2_blob, float* mu, float* s_q,
                    float* s_k, float* s_v, cudaStream_t stream);

/* apa_quantize() for callers that must not allocate device memory during the
 * call: engines that reserve the whole GPU for their own memory arena up front,
 * plugin interfaces that receive buffers but have no allocator to call, and
 * latency-critical paths where a device allocation (which can synchronize) is
 * not acceptable.  The blog has no counterpart to this entry point.
 *   Same arguments, outputs and results as apa_quantize(); no cudaMalloc,
 *   cudaFree or other allocating call is made.  The temporary statistics live in
 *   one fixed array of APA_NOALLOC_SCRATCH_BYTES in the library's device image,
 *   which every GPU that loads the library holds until the process exits.
 *   Problems whose statistics need more than that
 *   (apa_quantize_noalloc_scratch_bytes() > APA_NOALLOC_SCRATCH_BYTES, roughly
 *   B*Hkv*ceil(Nkv/64)*d*4 bytes) are rejected with APA_ERR_SCRATCH before any
 *   work is enqueued.
 *   The first call on a device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call before
 *   any stream capture.
 *   Every call shares the one array per device, and each call overwrites what
 *   the last one left there: calls that can overlap on the GPU (different
 *   streams without ordering between them) race on it and must be serialized by
 *   the caller. */
int apa_quantize_noalloc(const void* q, const void* k, const void* v, int B, int Hq, int Hkv, int Nq, int Nkv,
                         int d, uint8_t* kv_blob, uint8_t* q_blob, float* mu, float* s_q, float* s_k, float* s_v,
                         cudaStream_t stream);
/* Scratch bytes apa_quantize_noalloc needs for this problem (0 for invalid sizes). */
size_t apa_quantize_noalloc_scratch_bytes(int B, int Hq, int Hkv, int Nkv, int d);
size_t apa_q_blob_bytes(int B, int Hq, int Hkv, int Nq, int d);

/* ------------------------------------------------------------------ sliding window
 * Causal attention with a sliding window and sinks (first keys that stay visible):
 * query row i, at position p = i + Nkv - Nq, sees key j iff
 *     j <= p  and  (j > p - window  or  j < sinks).
 *   q        bf16 [B, Hq, Nq, d], contiguous
 *   k, v     bf16 [B, Hkv, Nkv, d], contiguous, Nkv >= Nq
 *   window   >= 1 keys, the row's own among them; sinks >= 0
 *   out      bf16 [B, Hq, Nq, d] (required)
 *   lse      fp32 [B, Hq, Nq], natural-log log-sum-exp of the scaled scores (nullable)
 * Exact attention, as the eps = 0 form of apa_attention: BF16 Q K^T and FP32
 * softmax statistics; here P is rounded to BF16 for the product with V itself
 * (relative error 2^-8 at most per weight, as the rounding of the output; apa_attention
 * at eps = 0 rounds it to FP16 and returns FP32).  Only the key tiles that a row block
 * sees are read.  V must be finite: a NaN or an infinity in it reaches, beside the rows
 * that see its key, others of their blocks of 128 packed rows.  A K that is not finite
 * reaches only the rows that see it.  No workspace. */
int apa_attention_window(const void* q, const void* k, const void* v, int B, int Hq, int Hkv, int Nq, int Nkv, int d,
                         int window, int sinks, void* out, float* lse, cudaStream_t stream);

/* ------------------------------------------------------------------ 4-bit K/V cache
 * Keys and values of decoding sequences in NVFP4 (E2M1 codes, one UE4M3 scale per
 * 16 channels of a key, one FP32 scale per KV head), in pages of 64 keys:
 *   pages    uint8 [num_pages][Hkv][72*d], 16-byte aligned, num_pages < 2^25
 * A page holds, per KV head, four blocks of 16 keys of 18*d bytes each:
 *   K codes   8*d bytes  key i, byte x: codes of channels 2x (low nibble), 2x + 1
 *   V codes   8*d bytes  key i, channels 16t + g (low nibble) and 16t + 8 + g, g < 8:
 *                        byte 512*(t/4) + 16*(4*g + i/4) + 4*(t%4) + i%4
 *   K scales    d bytes  key i, channels 16t .. 16t + 15: byte i*d/16 + t
 *   V scales    d bytes  key i, channels 16t .. 16t + 15: byte 4*((i/4)*d/16 + t) + i%4
 * (the V order is the one the attention's matrix products read in place, and every
 * key owns whole bytes, so tokens are appended independently of each other).
 * A value is E2M1 * UE4M3 * the head's FP32 scale.  Quantization is apa_quantize's,
 * bit for bit, with the caller's head scales (2^-100 .. 2^100; the largest
 * magnitude expected divided by 2688; larger values saturate): scale code
 * b = UE4M3(fp32(max|x| / fp32(6 s))); codes 0 if b is 0, else
 * E2M1(fp32(x * fp32(1 / fp32(b s)))).  Infinities saturate too; a NaN makes its
 * group of 16 NaN (b = 0x7F, codes 0).  Keys are not mean-centred (the mean would
 * change with every appended key).
 * A slot names a key's place in the pool: page * 64 + key within the page. */
size_t apa_cache_page_bytes(int Hkv, int d); /* bytes of one page: Hkv * 72 * d */

/* Grows, shrinks and places requests, and maps their new tokens to slots, on the
 * GPU: no length is read on the host.  Request b goes from old_lens[b] to
 * new_lens[b] keys (ends: to 0; begins: from 0).
 *   old_lens, new_lens  int32 [B], each in [0, 64 * max_pages]; 1 <= B <= 8192
 *   block_table  int32 [B][max_pages], updated in place: entries below
 *                ceil(old/64) are the request's pages; a request that grows gets
 *                entries ceil(old/64) .. ceil(new/64)-1; all others are left alone
 *   free_pages   int32 [free_capacity], a stack of free pages, updated in place;
 *                *free_count of them are free, the last one is on top
 * First the pages that shrinking requests give up, entries ceil(new/64) ..
 * ceil(old/64)-1, go on top of the stack, in request and entry order; then the
 * pages that growing requests need come off the top, in that order.
 *   slots      int32 [max_tokens]: the slots of the tokens old_lens[b] ..
 *              new_lens[b]-1 of request 0, then of request 1, ...; -1 behind the last
 *   positions  int32 [max_tokens]: their positions in the request; 0 behind the last
 *   starts     int32 [B+1]: where each request's tokens start in slots, and the end
 *   free_count_out  int32 [1]: the free pages left; may be free_count itself
 *   status     int32 [1]: 0, or why nothing was changed (all slots are -1, positions
 *              and starts 0, *free_count_out = *free_count): APA_TABLES_LENGTH a
 *              length out of range, APA_TABLES_TOKENS more tokens than max_tokens,
 *              APA_TABLES_PAGES too few free pages, APA_TABLES_FREE the stack's
 *              count out of range, or too many pages given back for its capacity
 * No workspace; the results do not depend on the launch's shape.  One launch for up
 * to 8192 tokens; for more, a second one fills slots and positions. */
#define APA_TABLES_LENGTH 1
#define APA_TABLES_TOKENS 2
#define APA_TABLES_PAGES 3
#define APA_TABLES_FREE 4
int apa_cache_tables(const int32_t* old_lens, const int32_t* new_lens, int B, int32_t* block_table, int max_pages,
                     int32_t* free_pages, int free_capacity, const int32_t* free_count, int max_tokens, int32_t* slots,
                     int32_t* positions, int32_t* starts, int32_t* free_count_out, int32_t* status,
                     cudaStream_t stream);

/* Quantizes T tokens' keys and values into their slots of the cache.
 *   k, v     dtype (APA_DTYPE_*) [Hkv][T][d]; channels contiguous, heads and tokens
 *            at the given strides (in elements, multiples of 8; of an axis of length 1
 *            any); 16-byte aligned.
 *            (A projection's [T][Hkv][d] output is such an array.)
 *   slots    int32 [T]; a negative slot's token is skipped (padding), one outside the
 *            pool is skipped and reported by apa_check_error.  Slots of one call differ
 *            (of two tokens with one slot, each byte there is from one or the other).
 *   k_scale, v_scale  fp32 [Hkv]
 * Everything else in the pool is left as it is.  T = 0 does nothing. */
int apa_cache_write(const void* k, const void* v, int dtype, int Hkv, int T, int d, long long k_head_stride,
                    long long k_token_stride, long long v_head_stride, long long v_token_stride, const int32_t* slots,
                    uint8_t* pages, int num_pages, const float* k_scale, const float* v_scale, cudaStream_t stream);

/* The values that cached tokens stand for: k, v of `dtype`, contiguous [Hkv][T][d]
 * (the layout of one sequence in apa_attention), fp32(fp32(E2M1 * UE4M3) * scale)
 * rounded to dtype.  Tokens of negative slots are zero; a slot outside the pool
 * gives zeros and is reported by apa_check_error.  T = 0 does nothing. */
int apa_cache_read(const uint8_t* pages, int num_pages, int dtype, int Hkv, int T, int d, const int32_t* slots,
                   const float* k_scale, const float* v_scale, void* k, void* v, cudaStream_t stream);

/* Attention of the last Nq query rows of each sequence over the cache (Nq = 1:
 * decoding; a few: drafted tokens, or the end of a prompt).  Row i of sequence b, at
 * position p = lens[b] - Nq + i, sees key j iff j <= p and, with window >= 1,
 * (j > p - window or j < sinks); window = 0: every key up to p.
 *   q        dtype [B][Hq][Nq][d]; channels contiguous, the rest at the given strides
 *            (in elements, multiples of 8; of an axis of length 1 any); 16-byte aligned
 *   block_table  int32 [B][max_pages]: entry t of sequence b is the page of its keys
 *            64t .. 64t+63; an entry outside the pool reads page 0 and is reported by
 *            apa_check_error (only entries of visible keys are read)
 *   lens     int32 [B]: keys per sequence, the rows' own among them, in
 *            [0, 64 * max_pages] (others are clamped to it and reported).  Keys past
 *            lens[b] or between the sinks and the first row's window, and whatever a
 *            page holds there, are never used.  (With Nq > 1, a NaN in V at a key that
 *            some of the sequence's rows see may reach the others' outputs too.)
 *   out      dtype [B][Hq][Nq][d], contiguous; a row that sees no key is zero
 *   lse      fp32 [B][Hq][Nq], natural log (nullable); -inf for such a row
 *   workspace  apa_attention_cache_workspace_bytes() bytes, 256-byte aligned, or null
 *            to have it allocated stream-ordered for the call.  Two calls that overlap
 *            on the GPU must not share one.
 * K, V and Q enter the products exactly (E2M1 * UE4M3 and a row of Q times a power of
 * two are FP16 values, but for values of Q below 2^-31 of their row's largest, which are
 * rounded at 2^-39 of it), with FP32 accumulation; the softmax weights are
 * rounded to FP16 for the product with V.  B <= 8192, B * max_pages < 2^29.  The work is
 * split over the GPU by the lengths alone, so reruns are bitwise equal. */
int apa_attention_cache(const void* q, int dtype, long long q_batch_stride, long long q_head_stride,
                        long long q_row_stride, const uint8_t* pages, int num_pages, const int32_t* block_table,
                        int max_pages, const int32_t* lens, const float* k_scale, const float* v_scale, int B, int Hq,
                        int Hkv, int Nq, int d, int window, int sinks, void* out, float* lse, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream);
size_t apa_attention_cache_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d);

/* Measurement aid, off by default.  While enabled, every apa_attention* call
 * records CUDA events on its stream around its three stages (quantizer, pass 1,
 * pass 2 with the merge); enabling or disabling resets the record. */
int apa_stage_timing(int enable);
/* Waits for the recorded events and returns the summed milliseconds per stage in
 * ms[0..2] (quantizer, pass 1, pass 2) and the number of calls in *calls, then
 * clears the record.  At eps = 0 only the pass-2 stage has work. */
int apa_stage_timing_read(float* ms, int* calls);

/* Synchronizes `stream`, then returns APA_ERR_DEVICE (and clears the word) if a
 * kernel of this library recorded a device-side timeout on the current device,
 * APA_ERR_CUDA if the stream reported an error, APA_OK otherwise. */
int apa_check_error(cudaStream_t stream);

/* Human-readable text for a status code (static storage). */
const char* apa_status_string(int status);

#ifdef __cplusplus
}
#endif
#endif /* APA_H */
