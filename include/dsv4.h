/*
 * dsv4.h -- C ABI of the GB300 (sm_103a) DeepSeek-V4 sparse-MLA decode library.
 *
 * One decode step for a batch of query tokens over a paged FP8 KV cache:
 *   1. per token, merge the top-k selected positions with the sliding window
 *      (SWA), dropping invalid, non-causal, in-window and repeated entries;
 *   2. translate each logical position to a physical cache slot through the
 *      block table and gather + dequantise the 656-byte entries;
 *   3. MQA attention of all heads over those keys: logits over the 576-d key
 *      (512 latent + 64 RoPE), values = the 512-d latent, an optional per-head
 *      sink logit in the softmax normaliser;
 *   4. BF16 output [T, H, 512] and a natural-log LSE per (token, head).
 *
 * Sources of the operations (vLLM pull-request summaries):
 *   - "[ROCm] [DSv4] [Perf] Support DeepSeek v4 MTP" (vllm #43385), section
 *     "关键源码片段 / rocm.py": _combine_topk_swa_indices_kernel / combine_topk_swa_indices
 *     (top-k entries then the window [pos - swa_len + 1, pos], swa_len = min(pos + 1, W),
 *     validity test, combined_lens = topk part + swa part, 128-aligned padded width).
 *   - "feat: add DeepSeek-V4 XPU attention decode path" (vllm #42953), section
 *     "xpu_sparse_decode_fp8.py": _dequant_gather_slots_kernel (slot -> block / offset,
 *     value = e4m3 * exp2(ue8m0 - 127), negative slot -> no contribution) and
 *     xpu_sparse_decode_fp8 / triton_bf16_mla_sparse_interface (sparse MLA over the
 *     gathered keys, with per-token top-k lengths).
 *   - "Enable DeepSeek V4 and GLM-5.1 on SM120" (vllm #43477), section
 *     "flashinfer_mla_sparse_sm120.py": forward_mqa converts per-request top-k indices to
 *     physical slots through the block table and writes output [T, h, kv_lora_rank = 512];
 *     "flashinfer_sparse.py": supports_sink.
 *
 * Conventions for every entry point:
 *   - All array pointers are DEVICE pointers unless stated otherwise; the caller owns
 *     all memory.  The library never allocates device memory in a call.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default stream)
 *     and never synchronise it.  Kernels run on the current CUDA device.
 *   - Argument errors are detected on the host and returned before anything is
 *     enqueued.  Errors that depend on device data (an out-of-range block-table entry,
 *     an out-of-range request index) do not stop the kernels: the offending key is left
 *     out of the result and a sticky per-device status word records the error; read it
 *     with dsv4_get_device_status().
 *   - All integer sizes and strides are in elements of the array's own type.
 *
 * KV-cache entry (656 bytes; entries are token-major inside a page, page stride
 * page_block * 656 bytes):
 *   [0, 512)    512 E4M3FN latent codes (OCP FP8: bias 7, max 448, S.1111.111 = NaN)
 *   [512, 640)  64 BF16 RoPE values, little-endian
 *   [640, 644)  4 UE8M0 scale bytes; byte b scales latent dims [128 b, 128 b + 128) by 2^(byte - 127)
 *   [644, 656)  padding (not read as data)
 * The key is k = [latent * scale, rope] (576 dims); the value is v = latent * scale (512 dims).
 */
#ifndef DSV4_H_
#define DSV4_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define DSV4_API __attribute__((visibility("default")))
#else
#define DSV4_API
#endif

struct CUstream_st;
/* Same type as cudaStream_t. */
typedef struct CUstream_st *dsv4_stream_t;

typedef enum dsv4_status {
    DSV4_OK = 0,
    DSV4_ERR_INVALID_ARG = 1,   /* bad pointer, size, stride, alignment or workspace size */
    DSV4_ERR_BAD_INDEX = 2,     /* device status only: a block-table or request index was out of range */
    DSV4_ERR_TIMEOUT = 3,       /* device status only: a bounded wait inside a kernel gave up */
    DSV4_ERR_CUDA = 4,          /* a CUDA runtime call or kernel launch failed */
    DSV4_ERR_UNSUPPORTED = 5    /* valid request this build does not implement (e.g. num_heads) */
} dsv4_status;

/*
 * dsv4_combine_topk_swa_indices -- per-token index list: kept top-k entries, then the window.
 *
 * Source: vllm #43385 "[ROCm] [DSv4] [Perf] Support DeepSeek v4 MTP", section
 * "关键源码片段 / rocm.py", _combine_topk_swa_indices_kernel.  This library reads one
 * cache region for both parts, so (where the page's kernel indexes two disjoint regions)
 * it additionally drops top-k entries that the window already covers and repeats, and
 * compacts the kept entries.
 *
 * For token t with pos = seq_lens[t] - 1 and n = min(max(topk_lens[t], 0), topk_width)
 * (n = topk_width when topk_lens is NULL):
 *   window   = [max(0, pos - window + 1), pos]   (empty when pos < 0 or window == 0)
 *   kept     = topk_idx[t][i] for i < n, in order of i, when 0 <= value <= pos, value is
 *              not inside the window, and no earlier i' < i holds the same value
 *   combined[t][0 .. L)      = kept entries, then the window positions ascending
 *   combined[t][L .. width)  = -1
 *   combined_lens[t]         = L = |kept| + window length
 *
 * Arguments:
 *   topk_idx        int32 [num_tokens, topk_width], row stride topk_stride (>= topk_width);
 *                   may be NULL when topk_width == 0.
 *   topk_width      0 .. 8192.
 *   topk_lens       int32 [num_tokens] or NULL.
 *   seq_lens        int32 [num_tokens]: causal visible length of each token (its position + 1).
 *   num_tokens      >= 0 (0 enqueues nothing).
 *   window          >= 0.
 *   combined        int32 [num_tokens, combined_width], row stride combined_stride (>= combined_width).
 *   combined_width  >= topk_width + window (callers usually round up to a multiple of 128).
 *   combined_lens   int32 [num_tokens].
 * Returns DSV4_OK, DSV4_ERR_INVALID_ARG, DSV4_ERR_UNSUPPORTED (topk_width > 8192) or DSV4_ERR_CUDA.
 */
DSV4_API dsv4_status dsv4_combine_topk_swa_indices(const int32_t *topk_idx, int64_t topk_stride, int32_t topk_width,
                                          const int32_t *topk_lens, const int32_t *seq_lens, int32_t num_tokens,
                                          int32_t window, int32_t *combined, int64_t combined_stride,
                                          int32_t combined_width, int32_t *combined_lens, dsv4_stream_t stream);

/*
 * dsv4_combine_topk_swa_indices_compressed -- per-token index lists over a compressed region
 * plus the raw window, for batches of multi-token requests (prefill chunks, speculative verify).
 *
 * Source: vllm #43385 "[ROCm] [DSv4] [Perf] Support DeepSeek v4 MTP", section
 * "关键源码片段 / rocm.py", _combine_topk_swa_indices_kernel with COMPRESS_RATIO, gather_lens
 * and query_start_loc.  Request b owns a gathered region of region_stride (M) entries:
 * compressed_len (N) compressed entries, which top-k indexes, then the raw positions from
 * gather_start = seq_lens[b] - gather_lens[b] on.  Its tokens are rows
 * [query_start_loc[b] - query_start_loc[0], query_start_loc[b + 1] - query_start_loc[0]);
 * token i of a request with query_len tokens sits at pos = seq_lens[b] - query_len + i and gets
 *   topk_len = min((pos + 1) / compress_ratio, top_k)   (0 when pos + 1 <= 0)
 *   swa_len  = min(pos + 1, window)                      (0 when pos + 1 <= 0)
 *   combined[t][k]            = M*b + topk_idx[t][k] when 0 <= topk_idx[t][k] < N, else -1
 *                               (k < topk_len; invalid entries stay in place, -1)
 *   combined[t][topk_len + j] = M*b + N + (pos - swa_len + 1 - gather_start) + j   (j < swa_len)
 *   combined[t][topk_len + swa_len .. combined_width) = -1
 *   combined_lens[t]          = topk_len + swa_len
 * The two parts index different regions, so nothing is deduplicated.  The arithmetic is 32-bit
 * two's complement, as on the page.
 *
 * Arguments:
 *   topk_idx         int32 [num_tokens, topk_width], row stride topk_stride (>= topk_width);
 *                    may be NULL when top_k == 0.
 *   query_start_loc  int32 [num_reqs + 1], non-decreasing, query_start_loc[num_reqs] -
 *                    query_start_loc[0] == num_tokens (rows no request covers are set to -1
 *                    with length 0 and flag DSV4_ERR_BAD_INDEX in the device status word).
 *   seq_lens, gather_lens  int32 [num_reqs].
 *   num_reqs         >= 0; num_tokens >= 0 (either 0 enqueues nothing).
 *   region_stride, compressed_len  >= 0, region_stride * num_reqs < 2^31.
 *   top_k            0 .. topk_width (<= 8192); compress_ratio >= 1; window >= 0.
 *   combined         int32 [num_tokens, combined_width], row stride combined_stride
 *                    (>= combined_width); combined_width >= top_k + window.
 *   combined_lens    int32 [num_tokens].
 * Returns DSV4_OK, DSV4_ERR_INVALID_ARG, DSV4_ERR_UNSUPPORTED (topk_width > 8192) or DSV4_ERR_CUDA.
 */
DSV4_API dsv4_status dsv4_combine_topk_swa_indices_compressed(
    const int32_t *topk_idx, int64_t topk_stride, int32_t topk_width, const int32_t *query_start_loc,
    const int32_t *seq_lens, const int32_t *gather_lens, int32_t num_reqs, int32_t num_tokens, int32_t region_stride,
    int32_t compressed_len, int32_t top_k, int32_t compress_ratio, int32_t window, int32_t *combined,
    int64_t combined_stride, int32_t combined_width, int32_t *combined_lens, dsv4_stream_t stream);

/*
 * dsv4_selftest_wait_timeout -- checks the bounded waits and the status path without a fault.
 *
 * Every wait of the tensor-core decode kernel on an mbarrier gives up after a limit (about two
 * seconds), records DSV4_ERR_TIMEOUT in the device status word and lets the kernel run to its
 * end, so a lost arrival never hangs the GPU.  This call launches one small kernel whose single
 * thread runs that same bounded wait, with a limit of `cycles` SM clock cycles (1 .. 2^31), on
 * an mbarrier nothing arrives on: the next dsv4_get_device_status returns DSV4_ERR_TIMEOUT and
 * the context stays usable.  Returns DSV4_OK, DSV4_ERR_INVALID_ARG or DSV4_ERR_CUDA.
 */
DSV4_API dsv4_status dsv4_selftest_wait_timeout(int64_t cycles, dsv4_stream_t stream);

/*
 * dsv4_qnorm_rope_kv_insert -- the step before the decode: normalise and rotate the queries and
 * write each token's key into the FP8 cache.
 *
 * Source: vllm #42953 "feat: add DeepSeek-V4 XPU attention decode path", section 实现拆解 4
 * (xpu_qnorm_rope_kv_fp8_insert: fused Q per-head RMSNorm, GPT-J RoPE and FP8 UE8M0 KV insert,
 * called from forward_mqa with q, kv, kv_cache, slot_mapping and positions).  The page names
 * the steps, not their formulas; this library's readings:
 *   q_out[t][h] = RoPE(q[t][h] / sqrt(mean over 576 dims of q[t][h]^2 + eps) * w)
 *   kv_cache[slot_mapping[t]] = entry(kv[t]): per 128 latent values the smallest e with
 *       448 * 2^e >= amax (0 for amax 0, clamped to [-127, 127]), E4M3 codes of x * 2^-e
 *       (nearest, ties to even), scale byte e + 127; the rotated rope part in BF16; zero padding
 * GPT-J RoPE rotates the interleaved pairs (512 + 2i, 513 + 2i), i < 32, by the angle whose
 * cosine and sine are cos_sin_cache[positions[t]][i] and [32 + i].  The arithmetic is fp32 with
 * one rounding to BF16 (queries) or E4M3/BF16 (entries) at the end.
 *
 * Arguments:
 *   q, q_out         BF16 [num_tokens, num_heads, 576], token strides in elements (even, >=
 *                    num_heads * 576); q_out may be q (with its stride).  Both 4-byte aligned.
 *   num_heads        1..128; q_norm_weight fp32 [576] or NULL (all ones); eps >= 0.
 *   kv               BF16 [num_tokens, 576] (512 latent, then 64 rope), token stride even, >= 576.
 *   positions, slot_mapping  int64 [num_tokens].
 *   cos_sin_cache    fp32 [max_position, 64]: 32 cosines, then 32 sines per position.
 *   kv_cache         uint8 [num_slots, 656] (a paged cache [num_blocks, page, 656] has
 *                    num_blocks * page slots), 16-byte aligned.
 * A negative slot writes nothing (a padding token).  A slot >= num_slots, or a position outside
 * [0, max_position), writes no entry and sets DSV4_ERR_BAD_INDEX in the device status word; such
 * a token's query is normalised but not rotated.  Nothing is allocated.  Returns DSV4_OK,
 * DSV4_ERR_INVALID_ARG or DSV4_ERR_CUDA.
 */
DSV4_API dsv4_status dsv4_qnorm_rope_kv_insert(const void *q, int64_t q_token_stride, void *q_out,
                                               int64_t q_out_token_stride, int32_t num_tokens, int32_t num_heads,
                                               const float *q_norm_weight, float eps, const void *kv,
                                               int64_t kv_token_stride, const int64_t *positions,
                                               const int64_t *slot_mapping, const float *cos_sin_cache,
                                               int32_t max_position, void *kv_cache, int64_t num_slots,
                                               dsv4_stream_t stream);

/*
 * dsv4_topk_select -- each token's top-k row from its indexer scores (the step that produces
 * topk_idx for the decode).
 *
 * Source: vllm #40860 "[Model] DeepSeek V4", section 实现拆解 2 (the MLA wrapper runs the
 * Indexer ahead of the sparse attention).  The pages print no selection rule; this is the
 * plain definition.  Token t's candidates are positions [0, n), n = num_cand[t] clamped to
 * [0, score_width]; the selected set is the min(top_k, n) candidates that come first in the
 * order "larger score first, then the smaller position", where -0 equals +0 and a NaN score
 * ranks below every number.
 *   topk_idx[t][0 .. m)        the selected positions in ascending order, m = min(top_k, n)
 *   topk_idx[t][m .. top_k)    -1
 *   topk_lens[t]               m
 *
 * Arguments:
 *   scores       fp32 [num_tokens, score_width], row stride score_stride (>= score_width).
 *   num_cand     int32 [num_tokens]: candidates per token (a decode token at position pos
 *                has pos + 1 raw positions, or (pos + 1) / ratio compressed entries).
 *   num_tokens   >= 0 (0 enqueues nothing); top_k >= 1.
 *   topk_idx     int32 [num_tokens, top_k], row stride topk_stride (>= top_k).
 *   topk_lens    int32 [num_tokens], or NULL.
 * All buffers are device memory owned by the caller; nothing is allocated.  The scores are
 * read from HBM once and up to four more times from L2 (the histogram rounds and the final
 * pass).  Returns DSV4_OK, DSV4_ERR_INVALID_ARG or DSV4_ERR_CUDA.
 */
DSV4_API dsv4_status dsv4_topk_select(const float *scores, int64_t score_stride, int32_t score_width,
                                      const int32_t *num_cand, int32_t num_tokens, int32_t top_k, int32_t *topk_idx,
                                      int64_t topk_stride, int32_t *topk_lens, dsv4_stream_t stream);

/*
 * dsv4_sparse_mla_decode_workspace_size -- bytes of device workspace dsv4_sparse_mla_decode needs.
 *
 * The size depends on the arguments and on the multiprocessor count of the current
 * CUDA device (it fixes how many workers share one token's keys); query it with the
 * device that will run the decode current.  Returns 0 for arguments the decode rejects.
 */
DSV4_API size_t dsv4_sparse_mla_decode_workspace_size(int32_t num_tokens, int32_t num_heads, int32_t topk_width,
                                             int32_t window);

/*
 * dsv4_sparse_mla_decode -- one sparse-MLA decode step (combine + gather/dequant + attention).
 *
 * Sources: the three pages named at the top of this file (combine: vllm #43385 rocm.py;
 * gather + dequant + BF16 sparse MLA: vllm #42953 xpu_sparse_decode_fp8.py; block-table
 * conversion, output [T, h, 512], sinks: vllm #43477 flashinfer_mla_sparse_sm120.py).
 *
 * For each token t and head h, with K_t the token's combined index list (as
 * dsv4_combine_topk_swa_indices with this call's arguments), row r = req_idx[t] (t when
 * req_idx is NULL), and for each logical position p in K_t the cache entry at
 *     slot = block_table[r][p / page_block] * page_block + p % page_block:
 *   s_p        = softmax_scale * sum_{d < 576} q[t][h][d] * k_p[d]
 *   lse[t][h]  = ln( sum_p e^{s_p} + e^{sink[h]} )        (no sink term when sink is NULL)
 *   out[t][h]  = sum_p e^{s_p - lse[t][h]} * v_p            (BF16, round-to-nearest-even)
 * A token with no key and no sink gets out = 0 and lse = -inf.  The sink is a logit in
 * the same units as s (it is not multiplied by softmax_scale).
 *
 * Arguments:
 *   q               BF16 [num_tokens, num_heads, 576]; heads contiguous (stride 576),
 *                   tokens at stride q_token_stride (>= num_heads * 576, multiple of 8).
 *                   16-byte aligned.
 *   kv_cache        uint8 [num_blocks, page_block, 656] (layout above), 16-byte aligned.
 *   block_table     int32 [num_reqs, max_blocks], row stride bt_stride (>= max_blocks).
 *                   Entries read must lie in [0, num_blocks); others are data errors.
 *   req_idx         int32 [num_tokens]: the block-table row of each token, in [0, num_reqs);
 *                   NULL means row t (then num_reqs >= num_tokens).  Several tokens may
 *                   share a row (speculative verify: one request, several positions).
 *   topk_idx, topk_stride, topk_width, topk_lens, seq_lens, window: as in
 *                   dsv4_combine_topk_swa_indices.  seq_lens[t] - 1 must be < max_blocks *
 *                   page_block for positions the token reads; others are data errors.
 *   num_tokens      >= 0 (0 enqueues nothing).
 *   num_heads       16, 32, 64 or 128 (others: DSV4_ERR_UNSUPPORTED).
 *   sink            float32 [num_heads] or NULL.
 *   softmax_scale   finite and >= 0 (a negative scale returns DSV4_ERR_INVALID_ARG; 0 gives uniform weights).
 *   out             BF16 [num_tokens, num_heads, 512], contiguous, 16-byte aligned.
 *   lse             float32 [num_tokens, num_heads], contiguous, or NULL.
 *   workspace       device scratch of at least dsv4_sparse_mla_decode_workspace_size(...)
 *                   bytes, 256-byte aligned, not used by anything else until the work
 *                   enqueued by this call has finished.  Its contents on entry do not matter.
 *   stream          CUDA stream.
 * When topk_lens is given and num_tokens * ceil(num_heads / 64) exceeds the device's
 * multiprocessor count, the call enqueues a one-CTA ordering kernel ahead of the decode kernel,
 * so that the tokens with the longest lists start first; the results do not depend on it.
 * Returns DSV4_OK, DSV4_ERR_INVALID_ARG, DSV4_ERR_UNSUPPORTED or DSV4_ERR_CUDA.
 */
DSV4_API dsv4_status dsv4_sparse_mla_decode(const void *q, int64_t q_token_stride, const void *kv_cache, int32_t num_blocks,
                                   int32_t page_block, const int32_t *block_table, int64_t bt_stride,
                                   int32_t max_blocks, int32_t num_reqs, const int32_t *req_idx,
                                   const int32_t *topk_idx, int64_t topk_stride, int32_t topk_width,
                                   const int32_t *topk_lens, const int32_t *seq_lens, int32_t num_tokens,
                                   int32_t num_heads, int32_t window, const float *sink, float softmax_scale,
                                   void *out, float *lse, void *workspace, size_t workspace_bytes,
                                   dsv4_stream_t stream);

/*
 * dsv4_sparse_mla_decode_trace -- dsv4_sparse_mla_decode that also records, from inside the
 * decode kernel, the combined index list each token was decoded over.
 *
 * A verification aid with no counterpart on the pages: the decode kernel combines each
 * token's top-k row with its window itself (the combine of dsv4_combine_topk_swa_indices,
 * vllm #43385 rocm.py, fused into the kernel's prologue); this entry point runs exactly that
 * kernel and lets a test compare the list it built with the definition bit for bit.
 *
 * Arguments: those of dsv4_sparse_mla_decode, then
 *   combined        int32 [num_tokens, combined_width], row stride combined_stride
 *                   (>= combined_width >= topk_width + window): entries [0, L) of row t
 *                   receive the logical positions of token t's keys in list order (the
 *                   kept top-k entries, then the window ascending); entries from L on are
 *                   not written.
 *   combined_lens   int32 [num_tokens]: L of each token.
 * The decode's out and lse are written as by dsv4_sparse_mla_decode.  Returns the codes of
 * dsv4_sparse_mla_decode, and DSV4_ERR_INVALID_ARG for a missing or too narrow record.
 */
DSV4_API dsv4_status dsv4_sparse_mla_decode_trace(const void *q, int64_t q_token_stride, const void *kv_cache,
                                                 int32_t num_blocks, int32_t page_block, const int32_t *block_table,
                                                 int64_t bt_stride, int32_t max_blocks, int32_t num_reqs,
                                                 const int32_t *req_idx, const int32_t *topk_idx,
                                                 int64_t topk_stride, int32_t topk_width, const int32_t *topk_lens,
                                                 const int32_t *seq_lens, int32_t num_tokens, int32_t num_heads,
                                                 int32_t window, const float *sink, float softmax_scale, void *out,
                                                 float *lse, void *workspace, size_t workspace_bytes,
                                                 int32_t *combined, int64_t combined_stride, int32_t combined_width,
                                                 int32_t *combined_lens, dsv4_stream_t stream);

/*
 * dsv4_sparse_mla_decode_noalloc -- dsv4_sparse_mla_decode without a workspace argument.
 *
 * The pages have no counterpart to this entry point; it exists for callers that cannot
 * allocate device memory when they decode: code replaying a pipeline whose memory was
 * fixed at set-up, plug-ins whose host framework owns every allocation, and runtimes that
 * forbid cudaMalloc between start-up and shutdown.  It computes exactly what
 * dsv4_sparse_mla_decode computes, with the same arguments except `workspace` and
 * `workspace_bytes`: the scratch comes from one static device array inside the library,
 * 32 MiB (33,554,432 bytes), which every GPU that loads the library holds until the process
 * exits.  Nothing is allocated in the call.
 *
 * - A batch whose dsv4_sparse_mla_decode_workspace_size(...) exceeds 32 MiB is rejected with
 *   DSV4_ERR_UNSUPPORTED before anything is enqueued; use dsv4_sparse_mla_decode for it.
 * - The first call on a device looks up the array's device address (cudaGetSymbolAddress);
 *   make that first call before any stream capture on that device.
 * - All calls on a device share the one array and leave their scratch in it.  Nothing in it
 *   needs to start at zero (each call writes every scratch value before reading it), but
 *   calls whose work overlaps on the GPU -- on different streams, or on one stream without
 *   ordering -- race on the array; serialise them.
 * Returns the same codes as dsv4_sparse_mla_decode, plus DSV4_ERR_UNSUPPORTED for a batch
 * too large for the array and DSV4_ERR_CUDA when the address lookup fails.
 */
DSV4_API dsv4_status dsv4_sparse_mla_decode_noalloc(const void *q, int64_t q_token_stride, const void *kv_cache,
                                                   int32_t num_blocks, int32_t page_block, const int32_t *block_table,
                                                   int64_t bt_stride, int32_t max_blocks, int32_t num_reqs,
                                                   const int32_t *req_idx, const int32_t *topk_idx,
                                                   int64_t topk_stride, int32_t topk_width, const int32_t *topk_lens,
                                                   const int32_t *seq_lens, int32_t num_tokens, int32_t num_heads,
                                                   int32_t window, const float *sink, float softmax_scale, void *out,
                                                   float *lse, dsv4_stream_t stream);

/*
 * dsv4_sparse_mla_decode_mtp_union -- dsv4_sparse_mla_decode for speculative-verify batches in
 * which the two query tokens of a request run in one tile over the union of their key lists.
 *
 * Source: "[ROCm] [DSv4] [Perf] Support DeepSeek v4 MTP" (vllm #43385), 风险 1 (MTP throughput
 * falls at high concurrency because each request's tokens gather their keys separately); the
 * per-token result is that of dsv4_sparse_mla_decode.
 *
 * Computes exactly what dsv4_sparse_mla_decode computes for the same arguments (up to the
 * order in which a token's keys are summed), with this batch layout: num_tokens is even and
 * tokens 2r and 2r + 1 are the two query tokens of request r, which share a block-table row
 * (req_idx[2r] == req_idx[2r + 1]).  Each CTA takes 32 heads of both tokens (64 tile columns)
 * and the union of the two tokens' combined lists, each key masked for the token that does not
 * list it; a CTA of dsv4_sparse_mla_decode takes 64 heads of one token.
 *
 * Arguments: those of dsv4_sparse_mla_decode, with
 *   req_idx         required (not NULL);
 *   num_tokens      even, >= 0;
 *   num_heads       32, 64 or 128 (others: DSV4_ERR_UNSUPPORTED);
 *   num_blocks * page_block < 2^29;
 *   workspace       at least dsv4_sparse_mla_decode_mtp_union_workspace_size(...) bytes.
 * A request whose two tokens name different block-table rows, or a position of 2^29 or more,
 * is a data error (recorded in the status word; the request's outputs are then not defined).
 * Enqueues the combine of every token, one union kernel (one CTA a request) and the decode
 * kernel.  Returns the codes of dsv4_sparse_mla_decode.
 */
DSV4_API dsv4_status dsv4_sparse_mla_decode_mtp_union(const void *q, int64_t q_token_stride, const void *kv_cache,
                                                     int32_t num_blocks, int32_t page_block,
                                                     const int32_t *block_table, int64_t bt_stride,
                                                     int32_t max_blocks, int32_t num_reqs, const int32_t *req_idx,
                                                     const int32_t *topk_idx, int64_t topk_stride,
                                                     int32_t topk_width, const int32_t *topk_lens,
                                                     const int32_t *seq_lens, int32_t num_tokens, int32_t num_heads,
                                                     int32_t window, const float *sink, float softmax_scale,
                                                     void *out, float *lse, void *workspace, size_t workspace_bytes,
                                                     dsv4_stream_t stream);

/*
 * dsv4_sparse_mla_decode_mtp_union_workspace_size -- bytes of device workspace
 * dsv4_sparse_mla_decode_mtp_union needs (0 for arguments it rejects); depends on the current
 * device's multiprocessor count, as dsv4_sparse_mla_decode_workspace_size.
 */
DSV4_API size_t dsv4_sparse_mla_decode_mtp_union_workspace_size(int32_t num_tokens, int32_t num_heads,
                                                               int32_t topk_width, int32_t window);

/*
 * ---- the 4-bit cache --------------------------------------------------------------------------
 *
 * Cache entry in 4 bits (400 bytes; entries are token-major inside a page, page stride
 * page_block * 400 bytes):
 *   [0, 256)    512 E2M1 latent codes, element 2i in the low half of byte i, 2i + 1 in the high half
 *               (code s.ee.m: magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6)
 *   [256, 384)  64 BF16 RoPE values, little-endian
 *   [384, 400)  16 UE8M0 scale bytes; byte b scales latent dims [32 b, 32 b + 32) by 2^(byte - 127)
 *               (255: NaN)
 * The key is k = [latent * scale, rope] (576 dims); the value is v = latent * scale (512 dims).
 */

/*
 * dsv4_sparse_mla_decode_fp4 -- dsv4_sparse_mla_decode over a cache of 4-bit entries.
 *
 * No page has a 4-bit cache: this is the decode of dsv4_sparse_mla_decode (same lists, same
 * formulas, same outputs) with the entry above, which takes 61 % of the bytes.  The dequantised
 * keys are exact in BF16 (a product past its range becomes an infinity, as rounding to BF16 does).
 * The softmax's weights are rounded to BF16 for their product with the values, as there.  With few tokens
 * (num_tokens * ceil(num_heads / 64) up to half the multiprocessors) the output is divided by the sum of the
 * rounded weights, so that the rounding of a key that has most of the weight cancels; with more by that of
 * the exact ones: a token's last bits depend on the size of its batch.  The lse is that of the exact weights.
 * Weights are held relative to a logit that may lie 40 ln 2 below the largest, so the fp32 sums over a list of
 * up to 2^24 keys stay in range for latent values below 2^64; larger ones may become infinite.
 *
 * Arguments: those of dsv4_sparse_mla_decode, with
 *   kv_cache        uint8 [num_blocks, page_block, 400], 16-byte aligned (num_blocks may be 0);
 *   workspace       at least dsv4_sparse_mla_decode_fp4_workspace_size(...) bytes, 256-byte aligned,
 *                   not used by anything else until the work enqueued by this call has finished (two
 *                   captured graphs that may run at the same time need a workspace each).  It
 *                   holds the tokens' lists (4 (topk_width + window) bytes a token) and, where several
 *                   thread blocks share a token, their parts (264 KB a multiprocessor at most).
 * One to three launches: the lists (few tokens: made by the decode), the decode, and a join where thread
 * blocks share a token.  Results do not depend on timing.  A token whose list is empty gets out = 0 and
 * lse = the sink (-inf without one), as does a head whose logits are all -inf; a sink of +inf gives
 * out = 0 and lse = +inf.
 * Returns DSV4_OK, DSV4_ERR_INVALID_ARG, DSV4_ERR_UNSUPPORTED (num_heads, topk_width) or DSV4_ERR_CUDA.
 */
DSV4_API dsv4_status dsv4_sparse_mla_decode_fp4(const void *q, int64_t q_token_stride, const void *kv_cache,
                                                int32_t num_blocks, int32_t page_block, const int32_t *block_table,
                                                int64_t bt_stride, int32_t max_blocks, int32_t num_reqs,
                                                const int32_t *req_idx, const int32_t *topk_idx, int64_t topk_stride,
                                                int32_t topk_width, const int32_t *topk_lens, const int32_t *seq_lens,
                                                int32_t num_tokens, int32_t num_heads, int32_t window,
                                                const float *sink, float softmax_scale, void *out, float *lse,
                                                void *workspace, size_t workspace_bytes, dsv4_stream_t stream);

/* Bytes of device workspace dsv4_sparse_mla_decode_fp4 needs; 0 for arguments it rejects. */
DSV4_API size_t dsv4_sparse_mla_decode_fp4_workspace_size(int32_t num_tokens, int32_t num_heads, int32_t topk_width,
                                                          int32_t window);

/*
 * dsv4_qk_norm_rope_kv_insert_fp4 -- norms of the queries (per head) and of the key, the rotation of
 * both, and the insert of the key as a 4-bit entry.
 *
 * Source of the step: vllm #42953, section 实现拆解 4, as dsv4_qnorm_rope_kv_insert; the key's norm is
 * that of vllm #40860 "[Model] DeepSeek V4", section 实现拆解 2 (fused RMSNorm + Rope + Quant).
 *   q_out[t][h] = RoPE(q[t][h] / sqrt(mean over 576 dims of q[t][h]^2 + eps) * w_q)
 *   k[t]        = RoPE(kv[t]), its first n = kv_norm_dims dims divided by sqrt(mean of their squares
 *                 + eps) and multiplied by w_kv before the rotation
 *   kv_cache[slot_mapping[t]] = entry(k[t]): per 32 latent values the smallest e with 6 * 2^e >= amax
 *                 (0 for amax 0, clamped to [-127, 125]), E2M1 codes of k * 2^-e (nearest, ties to
 *                 even), scale byte e + 127; the rope part in BF16
 *   k_out[t]    = the values of that entry in BF16 (what a later decode reads: the chunk's own
 *                 attention can use them without the cache)
 * The rotation is that of dsv4_qnorm_rope_kv_insert.  Queries are computed in fp32 and rounded once;
 * the codes and scales are those of the exact k (fp64 where fp32 could decide otherwise).  A NaN is
 * stored as the code of 6, an infinity as 6 * 2^125.
 *
 * Arguments:
 *   q, q_out         BF16 [num_tokens, num_heads, 576], token strides in elements (even, >=
 *                    num_heads * 576); q_out may be q (with its stride).  Both 4-byte aligned.
 *   num_heads        1..128; q_norm_weight fp32 [576] or NULL (all ones); eps >= 0.
 *   kv_norm_dims     0 (the key is not normalised), 512 (its latent) or 576 (all of it);
 *                    kv_norm_weight fp32 [kv_norm_dims] or NULL (all ones).
 *   kv               BF16 [num_tokens, 576] (512 latent, then 64 rope), token stride even, >= 576.
 *   positions, slot_mapping  int64 [num_tokens].
 *   cos_sin_cache    fp32 [max_position, 64]: 32 cosines, then 32 sines per position.
 *   kv_cache         uint8 [num_slots, 400], 16-byte aligned.
 *   k_out            BF16 [num_tokens, 576], token stride even, >= 576; or NULL.
 * But for q_out = q, a row of q_out or k_out shares no byte with a row of q, kv or the other output (rows may
 * lie between those of another array); such calls are refused.
 * A negative slot writes no entry (a padding token; its queries and k_out are computed).  A slot >=
 * num_slots, or a position outside [0, max_position), writes no entry and sets DSV4_ERR_BAD_INDEX in
 * the device status word; at such a position nothing is rotated.  Two tokens of a call must not name
 * one slot.  Nothing is allocated.  Returns DSV4_OK, DSV4_ERR_INVALID_ARG or DSV4_ERR_CUDA.
 */
DSV4_API dsv4_status dsv4_qk_norm_rope_kv_insert_fp4(
    const void *q, int64_t q_token_stride, void *q_out, int64_t q_out_token_stride, int32_t num_tokens,
    int32_t num_heads, const float *q_norm_weight, const float *kv_norm_weight, int32_t kv_norm_dims, double eps,
    const void *kv, int64_t kv_token_stride, const int64_t *positions, const int64_t *slot_mapping,
    const float *cos_sin_cache, int32_t max_position, void *kv_cache, int64_t num_slots, void *k_out,
    int64_t k_out_token_stride, dsv4_stream_t stream);

/*
 * ---- pages of a cache -------------------------------------------------------------------------
 *
 * A pool is num_layers caches of num_blocks pages, layer l at cache + l * layer_stride bytes, page b of
 * a layer at b * page_block * entry_bytes (entries of 656, 400 or any other multiple of 16 bytes; the
 * base 16-byte aligned, layer_stride a multiple of 16).  All layers share one block table, the rows'
 * lengths and one reference count per page:
 *   block_table  int32 [num_rows, max_blocks]: row r's pages in order, ceil(seq_lens[r] / page_block) of
 *                them; the cells after those are not read
 *   seq_lens     int32 [num_rows] (0 or less: an empty row)
 *   ref_counts   int32 [num_blocks]: the rows (and other holders) that name a page; 0: the page is free
 * The operators below run on the device alone: they can be captured, and no length, count or page number
 * passes through the host.  A page number outside [0, num_blocks), or a length past max_blocks *
 * page_block, in a row that is read sets DSV4_ERR_BAD_INDEX in the device status word; the cell becomes
 * -1, the length is cut (the compact writes no lengths: it reads the row as far as the table goes).
 * ref_counts must count every row of the table that is given.
 *
 * workspace: at least dsv4_cache_pages_workspace_size(num_rows, num_rows_out, num_blocks) bytes (the
 * compact and the copies need no rows: 0, 0), 256-byte aligned, not used by anything else until the
 * call's work has finished.
 */
DSV4_API size_t dsv4_cache_pages_workspace_size(int32_t num_rows, int32_t num_rows_out, int32_t num_blocks);

/*
 * dsv4_cache_fork_rows -- replace the table's rows by copies of them: forking, beam search's choice of
 * parents, and freeing, in one call.
 *
 * Row r of the result is a copy of row parent[r]; a negative parent gives an empty row, and a row that is
 * nobody's parent is freed (parent = 0, 1, .. with -1 for the finished rows frees those and keeps the
 * rest).  Page j of a row is
 *   shared   the parent's page, with one more reference, when `share` is not 0 and the page is full;
 *   kept     the parent's page, for the lowest row of that parent, when its count on entry is 1;
 *   taken    else: a free page that the page's entries are copied into, in every layer, count 1.
 * So a partly filled page always ends with one holder, and appending to a row never writes into
 * another's.  With share = 0 no two rows of the result share a page.  Pages that are free on entry are
 * taken lowest first, in the order of (row, page); pages that this call frees are not taken by it.  A row
 * that would need pages past the last free one becomes an empty row and sets DSV4_ERR_BAD_INDEX in the
 * device status word.
 *
 * Arguments: the pool; block_table, seq_lens [num_rows], ref_counts: the state before the call;
 *   parent           int32 [num_rows_out], each < num_rows (others: an empty row, and the status bit)
 *   block_table_out  int32 [num_rows_out, max_blocks], row stride bt_out_stride; every cell is written
 *                    (-1 after a row's pages).  Must not overlap block_table.
 *   seq_lens_out     int32 [num_rows_out].  Must not overlap seq_lens.
 *   ref_counts_out   int32 [num_blocks]; may be ref_counts.
 * max_blocks <= 2^20, num_blocks <= 2^30.  Of a taken page only the entries that the row holds are
 * written.  Returns DSV4_OK, DSV4_ERR_INVALID_ARG or DSV4_ERR_CUDA.
 */
DSV4_API dsv4_status dsv4_cache_fork_rows(void *cache, int32_t num_layers, int64_t layer_stride, int32_t num_blocks,
                                          int32_t page_block, int32_t entry_bytes, const int32_t *block_table,
                                          int64_t bt_stride, const int32_t *seq_lens, int32_t num_rows,
                                          const int32_t *parent, int32_t num_rows_out, int32_t max_blocks,
                                          int32_t *block_table_out, int64_t bt_out_stride, int32_t *seq_lens_out,
                                          const int32_t *ref_counts, int32_t *ref_counts_out, int32_t share,
                                          void *workspace, size_t workspace_bytes, dsv4_stream_t stream);

/*
 * dsv4_cache_compact -- move the live pages to the front of the pool.
 *
 * With L pages of a count > 0, the k-th of them at or past L (ascending) moves, in every layer, to the k-th
 * free page below L; the other live pages stay.  Afterwards pages [0, L) are live and [L, num_blocks) free.
 *   block_table_out  int32 [num_rows, max_blocks]: block_table with the pages' new numbers, -1 after a
 *                    row's pages; may be block_table (with the same stride)
 *   ref_counts_out   int32 [num_blocks]: the counts of the pages in their new places; may be ref_counts
 *   page_map         int32 [num_blocks]: the new number of each page, -1 for a free one (for page numbers
 *                    that are held elsewhere)
 *   num_live         int32 [1]: L
 * A cell that names a page whose count is 0 becomes -1 and sets DSV4_ERR_BAD_INDEX in the device status
 * word.  The entries of the pages from L on are left as they were.  Returns DSV4_OK, DSV4_ERR_INVALID_ARG
 * or DSV4_ERR_CUDA.
 */
DSV4_API dsv4_status dsv4_cache_compact(void *cache, int32_t num_layers, int64_t layer_stride, int32_t num_blocks,
                                        int32_t page_block, int32_t entry_bytes, const int32_t *block_table,
                                        int64_t bt_stride, const int32_t *seq_lens, int32_t num_rows,
                                        int32_t max_blocks, int32_t *block_table_out, int64_t bt_out_stride,
                                        const int32_t *ref_counts, int32_t *ref_counts_out, int32_t *page_map,
                                        int32_t *num_live, void *workspace, size_t workspace_bytes,
                                        dsv4_stream_t stream);

/*
 * dsv4_cache_copy_pages -- copy the listed pages, in every layer, within a pool or into another one.
 *
 * Page src_pages[i] of src_cache goes to page dst_pages[i] of dst_cache, i < num_pages.  A target that is
 * listed more than once receives its last pair.  In one pool (the same base, layer stride and number of
 * pages), a pair whose source is also a target of the call is left out and sets DSV4_ERR_BAD_INDEX in the
 * device status word, as does a page number out of range; two different pools must not overlap.
 * Workspace: dsv4_cache_pages_workspace_size(0, 0, dst_num_blocks).  Returns DSV4_OK,
 * DSV4_ERR_INVALID_ARG or DSV4_ERR_CUDA.
 */
DSV4_API dsv4_status dsv4_cache_copy_pages(void *dst_cache, int64_t dst_layer_stride, int32_t dst_num_blocks,
                                           const void *src_cache, int64_t src_layer_stride, int32_t src_num_blocks,
                                           int32_t num_layers, int32_t page_block, int32_t entry_bytes,
                                           const int32_t *src_pages, const int32_t *dst_pages, int32_t num_pages,
                                           void *workspace, size_t workspace_bytes, dsv4_stream_t stream);

/*
 * ---- between two decode steps -----------------------------------------------------------------
 *
 * dsv4_verify_drafts -- which of the drafted tokens stand, and the token after them, from given random numbers.
 *
 * The decode's batches of several query tokens a request (vllm #43385 "[ROCm] [DSv4] [Perf] Support DeepSeek v4 MTP") end
 * in this step; the pages print no rule for it.  This is the one that leaves the tokens with the target's distribution.
 * Request b has rows [query_start_loc[b], query_start_loc[b + 1]) - query_start_loc[0] of target probabilities, one for
 * each of its k drafted tokens and one for the token after them.  Draft j of it is
 * row query_start_loc[b] - query_start_loc[0] - b + j of draft_tokens and draft_probs.  With p_j, q_j the probabilities,
 * d_j the drafted tokens and u_j = uniform[row j]:
 *   a         = the number of leading drafts with u_j * q_j(d_j) < p_j(d_j)   (q_j(d_j) = 1 without draft_probs)
 *   w         = p_k when a = k; max(p_a - q_a, 0), or without draft_probs p_a without d_a, when a < k (p_a itself where
 *               that leaves nothing)
 *   token     = the lowest i with w_0 + .. + w_i > u_k * (w_0 + .. + w_{vocab - 1})
 * A greedy request (greedy[b] != 0) accepts while d_j is the index of the largest value of row j (the lowest of equal ones,
 * NaN below every number) and then takes that of row a; its rows may be logits.  One row (k = 0) is plain sampling.
 *   tokens[b]       = d_0 .. d_{a-1}, token, then -1
 *   num_accepted[b] = a
 *   seq_lens_out[b] = seq_lens[b] - (k - a)   (the cache's entries of the drafts that do not stand are dropped)
 * Products and comparisons are exact; sums are held to 2^-40 of themselves or better.  Probabilities are finite (they
 * need not sum to 1, but the positive ones of a row to less than 2^127); negative values and NaN count as 0, in the
 * comparisons as in the sums.
 *
 * Arguments:
 *   target_probs     fp32, or BF16 when probs_bf16 != 0, [num_rows, vocab], row stride target_stride (>= vocab).
 *   draft_probs      the same type, [num_drafts, vocab], row stride draft_stride; or NULL.
 *   vocab            1 .. 2^22.
 *   draft_tokens     int32 [num_drafts]; one outside [0, vocab) does not stand, and wherever it is among its request's
 *                    drafts sets DSV4_ERR_BAD_INDEX in the device status word.
 *   query_start_loc  int32 [num_reqs + 1], increasing: every request has a row or more; num_reqs <= 2^24.
 *   uniform          fp32 [num_rows] in [0, 1).
 *   greedy           uint8 [num_reqs] or NULL (none is).
 *   tokens           int32 [num_reqs, tokens_width], row stride tokens_stride; tokens_width >= k + 1.
 *   num_accepted     int32 [num_reqs].
 *   seq_lens, seq_lens_out  int32 [num_reqs], both or neither; may be one array.
 * tokens, num_accepted and seq_lens_out must not overlap the inputs (seq_lens_out == seq_lens apart) or one another
 * (DSV4_ERR_INVALID_ARG).
 * A request without a row, with rows or drafts outside the arrays, or with more of them than tokens_width gets -1 and
 * a = 0 (its length is kept); one whose row a has no positive value, or sums to 2^127 or more, gets a token of -1.  Both set
 * DSV4_ERR_BAD_INDEX in the device status word.  Nothing is allocated.  Returns DSV4_OK, DSV4_ERR_INVALID_ARG or DSV4_ERR_CUDA.
 */
DSV4_API dsv4_status dsv4_verify_drafts(const void *target_probs, int64_t target_stride, const void *draft_probs,
                                        int64_t draft_stride, int32_t probs_bf16, int32_t vocab,
                                        const int32_t *draft_tokens, int32_t num_drafts, const int32_t *query_start_loc,
                                        int32_t num_reqs, int32_t num_rows, const float *uniform, const uint8_t *greedy,
                                        int32_t *tokens, int64_t tokens_stride, int32_t tokens_width,
                                        int32_t *num_accepted, const int32_t *seq_lens, int32_t *seq_lens_out,
                                        dsv4_stream_t stream);

/*
 * dsv4_sparse_mla_key_weights -- add the attention weight that a decode step gave each key to its place in a table.
 *
 *   weights[row][p] += sum over heads h of e^{s_p - lse[t][h]}
 * for each token t, with row, the positions p of its list K_t and the logits s_p as in dsv4_sparse_mla_decode (8-bit
 * entries) or dsv4_sparse_mla_decode_fp4 (4-bit ones), and the lse that it returned.  A head whose lse is -inf gives
 * nothing, whatever its query is; what a head gives below 2^-126 is 0.  Tokens of one row are added in ascending order,
 * one rounding to fp32 each.  Several layers may be added to one table, a call each.
 * Where some of the tokens are drafts, the call belongs after dsv4_verify_drafts, with a length of 0 for tokens
 * num_accepted + 1 and on of each request: before it, the attention of the drafts that fall is added for good, and their
 * own positions keep a weight that the tokens after them inherit (until an eviction, which clears what lies past a row's end).
 *
 * Arguments: those of the decode, with
 *   entry_bytes     656 or 400 (others: DSV4_ERR_UNSUPPORTED): kv_cache uint8 [num_blocks, page_block, entry_bytes];
 *   lse             fp32 [num_tokens, num_heads];
 *   weights         fp32 [num_reqs, weights_width], row stride weights_stride; weights_width >= max_blocks * page_block;
 *   workspace       at least dsv4_sparse_mla_key_weights_workspace_size(...) bytes, 256-byte aligned, not used by
 *                   anything else until the work enqueued by this call has finished.
 * weights and the workspace must not overlap the inputs or each other (DSV4_ERR_INVALID_ARG).
 * Block-table entries and rows out of range are data errors, as in the decode; such keys are left out.
 * Returns DSV4_OK, DSV4_ERR_INVALID_ARG, DSV4_ERR_UNSUPPORTED (num_heads, topk_width, entry_bytes) or DSV4_ERR_CUDA.
 */
DSV4_API dsv4_status dsv4_sparse_mla_key_weights(
    const void *q, int64_t q_token_stride, const void *kv_cache, int32_t num_blocks, int32_t page_block,
    int32_t entry_bytes, const int32_t *block_table, int64_t bt_stride, int32_t max_blocks, int32_t num_reqs,
    const int32_t *req_idx, const int32_t *topk_idx, int64_t topk_stride, int32_t topk_width, const int32_t *topk_lens,
    const int32_t *seq_lens, int32_t num_tokens, int32_t num_heads, int32_t window, const float *lse,
    float softmax_scale, float *weights, int64_t weights_stride, int32_t weights_width, void *workspace,
    size_t workspace_bytes, dsv4_stream_t stream);

/* Bytes of device workspace dsv4_sparse_mla_key_weights needs; 0 for arguments it rejects. */
DSV4_API size_t dsv4_sparse_mla_key_weights_workspace_size(int32_t num_tokens, int32_t num_heads, int32_t topk_width,
                                                           int32_t window);

/*
 * dsv4_cache_evict -- cut long rows of a cache to a budget of entries, by accumulated attention weight.
 *
 * The pool, block table, lengths and reference counts are those of the page operators above.  A row of n > limit entries
 * keeps its first `first` entries, its last `recent` ones and, of those between, the heaviest: budget in all, in their
 * order (larger weight first, then the lower position; -0 is +0, NaN below every number).  Shorter rows are not changed.
 * Entries move down within the row in every layer.  A decode of the row afterwards takes its length as the number of
 * entries left; they keep the rotation of the positions that they were inserted with.
 *
 * Page j of a row that is cut
 *   stays    when it is full and all of its entries stay where they are, shared or not;
 *   is written in place  otherwise, when its count on entry is 1;
 *   is replaced  else, by a free page (count 1) that receives all of its entries.
 * Pages past the new end, and those replaced, lose a reference.  Pages that are free on entry are taken lowest first, in
 * the order of (row, page); pages that this call frees are not taken by it.  A row that would need pages past the last
 * free one stays as it was and sets DSV4_ERR_BAD_INDEX in the device status word.
 *
 * Arguments: the pool; block_table, seq_lens [num_rows], ref_counts: the state before the call (ref_counts must count
 * every row of the table);
 *   weights          fp32 [num_rows, weights_width], row stride weights_stride; weights_width >= max_blocks * page_block.
 *   budget, limit    1 <= budget <= limit; first, recent >= 0, first + recent <= budget.
 *   block_table_out  int32 [num_rows, max_blocks], row stride bt_out_stride; every cell is written (-1 after a row's
 *                    pages).  Must not overlap block_table.
 *   seq_lens_out     int32 [num_rows].  Must not overlap seq_lens.
 *   ref_counts_out   int32 [num_blocks]; may be ref_counts.
 *   weights_out      fp32 [num_rows, weights_width], row stride weights_out_stride: the kept entries' weights, then 0;
 *                    may be weights (with the same stride).
 *   workspace        at least dsv4_cache_evict_workspace_size(...) bytes, 256-byte aligned, not used by anything else
 *                    until the call's work has finished.
 * The outputs and the workspace must not overlap the inputs, those two pairs apart, or one another (DSV4_ERR_INVALID_ARG).
 * max_blocks <= 2^20, num_blocks <= 2^30.  A page number outside [0, num_blocks) in a row that is read becomes -1, entries
 * on such pages are not moved, a length past max_blocks * page_block is cut; both set DSV4_ERR_BAD_INDEX.  Nothing is
 * allocated; the call can be captured.  Returns DSV4_OK, DSV4_ERR_INVALID_ARG or DSV4_ERR_CUDA.
 */
DSV4_API dsv4_status dsv4_cache_evict(void *cache, int32_t num_layers, int64_t layer_stride, int32_t num_blocks,
                                      int32_t page_block, int32_t entry_bytes, const int32_t *block_table,
                                      int64_t bt_stride, const int32_t *seq_lens, int32_t num_rows, int32_t max_blocks,
                                      const float *weights, int64_t weights_stride, int32_t weights_width,
                                      int32_t budget, int32_t limit, int32_t first, int32_t recent,
                                      int32_t *block_table_out, int64_t bt_out_stride, int32_t *seq_lens_out,
                                      const int32_t *ref_counts, int32_t *ref_counts_out, float *weights_out,
                                      int64_t weights_out_stride, void *workspace, size_t workspace_bytes,
                                      dsv4_stream_t stream);

/* Bytes of device workspace dsv4_cache_evict needs; 0 for arguments it rejects. */
DSV4_API size_t dsv4_cache_evict_workspace_size(int32_t num_rows, int32_t max_blocks, int32_t num_blocks,
                                                int32_t num_layers, int32_t page_block, int32_t entry_bytes,
                                                int32_t budget);

/*
 * dsv4_get_device_status -- synchronise `stream`, then read and clear the current
 * device's sticky status word.
 *
 * Returns DSV4_OK when no kernel of this library on the current device recorded a data
 * error since the last call, DSV4_ERR_BAD_INDEX or DSV4_ERR_TIMEOUT for the recorded
 * error (BAD_INDEX wins when both were recorded), or DSV4_ERR_CUDA when the
 * synchronisation or the read failed.  The word is shared by all streams of the device.
 */
DSV4_API dsv4_status dsv4_get_device_status(dsv4_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DSV4_H_ */
