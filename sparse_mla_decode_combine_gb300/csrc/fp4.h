// fp4.h -- the 4-bit cache entry and the launch interface of its kernels.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.h"

namespace dsv4 {

// 4-bit cache entry (400 bytes): 512 E2M1 latent codes (element 2i in the low half of byte i),
// 64 BF16 rope values, 16 UE8M0 scale bytes (one for each 32 latent values).
constexpr int kEntry4Bytes = 400;
constexpr int kRope4Offset = 256;
constexpr int kScale4Offset = 384;
constexpr int kScale4Block = 32;

// A launch that may begin while the kernel before it in the stream ends (its CTAs are set up by then; 1 to 2 us a launch
// in a stream of small kernels).  The kernel waits for that one with griddep_wait() before it touches memory, and only
// then lets its own dependent begin: what that one reads ahead of its own wait was complete before this kernel.
// Such a kernel is there while the one that writes its inputs runs, so it never takes the non-coherent path of __ldg, which
// wants data that nobody writes during the kernel: __ldca, __ldcg and plain loads (level with it within 0.5 %).
template <typename Params>
cudaError_t launch_dependent(void (*kernel)(const Params), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                             const Params &p)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e != cudaSuccess)
        (void)cudaGetLastError();   // (returned here: a later call of this library must not find it as its own)
    return e;
}

#ifdef __CUDACC__
__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

struct Insert4Params {
    const uint32_t *q;          // BF16 pairs
    int64_t q_stride;           // pairs per token
    uint32_t *q_out;
    int64_t q_out_stride;
    int32_t num_tokens;
    int32_t num_heads;
    const float *q_w;           // [576] or null
    const float *kv_w;          // [kv_norm_dims] or null
    int32_t kv_norm_dims;       // 0, 512 or 576
    double eps;
    const uint32_t *kv;         // BF16 pairs [T][288]
    int64_t kv_stride;          // pairs per token
    const int64_t *positions;
    const int64_t *slots;
    const float *cos_sin;       // [max_pos][64]
    int32_t max_pos;
    uint8_t *cache;
    int64_t num_slots;
    uint32_t *k_out;            // BF16 pairs [T][288] or null
    int64_t k_out_stride;
    unsigned *status;
};
cudaError_t launch_qk_norm_rope_kv_insert_fp4(const Insert4Params &p, cudaStream_t stream);

struct Lists4Params {
    const int32_t *topk;
    int64_t topk_stride;
    int32_t topk_width;
    const int32_t *topk_lens;
    const int32_t *seq_lens;
    int32_t num_tokens;
    int32_t window;
    const int32_t *block_table;
    int64_t bt_stride;
    int32_t max_blocks;
    int32_t num_reqs;
    const int32_t *req_idx;
    int32_t num_blocks;
    int32_t page;
    int32_t *slots;            // [T, list_w]
    int32_t *lens;             // [T]
    int32_t list_w;            // topk_width + window
    int2 *joins;               // [groups * T] set to zero
    int32_t groups;
    // the outputs of tokens without a key
    const float *sink;
    int32_t num_heads;
    uint16_t *out;
    float *lse;
    int32_t smem_bytes;        // shared memory for the sets: lists_fp4_smem_bytes(topk_width)
    unsigned *status;
    // launch_lists_positions alone:
    int32_t *positions;        // [T, list_w]
    int32_t *later;            // [T] 1: a token with keys before this one names its row
};
// the hash set of a row; as a bitmap at least 262144 positions (131072 bytes at the widest rows)
inline int lists_fp4_smem_bytes(int topk_width)
{
    int bytes = 32768;
    while (bytes < 16 * topk_width)
        bytes *= 2;
    return bytes;
}
cudaError_t launch_lists_fp4(const Lists4Params &p, cudaStream_t stream);
// slots, positions and lengths alone (no joins, no outputs of tokens without a key)
cudaError_t launch_lists_positions(const Lists4Params &p, int sms, cudaStream_t stream);

struct Decode4Params {
    const uint16_t *q;
    int64_t q_token_stride;
    const uint8_t *kv;
    const int32_t *slots;      // [T, list_w] cache slots (-1: no key), and how many each token has
    const int32_t *lens;
    int32_t list_w;
    int32_t num_tokens;
    int32_t num_heads;
    const float *sink;
    float scale;
    uint16_t *out;             // BF16 [T, H, 512]
    float *lse;                // [T, H] or null
    int32_t groups;            // 64-head groups
    int32_t grid;              // CTAs
    int32_t ctas_per_unit;     // CTAs that share each unit; 0: every CTA takes an equal run of the blocks of all units
    bool split;                // whether several CTAs may share a unit
    float *parts;              // [2 * grid] partial results of units that several CTAs share
    int2 *joins;               // [groups * T] such a unit's first part and their number, zeros for units that are not shared
    bool own_lists;            // (ctas_per_unit > 0) the CTAs make their token's list themselves:
    Lists4Params lists;
    unsigned *status;
};
cudaError_t launch_decode_fp4(const Decode4Params &p, cudaStream_t stream);
int decode_fp4_block_keys();
int decode_fp4_own_list_width();   // widest top-k rows of which the decode makes the lists itself
size_t decode_fp4_part_bytes();

// ---- page operators

// A pool of pages: num_layers caches of num_blocks pages each, layer_stride bytes apart.
struct PagePool {
    uint8_t *base;
    int32_t num_layers;
    int64_t layer_stride;
    int32_t num_blocks;
    int32_t page;              // entries per page
    int32_t entry_bytes;
};

struct ForkParams {
    PagePool pool;
    const int32_t *table;
    int64_t table_stride;
    const int32_t *lens;
    int32_t rows;
    const int32_t *parent;
    int32_t rows_out;
    int32_t max_blocks;
    int32_t *table_out;
    int64_t table_out_stride;
    int32_t *lens_out;
    const int32_t *refs;
    int32_t *refs_out;
    int32_t share;
    unsigned *status;
    // workspace
    int32_t *first;            // [rows] lowest output row of each parent
    int32_t *kids;             // [rows] output rows that were given room
    int32_t *need;             // [rows_out] pages to take
    int32_t *offset;           // [rows_out] exclusive sums of need
    int32_t *free_list;        // [num_blocks]
    int4 *copies;              // [num_blocks] (source, target, entries, 0)
    int32_t *num_copies;       // [1]
};
cudaError_t launch_fork(const ForkParams &p, int sms, cudaStream_t stream);

struct CompactParams {
    PagePool pool;
    const int32_t *table;
    int64_t table_stride;
    const int32_t *lens;
    int32_t rows;
    int32_t max_blocks;
    int32_t *table_out;
    int64_t table_out_stride;
    const int32_t *refs;
    int32_t *refs_out;
    int32_t *page_map;
    int32_t *num_live;
    unsigned *status;
    // workspace
    int4 *copies;
    int32_t *num_copies;
};
cudaError_t launch_compact(const CompactParams &p, int sms, cudaStream_t stream);

struct CopyPagesParams {
    PagePool dst, src;
    bool one_pool;
    const int32_t *src_pages;
    const int32_t *dst_pages;
    int32_t num_pages;
    unsigned *status;
    // workspace
    int32_t *claim;            // [dst.num_blocks] the pair that writes a target
};
cudaError_t launch_copy_pages(const CopyPagesParams &p, int sms, cudaStream_t stream);

}  // namespace dsv4
