// api_fp4.cu -- the C ABI of the 4-bit cache and of the page operators (include/dsv4.h): argument
// validation, the carving of the caller's workspace, and the launches on the caller's stream.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdlib>

#include "../../include/dsv4.h"
#include "fp4.h"

using namespace dsv4;

namespace {

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int kMaxWindow = 1 << 24;

// whether [a, a + na) and [b, b + nb) share a byte
bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

// whether any of the `rows` rows of wa bytes from a on, sa bytes apart, shares a byte with one of b's (rows that lie between
// the other array's, as in a buffer that holds queries and keys side by side, do not)
bool rows_overlap(const void *a, int64_t sa, int64_t wa, const void *b, int64_t sb, int64_t wb, int64_t rows)
{
    if (!overlap(a, (size_t)((rows - 1) * sa + wa), b, (size_t)((rows - 1) * sb + wb)))
        return false;
    if (sa != sb || rows == 1)
        return true;
    const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
    const int64_t k = d / sa - (d % sa < 0 ? 1 : 0), r = d - k * sa;   // row j of b begins r bytes into row j + k of a
    return (r < wa && std::llabs(k) < rows) || (r + wb > sa && std::llabs(k + 1) < rows);
}

// ---- the decode's workspace: the tokens' slot lists, their lengths, and the parts of split units
struct Plan4 {
    int list_w, groups, grid, ctas_per_unit;
    bool split;
    size_t off_lens, off_joins, off_parts, total;
};

bool plan4(int num_tokens, int num_heads, int topk_width, int window, int sms, Plan4 *pl)
{
    if (num_tokens < 0 || topk_width < 0 || topk_width > kMaxTopkWidth || window < 0 || window > kMaxWindow)
        return false;
    if (num_heads != 16 && num_heads != 32 && num_heads != 64 && num_heads != 128)
        return false;
    pl->list_w = topk_width + window;
    pl->groups = (num_heads + 63) / 64;
    const int tile = decode_fp4_block_keys();
    if ((long long)num_tokens * pl->groups * std::max(1, (pl->list_w + tile - 1) / tile) > INT_MAX)
        return false;
    // Half as many units as multiprocessors or fewer: each unit is shared by as many CTAs as there are for it (two
    // blocks or more to each).  Otherwise every multiprocessor's CTA takes an equal run of all blocks, which splits units
    // at the runs' ends; with eight or more units to a CTA the runs end between units, which leaves at most an eighth of
    // a CTA's work uneven and nothing to join.
    const int units = num_tokens * pl->groups;
    const int most = std::max(1, (pl->list_w + 2 * tile - 1) / (2 * tile));   // CTAs that a unit's list can use
    pl->ctas_per_unit = units <= sms / 2 ? std::max(1, std::min(sms / std::max(1, units), most)) : 0;
    pl->grid = pl->ctas_per_unit > 0 ? std::max(1, units * pl->ctas_per_unit) : sms;
    pl->split = pl->ctas_per_unit > 0 ? pl->ctas_per_unit > 1 : most > 1 && units < 8ll * sms;
    pl->off_lens = align_up(sizeof(int32_t) * (size_t)num_tokens * (size_t)pl->list_w, 256);
    pl->off_joins = align_up(pl->off_lens + sizeof(int32_t) * (size_t)num_tokens, 256);
    pl->off_parts = align_up(pl->off_joins + sizeof(int2) * (size_t)num_tokens * pl->groups, 256);
    pl->total = std::max<size_t>(256, pl->off_parts + (pl->split ? 2 * decode_fp4_part_bytes() * (size_t)pl->grid : 0));
    return true;
}

// ---- the page operators' workspace
struct PagesPlan {
    size_t first, kids, need, offset, free_list, copies, num_copies, total;
};

constexpr int kMaxPages = 1 << 30, kMaxRowPages = 1 << 20;

bool pages_plan(int rows, int rows_out, int num_blocks, PagesPlan *pl)
{
    if (rows < 0 || rows_out < 0 || num_blocks < 0 || num_blocks > kMaxPages)
        return false;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes, 256);
        return at;
    };
    pl->copies = take(16 * (size_t)num_blocks);
    pl->free_list = take(4 * (size_t)num_blocks);   // (copies of listed pages: the claims)
    pl->first = take(4 * (size_t)rows);
    pl->kids = take(4 * (size_t)rows);
    pl->need = take(4 * (size_t)rows_out);
    pl->offset = take(4 * (size_t)rows_out);
    pl->num_copies = take(4);
    pl->total = off;
    return true;
}

bool pool_ok(const void *cache, int num_layers, int64_t layer_stride, int num_blocks, int page, int entry_bytes)
{
    if (num_layers < 1 || num_blocks < 0 || num_blocks > kMaxPages || page < 1 || entry_bytes < 16 || entry_bytes % 16 != 0)
        return false;
    if ((long long)page * entry_bytes > INT_MAX)
        return false;
    if (num_layers > 1 && (layer_stride % 16 != 0 || layer_stride < (int64_t)num_blocks * page * entry_bytes))
        return false;
    return num_blocks == 0 || (cache != nullptr && aligned(cache, 16));
}

size_t pool_bytes(int num_layers, int64_t layer_stride, int num_blocks, int page, int entry_bytes)
{
    return (size_t)(num_layers - 1) * (size_t)layer_stride + (size_t)num_blocks * page * entry_bytes;
}

size_t table_bytes(int rows, int64_t stride, int max_blocks)
{
    return rows > 0 && max_blocks > 0 ? 4 * ((size_t)(rows - 1) * (size_t)stride + (size_t)max_blocks) : 0;
}

}  // namespace

extern "C" DSV4_API size_t dsv4_sparse_mla_decode_fp4_workspace_size(int32_t num_tokens, int32_t num_heads,
                                                                     int32_t topk_width, int32_t window)
{
    int sms = 0;
    Plan4 pl;
    return device_info(nullptr, &sms) == cudaSuccess && plan4(num_tokens, num_heads, topk_width, window, sms, &pl) ? pl.total : 0;
}

extern "C" DSV4_API dsv4_status dsv4_sparse_mla_decode_fp4(
    const void *q, int64_t q_token_stride, const void *kv_cache, int32_t num_blocks, int32_t page_block,
    const int32_t *block_table, int64_t bt_stride, int32_t max_blocks, int32_t num_reqs, const int32_t *req_idx,
    const int32_t *topk_idx, int64_t topk_stride, int32_t topk_width, const int32_t *topk_lens,
    const int32_t *seq_lens, int32_t num_tokens, int32_t num_heads, int32_t window, const float *sink,
    float softmax_scale, void *out, float *lse, void *workspace, size_t workspace_bytes, dsv4_stream_t stream)
{
    if (num_tokens < 0 || topk_width < 0 || window < 0 || window > kMaxWindow)
        return DSV4_ERR_INVALID_ARG;
    if (topk_width > kMaxTopkWidth)
        return DSV4_ERR_UNSUPPORTED;
    if (num_tokens > 0 && (seq_lens == nullptr || (topk_width > 0 && (topk_idx == nullptr || topk_stride < topk_width))))
        return DSV4_ERR_INVALID_ARG;
    if (num_heads != 16 && num_heads != 32 && num_heads != 64 && num_heads != 128)
        return DSV4_ERR_UNSUPPORTED;
    if (!std::isfinite(softmax_scale) || softmax_scale < 0.f)
        return DSV4_ERR_INVALID_ARG;
    if (num_tokens == 0)
        return DSV4_OK;
    if (q == nullptr || (kv_cache == nullptr && num_blocks > 0) || block_table == nullptr || out == nullptr ||
        workspace == nullptr)
        return DSV4_ERR_INVALID_ARG;
    if (q_token_stride < (int64_t)num_heads * kDim || q_token_stride % 8 != 0)
        return DSV4_ERR_INVALID_ARG;
    if (num_blocks < 0 || page_block <= 0 || max_blocks <= 0 || num_reqs <= 0 || bt_stride < max_blocks)
        return DSV4_ERR_INVALID_ARG;
    if (req_idx == nullptr && num_reqs < num_tokens)
        return DSV4_ERR_INVALID_ARG;
    if ((long long)max_blocks * page_block > INT_MAX || (long long)num_blocks * page_block > INT_MAX)
        return DSV4_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(workspace, 256))
        return DSV4_ERR_INVALID_ARG;
    unsigned *status = nullptr;
    int sms = 1;
    Plan4 pl;
    if (!plan4(num_tokens, num_heads, topk_width, window, sms, &pl) || workspace_bytes < pl.total)   // (on any device)
        return DSV4_ERR_INVALID_ARG;
    if (device_info(&status, &sms) != cudaSuccess)
        return DSV4_ERR_CUDA;
    if (!plan4(num_tokens, num_heads, topk_width, window, sms, &pl) || workspace_bytes < pl.total)
        return DSV4_ERR_INVALID_ARG;
    char *ws = static_cast<char *>(workspace);
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    Lists4Params l{};
    l.topk = topk_idx;
    l.topk_stride = topk_stride;
    l.topk_width = topk_width;
    l.topk_lens = topk_lens;
    l.seq_lens = seq_lens;
    l.num_tokens = num_tokens;
    l.window = window;
    l.block_table = block_table;
    l.bt_stride = bt_stride;
    l.max_blocks = max_blocks;
    l.num_reqs = num_reqs;
    l.req_idx = req_idx;
    l.num_blocks = num_blocks;
    l.page = page_block;
    l.slots = reinterpret_cast<int32_t *>(ws);
    l.lens = reinterpret_cast<int32_t *>(ws + pl.off_lens);
    l.list_w = pl.list_w;
    l.joins = reinterpret_cast<int2 *>(ws + pl.off_joins);
    l.groups = pl.groups;
    l.sink = sink;
    l.num_heads = num_heads;
    l.out = static_cast<uint16_t *>(out);
    l.lse = lse;
    l.status = status;
    l.smem_bytes = lists_fp4_smem_bytes(topk_width);
    // The decode's CTAs make the lists themselves where each has one token and its row takes them one round of loads (a launch
    // less: 10.7 against 12.4 us for 2 tokens x 16 heads in a loop of calls); wider rows go faster by the list kernel's 512
    // threads (16 tokens x 64 heads, 2048 + 256 keys: 25.0 against 26.7).
    const bool own_lists = pl.ctas_per_unit > 0 && topk_width <= decode_fp4_own_list_width();
    if (!own_lists && launch_lists_fp4(l, cs) != cudaSuccess)
        return DSV4_ERR_CUDA;
    Decode4Params p{};
    p.groups = pl.groups;
    p.grid = pl.grid;
    p.ctas_per_unit = pl.ctas_per_unit;
    p.split = pl.split;
    p.parts = reinterpret_cast<float *>(ws + pl.off_parts);
    p.joins = l.joins;
    p.q = static_cast<const uint16_t *>(q);
    p.q_token_stride = q_token_stride;
    p.kv = static_cast<const uint8_t *>(kv_cache);
    p.slots = l.slots;
    p.lens = l.lens;
    p.list_w = pl.list_w;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.sink = sink;
    p.scale = softmax_scale;
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.own_lists = own_lists;
    p.lists = l;
    p.status = status;
    return launch_decode_fp4(p, cs) == cudaSuccess ? DSV4_OK : DSV4_ERR_CUDA;
}

extern "C" DSV4_API dsv4_status dsv4_qk_norm_rope_kv_insert_fp4(
    const void *q, int64_t q_token_stride, void *q_out, int64_t q_out_token_stride, int32_t num_tokens,
    int32_t num_heads, const float *q_norm_weight, const float *kv_norm_weight, int32_t kv_norm_dims, double eps,
    const void *kv, int64_t kv_token_stride, const int64_t *positions, const int64_t *slot_mapping,
    const float *cos_sin_cache, int32_t max_position, void *kv_cache, int64_t num_slots, void *k_out,
    int64_t k_out_token_stride, dsv4_stream_t stream)
{
    if (num_tokens < 0 || num_heads < 1 || num_heads > 128 || !(eps >= 0.0) || !std::isfinite(eps) ||
        max_position < 1 || num_slots < 0 || (kv_norm_dims != 0 && kv_norm_dims != kLatent && kv_norm_dims != kDim))
        return DSV4_ERR_INVALID_ARG;
    if (num_tokens == 0)
        return DSV4_OK;
    const int64_t row = (int64_t)num_heads * kDim;
    if (q == nullptr || q_out == nullptr || kv == nullptr || positions == nullptr || slot_mapping == nullptr ||
        cos_sin_cache == nullptr || (num_slots > 0 && kv_cache == nullptr) || q_token_stride < row ||
        q_out_token_stride < row || kv_token_stride < kDim || (k_out != nullptr && k_out_token_stride < kDim))
        return DSV4_ERR_INVALID_ARG;
    if (((q_token_stride | q_out_token_stride | kv_token_stride) & 1) != 0 || !aligned(q, 4) || !aligned(q_out, 4) ||
        !aligned(kv, 4) || (k_out != nullptr && (!aligned(k_out, 4) || (k_out_token_stride & 1) != 0)) ||
        (num_slots > 0 && !aligned(kv_cache, 16)))
        return DSV4_ERR_INVALID_ARG;
    // queries in place keep their rows' places; a key's blocks are read again after the first of k_out are written, and other
    // rows that share bytes would be read before or after they are written
    if (q_out == q ? num_tokens > 1 && q_out_token_stride != q_token_stride
                   : rows_overlap(q, 2 * q_token_stride, 2 * row, q_out, 2 * q_out_token_stride, 2 * row, num_tokens))
        return DSV4_ERR_INVALID_ARG;
    const int64_t key = 2 * kDim;
    if (rows_overlap(kv, 2 * kv_token_stride, key, q_out, 2 * q_out_token_stride, 2 * row, num_tokens) ||
        (k_out != nullptr && (rows_overlap(kv, 2 * kv_token_stride, key, k_out, 2 * k_out_token_stride, key, num_tokens) ||
                              rows_overlap(q, 2 * q_token_stride, 2 * row, k_out, 2 * k_out_token_stride, key, num_tokens) ||
                              rows_overlap(q_out, 2 * q_out_token_stride, 2 * row, k_out, 2 * k_out_token_stride, key, num_tokens))))
        return DSV4_ERR_INVALID_ARG;
    Insert4Params p{};
    if (device_info(&p.status, nullptr) != cudaSuccess)
        return DSV4_ERR_CUDA;
    p.q = static_cast<const uint32_t *>(q);
    p.q_stride = q_token_stride / 2;
    p.q_out = static_cast<uint32_t *>(q_out);
    p.q_out_stride = q_out_token_stride / 2;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.q_w = q_norm_weight;
    p.kv_w = kv_norm_dims > 0 ? kv_norm_weight : nullptr;
    p.kv_norm_dims = kv_norm_dims;
    p.eps = eps;
    p.kv = static_cast<const uint32_t *>(kv);
    p.kv_stride = kv_token_stride / 2;
    p.positions = positions;
    p.slots = slot_mapping;
    p.cos_sin = cos_sin_cache;
    p.max_pos = max_position;
    p.cache = static_cast<uint8_t *>(kv_cache);
    p.num_slots = num_slots;
    p.k_out = static_cast<uint32_t *>(k_out);
    p.k_out_stride = k_out_token_stride / 2;
    return launch_qk_norm_rope_kv_insert_fp4(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? DSV4_OK
                                                                                                       : DSV4_ERR_CUDA;
}

extern "C" DSV4_API size_t dsv4_cache_pages_workspace_size(int32_t num_rows, int32_t num_rows_out, int32_t num_blocks)
{
    PagesPlan pl;
    return pages_plan(num_rows, num_rows_out, num_blocks, &pl) ? pl.total : 0;
}

extern "C" DSV4_API dsv4_status dsv4_cache_fork_rows(
    void *cache, int32_t num_layers, int64_t layer_stride, int32_t num_blocks, int32_t page_block, int32_t entry_bytes,
    const int32_t *block_table, int64_t bt_stride, const int32_t *seq_lens, int32_t num_rows, const int32_t *parent,
    int32_t num_rows_out, int32_t max_blocks, int32_t *block_table_out, int64_t bt_out_stride, int32_t *seq_lens_out,
    const int32_t *ref_counts, int32_t *ref_counts_out, int32_t share, void *workspace, size_t workspace_bytes,
    dsv4_stream_t stream)
{
    if (!pool_ok(cache, num_layers, layer_stride, num_blocks, page_block, entry_bytes) || num_rows < 0 ||
        num_rows_out < 0 || max_blocks < 0 || max_blocks > kMaxRowPages || (long long)max_blocks * page_block > INT_MAX)
        return DSV4_ERR_INVALID_ARG;
    if (num_rows == 0 && num_rows_out == 0 && ref_counts == ref_counts_out)
        return DSV4_OK;
    if ((num_rows > 0 && (seq_lens == nullptr || (max_blocks > 0 && (block_table == nullptr || bt_stride < max_blocks)))) ||
        (num_rows_out > 0 && (parent == nullptr || seq_lens_out == nullptr ||
                              (max_blocks > 0 && (block_table_out == nullptr || bt_out_stride < max_blocks)))) ||
        (num_blocks > 0 && (ref_counts == nullptr || ref_counts_out == nullptr)) || workspace == nullptr ||
        !aligned(workspace, 256))
        return DSV4_ERR_INVALID_ARG;
    // the old rows are read while the new ones are written; the counts may be updated in place
    if (overlap(block_table, table_bytes(num_rows, bt_stride, max_blocks), block_table_out,
                table_bytes(num_rows_out, bt_out_stride, max_blocks)) ||
        overlap(seq_lens, 4 * (size_t)num_rows, seq_lens_out, 4 * (size_t)num_rows_out) ||
        (ref_counts != ref_counts_out && overlap(ref_counts, 4 * (size_t)num_blocks, ref_counts_out, 4 * (size_t)num_blocks)))
        return DSV4_ERR_INVALID_ARG;
    PagesPlan pl;
    if (!pages_plan(num_rows, num_rows_out, num_blocks, &pl) || workspace_bytes < pl.total)
        return DSV4_ERR_INVALID_ARG;
    ForkParams p{};
    int sms = 0;
    if (device_info(&p.status, &sms) != cudaSuccess)
        return DSV4_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    p.pool = PagePool{static_cast<uint8_t *>(cache), num_layers, layer_stride, num_blocks, page_block, entry_bytes};
    p.table = block_table;
    p.table_stride = bt_stride;
    p.lens = seq_lens;
    p.rows = num_rows;
    p.parent = parent;
    p.rows_out = num_rows_out;
    p.max_blocks = max_blocks;
    p.table_out = block_table_out;
    p.table_out_stride = bt_out_stride;
    p.lens_out = seq_lens_out;
    p.refs = ref_counts;
    p.refs_out = ref_counts_out;
    p.share = share != 0;
    p.first = reinterpret_cast<int32_t *>(ws + pl.first);
    p.kids = reinterpret_cast<int32_t *>(ws + pl.kids);
    p.need = reinterpret_cast<int32_t *>(ws + pl.need);
    p.offset = reinterpret_cast<int32_t *>(ws + pl.offset);
    p.free_list = reinterpret_cast<int32_t *>(ws + pl.free_list);
    p.copies = reinterpret_cast<int4 *>(ws + pl.copies);
    p.num_copies = reinterpret_cast<int32_t *>(ws + pl.num_copies);
    return launch_fork(p, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? DSV4_OK : DSV4_ERR_CUDA;
}

extern "C" DSV4_API dsv4_status dsv4_cache_compact(
    void *cache, int32_t num_layers, int64_t layer_stride, int32_t num_blocks, int32_t page_block, int32_t entry_bytes,
    const int32_t *block_table, int64_t bt_stride, const int32_t *seq_lens, int32_t num_rows, int32_t max_blocks,
    int32_t *block_table_out, int64_t bt_out_stride, const int32_t *ref_counts, int32_t *ref_counts_out,
    int32_t *page_map, int32_t *num_live, void *workspace, size_t workspace_bytes, dsv4_stream_t stream)
{
    if (!pool_ok(cache, num_layers, layer_stride, num_blocks, page_block, entry_bytes) || num_rows < 0 ||
        max_blocks < 0 || max_blocks > kMaxRowPages || (long long)max_blocks * page_block > INT_MAX)
        return DSV4_ERR_INVALID_ARG;
    if ((num_rows > 0 && (seq_lens == nullptr ||
                          (max_blocks > 0 && (block_table == nullptr || bt_stride < max_blocks ||
                                              block_table_out == nullptr || bt_out_stride < max_blocks)))) ||
        (num_blocks > 0 && (ref_counts == nullptr || ref_counts_out == nullptr || page_map == nullptr)) ||
        num_live == nullptr || workspace == nullptr || !aligned(workspace, 256))
        return DSV4_ERR_INVALID_ARG;
    // the table and the counts may be updated in place
    const bool same_table = block_table == block_table_out && bt_stride == bt_out_stride;
    if ((!same_table && overlap(block_table, table_bytes(num_rows, bt_stride, max_blocks), block_table_out,
                                table_bytes(num_rows, bt_out_stride, max_blocks))) ||
        (ref_counts != ref_counts_out && overlap(ref_counts, 4 * (size_t)num_blocks, ref_counts_out, 4 * (size_t)num_blocks)) ||
        overlap(page_map, 4 * (size_t)num_blocks, ref_counts, 4 * (size_t)num_blocks) ||
        overlap(page_map, 4 * (size_t)num_blocks, ref_counts_out, 4 * (size_t)num_blocks))
        return DSV4_ERR_INVALID_ARG;
    PagesPlan pl;
    if (!pages_plan(0, 0, num_blocks, &pl) || workspace_bytes < pl.total)
        return DSV4_ERR_INVALID_ARG;
    CompactParams p{};
    int sms = 0;
    if (device_info(&p.status, &sms) != cudaSuccess)
        return DSV4_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    p.pool = PagePool{static_cast<uint8_t *>(cache), num_layers, layer_stride, num_blocks, page_block, entry_bytes};
    p.table = block_table;
    p.table_stride = bt_stride;
    p.lens = seq_lens;
    p.rows = num_rows;
    p.max_blocks = max_blocks;
    p.table_out = block_table_out;
    p.table_out_stride = bt_out_stride;
    p.refs = ref_counts;
    p.refs_out = ref_counts_out;
    p.page_map = page_map;
    p.num_live = num_live;
    p.copies = reinterpret_cast<int4 *>(ws + pl.copies);
    p.num_copies = reinterpret_cast<int32_t *>(ws + pl.num_copies);
    return launch_compact(p, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? DSV4_OK : DSV4_ERR_CUDA;
}

extern "C" DSV4_API dsv4_status dsv4_cache_copy_pages(
    void *dst_cache, int64_t dst_layer_stride, int32_t dst_num_blocks, const void *src_cache, int64_t src_layer_stride,
    int32_t src_num_blocks, int32_t num_layers, int32_t page_block, int32_t entry_bytes, const int32_t *src_pages,
    const int32_t *dst_pages, int32_t num_pages, void *workspace, size_t workspace_bytes, dsv4_stream_t stream)
{
    if (!pool_ok(dst_cache, num_layers, dst_layer_stride, dst_num_blocks, page_block, entry_bytes) ||
        !pool_ok(src_cache, num_layers, src_layer_stride, src_num_blocks, page_block, entry_bytes) || num_pages < 0)
        return DSV4_ERR_INVALID_ARG;
    if (num_pages == 0)
        return DSV4_OK;
    if (src_pages == nullptr || dst_pages == nullptr || workspace == nullptr || !aligned(workspace, 256))
        return DSV4_ERR_INVALID_ARG;
    const bool one_pool = dst_cache == src_cache && dst_num_blocks == src_num_blocks &&
                          (num_layers == 1 || dst_layer_stride == src_layer_stride);
    if (!one_pool && overlap(dst_cache, pool_bytes(num_layers, dst_layer_stride, dst_num_blocks, page_block, entry_bytes),
                             src_cache, pool_bytes(num_layers, src_layer_stride, src_num_blocks, page_block, entry_bytes)))
        return DSV4_ERR_INVALID_ARG;
    PagesPlan pl;
    if (!pages_plan(0, 0, dst_num_blocks, &pl) || workspace_bytes < pl.total)
        return DSV4_ERR_INVALID_ARG;
    CopyPagesParams p{};
    int sms = 0;
    if (device_info(&p.status, &sms) != cudaSuccess)
        return DSV4_ERR_CUDA;
    p.dst = PagePool{static_cast<uint8_t *>(dst_cache), num_layers, dst_layer_stride, dst_num_blocks, page_block, entry_bytes};
    p.src = PagePool{static_cast<uint8_t *>(const_cast<void *>(src_cache)), num_layers, src_layer_stride, src_num_blocks,
                     page_block, entry_bytes};
    p.one_pool = one_pool;
    p.src_pages = src_pages;
    p.dst_pages = dst_pages;
    p.num_pages = num_pages;
    p.claim = reinterpret_cast<int32_t *>(static_cast<char *>(workspace) + pl.free_list);
    return launch_copy_pages(p, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? DSV4_OK : DSV4_ERR_CUDA;
}
