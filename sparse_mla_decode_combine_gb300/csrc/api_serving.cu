// api_serving.cu -- the C ABI of the operators between two decode steps (include/dsv4.h): argument validation, the carving
// of the caller's workspace, and the launches on the caller's stream.
#include <algorithm>
#include <climits>
#include <cmath>

#include "../../include/dsv4.h"
#include "overlap.h"
#include "serving.h"

using namespace dsv4;

namespace {

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int kMaxWindow = 1 << 24;
constexpr int kMaxVocab = 1 << 22;
constexpr int kMaxPages = 1 << 30, kMaxRowPages = 1 << 20;

// `rows` rows of `width` values of `unit` bytes
Rows rows_of(const void *at, int rows, int64_t stride, int64_t width, int64_t unit = 4)
{
    return Rows{at, rows, stride * unit, width * unit};
}

// ---- the key weights' workspace: the tokens' slots, positions and lengths, and what each key received
struct WeightsPlan {
    int list_w;
    size_t off_positions, off_got, off_lens, off_later, total;
};

bool weights_plan(int num_tokens, int num_heads, int topk_width, int window, WeightsPlan *pl)
{
    if (num_tokens < 0 || topk_width < 0 || topk_width > kMaxTopkWidth || window < 0 || window > kMaxWindow)
        return false;
    if (num_heads != 16 && num_heads != 32 && num_heads != 64 && num_heads != 128)
        return false;
    pl->list_w = topk_width + window;
    const int tile = key_weights_block_keys();
    if ((long long)num_tokens * ((pl->list_w + tile - 1) / tile + 4) > INT_MAX)   // (and a few blocks' worth for a token's start)
        return false;
    const size_t lists = align_up(4 * (size_t)num_tokens * (size_t)pl->list_w, 256);
    pl->off_positions = lists;
    pl->off_got = 2 * lists;
    pl->off_lens = 3 * lists;
    pl->off_later = align_up(pl->off_lens + 4 * (size_t)num_tokens, 256);
    pl->total = std::max<size_t>(256, align_up(pl->off_later + 4 * (size_t)num_tokens, 256));
    return true;
}

// ---- the eviction's workspace
struct EvictPlan {
    EvictShape shape;
    size_t picked, between, moved, need, offset, free_list, read, ticket, total;
};

bool evict_plan(int rows, int max_blocks, int num_blocks, int num_layers, int page, int entry_bytes, int budget, int weights_width,
                EvictPlan *pl)
{
    if (rows < 0 || max_blocks < 0 || max_blocks > kMaxRowPages || num_blocks < 0 || num_blocks > kMaxPages || num_layers < 1 ||
        page < 1 || entry_bytes < 16 || entry_bytes % 16 != 0 || budget < 1 || (long long)max_blocks * page > INT_MAX ||
        (long long)page * entry_bytes > INT_MAX)
        return false;
    budget = (int)std::max(1ll, std::min((long long)budget, (long long)max_blocks * page));   // (no row is longer)
    const long long columns = (long long)num_layers * ((entry_bytes + 16383) / 16384);
    if (columns > INT_MAX / 4 || (long long)rows * columns > INT_MAX / 4)
        return false;
    pl->shape = evict_shape(num_layers, entry_bytes, budget, weights_width);
    if ((double)rows * ((double)pl->shape.columns * pl->shape.tiles + pl->shape.weight_tiles + pl->shape.zero_tiles) > INT_MAX / 2)
        return false;   // (tickets)
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes, 256);
        return at;
    };
    pl->picked = take(4 * (size_t)rows * (size_t)budget);
    pl->between = take(4 * (size_t)rows);
    pl->moved = take(4 * (size_t)rows);
    pl->need = take(4 * (size_t)rows);
    pl->offset = take(4 * (size_t)rows);
    pl->free_list = take(4 * (size_t)num_blocks);
    pl->read = take(4 * (size_t)rows * ((size_t)pl->shape.columns * (size_t)pl->shape.words + (size_t)pl->shape.weight_words));
    pl->ticket = take(4);
    pl->total = off;
    return true;
}

}  // namespace

extern "C" DSV4_API dsv4_status dsv4_verify_drafts(
    const void *target_probs, int64_t target_stride, const void *draft_probs, int64_t draft_stride, int32_t probs_bf16,
    int32_t vocab, const int32_t *draft_tokens, int32_t num_drafts, const int32_t *query_start_loc, int32_t num_reqs,
    int32_t num_rows, const float *uniform, const uint8_t *greedy, int32_t *tokens, int64_t tokens_stride,
    int32_t tokens_width, int32_t *num_accepted, const int32_t *seq_lens, int32_t *seq_lens_out, dsv4_stream_t stream)
{
    if (num_reqs < 0 || num_rows < 0 || num_drafts < 0 || vocab < 1 || vocab > kMaxVocab || num_reqs > (1 << 24))
        return DSV4_ERR_INVALID_ARG;
    if (num_reqs == 0)
        return DSV4_OK;
    if (query_start_loc == nullptr || num_accepted == nullptr || tokens == nullptr || tokens_width < 1 ||
        tokens_stride < tokens_width || (num_rows > 0 && (target_probs == nullptr || target_stride < vocab || uniform == nullptr)) ||
        (num_drafts > 0 && (draft_tokens == nullptr || (draft_probs != nullptr && draft_stride < vocab))) ||
        (seq_lens == nullptr) != (seq_lens_out == nullptr))
        return DSV4_ERR_INVALID_ARG;
    const int64_t unit = probs_bf16 ? 2 : 4;
    if (!aligned(target_probs, unit) || !aligned(draft_probs, unit))
        return DSV4_ERR_INVALID_ARG;
    // the CTAs of a request, and other requests, read their inputs at different times; lengths may be updated in place
    const Rows target = rows_of(target_probs, num_rows, target_stride, vocab, unit),
               draft = rows_of(draft_probs, num_drafts, draft_stride, vocab, unit), drafted = bytes(draft_tokens, 4ll * num_drafts),
               starts = bytes(query_start_loc, 4 * (num_reqs + 1ll)), numbers = bytes(uniform, 4ll * num_rows),
               modes = bytes(greedy, num_reqs), lens = bytes(seq_lens, 4ll * num_reqs),
               out = rows_of(tokens, num_reqs, tokens_stride, tokens_width), accepted = bytes(num_accepted, 4ll * num_reqs),
               new_lens = bytes(seq_lens_out, 4ll * num_reqs);
    if (share(out, {target, draft, drafted, starts, numbers, modes, lens, accepted, new_lens}) ||
        share(accepted, {target, draft, drafted, starts, numbers, modes, lens, new_lens}) ||
        share(new_lens, {target, draft, drafted, starts, numbers, modes}) || (seq_lens_out != seq_lens && share(new_lens, lens)))
        return DSV4_ERR_INVALID_ARG;
    VerifyParams p{};
    int sms = 0;
    if (device_info(&p.status, &sms) != cudaSuccess)
        return DSV4_ERR_CUDA;
    p.target = target_probs;
    p.target_stride = target_stride;
    p.draft = num_drafts > 0 ? draft_probs : nullptr;
    p.draft_stride = draft_stride;
    p.vocab = vocab;
    p.tokens = draft_tokens;
    p.num_drafts = num_drafts;
    p.start = query_start_loc;
    p.num_reqs = num_reqs;
    p.num_rows = num_rows;
    p.uniform = uniform;
    p.greedy = greedy;
    p.out = tokens;
    p.out_stride = tokens_stride;
    p.out_width = tokens_width;
    p.accepted = num_accepted;
    p.seq = seq_lens;
    p.seq_out = seq_lens_out;
    p.cluster = verify_cluster_size(num_reqs, vocab, sms);
    p.tile = verify_tile(vocab, p.cluster);
    return launch_verify(p, probs_bf16 != 0, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? DSV4_OK : DSV4_ERR_CUDA;
}

extern "C" DSV4_API size_t dsv4_sparse_mla_key_weights_workspace_size(int32_t num_tokens, int32_t num_heads,
                                                                      int32_t topk_width, int32_t window)
{
    WeightsPlan pl;
    return weights_plan(num_tokens, num_heads, topk_width, window, &pl) ? pl.total : 0;
}

extern "C" DSV4_API dsv4_status dsv4_sparse_mla_key_weights(
    const void *q, int64_t q_token_stride, const void *kv_cache, int32_t num_blocks, int32_t page_block,
    int32_t entry_bytes, const int32_t *block_table, int64_t bt_stride, int32_t max_blocks, int32_t num_reqs,
    const int32_t *req_idx, const int32_t *topk_idx, int64_t topk_stride, int32_t topk_width, const int32_t *topk_lens,
    const int32_t *seq_lens, int32_t num_tokens, int32_t num_heads, int32_t window, const float *lse,
    float softmax_scale, float *weights, int64_t weights_stride, int32_t weights_width, void *workspace,
    size_t workspace_bytes, dsv4_stream_t stream)
{
    if (num_tokens < 0 || topk_width < 0 || window < 0 || window > kMaxWindow)
        return DSV4_ERR_INVALID_ARG;
    if (topk_width > kMaxTopkWidth)
        return DSV4_ERR_UNSUPPORTED;
    if (num_heads != 16 && num_heads != 32 && num_heads != 64 && num_heads != 128)
        return DSV4_ERR_UNSUPPORTED;
    if (entry_bytes != kEntryBytes && entry_bytes != kEntry4Bytes)
        return DSV4_ERR_UNSUPPORTED;
    if (!std::isfinite(softmax_scale) || softmax_scale < 0.f)
        return DSV4_ERR_INVALID_ARG;
    if (num_tokens == 0)
        return DSV4_OK;
    if (q == nullptr || (kv_cache == nullptr && num_blocks > 0) || block_table == nullptr || seq_lens == nullptr ||
        (topk_width > 0 && (topk_idx == nullptr || topk_stride < topk_width)) || lse == nullptr || weights == nullptr ||
        workspace == nullptr)
        return DSV4_ERR_INVALID_ARG;
    if (q_token_stride < (int64_t)num_heads * kDim || q_token_stride % 8 != 0)
        return DSV4_ERR_INVALID_ARG;
    if (num_blocks < 0 || page_block <= 0 || max_blocks <= 0 || num_reqs <= 0 || bt_stride < max_blocks ||
        (req_idx == nullptr && num_reqs < num_tokens))
        return DSV4_ERR_INVALID_ARG;
    if ((long long)max_blocks * page_block > INT_MAX || (long long)num_blocks * page_block > INT_MAX ||
        weights_width < (long long)max_blocks * page_block || weights_stride < weights_width)
        return DSV4_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(workspace, 256) || !aligned(weights, 4) || !aligned(lse, 4))
        return DSV4_ERR_INVALID_ARG;
    WeightsPlan pl;
    if (!weights_plan(num_tokens, num_heads, topk_width, window, &pl) || workspace_bytes < pl.total)
        return DSV4_ERR_INVALID_ARG;
    // the table is written, and the workspace, while lists, rows and queries are read again
    const Rows table = rows_of(weights, num_reqs, weights_stride, weights_width), ws_bytes = bytes(workspace, (int64_t)pl.total);
    for (const Rows &in : {rows_of(q, num_tokens, q_token_stride, (int64_t)num_heads * kDim, 2),
                           bytes(kv_cache, (int64_t)num_blocks * page_block * entry_bytes),
                           rows_of(block_table, num_reqs, bt_stride, max_blocks), bytes(req_idx, 4ll * num_tokens),
                           rows_of(topk_idx, num_tokens, topk_stride, topk_width), bytes(topk_lens, 4ll * num_tokens),
                           bytes(seq_lens, 4ll * num_tokens), bytes(lse, 4ll * num_tokens * num_heads)})
        if (share(table, in) || share(ws_bytes, in))
            return DSV4_ERR_INVALID_ARG;
    if (share(table, ws_bytes))
        return DSV4_ERR_INVALID_ARG;
    if (pl.list_w == 0)
        return DSV4_OK;
    unsigned *status = nullptr;
    int sms = 1;
    if (device_info(&status, &sms) != cudaSuccess)
        return DSV4_ERR_CUDA;
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
    l.positions = reinterpret_cast<int32_t *>(ws + pl.off_positions);
    l.lens = reinterpret_cast<int32_t *>(ws + pl.off_lens);
    l.later = reinterpret_cast<int32_t *>(ws + pl.off_later);
    l.list_w = pl.list_w;
    l.status = status;
    l.smem_bytes = lists_fp4_smem_bytes(topk_width);
    if (launch_lists_positions(l, sms, cs) != cudaSuccess)
        return DSV4_ERR_CUDA;
    KeyWeightsParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.q_token_stride = q_token_stride;
    p.kv = static_cast<const uint8_t *>(kv_cache);
    p.entry_bytes = entry_bytes;
    p.slots = l.slots;
    p.positions = l.positions;
    p.lens = l.lens;
    p.later = l.later;
    p.list_w = pl.list_w;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.req_idx = req_idx;
    p.num_reqs = num_reqs;
    p.lse = lse;
    p.scale = softmax_scale;
    p.got = reinterpret_cast<float *>(ws + pl.off_got);
    p.weights = weights;
    p.weights_stride = weights_stride;
    p.status = status;
    return launch_key_weights(p, sms, cs) == cudaSuccess ? DSV4_OK : DSV4_ERR_CUDA;
}

extern "C" DSV4_API size_t dsv4_cache_evict_workspace_size(int32_t num_rows, int32_t max_blocks, int32_t num_blocks,
                                                           int32_t num_layers, int32_t page_block, int32_t entry_bytes,
                                                           int32_t budget)
{
    EvictPlan pl;
    return evict_plan(num_rows, max_blocks, num_blocks, num_layers, page_block, entry_bytes, budget, 0, &pl) ? pl.total : 0;
}

extern "C" DSV4_API dsv4_status dsv4_cache_evict(
    void *cache, int32_t num_layers, int64_t layer_stride, int32_t num_blocks, int32_t page_block, int32_t entry_bytes,
    const int32_t *block_table, int64_t bt_stride, const int32_t *seq_lens, int32_t num_rows, int32_t max_blocks,
    const float *weights, int64_t weights_stride, int32_t weights_width, int32_t budget, int32_t limit, int32_t first,
    int32_t recent, int32_t *block_table_out, int64_t bt_out_stride, int32_t *seq_lens_out, const int32_t *ref_counts,
    int32_t *ref_counts_out, float *weights_out, int64_t weights_out_stride, void *workspace, size_t workspace_bytes,
    dsv4_stream_t stream)
{
    EvictPlan pl;
    if (budget < 1 || limit < budget || first < 0 || recent < 0 || first > budget || recent > budget - first ||
        weights_width < 0 ||
        !evict_plan(num_rows, max_blocks, num_blocks, num_layers, page_block, entry_bytes, budget, weights_width, &pl))
        return DSV4_ERR_INVALID_ARG;
    if ((num_layers > 1 && (layer_stride % 16 != 0 || layer_stride < (int64_t)num_blocks * page_block * entry_bytes)) ||
        (num_blocks > 0 && (cache == nullptr || !aligned(cache, 16) || ref_counts == nullptr || ref_counts_out == nullptr)))
        return DSV4_ERR_INVALID_ARG;
    if (num_rows == 0 && ref_counts == ref_counts_out)
        return DSV4_OK;
    if (num_rows > 0 && (seq_lens == nullptr || seq_lens_out == nullptr))
        return DSV4_ERR_INVALID_ARG;
    if (num_rows > 0 && max_blocks > 0 &&
        (block_table == nullptr || bt_stride < max_blocks || block_table_out == nullptr || bt_out_stride < max_blocks))
        return DSV4_ERR_INVALID_ARG;
    if (weights_width < (long long)max_blocks * page_block ||
        (num_rows > 0 && weights_width > 0 &&
         (weights == nullptr || weights_out == nullptr || weights_stride < weights_width || weights_out_stride < weights_width ||
          !aligned(weights, 4) || !aligned(weights_out, 4))))
        return DSV4_ERR_INVALID_ARG;
    if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < pl.total)
        return DSV4_ERR_INVALID_ARG;
    // the old rows are read while the new ones are written; counts and weights may be updated in place
    const bool same_weights = weights == weights_out && (num_rows <= 1 || weights_stride == weights_out_stride);
    const Rows table = rows_of(block_table, num_rows, bt_stride, max_blocks), lens = bytes(seq_lens, 4ll * num_rows),
               refs = bytes(ref_counts, 4ll * num_blocks), had = rows_of(weights, num_rows, weights_stride, weights_width),
               new_table = rows_of(block_table_out, num_rows, bt_out_stride, max_blocks),
               new_lens = bytes(seq_lens_out, 4ll * num_rows), new_refs = bytes(ref_counts_out, 4ll * num_blocks),
               left = rows_of(weights_out, num_rows, weights_out_stride, weights_width);
    const Rows ws_bytes = bytes(workspace, (int64_t)pl.total);
    if ((ref_counts != ref_counts_out && share(refs, new_refs)) || (!same_weights && share(had, left)) ||
        share(new_table, {table, lens, refs, had, new_lens, new_refs, left, ws_bytes}) ||
        share(new_lens, {table, lens, refs, had, new_refs, left, ws_bytes}) || share(new_refs, {table, lens, had, left, ws_bytes}) ||
        share(left, {table, lens, refs, ws_bytes}) || share(ws_bytes, {table, lens, refs, had}))
        return DSV4_ERR_INVALID_ARG;
    EvictParams p{};
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
    p.weights = weights;
    p.weights_stride = weights_stride;
    p.weights_width = weights_width;
    p.budget = budget;
    p.limit = limit;
    p.first = first;
    p.recent = recent;
    p.table_out = block_table_out;
    p.table_out_stride = bt_out_stride;
    p.lens_out = seq_lens_out;
    p.refs = ref_counts;
    p.refs_out = ref_counts_out;
    p.weights_out = weights_out;
    p.weights_out_stride = weights_out_stride;
    p.picked = reinterpret_cast<int32_t *>(ws + pl.picked);
    p.between = reinterpret_cast<int32_t *>(ws + pl.between);
    p.moved = reinterpret_cast<int32_t *>(ws + pl.moved);
    p.need = reinterpret_cast<int32_t *>(ws + pl.need);
    p.offset = reinterpret_cast<int32_t *>(ws + pl.offset);
    p.free_list = reinterpret_cast<int32_t *>(ws + pl.free_list);
    p.read = reinterpret_cast<uint32_t *>(ws + pl.read);
    p.ticket = reinterpret_cast<int32_t *>(ws + pl.ticket);
    p.tile = pl.shape.tile;
    p.column_bytes = pl.shape.column_bytes;
    p.columns = pl.shape.columns;
    p.tiles = pl.shape.tiles;
    p.words = pl.shape.words;
    p.weight_tiles = pl.shape.weight_tiles;
    p.weight_words = pl.shape.weight_words;
    p.zero_tiles = pl.shape.zero_tiles;
    return launch_evict(p, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? DSV4_OK : DSV4_ERR_CUDA;
}
