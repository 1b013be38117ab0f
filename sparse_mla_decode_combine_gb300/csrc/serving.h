// serving.h -- launch interface of the operators between two decode steps: verification of drafted tokens, the keys'
// attention weights, and eviction.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "fp4.h"

namespace dsv4 {

struct VerifyParams {
    const void *target;        // [rows, vocab] probabilities
    int64_t target_stride;
    const void *draft;         // [num_drafts, vocab] or null
    int64_t draft_stride;
    int32_t vocab;
    const int32_t *tokens;     // [num_drafts]
    int32_t num_drafts;
    const int32_t *start;      // [num_reqs + 1]
    int32_t num_reqs;
    int32_t num_rows;
    const float *uniform;      // [num_rows]
    const uint8_t *greedy;     // [num_reqs] or null
    int32_t *out;              // [num_reqs, out_width]
    int64_t out_stride;
    int32_t out_width;
    int32_t *accepted;         // [num_reqs]
    const int32_t *seq;        // [num_reqs] or null
    int32_t *seq_out;
    int32_t cluster;           // CTAs per request
    int32_t tile;              // values of a row whose sum is held for the search
    unsigned *status;
};
int verify_cluster_size(int num_reqs, int vocab, int sms);
int verify_tile(int vocab, int cluster);
cudaError_t launch_verify(const VerifyParams &p, bool bf16, cudaStream_t stream);

struct KeyWeightsParams {
    const uint16_t *q;
    int64_t q_token_stride;
    const uint8_t *kv;
    int32_t entry_bytes;
    const int32_t *slots;      // [T, list_w] cache slots (-1: no key), the positions that they hold, how many a token has
    const int32_t *positions;
    const int32_t *lens;
    const int32_t *later;      // [T] not 0: a token with keys before this one names its row
    int32_t list_w;
    int32_t num_tokens;
    int32_t num_heads;
    const int32_t *req_idx;
    int32_t num_reqs;
    const float *lse;          // [T, H]
    float scale;
    float *got;                // [T, list_w] what each key of such a later token received
    float *weights;            // [num_reqs, weights_width]
    int64_t weights_stride;
    unsigned *status;
};
int key_weights_block_keys();
cudaError_t launch_key_weights(const KeyWeightsParams &p, int sms, cudaStream_t stream);

struct EvictParams {
    PagePool pool;
    const int32_t *table;
    int64_t table_stride;
    const int32_t *lens;
    int32_t rows;
    int32_t max_blocks;
    const float *weights;
    int64_t weights_stride;
    int32_t weights_width;
    int32_t budget, limit, first, recent;
    int32_t *table_out;
    int64_t table_out_stride;
    int32_t *lens_out;
    const int32_t *refs;
    int32_t *refs_out;
    float *weights_out;
    int64_t weights_out_stride;
    unsigned *status;
    // workspace
    int32_t *picked;           // [rows, budget - first - recent] the positions kept between the first and the recent ones, less `first`
    int32_t *between;          // [rows] entries between the first and the recent ones
    int32_t *moved;            // [rows] first entry that is written (the row's length: none)
    int32_t *need;             // [rows] pages to take
    int32_t *offset;           // [rows] exclusive sums of need
    int32_t *free_list;        // [num_blocks]
    uint32_t *read;            // [rows, columns, words] bit i: the entries that tile i writes have been read; then
                               // [rows, weight_words] the same of the weights' tiles
    int32_t words;             // words per (row, column)
    int32_t tile;              // entries per tile
    int32_t column_bytes;      // bytes of an entry that a column covers (entries larger than a tile have several)
    int32_t columns;           // layers * columns of an entry
    int32_t tiles;             // tiles per (row, column)
    int32_t weight_tiles, weight_words;   // tiles of a row's kept weights, and words for them
    int32_t zero_tiles;        // tiles of a row of weights_out that may have to be set to zero
    int32_t *ticket;           // [1]
    bool selected;             // the selection wrote `moved`
};
struct EvictShape {
    int32_t tile, column_bytes, columns, tiles, words, weight_tiles, weight_words, zero_tiles;
};
EvictShape evict_shape(int num_layers, int entry_bytes, int budget, int weights_width);
cudaError_t launch_evict(EvictParams p, int sms, cudaStream_t stream);

}  // namespace dsv4
