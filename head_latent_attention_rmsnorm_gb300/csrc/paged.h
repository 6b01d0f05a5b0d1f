// paged.h -- host interface of the paged-cache kernels (paged*.cu).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tc.h"

namespace mla {

constexpr int PAGED_MAX_BATCH = 16384;   // requests of one mla_paged_tables call (its prefix sums stay in shared memory)

cudaError_t launch_paged_tables(int B, int page, int max_pages, int n_free, int n_tokens, const int *past,
                                const int *fresh, const int *free_pages, int *table, int *kv_lens, int *cu, int *slots,
                                int *positions, int *counts, cudaStream_t st);

// gone [B], pick [B][segments]: scratch.
int paged_evict_segments(int max_pages);
cudaError_t launch_paged_evict(int B, int page, int max_pages, int room, int keep, int first, int last, const int *lens,
                               const int *table, const float *weights, int *table_out, float *weights_out, int *freed,
                               int *counts, int *gone, uint4 *pick, cudaStream_t st);

// c rows at c + t * c_stride elements, k rows at k + t * k_stride.
cudaError_t launch_paged_append(int ty, int T, long n_slots, int Dk, int Dr, float base, float eps, const void *c,
                                long c_stride, const void *k, long k_stride, const void *w, const int *slots,
                                const int *positions, void *c_cache, void *kpe_cache, cudaStream_t st);

// One absorbed-form call: decode (one query per request), or the tokens of a step.  A query row is a head of a
// token, rows T H.  Rows of one request that lie together form a group: a decode's request with its H
// rows, or a few tokens of one request, as many as fit `row_tile` rows (of more heads one).  A work item is
// (group b, row tile of `row_tile` rows); its keys are cut
// into tiles of `tile` keys, all items' T tiles are numbered through, and worker c of W takes tiles
// [c q, (c + 1) q) with q = max(min_tiles, ceil(T / W)).  The part of item i that worker c computes goes
// to partial slot c + i: unique, because going along the tiles every cut raises c or i.
struct alignas(16) PagedPart {   // what a worker computes of one item
    int row, q, k0, nt;          // row of the block table, first query row, first key tile, key tiles
    int keys, next;              // the group's length; distance to the worker's next part, 0 for none
    int rows, pad;               // query rows of the item
};
struct PagedDecode {
    int B, H, Dk, Dn, Dr, Dv;        // groups (decode: requests), ..
    int T;                           // tokens (decode: B)
    int num_pages, page, max_pages;
    int ty;
    bool tc;                         // the tensor-core form
    float scale, base;
    const void *q_nope, *q_pe, *c_cache, *kpe_cache, *w;
    const int *table, *lens;         // lens [B]: the groups' keys
    // The tokens of a step (null for decode): each one's position, group (-1: not computed here, its output
    // stays) and first row in the group, and the keys that it sees; each group's row of the table, first query
    // row and number of rows.
    const int *pos;
    const int2 *of;
    const int *limits;
    const int4 *groups;
    // list: the step's tokens that are computed here, T of them from there on at most, *n_list - list_at in fact; then a
    // token in all of the above is its place in the list, but for pos, q_nope, q_pe, out and lse, which are the step's
    // (null: the tokens themselves, T of them).
    const int *list, *n_list;
    int list_at;
    bool scores_only;                // the absorb leaves the third parts of the queries out
    void *out;
    float *lse;
    int row_tile, row_tiles, tile;   // rows per item, items per group, keys per tile
    int workers, min_tiles;          // most workers, fewest tiles that make one worker more
    long *tile_off;                  // [B + 1] first tile of group b, for one row tile
    PagedPart *parts;                // [slots], the tensor-core form's
    int *first;                      // [2][workers]: a worker's first part, its number of tiles
    int2 *spans;                     // [B row_tiles]: an item's first part, its number of parts
    void *qabs, *qpe;                // absorbed and rotated queries
    // partials [slots][row_tile][Dk] and their log-sum-exps [slots][row_tile], slots = workers + B row_tiles:
    // fp32, or fp16 times a scale per half row [slots][row_tile][2] in the tensor-core form
    float *po32, *pl, *pscale;
    __half *po;
};
// A step: request b's tokens are rows cu[b] .. cu[b + 1] - 1 of n_tokens, each at its position; the request
// holds lens[b] tokens, its new ones among them.
struct PagedStep {
    int B, n_tokens;
    const int *cu, *positions, *lens;
};
// Tokens of one round of the absorbed form: a step of more takes several (queries and partials are 570 KB a token at 128
// heads; a round costs four launches, of which a step whose tokens all go explicit has nothing).
constexpr int PAGED_ROUND = 4096;
// The plan of tokens s0 .. s0 + p.T - 1: their groups of `most` at most, and the division of the groups' tiles (what is
// written are p's lens, of, limits and groups; p.B = p.T); n_zero words at `zero` are set to zero.
struct PagedPlan {
    PagedStep s;
    int s0, most;
    int *lens, *limits;
    int2 *of;
    int4 *groups;
    unsigned long long *zero;
    long n_zero;
};
cudaError_t launch_paged_plan(const PagedDecode &p, const PagedPlan &s, cudaStream_t st);
// Few tokens, not of a list: the absorb's first block divides them, as decode's does, which saves a launch.
inline bool plan_in_absorb(const PagedDecode &p, const PagedPlan &s) {
    return p.T <= 128 && !p.list && s.s.B <= 1024 && s.n_zero <= 4096;
}

// The launches of a call: absorb, attention, join.  `plan` of a step's tokens: theirs, for the absorb to make (null: made
// by launch_paged_plan in front, or decode's).
cudaError_t paged_decode_simt(const PagedDecode &p, const PagedPlan *plan, cudaStream_t st);
cudaError_t paged_absorb_simt(const PagedDecode &p, const PagedPlan *plan, cudaStream_t st);

// The explicit form of the requests with many tokens (tensor cores), CHUNK_MIN and more, in calls of CHUNK_CALL tokens and
// more (its launches, with nothing to do, are 10 to 16 us).  Tiles of 128 tokens: at most n_tokens / 128 and one more a
// request.  Tiles of 128 keys that have the rest of K_nope: CHUNK_RESTS a request, and one for CHUNK_REST_TOKENS tokens.
constexpr int CHUNK_CALL = 64, CHUNK_MIN = 32, CHUNK_RESTS = 4, CHUNK_REST_TOKENS = 16, CHUNK_SORT = 2048;
struct PagedChunk {
    int key_rows;                // rows of the key buffers, a multiple of 256
    int max_tiles, max_rests;    // tiles of 128 tokens; tiles of 128 keys with a rest
    int *rest_of;                // [key_rows / 128]
    void *rest;
    int heads;                   // of a shard
    int *ctl;                    // [4]: rows in use, tiles, tokens of the list, whether the tiles are in falling order
    int *key0, *holes;           // [B]: a request's first key row (-1: absorbed); nonzero: some page is missing
    unsigned *w_max, *c_max;     // [H], [B]: as TcStep's
    int *block_of;               // [key_rows / 128]: the request of each 128 rows
    int *limits, *done, *list;   // [n_tokens]: keys seen; nonzero: explicit; the requests' other tokens
    StepTile *raw, *tiles;
    uint32_t *held;              // a bit per key row
    void *chat, *kpe, *qpe, *kws, *vws;
};
inline int chunk_rests(int n_tokens, int key_rows) {
    const int a = key_rows / 128, b = n_tokens / CHUNK_REST_TOKENS;
    return b < a ? b : a;
}
inline int chunk_tiles(int n_tokens) { return n_tokens / 128 + n_tokens / CHUNK_MIN + 1; }
// Whether n tokens of a request of `keys` keys, `tiled` rounded up to whole tiles, go explicit: the cheaper form (its reasons
// and measurements are at paged_chunk_kernel).  rows: query rows of an item of the absorbed form.
__host__ __device__ inline bool chunk_pays(long n, long keys, long tiled, long rows) {
    return n >= CHUNK_MIN && keys >= CHUNK_MIN && 6 * n * (keys + 12 * rows) >= 11 * rows * (tiled + 64);
}
inline int chunk_item_rows(const PagedDecode &p) { return p.row_tiles > 1 ? p.H / p.row_tiles : p.row_tile / p.H * p.H; }
// A bound of the key rows that the requests of a step can take together; cap: keys of a row of the table.
long chunk_most_rows(int B, int n_tokens, long cap, int rows);
// The plan and the gathered rows; p.q_pe of the whole step.
cudaError_t launch_paged_chunk(const PagedDecode &p, const PagedStep &s, const PagedChunk &c, cudaStream_t st);

// The weights that the tokens of p gave the pages of their requests, added to acc [requests][max_pages] as integers of
// 2^-bits, behind the plan and the absorb (scores_only): tensor cores with items of 128 rows and tiles of 256 keys, CUDA
// cores with 16 and 32.  lse [T H].
constexpr int PAGED_W_ROWS = 128, PAGED_W_TILE = 256;
cudaError_t launch_paged_weights(const PagedDecode &p, const float *lse, unsigned long long *acc, int bits, cudaStream_t st);
// out [n] = acc 2^-bits + prior (null: 0)
cudaError_t launch_paged_weights_out(long n, const unsigned long long *acc, int bits, const float *prior, float *out, cudaStream_t st);
cudaError_t paged_weights_read_and_clear_error(unsigned *flags, cudaStream_t st);

// The tensor-core form (bf16): these dimensions and page size, any number of heads.
// pairs of SMs of a GB300, keys per tile (no worker waits for another: with fewer SMs free they take turns)
constexpr int PAGED_TC_WORKERS = 76, PAGED_TC_TILE = 64;
bool paged_tc_supported(int Dk, int Dn, int Dr, int Dv, int page);
cudaError_t paged_decode_tc(const PagedDecode &p, const PagedPlan *plan, cudaStream_t st);
cudaError_t paged_absorb_tc(const PagedDecode &p, const PagedPlan *plan, cudaStream_t st);
cudaError_t paged_tc_read_and_clear_error(unsigned *flags, cudaStream_t st);
cudaError_t paged_many_read_and_clear_error(unsigned *flags, cudaStream_t st);

}  // namespace mla
