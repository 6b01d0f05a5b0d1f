// paged.h -- host interface of the paged-cache kernels (paged.cu, paged_simt.cu).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mla {

constexpr int PAGED_MAX_BATCH = 16384;   // requests of one mla_paged_tables call (its prefix sums stay in shared memory)

cudaError_t launch_paged_tables(int B, int page, int max_pages, int n_free, int n_tokens, const int *past,
                                const int *fresh, const int *free_pages, int *table, int *kv_lens, int *cu, int *slots,
                                int *positions, int *counts, cudaStream_t st);

// c rows at c + t * c_stride elements, k rows at k + t * k_stride.
cudaError_t launch_paged_append(int ty, int T, long n_slots, int Dk, int Dr, float base, float eps, const void *c,
                                long c_stride, const void *k, long k_stride, const void *w, const int *slots,
                                const int *positions, void *c_cache, void *kpe_cache, cudaStream_t st);

// One decode call.  A work item is (request b, row tile of `row_tile` heads); its keys are cut
// into tiles of `tile` keys, all items' T tiles are numbered through, and worker c of W takes tiles
// [c q, (c + 1) q) with q = max(min_tiles, ceil(T / W)).  The part of item i that worker c computes goes
// to partial slot c + i: unique, because going along the tiles every cut raises c or i.
struct alignas(16) PagedPart {   // what a worker computes of one item
    int b, rt, k0, nt;           // request, row tile, first key tile, key tiles
    int keys, next;              // the request's length; distance to the worker's next part, 0 for none
    int pad[2];
};
struct PagedDecode {
    int B, H, Dk, Dn, Dr, Dv;
    int num_pages, page, max_pages;
    int ty;
    bool tc;                         // the tensor-core form
    float scale, base;
    const void *q_nope, *q_pe, *c_cache, *kpe_cache, *w;
    const int *table, *lens;
    void *out;
    float *lse;
    int row_tile, row_tiles, tile;   // heads per item, items per request, keys per tile
    int workers, min_tiles;          // most workers, fewest tiles that make one worker more
    long *tile_off;                  // [B + 1] first tile of request b, for one row tile
    PagedPart *parts;                // [slots], the tensor-core form's
    int *first;                      // [2][workers]: a worker's first part, its number of tiles
    int2 *spans;                     // [B row_tiles]: an item's first part, its number of parts
    void *qabs, *qpe;                // absorbed and rotated queries
    // partials [slots][row_tile][Dk] and their log-sum-exps [slots][row_tile], slots = workers + B row_tiles:
    // fp32, or fp16 times a scale per half row [slots][row_tile][2] in the tensor-core form
    float *po32, *pl, *pscale;
    __half *po;
};
cudaError_t paged_decode_simt(const PagedDecode &p, cudaStream_t st);

// The tensor-core form (bf16): these dimensions and page size, any number of heads.
// pairs of SMs of a GB300, keys per tile (no worker waits for another: with fewer SMs free they take turns)
constexpr int PAGED_TC_WORKERS = 76, PAGED_TC_TILE = 64;
bool paged_tc_supported(int Dk, int Dn, int Dr, int Dv, int page);
cudaError_t paged_decode_tc(const PagedDecode &p, cudaStream_t st);
cudaError_t paged_tc_read_and_clear_error(unsigned *flags, cudaStream_t st);

}  // namespace mla
