// paged_evict.cu -- eviction from the paged cache: the pages of least accumulated attention weight leave the
// requests that hold more than a budget.
//
// Two launches.  pick, a block per request: how many pages go, k = min(held - keep, candidates), and the k-th
// smallest weight among the candidates by radix selection, a byte a pass (weights as integers in the order
// of the numbers); of pages with exactly that weight the first ones go.  apply, a block per request: where the
// request's list begins (the sum of k over the requests before it), then the row in order of its columns, with
// running counts of the evicted and of those with the k-th weight.
#include <algorithm>

#include "paged_common.cuh"
#include "tc_common.cuh"

namespace mla {

using namespace paged;
using tc::pdl_launch_dependents;
using tc::pdl_wait;

namespace {

struct Evict {
    int B, page, max_pages, room, keep, first, last;
    const int *lens, *table;
    const float *weights;
    int *table_out;
    float *weights_out;
    int *freed, *counts;
    int *gone;      // [B] pages that go
    uint2 *pick;    // [B] the k-th weight, how many of exactly that weight go
};

// A weight as an integer of the same order: -0 as 0, NaN above all.
__device__ __forceinline__ unsigned ordered(float w) {
    if (w != w) return 0xffffffffu;
    const unsigned u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ int columns_of(const Evict &a, int b) {
    const int n = min(max(a.lens[b], 0), a.max_pages * a.page);
    return n / a.page + (n % a.page != 0);
}
// The sum of x over the block's threads, in all of them; `sm` 32 ints.
__device__ __forceinline__ int block_sum(int x, int *sm) {
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
    __syncthreads();
    int s = 0;
    for (int i = 0; i < (int)blockDim.x >> 5; ++i) s += sm[i];
    return s;
}

__global__ void __launch_bounds__(1024) paged_evict_pick_kernel(const __grid_constant__ Evict a) {
    __shared__ int sm[32], bins[256];
    __shared__ unsigned at[2];   // the byte found, candidates below it
    const int tid = threadIdx.x, nt = blockDim.x, b = blockIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    const int *ids = a.table + (long)b * a.max_pages;
    const float *w = a.weights + (long)b * a.max_pages;
    const int cols = columns_of(a, b), c0 = min(a.first, cols), c1 = cols - min(a.last, cols);
    int held = 0, may = 0;
    for (int c = tid; c < cols; c += nt)
        if (ids[c] >= 0) {
            ++held;
            may += c >= c0 && c < c1;
        }
    held = block_sum(held, sm);
    may = block_sum(may, sm);
    const int k = min(max(held - a.keep, 0), may);
    if (k == 0) {
        if (tid == 0) {
            a.gone[b] = 0;
            a.pick[b] = make_uint2(0, 0);
        }
        return;
    }
    unsigned prefix = 0;
    int left = k;   // rank of the sought one among those of the prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += nt) bins[i] = 0;
        __syncthreads();
        for (int c = c0 + tid; c < c1; c += nt)
            if (ids[c] >= 0) {
                const unsigned u = ordered(w[c]);
                if (shift == 24 || u >> (shift + 8) == prefix >> (shift + 8)) atomicAdd(&bins[u >> shift & 255], 1);
            }
        __syncthreads();
        if (tid < 32) {   // eight bins a lane
            int n = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) n += bins[tid * 8 + i];
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (tid >= o) x += y;
            }
            int below = x - n;
            if (below < left && left <= x) {
                int i = 0;
                while (below + bins[tid * 8 + i] < left) below += bins[tid * 8 + i++];
                at[0] = tid * 8 + i;
                at[1] = below;
            }
        }
        __syncthreads();
        prefix |= at[0] << shift;
        left -= (int)at[1];
        __syncthreads();
    }
    if (tid == 0) {
        a.gone[b] = k;
        a.pick[b] = make_uint2(prefix, left);
    }
}

constexpr int PER = 4;   // columns of a thread and round

__global__ void __launch_bounds__(1024) paged_evict_apply_kernel(const __grid_constant__ Evict a) {
    __shared__ int sm[32], tot[2][32];
    const int tid = threadIdx.x, nt = blockDim.x, b = blockIdx.x, lane = tid & 31, wp = tid >> 5;
    pdl_wait();
    int before = 0;
    for (int i = tid; i < b; i += nt) before += a.gone[i];
    before = block_sum(before, sm);
    const int k = b < a.B ? a.gone[b] : 0;
    if (b >= a.B - 1 && tid == 0) {
        a.counts[0] = min(before + k, a.room);
        a.counts[1] = before + k;
    }
    if (b >= a.B) return;
    const uint2 pick = a.pick[b];
    const long row = (long)b * a.max_pages;
    const int cols = columns_of(a, b), c0 = min(a.first, cols), c1 = cols - min(a.last, cols);
    int ties = 0, out = before;   // of exactly the k-th weight so far; evicted so far
    for (int base = 0; base < a.max_pages; base += nt * PER) {
        const int c = base + tid * PER;
        int id[PER], tie = 0, less = 0;   // (masks)
        float w[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e)
            if (c + e < a.max_pages) {
                id[e] = a.table[row + c + e];
                w[e] = a.weights[row + c + e];
                if (k && id[e] >= 0 && c + e >= c0 && c + e < c1) {
                    const unsigned u = ordered(w[e]);
                    tie |= (u == pick.x) << e;
                    less |= (u < pick.x) << e;
                }
            }
        if (k && base < cols) {   // (the same answer in every thread)
            // a thread's place among the ties, then among the evicted
            auto place = [&](int n, int *t, int &all) {
                int x = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                __syncthreads();   // the last round's totals have been read
                if (lane == 31) t[wp] = x;
                __syncthreads();
                int p = x - n;
                all = 0;
                for (int i = 0; i < nt >> 5; ++i) {
                    if (i < wp) p += t[i];
                    all += t[i];
                }
                return p;
            };
            int all;
            int t = ties + place(__popc(tie), tot[0], all);
            ties += all;
#pragma unroll
            for (int e = 0; e < PER; ++e)
                if (tie >> e & 1) {
                    if ((unsigned)t++ < pick.y) less |= 1 << e;
                }
            int at = out + place(__popc(less), tot[1], all);
            out += all;
#pragma unroll
            for (int e = 0; e < PER; ++e)
                if (less >> e & 1) {
                    if (at < a.room) {
                        a.freed[at] = id[e];
                        id[e] = -1;
                        w[e] = 0.f;
                    }
                    ++at;
                }
        }
#pragma unroll
        for (int e = 0; e < PER; ++e)
            if (c + e < a.max_pages) {
                a.table_out[row + c + e] = id[e];
                a.weights_out[row + c + e] = w[e];
            }
    }
}

}  // namespace

cudaError_t launch_paged_evict(int B, int page, int max_pages, int room, int keep, int first, int last, const int *lens,
                               const int *table, const float *weights, int *table_out, float *weights_out, int *freed,
                               int *counts, int *gone, uint2 *pick, cudaStream_t st) {
    const Evict a{B, page, max_pages, room, keep, first, last, lens, table, weights, table_out, weights_out, freed, counts, gone, pick};
    const unsigned threads = max_pages <= 512 ? 128 : max_pages <= 4096 ? 256 : 1024;
    if (B > 0) {
        ProfScope ps("paged_evict", st);
        const cudaError_t e = launch_after(paged_evict_pick_kernel, (unsigned)B, threads, 0, st, a);
        if (e != cudaSuccess) return e;
    }
    ProfScope ps("paged_evict", st);
    return launch_after(paged_evict_apply_kernel, (unsigned)std::max(B, 1), threads, 0, st, a);
}

}  // namespace mla
