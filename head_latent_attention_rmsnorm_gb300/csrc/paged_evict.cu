// paged_evict.cu -- eviction from the paged cache: the pages of least accumulated attention weight leave the
// requests that hold more than a budget.
//
// Two launches; a request's columns are cut into segments, a block each.  pick, the request's blocks as a cluster:
// how many pages go, k = min(held - keep, candidates), and the k-th smallest weight among the candidates by radix
// selection, a byte a pass (weights as integers in the order of the numbers; the blocks' counts meet through distributed
// shared memory); of pages with exactly that weight the first ones go.  apply, a block per segment: where its list
// begins (the sum of k over the requests before it, and the segments' counts), then its columns in order, with
// running counts of the evicted and of those with the k-th weight.
//
// Bound by latency: launches, loads and some twenty barriers for 16 bytes a column.  The segments are what a block holds
// in registers (a row of 65536 columns by one block took 176 us).
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
    int segs, seg;  // segments of a request, columns of each
    const int *lens, *table;
    const float *weights;
    int *table_out;
    float *weights_out;
    int *freed, *counts;
    int *gone;      // [B] pages that go
    uint4 *pick;    // [B][segs] the k-th weight, how many of exactly that weight go; in front of the segment: evicted, of that weight
};
constexpr int PER = 8;   // columns that a thread of the second launch holds

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
// The sums of x and y over the block's threads, in all of them; `sm` 32 pairs.
__device__ __forceinline__ int2 block_sums(int x, int y, int2 *sm) {
    x = __reduce_add_sync(0xffffffffu, x);
    y = __reduce_add_sync(0xffffffffu, y);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = make_int2(x, y);
    __syncthreads();
    const int n = (int)blockDim.x >> 5, lane = threadIdx.x & 31;
    const int2 v = lane < n ? sm[lane] : make_int2(0, 0);
    return make_int2(__reduce_add_sync(0xffffffffu, v.x), __reduce_add_sync(0xffffffffu, v.y));
}

// HOLD: columns of a thread, kept in registers; 0: read again for every pass.
template <int HOLD>
__global__ void __launch_bounds__(1024) paged_evict_pick_kernel(const __grid_constant__ Evict a) {
    __shared__ int2 sm[32], mine, cand;
    __shared__ int bins[2][256], all[256];   // bins: by parity of the pass
    __shared__ unsigned at[2][2];             // the byte found, candidates below it
    const int tid = threadIdx.x, nt = blockDim.x, segs = a.segs, rank = segs > 1 ? (int)tc::cluster_ctarank() : 0;
    const int b = blockIdx.x / segs;
    pdl_wait();
    pdl_launch_dependents();
    const int *ids = a.table + (long)b * a.max_pages;
    const float *w = a.weights + (long)b * a.max_pages;
    const int cols = columns_of(a, b), c0 = min(a.first, cols), c1 = cols - min(a.last, cols);
    const int s0 = rank * a.seg, s1 = min(s0 + a.seg, cols);
    // block `from`'s value of a shared variable of the cluster
    auto remote = [&](const int *x, int from) {
        if (segs == 1) return *x;
        int v;
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(tc::map_peer(tc::smem_u32(x), from)) : "memory");
        return v;
    };
    auto meet = [&] {
        if (segs > 1) tc::cluster_sync();
        else __syncthreads();
    };
    constexpr bool FITS = HOLD > 0;
    unsigned key[FITS ? HOLD : 1];
    unsigned may = 0;   // (mask) candidates among the held ones
    int held = 0, n_may = 0;
    if (FITS) {
        int id[FITS ? HOLD : 1];
#pragma unroll
        for (int e = 0; e < HOLD; ++e) {
            const int c = s0 + tid + e * nt;
            id[e] = c < s1 ? ids[c] : -1;
            key[e] = c < s1 ? ordered(w[c]) : 0;
        }
#pragma unroll
        for (int e = 0; e < HOLD; ++e) {
            const int c = s0 + tid + e * nt;
            held += id[e] >= 0;
            may |= (unsigned)(id[e] >= 0 && c >= c0 && c < c1) << e;
        }
        n_may = __popc(may);
    } else {
        for (int c = s0 + tid; c < s1; c += nt)
            if (ids[c] >= 0) {
                ++held;
                n_may += c >= c0 && c < c1;
            }
    }
    // f(key) of every candidate
    auto each = [&](auto f) {
        if (FITS) {
#pragma unroll
            for (int e = 0; e < HOLD; ++e)
                if (may >> e & 1) f(key[e]);
        } else {
            for (int c = max(s0, c0) + tid; c < min(s1, c1); c += nt)
                if (ids[c] >= 0) f(ordered(w[c]));
        }
    };
    for (int i = tid; i < 512; i += nt) bins[i >> 8][i & 255] = 0;
    const int2 sums = block_sums(held, n_may, sm);
    held = sums.x;
    n_may = sums.y;
    if (segs > 1) {
        if (tid == 0) mine = sums;
        meet();
        const int lane = tid & 31, h = lane < segs ? remote(&mine.x, lane) : 0, m = lane < segs ? remote(&mine.y, lane) : 0;
        held = __reduce_add_sync(0xffffffffu, h);
        n_may = __reduce_add_sync(0xffffffffu, m);
    }
    const int k = min(max(held - a.keep, 0), n_may);
    if (k == 0) {   // (the same in all of the cluster)
        if (tid == 0) {
            if (rank == 0) a.gone[b] = 0;
            a.pick[(long)b * segs + rank] = make_uint4(0, 0, 0, 0);
        }
        meet();   // nobody leaves while another reads its numbers
        return;
    }
    unsigned prefix = 0;
    int left = k;   // rank of the sought one among those of the prefix
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        int *bin = bins[pass & 1];
        each([&](unsigned u) {
            if (pass == 0 || u >> (shift + 8) == prefix >> (shift + 8)) atomicAdd(&bin[u >> shift & 255], 1);
        });
        meet();
        const int *sum = bin;
        if (segs > 1) {
            for (int i = tid; i < 256; i += nt) {
                int n = 0;
                for (int j = 0; j < segs; ++j) n += remote(&bin[i], j);
                all[i] = n;
            }
            __syncthreads();
            sum = all;
        }
        // (all have read the last pass's counts: they got to this one's meeting)
        if (pass > 0)
            for (int i = tid; i < 256; i += nt) bins[(pass & 1) ^ 1][i] = 0;
        if (tid < 32) {   // eight bins a lane
            int n = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) n += sum[tid * 8 + i];
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (tid >= o) x += y;
            }
            int below = x - n;
            if (below < left && left <= x) {
                int i = 0;
                while (below + sum[tid * 8 + i] < left) below += sum[tid * 8 + i++];
                at[pass & 1][0] = tid * 8 + i;
                at[pass & 1][1] = below;
            }
        }
        __syncthreads();
        prefix |= at[pass & 1][0] << shift;
        left -= (int)at[pass & 1][1];
    }
    if (segs == 1) {   // nothing in front
        if (tid == 0) {
            a.gone[b] = k;
            a.pick[b] = make_uint4(prefix, left, 0, 0);
        }
        return;
    }
    // the segments in front
    int less = 0, ties = 0;
    each([&](unsigned u) {
        less += u < prefix;
        ties += u == prefix;
    });
    const int2 of = block_sums(less, ties, sm);
    if (tid == 0) cand = of;
    meet();
    if (tid < 32) {
        less = __reduce_add_sync(0xffffffffu, tid < rank ? remote(&cand.x, tid) : 0);
        ties = __reduce_add_sync(0xffffffffu, tid < rank ? remote(&cand.y, tid) : 0);
        if (tid == 0) {
            if (rank == 0) a.gone[b] = k;
            a.pick[(long)b * segs + rank] = make_uint4(prefix, left, less + min(ties, left), ties);
        }
    }
    meet();   // nobody leaves while another reads its numbers
}

__global__ void __launch_bounds__(1024) paged_evict_apply_kernel(const __grid_constant__ Evict a) {
    __shared__ int2 sm[32];
    __shared__ int tot[2][32];
    const int tid = threadIdx.x, nt = blockDim.x, b = blockIdx.x / a.segs, s = blockIdx.x % a.segs, lane = tid & 31, wp = tid >> 5;
    const long row = (long)b * a.max_pages;
    const int first = s * a.seg, s1 = min(first + a.seg, a.max_pages);
    // a warp's 256 columns, 32 neighbours at a time; the first ones are inputs of the launch in front too, which began
    // behind what wrote them
    int id[PER];
    float w[PER];
    auto load = [&](int c) {
#pragma unroll
        for (int e = 0; e < PER; ++e)
            if (c + 32 * e < s1) {
                id[e] = a.table[row + c + 32 * e];
                w[e] = a.weights[row + c + 32 * e];
            }
    };
    const int at0 = wp * 32 * PER + lane;
    if (b < a.B) load(first + at0);
    pdl_wait();
    const int k = b < a.B ? a.gone[b] : 0;
    int before = 0;
    if (k || b >= a.B - 1) {   // (the same in all threads)
        for (int i = tid; i < b; i += nt) before += a.gone[i];
        before = block_sums(before, 0, sm).x;
    }
    if (b >= a.B - 1 && s == 0 && tid == 0) {
        a.counts[0] = min(before + k, a.room);
        a.counts[1] = before + k;
    }
    if (b >= a.B) return;
    const uint4 pick = a.pick[(long)b * a.segs + s];
    const int cols = columns_of(a, b), c0 = min(a.first, cols), c1 = cols - min(a.last, cols);
    int ties = (int)pick.w, out = before + (int)pick.z;   // of exactly the k-th weight so far; evicted so far
    for (int base = first; base < s1; base += nt * PER) {
        const int c = base + at0;
        if (base > first) load(c);
        if (k && base < cols) {   // (the same answer in every thread)
            unsigned tie[PER], less[PER];   // of the warp's columns, by 32
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int col = c + 32 * e;
                const bool may = col < s1 && col >= c0 && col < c1 && id[e] >= 0;
                const unsigned u = may ? ordered(w[e]) : 0;
                tie[e] = __ballot_sync(0xffffffffu, may && u == pick.x);
                less[e] = __ballot_sync(0xffffffffu, may && u < pick.x);
            }
            // how many bits the warps in front have, and all
            auto before_warp = [&](const unsigned (&x)[PER], int *t, int &all) {
                int n = 0;
#pragma unroll
                for (int e = 0; e < PER; ++e) n += __popc(x[e]);
                __syncthreads();   // the last round's totals have been read
                if (lane == 0) t[wp] = n;
                __syncthreads();
                const int v = lane < nt >> 5 ? t[lane] : 0;
                all = __reduce_add_sync(0xffffffffu, v);
                return (int)__reduce_add_sync(0xffffffffu, lane < wp ? v : 0);
            };
            const unsigned below = (1u << lane) - 1;
            int all, t = ties + before_warp(tie, tot[0], all);
            ties += all;
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const bool goes = (tie[e] >> lane & 1) && (unsigned)(t + __popc(tie[e] & below)) < pick.y;
                t += __popc(tie[e]);
                less[e] |= __ballot_sync(0xffffffffu, goes);
            }
            int at = out + before_warp(less, tot[1], all);
            out += all;
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int place = at + __popc(less[e] & below);
                if ((less[e] >> lane & 1) && place < a.room) {
                    a.freed[place] = id[e];
                    id[e] = -1;
                    w[e] = 0.f;
                }
                at += __popc(less[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < PER; ++e)
            if (c + 32 * e < s1) {
                a.table_out[row + c + 32 * e] = id[e];
                a.weights_out[row + c + 32 * e] = w[e];
            }
    }
}

}  // namespace

int paged_evict_segments(int max_pages) {
    int n = 1;
    while (n < 8 && n * 1024 * PER < max_pages) n *= 2;
    return n;
}

cudaError_t launch_paged_evict(int B, int page, int max_pages, int room, int keep, int first, int last, const int *lens,
                               const int *table, const float *weights, int *table_out, float *weights_out, int *freed,
                               int *counts, int *gone, uint4 *pick, cudaStream_t st) {
    const int segs = paged_evict_segments(max_pages), seg = (max_pages + segs - 1) / segs;
    const Evict a{B, page, max_pages, room, keep, first, last, segs, seg, lens, table, weights, table_out, weights_out, freed, counts, gone, pick};
    const int threads = std::min(1024, std::max(64, (seg + PER - 1) / PER + 31) / 32 * 32);
    if (B > 0) {
        auto kern = seg <= threads * PER       ? paged_evict_pick_kernel<PER>
                    : seg <= threads * 2 * PER ? paged_evict_pick_kernel<2 * PER>
                                               : paged_evict_pick_kernel<0>;
        cudaLaunchAttribute at[2];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim.x = segs;
        at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)B * segs);
        cfg.blockDim = dim3(threads);
        cfg.stream = st;
        cfg.attrs = at;
        cfg.numAttrs = segs > 1 ? 2 : 1;
        ProfScope ps("paged_evict", st);
        const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
        if (e != cudaSuccess) return e;
    }
    ProfScope ps("paged_evict", st);
    return launch_after(paged_evict_apply_kernel, (unsigned)std::max(B * segs, 1), (unsigned)threads, 0, st, a);
}

}  // namespace mla
