// paged.cu -- bookkeeping and writes of the paged latent cache: block tables and slot maps from
// request lengths, and the cache write of new tokens (RMSNorm of the latent, RoPE of the key
// band, scatter to the tokens' slots).
#include <algorithm>

#include "paged_common.cuh"
#include "tc_common.cuh"

namespace mla {

using namespace paged;
using tc::pdl_wait;

const unsigned long long *paged_turns(float base, int Dr) {
    static thread_local unsigned long long v[MAX_HALF];
    static thread_local float last_base = 0.f;
    static thread_local int last_dr = 0;
    if (last_base != base || last_dr != Dr) {
        for (int t = 0; t < Dr / 2; ++t) {
            const double f = pow((double)base, -2.0 * t / Dr) / 6.283185307179586476925286766559;
            v[t] = (unsigned long long)ldexp(f - floor(f), 64);
        }
        last_base = base;
        last_dr = Dr;
    }
    return v;
}

namespace {

// ------------------------------------------------------------------------ tables ----
// Each block forms both prefix sums (tokens, pages taken) over all requests in its own shared
// memory and then fills its share of the token and page rows; no block waits for another.  The rows
// are found by binary search in shared memory; everything per row is 32-bit arithmetic, with the
// division by the page size as a multiplication (64-bit divisions took 9 of 15 us at 2001 requests
// and half a million tokens).  Of the 10.2-10.5 us that 2001 requests of 576 thousand tokens take in a graph,
// launch and loads are 1.9, the scans of the first 1024 lengths 2.4, of the rest 3.0 (two scans of 64-bit sums a
// round, in every block, whose warp totals each thread adds up by itself), searches and rows 2.9.
struct Tables {
    int B, page, max_pages, n_free, n_tokens;
    Divisor by_page;
    const int *past, *fresh, *free_pages;
    int *table, *kv_lens, *cu, *slots, *positions, *counts;
};

__device__ __forceinline__ int sat(long v) { return (int)min(v, 2147483647l); }

// Exclusive prefix of one value per thread over the block; the total in `all`.
__device__ __forceinline__ long block_scan(long n, long *warp_tot, long &all) {
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    long x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();   // the previous scan's totals have been read
    if (lane == 31) warp_tot[wp] = x;
    __syncthreads();
    long before = 0, sum = 0;
    const int nw = blockDim.x >> 5;
    for (int i = 0; i < nw; ++i) {
        if (i < wp) before += warp_tot[i];
        sum += warp_tot[i];
    }
    all = sum;
    return before + x - n;
}

// The last of n requests whose prefix is <= x.
__device__ __forceinline__ int owner(const int *prefix, int n, int x) {
    int lo = 0;
    while (n > 1) {
        const int half = n >> 1;
        if (prefix[lo + half] <= x) lo += half;
        n -= half;
    }
    return lo;
}

// PER: token rows of a thread.
template <int PER>
__global__ void __launch_bounds__(1024) paged_tables_kernel(const __grid_constant__ Tables a) {
    extern __shared__ int sm[];
    __shared__ long warp_tot[32];
    int *cu = sm, *off = cu + a.B + 1, *past = off + a.B + 1;
    const int tid = threadIdx.x, cap = a.max_pages * a.page;
    pdl_wait();
    long tok = 0, pages = 0;
    for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
        const int b = b0 + tid;
        const bool in = b < a.B;
        const int p0 = in ? min(max(a.past[b], 0), cap) : 0, fresh = in ? max(a.fresh[b], 0) : 0;
        long all;
        const long c = tok + block_scan(fresh, warp_tot, all);
        tok += all;
        const int placed = max((int)min(min((long)fresh, (long)a.n_tokens - c), (long)(cap - p0)), 0);
        const int have = quotient(a.by_page, p0 + a.page - 1), extra = quotient(a.by_page, p0 + placed + a.page - 1) - have;
        const long o = pages + block_scan(extra, warp_tot, all);
        pages += all;
        if (in) {
            cu[b] = sat(c);
            off[b] = sat(o);
            past[b] = p0;
            if (blockIdx.x == 0) {
                const int got = (int)min(max((long)a.n_free - o, 0l), (long)extra);
                a.cu[b] = sat(c);
                a.kv_lens[b] = got == extra ? p0 + placed : max(p0, (have + got) * a.page);
            }
        }
    }
    if (tid == 0) {
        cu[a.B] = sat(tok);
        off[a.B] = sat(pages);
        if (blockIdx.x == 0) {
            a.cu[a.B] = sat(tok);
            a.counts[0] = sat(min(pages, (long)a.n_free));
            a.counts[1] = sat(pages);
        }
    }
    __syncthreads();
    const long step = (long)gridDim.x * blockDim.x, first = (long)blockIdx.x * blockDim.x + tid;
    // pages: entry e of the free list goes to the request whose prefix range holds e
    const int taken = min(off[a.B], a.n_free), tokens = min(cu[a.B], a.n_tokens);
    for (long e = first; e < taken; e += step) {
        const int b = owner(off, a.B, (int)e);
        const int have = quotient(a.by_page, past[b] + a.page - 1);
        a.table[(long)b * a.max_pages + have + ((int)e - off[b])] = a.free_pages[e];
    }
    // tokens, PER neighbours to a thread: one search, then a walk; rows behind the last token belong to no
    // request
    const bool wide = PER == 4 && (((uintptr_t)a.slots | (uintptr_t)a.positions) & 15) == 0;
    for (long t4 = first * PER; t4 < a.n_tokens; t4 += step * PER) {
        int slot[PER], pos[PER];
        int b = t4 < tokens ? owner(cu, a.B, (int)t4) : 0;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const long t = t4 + k;
            slot[k] = -1;
            pos[k] = 0;
            if (t >= tokens) continue;
            while (cu[b + 1] <= t) ++b;
            const int p0 = past[b];
            const unsigned at = (unsigned)p0 + (unsigned)((int)t - cu[b]);   // below 2^30 + 2^31
            pos[k] = (int)min(at, 2147483647u);
            if (at >= (unsigned)cap) continue;
            const int col = quotient(a.by_page, pos[k]), have = quotient(a.by_page, p0 + a.page - 1);
            const long e = (long)off[b] + col - have;
            int id = -1;
            if (col < have) id = a.table[(long)b * a.max_pages + col];
            else if (e < a.n_free) id = a.free_pages[e];
            const long s = (long)id * a.page + (pos[k] - col * a.page);
            if (id >= 0 && s <= 2147483647l) slot[k] = (int)s;
        }
        if (wide && t4 + 4 <= a.n_tokens) {
            *(int4 *)(a.slots + t4) = make_int4(slot[0], slot[PER / 4], slot[PER / 2], slot[PER - 1]);
            *(int4 *)(a.positions + t4) = make_int4(pos[0], pos[PER / 4], pos[PER / 2], pos[PER - 1]);
        } else {
#pragma unroll
            for (int k = 0; k < PER; ++k)
                if (t4 + k < a.n_tokens) {
                    a.slots[t4 + k] = slot[k];
                    a.positions[t4 + k] = pos[k];
                }
        }
    }
}

// ------------------------------------------------------------------------ append ----
// One warp per token: chat = c w / sqrt(mean c^2 + eps) and the rotated key band, both rounded
// once to the cache's type at the token's slot.  Slots outside [0, n_slots) are skipped.  The band's position and
// elements are loaded behind the latent's stores (which may alias them, for all the compiler knows), element by
// element: a second trip to memory in a row.  16384 tokens of 512 + 64 bf16 take 8.2 us in a graph; their bytes
// need 5.6.
struct Append {
    int T, Dk, Dr;
    long n_slots, c_stride, k_stride;
    float eps;
    const void *c, *k, *w;
    const int *slots, *positions;
    void *c_cache, *kpe_cache;
};

template <typename T, typename TU>
__device__ __forceinline__ void rotate_row(const Append &a, const TU &turns, long t, long slot, int lane) {
    const int half = a.Dr / 2, pos = a.positions[t];
    const T *k = (const T *)a.k + t * a.k_stride;
    T *o = (T *)a.kpe_cache + slot * a.Dr;
    for (int i = lane; i < half; i += 32) {
        const float x = to_f<T>(k[i]), y = to_f<T>(k[i + half]);
        const float2 cs = turn_cs(turns.v[i], pos);
        o[i] = from_f<T>(x * cs.x - y * cs.y);
        o[i + half] = from_f<T>(y * cs.x + x * cs.y);
    }
}

// Any width and row pitch.
template <typename T>
__global__ void __launch_bounds__(256) paged_append_kernel(const __grid_constant__ Append a, const __grid_constant__ Turns turns) {
    const int lane = threadIdx.x & 31;
    pdl_wait();
    const long t = ((long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (t >= a.T) return;
    const long slot = a.slots[t];
    if (slot < 0 || slot >= a.n_slots) return;
    const T *c = (const T *)a.c + t * a.c_stride, *w = (const T *)a.w;
    T *co = (T *)a.c_cache + slot * a.Dk;
    float s = 0.f;
    for (int d = lane; d < a.Dk; d += 32) {
        const float v = to_f<T>(c[d]);
        s = fmaf(v, v, s);
    }
    const float r = 1.f / sqrtf(warp_sum(s) / (float)a.Dk + a.eps);
    for (int d = lane; d < a.Dk; d += 32) co[d] = from_f<T>(to_f<T>(c[d]) * r * to_f<T>(w[d]));
    rotate_row<T>(a, turns, t, slot, lane);
}

// 16-byte pieces: rows of a whole number of pieces, up to 32 NC, held in registers between the sum and
// the write; one read and one write of every byte.  16384 tokens of 512 + 64 bf16: 13.3 us by single
// elements.
template <typename T, int NC, typename TU>
__global__ void __launch_bounds__(256) paged_append_vec_kernel(const __grid_constant__ Append a, const __grid_constant__ TU turns) {
    constexpr int E = 16 / (int)sizeof(T);
    const int lane = threadIdx.x & 31, pieces = a.Dk / E;
    pdl_wait();
    const long t = ((long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (t >= a.T) return;
    const long slot = a.slots[t];
    const uint4 *c = (const uint4 *)((const T *)a.c + t * a.c_stride), *w = (const uint4 *)a.w;
    uint4 x[NC], y[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i)
        if (lane + 32 * i < pieces) {
            x[i] = __ldcs(c + lane + 32 * i);
            y[i] = __ldg(w + lane + 32 * i);
        } else {
            x[i] = y[i] = make_uint4(0, 0, 0, 0);
        }
    if (slot < 0 || slot >= a.n_slots) return;
    float f[NC][E], s = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        alignas(16) T v[E];
        *(uint4 *)v = x[i];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            f[i][e] = to_f<T>(v[e]);
            s = fmaf(f[i][e], f[i][e], s);
        }
    }
    const float r = 1.f / sqrtf(warp_sum(s) / (float)a.Dk + a.eps);
    uint4 *o = (uint4 *)((T *)a.c_cache + slot * a.Dk);
#pragma unroll
    for (int i = 0; i < NC; ++i)
        if (lane + 32 * i < pieces) {
            alignas(16) T v[E];
            *(uint4 *)v = y[i];
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = from_f<T>(f[i][e] * r * to_f<T>(v[e]));
            o[lane + 32 * i] = *(const uint4 *)v;
        }
    rotate_row<T>(a, turns, t, slot, lane);
}

template <typename T, int NC>
cudaError_t append_vec(const Append &a, const unsigned long long *v, cudaStream_t st) {
    const unsigned blocks = (unsigned)(((long)a.T + 7) / 8);
    if (a.Dr <= 64) {
        Turns64 turns{};
        std::copy(v, v + a.Dr / 2, turns.v);
        return launch_after(paged_append_vec_kernel<T, NC, Turns64>, blocks, 256, 0, st, a, turns);
    }
    Turns turns{};
    std::copy(v, v + a.Dr / 2, turns.v);
    return launch_after(paged_append_vec_kernel<T, NC, Turns>, blocks, 256, 0, st, a, turns);
}

template <typename T>
cudaError_t append(const Append &a, const unsigned long long *v, cudaStream_t st) {
    constexpr int E = 16 / (int)sizeof(T);
    const int pieces = a.Dk % E == 0 && a.c_stride % E == 0 ? a.Dk / E : 0;
    if (pieces > 0 && pieces <= 32) return append_vec<T, 1>(a, v, st);
    if (pieces > 0 && pieces <= 64) return append_vec<T, 2>(a, v, st);
    if (pieces > 0 && pieces <= 128) return append_vec<T, 4>(a, v, st);
    Turns turns{};
    std::copy(v, v + a.Dr / 2, turns.v);
    return launch_after(paged_append_kernel<T>, (unsigned)(((long)a.T + 7) / 8), 256, 0, st, a, turns);
}

}  // namespace

cudaError_t launch_paged_tables(int B, int page, int max_pages, int n_free, int n_tokens, const int *past,
                                const int *fresh, const int *free_pages, int *table, int *kv_lens, int *cu, int *slots,
                                int *positions, int *counts, cudaStream_t st) {
    Tables a{B, page, max_pages, n_free, n_tokens, divisor(page), past, fresh, free_pages, table, kv_lens, cu, slots, positions, counts};
    const int smem = (3 * B + 2) * (int)sizeof(int);
    // A block per 1024 threads, one per SM at most, small steps in a small block (fewer warps to bring
    // together); four rows a thread once one a thread would fill the GPU (half a million tokens of 2001
    // requests: 10.6 against 12.0 us; 66 thousand of eight: 6.9 against 5.4 us).
    const bool four = n_tokens > 152 * 1024;
    const long rows = std::max(four ? ((long)n_tokens + 3) / 4 : (long)n_tokens, (long)B);
    const int threads = rows <= 128 ? 128 : rows <= 512 ? 256 : 1024;
    const int blocks = (int)std::min(152l, std::max(1l, (rows + threads - 1) / threads));
    auto kern = four ? paged_tables_kernel<4> : paged_tables_kernel<1>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    ProfScope ps("paged_tables", st);
    return launch_after(kern, (unsigned)blocks, (unsigned)threads, (size_t)smem, st, a);
}

cudaError_t launch_paged_append(int ty, int T, long n_slots, int Dk, int Dr, float base, float eps, const void *c,
                                long c_stride, const void *k, long k_stride, const void *w, const int *slots,
                                const int *positions, void *c_cache, void *kpe_cache, cudaStream_t st) {
    Append a{T, Dk, Dr, n_slots, c_stride, k_stride, eps, c, k, w, slots, positions, c_cache, kpe_cache};
    const unsigned long long *v = paged_turns(base, Dr);
    ProfScope ps("paged_append", st);
    return ty == TY_F32 ? append<float>(a, v, st) : append<__nv_bfloat16>(a, v, st);
}

}  // namespace mla
