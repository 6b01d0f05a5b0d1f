// paged.cu -- bookkeeping and writes of the paged latent cache: block tables and slot maps from
// request lengths, and the cache write of new tokens (RMSNorm of the latent, RoPE of the key
// band, scatter to the tokens' slots).
#include <algorithm>

#include "paged_common.cuh"

namespace mla {

void paged_turns(float base, int Dr, unsigned long long *v) {
    for (int t = 0; t < Dr / 2; ++t) {
        const double f = pow((double)base, -2.0 * t / Dr) / 6.283185307179586476925286766559;
        v[t] = (unsigned long long)ldexp(f - floor(f), 64);
    }
}

namespace {

using namespace paged;

// ------------------------------------------------------------------------ tables ----
// Each block forms both prefix sums (tokens, pages taken) over all requests in its own shared
// memory and then fills its share of the token and page rows; no block waits for another.
constexpr int TB = 1024;

struct Tables {
    int B, page, max_pages, n_free, n_tokens;
    const int *past, *fresh, *free_pages;
    int *table, *kv_lens, *cu, *slots, *positions, *counts;
};

__device__ __forceinline__ int sat(long v) { return (int)min(v, 2147483647l); }

struct Request {
    int past, have;   // tokens and pages held before
    long placed, extra;
};
__device__ __forceinline__ Request request(const Tables &a, int b, long cu) {
    const long cap = (long)a.max_pages * a.page;
    Request r;
    r.past = (int)min((long)max(a.past[b], 0), cap);
    r.placed = max(min(min((long)a.fresh[b], (long)a.n_tokens - cu), cap - r.past), 0l);
    r.have = (r.past + a.page - 1) / a.page;
    r.extra = (r.past + r.placed + a.page - 1) / a.page - r.have;
    return r;
}

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

__global__ void __launch_bounds__(TB) paged_tables_kernel(Tables a) {
    extern __shared__ int sm[];
    __shared__ long warp_tot[TB / 32];
    int *cu = sm, *off = sm + a.B + 1;
    const int tid = threadIdx.x;
    long tok = 0, pages = 0;
    for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {   // the last request's successor holds the totals
        const int b = b0 + tid;
        long all;
        const long n = b < a.B ? max(a.fresh[b], 0) : 0;
        const long c = tok + block_scan(n, warp_tot, all);
        tok += all;
        Request r{};
        if (b < a.B) r = request(a, b, c);
        const long o = pages + block_scan(r.extra, warp_tot, all);
        pages += all;
        if (b < a.B) {
            cu[b] = sat(c);
            off[b] = sat(o);
            if (blockIdx.x == 0) {
                const long got = min(max((long)a.n_free - o, 0l), r.extra);
                a.cu[b] = sat(c);
                a.kv_lens[b] = (int)(got == r.extra ? r.past + r.placed
                                                    : max((long)r.past, (r.have + got) * (long)a.page));
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
    const long step = (long)gridDim.x * blockDim.x;
    // pages: entry e of the free list goes to the request whose prefix range holds e
    const long taken = min((long)off[a.B], (long)a.n_free);
    for (long e = (long)blockIdx.x * blockDim.x + tid; e < taken; e += step) {
        int lo = 0, hi = a.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (off[mid] <= e) lo = mid;
            else hi = mid - 1;
        }
        const Request r = request(a, lo, cu[lo]);
        a.table[(long)lo * a.max_pages + r.have + (e - off[lo])] = a.free_pages[e];
    }
    // tokens
    for (long t = (long)blockIdx.x * blockDim.x + tid; t < a.n_tokens; t += step) {
        int slot = -1, pos = 0;
        if (t < cu[a.B]) {
            int lo = 0, hi = a.B - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cu[mid] <= t) lo = mid;
                else hi = mid - 1;
            }
            const Request r = request(a, lo, cu[lo]);
            const long i = t - cu[lo], at = r.past + i;
            pos = sat(at);
            if (i < r.placed) {
                const int col = (int)(at / a.page), in = (int)(at % a.page);
                int id = -1;
                if (col < r.have) {
                    id = a.table[(long)lo * a.max_pages + col];
                } else {
                    const long e = (long)off[lo] + col - r.have;
                    if (e < a.n_free) id = a.free_pages[e];
                }
                const long s = (long)id * a.page + in;
                if (id >= 0 && s <= 2147483647l) slot = (int)s;
            }
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
    }
}

// ------------------------------------------------------------------------ append ----
// One warp per token: chat = c w / sqrt(mean c^2 + eps) and the rotated key band, both rounded
// once to the cache's type at the token's slot.  Slots outside [0, n_slots) are skipped.
struct Append {
    int T, Dk, Dr;
    long n_slots, c_stride, k_stride;
    float eps;
    const void *c, *k, *w;
    const int *slots, *positions;
    void *c_cache, *kpe_cache;
    Turns turns;
};

template <typename T>
__global__ void __launch_bounds__(256) paged_append_kernel(const __grid_constant__ Append a) {
    const int lane = threadIdx.x & 31, half = a.Dr / 2;
    const long warp = ((long)blockIdx.x * blockDim.x + threadIdx.x) >> 5, nwarps = ((long)gridDim.x * blockDim.x) >> 5;
    for (long t = warp; t < a.T; t += nwarps) {
        const long slot = a.slots[t];
        if (slot < 0 || slot >= a.n_slots) continue;
        const int pos = a.positions[t];
        const T *c = (const T *)a.c + t * a.c_stride, *k = (const T *)a.k + t * a.k_stride, *w = (const T *)a.w;
        T *co = (T *)a.c_cache + slot * a.Dk, *ko = (T *)a.kpe_cache + slot * a.Dr;
        float s = 0.f;
        for (int d = lane; d < a.Dk; d += 32) {
            const float v = to_f<T>(c[d]);
            s = fmaf(v, v, s);
        }
        const float r = 1.f / sqrtf(warp_sum(s) / (float)a.Dk + a.eps);
        for (int d = lane; d < a.Dk; d += 32) co[d] = from_f<T>(to_f<T>(c[d]) * r * to_f<T>(w[d]));
        for (int i = lane; i < half; i += 32) {
            const float2 cs = turn_cs(a.turns.v[i], pos);
            const float x = to_f<T>(k[i]), y = to_f<T>(k[i + half]);
            ko[i] = from_f<T>(x * cs.x - y * cs.y);
            ko[i + half] = from_f<T>(y * cs.x + x * cs.y);
        }
    }
}

}  // namespace

cudaError_t launch_paged_tables(int B, int page, int max_pages, int n_free, int n_tokens, const int *past,
                                const int *fresh, const int *free_pages, int *table, int *kv_lens, int *cu, int *slots,
                                int *positions, int *counts, cudaStream_t st) {
    Tables a{B, page, max_pages, n_free, n_tokens, past, fresh, free_pages, table, kv_lens, cu, slots, positions, counts};
    const int smem = 2 * (B + 1) * (int)sizeof(int);
    const int blocks = (int)std::min(152l, std::max(1l, ((long)n_tokens + TB - 1) / TB));
    cudaError_t e = cudaFuncSetAttribute(paged_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ProfScope ps("paged_tables", st);
    paged_tables_kernel<<<blocks, TB, smem, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_paged_append(int ty, int T, long n_slots, int Dk, int Dr, float base, float eps, const void *c,
                                long c_stride, const void *k, long k_stride, const void *w, const int *slots,
                                const int *positions, void *c_cache, void *kpe_cache, cudaStream_t st) {
    Append a{T, Dk, Dr, n_slots, c_stride, k_stride, eps, c, k, w, slots, positions, c_cache, kpe_cache, {}};
    paged_turns(base, Dr, a.turns.v);
    const int blocks = (int)std::min(152l * 8, ((long)T + 7) / 8);
    ProfScope ps("paged_append", st);
    if (ty == TY_F32) paged_append_kernel<float><<<blocks, 256, 0, st>>>(a);
    else paged_append_kernel<__nv_bfloat16><<<blocks, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace mla
