// paged_step.cu -- a serving step's tokens over the paged latent cache: which tokens share a work item, the
// division of the items among the workers; which requests' tokens go in the explicit form, and their keys'
// rows gathered from the pages.
#include <cuda_fp16.h>

#include <algorithm>

#include "paged_common.cuh"
#include "tc_common.cuh"

namespace mla {

using namespace paged;
using tc::pdl_launch_dependents;
using tc::pdl_wait;

namespace {

// -------------------------------------------------------------------------- plan ----
// Block 0 divides (plan_tokens); the others set `zero` to zero.
constexpr int PNT = 1024;
constexpr int SOME = 512;   // tokens up to which a block of as many threads is enough (fewer warps to bring together)

struct Plan {
    PagedDecode p;
    PagedPlan s;
};

template <int NT, int PER>
__global__ void __launch_bounds__(NT) paged_plan_kernel(const __grid_constant__ Plan a) {
    extern __shared__ int sm[];
    const PagedDecode &p = a.p;
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();   // the absorb beside this; what follows it waits for both
    if (blockIdx.x > 0) {
        for (long i = (long)(blockIdx.x - 1) * NT + tid; i < a.s.n_zero; i += (long)(gridDim.x - 1) * NT) a.s.zero[i] = 0;
        return;
    }
    const int T = tokens_of(p);
    if (p.list && T == 0) {   // (the join has no token to look anything up for)
        for (int i = tid; i < 2 * p.workers; i += NT) p.first[i] = 0;
        return;
    }
    plan_tokens<NT, PER>(p, a.s, T, sm);
}

// The sum of the values of the threads in front, and of all, by a block of NT threads.
template <int NT>
__device__ long block_before(long n, long *warp_tot, long &all) {
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    long x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();   // the previous call's totals have been read
    if (lane == 31) warp_tot[wp] = x;
    __syncthreads();
    long before = x - n;
    all = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        if (i < wp) before += warp_tot[i];
        all += warp_tot[i];
    }
    return before;
}

// ----------------------------------------------------------------- explicit plan ----
// Which form is cheaper.  Absorbed, a token costs its share of an item, r query rows of up to 128 (or 64, which take as
// long): 0.17 ns a key of its own and as much as 12 r keys more for its queries, a part's beginning and end and its share of
// the join.  Explicit, a request costs the rebuild of its keys, rounded up to whole tiles, 0.3 ns a key and head, once for
// all of its tokens, and a tenth of the absorbed form's time for a token.  So a request goes explicit from 11 r (tiled keys
// + 64) / (6 keys + 72 r) tokens on, at least CHUNK_MIN, where its rows fit in what the requests in front of it left of the
// buffers.  Measured, explicit / absorbed, us: 128 heads, one request of 8192 keys, 192 tokens 384 / 357, 224 385 / 411;
// four of 2048, 96 tokens 373 / 304, 128 375 / 382; 16 of 200, 40 tokens 273 / 226, 56 276 / 292; 16 of none, 32 tokens
// 175 / 217; 64 heads, eight of 2048, 64 tokens 359 / 289, 96 363 / 424; 16 heads, four of 8192, 96 tokens 216 / 209, 128
// 215 / 250; 16 of 2048, 80 tokens 215 / 214, 96 215 / 243; 48 of 200, 40 tokens 125 / 125, 56 131 / 161.
// One block: prefix sums over the requests, then a warp per 128 tokens, then the order of the tiles: in falling order of
// their keys where L2 holds all K_nope and V^T of a shard's heads, which then take turns; else request by request, the
// longest first, so that the tiles of one head and request, which read the same rows, run together.
struct Chunk {
    PagedStep s;
    PagedChunk c;
    int cap, key_rows, heads;   // heads of a shard
    int all_heads;
    int rows;                   // of an item of the absorbed form
};
constexpr int L2_KEYS = (112 << 20) / 512;   // (key, head) pairs whose K_nope and V^T stay in L2 (of 129 MB)

template <int NT>
__global__ void __launch_bounds__(NT) paged_chunk_kernel(const __grid_constant__ Chunk a) {
    __shared__ long warp_tot[NT / 32];
    __shared__ int2 order[CHUNK_SORT];   // a tile's key tiles, its request
    __shared__ int explicit_tokens;
    __shared__ int room[NT];             // a request's need of rows, then its place
    __shared__ long taken;
    const int tid = threadIdx.x, lane = tid & 31, N = a.s.n_tokens;
    pdl_wait();
    pdl_launch_dependents();
    for (int i = tid; i < N; i += NT) a.c.done[i] = 0;
    for (int i = tid; i < a.all_heads; i += NT) a.c.w_max[i] = 0;
    if (tid == 0) explicit_tokens = 0;
    long rows = 0, tiles = 0, rests = 0;
    for (int b0 = 0; b0 < a.s.B; b0 += NT) {
        const int b = b0 + tid;
        int t0 = 0, n = 0, keys = 0;
        if (b < a.s.B) {
            t0 = min(max(a.s.cu[b], 0), N);
            n = min(max(a.s.cu[b + 1], 0), N) - t0;
            keys = min(max(a.s.lens[b], 0), a.cap);
        }
        const long tiled = (keys + 127l) / 128 * 128;
        const bool may = chunk_pays(n, keys, tiled, a.rows);
        const long need = may ? tiled : 0;
        long all, r0 = rows + block_before<NT>(need, warp_tot, all);
        bool fits = may;
        if (rows + all <= a.key_rows) {
            rows += all;
        } else {   // not all of them: in their order, each that fits in what is left
            room[tid] = (int)need;
            __syncthreads();
            if (tid < 32) {
                long at = rows;
                for (int i = lane; i < NT; i += 32) {
                    const int x = room[i];
                    int place = -1;
                    for (unsigned some = __ballot_sync(0xffffffffu, x > 0); some; some &= some - 1) {
                        const int l = __ffs(some) - 1, y = __shfl_sync(0xffffffffu, x, l);
                        if (at + y > a.key_rows) continue;
                        if (l == lane) place = (int)at;
                        at += y;
                    }
                    room[i] = place;
                }
                if (lane == 0) taken = at;
            }
            __syncthreads();
            r0 = room[tid];
            fits = may && r0 >= 0;
            rows = taken;
        }
        const int mine = fits ? (n + 127) / 128 : 0;
        const long e0 = tiles + block_before<NT>(mine, warp_tot, all);
        tiles += all;
        int rest = fits ? (int)min(need / 128, (long)min(n / CHUNK_REST_TOKENS, CHUNK_RESTS)) : 0;
        const long p0 = rests + block_before<NT>(rest, warp_tot, all);
        rests += all;
        if (p0 + rest > a.c.max_rests) rest = 0;   // (only where cu decreases)
        if (b < a.s.B) {
            a.c.key0[b] = fits ? (int)r0 : -1;
            a.c.holes[b] = 0;
            a.c.c_max[b] = 0;
            if (fits) {
                for (int e = 0; e < mine && e0 + e < a.c.max_tiles; ++e) {   // (more only where cu decreases)
                    StepTile x{};
                    x.token = t0 + 128 * e;
                    x.rows = min(128, n - 128 * e);
                    x.key = (int)r0;
                    x.request = b;
                    x.rest = (int)p0 * 128;
                    x.rests = rest;
                    a.c.raw[e0 + e] = x;
                }
                for (int i = 0; i < (int)(need / 128); ++i) {
                    a.c.block_of[r0 / 128 + i] = b;
                    a.c.rest_of[r0 / 128 + i] = i < rest ? (int)p0 + i : -1;
                }
            }
        }
    }
    __syncthreads();
    const int n = (int)min(tiles, (long)a.c.max_tiles);
    const bool sorted = n <= CHUNK_SORT;
    constexpr int AT_ONCE = 3;   // tiles of a warp whose loads are in flight together
    for (int e0 = tid >> 5; e0 < n; e0 += AT_ONCE * (NT / 32)) {
        StepTile x[AT_ONCE];
        int keys[AT_ONCE], pos[AT_ONCE][4];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            x[k].rows = x[k].token = x[k].request = 0;
            if (e0 + k * (NT / 32) < n) x[k] = a.c.raw[e0 + k * (NT / 32)];
        }
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            keys[k] = a.s.lens[x[k].request];
#pragma unroll
            for (int i = 0; i < 4; ++i) pos[k][i] = lane + 32 * i < x[k].rows ? a.s.positions[x[k].token + lane + 32 * i] : -1;
        }
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const int e = e0 + k * (NT / 32);
            if (e >= n) break;
            int most = 0, mine = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = lane + 32 * i, t = x[k].token + r, p = pos[k][i];
                if (r >= x[k].rows) continue;
                const int sees = p < 0 ? 0 : min(min(max(keys[k], 0), a.cap), p == 2147483647 ? p : p + 1);
                a.c.limits[t] = sees;
                if (sees > 0) {
                    a.c.done[t] = 1;
                    ++mine;
                    most = max(most, sees);
                }
            }
            most = __reduce_max_sync(0xffffffffu, most);
            mine = __reduce_add_sync(0xffffffffu, mine);
            if (lane == 0) {
                a.c.raw[e].tiles = (most + 127) / 128;
                atomicAdd(&explicit_tokens, mine);
                if (sorted) order[e] = make_int2((most + 127) / 128, x[k].request);
            }
        }
    }
    __syncthreads();
    // the tiles that have keys here in their order (a step of more than CHUNK_SORT tiles: as they come, heads in turns)
    const bool heaviest = !sorted || rows * a.heads <= L2_KEYS;
    long out = 0;
    for (int base = 0; base < n; base += NT) {
        const int e = base + tid;
        StepTile x{};
        if (e < n) x = a.c.raw[e];
        long all, at = out + block_before<NT>(x.tiles > 0, warp_tot, all);
        out += all;
        if (x.tiles == 0) continue;
        if (sorted && heaviest) {
            at = 0;
            for (int i = 0; i < n; ++i) at += order[i].x > x.tiles || (order[i].x == x.tiles && i < e);
        } else if (sorted) {   // by the request's longest tile, then as they come: a request's tiles are neighbours in raw
            int lo = e, hi = e + 1, most = x.tiles, count = 0, before = 0;
            while (lo > 0 && order[lo - 1].y == x.request) --lo;
            while (hi < n && order[hi].y == x.request) ++hi;
            for (int i = lo; i < hi; ++i) {
                most = max(most, order[i].x);
                count += order[i].x > 0;
                before += i < e && order[i].x > 0;
            }
            at = 0;   // tiles of the requests in front
            for (int i = 0; i < n;) {
                int j = i, m = 0, c = 0;
                for (; j < n && order[j].y == order[i].y; ++j) {
                    m = max(m, order[j].x);
                    c += order[j].x > 0;
                }
                if (m > most || (m == most && i < lo)) at += c;
                i = j;
            }
            x.place = (int)at << 16 | count;
            at += before;
        }
        a.c.tiles[at] = x;
    }
    // the requests' other tokens, eight neighbours a thread
    long listed = 0;
    const int first = min(max(a.s.cu[0], 0), N), last = min(max(a.s.cu[a.s.B], 0), N);
    for (int base = explicit_tokens == last - first ? last : first; base < last; base += 8 * NT) {
        const int t0 = base + 8 * tid;
        int mine = 0;   // (mask)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (t0 + i < last && !a.c.done[t0 + i]) mine |= 1 << i;
        long all;
        int *at = a.c.list + listed + block_before<NT>(__popc(mine), warp_tot, all);
        listed += all;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (mine >> i & 1) *at++ = t0 + i;
    }
    if (tid == 0) {
        a.c.ctl[0] = (int)rows;
        a.c.ctl[1] = (int)out;
        a.c.ctl[2] = (int)listed;
        a.c.ctl[3] = heaviest;
    }
}

// ------------------------------------------------------------------------ gather ----
// A warp per 32 key rows of the explicit requests: the keys' latent rows as they are, their bands in fp16, zeros and no bit
// where there is no key (behind the length, a missing page); a warp per token and 32 heads: the rotated
// band in fp16, as a rounding and its rest; and a warp per eight rows of W_V.  The largest |c| of a request and the largest
// sum |W_V row| of a head bound V, which is held in fp16 times a power of two of theirs (value_shift): bf16 models whose
// values are small or large lose nothing by the form.  Numbers that are not finite do not count: they show in V as they are.
struct Gather {
    PagedDecode p;
    PagedStep s;
    PagedChunk c;
    Divisor by_page;
    Turns64 turns;
};
// Pairs of bf16: |x|, with FINITE 0 for what is not finite; the larger ones of pairs; the sum of a pair
template <bool FINITE>
__device__ __forceinline__ uint32_t magnitudes(uint32_t x) {
    x &= 0x7fff7fffu;
    return FINITE ? x & ~__vcmpgeu2(x, 0x7f807f80u) : x;
}
template <bool FINITE>
__device__ __forceinline__ uint32_t largest(const uint4 (&x)[8][2]) {
    uint32_t m[4] = {};
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const uint4 &v = x[e >> 1][e & 1];
        m[0] = __vmaxu2(m[0], magnitudes<FINITE>(v.x));
        m[1] = __vmaxu2(m[1], magnitudes<FINITE>(v.y));
        m[2] = __vmaxu2(m[2], magnitudes<FINITE>(v.z));
        m[3] = __vmaxu2(m[3], magnitudes<FINITE>(v.w));
    }
    return __vmaxu2(__vmaxu2(m[0], m[1]), __vmaxu2(m[2], m[3]));
}
// The largest sum of magnitudes of the warp's eight rows of 512; NaN where one of them is NaN
template <bool FINITE>
__device__ __forceinline__ float largest_sum(const uint4 (&x)[8][2]) {
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const uint32_t w[8] = {x[r][0].x, x[r][0].y, x[r][0].z, x[r][0].w, x[r][1].x, x[r][1].y, x[r][1].z, x[r][1].w};
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t m = magnitudes<FINITE>(w[e]);
            sum[0] += __uint_as_float(m << 16);
            sum[1] += __uint_as_float(m & 0xffff0000u);
        }
        const float all = warp_sum(sum[0] + sum[1]);
        top = max(top, __float_as_uint(all));   // (as integers: NaN the largest)
    }
    return __uint_as_float(top);
}
__device__ __forceinline__ uint32_t half_pair(uint32_t bf) {   // two bf16 as two fp16
    const __half2 h = __floats2half2_rn(__uint_as_float(bf << 16), __uint_as_float(bf & 0xffff0000u));
    return *(const uint32_t *)&h;
}

__global__ void __launch_bounds__(256) paged_gather_kernel(const __grid_constant__ Gather a) {
    const PagedDecode &p = a.p;
    const int lane = threadIdx.x & 31, warps = gridDim.x * 8;
    pdl_wait();
    pdl_launch_dependents();
    const int R = __ldcg(a.c.ctl) / 32, per = (p.H + 31) / 32;
    if (R == 0) return;
    const long heads = R + (long)a.s.n_tokens * per, total = heads + p.H * 16l;
#pragma unroll 1
    for (long u = blockIdx.x * 8 + (threadIdx.x >> 5); u < total; u += warps) {
        if (u < R) {
            const int r0 = (int)u * 32, b = a.c.block_of[r0 / 128];
            const int keys = min(max(a.s.lens[b], 0), p.max_pages * p.page), key = r0 - a.c.key0[b] + lane;
            int row = -1;
            if (key < keys) {
                const int col = quotient(a.by_page, key), id = p.table[(long)b * p.max_pages + col];
                if ((unsigned)id < (unsigned)p.num_pages) row = id * p.page + (key - col * p.page);
            }
            const unsigned held = __ballot_sync(0xffffffffu, row >= 0);
            if (lane == 0) {
                a.c.held[u] = held;
                if (held != (keys - key >= 32 ? 0xffffffffu : keys > key ? (1u << (keys - key)) - 1 : 0u)) a.c.holes[b] = 1;
            }
            const uint4 zero = make_uint4(0, 0, 0, 0);
            uint32_t most = 0;
#pragma unroll 1
            for (int r = 0; r < 32; r += 8) {
                uint4 x[8][2], y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int from = __shfl_sync(0xffffffffu, row, r + e);
                    const uint4 *c = (const uint4 *)p.c_cache + (long)from * 64, *k = (const uint4 *)p.kpe_cache + (long)from * 8;
                    x[e][0] = from >= 0 ? __ldcg(c + lane) : zero;
                    x[e][1] = from >= 0 ? __ldcg(c + lane + 32) : zero;
                    y[e] = from >= 0 && lane < 8 ? __ldcg(k + lane) : zero;
                }
                uint32_t here = largest<false>(x);
                if (__vcmpgeu2(here, 0x7f807f80u)) here = largest<true>(x);   // (seldom)
                most = __vmaxu2(most, here);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    uint4 *c = (uint4 *)a.c.chat + (long)(r0 + r + e) * 64;
                    c[lane] = x[e][0];
                    c[lane + 32] = x[e][1];
                    if (lane < 8)
                        ((uint4 *)a.c.kpe)[(long)(r0 + r + e) * 8 + lane] =
                            make_uint4(half_pair(y[e].x), half_pair(y[e].y), half_pair(y[e].z), half_pair(y[e].w));
                }
            }
            most = __reduce_max_sync(0xffffffffu, max(most & 0xffff, most >> 16));
            if (lane == 0) atomicMax(a.c.c_max + b, most << 16);
        } else if (u >= heads) {
            const long row = (u - heads) * 8;   // of all heads' W_V
            const int h = (int)(row / 128);
            const uint4 *w = (const uint4 *)p.w + ((long)h * 256 + 128 + row % 128) * 64;
            uint4 x[8][2];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e >> 1][e & 1] = __ldcg(w + (e >> 1) * 64 + (e & 1) * 32 + lane);
            float top = largest_sum<false>(x);
            if (!(top <= 3e38f)) top = fminf(largest_sum<true>(x), 3e38f);   // (seldom; the same in all lanes)
            if (lane == 0) atomicMax(a.c.w_max + h, __float_as_uint(top));
        } else {
            const long i = u - R;
            const int t = (int)(i / per), h0 = (int)(i % per) * 32, h1 = min(h0 + 32, p.H);
            if (!a.c.done[t]) continue;
            const float2 cs = turn_cs(a.turns.v[lane], a.s.positions[t]);
#pragma unroll 1
            for (int h = h0; h < h1; h += 8) {
                uint16_t x0[8], x1[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint16_t *x = (const uint16_t *)p.q_pe + ((long)t * p.H + min(h + j, h1 - 1)) * 64 + lane;
                    x0[j] = x[0];
                    x1[j] = x[32];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (h + j >= h1) break;
                    const float f0 = __uint_as_float((uint32_t)x0[j] << 16), f1 = __uint_as_float((uint32_t)x1[j] << 16);
                    __half *y = (__half *)a.c.qpe + ((long)t * p.H + h + j) * 128 + lane;
                    const float r0 = f0 * cs.x - f1 * cs.y, r1 = f1 * cs.x + f0 * cs.y;
                    const __half h0r = __float2half_rn(r0), h1r = __float2half_rn(r1);
                    y[0] = h0r;
                    y[32] = h1r;
                    y[64] = __float2half_rn(r0 - __half2float(h0r));
                    y[96] = __float2half_rn(r1 - __half2float(h1r));
                }
            }
        }
    }
}

}  // namespace

// n tokens of one request take at most f(n) rows: whole tiles t <= L, L a row of the table, with
// t (11 rows - 6 n) <= rows (72 n - 704).  Up to L that is a convex function, below 0 at 0, so while no request can have a
// whole row of the table, all tokens in one request take the most; else no token brings more rows than the largest f(n) / n.
long chunk_most_rows(int B, int n_tokens, long cap, int rows) {
    const long L = (cap + 127) / 128 * 128, r = rows;
    auto most = [&](long n) {
        if (n < CHUNK_MIN) return 0l;
        const long num = r * (72 * n - 704), den = 11 * r - 6 * n;
        return den <= 0 ? L : std::min(L, num / den / 128 * 128);
    };
    const long requests = std::min((long)B, (long)n_tokens / CHUNK_MIN);
    long whole = CHUNK_MIN;   // tokens that may have a whole row of the table
    while (most(whole) < L) ++whole;
    if (n_tokens < whole) return requests > 0 ? most(n_tokens) : 0;
    long top = 0, by = 1;   // the largest f(n) / n
    for (long n = CHUNK_MIN; n <= whole; ++n)
        if (most(n) * by > top * n) {
            top = most(n);
            by = n;
        }
    return std::min(requests * L, (n_tokens * top + by - 1) / by);
}

cudaError_t launch_paged_chunk(const PagedDecode &p, const PagedStep &s, const PagedChunk &c, cudaStream_t st) {
    cudaError_t e;
    {
        const Chunk a{s, c, p.max_pages * p.page, c.key_rows, c.heads, p.H, chunk_item_rows(p)};
        ProfScope ps("paged_chunk", st);
        const bool few = s.n_tokens <= 2048 && s.B <= 256;   // few warps come together sooner
        auto kern = few ? paged_chunk_kernel<256> : paged_chunk_kernel<PNT>;
        if ((e = launch_after(kern, 1, few ? 256 : PNT, 0, st, a)) != cudaSuccess) return e;
    }
    Gather g{p, s, c, divisor(p.page), {}};
    std::copy_n(paged_turns(p.base, p.Dr), 32, g.turns.v);
    ProfScope ps("paged_gather", st);
    return launch_after(paged_gather_kernel, 152 * 4, 256, 0, st, g);
}

cudaError_t launch_paged_plan(const PagedDecode &p, const PagedPlan &s, cudaStream_t st) {
    const Plan a{p, s};
    const unsigned nt = p.T <= SOME ? SOME : PNT;
    auto kern = nt == SOME ? paged_plan_kernel<SOME, 1> : paged_plan_kernel<PNT, PAGED_ROUND / PNT>;
    const size_t sm = plan_ints(nt == SOME ? SOME : PAGED_ROUND, s.s.B) * sizeof(int);
    if (sm > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
        if (e != cudaSuccess) return e;
    }
    ProfScope ps("paged_plan", st);
    return launch_after(kern, 1 + (unsigned)std::min((s.n_zero + nt - 1) / nt, 150l), nt, sm, st, a);
}

}  // namespace mla
