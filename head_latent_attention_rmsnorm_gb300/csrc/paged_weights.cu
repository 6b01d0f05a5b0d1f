// paged_weights.cu -- the attention weight that a step's tokens gave each page of their requests.
//
// Mathematics, per request and page c: w_c = prior_c + sum over the request's tokens t of the step, heads h and the
// page's keys j that t sees of exp(s_tjh - lse_th), s_tjh = scale (q_th . c_j + rot(q_pe_th, p_t) . kpe_j) with the
// absorbed query q_th = W_K(h)^T q_nope_th; lse as the attention call returned it.  One pass over the cache, no
// maximum: the log-sum-exp is known.  Launches: plan and absorb as for the attention of a step, the
// weights, a last one that rounds to fp32.
//
// Sums.  A page's sum meets in a 64-bit fixed-point number (integer additions have no order, so the bits
// do not depend on timing), with as many bits behind the point as n_tokens H page weights of 2 leave.  A weight is
// cut to [0, 2]; NaN counts as 0.
//
// Tensor cores (bf16, 512 + 64 dims, pages of a multiple of eight).  Persistent clusters of two CTAs walk equal
// shares of all items' tiles of 256 keys, cta_group::2 MMAs: S = K Q^T with the keys as the 256 rows
// (128 in each SM), and Q's bf16 high halves as the columns that CTA 0 holds, its low halves those of CTA 1:
// N = 2 x rows.  So a key is loaded by one SM only, the scores are exact to the queries' 2^-17, and a
// key's weights of all rows lie in one thread's TMEM lane: their sum needs no exchange.  Per CTA: three warps that
// load the keys' 64-dim blocks (16 KB a stage) in turns, one that loads the queries, four that take the exponentials; CTA
// 0's second warp issues the MMAs.
//
// What bounds it.  64 ragged requests of up to 32768 keys, 128 heads: 218 us, 6.2 TB/s, 0.92 of a copy's rate; 8 requests'
// last 32 tokens over 8192 keys, 16 heads: 48 us, 3.4 us a tile, in which the tensor pipes are busy 2.2 (their operands,
// from L2, come in stages of which five are in flight).  What it took: no L2 prefetch (asking for tiles one to five
// ahead, by bulk copies or line by line, cost 0.1-0.17 ms of the first case), three loading warps (one issues
// the boxes of 16-row pages too slowly: 76 us for the second case, 55 with three), five stages (238 us with four).
// Eight warps for the exponentials gained 2 us of the second case and cost 7 of the first.
#include <cuda_bf16.h>

#include <algorithm>

#include "paged_common.cuh"
#include "tc_common.cuh"
#include "tc_internal.h"

namespace mla {

__device__ unsigned g_paged_weights_err = 0;

namespace {

using namespace paged;
using namespace tc;
using bf16 = __nv_bfloat16;

constexpr unsigned FULL = 0xffffffffu;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A weight as it is counted.
__device__ __forceinline__ float counted(float w) { return w > 0.f ? fminf(w, 2.f) : 0.f; }

__device__ __forceinline__ void add_fixed(unsigned long long *at, float x, float one) {
    atomicAdd(at, (unsigned long long)__float2ll_rn(x * one));
}

// ------------------------------------------------------------------- tensor cores ----
constexpr int DK = 512, DR = 64;
constexpr int ROWS = 128, KT = 128;                // query rows of an item, keys of a CTA's half of a tile
constexpr int BLOCKS = (DK + DR) / 64, STAGES = 5;
constexpr uint32_t BLK = 128 * 128;                // 128 rows of 64 dims
// warps: 0, 7, 8 load keys, 1 issues, 2-5 weigh, 6 loads queries
constexpr int LOADERS = 3, NTHREADS = 32 * (6 + LOADERS);
constexpr uint32_t OFF_K = BLOCKS * BLK, OFF_ROW = OFF_K + STAGES * BLK, OFF_BAR = OFF_ROW + 2 * ROWS * 8 + 64;
constexpr uint32_t W_SMEM = OFF_BAR + 256;
static_assert(W_SMEM <= 232448, "shared memory budget");
enum : int {
    B_FULL = 0,                   // leader [stage]: both CTAs' block landed
    B_EMPTY = B_FULL + STAGES,    // both [stage]: read by the MMAs
    B_QFULL = B_EMPTY + STAGES,   // leader: both CTAs' queries landed
    B_QFREE = B_QFULL + 1,        // both: read by the part's MMAs
    B_SFULL = B_QFREE + 1,        // both [buffer]: scores done
    B_SFREE = B_SFULL + 2,        // leader [buffer]: read by both CTAs' warps
    B_COUNT = B_SFREE + 2
};

__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *m, uint32_t bar_cluster, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4}], [%2];" ::"r"(smem_u32(dst)),
        "l"((uint64_t)m), "r"(bar_cluster), "r"(c0), "r"(c1)
        : "memory");
}

struct WMaps {
    CUtensorMap c, r;          // a unit's rows, 64 dims
    CUtensorMap q[2], qr[2];   // query rows of 64 dims: hi, lo
};
struct Weights {
    PagedDecode p;
    Divisor by_page;
    const float *lse;            // [T H]
    unsigned long long *acc;     // [requests][max_pages]
    float scale_log2, one;       // one: 2^bits behind the point
};

__device__ __forceinline__ int row_of(const Weights &a, const PagedPart &w, int key) {
    if (key >= w.keys) return -1;
    const int col = quotient(a.by_page, key);
    const int id = __ldg(a.p.table + (long)w.row * a.p.max_pages + col);
    return (unsigned)id < (unsigned)a.p.num_pages ? id * a.p.page + (key - col * a.p.page) : -1;
}

template <int UNIT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NTHREADS, 1)
    paged_weights_tc_kernel(const __grid_constant__ WMaps m, const __grid_constant__ Weights a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {   // no room to align by hand; the same answer in every CTA
        if (threadIdx.x == 0) atomicOr(&g_paged_weights_err, 2u);
        return;
    }
    constexpr int UNITS = KT / UNIT;
    float *row_lse = (float *)(smem + OFF_ROW);    // [part parity][row]: log-sum-exp in log2 units
    int *row_lim = (int *)(row_lse + 2 * ROWS);    // keys that the row sees, 0 for none
    int *least = row_lim + 2 * ROWS;               // [part parity][warp]: the least of them
    uint64_t *bars = (uint64_t *)(smem + OFF_BAR);
    uint32_t *tslot = (uint32_t *)(bars + B_COUNT);
    volatile int *abort = (volatile int *)(tslot + 1);
    const PagedDecode &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();

    if (tid == 0) {
        for (int i = 0; i < B_COUNT; ++i) mbar_init(&bars[i], i >= B_SFREE ? 8 : 1);
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tslot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers and TMEM exist before any cross-CTA traffic
    tc_fence_after();
    const uint32_t tmem = *tslot;
    pdl_wait();
    pdl_launch_dependents();

    const PagedPart *part = p.parts + __ldcg(p.first + (blockIdx.x >> 1));
    bool more = __ldcg(p.first + p.workers + (blockIdx.x >> 1)) > 0;
    PagedPart w{};
    auto load = [&]() {
        const int4 x = __ldcg((const int4 *)part), y = __ldcg((const int4 *)part + 1);
        w.row = x.x;
        w.q = x.y;
        w.k0 = x.z;
        w.nt = x.w;
        w.keys = y.x;
        w.next = y.y;
        w.rows = y.z;
    };
    if (more) load();
    auto next = [&]() {
        more = w.next > 0;
        part += w.next;
        if (more) load();
    };
    auto wait = [&](int i, uint32_t parity) { return mbar_wait(&bars[i], parity, abort, &g_paged_weights_err); };
    auto wait_pair = [&](int i, uint32_t parity) { return mbar_wait_cluster(&bars[i], parity, abort, &g_paged_weights_err); };

    if (warp == 0 || warp >= 7) {
        // ------------------------------------------------------------ the keys' blocks in turns, a lane per unit
        const uint32_t full0 = map_peer(smem_u32(&bars[B_FULL]), 0);
        const int none = p.num_pages * p.page;   // a row outside the cache: zeros
        const int me = warp == 0 ? 0 : warp - 6;
        int it = 0;
        bool go = true;
        for (; more && go; next()) {
            const int key0 = (int)rank * KT + lane * UNIT;   // of the lane's unit in a tile
            int ahead = lane < UNITS ? row_of(a, w, w.k0 * 2 * KT + key0) : -1;
            for (int i = 0; i < w.nt && go; ++i) {
                const int row = ahead >= 0 ? ahead : none;
                if (i + 1 < w.nt && lane < UNITS) ahead = row_of(a, w, (w.k0 + i + 1) * 2 * KT + key0);
#pragma unroll 1
                for (int j = 0; j < BLOCKS; ++j, ++it) {
                    if (it % LOADERS != me) continue;
                    const int s = it % STAGES;
                    go = __all_sync(FULL, wait_pair(B_EMPTY + s, ((it / STAGES) & 1) ^ 1));   // (passes at first)
                    if (!go) break;
                    if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&bars[B_FULL + s], 2 * BLK);
                    __syncwarp();
                    if (lane < UNITS) {
                        uint8_t *dst = smem + OFF_K + s * BLK + lane * UNIT * 128;
                        if (j < DK / 64) tma_load_2d_pair(dst, &m.c, full0 + s * 8, 64 * j, row);
                        else tma_load_2d_pair(dst, &m.r, full0 + s * 8, 0, row);
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp == 6) {
        // ------------------------------------------------------------ a part's queries: hi here, lo in the peer
        const uint32_t full0 = map_peer(smem_u32(&bars[B_QFULL]), 0);
        int seg = 0;
        bool go = lane == 0;
        for (; more && go; next(), ++seg) {
            go = wait_pair(B_QFREE, (seg & 1) ^ 1);   // (passes at first)
            if (!go) break;
            if (rank == 0) mbar_arrive_expect_tx(&bars[B_QFULL], 2 * BLOCKS * BLK);
#pragma unroll 1
            for (int j = 0; j < BLOCKS; ++j)
                tma_load_2d_pair(smem + j * BLK, j < DK / 64 ? &m.q[rank] : &m.qr[rank], full0, j < DK / 64 ? 64 * j : 0, w.q);
        }
    } else if (warp == 1 && rank == 0) {
        // ------------------------------------------------------------ S = K Q^T
        int it = 0, n = 0, seg = 0;
        bool ok = true;
        for (; more && ok; next(), ++seg) {
            const uint32_t cols = (w.rows + 7) / 8 * 8;
            const uint32_t idesc = idesc_f16(256, 0, false) | ((2 * cols) >> 3) << 17;
            ok = __all_sync(FULL, wait(B_QFULL, seg & 1));
#pragma unroll 1
            for (int i = 0; i < w.nt && ok; ++i, ++n) {
                const int buf = n & 1;
                ok = __all_sync(FULL, wait_pair(B_SFREE + buf, ((n >> 1) & 1) ^ 1));   // (passes at first)
#pragma unroll 1
                for (int j = 0; j < BLOCKS && ok; ++j, ++it) {
                    const int s = it % STAGES;
                    ok = __all_sync(FULL, wait(B_FULL + s, (it / STAGES) & 1));
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t k = sdesc_kmajor(smem + OFF_K + s * BLK), q = sdesc_kmajor(smem + j * BLK);
#pragma unroll
                        for (int e = 0; e < 4; ++e) mma_ss_pair(tmem + buf * 256, k + 2 * e, q + 2 * e, idesc, (j | e) != 0);
                        mma_commit_pair(&bars[B_EMPTY + s], 3);
                        if (j == BLOCKS - 1) mma_commit_pair(&bars[B_SFULL + buf], 3);
                    }
                    __syncwarp();
                }
            }
            if (ok && w.next > 0 && elect_one()) mma_commit_pair(&bars[B_QFREE], 3);   // (the peer has left after the last)
            __syncwarp();
        }
    } else if (warp >= 2 && warp < 6) {
        // ------------------------------------------------------------ weights: a thread per key
        const int quad = warp & 3, row = quad * 32 + lane;
        const uint32_t free0 = map_peer(smem_u32(&bars[B_SFREE]), 0);
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        int n = 0, seg = 0;
        bool ok = true;   // an abandoned wait clears it; the walk goes on without waiting
        for (; more; next(), ++seg) {
            float *lse2 = row_lse + (seg & 1) * ROWS;
            int *lim = row_lim + (seg & 1) * ROWS;
            {
                float x = 0.f;
                int l = 0;
                if (row < w.rows) {
                    x = __ldg(a.lse + w.q + row) * 1.4426950408889634f;
                    l = __ldcg(p.limits + (w.q + row) / p.H);
                    if (x == -INFINITY) l = 0;   // saw no key
                }
                lse2[row] = x;
                lim[row] = l;
                const int low = __reduce_min_sync(FULL, row < (w.rows + 31) / 32 * 32 ? l : 2147483647);
                if (lane == 0) least[(seg & 1) * 4 + quad] = low;
            }
            named_bar_sync(1, 128);   // (a part's numbers are read before its successor's barrier, written behind that)
            const int *lo = least + (seg & 1) * 4;
            const int all_see = min(min(lo[0], lo[1]), min(lo[2], lo[3]));
            const int cols = (w.rows + 7) / 8 * 8;
#pragma unroll 1
            for (int i = 0; i < w.nt; ++i, ++n) {
                const int buf = n & 1, end = ((w.k0 + i) * 2 + (int)rank + 1) * KT, key = end - KT + row;
                const bool held = row_of(a, w, key) >= 0;
                const int col = held ? quotient(a.by_page, key) : 0;
                ok = __all_sync(FULL, ok && wait(B_SFULL + buf, (n >> 1) & 1));
                tc_fence_after();
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                for (int r0 = 0; r0 < w.rows; r0 += 32) {
                    uint32_t hi[32], low[32];
                    tmem_ld32_wait(lanes + buf * 256 + r0, hi);
                    tmem_ld32_wait(lanes + buf * 256 + cols + r0, low);
                    if (end <= all_see) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 z = *(const float4 *)(lse2 + r0 + e);
                            const float zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                sum[q] += counted(ex2(fmaf(__uint_as_float(hi[e + q]) + __uint_as_float(low[e + q]), a.scale_log2, -zs[q])));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 z = *(const float4 *)(lse2 + r0 + e);
                            const int4 l = *(const int4 *)(lim + r0 + e);
                            const float zs[4] = {z.x, z.y, z.z, z.w};
                            const int ls[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const float x = counted(ex2(fmaf(__uint_as_float(hi[e + q]) + __uint_as_float(low[e + q]), a.scale_log2, -zs[q])));
                                sum[q] += key < ls[q] ? x : 0.f;
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_peer(free0 + buf * 8);
                // the keys of a unit of up to 32 share a page
                constexpr int SHARE = UNIT < 32 ? UNIT : 32;
                float x = held ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : 0.f;
#pragma unroll
                for (int o = SHARE / 2; o > 0; o >>= 1) x += __shfl_xor_sync(FULL, x, o);
                if (ok && held && lane % SHARE == 0 && x > 0.f) add_fixed(a.acc + (long)w.row * p.max_pages + col, x, a.one);
            }
        }
    }
    __syncwarp();
    if (tid == 0 && *abort) settle();
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // the leader's MMAs read this CTA's shared memory until here
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

cudaError_t weights_tc(const PagedDecode &p, const float *lse, unsigned long long *acc, float one, cudaStream_t st) {
    using ull = unsigned long long;
    cudaError_t e;
    const ull rows = (ull)p.num_pages * p.page, heads = (ull)p.T * p.H;
    int unit = 64;   // rows that always share a page: the largest power of two up to 64 that divides one
    while (p.page % unit) unit /= 2;
    WMaps m{};
    {
        const ull d[2] = {DK, rows}, s[1] = {DK * 2}, dr[2] = {DR, rows}, sr[1] = {DR * 2};
        const unsigned b[2] = {64, (unsigned)unit};
        if ((e = make_tma_map(&m.c, p.c_cache, 2, d, s, b)) != cudaSuccess) return e;
        if ((e = make_tma_map(&m.r, p.kpe_cache, 2, dr, sr, b)) != cudaSuccess) return e;
        const ull dq[2] = {DK, heads}, dqr[2] = {DR, heads};
        const unsigned bq[2] = {64, ROWS};
        const bf16 *q = (const bf16 *)p.qabs, *qr = (const bf16 *)p.qpe;   // hi, then lo
        for (int i = 0; i < 2; ++i) {
            if ((e = make_tma_map(&m.q[i], q + i * heads * DK, 2, dq, s, bq)) != cudaSuccess) return e;
            if ((e = make_tma_map(&m.qr[i], qr + i * heads * DR, 2, dqr, sr, bq)) != cudaSuccess) return e;
        }
    }
    const Weights a{p, divisor(p.page), lse, acc, p.scale * 1.4426950408889634f, one};
    auto kern = unit == 64   ? paged_weights_tc_kernel<64>
                : unit == 32 ? paged_weights_tc_kernel<32>
                : unit == 16 ? paged_weights_tc_kernel<16>
                             : paged_weights_tc_kernel<8>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)W_SMEM)) != cudaSuccess) return e;
    ProfScope ps("paged_weights", st);
    return launch_after(kern, 2 * (unsigned)p.workers, NTHREADS, W_SMEM, st, m, a);
}

// --------------------------------------------------------------------- CUDA cores ----
// fp32, and bf16 of other dims or pages: a block walks its share of the tiles of 32 keys; queries and keys as fp32 in
// shared memory, a lane per key, two of the item's 16 rows a warp.
constexpr int SNT = 256, SROWS = 16, SKEYS = 32;
__host__ __device__ inline int pitch_of(int Dq) { return (Dq + 3) / 4 * 4 + 4; }   // rows four banks apart

template <typename T>
__global__ void __launch_bounds__(SNT) paged_weights_simt_kernel(const __grid_constant__ Weights a) {
    extern __shared__ float sm[];
    __shared__ float sum[SNT / 32][SKEYS], lse[SROWS];
    __shared__ int lim[SROWS], src[SKEYS], cols[SKEYS];
    const PagedDecode &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, Dq = p.Dk + p.Dr, pitch = pitch_of(Dq);
    float *sq = sm, *sk = sm + SROWS * pitch;
    pdl_launch_dependents();
    pdl_wait();
    const long total = p.tile_off[p.B] * p.row_tiles, q = share_of(p, total);
    long t = blockIdx.x * q;
    const long tend = min(t + q, total);
    while (t < tend) {
        const int b = request_of(p, p.tile_off, t);
        const long first = p.tile_off[b], per = p.tile_off[b + 1] - first, in = t - first * p.row_tiles;
        const int rt = (int)(in / per), keys = keys_of(p, b);
        const long k0 = in % per, k1 = min(per, k0 + tend - t);
        const int4 g = p.groups[b];
        const int q0 = g.y + rt * SROWS, rows = min(SROWS, g.z - rt * SROWS);
        __syncthreads();
        for (int i = tid; i < SROWS * pitch; i += SNT) {
            const int r = i / pitch, d = i % pitch;
            float v = 0.f;
            if (r < rows && d < Dq)
                v = d < p.Dk ? ((const float *)p.qabs)[(long)(q0 + r) * p.Dk + d] : ((const float *)p.qpe)[(long)(q0 + r) * p.Dr + d - p.Dk];
            sq[i] = v;
        }
        if (tid < SROWS) {
            const float x = tid < rows ? a.lse[q0 + tid] : -INFINITY;
            lse[tid] = x;
            lim[tid] = x == -INFINITY ? 0 : p.limits[(q0 + tid) / p.H];
        }
        for (long kt = k0; kt < k1; ++kt) {
            __syncthreads();   // the previous tile has been read
            if (tid < SKEYS) {
                const int key = (int)(kt * SKEYS) + tid;
                int row = -1, col = 0;
                if (key < keys) {
                    col = quotient(a.by_page, key);
                    const int id = p.table[(long)g.x * p.max_pages + col];
                    if ((unsigned)id < (unsigned)p.num_pages) row = id * p.page + (key - col * p.page);
                }
                src[tid] = row;
                cols[tid] = col;
            }
            __syncthreads();
            for (int k = warp; k < SKEYS; k += SNT / 32) {
                const int row = src[k];
                const T *c = (const T *)p.c_cache + (long)row * p.Dk, *r = (const T *)p.kpe_cache + (long)row * p.Dr;
                for (int d = lane; d < pitch; d += 32) sk[k * pitch + d] = row < 0 || d >= Dq ? 0.f : d < p.Dk ? to_f<T>(c[d]) : to_f<T>(r[d - p.Dk]);
            }
            __syncthreads();
            const int r0 = 2 * warp, key = (int)(kt * SKEYS) + lane;
            float x[2] = {0.f, 0.f};
            for (int d = 0; d < Dq; d += 4) {
                const float4 k = *(const float4 *)(sk + lane * pitch + d);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float4 v = *(const float4 *)(sq + (r0 + e) * pitch + d);
                    x[e] = fmaf(v.x, k.x, fmaf(v.y, k.y, fmaf(v.z, k.z, fmaf(v.w, k.w, x[e]))));
                }
            }
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float wgt = counted(expf(x[e] * p.scale - lse[r0 + e]));
                if (src[lane] >= 0 && key < lim[r0 + e]) s += wgt;
            }
            sum[warp][lane] = s;
            __syncthreads();
            if (warp == 0 && src[lane] >= 0) {
                float all = 0.f;
#pragma unroll
                for (int i = 0; i < SNT / 32; ++i) all += sum[i][lane];
                if (all > 0.f) add_fixed(a.acc + (long)g.x * p.max_pages + cols[lane], all, a.one);
            }
        }
        t += k1 - k0;
    }
}

template <typename T>
cudaError_t weights_simt(const PagedDecode &p, const float *lse, unsigned long long *acc, float one, cudaStream_t st) {
    const Weights a{p, divisor(p.page), lse, acc, 0.f, one};
    const size_t sm = (size_t)(SROWS + SKEYS) * pitch_of(p.Dk + p.Dr) * 4;
    const cudaError_t e = cudaFuncSetAttribute(paged_weights_simt_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
    if (e != cudaSuccess) return e;
    ProfScope ps("paged_weights", st);
    return launch_after(paged_weights_simt_kernel<T>, (unsigned)p.workers, SNT, sm, st, a);
}

// out = prior + the sums
__global__ void __launch_bounds__(256) paged_weights_out_kernel(long n, const unsigned long long *acc, double unit, const float *prior, float *out) {
    pdl_wait();
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256)
        out[i] = (float)((double)(long long)acc[i] * unit + (prior ? (double)prior[i] : 0.0));
}

}  // namespace

cudaError_t launch_paged_weights(const PagedDecode &p, const float *lse, unsigned long long *acc, int bits, cudaStream_t st) {
    const float one = ldexpf(1.f, bits);
    if (p.tc) return weights_tc(p, lse, acc, one, st);
    return p.ty == TY_F32 ? weights_simt<float>(p, lse, acc, one, st) : weights_simt<bf16>(p, lse, acc, one, st);
}

cudaError_t launch_paged_weights_out(long n, const unsigned long long *acc, int bits, const float *prior, float *out, cudaStream_t st) {
    ProfScope ps("paged_weights_out", st);
    return launch_after(paged_weights_out_kernel, (unsigned)std::min((n + 255) / 256, 1216l), 256, 0, st, n, acc, ldexp(1.0, -bits), prior, out);
}

cudaError_t paged_weights_read_and_clear_error(unsigned *flags, cudaStream_t st) {
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_paged_weights_err, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
    if (e != cudaSuccess) return e;
    if ((e = cudaStreamSynchronize(st)) != cudaSuccess) return e;
    if (v) {
        unsigned z = 0;
        e = cudaMemcpyToSymbolAsync(g_paged_weights_err, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
        if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    }
    *flags |= v;
    return e;
}

}  // namespace mla
