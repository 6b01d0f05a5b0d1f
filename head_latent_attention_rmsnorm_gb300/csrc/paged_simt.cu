// paged_simt.cu -- one-token decode over the paged latent cache on the CUDA cores: fp32, and bf16
// at dimensions or page sizes that the tensor-core kernels do not take.  fp32 arithmetic.
//
// Three launches: absorb (q_abs = W_K^T q_nope, the query's rotation, the division of the batch
// among the workers), attention (each worker walks its key tiles with the running maximum and sum
// of the softmax and writes one normalised partial per request it met), join (the partials'
// log-sum-exp merge and out = W_V o), each launched early.  16 heads of 512 + 64 dims, fp32: 4
// ragged requests of up to 1000 keys 23.5 us (one tile per worker: three launches' latency; 46 before the
// loads of queries, tiles, parts and W_V went out together), 16 requests of 3000 keys 101 us: 8 us a
// tile, in which shared-memory reads take about twice the time of the 557 thousand multiply-adds.  512
// threads take 8.8 us a tile (registers for the next tile's loads run out), the same otherwise.
#include <algorithm>

#include "paged_common.cuh"
#include "tc_common.cuh"

namespace mla {
namespace {

using namespace paged;
using tc::pdl_launch_dependents;
using tc::pdl_wait;

constexpr int NT = 256;         // threads
constexpr int HT = 16;          // heads per work item
constexpr int KT = 32;          // keys per tile
constexpr int DK_MAX = 512, DQ_MAX = 640;
constexpr int BT = 4;           // requests per block of the two weight products
constexpr int DC = 128;         // latent dims of an absorb block
constexpr int VC = 32;          // value dims of a join block

// ------------------------------------------------------------------------ absorb ----
// Block (head, DC latent dims, group of BT requests): the warps share out the rows of W_K(h), a lane
// holds four dims 32 apart, and the warps' sums meet in shared memory.  The grid is cut that fine
// because few heads over few requests are a matter of latency: every weight load of a block is in
// flight at once.  One block more forms the tile prefix sums.
template <typename T>
__global__ void __launch_bounds__(NT) paged_absorb_simt_kernel(const __grid_constant__ PagedDecode p,
                                                               const __grid_constant__ Turns turns) {
    extern __shared__ float sm[];   // q [BT][Dn], sums [8 warps][BT][DC]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int groups = (p.B + BT - 1) / BT, chunks = (p.Dk + DC - 1) / DC;
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == 0) {
        plan_block<NT>(p);
        return;
    }
    int u = blockIdx.x - 1;
    const int ch = u % chunks;
    u /= chunks;
    const int h = u / groups, b0 = (u % groups) * BT, nb = min(BT, p.B - b0), d0 = ch * DC;
    for (int i = tid; i < BT * p.Dn; i += NT) {
        const int j = i / p.Dn, n = i % p.Dn;
        sm[i] = j < nb ? to_f<T>(((const T *)p.q_nope)[((long)(b0 + j) * p.H + h) * p.Dn + n]) : 0.f;
    }
    if (ch == 0) {   // the query sits at its request's last key
        const int half = p.Dr / 2;
        for (int i = tid; i < nb * half; i += NT) {
            const int j = i / half, t = i % half;
            const long row = (long)(b0 + j) * p.H + h;
            const float2 cs = turn_cs(turns.v[t], keys_of(p, b0 + j) - 1);
            const T *x = (const T *)p.q_pe + row * p.Dr;
            const float x0 = to_f<T>(x[t]), x1 = to_f<T>(x[t + half]);
            float *y = (float *)p.qpe + row * p.Dr;
            y[t] = x0 * cs.x - x1 * cs.y;
            y[t + half] = x1 * cs.x + x0 * cs.y;
        }
    }
    __syncthreads();
    const T *w = (const T *)p.w + (long)h * (p.Dn + p.Dv) * p.Dk + d0 + lane;
    float acc[BT][4] = {};
#pragma unroll 8
    for (int n = warp; n < p.Dn; n += NT / 32) {
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = d0 + lane + 32 * k < p.Dk ? to_f<T>(w[(long)n * p.Dk + 32 * k]) : 0.f;
#pragma unroll
        for (int j = 0; j < BT; ++j) {
            const float q = sm[j * p.Dn + n];
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[j][k] = fmaf(v[k], q, acc[j][k]);
        }
    }
    float *sum = sm + BT * p.Dn;
#pragma unroll
    for (int j = 0; j < BT; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[(warp * BT + j) * DC + lane + 32 * k] = acc[j][k];
    __syncthreads();
    for (int i = tid; i < BT * DC; i += NT) {
        const int j = i / DC, d = i % DC;
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < NT / 32; ++k) x += sum[(k * BT + j) * DC + d];
        if (j < nb && d0 + d < p.Dk) ((float *)p.qabs)[((long)(b0 + j) * p.H + h) * p.Dk + d0 + d] = x;
    }
}

// --------------------------------------------------------------------- attention ----
// Scores: 16 heads x 32 keys of a tile; the 640 query dims are cut among the 8 warps in chunks of
// four, each lane holding 4 heads x 4 keys, and the warps' sums meet in shared memory (eight
// 16-byte shared loads feed 64 FMAs).  Values: a thread owns two latent dims of every head, for one of up to
// four groups of the tile's keys, whose sums meet at the item's end (16 requests of 3000 keys at 64 + 16
// dims, bf16: 48 us with one group, 41 with four).
struct Lay {   // shared memory, in floats
    int dqp, q, k, s, flag, total;
    int per, groups;   // threads and number of the groups
};
__host__ __device__ inline Lay layout(int Dk, int Dr) {
    Lay l;
    const int Dq = Dk + Dr;
    l.per = 64;
    while (2 * l.per < Dk) l.per *= 2;
    l.groups = NT / l.per;
    l.dqp = (Dq + 3) / 4 * 4 + 4;   // row pitch: rows four banks apart
    l.q = 0;
    l.k = HT * l.dqp;
    l.s = l.k + KT * l.dqp;
    l.flag = l.s + NT / 32 * HT * KT;
    const int meet = NT * HT * 2;   // the groups' sums, over the rest
    if (l.flag < meet) l.flag = meet;
    l.total = l.flag + 2 * KT + 3 * HT;
    return l;
}

template <typename T>
struct Four;   // four elements as they are loaded
template <>
struct Four<float> {
    float4 x;
    __device__ __forceinline__ void load(const float *p) { x = __ldg((const float4 *)p); }
    __device__ __forceinline__ void zero() { x = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ float4 f() const { return x; }
};
template <>
struct Four<__nv_bfloat16> {
    uint2 x;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { x = __ldg((const uint2 *)p); }
    __device__ __forceinline__ void zero() { x = make_uint2(0, 0); }
    __device__ __forceinline__ float4 f() const {
        return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                           __uint_as_float(x.y & 0xffff0000u));
    }
};
constexpr int KR = KT / (NT / 32), KC = DQ_MAX / 4 / 32;   // rows of a tile per warp, groups of four per lane

template <typename T>
__global__ void __launch_bounds__(NT, 1) paged_attn_simt_kernel(const __grid_constant__ PagedDecode p) {
    extern __shared__ float sm[];
    const int Dq = p.Dk + p.Dr;
    const Lay L = layout(p.Dk, p.Dr);
    float *sQ = sm + L.q, *sK = sm + L.k, *sS = sm + L.s;
    int *sRow = (int *)(sm + L.flag);                   // the keys' cache rows, -1 = no key; by parity of the tile
    float *sM = sm + L.flag + 2 * KT, *sL = sM + HT, *sA = sL + HT;   // running maximum, sum, rescale
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    pdl_wait();
    const long total = p.tile_off[p.B] * p.row_tiles;
    const long q = share_of(p, total);
    long t = blockIdx.x * q;
    const long tend = min(t + q, total);
    const int chunks = (Dq + 3) / 4, grp = tid / L.per, d = tid % L.per * 2;   // group, first latent dim
    const bool four = p.Dk % 4 == 0 && p.Dr % 4 == 0;
    while (t < tend) {
        const int b = request_of(p, p.tile_off, t);
        const long first = p.tile_off[b], per = p.tile_off[b + 1] - first;
        const int rt = (int)((t - first * p.row_tiles) / per);
        const long k0 = (t - first * p.row_tiles) % per;        // first tile of the item here
        const long k1 = min(per, k0 + tend - t);
        const int keys = keys_of(p, b), h0 = rt * HT, nh = min(HT, p.H - h0);
        // the rows of tile kt's keys
        auto look_up = [&](long kt) {
            if (tid < KT) {
                int row = -1;
                const long key = kt * KT + tid;
                if (key < keys) {
                    const int id = p.table[(long)b * p.max_pages + (int)key / p.page];
                    if (id >= 0 && id < p.num_pages) row = id * p.page + (int)key % p.page;
                }
                sRow[(kt & 1) * KT + tid] = row;
            }
        };
        // tile kt into registers: rows of whole groups of four, a lane per group, a warp's rows and groups
        // all in flight
        const int ck = p.Dk / 4, c4 = ck + p.Dr / 4;
        Four<T> v[KR][KC];
        auto fetch = [&](long kt) {
#pragma unroll
            for (int k = 0; k < KR; ++k) {
                const int row = sRow[(kt & 1) * KT + warp + 8 * k];
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    const int i = lane + 32 * c;
                    v[k][c].zero();
                    if (row >= 0 && i < c4)
                        v[k][c].load(i < ck ? (const T *)p.c_cache + (long)row * p.Dk + 4 * i
                                            : (const T *)p.kpe_cache + (long)row * p.Dr + 4 * (i - ck));
                }
            }
        };
        __syncthreads();   // the previous item has been read
        look_up(k0);
        __syncthreads();
        if (four) fetch(k0);
        if (four) {
            constexpr int QN = (HT * DQ_MAX / 4 + NT - 1) / NT;   // ten groups a thread, in flight at once
            float4 x[QN];
#pragma unroll
            for (int k = 0; k < QN; ++k) {
                const int i = tid + k * NT, h = i / c4, d = i % c4;
                const long row = (long)b * p.H + h0 + h;
                x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (h < nh)
                    x[k] = __ldcg((const float4 *)(d < ck ? (const float *)p.qabs + row * p.Dk + 4 * d
                                                          : (const float *)p.qpe + row * p.Dr + 4 * (d - ck)));
            }
#pragma unroll
            for (int k = 0; k < QN; ++k) {
                const int i = tid + k * NT, h = i / c4, d = i % c4;
                if (h < HT) *(float4 *)(sQ + h * L.dqp + 4 * d) = x[k];
            }
        } else {
            for (int i = tid; i < HT * L.dqp; i += NT) {
                const int h = i / L.dqp, d = i % L.dqp;
                float v = 0.f;
                if (h < nh && d < Dq) {
                    const long row = (long)b * p.H + h0 + h;
                    v = d < p.Dk ? ((const float *)p.qabs)[row * p.Dk + d] : ((const float *)p.qpe)[row * p.Dr + d - p.Dk];
                }
                sQ[i] = v;
            }
        }
        if (tid < HT) {
            sM[tid] = -INFINITY;
            sL[tid] = 0.f;
        }
        float o[HT][2];
#pragma unroll
        for (int h = 0; h < HT; ++h) o[h][0] = o[h][1] = 0.f;
        for (long kt = k0; kt < k1; ++kt) {
            const int *rows = sRow + (kt & 1) * KT;
            __syncthreads();   // the previous tile has been read
            if (four) {
#pragma unroll
                for (int k = 0; k < KR; ++k)
#pragma unroll
                    for (int c = 0; c < KC; ++c)
                        if (lane + 32 * c < c4) *(float4 *)(sK + (warp + 8 * k) * L.dqp + 4 * (lane + 32 * c)) = v[k][c].f();
            } else {
                for (int k = warp; k < KT; k += NT / 32) {   // a warp per key row; absent keys as zeros
                    const int row = rows[k];
                    const T *c = (const T *)p.c_cache + (long)row * p.Dk, *r = (const T *)p.kpe_cache + (long)row * p.Dr;
                    for (int d = lane; d < L.dqp; d += 32) {
                        float v = 0.f;
                        if (row >= 0 && d < Dq) v = d < p.Dk ? to_f<T>(c[d]) : to_f<T>(r[d - p.Dk]);
                        sK[k * L.dqp + d] = v;
                    }
                }
            }
            if (kt + 1 < k1) look_up(kt + 1);
            __syncthreads();
            if (four && kt + 1 < k1) fetch(kt + 1);   // under this tile's products
            {
                const int hg = lane >> 3, kg = lane & 7;   // heads 4 hg .., keys kg, kg + 8, ..
                float acc[4][4] = {};
#pragma unroll 2
                for (int c = warp; c < chunks; c += NT / 32) {
                    float4 q[4], k[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) q[i] = *(const float4 *)(sQ + (4 * hg + i) * L.dqp + 4 * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) k[i] = *(const float4 *)(sK + (kg + 8 * i) * L.dqp + 4 * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            acc[i][j] = fmaf(q[i].x, k[j].x, acc[i][j]);
                            acc[i][j] = fmaf(q[i].y, k[j].y, acc[i][j]);
                            acc[i][j] = fmaf(q[i].z, k[j].z, acc[i][j]);
                            acc[i][j] = fmaf(q[i].w, k[j].w, acc[i][j]);
                        }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sS[(warp * HT + 4 * hg + i) * KT + kg + 8 * j] = acc[i][j];
            }
            __syncthreads();
            for (int h = warp; h < HT; h += NT / 32) {   // a warp per head, a lane per key
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < NT / 32; ++w) s += sS[(w * HT + h) * KT + lane];
                s = rows[lane] >= 0 ? s * p.scale : -INFINITY;
                float m = s;
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
                const float mo = sM[h], mn = fmaxf(mo, m);
                const float e = s == -INFINITY ? 0.f : expf(s - mn);   // a NaN score stays one
                const float sum = warp_sum(e);
                __syncwarp();
                sS[h * KT + lane] = e;   // warp w's own slice of head h is read; slice 0 takes P
                if (lane == 0) {
                    const float al = mo == -INFINITY ? 0.f : expf(mo - mn);
                    sM[h] = mn;
                    sL[h] = sL[h] * al + sum;
                    sA[h] = al;
                }
            }
            __syncthreads();
#pragma unroll
            for (int h = 0; h < HT; ++h) {
                o[h][0] *= sA[h];
                o[h][1] *= sA[h];
            }
            if (d < p.Dk) {
                const int n = KT / L.groups;
                for (int k = grp * n; k < (grp + 1) * n; k += 4) {
                    float2 v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = *(const float2 *)(sK + (k + j) * L.dqp + d);
#pragma unroll
                    for (int h = 0; h < HT; ++h) {
                        const float4 w = *(const float4 *)(sS + h * KT + k);
                        o[h][0] = fmaf(w.x, v[0].x, fmaf(w.y, v[1].x, fmaf(w.z, v[2].x, fmaf(w.w, v[3].x, o[h][0]))));
                        o[h][1] = fmaf(w.x, v[0].y, fmaf(w.y, v[1].y, fmaf(w.z, v[2].y, fmaf(w.w, v[3].y, o[h][1]))));
                    }
                }
            }
        }
        const long slot = (long)blockIdx.x + (long)b * p.row_tiles + rt;
        float *po = p.po32 + slot * HT * p.Dk + d;
        auto store = [&](int h, float x, float y) {
            const float inv = sL[h] == 0.f ? 0.f : 1.f / sL[h];
            po[(long)h * p.Dk] = x * inv;
            if (d + 1 < p.Dk) po[(long)h * p.Dk + 1] = y * inv;
        };
        if (L.groups == 1) {
#pragma unroll
            for (int h = 0; h < HT; ++h)
                if (h < nh && d < p.Dk) store(h, o[h][0], o[h][1]);
        } else {
            __syncthreads();   // the last tile has been read
            float2 *meet = (float2 *)sm + tid % L.per;
#pragma unroll
            for (int h = 0; h < HT; ++h) meet[(grp * HT + h) * L.per] = make_float2(o[h][0], o[h][1]);
            __syncthreads();
            for (int h = grp; h < nh && d < p.Dk; h += L.groups) {   // the groups share out the heads
                float2 x = make_float2(0.f, 0.f);
                for (int g = 0; g < L.groups; ++g) {
                    const float2 y = meet[(g * HT + h) * L.per];
                    x.x += y.x;
                    x.y += y.y;
                }
                store(h, x.x, x.y);
            }
        }
        if (tid < nh) p.pl[slot * HT + tid] = sL[tid] == 0.f ? -INFINITY : sM[tid] + logf(sL[tid]);
        t += k1 - k0;
    }
}

// -------------------------------------------------------------------------- join ----
// Block (head, VC value dims, group of BT requests): four rows of W_V per warp into registers, before
// the attention ends; the parts' weights; their merge (a thread per four latent dims of a request, eight
// parts in flight); the product.
constexpr int JP = 160;   // parts of an item at most (the workers)

template <typename T>
__global__ void __launch_bounds__(NT) paged_join_simt_kernel(const __grid_constant__ PagedDecode p) {
    extern __shared__ float sm[];   // o [BT][Dk]
    __shared__ float sw[BT][JP];
    __shared__ long ss[BT];
    __shared__ int sn[BT];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int groups = (p.B + BT - 1) / BT, chunks = (p.Dv + VC - 1) / VC;
    int u = blockIdx.x;
    const int ch = u % chunks;
    u /= chunks;
    const int h = u / groups, b0 = (u % groups) * BT, nb = min(BT, p.B - b0);
    const int rt = h / p.row_tile, r = h % p.row_tile;
    constexpr int WN = DK_MAX / 32;
    const int v0 = ch * VC + warp * 4;
    const T *w = (const T *)p.w + ((long)h * (p.Dn + p.Dv) + p.Dn + v0) * p.Dk + lane;
    T wr[4][WN];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < WN; ++i) wr[k][i] = v0 + k < p.Dv && lane + 32 * i < p.Dk ? w[(long)k * p.Dk + 32 * i] : from_f<T>(0.f);
    pdl_wait();
    if (warp < BT) {
        const int b = b0 + warp;
        long s0 = 0;
        int n = 0;
        if (warp < nb) {
            const long total = p.tile_off[p.B] * p.row_tiles;
            const long per = p.tile_off[b + 1] - p.tile_off[b], first = p.tile_off[b] * p.row_tiles + rt * per;
            if (per > 0) {
                const long q = share_of(p, total), c0 = first / q;
                n = (int)((first + per - 1) / q - c0) + 1;
                s0 = c0 + (long)b * p.row_tiles + rt;
            }
        }
        const float *pl = p.pl + s0 * p.row_tile + r;
        float m = -INFINITY, sum = 0.f;
        for (int c = lane; c < n; c += 32) m = fmaxf(m, pl[(long)c * p.row_tile]);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        for (int c = lane; c < n; c += 32) {
            const float x = pl[(long)c * p.row_tile];
            sum += sw[warp][c] = x == -INFINITY ? 0.f : expf(x - m);
        }
        sum = warp_sum(sum);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        for (int c = lane; c < n; c += 32) sw[warp][c] *= inv;
        if (lane == 0) {
            ss[warp] = s0;
            sn[warp] = n;
            if (ch == 0 && warp < nb) p.lse[(long)b * p.H + h] = sum == 0.f ? -INFINITY : m + logf(sum);
        }
    }
    __syncthreads();
    const long pitch = (long)p.row_tile * p.Dk;
    if (p.Dk % 4 == 0) {
        const int d4 = p.Dk / 4;
        for (int i = tid; i < BT * d4; i += NT) {
            const int j = i / d4, n = sn[j];
            const float *po = p.po32 + (ss[j] * p.row_tile + r) * p.Dk + i % d4 * 4;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int c = 0; c < n; c += 8) {
                float4 x[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (c + u < n) x[u] = __ldcg((const float4 *)(po + (c + u) * pitch));
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (c + u < n) {
                        const float f = sw[j][c + u];
                        o.x = fmaf(f, x[u].x, o.x);
                        o.y = fmaf(f, x[u].y, o.y);
                        o.z = fmaf(f, x[u].z, o.z);
                        o.w = fmaf(f, x[u].w, o.w);
                    }
            }
            *(float4 *)(sm + 4 * i) = o;
        }
    } else {
        for (int i = tid; i < BT * p.Dk; i += NT) {
            const int j = i / p.Dk, d = i % p.Dk;
            const float *po = p.po32 + (ss[j] * p.row_tile + r) * p.Dk + d;
            float o = 0.f;
#pragma unroll 4
            for (int c = 0; c < sn[j]; ++c) o = fmaf(sw[j][c], po[c * pitch], o);
            sm[i] = o;
        }
    }
    __syncthreads();
    float acc[4][BT] = {};
#pragma unroll
    for (int i = 0; i < WN; ++i) {
        const int d = lane + 32 * i;
        if (d < p.Dk)
#pragma unroll
            for (int j = 0; j < BT; ++j) {
                const float x = sm[j * p.Dk + d];
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[k][j] = fmaf(to_f<T>(wr[k][i]), x, acc[k][j]);
            }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < BT; ++j) {
            const float x = warp_sum(acc[k][j]);
            if (lane == 0 && j < nb && v0 + k < p.Dv) ((T *)p.out)[((long)(b0 + j) * p.H + h) * p.Dv + v0 + k] = from_f<T>(x);
        }
}

template <typename T>
cudaError_t decode_simt(const PagedDecode &p, cudaStream_t st) {
    Turns turns{};
    std::copy_n(paged_turns(p.base, p.Dr), p.Dr / 2, turns.v);
    const unsigned units = (unsigned)((p.B + BT - 1) / BT) * (unsigned)p.H;
    const unsigned blocks = units * (unsigned)((p.Dk + DC - 1) / DC), jblocks = units * (unsigned)((p.Dv + VC - 1) / VC);
    const size_t s1 = ((size_t)BT * p.Dn + (size_t)NT / 32 * BT * DC) * 4, s2 = (size_t)layout(p.Dk, p.Dr).total * 4, s3 = (size_t)BT * p.Dk * 4;
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(paged_absorb_simt_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s1)) != cudaSuccess)
        return e;
    if ((e = cudaFuncSetAttribute(paged_attn_simt_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s2)) != cudaSuccess)
        return e;
    {
        ProfScope ps("paged_absorb", st);
        e = launch_after(paged_absorb_simt_kernel<T>, blocks + 1, NT, s1, st, p, turns);
    }
    if (e != cudaSuccess) return e;
    {
        ProfScope ps("paged_attn", st);
        e = launch_after(paged_attn_simt_kernel<T>, (unsigned)p.workers, NT, s2, st, p);
    }
    if (e != cudaSuccess) return e;
    {
        ProfScope ps("paged_join", st);
        e = launch_after(paged_join_simt_kernel<T>, jblocks, NT, s3, st, p);
    }
    return e;
}

}  // namespace

cudaError_t paged_decode_simt(const PagedDecode &p, cudaStream_t st) {
    return p.ty == TY_F32 ? decode_simt<float>(p, st) : decode_simt<__nv_bfloat16>(p, st);
}

}  // namespace mla
