// paged_many.cu -- the first and the last launch of the absorbed form on the tensor cores (paged_tc.cu) for many tokens
// of a step: hundreds of rows share a head's 128 x 512 weights, so both are products of 128 tokens a tile.
//
//   absorb     q[t, h, :] = W_K(h)^T q_nope[t, h, :] as bf16 hi + lo (and a third part where a token sees few keys), and
//              the rotated q_pe;
//   join       out[t, h, :] = W_V(h) sum_c w_c o_c, the merge of a token's parts, and its log-sum-exp.
// Persistent blocks, one an SM, walk equal shares of all (head, 128 tokens) in the heads' order and hold the head's
// weights in shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "paged_tc.cuh"
#include "tc_internal.h"

namespace mla {

__device__ unsigned g_paged_many_err = 0;

namespace {

using namespace tc;
using namespace paged;

constexpr unsigned FULL = 0xffffffffu;
constexpr int TOK = 128;                       // tokens of a tile
constexpr int W_BYTES = 128 * DK * 2;          // W_K(h) or W_V(h): eight boxes of 64 dims x 128 rows
constexpr int BOX = 128 * 128;                 // 64 dims x 128 rows

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, int *abort) {
    return mbar_wait(bar, parity, (volatile int *)abort, &g_paged_many_err);
}

// The block's share of the (head, tile) units: [from, to).
struct Share {
    int from, to, tiles;
};
__device__ __forceinline__ Share share(int H, int T) {
    const int tiles = (T + TOK - 1) / TOK;
    const long units = (long)H * tiles;
    return {(int)(units * blockIdx.x / gridDim.x), (int)(units * (blockIdx.x + 1) / gridDim.x), tiles};
}

// -------------------------------------------------------------------------- join ----
// Sixteen warps merge (four lanes a token's 64 dims, the loads two blocks of 64 dims ahead) into two stages of [128
// tokens][64 dims] hi and lo; one issues the MMAs (M = 128 tokens, N = 128 value dims, o's hi and lo one after the other,
// so that it is as exact as fp32 o); three find the next tiles' parts and the weights of the first two while the others
// work; four write a finished tile.
// 128 heads, events around it alone: 144 tokens 29 us, 512 53 us, 1024 84 us (2.3 KB a token and head, 3.6 TB/s); the
// kernel of 32 tokens a turn 55, 168 and 325 us.  What a turn of that one spends is latency, a chain of five loads, the
// merge, 64 MMAs and the output one after the other; here they overlap.  A tile's 5 us without its loads are the two
// stages' exchange with the MMAs.  What it took (512 tokens): the parts found by warps of their own (the writing ones did
// it: 66), no branch between the merge's loads and no spill (76), 96 or 104 registers a merging thread.  Loads of whole
// rows into L2 ahead gained nothing, nor did stages of 32 dims by two groups of warps (80).
// At 768 threads a thread may have 80 registers, fewer than the merge's loads need: its warps take over what the others give
// up (their sum is what the block was launched with).
constexpr int JM_MERGE = 512, JM_NT = JM_MERGE + 128 + 128;
constexpr int JM_REGS = 80, REGS_MERGE = 104, REGS_OUT = 24, REGS_FIND = 40;
static_assert(JM_MERGE * REGS_MERGE + 128 * REGS_OUT + 128 * REGS_FIND <= JM_NT * JM_REGS, "registers of the block");
constexpr int JM_AHEAD = 3;    // tiles whose parts are known
struct Parts {                 // of a tile's tokens
    int row[TOK], n[TOK];      // the first part's row of partials; parts, -1 for a token that is not computed here
    int ex[TOK];
    float w[2][2][TOK];        // [part 0 or 1][half of the dims]
    float top[TOK], inv[TOK];  // the parts' largest log-sum-exp, 1 / the sum of their weights
    int tok[TOK];              // the token's row in the step, -1 for one that is not computed here
    float lse[TOK], dot[TOK];  // the log-sum-exp without the q_lo term; q_lo . o
};
struct JoinCtl {
    Parts parts[JM_AHEAD];
    uint64_t w_full, full[2], empty[2], d_full[2], d_empty[2], parts_full[JM_AHEAD], parts_empty[JM_AHEAD], dots[JM_AHEAD];
    uint32_t tslot;
    int abort;
};
constexpr int JM_SMEM = W_BYTES + 2 * 2 * BOX + (int)sizeof(JoinCtl);
static_assert(JM_SMEM <= 232448, "shared memory budget");

__device__ __forceinline__ void load32(uint32_t (&v)[8], const void *p) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
}
// Two fp32 numbers in one register pair: an instruction for both.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(*(uint64_t *)&a), "l"(*(uint64_t *)&b), "l"(*(uint64_t *)&c));
    return *(float2 *)&d;
}
__device__ __forceinline__ void add_part(float2 (&o)[8], const uint32_t (&x)[8], float w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = fma2(make_float2(w, w), __half22float2(*(const __half2 *)&x[e]), o[e]);
}
__device__ __forceinline__ void dot16(float2 &s, const float2 (&o)[8], const uint32_t (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fma2(o[e], make_float2(__uint_as_float(x[e] << 16), __uint_as_float(x[e] & 0xffff0000u)), s);
}
// split2
__device__ __forceinline__ void split_pair(float2 x, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(x.x, x.y);
    const float2 rest = fma2(make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)), make_float2(-1.f, -1.f), x);
    lo = pack_bf16(rest.x, rest.y);
}

__global__ void __launch_bounds__(JM_NT, 1) paged_join_many_kernel(const __grid_constant__ CUtensorMap mW,
                                                                   const __grid_constant__ PagedDecode p, const bf16 *qlo,
                                                                   const bf16 *qrest) {
    extern __shared__ __align__(1024) uint8_t sm[];
    if (smem_u32(sm) & 1023) {   // the same answer in every block
        if (threadIdx.x == 0) atomicOr(&g_paged_many_err, 2u);
        return;
    }
    uint8_t *so = sm + W_BYTES;
    JoinCtl &ct = *(JoinCtl *)(so + 2 * 2 * BOX);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int T = tokens_of(p);   // (a list's length is of a launch long ended)
    const Share my = share(p.H, T);
    if (my.from == my.to) {
        pdl_wait();
        return;
    }
    if (tid == 0) {
        mbar_init(&ct.w_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ct.full[i], JM_MERGE / 32);
            mbar_init(&ct.empty[i], 1);
            mbar_init(&ct.d_full[i], 1);
            mbar_init(&ct.d_empty[i], 4);
        }
        for (int i = 0; i < JM_AHEAD; ++i) {
            mbar_init(&ct.parts_full[i], 3);
            mbar_init(&ct.parts_empty[i], JM_MERGE / 32 + 4);
            mbar_init(&ct.dots[i], JM_MERGE / 32);
        }
        ct.abort = 0;
        fence_mbar_init();
    }
    if (warp == 20) {
        tmem_alloc(&ct.tslot, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ct.tslot;
    const bool paired = p.row_tile <= 64;
    if (warp < 16) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_MERGE));
        pdl_wait();
        const int v = tid & 3, r = tid >> 2;   // 16 of the 64 dims, the token
        bool ok = true;
#pragma unroll 1
        for (int u = my.from, k = 0; ok && u < my.to; ++u, ++k) {
            Parts &pt = ct.parts[k % JM_AHEAD];
            const int h = u / my.tiles, t0 = u % my.tiles * TOK;
            if (!(ok = __all_sync(FULL, wait(&ct.parts_full[k % JM_AHEAD], (k / JM_AHEAD) & 1, &ct.abort)))) break;
            const int n = pt.n[r];
            const unsigned skip = paired || n <= 0 ? 0xff : lo_blocks((Extra)pt.ex[r]);   // blocks of 64 dims whose q_lo the scores have
            const __half *const po = p.po + (long)pt.row[r] * DK + 16 * v;   // its first part
            const long q0 = ((long)(t0 + r) * p.H + h) * DK + 16 * v, pitch = (long)p.row_tile * DK;
            const bool band = n > 0 && pt.ex[r] == EX_BAND;
            float2 dots = make_float2(0.f, 0.f);
            auto put = [&](int c, int s, const float2 (&o)[8]) {   // block c of o, to stage s
                if (!(ok = __all_sync(FULL, wait(&ct.empty[s], ((k * 4 + (c >> 1)) & 1) ^ 1, &ct.abort)))) return;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int f = 0; f < 4; ++f) split_pair(o[4 * e + f], hi[f], lo[f]);
                    uint4 *y = (uint4 *)(so + s * 2 * BOX + r * 128 + (((2 * v + e) ^ (r & 7)) << 4));   // 128-byte swizzle
                    y[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    y[BOX / 16] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ct.full[s]);
            };
            if (__all_sync(FULL, n != 0 && n <= 2 && !band)) {
                // The usual ones, without a branch between the loads: a token of one part reads it twice (the second time
                // from L1) with no weight, one that is not computed whatever its row of 0 names, which nobody reads.
                const __half *const p1 = n > 1 ? po + pitch : po;
                const unsigned want = __reduce_or_sync(FULL, ~skip & 0xff);
                uint32_t x[2][8], x1[2][8], q[2][8];
                auto load = [&](int c, int s) {
                    load32(x[s], po + 64 * c);
                    load32(x1[s], p1 + 64 * c);
                    if (want >> c & 1) load32(q[s], qlo + (skip == 0xff ? 0 : q0) + 64 * c);
                };
                load(0, 0);
                load(1, 1);
#pragma unroll 1
                for (int c2 = 0; ok && c2 < 8; c2 += 2)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int c = c2 + s;
                        float2 o[8] = {};
                        add_part(o, x[s], pt.w[0][c >> 2][r]);
                        add_part(o, x1[s], pt.w[1][c >> 2][r]);
                        if (want >> c & 1) {
                            float2 more = dots;
                            dot16(more, o, q[s]);
                            if (!(skip >> c & 1)) dots = more;
                        }
                        if (c + 2 < 8) load(c + 2, s);
                        put(c, s, o);
                        if (!ok) break;
                    }
            } else {
#pragma unroll 1
                for (int c = 0; ok && c < 8; ++c) {
                    float2 o[8] = {};
                    uint32_t y[2][8];
#pragma unroll 1
                    for (int j = 0; j < n; j += 2) {
                        float w[2] = {0.f, 0.f};
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (j + e < n) {
                                load32(y[e], po + (j + e) * pitch + 64 * c);
                                if (j < 2) {
                                    w[e] = pt.w[e][c >> 2][r];
                                } else {
                                    const long at = pt.row[r] + (long)(j + e) * p.row_tile;
                                    const float l = __ldcg(p.pl + at);
                                    w[e] = l == -INFINITY ? 0.f : expf(l - pt.top[r]) * pt.inv[r] * __ldcg(p.pscale + 2 * at + (c >> 2));
                                }
                            }
                        add_part(o, y[0], w[0]);
                        if (j + 1 < n) add_part(o, y[1], w[1]);
                    }
                    if (!(skip >> c & 1)) {
                        load32(y[0], qlo + q0 + 64 * c);
                        dot16(dots, o, y[0]);
                    }
                    if (band) {
                        load32(y[0], qrest + q0 + 64 * c);
                        dot16(dots, o, y[0]);
                    }
                    put(c, c & 1, o);
                }
            }
            float dot = dots.x + dots.y;
            dot += __shfl_xor_sync(FULL, dot, 1);
            dot += __shfl_xor_sync(FULL, dot, 2);
            if (v == 0) pt.dot[r] = dot;
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&ct.dots[k % JM_AHEAD]);
                mbar_arrive(&ct.parts_empty[k % JM_AHEAD]);
            }
        }
    } else if (warp >= 20) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_FIND));
        if (warp == 20) {
            bool ok = true;
            int head = -1;
            uint32_t wp = 0;
            const uint64_t a0 = sdesc_kmajor(so), b0 = sdesc_kmajor(sm);
            constexpr uint32_t idesc = idesc_f16(TOK, DV, false);
#pragma unroll 1
            for (int u = my.from, k = 0; ok && u < my.to; ++u, ++k) {
                const int h = u / my.tiles;
                if (h != head) {   // (the last tile's MMAs read the weights that lie there)
                    if (k > 0) ok = __all_sync(FULL, wait(&ct.d_full[(k - 1) & 1], ((k - 1) >> 1) & 1, &ct.abort));
                    if (!ok) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&ct.w_full, W_BYTES);
#pragma unroll 1
                        for (int i = 0; i < 8; ++i) tma_load_2d(sm + i * BOX, &mW, &ct.w_full, 64 * i, h * (DN + DV) + DN);
                    }
                    __syncwarp();
                    pdl_wait();   // (here and in the other roles: no wait runs out while the attention still works)
                    ok = __all_sync(FULL, wait(&ct.w_full, wp, &ct.abort));
                    wp ^= 1;
                    head = h;
                    if (!ok) break;
                }
                ok = __all_sync(FULL, wait(&ct.d_empty[k & 1], ((k >> 1) & 1) ^ 1, &ct.abort));
#pragma unroll 1
                for (int c = 0; ok && c < 8; ++c) {
                    const int s = c & 1;
                    ok = __all_sync(FULL, wait(&ct.full[s], (k * 4 + (c >> 1)) & 1, &ct.abort));
                    tc_fence_after();
                    if (ok && elect_one()) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint64_t a = a0 + (uint64_t)(s * (2 * BOX >> 4) + 2 * q), b = b0 + (uint64_t)(c * (BOX >> 4) + 2 * q);
                            mma_ss(tmem + (k & 1) * DV, a, b, idesc, (c | q) != 0);
                            mma_ss(tmem + (k & 1) * DV, a + (BOX >> 4), b, idesc, 1);
                        }
                        mma_commit(&ct.empty[s]);
                        if (c == 7) mma_commit(&ct.d_full[k & 1]);
                    }
                    __syncwarp();
                }
            }
        } else {   // a token's parts: their largest log-sum-exp, the sum of the weights, the first two's weights
            pdl_wait();
#pragma unroll 1
            for (int u = my.from, k = 0; u < my.to; ++u, ++k) {
                Parts &pt = ct.parts[k % JM_AHEAD];
                if (!__all_sync(FULL, wait(&ct.parts_empty[k % JM_AHEAD], ((k / JM_AHEAD) & 1) ^ 1, &ct.abort))) break;
                const int h = u / my.tiles;
#pragma unroll 1
                for (int r = tid - 21 * 32; r < TOK; r += 96) {
                    const int t = u % my.tiles * TOK + r;
                    int n = -1, ex = EX_NONE, tok = -1;
                    int at = 0;
                    if (t < T) {
                        const int2 of = __ldcg(p.of + t);
                        if (of.x >= 0) {
                            tok = token_of(p, t);
                            const int2 sp = __ldcg(p.spans + (long)of.x * p.row_tiles + (of.y + h) / p.row_tile);
                            ex = extra_of(paired, keys_of(p, of.x));
                            at = sp.x * p.row_tile + (of.y + h) % p.row_tile;
                            n = sp.y;
                        }
                    }
                    float2 scale[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) scale[e] = e < n ? __ldcg((const float2 *)p.pscale + at + e * p.row_tile) : make_float2(0.f, 0.f);
                    float m = -INFINITY, sum = 0.f, x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll 1
                    for (int j = 0; j < n; j += 4) {
                        float x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[e] = j + e < n ? __ldcg(p.pl + at + (j + e) * p.row_tile) : -INFINITY;
                        if (j == 0) x0 = x[0], x1 = x[1];
                        const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                        if (top > m) {
                            sum *= m == -INFINITY ? 0.f : expf(m - top);
                            m = top;
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum += x[e] == -INFINITY ? 0.f : expf(x[e] - m);
                    }
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    x0 = x0 == -INFINITY ? 0.f : expf(x0 - m) * inv;
                    x1 = x1 == -INFINITY ? 0.f : expf(x1 - m) * inv;
                    pt.row[r] = at;
                    pt.n[r] = n;
                    pt.ex[r] = ex;
                    pt.w[0][0][r] = x0 * scale[0].x;
                    pt.w[0][1][r] = x0 * scale[0].y;
                    pt.w[1][0][r] = x1 * scale[1].x;
                    pt.w[1][1][r] = x1 * scale[1].y;
                    pt.top[r] = m;
                    pt.inv[r] = inv;
                    pt.tok[r] = tok;
                    pt.lse[r] = sum == 0.f ? -INFINITY : m + logf(sum);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ct.parts_full[k % JM_AHEAD]);
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OUT));
        pdl_wait();
        const int quarter = warp & 3, r = quarter * 32 + lane;   // the tensor memory's lanes that the warp reads
#pragma unroll 1
        for (int u = my.from, k = 0; u < my.to; ++u, ++k) {
            const Parts &pt = ct.parts[k % JM_AHEAD];
            const bool ok = wait(&ct.parts_full[k % JM_AHEAD], (k / JM_AHEAD) & 1, &ct.abort) &&
                 wait(&ct.dots[k % JM_AHEAD], (k / JM_AHEAD) & 1, &ct.abort) && wait(&ct.d_full[k & 1], (k >> 1) & 1, &ct.abort);
            if (!__all_sync(FULL, ok)) break;
            tc_fence_after();
            const int tok = pt.tok[r];
            const long at = (long)max(tok, 0) * p.H + u / my.tiles;
            // (no keys: -inf stays, whatever the queries hold; 0 * NaN is not added)
            if (tok >= 0) p.lse[at] = pt.lse[r] == -INFINITY ? pt.lse[r] : pt.lse[r] + p.scale * pt.dot[r];
            bf16 *out = (bf16 *)p.out + at * DV;
#pragma unroll 1
            for (int c = 0; c < DV; c += 8) {
                uint32_t y[8], z[4];
                tmem_ld8_wait(tmem + (k & 1) * DV + c + ((uint32_t)(quarter * 32) << 16), y);
#pragma unroll
                for (int e = 0; e < 4; ++e) z[e] = pack_bf16(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1]));
                if (tok >= 0) *(uint4 *)(out + c) = make_uint4(z[0], z[1], z[2], z[3]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&ct.d_empty[k & 1]);
                mbar_arrive(&ct.parts_empty[k % JM_AHEAD]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*(volatile int *)&ct.abort) settle();
    if (warp == 20) tmem_dealloc(tmem, 256);
}

// ------------------------------------------------------------------------ absorb ----
// One warp issues the MMAs (M = 128 tokens, N = 256 latent dims: the product is all of the tensor memory, in two halves)
// and brings the weights, four bring the queries a tile ahead, three rotate q_pe, eight write the halves of q, 64 dims at a
// time through shared memory.  Bound by its writes, 2 KB a token and head; the third part is written for the tokens that
// need it alone (the plan has found them by then).
// 128 heads, events around it alone: 144 tokens 25 us, 512 41 us, 1024 75 us (3.6 TB/s of writes); the kernel of 64 tokens
// a block, which writes all third parts, 34, 91 and 168 us.  TMA stores of the 32 x 64 pieces were no faster than the
// warps' own; one buffer of queries 48 us, two warps to bring them 48.
constexpr int AM_NT = 512, AM_LOAD = 128;
constexpr int AM_Q = W_BYTES, AM_STG = AM_Q + 2 * 2 * BOX;   // two tiles of queries, two boxes of 64 dims each; staging: 32 tokens x 64 dims a warp
struct AbsorbCtl {
    uint64_t w_full, q_full[2], q_empty[2], d_full[2], d_empty[2];
    uint32_t tslot;
    int abort;
};
constexpr int AM_SMEM = AM_STG + 8 * 4096 + (int)sizeof(AbsorbCtl);
static_assert(AM_SMEM <= 232448, "shared memory budget");

__global__ void __launch_bounds__(AM_NT, 1) paged_absorb_many_kernel(const __grid_constant__ CUtensorMap mW,
                                                                     const __grid_constant__ Absorb a) {
    extern __shared__ __align__(1024) uint8_t sm[];
    const PagedDecode &p = a.p;
    // The plan is the launch in front and runs beside this one (it began behind the end of all before it): only what
    // depends on a token's keys waits for it.
    pdl_launch_dependents();
    if (smem_u32(sm) & 1023) {   // the same answer in every block
        if (threadIdx.x == 0) atomicOr(&g_paged_many_err, 2u);
        pdl_wait();
        return;
    }
    AbsorbCtl &ct = *(AbsorbCtl *)(sm + AM_STG + 8 * 4096);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int T = tokens_of(p);
    const Share my = share(p.H, T);
    if (T == 0) {
        pdl_wait();
        return;
    }
    if (tid == 0) {
        mbar_init(&ct.w_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ct.q_full[i], AM_LOAD / 32);
            mbar_init(&ct.q_empty[i], 2);
            mbar_init(&ct.d_full[i], 1);
            mbar_init(&ct.d_empty[i], 4);
        }
        ct.abort = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(&ct.tslot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ct.tslot;
    bool ok = true;
    if (warp < 8) {
        pdl_wait();
        const int half = warp >> 2, quarter = warp & 3;
        uint8_t *to = sm + AM_STG + warp * 4096;
        auto group = [&](int u) {   // of the thread's token, -1 where its keys do not matter
            const int t = u % my.tiles * TOK + quarter * 32 + lane;
            return p.scores_only || t >= T || u >= my.to ? -1 : __ldcg(&p.of[t].x);
        };
        int g = group(my.from);
        bool few = g >= 0 && keys_of(p, g) <= SHORT_KEYS, next_few = false;
#pragma unroll 1
        for (int u = my.from, k = 0; u < my.to; ++u, ++k, few = next_few) {
            const int h = u / my.tiles, t = u % my.tiles * TOK + quarter * 32;
            g = group(u + 1);
            if (!(ok = __all_sync(FULL, wait(&ct.d_full[half], k & 1, &ct.abort)))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {   // 64 dims' high halves, then their low ones
                const bool low = c & 1;
                if (c == 4) next_few = g >= 0 && keys_of(p, g) <= SHORT_KEYS;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int dim = half * 256 + (c >> 1) * 64 + i * 32;
                    uint32_t y[32], x[16];
                    tmem_ld32_wait(tmem + dim + ((uint32_t)(quarter * 32) << 16), y);
                    if (!low) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) x[e] = pack_bf16(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1]));
                    } else {
                        uint32_t rest[16], hi;
#pragma unroll
                        for (int e = 0; e < 16; ++e) split3(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1]), hi, x[e], rest[e]);
                        if (few) {
                            uint4 *r = (uint4 *)(a.qrest + ((long)(t + lane) * p.H + h) * DK + dim);
#pragma unroll
                            for (int e = 0; e < 4; ++e) r[e] = make_uint4(rest[4 * e], rest[4 * e + 1], rest[4 * e + 2], rest[4 * e + 3]);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)   // 128-byte swizzle
                        *(uint4 *)(to + lane * 128 + ((((i * 4 + e) ^ lane) & 7) << 4)) = make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                }
                if (c == 7) {   // the half is read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ct.d_empty[half]);
                }
                __syncwarp();
                bf16 *q = (low ? a.qlo : a.qhi) + half * 256 + (c >> 1) * 64 + (lane & 7) * 8;
#pragma unroll
                for (int e = 0; e < 8; ++e) {   // four tokens' 128 bytes
                    const int r = 4 * e + (lane >> 3);
                    const uint4 x = *(const uint4 *)(to + r * 128 + (((lane ^ r) & 7) << 4));
                    if (t + r < T) *(uint4 *)(q + ((long)(t + r) * p.H + h) * DK) = x;
                }
                __syncwarp();
            }
        }
    } else if (warp == 8) {
        int head = -1;
        uint32_t wp = 0;
        const uint64_t a0 = sdesc_kmajor(sm + AM_Q), b0 = sdesc_mnmajor(sm, BOX);
        constexpr uint32_t idesc = idesc_f16(TOK, 256, false, true);
#pragma unroll 1
        for (int u = my.from, k = 0; ok && u < my.to; ++u, ++k) {
            const int h = u / my.tiles;
            if (h != head) {   // (the last tile's MMAs read the weights that lie there)
                if (k > 0) ok = __all_sync(FULL, wait(&ct.q_empty[(k - 1) & 1], ((k - 1) >> 1) & 1, &ct.abort));
                if (!ok) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&ct.w_full, W_BYTES);
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) tma_load_2d(sm + i * BOX, &mW, &ct.w_full, 64 * i, h * (DN + DV));
                }
                __syncwarp();
                ok = __all_sync(FULL, wait(&ct.w_full, wp, &ct.abort));
                wp ^= 1;
                head = h;
                if (!ok) break;
            }
            ok = __all_sync(FULL, wait(&ct.q_full[k & 1], (k >> 1) & 1, &ct.abort));
#pragma unroll 1
            for (int half = 0; ok && half < 2; ++half) {
                ok = __all_sync(FULL, wait(&ct.d_empty[half], (k & 1) ^ 1, &ct.abort));
                tc_fence_after();
                if (ok && elect_one()) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)   // 16 of the summed dims
                        mma_ss(tmem + half * 256, a0 + (uint64_t)((k & 1) * (2 * BOX >> 4) + (q >> 2) * (BOX >> 4) + 2 * (q & 3)),
                               b0 + (uint64_t)(half * (4 * BOX >> 4) + q * (2048 >> 4)), idesc, q != 0);
                    mma_commit(&ct.d_full[half]);
                    mma_commit(&ct.q_empty[k & 1]);
                }
                __syncwarp();
            }
        }
    } else if (warp < 9 + AM_LOAD / 32) {
        const int i0 = tid - 9 * 32;
#pragma unroll 1
        for (int u = my.from, k = 0; u < my.to; ++u, ++k) {
            const int h = u / my.tiles, t0 = u % my.tiles * TOK;
            if (!(ok = __all_sync(FULL, wait(&ct.q_empty[k & 1], ((k >> 1) & 1) ^ 1, &ct.abort)))) break;
#pragma unroll 4
            for (int i = i0; i < TOK * 16; i += AM_LOAD) {   // (rows behind the last token: its again)
                const int r = i >> 4, c = i & 15;
                cp16(sm + AM_Q + (k & 1) * 2 * BOX + (c >> 3) * BOX + r * 128 + (((c ^ r) & 7) << 4),
                     (const bf16 *)p.q_nope + ((long)token_of(p, min(t0 + r, T - 1)) * p.H + h) * DN + c * 8);
            }
            asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ct.q_full[k & 1]);
        }
    } else {
        pdl_wait();
        const long n = (long)T * ((p.H + 31) / 32);
#pragma unroll 1
        for (long i = (long)(warp - 9 - AM_LOAD / 32) * gridDim.x + blockIdx.x; i < n; i += (AM_NT - 288l - AM_LOAD) / 32 * gridDim.x)
            rotate_queries<true, true, 16>(a, (int)i, lane);
    }
    tc_fence_before();
    __syncthreads();
    if (*(volatile int *)&ct.abort) settle();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t paged_absorb_many(const paged::Absorb &ab, cudaStream_t st) {
    using ull = unsigned long long;
    const PagedDecode &p = ab.p;
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(paged_absorb_many_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, AM_SMEM)) != cudaSuccess) return e;
    CUtensorMap mW;
    const ull dw[2] = {DK, (ull)p.H * (DN + DV)}, sw[1] = {DK * 2};
    const unsigned bw[2] = {64, DN};
    if ((e = make_tma_map(&mW, p.w, 2, dw, sw, bw)) != cudaSuccess) return e;
    ProfScope ps("paged_absorb", st);
    return launch_after(paged_absorb_many_kernel, 2 * PAGED_TC_WORKERS, AM_NT, AM_SMEM, st, mW, ab);
}

cudaError_t paged_join_many(const PagedDecode &p, const __nv_bfloat16 *qlo, const __nv_bfloat16 *qrest, cudaStream_t st) {
    using ull = unsigned long long;
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(paged_join_many_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, JM_SMEM)) != cudaSuccess) return e;
    // the register split waits for ever where the launch has fewer to draw on: another compiler's choice is refused
    static std::atomic<int> regs{0};   // (of the kernel: the same from any host thread and device)
    if (regs == 0) {
        cudaFuncAttributes at;
        if ((e = cudaFuncGetAttributes(&at, paged_join_many_kernel)) != cudaSuccess) return e;
        regs = at.numRegs;
    }
    if (regs < JM_REGS) return cudaErrorInvalidConfiguration;
    CUtensorMap mW;
    const ull d[2] = {DK, (ull)p.H * (DN + DV)}, s[1] = {DK * 2};
    const unsigned b[2] = {64, DV};
    if ((e = make_tma_map(&mW, p.w, 2, d, s, b)) != cudaSuccess) return e;
    const int units = p.H * ((p.T + TOK - 1) / TOK);
    ProfScope ps("paged_join", st);
    return launch_after(paged_join_many_kernel, (unsigned)std::min(units, 2 * PAGED_TC_WORKERS), JM_NT, JM_SMEM, st, mW, p, qlo, qrest);
}

cudaError_t paged_many_read_and_clear_error(unsigned *flags, cudaStream_t st) {
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_paged_many_err, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
    if (e != cudaSuccess) return e;
    if ((e = cudaStreamSynchronize(st)) != cudaSuccess) return e;
    if (v) {
        unsigned z = 0;
        e = cudaMemcpyToSymbolAsync(g_paged_many_err, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
        if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    }
    *flags |= v;
    return e;
}

}  // namespace mla
