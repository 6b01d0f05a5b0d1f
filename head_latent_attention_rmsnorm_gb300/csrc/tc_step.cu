// tc_step.cu -- the explicit form of a paged step's tokens on the sm_103a tensor cores: K_nope and V^T rebuilt from the
// gathered pages by the pair GEMM, then causal attention of 128-token tiles over them.
//
// Mathematics: s_tj = scale (q_nope_t . K_nope_j + rot(q_pe_t) . k_pe_j) for the keys j that token t sees, softmax, O =
// P V, log-sum-exp.  How many key rows and tiles there are is known on the device only: fixed grids of persistent CTAs walk
// the units (128 tokens of one request, head) of a list made there.
//
// Per CTA, 12 warps.  Warp 0 loads Q of each unit and the K tiles (128 keys: K_nope and the band), warp 2 the V^T
// tiles, two-deep rings; warp 1 issues S = Q K^T (Q in TMEM) into S buffer T & 1, warp 3 O += P V.  Warps 4-7 and 8-11 are
// two softmax groups, one thread per query row each: group T & 1 takes tile T, so that one's exponentials run under the
// other's loads and maximum.  What a tile hands to the next is its row's maximum, through shared memory and a named
// barrier of the two warps of a row; each group keeps its own part of the row sum, and they meet at the unit's end.
// O in TMEM is rescaled only when a row's maximum grows by more than 2^8.
//
// Precision.  Operands are fp16 (11 bits).  The row sums are fp32 and of the unrounded weights: a column of ones in
// the P V product would gather them 16 at a time in an accumulator that cuts off, 3e-5 of the sum at 16384 keys.  The
// rotated q_pe has its fp16 rest too (four score MMAs of 16): its rounding is the same for all keys, and shifted a
// log-sum-exp by 1.5e-5 whatever their number.  K_nope's rounding errs by 1.6e-4 in each score, 1.6e-4 / sqrt(0.4 keys) in
// a row's log-sum-exp: little but for rows of few keys, so the request's first 512 keys have K_nope's rest in the scores too
// (eight MMAs more for those tiles, an entry of their own in the K ring).  V is held times a power of two of its head and
// request (value_shift), which each row's last division takes out again: fp16's narrow range bounds scores only.
//
// What bounds it.  2048 tokens over 16384 keys, 128 heads in shards of 64: 2.04 ms, 1265 TFLOP/s of the 640 a (token, key,
// head) and 1520 of the MMAs that it issues (1.2 times those: the band's rest), where a product that runs for seconds under the
// power cap reaches 1726.  A tile's 24 MMAs of 64 cycles take 1536; the chain of one S buffer, scores 1024, softmax some 1300, P V
// 512, is two tiles' time.  Measured: one softmax group of four warps 2.05 ms (109 us against 109 for three prompts of up to 4096
// tokens, 16 heads), two groups with the product behind the whole of P 2.12 ms (113 us), by halves 2.04 ms; without the
// band's rest 1.78-1.95 ms, with a log-sum-exp six times less exact.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "mla_internal.h"
#include "tc.h"
#include "tc_common.cuh"
#include "tc_internal.h"

namespace mla {

__device__ unsigned g_tc_step_err = 0;

namespace {

using namespace tc;

constexpr unsigned FULL = 0xffffffffu;
constexpr int BKV = 128;
constexpr uint32_t BOX = 128 * 128;       // 128 rows of 64 16-bit elements
constexpr uint32_t K_BYTES = 3 * BOX;     // K_nope lo, hi, band
constexpr uint32_t V_BYTES = 2 * BOX;     // V^T: 128 dims x 2 key halves
constexpr int KST = 2, VST = 2;
constexpr int Q_BOXES = 4;                // q_nope lo, hi (bf16), rotated q_pe, its rest (fp16)
constexpr uint32_t QS_BYTES = Q_BOXES * BOX;
constexpr uint32_t OFF_K = QS_BYTES, OFF_V = OFF_K + KST * K_BYTES, OFF_ROW = OFF_V + VST * V_BYTES;
// the rows' maxima [parity of the tile][row], their sums [group][row]
constexpr uint32_t OFF_BAR = OFF_ROW + 2 * 2 * 128 * 4, S_BYTES = OFF_BAR + 256;
static_assert(S_BYTES <= 232448, "shared memory budget");
constexpr uint32_t T_O = 256, T_Q = 384;  // TMEM: S buffers 0-127, 128-255, O, Q (32 columns a box)
constexpr float RESCALE_LOG2 = 8.0f;
constexpr int NTHREADS = 384;
// registers of a thread of the first warpgroup and of the softmax groups, in place of the launch's 168: 128 (80 + 2 208) =
// 63488 of 384 x 168 = 64512
constexpr int REGS_ISSUE = 80, REGS_SOFTMAX = 208;
static_assert(128 * (REGS_ISSUE + 2 * REGS_SOFTMAX) <= NTHREADS * 168, "the split draws on the launch's registers");

struct StepK {
    const StepTile *tiles;
    const int *ctl;           // as TcStep's
    const int *limits, *done; // [tokens]: keys seen; nonzero: computed here
    const uint32_t *held;     // a bit per key row: there is such a key
    const int *holes;         // [requests]: nonzero: some page is missing
    const unsigned *w_max, *c_max;   // [heads of the model], [requests]: V is held times 2^value_shift of the two
    int head_off, nh;         // first head, heads of this launch
    float scale_log2;
    __nv_bfloat16 *out;
    long H;
    int out_v8;               // the output's rows are 32-byte aligned
    float *lse;
    uint32_t idesc_s, idesc_pv;
};

struct Work {
    int hl, q0, rows, nt;     // head, first token, tokens, key tiles
    int k0, request, r0, nr;  // first key row, request, first row of K_nope's rest, key tiles that have one
};
__device__ __forceinline__ Work work_of(const StepK &s, bool heaviest, int u) {
    // The heaviest tiles first, heads in turns, where L2 holds all heads' K_nope and V^T; else a request's tiles of one
    // head behind one another, so that L2 holds those of the ten or so heads in work (three prompts of up to 4096
    // tokens, 16 heads, 103 MB: 102 us against 127; 2048 tokens over 16384 keys, 64 heads a shard: 2.07 ms against 2.17).
    // A request of tiles f .. f + c - 1 then has units f nh .. (f + c) nh - 1, so unit u / nh is one of its tiles.
    int i = u / s.nh, h = u - i * s.nh;
    const int4 *e = (const int4 *)(s.tiles + i);
    if (!heaviest) {
        const int place = __ldcg(&e[1].w), f = place >> 16, c = place & 0xffff, v = u - f * s.nh;
        h = v / c;
        e = (const int4 *)(s.tiles + f + (v - h * c));
    }
    const int4 x = __ldcg(e), y = __ldcg(e + 1);
    return Work{h, x.x, x.y, x.w, x.z, y.x, y.y, min(y.z, x.w)};
}
// Unit of round k for CTA c of G: rounds alternate direction, so that every CTA gets a mix of heavy and light ones.
__device__ __forceinline__ int unit_at(int k, int c, int G) { return (k & 1) ? (k + 1) * G - 1 - c : k * G + c; }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void bar_arrive(int id, int n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }

enum : int {
    B_QREADY = 0,
    B_KFULL = 1,
    B_KEMPTY = B_KFULL + KST,
    B_VFULL = B_KEMPTY + KST,
    B_VEMPTY = B_VFULL + VST,
    B_SFULL = B_VEMPTY + VST,
    B_PFULL = B_SFULL + 2,
    B_PVDONE = B_PFULL + 4,      // (B_PFULL: [buffer][half of the keys])
    B_ODONE = B_PVDONE + 2,
    B_OFINAL,
    B_OFREE,
    B_QSFULL,
    B_COUNT
};
__device__ __forceinline__ uint32_t arrivals(int i) {
    if (i == B_QREADY || i == B_OFREE) return 8;          // the softmax warps
    return i >= B_PFULL && i < B_PVDONE ? 4 : 1;          // a group's warps
}

__global__ void __launch_bounds__(NTHREADS, 1)
    tc_step_kernel(const __grid_constant__ CUtensorMap mQn, const __grid_constant__ CUtensorMap mQr,
                   const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mKr,
                   const __grid_constant__ CUtensorMap mV, const __grid_constant__ CUtensorMap mR,
                   const __grid_constant__ StepK p) {
    if (__ldcg(p.ctl + 1) == 0) {   // (of a launch that ended before the one in front began its work)
        pdl_wait();
        return;
    }
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {   // no room to align by hand; the same answer in every CTA
        if (threadIdx.x == 0) atomicOr(&g_tc_step_err, 2u);
        return;
    }
    uint8_t *sK = smem + OFF_K, *sV = smem + OFF_V;
    float(*row_max)[128] = (float(*)[128])(smem + OFF_ROW), (*row_sum)[128] = row_max + 2;
    uint64_t *bars = (uint64_t *)(smem + OFF_BAR);
    uint32_t *tslot = (uint32_t *)(bars + B_COUNT);
    volatile int *abort = (volatile int *)(tslot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = gridDim.x, c = blockIdx.x;
    auto wait = [&](int i, uint32_t parity) { return mbar_wait(&bars[i], parity, abort, &g_tc_step_err); };
    auto wait_all = [&](int i, uint32_t parity) { return __all_sync(FULL, wait(i, parity)); };

    if (tid == 0) {
        for (int i = 0; i < B_COUNT; ++i) mbar_init(&bars[i], arrivals(i));
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    pdl_wait();   // units, limits, rows: all from the launches in front
    const int units = __ldcg(p.ctl + 1) * p.nh;
    const bool heaviest = __ldcg(p.ctl + 3) != 0;
    // Every role walks the same units in the same order and counts key tiles T across units, so ring slots and barrier
    // parities continue from one unit to the next.  This CTA's next unit from round k on, -1 behind the last:
    auto next_unit = [&](int &k) {
        for (; k * G < units; ++k)
            if (unit_at(k, c, G) < units) return unit_at(k, c, G);
        return -1;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_ISSUE));
        if (warp == 0) {
            // ------------------------------------------- Q of each unit and K tiles (TMA)
            if (lane == 0) {
                tma_prefetch_desc(&mQn);
                tma_prefetch_desc(&mQr);
                tma_prefetch_desc(&mK);
                tma_prefetch_desc(&mKr);
                tma_prefetch_desc(&mR);
                bool ok = true;
                int E = 0, n = 0, k = 0;   // ring entries, units so far
                for (int u; ok && (u = next_unit(k)) >= 0; ++k) {
                    const Work w = work_of(p, heaviest, u);
                    const int h = p.head_off + w.hl;
                    // once the softmax warps have moved the last unit's Q into TMEM
                    if (n > 0 && !wait(B_QREADY, (n - 1) & 1)) break;
                    ++n;
                    mbar_arrive_expect_tx(&bars[B_QSFULL], QS_BYTES);
                    tma_load_4d(smem, &mQn, &bars[B_QSFULL], 0, h, w.q0, 0);
                    tma_load_4d(smem + BOX, &mQn, &bars[B_QSFULL], 64, h, w.q0, 0);
                    tma_load_4d(smem + 2 * BOX, &mQr, &bars[B_QSFULL], 0, h, w.q0, 0);
                    tma_load_4d(smem + 3 * BOX, &mQr, &bars[B_QSFULL], 64, h, w.q0, 0);
                    for (int j = 0; j < w.nt && ok; ++j)
                        for (int r = 0; r < 1 + (j < w.nr); ++r, ++E) {   // the second entry: the tile's rest of K_nope
                            const int s = E % KST;
                            uint64_t *full = &bars[B_KFULL + s];
                            uint8_t *kd = sK + s * K_BYTES;
                            ok = wait(B_KEMPTY + s, ((E / KST) & 1) ^ 1);   // (passes at first)
                            if (!ok) break;
                            mbar_arrive_expect_tx(full, r ? 2 * BOX : K_BYTES);
                            const int row = (r ? w.r0 : w.k0) + j * BKV;
                            tma_load_3d(kd, r ? &mR : &mK, full, w.hl * 128, row, 0);
                            tma_load_3d(kd + BOX, r ? &mR : &mK, full, w.hl * 128 + 64, row, 0);
                            if (!r) tma_load_3d(kd + 2 * BOX, &mKr, full, 0, row, 0);
                        }
                }
            }
        } else if (warp == 2) {
            // ------------------------------------------------------------- V^T tiles (TMA)
            if (lane == 0) {
                tma_prefetch_desc(&mV);
                bool ok = true;
                int T = 0, k = 0;
                for (int u; ok && (u = next_unit(k)) >= 0; ++k) {
                    const Work w = work_of(p, heaviest, u);
                    for (int j = 0; j < w.nt; ++j, ++T) {
                        const int s = T % VST;
                        ok = wait(B_VEMPTY + s, ((T / VST) & 1) ^ 1);   // (passes at first)
                        if (!ok) break;
                        uint8_t *vd = sV + s * V_BYTES;
                        mbar_arrive_expect_tx(&bars[B_VFULL + s], V_BYTES);
                        tma_load_3d(vd, &mV, &bars[B_VFULL + s], w.k0 + j * BKV, w.hl * 128, 0);
                        tma_load_3d(vd + BOX, &mV, &bars[B_VFULL + s], w.k0 + j * BKV + 64, w.hl * 128, 0);
                    }
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------- scores: warp-uniform, one lane issues
            bool ok = true;
            int T = 0, E = 0, n = 0, k = 0;
            for (int u; ok && (u = next_unit(k)) >= 0; ++k) {
                const Work w = work_of(p, heaviest, u);
                ok = wait_all(B_QREADY, n & 1);   // this unit's Q is in TMEM
                ++n;
                for (int j = 0; j < w.nt && ok; ++j, ++T) {
                    const int b = T & 1;
                    const uint32_t s_tm = tmem + b * 128;
                    const bool rest = j < w.nr;
                    ok = wait_all(B_KFULL + E % KST, (E / KST) & 1);
                    // S buffer b last held P of tile T - 2: its product has read it
                    if (ok && T >= 2) ok = wait_all(B_PVDONE + b, ((T - 2) >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint8_t *kd = sK + E % KST * K_BYTES;
#pragma unroll
                        for (int kb = 0; kb < Q_BOXES; ++kb) {
                            const uint64_t db = sdesc_kmajor(kd + (kb < 3 ? kb : 2) * BOX);
#pragma unroll
                            for (int k4 = 0; k4 < 4; ++k4)
                                mma_ts(s_tm, tmem + T_Q + (kb * 4 + k4) * 8, db + 2 * k4, p.idesc_s, (kb | k4) != 0);
                        }
                        if (!rest) mma_commit(&bars[B_SFULL + b]);
                        mma_commit(&bars[B_KEMPTY + E % KST]);
                    }
                    __syncwarp();
                    ++E;
                    if (!rest) continue;
                    ok = wait_all(B_KFULL + E % KST, (E / KST) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint8_t *kd = sK + E % KST * K_BYTES;
#pragma unroll
                        for (int kb = 0; kb < 2; ++kb) {
                            const uint64_t db = sdesc_kmajor(kd + kb * BOX);
#pragma unroll
                            for (int k4 = 0; k4 < 4; ++k4)
                                mma_ts(s_tm, tmem + T_Q + (kb * 4 + k4) * 8, db + 2 * k4, p.idesc_s, 1);
                        }
                        mma_commit(&bars[B_SFULL + b]);
                        mma_commit(&bars[B_KEMPTY + E % KST]);
                    }
                    __syncwarp();
                    ++E;
                }
            }
        } else {
            // ------------------------------------------------------------- O += P V
            bool ok = true;
            int T = 0, n = 0, k = 0;
            for (int u; ok && (u = next_unit(k)) >= 0; ++k) {
                const Work w = work_of(p, heaviest, u);
                ok = wait_all(B_OFREE, (n & 1) ^ 1);   // the last unit's O has been read (passes at first)
                ++n;
                for (int j = 0; j < w.nt && ok; ++j, ++T) {
                    const int b = T & 1, s = T % VST;
                    ok = wait_all(B_VFULL + s, (T / VST) & 1);
                    // by halves of the keys: the first ones' product runs under the other ones' exponentials
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb) {
                        ok = ok && wait_all(B_PFULL + 2 * b + kb, (T >> 1) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t db = sdesc_kmajor(sV + s * V_BYTES + kb * BOX);
#pragma unroll
                            for (int k4 = 0; k4 < 4; ++k4)
                                mma_ts(tmem + T_O, tmem + b * 128 + kb * 32 + k4 * 8, db + 2 * k4, p.idesc_pv, (j | kb | k4) != 0);
                            if (kb == 1) {
                                mma_commit(&bars[B_VEMPTY + s]);
                                mma_commit(&bars[B_PVDONE + b]);
                                mma_commit(&bars[B_ODONE]);
                                if (j == w.nt - 1) mma_commit(&bars[B_OFINAL]);
                            }
                        }
                        __syncwarp();
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
        // ----------------------------------------------------------------- softmax groups
        const int quad = warp & 3, g = (warp >> 2) - 1, row = quad * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
        // named barriers of this row's two warps: a maximum for the other group, one from it, both at a unit's end
        const int b_send = 1 + quad * 2 + g, b_recv = 1 + quad * 2 + (g ^ 1), b_meet = 9 + quad;
        bool ok = true;   // an abandoned wait clears it; the walk goes on, so that every barrier is reached
        // a unit's Q from the staging buffer into TMEM: group 0 the row's q_nope (bf16 widened to fp16), group 1 the rotated
        // q_pe and its rest.  16-byte chunk i of row r of a staged box sits at chunk i ^ (r & 7).
        auto load_q = [&](int n) {
            ok = __all_sync(FULL, ok && wait(B_QSFULL, n & 1));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t *src = smem + (2 * g + h) * BOX + row * 128;
                uint32_t q[2][16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 v = *(const uint4 *)(src + ((i ^ (row & 7)) << 4));
                    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        q[i >> 2][4 * (i & 3) + e] =
                            g ? x[e] : pack_f16(__uint_as_float(x[e] << 16), __uint_as_float(x[e] & 0xffff0000u));
                }
                tmem_st16(lane_base + T_Q + 32 * (2 * g + h), q[0]);
                tmem_st16(lane_base + T_Q + 32 * (2 * g + h) + 16, q[1]);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_QREADY]);
        };
        int T = 0, n = 0, k = 0, u = next_unit(k);
        if (u >= 0) load_q(0);
        while (u >= 0) {
            const Work w = work_of(p, heaviest, u);
            ++k;
            const int u_next = next_unit(k);
            // keys that the row, that every row of the warp sees (rows behind the tile's tokens: no matter what)
            const int sees = row < w.rows ? __ldcg(p.limits + w.q0 + row) : 2147483647;
            const int all_see = __reduce_min_sync(FULL, sees), holes = __ldcg(p.holes + w.request);
            const float unscale = pow2(-value_shift(__ldcg(p.w_max + p.head_off + w.hl), __ldcg(p.c_max + w.request)));
            float m = -INFINITY, sum = 0.f;   // the row's maximum that this group last used; its part of the sum, relative to it
#pragma unroll 1
            for (int j = 0; j < w.nt; ++j, ++T) {
                if ((T & 1) != g) continue;
                ok = __all_sync(FULL, ok && wait(B_SFULL + g, (T >> 1) & 1));
                tc_fence_after();
                float x[128];
                {
                    uint32_t(&r)[4][32] = *reinterpret_cast<uint32_t(*)[4][32]>(x);
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld32(lane_base + g * 128 + 32 * q, r[q]);
                    tmem_ld_wait();
                }
                const int j0 = j * BKV;
                if (j0 + BKV > all_see || holes) {
                    const int lim = sees - j0;
#pragma unroll
                    for (int i = 0; i < 128; ++i) x[i] = i < lim ? x[i] : -INFINITY;
                    if (holes) {
                        const uint4 h = __ldcg((const uint4 *)(p.held + (w.k0 + j0) / 32));
                        const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
                        for (int i = 0; i < 128; ++i) x[i] = hw[i >> 5] >> (i & 31) & 1 ? x[i] : -INFINITY;
                    }
                }
                float mx[8];
#pragma unroll
                for (int a = 0; a < 8; ++a) mx[a] = x[a];
#pragma unroll
                for (int i = 8; i < 128; ++i) mx[i & 7] = fmaxf(mx[i & 7], x[i]);
                const float mt = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                       fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * p.scale_log2;
                // the maximum in use after the tile in front (of another unit: none)
                float m_old = -INFINITY;
                if (T > 0) {
                    named_bar_sync(b_recv, 64);
                    if (j > 0) m_old = row_max[g ^ 1][row];
                }
                const bool need = mt > m_old + RESCALE_LOG2;   // also true on the first finite maximum
                const float m_use = need ? mt : m_old;
                row_max[g][row] = m_use;
                if (u_next >= 0 || j < w.nt - 1) bar_arrive(b_send, 64);   // (nobody waits behind the last tile)
                if (j > 0 && __any_sync(FULL, need)) {
                    const float alpha = !need ? 1.f : m_old == -INFINITY ? 0.f : ex2(m_old - m_use);
                    ok = __all_sync(FULL, ok && wait(B_ODONE, (T - 1) & 1));   // O holds the tile in front's product
                    tc_fence_after();
#pragma unroll 1
                    for (int q = 0; q < 8; ++q) {
                        uint32_t o[16];
                        tmem_ld16_wait(lane_base + T_O + 16 * q, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st16(lane_base + T_O + 16 * q, o);
                    }
                    tmem_st_wait();
                }
                if (m_use != m) {
                    sum *= m == -INFINITY ? 0.f : ex2(m - m_use);
                    m = m_use;
                }
                const float nm = m == -INFINITY ? 0.f : -m;
                // P over the S columns it came from, 32 keys (16 columns) at a time
                float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float p0 = ex2(fmaf(x[32 * q + 2 * i], p.scale_log2, nm)),
                                    p1 = ex2(fmaf(x[32 * q + 2 * i + 1], p.scale_log2, nm));
                        pk[i] = pack_f16(p0, p1);
                        add[2 * (i & 1)] += p0;
                        add[2 * (i & 1) + 1] += p1;
                    }
                    tmem_st16(lane_base + g * 128 + 16 * q, pk);
                    if (q & 1) {
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars[B_PFULL + 2 * g + (q >> 1)]);
                    }
                }
                sum += (add[0] + add[1]) + (add[2] + add[3]);
            }
            // the next unit's Q, once this one's last scores are done (the other group's tile, for one of the groups), so that
            // its first scores overlap the last product and the epilogue
            if (u_next >= 0) {
                ok = __all_sync(FULL, ok && wait(B_SFULL + ((T - 1) & 1), ((T - 1) >> 1) & 1));
                load_q(n + 1);
            }
            // ---- the groups' sums meet; a group stores half of the row's outputs
            named_bar_sync(b_meet, 64);   // (the last tile's group has set its maximum)
            const float top = row_max[(T - 1) & 1][row];
            if (m != -INFINITY) sum *= ex2(m - top);   // (else 0, or NaN where a score is NaN)
            row_sum[g][row] = sum;
            named_bar_sync(b_meet, 64);   // (and the last unit's sums were read before the first of the two)
            const float s2 = row_sum[g ^ 1][row], l = g ? s2 + sum : sum + s2;
            const float inv = l == 0.f ? 0.f : unscale / l;
            ok = __all_sync(FULL, ok && wait(B_OFINAL, n & 1));
            tc_fence_after();
            uint32_t o[2][32];
            tmem_ld32(lane_base + T_O + 64 * g, o[0]);
            tmem_ld32(lane_base + T_O + 64 * g + 32, o[1]);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_OFREE]);   // the next unit's first product may overwrite O
            const int t = w.q0 + row, h = p.head_off + w.hl;
            if (ok && row < w.rows && __ldcg(p.done + t)) {
                uint32_t *dst = (uint32_t *)(p.out + (t * p.H + h) * 128 + 64 * g);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t wv[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        wv[i] = pack_bf16(__uint_as_float(o[q][2 * i]) * inv, __uint_as_float(o[q][2 * i + 1]) * inv);
                    if (p.out_v8) {
                        st_global_v8(dst + 16 * q, wv);
                        st_global_v8(dst + 16 * q + 8, wv + 8);
                    } else {
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            ((uint4 *)(dst + 16 * q))[v] = make_uint4(wv[4 * v], wv[4 * v + 1], wv[4 * v + 2], wv[4 * v + 3]);
                    }
                }
                if (g == 0) p.lse[t * p.H + h] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
            }
            ++n;
            u = u_next;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*abort) settle();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace

// How many key rows and units there are is known on the device only, so the grids are fixed.
cudaError_t tc_step_prefill(const TcStep &p, cudaStream_t st) {
    using ull = unsigned long long;
    const ull R = p.key_rows, H = p.H, T = p.T, hs = p.hs;
    cudaError_t e;
    CUtensorMap mQn, mQr, mK, mKr, mV, mR;
    {
        const ull d[4] = {128, H, T, 1}, s[3] = {256, H * 256, T * H * 256};
        const unsigned box[4] = {64, 1, 128, 1};
        if ((e = make_tma_map(&mQn, p.q_nope, 4, d, s, box)) != cudaSuccess) return e;
        if ((e = make_tma_map(&mQr, p.qpe, 4, d, s, box)) != cudaSuccess) return e;
    }
    {
        const ull nr = p.rest_rows;
        const ull dr[3] = {64, R, 1}, sr[2] = {128, R * 128}, dk[3] = {hs * 128, R, 1}, sk[2] = {hs * 256, R * hs * 256};
        const ull dv[3] = {R, hs * 128, 1}, sv[2] = {R * 2, R * hs * 256}, de[3] = {hs * 128, nr, 1}, se[2] = {hs * 256, nr * hs * 256};
        const unsigned box[3] = {64, 128, 1};
        if ((e = make_tma_map(&mKr, p.kpe, 3, dr, sr, box)) != cudaSuccess) return e;
        if ((e = make_tma_map(&mK, p.kws, 3, dk, sk, box)) != cudaSuccess) return e;
        if ((e = make_tma_map(&mR, p.rest, 3, de, se, box)) != cudaSuccess) return e;
        if ((e = make_tma_map(&mV, p.vws, 3, dv, sv, box)) != cudaSuccess) return e;
    }
    if ((e = cudaFuncSetAttribute(tc_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S_BYTES)) != cudaSuccess) return e;
    // the register split waits for ever where the launch has fewer to draw on: another compiler's choice is refused
    static std::atomic<int> regs{0};   // (of the kernel: the same from any host thread and device)
    if (regs == 0) {
        cudaFuncAttributes at;
        if ((e = cudaFuncGetAttributes(&at, tc_step_kernel)) != cudaSuccess) return e;
        regs = at.numRegs;
    }
    if (NTHREADS * regs < 128 * (REGS_ISSUE + 2 * REGS_SOFTMAX)) return cudaErrorInvalidConfiguration;
    int dev = 0, n_sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&n_sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    StepK a{};
    a.tiles = p.tiles;
    a.ctl = p.ctl;
    a.limits = p.limits;
    a.done = p.done;
    a.held = p.held;
    a.holes = p.holes;
    a.w_max = p.w_max;
    a.c_max = p.c_max;
    a.scale_log2 = p.scale * 1.4426950408889634f;
    a.out = (__nv_bfloat16 *)p.out;
    a.H = p.H;
    a.out_v8 = ((uintptr_t)p.out % 32) == 0;
    a.lse = p.lse;
    a.idesc_s = a.idesc_pv = idesc_f16(128, 128, true);
    for (int h0 = 0; h0 < p.H; h0 += p.hs) {
        const int nh = std::min(p.hs, p.H - h0);
        // bf16 rows and weights as they are: their products are exact in the fp32 accumulator
        TmaOperand latent{p.chat, 512, (long)R, 1, 1024, (long)R * 1024, (int)R, 0, 1};
        const char *w = (const char *)p.w + (long)h0 * 256 * 1024;
        TmaOperand wk{w, 512, 128, nh, 1024, 256 * 1024, 128, 0, 0}, wv{w + 128 * 1024, 512, 128, nh, 1024, 256 * 1024, 128, 0, 0};
        const GemmProblem kv[2] = {{latent, wk, (int)R, nh * 128, 512, 1, p.kws, (long)hs * 128, 1, 0, 0},
                                   {wv, latent, nh * 128, (int)R, 512, 1, p.vws, (long)R, 1, 0, 0}};
        const GemmStep gs{p.ctl, p.rest_of, p.rest, p.block_of, p.w_max + h0, p.c_max};
        if ((e = tc_gemm_group(kv, 2, false, st, &gs)) != cudaSuccess) return e;
        a.head_off = h0;
        a.nh = nh;
        ProfScope ps("tc_step_attn", st);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(n_sms);
        cfg.blockDim = dim3(NTHREADS);
        cfg.dynamicSmemBytes = S_BYTES;
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // overlap the GEMM's tail
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if ((e = cudaLaunchKernelEx(&cfg, tc_step_kernel, mQn, mQr, mK, mKr, mV, mR, a)) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t tc_step_read_and_clear_error(unsigned *flags, cudaStream_t st) {
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_tc_step_err, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
    if (e != cudaSuccess) return e;
    e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return e;
    if (v) {
        unsigned z = 0;
        e = cudaMemcpyToSymbolAsync(g_tc_step_err, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
        if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    }
    *flags |= v;
    return e;
}

}  // namespace mla
