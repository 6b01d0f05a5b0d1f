// paged_tc.cuh -- device code shared by the tensor-core kernels of the paged cache (paged_tc.cu, paged_many.cu): the
// queries' parts, and what is taken of them.
#pragma once

#include <cuda_bf16.h>

#include "paged_common.cuh"
#include "tc_common.cuh"

namespace mla {
namespace paged {

using bf16 = __nv_bfloat16;
using tc::pack_bf16;
using tc::smem_u32;

constexpr int DK = 512, DN = 128, DR = 64, DV = 128;

__device__ __forceinline__ void cp16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// x as hi + lo in bf16 (hi its rounding, lo the rounding of the rest)
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(x, y);
    lo = pack_bf16(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}
// the same, and what lo leaves
__device__ __forceinline__ void split3(float x, float y, uint32_t &hi, uint32_t &lo, uint32_t &rest) {
    hi = pack_bf16(x, y);
    x -= __uint_as_float(hi << 16);
    y -= __uint_as_float(hi & 0xffff0000u);
    split2(x, y, lo, rest);
}

// What a request's scores and log-sum-exp take of the queries besides q_hi and the band's hi and lo
// (the header's part on precision).
enum Extra { EX_NONE, EX_LATENT, EX_WIDE, EX_BAND };
constexpr int SHORT_KEYS = 64, WIDE_KEYS = 1024, MIDDLE_KEYS = 4096;
__device__ __forceinline__ Extra extra_of(bool paired, int keys) {
    if (keys <= SHORT_KEYS) return EX_BAND;
    return paired || keys > MIDDLE_KEYS ? EX_NONE : (keys > WIDE_KEYS ? EX_LATENT : EX_WIDE);
}
// The blocks of 64 latent dims, as bits, whose q_lo has MMAs of its own above 64 heads (up to 64 all have idle rows).
__device__ __forceinline__ unsigned lo_blocks(Extra ex) {
    return ex == EX_NONE ? 0 : (ex == EX_LATENT ? 0x3 : (ex == EX_WIDE ? 0xf : 0xe));
}

struct Absorb {
    PagedDecode p;
    bf16 *qhi, *qlo, *qrest, *rhi, *rlo, *rrest;   // [B][H][512], [B][H][64]; the rests of short requests only
    int groups, group;             // groups of `group` requests
    int blocks;                    // blocks that share them out, of each head and 128 dims: the groups, but for a list
    int rot_blocks;                // blocks 1 .. rot_blocks rotate the queries; block 0 divides the batch
    Turns64 turns;
};

// The keys of token b's group, for what is done besides where they are few (behind the plan).
__device__ __forceinline__ int group_keys(const PagedDecode &p, int b) {
    const int g = p.scores_only ? -1 : __ldcg(&p.of[b].x);
    return g < 0 ? 2147483647 : keys_of(p, g);
}

// The queries' rotation: a warp per token and 32 heads, a lane per pair of dims, the angle formed once, HB heads'
// loads in flight.  PLANNED: a step's,
// behind its plan.
template <bool STEP, bool PLANNED = false, int HB = 8>
__device__ void rotate_queries(const Absorb &a, int i, int lane) {
    const PagedDecode &p = a.p;
    const int per = (p.H + 31) / 32, b = i / per, h0 = i % per * 32;
    if (b >= (STEP ? tokens_of(p) : p.B)) return;
    const int t = STEP ? token_of(p, b) : b;
    // (a step's tokens may see few keys whatever their position)
    const int keys = !STEP ? keys_of(p, b) : PLANNED ? group_keys(p, b) : p.scores_only ? 2147483647 : 0;
    const float2 cs = turn_cs(a.turns.v[lane], STEP ? p.pos[t] : keys - 1);
    const int h1 = min(h0 + 32, p.H);
#pragma unroll 1
    for (int h = h0; h < h1; h += HB) {
        uint16_t x0[HB], x1[HB];
#pragma unroll
        for (int j = 0; j < HB; ++j) {
            const uint16_t *x = (const uint16_t *)p.q_pe + ((long)t * p.H + min(h + j, h1 - 1)) * DR + lane;
            x0[j] = x[0];
            x1[j] = x[32];
        }
#pragma unroll
        for (int j = 0; j < HB; ++j) {
            if (h + j >= h1) break;
            const long o = ((long)b * p.H + h + j) * DR + lane;
            const float f0 = __uint_as_float((uint32_t)x0[j] << 16), f1 = __uint_as_float((uint32_t)x1[j] << 16);
            uint32_t hi, lo, rest;
            split3(f0 * cs.x - f1 * cs.y, f1 * cs.x + f0 * cs.y, hi, lo, rest);
            ((uint16_t *)a.rhi)[o] = (uint16_t)hi;
            ((uint16_t *)a.rhi)[o + 32] = (uint16_t)(hi >> 16);
            ((uint16_t *)a.rlo)[o] = (uint16_t)lo;
            ((uint16_t *)a.rlo)[o + 32] = (uint16_t)(lo >> 16);
            if (keys <= SHORT_KEYS) {
                ((uint16_t *)a.rrest)[o] = (uint16_t)rest;
                ((uint16_t *)a.rrest)[o + 32] = (uint16_t)(rest >> 16);
            }
        }
    }
}

}  // namespace paged

// The absorb and the join of many tokens (paged_many.cu); the first behind launch_paged_plan.
cudaError_t paged_absorb_many(const paged::Absorb &ab, cudaStream_t st);
cudaError_t paged_join_many(const PagedDecode &p, const __nv_bfloat16 *qlo, const __nv_bfloat16 *qrest, cudaStream_t st);

}  // namespace mla
