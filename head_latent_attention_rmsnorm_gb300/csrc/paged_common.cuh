// paged_common.cuh -- device code shared by the paged-cache kernels: rotation angles, the
// division of a ragged batch among workers, element access.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <utility>

#include "mla_internal.h"
#include "paged.h"

namespace mla {
namespace paged {

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// RoPE angles in turns, as 64-bit fixed point: frequency t turns base^(-2t/Dr) / (2 pi) per
// position, kept modulo one turn in 64 bits.  pos * turns modulo 2^64 is then the angle's exact
// fraction of a turn (to pos * 2^-53 of the frequency's own rounding), at any 32-bit position and
// without a double-precision operation on the device.
constexpr int MAX_HALF = 320;   // d_rope <= 640
template <int N>
struct TurnsOf {
    unsigned long long v[N];
};
using Turns = TurnsOf<MAX_HALF>;
using Turns64 = TurnsOf<32>;    // d_rope <= 64: a tenth of the launch's parameters
__device__ __forceinline__ float2 turn_cs(unsigned long long turns, int pos) {
    const long long x = (long long)(turns * (unsigned long long)(long long)pos);
    float s, c;
    sincospif((float)(int)(x >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31 half turns
    return make_float2(c, s);
}

// x / d for 0 <= x < 2^31 by a multiplication (round-up multiplier, Granlund and Montgomery 1994; the sum cannot
// overflow, as the high product is at most x).
struct Divisor {
    uint32_t mul, shift;
};
__device__ __forceinline__ int quotient(const Divisor &d, int x) {
    return (int)((__umulhi(d.mul, (uint32_t)x) + (uint32_t)x) >> d.shift);
}
inline Divisor divisor(int d) {
    Divisor r{0, 0};
    while ((1u << r.shift) < (unsigned)d) ++r.shift;
    r.mul = (uint32_t)((((unsigned long long)1 << 32) * (((unsigned long long)1 << r.shift) - d)) / d + 1);
    return r;
}

// Tiles of a worker's share of T: worker c takes [c q, (c + 1) q).  Whole tiles, the same for all but the
// last, so that shares end where requests do as often as they can (a request's last part and the
// next one's first in one share cost some 5 us more than a tile each: 16 requests of 1000 keys went
// from 31 to 27 us against shares of T / W).
__device__ __forceinline__ long share_of(const PagedDecode &p, long T) {
    const long q = (T + p.workers - 1) / p.workers;
    return q > p.min_tiles ? q : p.min_tiles;
}

// A group's keys (decode: a request's): its length cut to what a table row can hold.
__device__ __forceinline__ int keys_of(const PagedDecode &p, int b) {
    const int cap = p.max_pages * p.page;   // checked to fit by the caller
    return min(max(p.lens[b], 0), cap);
}

// The tokens of the call, and token i's row in the step.
__device__ __forceinline__ int tokens_of(const PagedDecode &p) {
    return p.list ? min(max(__ldcg(p.n_list) - p.list_at, 0), p.T) : p.T;
}
__device__ __forceinline__ int token_of(const PagedDecode &p, int i) { return p.list ? __ldcg(p.list + i) : i; }

// The group whose tiles (for all its row tiles) hold tile t < T; `off`: the prefix sums.
template <typename I>
__device__ __forceinline__ int request_of(const PagedDecode &p, const I *off, long t) {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {   // the last b whose first tile is <= t: empty groups before it share that tile
        const int mid = (lo + hi + 1) >> 1;
        if ((long)off[mid] * p.row_tiles <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The parts begin where a worker's share begins and where an item does (one may be both): a thread per
// beginning finds its part's worker, item and end.
template <int NT, bool STEP, typename I>
__device__ void plan_parts(const PagedDecode &p, const I *off, long total) {
    const long q = share_of(p, total);
    const long items = (long)p.B * p.row_tiles;
#pragma unroll 1
    for (long k = threadIdx.x; k < p.workers + items; k += NT) {
        const bool worker = k < p.workers;
        long t0 = 0;
        int b = 0, c = (int)k, rt = 0;
        if (worker) {
            if (c * q >= total) {
                p.first[c] = p.first[p.workers + c] = 0;
                continue;
            }
            t0 = c * q;
            b = request_of(p, off, t0);
        } else {
            b = (int)((k - p.workers) / p.row_tiles);
            rt = (int)((k - p.workers) % p.row_tiles);
        }
        const long o = off[b], per = off[b + 1] - o;
        if (per == 0) {
            p.spans[k - p.workers] = make_int2(0, 0);
            continue;
        }
        if (worker) {
            rt = (int)((t0 - o * p.row_tiles) / per);
        } else {
            t0 = o * p.row_tiles + rt * per;
            c = (int)(t0 / q);
            p.spans[k - p.workers] = make_int2(c + (int)(k - p.workers), (int)((t0 + per - 1) / q) - c + 1);
        }
        const long i0 = o * p.row_tiles + rt * per, i1 = i0 + per, end = min((c + 1) * q, total), t1 = min(end, i1);
        const int item = b * p.row_tiles + rt;
        const int4 g = STEP ? p.groups[b] : make_int4(b, b * p.H, p.H, 0);
        PagedPart x{};
        x.row = g.x;
        x.q = g.y + rt * p.row_tile;
        x.rows = min(g.z - rt * p.row_tile, p.row_tile);
        x.k0 = (int)(t0 - i0);
        x.nt = (int)(t1 - t0);
        x.keys = keys_of(p, b);
        if (t1 < end) {   // the worker goes on with the next item that has tiles
            x.next = 1;
            if (rt == p.row_tiles - 1)
                for (int e = b + 1; off[e + 1] == off[e]; ++e) x.next += p.row_tiles;
        }
        p.parts[c + item] = x;
        if (worker) {
            p.first[c] = c + item;
            p.first[p.workers + c] = (int)(end - t0);
        }
    }
}

// The tile prefix sums of all groups and the workers' parts, by one block of NT threads; `room`
// ints of shared memory keep the sums at hand where they fit.
template <int NT, bool STEP>
__device__ void plan_block(const PagedDecode &p, int *sm = nullptr, int room = 0) {
    __shared__ long warp_tot[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
    const bool near = p.B < room && (long)p.B * ((p.max_pages * (long)p.page + p.tile - 1) / p.tile) < 1l << 31;
    long carry = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += NT) {
        const int b = b0 + tid;
        const long n = b < p.B ? (keys_of(p, b) + p.tile - 1) / p.tile : 0;
        long x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warp_tot[wp] = x;
        __syncthreads();
        long before = carry, all = carry;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) {
            if (i < wp) before += warp_tot[i];
            all += warp_tot[i];
        }
        if (b < p.B) {
            if (near) sm[b] = (int)(before + x - n);
            else p.tile_off[b] = before + x - n;
        }
        carry = all;
        __syncthreads();
    }
    if (tid == 0) {
        if (near) sm[p.B] = (int)carry;
        else p.tile_off[p.B] = carry;
    }
    if (!p.parts) return;
    __syncthreads();
    if (near) plan_parts<NT, STEP>(p, sm, carry * p.row_tiles);
    else plan_parts<NT, STEP>(p, p.tile_off, carry * p.row_tiles);
}

// ------------------------------------------------------------------ plan of a step ----
// A block of NT threads, PER tokens each: a token's request by binary search of the prefix sums, the keys that it
// sees; groups begin where a request's tokens do and after every `most` tokens; then the groups' tile sums and
// the workers' parts as for decode.  `sm`: plan_ints(NT PER, B) ints.
constexpr int CU_NEAR = 4096;   // requests whose prefix sums are kept at hand
inline size_t plan_ints(int most, int B) { return 4 * (size_t)most + 1 + (B < CU_NEAR ? B + 1 : 0); }

template <int NT, int PER>
__device__ void plan_tokens(const PagedDecode &p, const PagedPlan &a, int T, int *sm) {
    __shared__ int warp_tot[NT / 32];
    constexpr int MOST = NT * PER;
    const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
    int *lim = sm, *req = lim + MOST, *sums = req + MOST, *tok = sums + MOST + 1, *near = tok + MOST;
    const bool here = a.s.B < CU_NEAR;
    if (here) {
        for (int i = tid; i <= a.s.B; i += NT) near[i] = a.s.cu[i];
        __syncthreads();
    }
    const int *cu = here ? near : a.s.cu;
    const int cap = p.max_pages * p.page;
    for (int i = tid; i < T; i += NT) {
        const int t = p.list ? __ldcg(p.list + i) : a.s0 + i;
        int lo = 0, hi = a.s.B;   // the first request whose tokens end behind t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid + 1] > t) hi = mid;
            else lo = mid + 1;
        }
        const bool in = lo < a.s.B && cu[lo] <= t;
        req[i] = in ? lo : -1;
        tok[i] = t;
        int n = 0;
        if (in) {
            const int pos = a.s.positions[t], keys = min(max(a.s.lens[lo], 0), cap);
            n = pos < 0 ? 0 : min(keys, pos == 2147483647 ? pos : pos + 1);
        }
        lim[i] = a.limits[i] = n;
    }
    __syncthreads();
    // which tokens begin a group
    const int i0 = PER * tid;
    int first[PER], place[PER];   // place: among the request's tokens of this round
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const int i = i0 + e;
        first[e] = place[e] = 0;
        if (i >= T || req[i] < 0) continue;
        int lo = 0, hi = i;   // the request's first token here
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (tok[mid] >= cu[req[i]]) hi = mid;
            else lo = mid + 1;
        }
        place[e] = i - lo;
        first[e] = i == 0 || req[i - 1] != req[i] || place[e] % a.most == 0;
    }
    int own = 0;
#pragma unroll
    for (int e = 0; e < PER; ++e) own += first[e];
    int x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_tot[wp] = x;
    __syncthreads();
    int g = x - own, all = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        if (i < wp) g += warp_tot[i];
        all += warp_tot[i];
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const int i = i0 + e;
        if (i >= T) continue;
        if (req[i] < 0) a.of[i] = make_int2(-1, 0);
        if (!first[e]) continue;
        // the group's tokens: up to the next beginning
        const int b = req[i];
        int n = 0, most = 0;
        for (int k = i; k < T && req[k] == b && (k == i || (place[e] + k - i) % a.most); ++k, ++n) {
            a.of[k] = make_int2(g, n * p.H);
            most = max(most, lim[k]);
        }
        a.groups[g] = make_int4(b, i * p.H, n * p.H, 0);
        a.lens[g] = most;
        ++g;
    }
    for (int i = all + tid; i < p.B; i += NT) {
        a.lens[i] = 0;
        a.groups[i] = make_int4(0, 0, 0, 0);
    }
    __syncthreads();
    if (p.parts) plan_block<NT, true>(p, sums, MOST + 1);
    else plan_block<NT, true>(p);
}

// Started early, behind the kernel in front of it (programmatic dependent launch): the kernel waits for that one's
// end before it touches memory (pdl_wait).  Against plain launches a call that the GPU bounds took 2.7 us
// less back to back (one request of 4096 keys, 128 heads: 32.8 -> 30.0 us), a small kernel in a graph 0.2-0.6.
template <typename... Par, typename... Arg>
cudaError_t launch_after(void (*kern)(Par...), unsigned grid, unsigned block, size_t smem, cudaStream_t st, Arg &&...arg) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Arg>(arg)...);
}

}  // namespace paged

// The frequencies for one base and width (host), kept for the next call of the thread with the same two.
const unsigned long long *paged_turns(float base, int Dr);

}  // namespace mla
