// paged_step.cu -- a serving step's tokens over the paged latent cache: which tokens share a work item, and
// the division of the items among the workers.
#include <algorithm>

#include "paged_common.cuh"
#include "tc_common.cuh"

namespace mla {

using namespace paged;
using tc::pdl_launch_dependents;
using tc::pdl_wait;

namespace {

// -------------------------------------------------------------------------- plan ----
// Block 0, two tokens a thread: a token's request by binary search of the prefix sums, the keys that
// it sees; groups begin where a request's tokens do, where one is not computed here, and after every
// `most` tokens; then the groups' tile sums and the workers' parts as for decode.
constexpr int PNT = 1024, CU_NEAR = 4096;

struct Plan {
    PagedDecode p;
    PagedStep s;
    int s0, most;   // first token of the round; tokens of a group at most
    int *lens, *limits;
    int2 *of;
    int4 *groups;
    unsigned long long *zero;
    long n_zero;
};

__global__ void __launch_bounds__(PNT) paged_plan_kernel(const __grid_constant__ Plan a) {
    extern __shared__ int sm[];
    __shared__ int warp_tot[PNT / 32];
    const PagedDecode &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
    int *lim = sm, *req = lim + PAGED_ROUND, *sums = req + PAGED_ROUND, *near = sums + PAGED_ROUND + 1;
    pdl_wait();
    pdl_launch_dependents();   // the absorb beside this; what follows it waits for both
    if (blockIdx.x > 0) {
        for (long i = (long)(blockIdx.x - 1) * PNT + tid; i < a.n_zero; i += (long)(gridDim.x - 1) * PNT) a.zero[i] = 0;
        return;
    }
    const bool here = a.s.B < CU_NEAR;
    if (here) {
        for (int i = tid; i <= a.s.B; i += PNT) near[i] = a.s.cu[i];
        __syncthreads();
    }
    const int *cu = here ? near : a.s.cu;
    const int cap = p.max_pages * p.page;
    for (int i = tid; i < p.T; i += PNT) {
        const int t = a.s0 + i;
        int lo = 0, hi = a.s.B;   // the first request whose tokens end behind t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid + 1] > t) hi = mid;
            else lo = mid + 1;
        }
        const bool in = lo < a.s.B && cu[lo] <= t && !(p.done && p.done[i]);
        req[i] = in ? lo : -1;
        int n = 0;
        if (in) {
            const int pos = a.s.positions[t], keys = min(max(a.s.lens[lo], 0), cap);
            n = pos < 0 ? 0 : min(keys, pos == 2147483647 ? pos : pos + 1);
        }
        lim[i] = a.limits[i] = n;
    }
    __syncthreads();
    // which tokens begin a group
    const int i0 = 2 * tid;
    int first[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = i0 + e;
        first[e] = 0;
        if (i < p.T && req[i] >= 0)
            first[e] = i == 0 || req[i - 1] != req[i] || (a.s0 + i - max(cu[req[i]], a.s0)) % a.most == 0;
    }
    int x = first[0] + first[1];
    const int own = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_tot[wp] = x;
    __syncthreads();
    int g = x - own, all = 0;
#pragma unroll
    for (int i = 0; i < PNT / 32; ++i) {
        if (i < wp) g += warp_tot[i];
        all += warp_tot[i];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = i0 + e;
        if (i >= p.T) continue;
        if (req[i] < 0) a.of[i] = make_int2(-1, 0);
        if (!first[e]) continue;
        // the group's tokens: up to the next beginning
        const int b = req[i], in_request = a.s0 + i - max(cu[b], a.s0);
        int n = 0, most = 0;
        for (int k = i; k < p.T && req[k] == b && (k == i || (in_request + k - i) % a.most); ++k, ++n) {
            a.of[k] = make_int2(g, n * p.H);
            most = max(most, lim[k]);
        }
        a.groups[g] = make_int4(b, i * p.H, n * p.H, 0);
        a.lens[g] = most;
        ++g;
    }
    for (int i = all + tid; i < p.B; i += PNT) {
        a.lens[i] = 0;
        a.groups[i] = make_int4(0, 0, 0, 0);
    }
    __syncthreads();
    if (p.parts) plan_block<PNT>(p, sums, PAGED_ROUND + 1);
    else plan_block<PNT>(p);
}

}  // namespace

cudaError_t launch_paged_plan(const PagedDecode &p, const PagedStep &s, int s0, int *lens, int2 *of, int *limits, int4 *groups,
                              cudaStream_t st, unsigned long long *zero, long n_zero) {
    Plan a{p, s, s0, std::max(1, p.row_tile / p.H), lens, limits, of, groups, zero, n_zero};
    const size_t sm = (3 * PAGED_ROUND + 1 + (s.B < CU_NEAR ? s.B + 1 : 0)) * sizeof(int);
    ProfScope ps("paged_plan", st);
    return launch_after(paged_plan_kernel, 1 + (unsigned)std::min((n_zero + PNT - 1) / PNT, 150l), PNT, sm, st, a);
}

}  // namespace mla
