// A mixture-of-experts layer for 1 to 64 tokens in one kernel:
//   l = x·Wr, p = softmax(l), the top_k experts of each token,
//   h_e = act(x·Wgate_e) ⊙ (x·Wup_e),  y = Σ_j w_j·(h_{e_j}·Wdown_{e_j}) (+ R)
// with expert weights in bf16 (row-major, as the library's B operands) or in
// packed 4-bit chunks.
//
// Bound by the weights of the experts that were chosen, each read once however
// many tokens chose it: 1 token, 2 of 8 bf16 experts of 4096x14336, 119 us, 5.9 TB/s (87%
// of a copy); 64 tokens, 4 of 32 of 4096x2048, 298 us, 5.4 TB/s; 16 tokens, 8 of 64 4-bit
// experts, 198 us, 3.8 TB/s (the multiplications and conversions of 4-bit steps, not the
// memory, bound that one).  Small layers are bound by the chain of phases: 1 token, 8 of
// 64 of 2048x1024, takes 38 us for 15 us of weights.  One cooperative launch, one CTA to
// an SM, three phases:
//   route   the router product, split over token groups of 8 and slices of H.  Up to 8
//           tokens all CTAs then wait for one another, and each adds the slices and picks
//           the experts for itself; above, the slice of a token group that arrives last
//           does so for all, and then they wait;
//   up      for each chosen expert, tiles of 64 features (64 gate and 64 up
//           columns) by H, on the tokens that chose it; h in bf16;
//   down    tiles of 128 columns of y, each reducing over the intermediate
//           features of all chosen experts in turn.
// The steps of each phase (tile by tile, along K within one) divide evenly over the
// CTAs; the pieces of a cut tile are added in K order by the CTA that arrives last.
// Between up and down all CTAs wait for one another again; the copying warp
// does not: weights of the down phase fill its ring meanwhile, only the copies
// of h follow the wait.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "few_token.cuh"

namespace gemmgb {
namespace {

// Shared-memory tables of the routing (off_route).
struct RouteTables {
    unsigned long long mask[kMoeMaxExperts];   // tokens of each expert
    int32_t offset[kMoeMaxExperts];            // first of its rows in h
    int32_t act_expert[kMoeMaxExperts];        // experts chosen by any token, ascending
    int32_t act_count[kMoeMaxExperts];
    // The down phase's runs of a tile: an expert's rows, at most moe_down_tokens of them.
    int32_t down_expert[kMoeMaxRuns];
    uint16_t down_offset[kMoeMaxRuns], down_count[kMoeMaxRuns];
    float weight[kMoeMaxPairs];                // by row of h
    uint8_t token[kMoeMaxPairs];
    FtShare up, down;                          // how the two phases divide
    int32_t n_active, n_down;
    int32_t last;                              // this CTA's slice was the last of its token group
};

__device__ __forceinline__ void fence_proxy_async_all()
{
    asm volatile("fence.proxy.async;" ::: "memory");
}

// The CTAs' meeting points.  Every launch adds a whole number of times gridDim.x
// arrivals to a count that only grows, so the count read before this CTA's first
// arrival lies less than gridDim.x above the launch's own start, a multiple of it.
__device__ __forceinline__ void grid_arrive(int32_t *ctl)
{
    atom_acq_rel_gpu_add_u64(reinterpret_cast<uint64_t *>(ctl + 2), 1);
}

__device__ __forceinline__ uint64_t grid_start(const int32_t *ctl)
{
    uint64_t v;
    asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(ctl + 2) : "memory");
    return v - v % gridDim.x;
}

// Bounded wait until all CTAs have arrived `n` times since `start`.
__device__ __noinline__ bool grid_wait(const int32_t *ctl, uint64_t start, int n, const WaitCtl &c)
{
    const uint64_t target = start + (uint64_t)n * gridDim.x;
    const long long limit = (long long)((double)c.timeout_ns * 2.2);
    const long long t0 = clock64();
    for (uint32_t it = 1;; ++it) {
        if (ld_acquire_gpu_u64(reinterpret_cast<const uint64_t *>(ctl + 2)) >= target) return true;
        if ((it & 63u) == 0) {
            if (*c.abort) return false;
            if (clock64() - t0 > limit) {
                *c.abort = 1;
                atomicCAS(c.status, 0, SITE_FIXUP);
                return false;
            }
        }
    }
}

// A logit as an unsigned key in the order of its value, equal for -0 and +0, NaN
// above all.
__device__ __forceinline__ uint32_t rank_key(float v)
{
    v += 0.0f;
    const uint32_t b = __float_as_uint(v);
    return v != v ? 0xFFFFFFFFu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// out[0..n) = the slices' sums of the logits from `at` on.  Where there are fewer
// numbers than workers, several workers take a share of the slices each (scratch:
// one word a worker); always the same order of additions.
__device__ __forceinline__ void add_slices(const MoeParams &p, int64_t at, int n, float *out, float *scratch, int tid,
                                           int workers)
{
    constexpr int kAtOnce = 8;
    const int slices = p.route_slices;
    const int64_t slice = (int64_t)p.T * p.E;
    const int shares = n < workers ? min(workers / n, (slices + kAtOnce - 1) / kAtOnce) : 1;
    const int each = (slices + shares - 1) / shares;
    for (int i = tid; i < n * shares; i += workers) {
        const int k = i % n, q0 = i / n * each, q1 = min(slices, q0 + each);
        float v = 0.0f;
        for (int q = q0; q < q1; q += kAtOnce) {
            float part[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) part[u] = __ldcg(p.logits + (int64_t)min(q + u, q1 - 1) * slice + at + k);
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) v += q + u < q1 ? part[u] : 0.0f;
        }
        if (shares == 1) out[k] = v;
        else scratch[i] = v;
    }
    named_bar_sync(1, workers);
    if (shares > 1) {
        for (int k = tid; k < n; k += workers) {
            float v = 0.0f;
            for (int s = 0; s < shares; ++s) v += scratch[s * n + k];
            out[k] = v;
        }
        named_bar_sync(1, workers);
    }
}

// The choice of nt tokens from their logits [nt][E] in shared memory, by all
// workers: an expert's rank is the number of experts before it (a larger logit, or
// an equal one of a lower index), and the first top_k ranks are the choice.
// keys: [nt][E] words of scratch; ids and weights: [nt][top_k] in shared memory.
__device__ __forceinline__ void choose_tokens(const MoeParams &p, float *logits, uint32_t *keys, int nt, int32_t *ids,
                                              float *weights, int tid, int workers)
{
    const int n = nt * p.E, pairs = nt * p.top_k;
    for (int i = tid; i < n; i += workers) keys[i] = rank_key(logits[i]);
    named_bar_sync(1, workers);
    for (int i = tid; i < n; i += workers) {
        const int t = i / p.E, e = i - t * p.E;
        const uint32_t *const row = keys + t * p.E;
        const uint32_t k = row[e];
        int rank = 0;
#pragma unroll 8
        for (int o = 0; o < p.E; ++o) rank += (int)(row[o] > k) | ((int)(row[o] == k) & (int)(o < e));
        if (rank < p.top_k) ids[t * p.top_k + rank] = e;
    }
    named_bar_sync(1, workers);
    if (!p.normalize) {   // every expert's exponential, for the sum over all
        for (int i = tid; i < n; i += workers) {
            const int t = i / p.E;
            keys[i] = __float_as_uint(expf(logits[i] - logits[t * p.E + ids[t * p.top_k]]));
        }
        named_bar_sync(1, workers);
    }
    for (int i = tid; i < pairs; i += workers) {
        const int t = i / p.top_k;
        const int32_t *const mine = ids + t * p.top_k;
        const float *const l = logits + t * p.E;
        const float top = l[mine[0]];
        float d = 0.0f;
        if (p.normalize)
            for (int j = 0; j < p.top_k; ++j) d += expf(l[mine[j]] - top);
        else
#pragma unroll 8
            for (int o = 0; o < p.E; ++o) d += __uint_as_float(keys[t * p.E + o]);
        weights[i] = __fdiv_rn(expf(l[ids[i]] - top), d);
    }
    named_bar_sync(1, workers);
}

// The router product, a unit (8 tokens, a slice of H) at a time, into the
// workspace; with route_reduce the CTA whose slice comes last adds a token group's
// slices and chooses its experts.  All W workers; the scratch lies in the ring,
// before any copy is in flight.
template <int W>
__device__ __forceinline__ void route(const MoeParams &p, uint8_t *scratch, RouteTables *rt, int tid)
{
    const int groups = (p.T + 7) / 8, units = groups * p.route_slices;
    int ep = 8;                                    // experts a pass of the threads covers, a power of two
    while (ep < p.E && ep < W) ep *= 2;
    const int hgs = W / ep, e = tid % ep, hg = tid / ep;
    const bool adds = hg < hgs;                    // W need not be a power of two
    float *const sums = reinterpret_cast<float *>(scratch);          // [hgs][8][ep]
    float *const xs = sums + W * 8;                                  // [rows][8]
    __nv_bfloat16 *const ws = reinterpret_cast<__nv_bfloat16 *>(xs + kRouteRows * 8);   // [rows][E], a part of the slice
    const int rows_at_once = min(kRouteRows, kRouteWeightBytes / (2 * p.E) / 8 * 8);
    const __nv_bfloat16 *const x = static_cast<const __nv_bfloat16 *>(p.x);
    const __nv_bfloat16 *const wr = static_cast<const __nv_bfloat16 *>(p.router);
    const int64_t slice = (int64_t)p.T * p.E;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const int tg = u / p.route_slices, sl = u % p.route_slices;
        const int t0 = tg * 8, nt = min(8, p.T - t0);
        const int h0 = sl * p.route_rows, nh = max(0, min(p.H - h0, p.route_rows));   // multiples of 8
        float s[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) s[t] = 0.0f;
        for (int r0 = 0; r0 < nh; r0 += rows_at_once) {
            const int nr = min(rows_at_once, nh - r0);
            // Rows of the router weight are one contiguous piece.
            const uint8_t *const src = reinterpret_cast<const uint8_t *>(wr + (int64_t)(h0 + r0) * p.E);
            for (int i = tid; i < nr * p.E / 8; i += W) cp_async_16(smem_u32(ws) + (uint32_t)i * 16u, src + (int64_t)i * 16);
            for (int i = tid; i < nr; i += W) {    // 8 tokens side by side in shared memory
                const int t = i & 7, h = i >> 3;
                const uint4 v = t < nt ? __ldg(reinterpret_cast<const uint4 *>(x + (int64_t)(t0 + t) * p.H + h0 + r0 + h * 8))
                                       : make_uint4(0, 0, 0, 0);
                const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    xs[(h * 8 + 2 * k) * 8 + t] = bf16_lo(q[k]);
                    xs[(h * 8 + 2 * k + 1) * 8 + t] = bf16_hi(q[k]);
                }
            }
            cp_async_commit_wait_all();
            named_bar_sync(1, W);
            if (adds && e < p.E) {
#pragma unroll 4
                for (int h = hg; h < nr; h += hgs) {
                    const float w = __bfloat162float(ws[h * p.E + e]);
                    const float4 a = *reinterpret_cast<const float4 *>(xs + h * 8);
                    const float4 b = *reinterpret_cast<const float4 *>(xs + h * 8 + 4);
                    s[0] = fmaf(a.x, w, s[0]), s[1] = fmaf(a.y, w, s[1]), s[2] = fmaf(a.z, w, s[2]);
                    s[3] = fmaf(a.w, w, s[3]), s[4] = fmaf(b.x, w, s[4]), s[5] = fmaf(b.y, w, s[5]);
                    s[6] = fmaf(b.z, w, s[6]), s[7] = fmaf(b.w, w, s[7]);
                }
            }
            named_bar_sync(1, W);
        }
        if (adds) {
#pragma unroll
            for (int t = 0; t < 8; ++t) sums[(hg * 8 + t) * ep + e] = s[t];
        }
        named_bar_sync(1, W);
        for (int i = tid; i < nt * ep; i += W) {
            const int t = i / ep, ee = i % ep;
            if (ee >= p.E) continue;
            float v = 0.0f;
            for (int q = 0; q < hgs; ++q) v += sums[(q * 8 + t) * ep + ee];
            __stcg(p.logits + sl * slice + (int64_t)(t0 + t) * p.E + ee, v);
        }
        named_bar_sync(1, W);
        if (!p.route_reduce) continue;
        if (tid == 0) {
            const int before = atom_acq_rel_gpu_add(p.ctl + 8 + tg, 1);
            rt->last = before == p.route_slices - 1;
            if (before == p.route_slices - 1) p.ctl[8 + tg] = 0;
        }
        named_bar_sync(1, W);
        if (!rt->last) continue;
        // [8][E] logits and keys, [8][top_k] ids and weights over the staged weight.
        float *const logits = reinterpret_cast<float *>(ws);
        uint32_t *const keys = reinterpret_cast<uint32_t *>(logits + 8 * p.E);
        int32_t *const ids = reinterpret_cast<int32_t *>(keys + 8 * p.E);
        float *const weights = reinterpret_cast<float *>(ids + 8 * p.top_k);
        add_slices(p, (int64_t)t0 * p.E, nt * p.E, logits, sums, tid, W);
        choose_tokens(p, logits, keys, nt, ids, weights, tid, W);
        for (int i = tid; i < nt * p.top_k; i += W) {
            const int at = t0 * p.top_k + i;
            __stcg(p.ids + at, ids[i]);
            __stcg(p.weights + at, weights[i]);
            if (p.ids_out) p.ids_out[at] = ids[i];
            if (p.weights_out) p.weights_out[at] = weights[i];
        }
        named_bar_sync(1, W);
    }
}

// ids[T][top_k] and weights in shared memory: the caller's, or those chosen during
// route, or (few tokens) by every CTA for itself from the slices' sums, which saves
// a trip through global memory; one CTA a token then writes the caller's arrays.
template <int W>
__device__ __forceinline__ void choose(const MoeParams &p, float *logits, int32_t *ids, float *weights, int tid)
{
    const int pairs = p.T * p.top_k;
    if (p.routed || p.route_reduce) {
        const int32_t *const from = p.routed ? p.ids_in : p.ids;
        const float *const wfrom = p.routed ? p.weights_in : p.weights;
        for (int i = tid; i < pairs; i += W) ids[i] = __ldcg(from + i), weights[i] = __ldcg(wfrom + i);
    } else {
        uint32_t *const keys = reinterpret_cast<uint32_t *>(weights + pairs);
        add_slices(p, 0, p.T * p.E, logits, reinterpret_cast<float *>(keys), tid, W);
        choose_tokens(p, logits, keys, p.T, ids, weights, tid, W);
        for (int i = tid; i < pairs; i += W)
            if (i / p.top_k % gridDim.x == blockIdx.x) {
                if (p.ids_out) p.ids_out[i] = ids[i];
                if (p.weights_out) p.weights_out[i] = weights[i];
            }
    }
    named_bar_sync(1, W);
}

// Tables of the chosen experts, from ids and weights in shared memory.  An id
// outside [0, E) is an empty place; a second mention of an expert by the same
// token adds its weight to the first.
template <int W, int DOWN>
__device__ __forceinline__ void build_tables(const MoeParams &p, RouteTables *rt, const int32_t *ids, const float *wts,
                                             int tid)
{
    const int pairs = p.T * p.top_k;
    for (int e = tid; e < p.E; e += W) rt->mask[e] = 0;
    named_bar_sync(1, W);
    for (int i = tid; i < pairs; i += W) {
        const int id = ids[i];
        if (id >= 0 && id < p.E) atomicOr(&rt->mask[id], 1ull << (i / p.top_k));
    }
    named_bar_sync(1, W);
    if (tid < 32) {
        int rows = 0, active = 0, runs = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + tid;
            const int n = e < p.E ? __popcll(rt->mask[e]) : 0;
            const int parts = (n + DOWN - 1) / DOWN;
            int incl = n | parts << 16;            // rows and runs before, side by side
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (tid >= o) incl += v;
            }
            const int first = rows + (incl & 0xFFFF) - n;
            const uint32_t used = __ballot_sync(0xFFFFFFFFu, n > 0);
            if (e < p.E) rt->offset[e] = first;
            for (int i = 0; i < parts; ++i) {
                const int a = runs + (incl >> 16) - parts + i;
                rt->down_expert[a] = e;
                rt->down_offset[a] = (uint16_t)(first + i * DOWN);
                rt->down_count[a] = (uint16_t)min(DOWN, n - i * DOWN);
            }
            if (n > 0) {
                const int a = active + __popc(used & ((1u << tid) - 1u));
                rt->act_expert[a] = e;
                rt->act_count[a] = n;
            }
            const int all = __shfl_sync(0xFFFFFFFFu, incl, 31);
            rows += all & 0xFFFF, runs += all >> 16;
            active += __popc(used);
        }
        if (tid == 0) {
            rt->n_active = active, rt->n_down = runs;
            // Step by step: even shares at staggered places of the weights.
            rt->up = ft_share_of((int64_t)active * p.tiles_up, p.nkb_up, 1, gridDim.x);
            rt->down = ft_share_of(p.tiles_down, runs * p.nkb_down, 1, gridDim.x);
        }
    }
    named_bar_sync(1, W);
    for (int i = tid; i < pairs; i += W) {
        const int t = i / p.top_k, j0 = t * p.top_k, id = ids[i];
        if (id < 0 || id >= p.E) continue;
        float w = wts[i];
        bool first = true;
        for (int j = j0; j < j0 + p.top_k; ++j)
            if (j != i && ids[j] == id) {
                if (j < i) first = false;
                else w += wts[j];
            }
        if (!first) continue;
        const int row = rt->offset[id] + __popcll(rt->mask[id] & ((1ull << t) - 1ull));
        rt->token[row] = (uint8_t)t;
        rt->weight[row] = w;
    }
}

// A CTA's share of a phase as runs of steps on one tile and expert: in the up phase
// expert by expert, tile by tile; in the down phase tile by tile, expert by expert (an
// expert of many tokens in several runs).
// (Divides once: a 64-bit division for every run took as long as a step.)
struct Runs {
    int a, tile, k, left;   // place in the tables, tile, first K step; steps from here on
    int nkb, na, nt;
    bool up;
    __device__ __forceinline__ Runs(const MoeParams &p, const RouteTables *rt, bool up_) : up(up_)
    {
        const FtShare &sh = up ? rt->up : rt->down;
        nkb = up ? p.nkb_up : p.nkb_down, na = up ? rt->n_active : rt->n_down, nt = p.tiles_up;
        a = tile = k = left = 0;
        if ((int)blockIdx.x >= sh.parts) return;
        const int64_t s0 = ft_share_begin(sh, blockIdx.x), run = s0 / nkb;
        left = (int)(ft_share_begin(sh, blockIdx.x + 1) - s0);
        k = (int)(s0 % nkb);
        a = (int)(up ? run / nt : run % na), tile = (int)(up ? run % nt : run / na);
    }
    __device__ __forceinline__ int steps() const { return min(nkb - k, left); }
    // The run's rows of h.
    __device__ __forceinline__ int count(const RouteTables *rt) const { return up ? rt->act_count[a] : rt->down_count[a]; }
    __device__ __forceinline__ int offset(const RouteTables *rt) const
    {
        return up ? rt->offset[rt->act_expert[a]] : rt->down_offset[a];
    }
    __device__ __forceinline__ void next()
    {
        left -= steps();
        k = 0;
        if (up) {
            if (++tile == nt) tile = 0, ++a;
        } else {
            if (++a == na) a = 0, ++tile;
        }
    }
};

// Where a row of a tile of expert `expert` lies in its packed weight (ft_resolve).
__device__ __forceinline__ const uint8_t *moe_chunk(const MoeParams &p, bool up, int expert, int tile, int row, uint32_t &step,
                                                    uint32_t &where)
{
    const int ncg = up ? p.ncg_up : p.ncg_down, nkb = up ? p.nkb_up : p.nkb_down;
    step = (uint32_t)(min(4, ncg - 4 * tile) * p.chunk_bytes);
    where = (uint32_t)(row & 31) | (uint32_t)p.gpc << 5 | (uint32_t)p.has_zeros << 9;
    return (up ? p.gate_up : p.down) +
           ((int64_t)expert * ncg * nkb + wq_chunk_index(ncg, nkb, tile, 0) + (row >> 5)) * p.chunk_bytes;
}

// ft_resolve for a row of an up tile and a token.
__device__ __forceinline__ float moe_resolve_up(const MoeParams &p, int expert, int tile, int row, int token, float v)
{
    uint32_t step, where;
    const uint8_t *const chunk = moe_chunk(p, true, expert, tile, row, step, where);
    return ft_resolve(chunk, step, where, static_cast<const __nv_bfloat16 *>(p.x) + (int64_t)token * p.H, p.H, v);
}

// The same on a row of h, in blocks of 256 features `rows` rows apart: 0 if it holds neither an
// infinity (which lies there as ±2^14 among zeros, under an infinite power) nor NaN.
__device__ __noinline__ float ft_resolve_h(const uint8_t *chunk, uint32_t step, uint32_t where, const __half *h,
                                           const float *powers, int rows, int I)
{
    float sum = 0.0f;
#pragma unroll 1
    for (int k = 0; k < I; k += 8) {
        if ((k & 63) == 0 && __ldcg(powers + ((int64_t)(k >> 8) * rows * 4 + (k >> 6 & 3))) != INFINITY) {
            k += 56;
            continue;
        }
        const uint4 u = __ldcg(reinterpret_cast<const uint4 *>(h + ((int64_t)(k >> 8) * rows * kWqChunkK + (k & 255))));
        ft_add_special(chunk, step, where, k, u, 1u, 0x7C00u, sum);
        if (sum != sum) break;
    }
    return sum;
}

// A sum over a token's experts: each resolved and weighted; those whose h is finite add
// nothing to what the others make of it.
__device__ __forceinline__ float moe_resolve_down(const MoeParams &p, const RouteTables *rt, int tile, int row, int token, float v)
{
    // All CTAs met before the down phase; this read of the count makes their h visible here.
    ld_acquire_gpu_u64(reinterpret_cast<const uint64_t *>(p.ctl + 2));
    float sum = 0.0f;
    bool found = false;
#pragma unroll 1
    for (int a = 0; a < rt->n_down; ++a)
#pragma unroll 1
        for (int at = rt->down_offset[a]; at < rt->down_offset[a] + rt->down_count[a]; ++at) {
            if (rt->token[at] != token) continue;
            uint32_t step, where;
            const uint8_t *const chunk = moe_chunk(p, false, rt->down_expert[a], tile, row, step, where);
            const float one = ft_resolve_h(chunk, step, where, static_cast<const __half *>(p.h) + (int64_t)at * kWqChunkK,
                                           p.h_powers + (int64_t)at * 4, p.h_rows, p.I);
            if (one != 0.0f) sum += rt->weight[at] * one, found = true;   // an infinity or NaN
        }
    return found ? sum : v;
}

// FMT 0: bf16 experts; 1: packed 4-bit experts.  NTMAX: 8-token tiles of the call.
template <int FMT, int NTMAX>
struct MoeKernel {
    static constexpr int kWorkers = ft_workers(FMT, NTMAX), kConverters = ft_converters(FMT, NTMAX);
    static constexpr int kFirstStorer = kWorkers / 32, kFirstConverter = kFirstStorer + kFtStorers / 32;
    static constexpr int kCopier = kFirstConverter + kConverters;
    static constexpr int kStepK = FMT == 0 ? moe_step_k(NTMAX) : kWqChunkK;
    static constexpr int kBoxes = kStepK / 64;           // 64-K pieces of the tokens a step copies
    static constexpr uint32_t kColBox = kStepK * 128u;   // bf16: a step's K x 64 columns
    // Steps of 4-bit weights go round the K parts, whose number changes with the
    // expert's tokens in calls of more than 32; above 16 the ring may have three slots.
    // Every bf16 worker takes part in every step.
    static constexpr bool kAll = FMT == 1 && NTMAX > 2;
    using Walk = StepWalk<FMT == 0 ? 1 : ft_k_parts(FMT, NTMAX, 1), kAll>;

    // Multiplies `n` steps of one tile on n_tok tokens (NT tiles) of one expert, whose
    // rows of h begin at `off`, and hands the sums over; the ring position moves on.
    // up: the tokens' rows are those of x, else of h.
    template <int NT>
    static __device__ __forceinline__ void steps(const MoeParams &p, const Ring &ring, const HandOver &hand,
                                                 const WaitCtl &ctl, const RouteTables *rt, int n, Walk &walk, RingPos &h,
                                                 bool up, int n_tok, int off, int chunks, uint8_t *gbase, uint32_t base, int warp,
                                                 int lane)
    {
        constexpr int TP = ft_token_parts(NT), KP = ft_k_parts(FMT, NTMAX, NT), NW = NT / TP;
        const int cg = warp & 3, part = (warp >> 2) % KP, tok0 = (warp >> 2) / KP * NW * 8;
        const uint32_t box_bytes = up ? (uint32_t)p.t8 * 128u : (uint32_t)NT * 1024u;
        uint32_t xrow[NW];
#pragma unroll
        for (int q = 0; q < NW; ++q) {
            // ldmatrix takes row lane % 8 of each eight, the fp16 fragment column lane / 4;
            // columns past the tokens repeat the last one's row.
            const int i = min(tok0 + q * 8 + (FMT == 0 ? lane & 7 : lane >> 2), n_tok - 1);
            xrow[q] = up ? rt->token[off + i] : (uint32_t)i;
        }
        Acc<NW> acc;
        acc.zero();
        walk.run(n, p.stages, ctl, part, KP, [&](const RingPos &at, bool own) {
            const uint32_t st = ring.stage(at), xb = st + p.off_x;
            if constexpr (FMT == 0) {
#pragma unroll
                for (int k0 = 0; k0 < kStepK / KP; k0 += 32) {
                    const int k = part * (kStepK / KP) + k0;
                    const uint32_t xbox = xb + (uint32_t)(k >> 6) * box_bytes;
                    ft_box_bf16<NW>(st + (uint32_t)(cg >> 1) * kColBox, cg & 1, k, up, xbox,
                                    up ? 0u : xbox + (uint32_t)kBoxes * box_bytes, xrow, lane, acc);
                }
            } else {
                const float *const meta = reinterpret_cast<const float *>(gbase + (st - base) + p.off_meta);
                if (own && cg < chunks)
                    ft_chunk_w4<NW>(st + (uint32_t)(cg * p.chunk_bytes), base + kFtEights, xb, meta, p.t8, tok0, xrow, p.gpc,
                                    p.has_zeros, lane, acc);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(ring.empty(at));
        });
        if constexpr (FMT == 1) ft_scale_w4<NW>(acc);
        HandOver mine = hand;
        mine.part_floats = NT * 8 * kFtRowStride;
        ft_hand_over<NW>(mine, h, ctl, part, warp, tok0, lane, acc);
    }

    static __device__ __forceinline__ int tiles_of(int n_tok)
    {
        return n_tok <= 8 ? 1 : n_tok <= 16 ? 2 : n_tok <= 32 ? 4 : 8;
    }

    // The converting warps (4-bit): the rows of each step's tokens, in the order of
    // the copies.
    static __device__ __forceinline__ void conversion(const MoeParams &p, const Ring &ring, const WaitCtl &ctl,
                                                      const RouteTables *rt, uint8_t *gbase, uint32_t base, int cw, int lane)
    {
        RingPos pos;
        int first = cw;
        auto step = [&](int n_tok, int off, bool up) {
            const uint32_t st = ring.stage(pos);
            float *const meta = reinterpret_cast<float *>(gbase + (st - base) + p.off_meta);
            ft_convert_step(ring, pos, ctl, st + p.off_x, up ? 0u : st + p.off_powers, n_tok, first, kConverters,
                            [&](int i) { return up ? (int)rt->token[off + i] : i; }, meta, p.t8, p.gpc, lane);
            first = first + 1 == kConverters ? 0 : first + 1;
            pos.next(p.stages);
        };
        for (int phase = 0; phase < 2; ++phase)
            for (Runs run(p, rt, phase == 0); run.left > 0; run.next())
                for (int n = run.steps(); n > 0; --n) step(run.count(rt), run.offset(rt), run.up);
    }

    // The copying thread.
    static __device__ __forceinline__ void copies(const MoeMaps &m, const MoeParams &p, const Ring &ring,
                                                  const WaitCtl &ctl, const RouteTables *rt, uint64_t start, int waits)
    {
        const int A = rt->n_down;
        const uint32_t box = (uint32_t)p.t8 * 128u;
        const int64_t up_bytes = (int64_t)p.ncg_up * p.nkb_up * p.chunk_bytes;
        const int64_t down_bytes = (int64_t)p.ncg_down * p.nkb_down * p.chunk_bytes;
        // Weights of a step: tile t of expert e, K step kb.
        auto weight_bytes = [&](bool up, int t) {
            return FMT == 0 ? 2u * kColBox : (uint32_t)(min(4, (up ? p.ncg_up : p.ncg_down) - 4 * t) * p.chunk_bytes);
        };
        auto weights = [&](bool up, int e, int t, int kb, uint32_t dst, uint32_t full) {
            if constexpr (FMT == 0) {
                const CUtensorMap *w = up ? &m.gate_up : &m.down;
                if (up ? p.up_spans : p.down_spans) {
                    tma_load_4d(dst, w, full, 0, kb * kStepK, t * 2, e);
                } else {
                    tma_load_3d(dst, w, full, t * 128, kb * kStepK, e);
                    tma_load_3d(dst + kColBox, w, full, t * 128 + 64, kb * kStepK, e);
                }
            } else {
                const int ncg = up ? p.ncg_up : p.ncg_down, nkb = up ? p.nkb_up : p.nkb_down;
                const uint8_t *src =
                    (up ? p.gate_up + e * up_bytes : p.down + e * down_bytes) + wq_chunk_index(ncg, nkb, t, kb) * p.chunk_bytes;
                bulk_load(dst, src, weight_bytes(up, t), full);
            }
        };
        RingPos pos;
        int issued = 0;
        bool ok = true;

        // Up: all of the call's token rows with each step.
        if ((int)blockIdx.x < rt->up.parts) {
            const int64_t s0 = ft_share_begin(rt->up, blockIdx.x), s1 = ft_share_begin(rt->up, blockIdx.x + 1);
            const int tile = (int)(s0 / p.nkb_up);
            int kb = (int)(s0 % p.nkb_up), a = tile / p.tiles_up, t = tile % p.tiles_up;
            for (int left = (int)(s1 - s0); left > 0; --left, ++issued, pos.next(p.stages)) {
                if (!(ok = ring.wait_empty(pos, ctl))) break;
                const uint32_t full = ring.full(pos), dst = ring.stage(pos);
                mbar_arrive_expect_tx(full, weight_bytes(true, t) + (FMT == 0 ? (uint32_t)kBoxes * box : (uint32_t)p.T * 512u));
                weights(true, rt->act_expert[a], t, kb, dst, full);
                if constexpr (FMT == 0) load_tokens(dst + p.off_x, &m.x, full, kb * kBoxes, kBoxes, 0, box, p.x_spans);
                else tma_load_2d(dst + p.off_x, &m.x, full, kb * kWqChunkK, 0);
                if (++kb == p.nkb_up) {
                    kb = 0;
                    if (++t == p.tiles_up) t = 0, ++a;
                }
            }
        }
        // Down: weights up to a ring ahead of the wait for h.
        if ((int)blockIdx.x < rt->down.parts && ok) {
            const int64_t s0 = ft_share_begin(rt->down, blockIdx.x), s1 = ft_share_begin(rt->down, blockIdx.x + 1);
            struct At {
                int t, a, kb;
            } w, h;
            w.kb = (int)(s0 % p.nkb_down);
            w.a = (int)(s0 / p.nkb_down % A);
            w.t = (int)(s0 / p.nkb_down / A);
            h = w;
            auto next = [&](At &s) {
                if (++s.kb == p.nkb_down) {
                    s.kb = 0;
                    if (++s.a == A) s.a = 0, ++s.t;
                }
            };
            auto begin = [&](const RingPos &r) {
                const int nt = tiles_of(rt->down_count[w.a]);
                mbar_arrive_expect_tx(ring.full(r), weight_bytes(false, w.t) + (uint32_t)(FMT == 0 ? 2 * kBoxes * nt * 1024 : nt * 8 * (512 + 16)));
                weights(false, rt->down_expert[w.a], w.t, w.kb, ring.stage(r), ring.full(r));
                next(w);
            };
            auto rows_of_h = [&](const RingPos &r) {
                const int nt = tiles_of(rt->down_count[h.a]);
                const int row = rt->down_offset[h.a];
                if constexpr (FMT == 0) {
                    const CUtensorMap *hm = nt == 1 ? &m.h[0] : nt == 2 ? &m.h[1] : &m.h[2];   // moe_down_tokens
                    const uint32_t box = (uint32_t)nt * 1024u;
                    for (uint32_t part = 0; part < 2; ++part)
                        load_tokens(ring.stage(r) + p.off_x + part * kBoxes * box, hm, ring.full(r), h.kb * kBoxes, kBoxes,
                                    row + (int)part * p.h_rows, box, p.h_spans);
                } else {
                    const int64_t at = (int64_t)h.kb * p.h_rows + row;
                    bulk_load(ring.stage(r) + p.off_x, static_cast<const uint8_t *>(p.h) + at * 512, (uint32_t)nt * 4096u,
                              ring.full(r));
                    bulk_load(ring.stage(r) + p.off_powers, p.h_powers + at * 4, (uint32_t)nt * 128u, ring.full(r));
                }
                next(h);
            };
            const int n = (int)(s1 - s0);
            RingPos behind = pos;
            int sent = 0;
            for (; sent < min(n, p.stages); ++sent, ++issued, pos.next(p.stages)) {
                if (!(ok = ring.wait_empty(pos, ctl))) break;
                begin(pos);
            }
            // h is written by plain stores of all CTAs and read here by bulk copies.
            if (!grid_wait(p.ctl, start, waits, ctl)) ok = false;
            fence_proxy_async_all();
            // Even after an expired wait: the steps begun above must complete.
            for (int q = 0; q < sent; ++q, behind.next(p.stages)) rows_of_h(behind);
            for (; sent < n && ok; ++sent, ++issued, pos.next(p.stages)) {
                if (!(ok = ring.wait_empty(pos, ctl))) break;
                begin(pos);
                rows_of_h(pos);
            }
        }
        // After an expired wait copies may still be in flight: see them land.
        if (*ctl.abort)
            for (int n = max(0, issued - p.stages); n < issued; ++n)
                wait_teardown(ring.full0 + 8u * (uint32_t)(n % p.stages), (uint32_t)(n / p.stages) & 1u, ctl);
    }

    // Calls f with the instance for nt 8-token tiles.
    template <typename F>
    static __device__ __forceinline__ void with_tiles(int nt, F f)
    {
        if (NTMAX == 1 || nt == 1) f(std::integral_constant<int, 1>());
        else if (NTMAX == 2 || nt == 2) f(std::integral_constant<int, (NTMAX >= 2 ? 2 : 1)>());
        else if (NTMAX == 4 || nt == 4) f(std::integral_constant<int, (NTMAX >= 4 ? 4 : 1)>());
        else f(std::integral_constant<int, (NTMAX >= 8 ? 8 : 1)>());
    }

    // The workers: every piece of a tile of the up phase, then every expert's part of
    // a piece of the down phase.
    static __device__ __forceinline__ void products(const MoeParams &p, const Ring &ring, const HandOver &hand,
                                                    const WaitCtl &ctl, const RouteTables *rt, uint8_t *gbase, uint32_t base,
                                                    int warp, int lane)
    {
        RingPos h;
        Walk walk;
        walk.start(FMT == 0 ? ring.full0 : ring.ready0, FMT == 0 ? 0 : (warp >> 2) % ft_k_parts(FMT, NTMAX, 1), p.stages);
        for (int phase = 0; phase < 2; ++phase)
            for (Runs run(p, rt, phase == 0); run.left > 0; run.next()) {
                const int chunks = min(4, (run.up ? p.ncg_up : p.ncg_down) - 4 * run.tile);
                const int n_tok = run.count(rt), off = run.offset(rt);
                with_tiles(tiles_of(n_tok), [&](auto nt) {
                    steps<decltype(nt)::value>(p, ring, hand, ctl, rt, run.steps(), walk, h, run.up, n_tok, off, chunks, gbase, base,
                                               warp, lane);
                });
            }
    }

    // Two features of a row of h of 4-bit experts (a warp; v: 0 past the last), as fp16 with
    // their 64's power of two; false where it holds an infinity or NaN, unless MARK: then the
    // power is infinite, infinities are marked and what is finite is 0.
    template <bool MARK>
    static __device__ __forceinline__ bool store_row(const MoeParams &p, float (&v)[2], int at, int j, bool second, int lane)
    {
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu,
                                               max(__float_as_uint(v[0]) & 0x7FFFFFFFu, __float_as_uint(v[1]) & 0x7FFFFFFFu));
        const uint32_t e = max(top >> 23, 15u);              // biased exponent of the largest
        if (!MARK && e == 255u) return false;
        const float inv = __uint_as_float((268u - min(e, 254u)) << 23);
        const int64_t row = (int64_t)(j >> 2) * p.h_rows + at;
        __half *const out = static_cast<__half *>(p.h) + row * kWqChunkK + (j & 3) * 64 + lane;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (MARK && e == 255u) v[q] = isinf(v[q]) ? copysignf(16384.0f, v[q]) : isnan(v[q]) ? v[q] : 0.0f;
            else v[q] *= inv;
            if (q == 0 || second) out[q * 32] = __float2half_rn(v[q]);
        }
        if (lane == 0) p.h_powers[row * 4 + (j & 3)] = e == 255u ? INFINITY : __uint_as_float((e - 14u) << 23);
        return true;
    }

    // A row of h with sums that are not finite.
    static __device__ __forceinline__ void store_row_resolved(const MoeParams &p, const float *red, const RouteTables *rt, int at,
                                                           int j, int expert, bool second, int lane)
    {
        float v[2] = {0.0f, 0.0f};
#pragma unroll 1
        for (int q = 0; q < (second ? 2 : 1); ++q) {
            const int row = ft_gate_row(lane + q * 32);
            float gate = red[row], up = red[row + 8];
            if (!(fabsf(gate) < INFINITY)) gate = moe_resolve_up(p, expert, j, row, rt->token[at], gate);
            if (!(fabsf(up) < INFINITY)) up = moe_resolve_up(p, expert, j, row + 8, rt->token[at], up);
            v[q] = ft_act(gate, p.act) * up;
        }
        __syncwarp();
        store_row<true>(p, v, at, j, second, lane);
    }

    // Columns of y whose sums are not finite (one storer's).
    static __device__ __forceinline__ void store_y_resolved(const MoeParams &p, const RouteTables *rt, const float *yacc, int tile,
                                                         int tid)
    {
        const __nv_bfloat16 *const res = static_cast<const __nv_bfloat16 *>(p.residual);
#pragma unroll 1
        for (int e = tid; e < kFtTileRows * p.T; e += kFtStorers) {
            const int row = e % kFtTileRows, t = e / kFtTileRows, n = tile * kFtTileRows + row;
            float v = yacc[t * kFtRowStride + row];
            if (n >= p.H || fabsf(v) < INFINITY) continue;
            if (FMT == 1) v = moe_resolve_down(p, rt, tile, row, t, v);
            const int64_t at = (int64_t)t * p.H + n;
            static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(res ? v + __bfloat162float(res[at]) : v);
        }
    }

    // h of tile j for n_tok tokens from row `off` on, in the form that the down phase
    // multiplies.  bf16 experts: as a sum of two bf16 numbers, 16 significant bits; one, 8
    // bits, would add as much error to y as the rounding of y does, and the second doubles
    // only the products of h.  4-bit experts: in fp16, as their products read it anyway, 11
    // bits and an eighth of that error; a power of two for each 64 features of a row takes
    // the place of the exponents that fp16 lacks.
    static __device__ __forceinline__ void store_h(const MoeParams &p, const float *red, int n_tok, int off, int j, int expert,
                                                   const RouteTables *rt, int tid)
    {
        auto value = [&](int t, int f) {
            const float *const at = red + t * kFtRowStride + ft_gate_row(f);
            return ft_act(at[0], p.act) * at[8];
        };
        if constexpr (FMT == 0) {
            __nv_bfloat16 *const hs = static_cast<__nv_bfloat16 *>(p.h);
            for (int e = tid; e < 64 * n_tok; e += kFtStorers) {
                const int f = e & 63, t = e >> 6, col = j * 64 + f;
                if (col >= p.I) continue;
                const float v = value(t, f);
                const __nv_bfloat16 high = __float2bfloat16_rz(v);   // (a finite one stays finite)
                hs[(int64_t)(off + t) * p.I + col] = high;
                hs[(int64_t)(p.h_rows + off + t) * p.I + col] =
                    __float2bfloat16_rn(isinf(v) ? 0.0f : v - __bfloat162float(high));
            }
        } else {
            const int lane = tid & 31;
            const bool second = j * 64 + 32 < p.I;   // I is a multiple of 32
            for (int t = tid >> 5; t < n_tok; t += kFtStorers / 32) {
                float v[2] = {value(t, lane), second ? value(t, lane + 32) : 0.0f};
                if (!store_row<false>(p, v, off + t, j, second, lane))
                    store_row_resolved(p, red + t * kFtRowStride, rt, off + t, j, expert, second, lane);
            }
        }
    }

    // The storers: h of the up phase's tiles, the meeting of all CTAs, y.
    static __device__ __forceinline__ void finish(const MoeParams &p, const HandOver &hand, const WaitCtl &ctl,
                                                  const RouteTables *rt, float *yacc, volatile int32_t *flags, int tid)
    {
        const int lane = tid & 31, A = rt->n_down;
        RingPos h;
        // The sums of one expert's n_tok tokens, K parts added up.
        auto take = [&](int n_tok) {
            const int nt = tiles_of(n_tok);
            HandOver mine = hand;
            mine.part_floats = nt * 8 * kFtRowStride;
            return ft_take_over(mine, h, ctl, ft_k_parts(FMT, NTMAX, nt), n_tok, tid);
        };
        for (Runs run(p, rt, true); run.left > 0; run.next()) {
            const int n_tok = run.count(rt), off = run.offset(rt), j = run.tile;
            float *const red = take(n_tok);
            bool last = true;
            if (run.steps() < p.nkb_up) {
                const int tile = run.a * p.tiles_up + j;
                int first, pieces;
                ft_share_pieces(rt->up, tile, first, pieces);
                last = ft_exchange(p.partials, p.t8, red, n_tok, run.k == 0, p.ctl + kMoeCtlHead + tile, first, pieces, flags + 1,
                                   tid);
            }
            if (last) store_h(p, red, n_tok, off, j, rt->act_expert[run.a], rt, tid);
            ft_give_back(hand, h, lane);
        }
        fence_proxy_async_all();
        ft_storers_sync();
        if (tid == 0) grid_arrive(p.ctl);

        const __nv_bfloat16 *const res = static_cast<const __nv_bfloat16 *>(p.residual);
        __nv_bfloat16 *const y = static_cast<__nv_bfloat16 *>(p.y);
        if (A == 0) {   // no token chose any expert
            for (int64_t e = (int64_t)blockIdx.x * kFtStorers + tid; e < (int64_t)p.T * p.H;
                 e += (int64_t)gridDim.x * kFtStorers)
                y[e] = res ? res[e] : __float2bfloat16_rn(0.0f);
            return;
        }
        for (Runs run(p, rt, false); run.left > 0;) {
            const int tile = run.tile;
            const bool head = run.a == 0 && run.k == 0;
            bool whole = head;
            for (int e = tid; e < p.t8 * kFtRowStride; e += kFtStorers) yacc[e] = 0.0f;   // take's barrier comes before its use
            for (; run.left > 0 && run.tile == tile; run.next()) {
                const int n_tok = run.count(rt), off = run.offset(rt);
                whole &= run.steps() == p.nkb_down && (run.a + 1 == A || run.left > run.steps());
                const float *const red = take(n_tok);
                for (int e = tid; e < kFtTileRows * n_tok; e += kFtStorers) {
                    const int row = e % kFtTileRows, i = e / kFtTileRows;
                    float *const out = yacc + (int)rt->token[off + i] * kFtRowStride + row;
                    *out = fmaf(rt->weight[off + i], red[i * kFtRowStride + row], *out);
                }
                ft_give_back(hand, h, lane);
                ft_storers_sync();   // a token's next expert may be another thread's
            }
            bool last = true;
            if (!whole) {
                int first, pieces;
                ft_share_pieces(rt->down, tile, first, pieces);
                last = ft_exchange(p.partials, p.t8, yacc, p.T, head, p.ctl + kMoeCtlHead + p.max_tiles_up + tile, first,
                                   pieces, flags + 1, tid);
            }
            if (last) {
                const int n0 = tile * kFtTileRows;
                bool left = false;
                ft_batched<8>(
                    kFtTileRows * p.T, tid, kFtStorers,
                    [&](int e) {
                        const int n = n0 + e % kFtTileRows;
                        return res && n < p.H ? __bfloat162float(res[(int64_t)(e / kFtTileRows) * p.H + n]) : 0.0f;
                    },
                    [&](int e, float r) {
                        const int row = e % kFtTileRows, t = e / kFtTileRows, n = n0 + row;
                        if (n >= p.H) return;
                        const float v = yacc[t * kFtRowStride + row];
                        if (FMT == 1 && !(fabsf(v) < INFINITY)) {
                            left = true;
                            return;
                        }
                        y[(int64_t)t * p.H + n] = __float2bfloat16_rn(res ? v + r : v);
                    });
                if (left) store_y_resolved(p, rt, yacc, tile, tid);
            }
            ft_storers_sync();
        }
    }
};

template <int FMT, int NTMAX>
__global__ void __launch_bounds__(ft_threads(FMT, NTMAX), 1)
    moe_kernel(const __grid_constant__ MoeMaps m, const __grid_constant__ MoeParams p)
{
    using K = MoeKernel<FMT, NTMAX>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *const gbase = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = smem_u32(gbase);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Ring ring{base + p.off_ring, p.stage_bytes, base + kFtFull, base + kFtEmpty, base + kFtReady, p.stages};
    volatile int32_t *const flags = reinterpret_cast<volatile int32_t *>(gbase + kFtFlags);
    RouteTables *const rt = reinterpret_cast<RouteTables *>(gbase + p.off_route);
    const HandOver hand{reinterpret_cast<float *>(gbase + p.off_red), ft_k_parts(FMT, NTMAX, NTMAX) * NTMAX * 8 * kFtRowStride, 0,
                        base + kFtHandFull, base + kFtHandEmpty};
    float *const yacc = reinterpret_cast<float *>(gbase + p.off_acc);
    const WaitCtl ctl{flags, p.ctl, p.timeout_ns};

    ft_touch_params(p, warp);
    // Before this CTA arrives, by the threads that wait for the others.
    const bool waits_for_all = threadIdx.x == 0 || threadIdx.x == 32 * K::kCopier;
    const uint64_t start = waits_for_all ? grid_start(p.ctl) : 0;
    if (threadIdx.x == 0) {
        ft_init_shared(gbase, ring, FMT == 0 || K::kAll ? K::kWorkers / 32 : 4, K::kConverters, K::kWorkers);
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (threadIdx.x == 32 * K::kCopier) {
        prefetch_tmap(&m.x);
        if (FMT == 0) {
            prefetch_tmap(&m.h[0]);
            prefetch_tmap(&m.gate_up);
            prefetch_tmap(&m.down);
        }
    }
    __syncthreads();
    int waits = 0;
    float *const logits = reinterpret_cast<float *>(gbase + p.off_ring);   // of the CTA's own choice
    int32_t *const ids = reinterpret_cast<int32_t *>(logits + (p.routed || p.route_reduce ? 0 : p.T * p.E));
    float *const weights = reinterpret_cast<float *>(ids + p.T * p.top_k);
    if (!p.routed) {
        if (warp < K::kWorkers / 32) {
            route<K::kWorkers>(p, gbase + p.off_ring, rt, threadIdx.x);
            if (threadIdx.x == 0) grid_arrive(p.ctl);
        }
        waits = 1;
        if (threadIdx.x == 0) grid_wait(p.ctl, start, waits + (p.debug_stall ? 64 : 0), ctl);
        __syncthreads();
    }
    if (warp < K::kWorkers / 32) choose<K::kWorkers>(p, logits, ids, weights, threadIdx.x);
    if (warp < K::kWorkers / 32) build_tables<K::kWorkers, moe_down_tokens(FMT)>(p, rt, ids, weights, threadIdx.x);
    // The router's scratch in the ring was written by plain stores.
    fence_proxy_async_smem();
    __syncthreads();
    if (warp == K::kCopier) {
        if (lane == 0) K::copies(m, p, ring, ctl, rt, start, waits + 1 + (p.routed && p.debug_stall ? 64 : 0));
        return;
    }
    if (warp >= K::kFirstConverter) K::conversion(p, ring, ctl, rt, gbase, base, warp - K::kFirstConverter, lane);
    else if (warp >= K::kFirstStorer) K::finish(p, hand, ctl, rt, yacc, flags, threadIdx.x - K::kWorkers);
    else K::products(p, ring, hand, ctl, rt, gbase, base, warp, lane);
}

template <int FMT>
const void *moe_fn(int nt)
{
    return nt == 1   ? (const void *)moe_kernel<FMT, 1>
           : nt == 2 ? (const void *)moe_kernel<FMT, 2>
           : nt == 4 ? (const void *)moe_kernel<FMT, 4>
                     : (const void *)moe_kernel<FMT, 8>;
}

}  // namespace

cudaError_t moe_set_smem_limit(int bytes)
{
    for (int nt = 1; nt <= 8; nt *= 2)
        for (const void *f : {moe_fn<0>(nt), moe_fn<1>(nt)}) {
            cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

cudaError_t launch_moe(int nt, int wq, const MoeMaps &m, const MoeParams &p, int grid, int smem, cudaStream_t stream)
{
    void *args[] = {const_cast<MoeMaps *>(&m), const_cast<MoeParams *>(&p)};
    // Cooperative: the CTAs wait for one another between phases, so all must
    // be resident (the launch fails otherwise).
    return cudaLaunchCooperativeKernel(wq ? moe_fn<1>(nt) : moe_fn<0>(nt), dim3(grid), dim3(ft_threads(wq ? FT_MOE_W4 : FT_MOE_BF16, nt)), args,
                                       (size_t)smem, stream);
}

}  // namespace gemmgb
