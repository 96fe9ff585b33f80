// Few-token products with 4-bit weights:
//   y[t, n] = act(Σ_k x[t, k] · (q[k, n] - z[k/G, n]) · s[k/G, n] + bias[n]) (+ R[t, n])
// for 1 to 64 tokens, plain or gated, with the kernels that quantise a bf16
// weight and lay codes, scales and zero points out for the product.
//
// Product: bound by the weight's bytes (K·N/2, plus scales), read once: 1 token
// 8192x28672 with zero points 25.6 us, 4.8 TB/s (71% of a copy; 5 us of it are start-up
// and the last exchange, then a step of 17 KB takes 0.43 us an SM where the memory alone
// takes 0.37).  With more tokens the workers bound it: 64 tokens 14336x4096 41 us, 3,600
// cycles a step (tensor pipe 45% busy, 1.7 instructions a cycle from two warps a
// scheduler; four foursomes spill: 49 us), and above 32 tokens the library's bf16 GEMM
// takes less time with four times the bytes (25 us there).  One CTA to an SM; a copying warp
// fills a ring with a tile's packed chunks (one bulk copy for 128 columns x 256 K) and the
// matching piece of x; up to 8 tokens a few warps convert it in place, above a kernel
// ahead has prepared it (16 tokens 4096x28672: 26 us, 39 with converting warps; 1 token
// 8192x28672: 26.1 and 25.6); foursomes of workers multiply, and four storers finish tiles behind them.  Tiles are cut
// along K into as many pieces as keep the SMs evenly busy (FtShare).  Where there
// are few tiles the pieces of each are one thread-block cluster and add up through
// distributed shared memory; else through a workspace, the CTA that arrives last
// adding them.  Always in K order, so results do not depend on timing.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "few_token.cuh"

namespace gemmgb {
namespace {

__device__ __forceinline__ float4 ld_cluster(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Row of element e of the 16-row strips rank, rank + step, ... (`strips` of them),
// strip by strip within a token.
__device__ __forceinline__ int wq_strip_row(int e, int strips, int rank, int step)
{
    return (rank + (e >> 4) % strips * step) * 16 + (e & 15);
}

// ft_resolve for a row of a tile and a token.
__device__ __forceinline__ float wq_resolve(const WqParams &p, int tile, int row, int t, float v)
{
    const int here = min(4, p.ncg - 4 * tile);
    if (row >> 5 >= here) return v;
    return ft_resolve(p.packed + (wq_chunk_index(p.ncg, p.nkb, tile, 0) + (row >> 5)) * p.chunk_bytes,
                      (uint32_t)(here * p.chunk_bytes), (uint32_t)(row & 31) | (uint32_t)p.gpc << 5 | (uint32_t)p.has_zeros << 9,
                      static_cast<const __nv_bfloat16 *>(p.x) + (int64_t)t * p.K, p.K, v);
}

// Epilogue of the 16-row strips rank, rank + step, ... of a tile, from red[token][row],
// by `workers` threads.  A gated strip holds eight gates and their eight ups.  The sums
// that are finite; true if the thread left others, which RESOLVE then stores.
template <bool RESOLVE>
__device__ __forceinline__ bool wq_store_sums(const WqParams &p, const float *red, int tile, int rank, int step, int tid,
                                              int workers)
{
    bool left = false;
    constexpr int rstride = kFtRowStride;
    const __nv_bfloat16 *const bias = static_cast<const __nv_bfloat16 *>(p.bias);
    const __nv_bfloat16 *const res = static_cast<const __nv_bfloat16 *>(p.residual);
    __nv_bfloat16 *const y = static_cast<__nv_bfloat16 *>(p.y);
    const int strips = (8 - rank + step - 1) / step;
    if (!p.gated) {
        const int n0 = tile * kFtTileRows;
        ft_batched<RESOLVE ? 1 : 4>(
            strips * 16 * p.T, tid, workers,
            [&](int e) {
                const int n = n0 + wq_strip_row(e, strips, rank, step);
                return make_float2(bias && n < p.N ? __bfloat162float(bias[n]) : 0.0f,
                                   res && n < p.N ? __bfloat162float(res[(int64_t)((e >> 4) / strips) * p.N + n]) : 0.0f);
            },
            [&](int e, float2 r) {
                const int row = wq_strip_row(e, strips, rank, step), t = (e >> 4) / strips, n = n0 + row;
                if (n >= p.N) return;
                float v = red[t * rstride + row];
                if ((fabsf(v) < INFINITY) == RESOLVE) {
                    left = true;
                    return;
                }
                if (RESOLVE) v = wq_resolve(p, tile, row, t, v);
                if (bias) v += r.x;
                v = ft_act(v, p.act);
                y[(int64_t)t * p.N + n] = __float2bfloat16_rn(res ? v + r.y : v);
            });
    } else {
        const int o0 = tile * (kFtTileRows / 2);
        for (int e = tid; e < strips * 8 * p.T; e += workers) {   // (batched loads cost the products registers)
            const int strip = rank + (e >> 3) % strips * step, t = (e >> 3) / strips, o = o0 + strip * 8 + (e & 7);
            if (o >= p.N / 2) continue;
            const int gate_col = 64 * (o >> 5) + (o & 31);
            const float *const at = red + t * rstride + strip * 16 + (e & 7);
            float gate = at[0], up = at[8];
            if ((fabsf(gate) < INFINITY && fabsf(up) < INFINITY) == RESOLVE) {
                left = true;
                continue;
            }
            if (RESOLVE) {
                gate = fabsf(gate) < INFINITY ? gate : wq_resolve(p, tile, strip * 16 + (e & 7), t, gate);
                up = fabsf(up) < INFINITY ? up : wq_resolve(p, tile, strip * 16 + (e & 7) + 8, t, up);
            }
            if (bias) {
                gate += __bfloat162float(bias[gate_col]);
                up += __bfloat162float(bias[gate_col + 32]);
            }
            y[(int64_t)t * (p.N / 2) + o] = __float2bfloat16_rn(ft_act(gate, p.act) * up);
        }
    }
    return left;
}

__device__ __forceinline__ void wq_store(const WqParams &p, const float *red, int tile, int rank, int step, int tid, int workers)
{
    if (wq_store_sums<false>(p, red, tile, rank, step, tid, workers)) wq_store_sums<true>(p, red, tile, rank, step, tid, workers);
}

// The pieces of a tile are one cluster: each CTA adds up and stores the 16-row strips of
// its rank, reading the others' sums from their shared memory, which all threads see
// complete at the first meeting and leave at the second.  All warps of the CTA: the four
// storers alone, a word at a time, took 24,000 cycles for 64 tokens.
__device__ __forceinline__ void wq_join(const WqParams &p, float *red, int tile)
{
    cluster_sync_all();
    const int rank = (int)cluster_ctarank(), strips = (8 - rank + p.cluster - 1) / p.cluster;
    for (int e = threadIdx.x; e < strips * 4 * p.T; e += blockDim.x) {
        const int q4 = e % (strips * 4), row = (rank + (q4 >> 2) * p.cluster) * 16 + (q4 & 3) * 4;
        float *const at = red + e / (strips * 4) * kFtRowStride + row;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int q0 = 0; q0 < kFtMostCluster; q0 += 4) {
            float4 part[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q0 + q < p.cluster) part[q] = ld_cluster(mapa_u32(smem_u32(at), (uint32_t)(q0 + q)));
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q0 + q < p.cluster) v.x += part[q].x, v.y += part[q].y, v.z += part[q].z, v.w += part[q].w;
        }
        *reinterpret_cast<float4 *>(at) = v;    // no other CTA reads this rank's strips here
    }
    __syncthreads();
    wq_store(p, red, tile, rank, p.cluster, threadIdx.x, blockDim.x);
    cluster_sync_all();
}

// NT: 8-token tiles of the call.  JOIN: the pieces of each tile are a cluster.
template <int NT, bool JOIN>
__global__ void __launch_bounds__(ft_threads(FT_PRODUCT, NT), 1)
    wq_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ WqParams p)
{
    constexpr int workers = ft_workers(FT_PRODUCT, NT), converters = ft_converters(FT_PRODUCT, NT);
    constexpr int kFirstStorer = workers / 32, kFirstConverter = kFirstStorer + kFtStorers / 32;
    constexpr int kCopier = kFirstConverter + converters;
    constexpr int TP = ft_token_parts(NT), KP = ft_k_parts(FT_PRODUCT, NT, NT), NW = NT / TP;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *const gbase = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = smem_u32(gbase);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Ring ring{base + p.off_ring, p.stage_bytes, base + kFtFull, base + kFtEmpty, base + kFtReady, p.stages};
    const HandOver hand{reinterpret_cast<float *>(gbase + p.off_red), KP * NT * 8 * kFtRowStride, NT * 8 * kFtRowStride,
                        base + kFtHandFull, base + kFtHandEmpty};
    const uint32_t never = base + kFtNever;
    volatile int32_t *const flags = reinterpret_cast<volatile int32_t *>(gbase + kFtFlags);

    ft_touch_params(p, warp);
    if (threadIdx.x == 0) {
        ft_init_shared(gbase, ring, 4 * TP, converters, workers);   // a slot is left by one foursome a token part
        mbar_init(never, 1);
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (!wq_prepares(NT) && warp == kCopier && lane == 0) prefetch_tmap(&tm_x);
    __syncthreads();

    const WaitCtl ctl{flags, p.status, p.timeout_ns};
    const int64_t s0 = ft_share_begin(p.share, blockIdx.x), s1 = ft_share_begin(p.share, blockIdx.x + 1);
    const int n_steps = (int)(s1 - s0);
    int tile = (int)(s0 / p.nkb), kb = (int)(s0 % p.nkb);

    if (warp == kCopier) {
        // ---- copies ----
        if (lane == 0) {
            const uint8_t *src = p.packed + wq_chunk_index(p.ncg, p.nkb, tile, kb) * p.chunk_bytes;
            const uint32_t x_bytes = wq_prepares(NT) ? p.prepared_bytes : (uint32_t)p.T * 512u;
            auto w_bytes = [&](int t) { return (uint32_t)(min(4, p.ncg - 4 * t) * p.chunk_bytes); };
            auto load_w = [&](const RingPos &r, uint32_t bytes) {
                mbar_arrive_expect_tx(ring.full(r), bytes + x_bytes);
                bulk_load(ring.stage(r), src, bytes, ring.full(r));
                src += bytes;   // a tile's chunks lie along K, tiles one after another
            };
            // What lies past K comes back as zeros, which is what the weight's padding must meet.
            auto load_x = [&](const RingPos &r, int k) {
                if constexpr (wq_prepares(NT))
                    bulk_load(ring.stage(r) + p.off_x, p.prepared + (int64_t)k * x_bytes, x_bytes, ring.full(r));
                else tma_load_2d(ring.stage(r) + p.off_x, &tm_x, ring.full(r), k * kWqChunkK, 0);
            };
            auto next = [&](int &t, int &k) {
                if (++k == p.nkb) k = 0, ++t;
            };
            // Weights that the work before this launch does not write start at
            // once; everything else waits for that work.
            const int early = p.early_weights ? min(n_steps, p.stages) : 0;
            RingPos pos;
            {
                int t = tile, k = kb;
                for (int i = 0; i < early; ++i, pos.next(p.stages), next(t, k)) load_w(pos, w_bytes(t));
            }
            asm volatile("griddepcontrol.wait;" ::: "memory");
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            pos = RingPos();
            for (int i = 0; i < early; ++i, pos.next(p.stages), next(tile, kb)) load_x(pos, kb);
            int issued = early;
            for (; issued < n_steps; ++issued, pos.next(p.stages), next(tile, kb)) {
                if (!ring.wait_empty(pos, ctl)) break;
                load_w(pos, w_bytes(tile));
                load_x(pos, kb);
            }
            // After an expired wait copies may still be in flight: see them land.
            if (flags[0])
                for (int i = max(0, issued - p.stages); i < issued; ++i)
                    wait_teardown(ring.full0 + 8u * (uint32_t)(i % p.stages), (uint32_t)(i / p.stages) & 1u, ctl);
        }
        __syncwarp();
    } else if (converters > 0 && warp >= kFirstConverter) {
        // ---- conversion ----
        asm volatile("griddepcontrol.wait;" ::: "memory");
        RingPos pos;
        for (int i = 0; i < n_steps; ++i, pos.next(p.stages)) {
            float *const meta = reinterpret_cast<float *>(gbase + (ring.stage(pos) - base) + p.off_meta);
            ft_convert_step(ring, pos, ctl, ring.stage(pos) + p.off_x, 0u, p.T, (warp + i) % max(converters, 1), converters,
                            [](int r) { return r; }, meta, p.t8, p.gpc, lane);
        }
    } else if (warp >= kFirstStorer) {
        // ---- finished tiles ----
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const int tid = threadIdx.x - workers;
        RingPos h;
        for (int left = n_steps; left > 0; ++tile, kb = 0) {
            const int ks0 = kb, ks1 = min(p.nkb, kb + left);
            left -= ks1 - ks0;
            float *const red = ft_take_over(hand, h, ctl, KP, p.T, tid);
            if (JOIN) break;            // one piece of one tile, joined below
            bool finish = true;
            if (ks1 - ks0 < p.nkb) {    // a piece: the last one to arrive goes on
                int first, pieces;
                ft_share_pieces(p.share, tile, first, pieces);
                finish = ft_exchange(p.workspace, p.t8, red, p.T, ks0 == 0, p.counters + tile, first, pieces, flags + 1, tid);
            }
            if (finish) wq_store(p, red, tile, 0, 1, tid, kFtStorers);
            ft_give_back(hand, h, lane);
        }
    } else {
        // ---- products ----
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (p.debug_stall) wait_bar(never, 0, ctl, SITE_EPI_STALL);
        const int chunk = warp & 3, part = (warp >> 2) % KP, tok0 = (warp >> 2) / KP * NW * 8;
        uint32_t xrow[NW];   // columns past the tokens repeat the last one's row
#pragma unroll
        for (int n = 0; n < NW; ++n) xrow[n] = (uint32_t)min(tok0 + n * 8 + (lane >> 2), p.T - 1);
        Acc<NW> acc;

        RingPos h;
        StepWalk<KP, false> walk;   // steps go round the K parts
        walk.start(converters > 0 ? ring.ready0 : ring.full0, part, p.stages);
        for (int left = n_steps; left > 0; ++tile, kb = 0) {
            const int ks0 = kb, ks1 = min(p.nkb, kb + left);
            const bool here = tile * 4 + chunk < p.ncg;
            acc.zero();
            walk.run(ks1 - ks0, p.stages, ctl, part, KP, [&](const RingPos &pos, bool) {
                const uint32_t st = ring.stage(pos);
                const float *const meta = reinterpret_cast<const float *>(gbase + (st - base) + p.off_meta);
                if (here)
                    ft_chunk_w4<NW>(st + (uint32_t)(chunk * p.chunk_bytes), base + kFtEights, st + p.off_x, meta, p.t8, tok0,
                                    xrow, p.gpc, p.has_zeros, lane, acc);
                __syncwarp();
                if (lane == 0) mbar_arrive(ring.empty(pos));
            });
            left -= ks1 - ks0;
            ft_scale_w4<NW>(acc);
            ft_hand_over<NW>(hand, h, ctl, part, warp, tok0, lane, acc);
        }
    }
    if constexpr (JOIN) wq_join(p, hand.red, (int)(s0 / p.nkb));   // the first and only hand-over
}

// --- Activations ---------------------------------------------------------------------
//
// The products' form of x (few_token.cuh) for every 256 K, one warp to a row of it.
// Runs ahead of the product; only what follows the waits there needs it.
__global__ void __launch_bounds__(256) wq_prepare_kernel(const __grid_constant__ WqPrepareParams p)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, item = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item >= p.T * p.nkb) return;
    const int t = item % p.T, kb = item / p.T, k = kb * kWqChunkK + lane * 8;   // K is a multiple of 8
    const uint4 v = k < p.K ? __ldcg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.x) +
                                                                    (int64_t)t * p.K + k))
                            : make_uint4(0, 0, 0, 0);
    const uint32_t w[1][4] = {{v.x, v.y, v.z, v.w}};
    uint32_t out[1][4];
    float scale[1], sum[1];
    const int row[1] = {0};
    ft_convert<1>(w, 0u, row, lane, p.gpc, out, scale, sum);
    uint8_t *const piece = p.out + (int64_t)kb * p.piece_bytes;
    float *const meta = reinterpret_cast<float *>(piece + p.T * 512);
    *reinterpret_cast<uint4 *>(piece + t * 512 + ft_converted_place(t, lane)) = make_uint4(out[0][0], out[0][1], out[0][2], out[0][3]);
    if (lane == 0) meta[t] = scale[0];
    if ((lane & 3) == 0) meta[(1 + ((lane >> 2) * p.gpc >> 3)) * p.t8 + t] = sum[0];
    asm volatile("fence.proxy.async;" ::: "memory");   // read by bulk copies
}

// --- Layout ------------------------------------------------------------------------

// One thread to a word of codes; the chunk's first threads copy scales and
// zero points.  Columns and K beyond the weight get code 0, scale 0, zero 0.
__global__ void __launch_bounds__(256) wq_pack_kernel(const WqPackParams p)
{
    const int64_t chunks = (int64_t)p.ncg * p.nkb;
    const int64_t nb = (p.N + 1) / 2;
    const int64_t ng = p.group > 0 ? (p.K + p.group - 1) / p.group : 1;
    for (int64_t c = blockIdx.x; c < chunks * p.mats; c += gridDim.x) {
        const int64_t mat = c / chunks, in_mat = c % chunks;
        const int tile = (int)(in_mat / ((int64_t)4 * p.nkb)), here = min(4, p.ncg - 4 * tile);
        const int in_tile = (int)(in_mat - (int64_t)4 * p.nkb * tile);
        const int cg = tile * 4 + in_tile % here, kb = in_tile / here;
        const uint8_t *codes = p.codes + mat * p.K * nb;
        uint8_t *out = p.packed + c * p.chunk_bytes;
        for (int wd = threadIdx.x; wd < kWqChunkCodes / 4; wd += blockDim.x) {
            const int slot = wd & 3, lane = (wd >> 2) & 31, j = wd >> 7;
            const int n = wq_column(cg, slot, lane >> 2, p.gated);
            uint32_t word = 0;
            if (n < p.N)
                for (int q = 0; q < 8; ++q) {
                    const int64_t k = (int64_t)kb * 256 + j * 32 + 8 * (lane & 3) + 2 * (q & 3) + (q >> 2);
                    if (k < p.K) word |= ((codes[k * nb + n / 2] >> (4 * (n & 1))) & 15u) << (4 * q);
                }
            reinterpret_cast<uint32_t *>(out)[wd] = word;
        }
        for (int i = threadIdx.x; i < p.gpc * 32; i += blockDim.x) {
            const int gi = i >> 5, g = (i >> 2) & 7, slot = i & 3;
            const int n = wq_column(cg, slot, g, p.gated);
            const int64_t k = (int64_t)kb * 256 + gi * (256 / p.gpc);
            const bool in = n < p.N && k < p.K;
            const int64_t at = (mat * ng + (p.group > 0 ? k / p.group : 0)) * p.N + n;
            reinterpret_cast<uint16_t *>(out + kWqChunkCodes)[i] =
                in ? static_cast<const uint16_t *>(p.scales)[at] : (uint16_t)0;
            if (p.zeros) out[kWqChunkCodes + p.gpc * 64 + i] = in ? p.zeros[at] & 15 : 0;
        }
    }
}

// --- Quantisation ------------------------------------------------------------------
//
// Bound by the weight's bytes, read once (2·K·N) and written back at a quarter:
// 8192x28672 with zero points 126 us, 4.7 TB/s (70% of a copy).  Loads and stores alone
// take 115 us (a block is loaded, then worked on, then stored, two blocks to an SM); the
// arithmetic hides behind them but for the last of it, since it works on two columns at
// once (141 us with a column at a time).

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Scale and zero point of a group from its extremes (0 included).
__device__ __forceinline__ void wq_group_scale(float lo, float hi, bool zeros, float &scale, float &zero)
{
    const float span = zeros ? (hi - lo) * (1.0f / 15.0f) : fmaxf(hi, -lo) * (1.0f / 7.0f);
    scale = __bfloat162float(__float2bfloat16_rn(span));
    if (scale == 0.0f) scale = 1.0f;
    zero = zeros ? fminf(fmaxf(rintf(__fdiv_rn(-lo, scale)), 0.0f), 15.0f) : 8.0f;
}

// Any N, any group: one thread to a pair of columns and a group, the extremes in
// one walk along K, the codes in another (served by the caches).
__global__ void __launch_bounds__(128) wq_quantize_any_kernel(const WqQuantParams p)
{
    const int64_t nb = (p.N + 1) / 2;
    const int64_t pair = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (pair >= nb) return;
    const int n0 = (int)(2 * pair);
    const bool two = n0 + 1 < p.N;
    const __nv_bfloat16 *w = static_cast<const __nv_bfloat16 *>(p.w);
    const int group = p.group > 0 ? p.group : p.K;
    for (int64_t gi = blockIdx.y; gi * group < p.K; gi += gridDim.y) {
        const int64_t k0 = gi * group, k1 = min((int64_t)p.K, k0 + group);
        float lo[2] = {0.0f, 0.0f}, hi[2] = {0.0f, 0.0f};
#pragma unroll 8
        for (int64_t k = k0; k < k1; ++k)
            for (int c = 0; c < (two ? 2 : 1); ++c) {
                const float v = __bfloat162float(w[k * p.N + n0 + c]);
                lo[c] = fminf(lo[c], v);
                hi[c] = fmaxf(hi[c], v);
            }
        float scale[2], zero[2];
        for (int c = 0; c < 2; ++c) wq_group_scale(lo[c], hi[c], p.zeros != nullptr, scale[c], zero[c]);
#pragma unroll 4
        for (int64_t k = k0; k < k1; ++k) {
            uint32_t byte = 0;
            for (int c = 0; c < (two ? 2 : 1); ++c) {
                const float v = __bfloat162float(w[k * p.N + n0 + c]);
                const float q = fminf(fmaxf(rintf(__fdiv_rn(v, scale[c])) + zero[c], 0.0f), 15.0f);
                byte |= (uint32_t)q << (4 * c);
            }
            p.codes[k * nb + pair] = (uint8_t)byte;
        }
        for (int c = 0; c < (two ? 2 : 1); ++c) {
            static_cast<__nv_bfloat16 *>(p.scales)[gi * p.N + n0 + c] = __float2bfloat16_rn(scale[c]);
            if (p.zeros) p.zeros[gi * p.N + n0 + c] = (uint8_t)zero[c];
        }
    }
}

// N a multiple of 8 and a group of at most 16·STRIPS rows (the kernel above takes
// twice as long: 260 us at 8192x28672, 30 at 1024x4096 against 15): a block of 16·STRIPS rows
// by 256 columns stays in registers (a warp a strip of 16 rows, 16 bytes of each a
// lane) between the extremes and the codes, so the weight is read once.
//
// rint(w / s) without a division: w / s is a ratio of two 8-bit significands, so
// where it is not exactly between two integers it is at least 2^-11 away from
// there (|w / s| <= 16).  w · (1/s), off by 2^-20 at most, is rounded to multiples
// of 2^-12 by adding 2560 and so stays on its side, and a tie is exactly a tie
// again, which adding 1.5·2^23 rounds to even as the division would.
template <int STRIPS>
__global__ void __launch_bounds__(32 * STRIPS, STRIPS == 8 ? 2 : 1) wq_quantize_kernel(const WqQuantParams p)
{
    constexpr int kRows = 16 * STRIPS, kThreads = 32 * STRIPS;
    __shared__ __nv_bfloat162 ext[2][STRIPS][128];     // extremes by strip
    __shared__ float tab[2][kRows / 32][256];          // scales and zero points by group
    const int strip = threadIdx.x >> 5, col = (threadIdx.x & 31) * 8;
    const int64_t n0 = (int64_t)blockIdx.x * 256 + col, k0 = (int64_t)blockIdx.y * kRows + strip * 16;
    const bool in = n0 < p.N;
    const __nv_bfloat16 *w = static_cast<const __nv_bfloat16 *>(p.w);
    uint4 v[16];
#pragma unroll
    for (int r = 0; r < 16; ++r)
        v[r] = in && k0 + r < p.K ? __ldcs(reinterpret_cast<const uint4 *>(w + (k0 + r) * p.N + n0)) : make_uint4(0, 0, 0, 0);
    __nv_bfloat162 lo[4], hi[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) lo[c] = hi[c] = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(&v[r]);
#pragma unroll
        for (int c = 0; c < 4; ++c) lo[c] = __hmin2(lo[c], b[c]), hi[c] = __hmax2(hi[c], b[c]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) ext[0][strip][col / 2 + c] = lo[c], ext[1][strip][col / 2 + c] = hi[c];
    __syncthreads();
    const int groups = kRows / p.group, strips = p.group / 16;
    for (int i = threadIdx.x; i < groups * 256; i += kThreads) {
        const int gi = i >> 8, c = i & 255;
        float l = 0.0f, h = 0.0f;
        for (int q = 0; q < strips; ++q) {
            const float2 l2 = __bfloat1622float2(ext[0][gi * strips + q][c >> 1]);
            const float2 h2 = __bfloat1622float2(ext[1][gi * strips + q][c >> 1]);
            l = fminf(l, c & 1 ? l2.y : l2.x), h = fmaxf(h, c & 1 ? h2.y : h2.x);
        }
        float scale, zero;
        wq_group_scale(l, h, p.zeros != nullptr, scale, zero);
        tab[0][gi][c] = scale;
        tab[1][gi][c] = zero;
        const int64_t n = (int64_t)blockIdx.x * 256 + c, row = (int64_t)blockIdx.y * groups + gi;
        if (n < p.N && row * p.group < p.K) {
            static_cast<__nv_bfloat16 *>(p.scales)[row * p.N + n] = __float2bfloat16_rn(scale);
            if (p.zeros) p.zeros[row * p.N + n] = (uint8_t)zero;
        }
    }
    __syncthreads();
    if (!in) return;
    const int gi = strip * 16 / p.group;
    float scale[8], inv[8];
    int zero[8];
    bool tiny = false;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        scale[c] = tab[0][gi][col + c];
        zero[c] = (int)tab[1][gi][col + c];
        inv[c] = __frcp_rn(scale[c]);
        tiny |= scale[c] < 1e-36f;               // its reciprocal may not be finite
    }
    const int64_t nb = p.N / 2;
    const int rows = (int)min((int64_t)16, p.K - k0);
    uint8_t *out = p.codes + k0 * nb + n0 / 2;
    if (tiny) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const uint32_t ws[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
            uint32_t word = 0;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float x = c & 1 ? bf16_hi(ws[c >> 1]) : bf16_lo(ws[c >> 1]);
                word |= (uint32_t)min(max((int)rintf(__fdiv_rn(x, scale[c])) + zero[c], 0), 15) << (4 * c);
            }
            if (r < rows) *reinterpret_cast<uint32_t *>(out + r * nb) = word;
        }
        return;
    }
    // Columns c and c + 4 side by side: fp32 pairs, then 16-bit halves.
    float2 inv2[4];
    uint32_t zero2[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        inv2[c] = make_float2(inv[c], inv[c + 4]);
        zero2[c] = (uint32_t)zero[c] | (uint32_t)zero[c + 4] << 16;
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const uint32_t ws[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
        uint32_t word = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t a = ws[c >> 1], b = ws[(c >> 1) + 2];
            const float2 x = c & 1 ? make_float2(bf16_hi(a), bf16_hi(b)) : make_float2(bf16_lo(a), bf16_lo(b));
            // 1.5·2^23 + rint(x / scale): its low half is the integer
            const float2 q = add2(fma2(x, inv2[c], make_float2(2560.0f, 2560.0f)), make_float2(12580352.0f, 12580352.0f));
            const uint32_t n = __byte_perm(__float_as_uint(q.x), __float_as_uint(q.y), 0x5410);
            word += __viaddmin_s16x2_relu(n, zero2[c], 0x000F000Fu) << (4 * c);   // + zero point, within 0..15
        }
        if (r < rows) *reinterpret_cast<uint32_t *>(out + r * nb) = word;
    }
}

template <bool JOIN>
const void *wq_fn(int nt)
{
    return nt == 1   ? (const void *)wq_kernel<1, JOIN>
           : nt == 2 ? (const void *)wq_kernel<2, JOIN>
           : nt == 4 ? (const void *)wq_kernel<4, JOIN>
                     : (const void *)wq_kernel<8, JOIN>;
}

}  // namespace

cudaError_t wq_set_smem_limit(int bytes)
{
    for (int nt = 1; nt <= 8; nt *= 2)
        for (const void *f : {wq_fn<false>(nt), wq_fn<true>(nt)}) {
            cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

cudaError_t launch_wq(int nt, const CUtensorMap &x, const WqParams &p, int grid, int smem, cudaStream_t stream)
{
    void *args[] = {const_cast<CUtensorMap *>(&x), const_cast<WqParams *>(&p)};
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(ft_threads(FT_PRODUCT, nt));
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    // May start while the previous kernel drains (griddepcontrol.wait above).
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, p.cluster > 1 ? wq_fn<true>(nt) : wq_fn<false>(nt), args);
}

cudaError_t launch_wq_prepare(const WqPrepareParams &p, cudaStream_t stream)
{
    void *args[] = {const_cast<WqPrepareParams *>(&p)};
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)(((int64_t)p.T * p.nkb + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, (const void *)wq_prepare_kernel, args);
}

cudaError_t launch_wq_pack(const WqPackParams &p, cudaStream_t stream)
{
    const int64_t chunks = (int64_t)p.ncg * p.nkb * p.mats;
    const int grid = (int)(chunks < 152 * 8 ? chunks : 152 * 8);
    wq_pack_kernel<<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_wq_quantize(const WqQuantParams &p, cudaStream_t stream)
{
    const bool wide = p.N % 8 == 0 && p.group > 0 && ((uintptr_t)p.w & 15u) == 0 && ((uintptr_t)p.codes & 3u) == 0;
    const int rows = p.group > 128 ? 256 : 128;
    const int64_t bands = ((int64_t)p.K + rows - 1) / rows;
    if (wide && bands <= 65535) {
        const dim3 grid((unsigned)((p.N + 255) / 256), (unsigned)bands);
        if (rows == 128) wq_quantize_kernel<8><<<grid, 256, 0, stream>>>(p);
        else wq_quantize_kernel<16><<<grid, 512, 0, stream>>>(p);
        return cudaGetLastError();
    }
    const int64_t nb = ((int64_t)p.N + 1) / 2, ng = p.group > 0 ? ((int64_t)p.K + p.group - 1) / p.group : 1;
    const dim3 grid((unsigned)((nb + 127) / 128), (unsigned)(ng < 32768 ? ng : 32768));
    wq_quantize_any_kernel<<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gemmgb
