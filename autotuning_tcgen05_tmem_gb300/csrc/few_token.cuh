// Device code shared by the few-token kernels: fragments, the two weight
// formats' inner loops, and the exchange of partial tiles.
//
// All of them compute Cᵀ: the weights' columns are the M side of
// mma.sync and the tokens its N side, so that 1 to 8 tokens cost one instruction
// and no weight is read for a padded row.  These products are bound
// by the bytes of the weights (at 64 tokens a bf16 weight meets 64
// multiply-adds for 2 bytes), so what matters is the stream: weights go from
// global memory to a shared-memory ring by bulk copies, tens of KB ahead of
// the warps that multiply, and every CTA takes an equal share of the whole
// reduction whatever the shape.
//
// Why not the fifth-generation tensor core: codes expanded into tensor memory, tokens as
// its shared-memory operand and sums scaled on their way out came to 41 us for 16 tokens
// 4096x28672 and 57 us for 64 tokens 14336x4096, where this form takes 26 and 41.
// Issuing the multiplications (5 us of the 57) did not bound it; expanding the codes did,
// and the 33 KB of tokens copied with each step's 17 KB of weights.  Tokens that stay in
// shared memory over several tiles ask for another kernel.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "few_token.h"
#include "ptx.cuh"

namespace gemmgb {
namespace {

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first of a sum: the accumulator starts at zero.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Activations in fp32.  GELU is the erf form through erfc, which keeps its
// relative accuracy for negative arguments; SiLU x / (1 + e^-x) is -0 at -inf's
// side (e^-x = inf), as the limit is 0.
__device__ __forceinline__ float ft_act(float v, int act)
{
    if (act == FT_ACT_RELU) return v > 0.0f ? v : (v != v ? v : 0.0f);
    if (act == FT_ACT_GELU) return 0.5f * v * erfcf(-v * 0.70710678118654752440f);
    if (act == FT_ACT_SILU) return v / (1.0f + expf(-v));
    return v;
}

// Fragment accumulators of one warp: 32 weight columns (two 16-row halves of
// the MMA) by 8·NT tokens.  acc[mi][nt]: {row g, tokens 2t and 2t+1; row g+8}.
template <int NT>
struct Acc {
    float v[2][NT][4];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) v[m][n][i] = 0.0f;
    }
};

// A launch's parameters come through the constant cache, whose first read of every
// line takes most of a microsecond: one warp for each 64 bytes reads them all at
// the start, side by side, instead of the code one after another.
template <typename P>
__device__ __forceinline__ void ft_touch_params(const P &p, int warp)
{
    static_assert(sizeof(P) <= 64 * 8, "a line for each of eight warps");
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i * 16 < (int)(sizeof(P) / 4) && warp == i)
            asm volatile("" ::"r"(reinterpret_cast<const int32_t *>(&p)[i * 16]));
}

// --- The ring ------------------------------------------------------------------
//
// A position in it: slots in turn, the barriers' phase flipping with each lap.
struct RingPos {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next(int stages)
    {
        if (++slot == (uint32_t)stages) slot = 0, phase ^= 1u;
    }
    __device__ __forceinline__ void skip(int n, int stages)   // n <= stages
    {
        slot += (uint32_t)n;
        if (slot >= (uint32_t)stages) slot -= (uint32_t)stages, phase ^= 1u;
    }
};

struct Ring {
    uint32_t data, stage_bytes, full0, empty0, ready0;
    int stages;
    __device__ __forceinline__ uint32_t stage(const RingPos &r) const { return data + r.slot * stage_bytes; }
    __device__ __forceinline__ uint32_t full(const RingPos &r) const { return full0 + 8u * r.slot; }
    __device__ __forceinline__ uint32_t ready(const RingPos &r) const { return ready0 + 8u * r.slot; }
    __device__ __forceinline__ uint32_t empty(const RingPos &r) const { return empty0 + 8u * r.slot; }
    // The copying warp's side: a slot's first lap is free.
    __device__ __forceinline__ bool wait_empty(const RingPos &r, const WaitCtl &c) const
    {
        return wait_bar(empty(r), r.phase ^ 1u, c, SITE_PRODUCER_EMPTY);
    }
    __device__ __forceinline__ void wait_full(const RingPos &r, const WaitCtl &c) const
    {
        wait_bar(full(r), r.phase, c, SITE_MMA_FULL);
    }
};

// Barriers, flags and constants of a CTA; one thread.  `leave`: warps that leave a
// slot of the ring.
__device__ __forceinline__ void ft_init_shared(uint8_t *gbase, const Ring &ring, int leave, int converters, int workers)
{
    const uint32_t base = smem_u32(gbase);
    for (int s = 0; s < ring.stages; ++s) {
        mbar_init(ring.full0 + 8u * s, 1);
        mbar_init(ring.empty0 + 8u * s, leave);
        if (converters) mbar_init(ring.ready0 + 8u * s, converters);
    }
    for (int i = 0; i < 2; ++i) {
        mbar_init(base + kFtHandFull + 8u * i, workers / 32);
        mbar_init(base + kFtHandEmpty + 8u * i, kFtStorers / 32);
        reinterpret_cast<volatile int32_t *>(gbase + kFtFlags)[i] = 0;
    }
    for (int i = 0; i < 8; ++i) reinterpret_cast<uint32_t *>(gbase + kFtEights)[i] = 0x08080808u;
}

// A worker's walk over the steps of its CTA, of which every KP-th is its own (number
// `part` of each KP).  `bars`: the barriers that announce a slot (full, or ready:
// whoever converted the slot's activations saw its copies land, and so does who
// sees that).
//
// A phase bit tells a lap of the ring from the next only to who has seen every lap.
// So the ring's slots number a multiple of KP, which makes a worker's slots its own
// for good; or (ALL, where KP changes from expert to expert, or the slots are odd) it
// waits for the others' steps too and leaves their slots as it does its own.
//
// The next barrier is probed before the work on a step, which hides the probe (about
// 170 cycles beside a busy shared memory) where the slot is there.
template <int KP, bool ALL>
struct StepWalk {
    uint32_t bars;
    RingPos pos;       // of the next own step (ALL: of the next step)
    int ahead;         // steps of the stream before it
    bool seen;
    __device__ __forceinline__ void start(uint32_t bars_, int part, int stages)
    {
        bars = bars_;
        ahead = ALL ? 0 : part;
        seen = false;
        if (ahead) pos.skip(ahead, stages);
    }
    // Calls work(position, own) for the own ones of the stream's next n steps.  ALL: for
    // all of them, of which every kp-th from `part` on is its own.
    template <typename F>
    __device__ __forceinline__ void run(int n, int stages, const WaitCtl &c, int part, int kp, F work)
    {
        int turn = 0;
        for (; ahead < n; ahead += ALL ? 1 : KP) {
            if (!seen) wait_bar(bars + 8u * pos.slot, pos.phase, c, SITE_MMA_FULL);
            __syncwarp();   // lanes may have seen it at different probes; fragments want them together
            const RingPos here = pos;
            pos.skip(ALL ? 1 : KP, stages);
            seen = __all_sync(0xFFFFFFFFu, mbar_test_wait(bars + 8u * pos.slot, pos.phase));
            work(here, !ALL || turn == part);
            if (ALL) turn = turn + 1 == kp ? 0 : turn + 1;
        }
        ahead -= n;
    }
};

// Token pieces of a step: `boxes` spans of 64 K from span `box0` on, rows from
// `row` on, as one copy where the map views the matrix in spans.
__device__ __forceinline__ void load_tokens(uint32_t dst, const CUtensorMap *m, uint32_t bar, int box0, int boxes, int row,
                                            uint32_t box_bytes, int spans)
{
    if (spans) {
        tma_load_3d(dst, m, bar, 0, row, box0);
    } else {
        for (int b = 0; b < boxes; ++b) tma_load_2d(dst + (uint32_t)b * box_bytes, m, bar, (box0 + b) * 64, row);
    }
}

// --- 4-bit weights ---------------------------------------------------------------
//
// The products run in mma.m16n8k16 on fp16 operands, exactly:
//   * a code q (0..15) in the low bits of a half is the fp16 subnormal q·2^-24, four
//     bits higher q·2^-20: codes become operands by a mask (five instructions for
//     eight codes; placing them under an exponent and subtracting it again, as
//     their conversion to bf16 needs, takes eleven);
//   * a bf16 activation has eight significant bits and fits fp16's eleven once a
//     power of two brings the largest of its 256 of K into [2^14, 2^15).  Those that
//     meet the codes four bits up are a sixteenth of it.  Only values below 2^-25
//     of the largest lose bits, and at most 2^-35 of it.
// Σ (q - z)·x over a group is then Σ q·x from the tensor core (fp32 sums) minus
// z·Σ x; the group's scale and the activations' power of two multiply it in fp32.
// No weight is ever rounded.
//
// Activations in a stage: one row of 512 bytes for each token, 256 bf16 as they
// come, converted in place: the 16 bytes at (j ^ (row % 8))·64 + t·16 are
// k = 32j + 8t .. + 7.  Beside them (off_meta) for each token its power of two and,
// for each group, its sum.  Where a row of 256 holds an infinity the power of two is NaN,
// which makes the token's sums NaN; ft_resolve finds what they are.

// Conversion of R rows of 256 at once (so that their latencies overlap; one warp, 16
// bytes w[q] of each a lane): out[q] the lane's 16 bytes, scale[q] the power of two
// (all lanes), sum[q] the sum over the lane's group in the codes' unit.
//
// Rows are bf16, or (powers not 0) rows of h of 4-bit experts: fp16 with a power of two
// for each 64, the row's four at powers + 16·r[q], infinite where the 64 hold an infinity or
// NaN.  Brought to the row's largest power only values below 2^-20 of the
// largest lose bits.
template <int R>
__device__ __forceinline__ void ft_convert(const uint32_t (&w)[R][4], uint32_t powers, const int (&r)[R], int lane, int gpc,
                                           uint32_t (&out)[R][4], float (&scale)[R], float (&sum)[R])
{
    float f[R];            // of the lane's values
    if (powers) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const float4 all = ld_shared_v4(powers + (uint32_t)r[q] * 16u);
            const float e = (lane & 16) ? (lane & 8 ? all.w : all.z) : lane & 8 ? all.y : all.x;
            scale[q] = fmaxf(fmaxf(all.x, all.y), fmaxf(all.z, all.w));
            f[q] = e * __uint_as_float(0x7F000000u - __float_as_uint(scale[q]));   // 1 over a power of two
            if (scale[q] == INFINITY) scale[q] = NAN;
        }
    } else {
#pragma unroll
        for (int q = 0; q < R; ++q) {
            auto abs2 = [](uint32_t u) { return __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&u)); };
            const __nv_bfloat162 mx = __hmax2(__hmax2(abs2(w[q][0]), abs2(w[q][1])), __hmax2(abs2(w[q][2]), abs2(w[q][3])));
            const uint32_t mb = *reinterpret_cast<const uint32_t *>(&mx);
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, max(mb & 0xFFFFu, mb >> 16)) << 16;
            const uint32_t e = max(top >> 23, 15u);                               // biased exponent of the largest
            f[q] = __uint_as_float((268u - min(e, 254u)) << 23);                  // 2^(14 - exponent)
            scale[q] = e == 255u ? NAN : __uint_as_float((e - 14u) << 23);   // 2^(exponent - 14)
        }
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
        float xs[8];
        if (powers) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&w[q][k]));
                xs[2 * k] = h.x, xs[2 * k + 1] = h.y;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) xs[2 * k] = bf16_lo(w[q][k]), xs[2 * k + 1] = bf16_hi(w[q][k]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) xs[k] *= k & 2 ? f[q] * 0.0625f : f[q];
        sum[q] = fmaf(xs[2] + xs[3] + (xs[6] + xs[7]), 16.0f, xs[0] + xs[1] + (xs[4] + xs[5]));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __half2 h = __floats2half2_rn(xs[2 * k], xs[2 * k + 1]);
            out[q][k] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        if (o >= 4 && o * gpc >= 32) break;                           // blocks of one group
#pragma unroll
        for (int q = 0; q < R; ++q) sum[q] += __shfl_xor_sync(0xFFFFFFFFu, sum[q], o);
    }
#pragma unroll
    for (int q = 0; q < R; ++q) sum[q] *= 5.9604644775390625e-8f;     // 2^-24
}

// Place of a lane's 16 bytes in row r.
__device__ __forceinline__ uint32_t ft_converted_place(int r, int lane)
{
    return (uint32_t)((((lane >> 2) ^ (r & 7)) * 4 + (lane & 3)) * 16);
}

// Converts rows of a stage in place (one warp): row r[q] of the tile is token column
// i[q], and only the first n count.
template <int R>
__device__ __forceinline__ void ft_convert_rows(uint32_t x, uint32_t powers, const int (&r)[R], const int (&i)[R], int n,
                                                float *meta, int t8, int gpc, int lane)
{
    uint32_t w[R][4], out[R][4];
    float scale[R], sum[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
        const uint4 v = lds128(x + (uint32_t)r[q] * 512u + (uint32_t)lane * 16u);
        w[q][0] = v.x, w[q][1] = v.y, w[q][2] = v.z, w[q][3] = v.w;
    }
    ft_convert<R>(w, powers, r, lane, gpc, out, scale, sum);
    __syncwarp();                                                     // every lane holds its 16 bytes
#pragma unroll
    for (int q = 0; q < R; ++q) {
        if (q >= n) break;
        st_shared_v4(x + (uint32_t)r[q] * 512u + ft_converted_place(r[q], lane), out[q][0], out[q][1], out[q][2], out[q][3]);
        if (lane == 0) meta[i[q]] = scale[q];
        if ((lane & 3) == 0) meta[(1 + ((lane >> 2) * gpc >> 3)) * t8 + i[q]] = sum[q];
    }
}

// A converting warp's part of a step: of the token columns 0..n_tok-1, whose rows
// row(i) gives, every `warps`-th from `first` on (`first` changes from step to step,
// so that few tokens keep all warps busy).  A warp without a token waits and arrives
// like the others: its arrival is what holds the slot until it has seen this lap.
template <typename F>
__device__ __forceinline__ void ft_convert_step(const Ring &ring, const RingPos &pos, const WaitCtl &ctl, uint32_t x,
                                                uint32_t powers, int n_tok, int first, int warps, F row, float *meta,
                                                int t8, int gpc, int lane)
{
    ring.wait_full(pos, ctl);
    int i = first;
    for (; i + warps < n_tok; i += 3 * warps) {
        const int c[3] = {i, i + warps, min(i + 2 * warps, n_tok - 1)};
        const int r[3] = {row(c[0]), row(c[1]), row(c[2])};
        ft_convert_rows<3>(x, powers, r, c, i + 2 * warps < n_tok ? 3 : 2, meta, t8, gpc, lane);
    }
    if (i < n_tok) {
        const int c[1] = {i}, r[1] = {row(i)};
        ft_convert_rows<1>(x, powers, r, c, 1, meta, t8, gpc, lane);
    }
    fence_proxy_async_smem();   // the slot's next copy writes what plain stores wrote here
    __syncwarp();
    if (lane == 0) mbar_arrive(ring.ready(pos));
}

// acc += scale · Σ (code - zero) · x · 2^-24 over a chunk's 32 columns and 256 K in
// groups of GB·32, for 8·NW tokens: xrow[n] this lane's row (of the fragment's
// column lane/4), tok0 the first column in the meta data.  Zero points lie at
// `zeros`, zstride bytes from group to group.
template <int NW, int GB>
__device__ __forceinline__ void ft_groups_w4(uint32_t chunk, uint32_t zeros, uint32_t zstride, uint32_t xbase,
                                             const float *meta, int t8, int tok0, const uint32_t (&xrow)[NW], int lane,
                                             Acc<NW> &acc)
{
    const int g = lane >> 2, t = lane & 3;
    const uint32_t wl = chunk + (uint32_t)lane * 16u, sl = chunk + kWqChunkCodes + (uint32_t)g * 8u;
    meta += tok0 + 2 * t;
    uint32_t xl[NW];   // block j's 16 bytes are at xl ^ 64·j (rows are 512-byte aligned)
#pragma unroll
    for (int n = 0; n < NW; ++n) xl[n] = xbase + xrow[n] * 512u + (xrow[n] & 7u) * 64u + (uint32_t)t * 16u;
    // Of several groups in a chunk the activations' power of two multiplies the sum
    // once (few tokens: many accumulators leave no registers for it).
    constexpr bool kOnce = NW < 4 && GB < 8;
    float part[kOnce ? 2 : 1][kOnce ? NW : 1][4];
#pragma unroll(NW >= 4 ? 1 : 8)
    for (int gi = 0; gi < 8 / GB; ++gi) {
        float sum[2][NW][4];
        if constexpr (NW >= 4) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NW; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[m][n][i] = 0.0f;
        }
        // Many accumulators leave no registers to unroll with.
#pragma unroll(NW >= 4 ? 1 : 8)
        for (int b = 0; b < GB; ++b) {
            const uint32_t j = (uint32_t)(gi * GB + b);
            const uint4 w = lds128(wl + j * 512u);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
            uint32_t a[4][4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint32_t up = ws[s] >> 8;
                a[s][0] = ws[s] & 0x000F000Fu, a[s][1] = ws[s] & 0x00F000F0u;
                a[s][2] = up & 0x000F000Fu, a[s][3] = up & 0x00F000F0u;
            }
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                const uint4 x = lds128(xl[n] ^ (j * 64u));
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    if (NW < 4 && b == 0)
                        mma_f16_first(sum[m][n], a[2 * m][0], a[2 * m + 1][0], a[2 * m][1], a[2 * m + 1][1], x.x, x.y);
                    else
                        mma_f16(sum[m][n], a[2 * m][0], a[2 * m + 1][0], a[2 * m][1], a[2 * m + 1][1], x.x, x.y);
                    mma_f16(sum[m][n], a[2 * m][2], a[2 * m + 1][2], a[2 * m][3], a[2 * m + 1][3], x.z, x.w);
                }
            }
        }
        const uint2 s4 = lds64(sl + (uint32_t)(gi * 64));
        const float sc[4] = {bf16_lo(s4.x), bf16_hi(s4.x), bf16_lo(s4.y), bf16_hi(s4.y)};
        const uint32_t z4 = lds32(zeros + (uint32_t)gi * zstride + (uint32_t)g * 4u);
        float z[4];   // a byte under the exponent of 2^23, less 2^23
#pragma unroll
        for (int s = 0; s < 4; ++s) z[s] = __uint_as_float(__byte_perm(z4, 0x4B000000u, 0x7440u | s)) - 8388608.0f;
#pragma unroll
        for (int n = 0; n < NW; ++n) {
            const float2 sx = *reinterpret_cast<const float2 *>(meta + (1 + gi) * t8 + n * 8);
            float2 p2 = make_float2(1.0f, 1.0f);
            if constexpr (!kOnce) p2 = *reinterpret_cast<const float2 *>(meta + n * 8);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int s = 2 * m + (i >> 1);
                    const float inner = fmaf(-z[s], i & 1 ? sx.y : sx.x, sum[m][n][i]);
                    if constexpr (kOnce) part[m][n][i] = gi == 0 ? sc[s] * inner : fmaf(sc[s], inner, part[m][n][i]);
                    else acc.v[m][n][i] = fmaf(sc[s] * (i & 1 ? p2.y : p2.x), inner, acc.v[m][n][i]);
                }
        }
    }
    if constexpr (kOnce) {
#pragma unroll
        for (int n = 0; n < NW; ++n) {
            const float2 p2 = *reinterpret_cast<const float2 *>(meta + n * 8);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc.v[m][n][i] = fmaf(i & 1 ? p2.y : p2.x, part[m][n][i], acc.v[m][n][i]);
        }
    }
}

template <int NW>
__device__ __forceinline__ void ft_chunk_w4(uint32_t chunk, uint32_t eights, uint32_t xbase, const float *meta, int t8,
                                            int tok0, const uint32_t (&xrow)[NW], int gpc, int has_zeros, int lane,
                                            Acc<NW> &acc)
{
    const uint32_t zeros = has_zeros ? chunk + kWqChunkCodes + (uint32_t)gpc * 64u : eights;
    const uint32_t zstride = has_zeros ? 32u : 0u;
    if (gpc == 2) ft_groups_w4<NW, 4>(chunk, zeros, zstride, xbase, meta, t8, tok0, xrow, lane, acc);
    else if (gpc == 4) ft_groups_w4<NW, 2>(chunk, zeros, zstride, xbase, meta, t8, tok0, xrow, lane, acc);
    else if (gpc == 1) ft_groups_w4<NW, 8>(chunk, zeros, zstride, xbase, meta, t8, tok0, xrow, lane, acc);
    else ft_groups_w4<NW, 1>(chunk, zeros, zstride, xbase, meta, t8, tok0, xrow, lane, acc);
}

// The accumulators' unit, 2^-24, undone.
template <int NW>
__device__ __forceinline__ void ft_scale_w4(Acc<NW> &acc)
{
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NW; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc.v[m][n][i] *= 16777216.0f;
}

// A sum that is not finite, as the definition gives it.  Where the activations hold
// infinities or NaN it is the sum of (code - zero) · scale · x over those alone, product by
// product: an infinity, or NaN (of opposite ones, of a code that is its zero point).
// Otherwise it stands as it is (v).  Read again from global memory, by the storers where they
// meet such a sum: a look at each step's powers cost the products 3%.  (A lean function of
// its own: one with more registers, called or not, cost the kernels 4 to 10%.)
//
// chunk: of the column group, K block 0; step: bytes from one K block to the next; where:
// row (of 32) + 32·gpc + 512·has_zeros.
//
// Adds what eight activations from k on (16-bit, of a size from `least` on: infinities, and
// NaN above `nan`) make of their weights.
__device__ __forceinline__ void ft_add_special(const uint8_t *chunk, uint32_t step, uint32_t where, int k, const uint4 &u,
                                               uint32_t least, uint32_t nan, float &sum)
{
    const uint8_t *const c = chunk + (int64_t)(k >> 8) * step;
    const int row = where & 31, gpc = where >> 5 & 15, j = k >> 5 & 7;
    const int at = (j * gpc >> 3) * 32 + (row & 7) * 4 + (row >> 3);
    const uint32_t word = *reinterpret_cast<const uint32_t *>(c + j * 512 + ((row & 7) * 4 + (k >> 3 & 3)) * 16 + (row >> 3) * 4);
    const float scale = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(c + kWqChunkCodes)[at]);
    const int zero = where >> 9 ? c[kWqChunkCodes + gpc * 64 + at] : 8;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
        const uint32_t e = (i < 4 ? (i < 2 ? u.x : u.y) : (i < 6 ? u.z : u.w)) >> (16 * (i & 1)), size = e & 0x7FFFu;
        if (size < least) continue;
        const int code = (int)(word >> (4 * ((i >> 1) + 4 * (i & 1))) & 15u);
        sum += (float)(code - zero) * scale * (size > nan ? NAN : e & 0x8000u ? -INFINITY : INFINITY);
    }
}

// x: the token's row of K bf16 (K a multiple of 8).
__device__ __noinline__ float ft_resolve(const uint8_t *chunk, uint32_t step, uint32_t where, const __nv_bfloat16 *x, int K,
                                         float v)
{
    float sum = 0.0f;
#pragma unroll 1
    for (int k = 0; k < K; k += 8) {
        const uint4 u = *reinterpret_cast<const uint4 *>(x + k);
        auto any = [](uint32_t w) { return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; };
        if (!any(u.x) && !any(u.y) && !any(u.z) && !any(u.w)) continue;
        ft_add_special(chunk, step, where, k, u, 0x7F80u, 0x7F80u, sum);
        if (sum != sum) break;
    }
    return sum != 0.0f ? sum : v;   // (an infinity or NaN, once there is one)
}

// --- bf16 weights ----------------------------------------------------------------
//
// acc += W · x over 32 of K, from k0 on, of a box of 64 columns: a [K][64 columns]
// piece of the row-major weight with 128-byte swizzled rows.  `mh` picks the
// warp's 32 columns: plain, columns 32·mh + 16·m + row; gated (32 gate columns,
// then 32 up), features 16·mh + 8·m + g with the gate in the fragment's rows g
// and the up in rows g + 8.  xbox: the tokens' 64 K that hold k0; xlow: those of
// their second bf16 part (kept h, down phase), 0 where they have one part.
template <int NT>
__device__ __forceinline__ void ft_box_bf16(uint32_t box, int mh, int k0, bool gated, uint32_t xbox, uint32_t xlow,
                                            const uint32_t (&xrow)[NT], int lane, Acc<NT> &acc)
{
    uint32_t a[2][2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const uint32_t krow = (uint32_t)(k0 + ks * 16 + ((lane >> 4) & 1) * 8 + (lane & 7));
            const uint32_t mt = (uint32_t)(2 * mh + m), hi = (uint32_t)((lane >> 3) & 1);
            const uint32_t ck = gated ? mt + 4 * hi : 2 * mt + hi;
            ldmatrix_x4_trans(box + krow * 128u + ((ck ^ (krow & 7u)) << 4), a[m][ks]);
        }
    const uint32_t cx = (uint32_t)((k0 & 32) / 8 + (lane >> 3));
    auto multiply = [&](uint32_t box_of_tokens) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            uint32_t b[4];
            ldmatrix_x4(box_of_tokens + xrow[n] * 128u + ((cx ^ (xrow[n] & 7u)) << 4), b);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                mma_bf16(acc.v[m][n], a[m][0][0], a[m][0][1], a[m][0][2], a[m][0][3], b[0], b[1]);
                mma_bf16(acc.v[m][n], a[m][1][0], a[m][1][1], a[m][1][2], a[m][1][3], b[2], b[3]);
            }
        }
    };
    multiply(xbox);
    if (xlow) multiply(xlow);
}

// --- Sums across the warps of a CTA ------------------------------------------------
//
// [token][row], rows padded by 4 (conflict-free for the fragment's layout).
constexpr int kFtRowStride = kFtTileRows + 4;

template <int NW>
__device__ __forceinline__ void ft_store_red(float *red, int rstride, int row0, int tok0, int lane, const Acc<NW> &acc)
{
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NW; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[(tok0 + n * 8 + 2 * t + (i & 1)) * rstride + row0 + m * 16 + (i >> 1) * 8 + g] = acc.v[m][n][i];
}

// Hand-over of finished tiles from the workers to the storers: two buffers of sums,
// [K part][token][row], with a barrier each for "full" (all workers) and "empty"
// (all storers).  A RingPos over the two runs along on both sides.
struct HandOver {
    float *red;
    int red_floats, part_floats;       // of a buffer, of a K part
    uint32_t full0, empty0;
    __device__ __forceinline__ float *buffer(const RingPos &h) const { return red + h.slot * red_floats; }
};

// A worker's part: its accumulators (column group warp % 4, tokens from tok0 on).
template <int NW>
__device__ __forceinline__ void ft_hand_over(const HandOver &ho, RingPos &h, const WaitCtl &ctl, int part, int warp, int tok0,
                                             int lane, const Acc<NW> &acc)
{
    wait_bar(ho.empty0 + 8u * h.slot, h.phase ^ 1u, ctl, SITE_MMA_TMEM_EMPTY);
    ft_store_red<NW>(ho.buffer(h) + part * ho.part_floats, kFtRowStride, (warp & 3) * 32, tok0, lane, acc);
    __syncwarp();
    if (lane == 0) mbar_arrive(ho.full0 + 8u * h.slot);
    h.next(2);
}

__device__ __forceinline__ void ft_storers_sync() { named_bar_sync(1, kFtStorers); }

// The storers' side: waits for a tile's sums and adds up the K parts; returns the
// buffer, [token][row] of n_tok tokens, visible to all storers.
__device__ __forceinline__ float *ft_take_over(const HandOver &ho, const RingPos &h, const WaitCtl &ctl, int k_parts, int n_tok,
                                               int tid)
{
    wait_bar(ho.full0 + 8u * h.slot, h.phase, ctl, SITE_EPI_TMEM_FULL);
    float *const buf = ho.buffer(h);
    if (k_parts > 1) {
        for (int e = tid; e < n_tok * (kFtTileRows / 4); e += kFtStorers) {
            float *const at = buf + e / (kFtTileRows / 4) * kFtRowStride + e % (kFtTileRows / 4) * 4;
            float4 a = *reinterpret_cast<const float4 *>(at);
            for (int q = 1; q < k_parts; ++q) {
                const float4 b = *reinterpret_cast<const float4 *>(at + q * ho.part_floats);
                a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
            }
            *reinterpret_cast<float4 *>(at) = a;
        }
    }
    ft_storers_sync();
    return buf;
}

// ... and gives the buffer back.
__device__ __forceinline__ void ft_give_back(const HandOver &ho, RingPos &h, int lane)
{
    __syncwarp();
    if (lane == 0) mbar_arrive(ho.empty0 + 8u * h.slot);
    h.next(2);
}

// --- Tiles cut by a range boundary ---------------------------------------------------
//
// The piece in src[token][row] goes, by the storers, to this CTA's slot of the
// workspace ([cta][first piece of a tile or not][t8][128]); true for the CTA that
// arrives last at the tile's counter, which it clears, and whose src then holds
// the sum of all pieces in K order.
__device__ __noinline__ bool ft_exchange(float *workspace, int t8, float *src, int n_tok, bool first_piece,
                                         int32_t *counter, int first, int pieces, volatile int32_t *flag, int tid)
{
    constexpr int rstride = kFtRowStride, workers = kFtStorers;
    const int64_t slot = (int64_t)t8 * kFtTileRows;
    float *const mine = workspace + (int64_t)(blockIdx.x * 2 + (first_piece ? 1 : 0)) * slot;
    for (int e = tid; e < n_tok * (kFtTileRows / 4); e += workers) {
        const int t = e / (kFtTileRows / 4), r = e % (kFtTileRows / 4) * 4;
        __stcg(reinterpret_cast<float4 *>(mine + t * kFtTileRows + r), *reinterpret_cast<float4 *>(src + t * rstride + r));
    }
    ft_storers_sync();
    if (tid == 0) {
        const int32_t before = atom_acq_rel_gpu_add(counter, 1);
        *flag = before == pieces - 1;
        if (before == pieces - 1) *counter = 0;
    }
    ft_storers_sync();
    if (!*flag) return false;
    // Two places a thread and four pieces at a time: eight loads in flight.
    const int places = n_tok * (kFtTileRows / 4);
    const float *const from = workspace + (int64_t)(first * 2) * slot;
    for (int e0 = tid; e0 < places; e0 += 2 * workers) {
        float4 v[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
            v[u] = e0 + u * workers < places ? __ldcg(reinterpret_cast<const float4 *>(from + slot) + e0 + u * workers)
                                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int q0 = 1; q0 < pieces; q0 += 4) {
            float4 a[4][2];
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (q0 + q < pieces && e0 + u * workers < places)
                        a[q][u] = __ldcg(reinterpret_cast<const float4 *>(from + (int64_t)(2 * (q0 + q)) * slot) + e0 + u * workers);
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (q0 + q < pieces) v[u].x += a[q][u].x, v[u].y += a[q][u].y, v[u].z += a[q][u].z, v[u].w += a[q][u].w;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int e = e0 + u * workers;
            if (e < places)
                *reinterpret_cast<float4 *>(src + e / (kFtTileRows / 4) * rstride + e % (kFtTileRows / 4) * 4) = v[u];
        }
    }
    ft_storers_sync();
    return true;
}

// Row of the tile that holds feature f's gate (its up is 8 rows further).
__device__ __forceinline__ int ft_gate_row(int f) { return 16 * (f >> 3) + (f & 7); }

// Calls f(e, r) for e = tid, tid + workers, ... below n, in batches of B whose loads
// (r = load(e)) are all in flight before the first result is used.
template <int B, typename L, typename F>
__device__ __forceinline__ void ft_batched(int n, int tid, int workers, L load, F f)
{
    for (int e0 = tid; e0 < n; e0 += B * workers) {
        decltype(load(0)) r[B];
#pragma unroll
        for (int u = 0; u < B; ++u)
            if (e0 + u * workers < n) r[u] = load(e0 + u * workers);
#pragma unroll
        for (int u = 0; u < B; ++u)
            if (e0 + u * workers < n) f(e0 + u * workers, r[u]);
    }
}

// --- Equal shares ------------------------------------------------------------------
//
// Range c of a share: its first step (tile·n + step), and the range that holds a
// unit.  Range c starts at unit ⌊units·c/parts⌋.
__device__ __forceinline__ int64_t ft_share_begin(const FtShare &s, int c)
{
    const int64_t u = s.units * c / s.parts;
    return u / s.U * s.n + min((int64_t)s.n, u % s.U * s.L);
}
__device__ __forceinline__ int ft_share_range(const FtShare &s, int64_t unit)
{
    return (int)(((unit + 1) * s.parts - 1) / s.units);
}
// First range and number of ranges that a tile's pieces went to.
__device__ __forceinline__ void ft_share_pieces(const FtShare &s, int tile, int &first, int &pieces)
{
    first = ft_share_range(s, (int64_t)tile * s.U);
    pieces = ft_share_range(s, (int64_t)tile * s.U + s.U - 1) - first + 1;
}

}  // namespace
}  // namespace gemmgb
