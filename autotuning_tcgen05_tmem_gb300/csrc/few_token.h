// Launch records and layouts of the few-token kernels (wq.cu, moe.cu), shared
// by host and device.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gemmgb {

// Warps of a CTA, by kernel and 8-token tiles of the call.  Workers multiply:
// foursomes of one column group of 32 a warp, which share the steps (4-bit: in turn;
// bf16: half of a step's K each; above 32 tokens: half of the tokens each).  A 4-bit
// foursome takes about 1,700 cycles over a step, half of it latency, while the memory
// brings one every 700: as many foursomes of the product as the registers allow (16
// tokens 4096x28672: 25.1 us with three, 25.5 with two).  The expert layer has two: each
// more holds a slot of the ring, of which five or six fit (16 tokens over 4-bit experts:
// 195 us with two, 252 with three).  Four storers take
// the sums of a finished tile from shared memory and exchange, activate and store
// them while the workers go on.  Converters bring the activations of 4-bit steps
// into the form that the products read; the product for more than 8 tokens has them
// prepared by a kernel of their own instead, once and not by every CTA.  One warp
// copies.
enum FtKernel : int { FT_MOE_BF16 = 0, FT_MOE_W4 = 1, FT_PRODUCT = 2 };
__host__ __device__ constexpr int ft_groups(int kernel, int nt) { return kernel != FT_PRODUCT || nt > 2 ? 2 : nt == 2 ? 3 : 4; }
__host__ __device__ constexpr int ft_workers(int kernel, int nt) { return 128 * ft_groups(kernel, nt); }
constexpr int kFtStorers = 128;
__host__ __device__ constexpr bool wq_prepares(int nt) { return nt >= 2; }
__host__ __device__ constexpr int ft_converters(int kernel, int nt)
{
    return kernel == FT_MOE_BF16 ? 0 : kernel == FT_MOE_W4 ? 7 : wq_prepares(nt) ? 0 : 3;
}
__host__ __device__ constexpr int ft_threads(int kernel, int nt)
{
    return ft_workers(kernel, nt) + kFtStorers + 32 * (ft_converters(kernel, nt) + 1);
}
// Token parts and K parts of the workers on an expert of nt tiles in a call of ntmax.
__host__ __device__ constexpr int ft_token_parts(int nt) { return nt > 4 ? 2 : 1; }
__host__ __device__ constexpr int ft_k_parts(int kernel, int ntmax, int nt) { return ft_groups(kernel, ntmax) / ft_token_parts(nt); }
constexpr int kFtMaxTokens = 64;
constexpr int kFtMaxStages = 16;
constexpr int kFtTileRows = 128;                      // weight columns of a full tile
constexpr int kFtCtl = 1024;                          // barriers and flags, ahead of the ring:
constexpr uint32_t kFtFull = 0, kFtEmpty = 8 * kFtMaxStages, kFtReady = 16 * kFtMaxStages;
constexpr uint32_t kFtHandFull = 24 * kFtMaxStages, kFtHandEmpty = kFtHandFull + 16, kFtNever = kFtHandFull + 32;
constexpr uint32_t kFtFlags = kFtHandFull + 48;       // [0] abort, [1] last arrival
constexpr uint32_t kFtEights = 512;                   // the zero points of weights that have none

// --- Packed 4-bit weights ------------------------------------------------------
// A [K, N] weight is cut into chunks of 32 columns x 256 K.  Chunks lie tile by
// tile (four column groups; the last tile may have fewer), along K within a tile,
// column group by column group within a block of K, so that a tile's copy of any
// K range is one contiguous piece.  A chunk holds its codes (4096 bytes), then
// scales (bf16) and zero points (bytes, if any) of its 256/group groups.
//
// Codes: for each 32 of K (j = 0..7), each lane (g = lane/4, t = lane%4) and each
// of four column slots (column 8·slot + g), one word whose nibble i is
// k = 32j + 8t + 2(i%4) + i/4: masking the low nibble of every byte pair, or the
// one above it, gives two codes of one mma fragment register.  Scales and zero
// points of group i: [g][slot].
//
// Gated weights (32 gate and 32 up columns in turn): the chunk's slots 0 and 2
// hold gate columns, 1 and 3 the up columns 32 further on, so that a thread
// finds a gate and its up in the same fragment.
constexpr int kWqChunkCols = 32;
constexpr int kWqChunkK = 256;
constexpr int kWqChunkCodes = kWqChunkCols * kWqChunkK / 2;

__host__ __device__ inline int wq_groups_per_chunk(int group) { return group >= kWqChunkK ? 1 : kWqChunkK / group; }
__host__ __device__ inline int wq_chunk_bytes(int group, int zeros)
{
    return kWqChunkCodes + wq_groups_per_chunk(group) * kWqChunkCols * (zeros ? 3 : 2);
}

// First chunk of tile `tile` at K block kb, in chunks.
__host__ __device__ inline int64_t wq_chunk_index(int ncg, int nkb, int tile, int kb)
{
    const int here = ncg - 4 * tile < 4 ? ncg - 4 * tile : 4;
    return (int64_t)4 * tile * nkb + (int64_t)here * kb;
}

// Column of the weight held by slot `slot`, lane group g of chunk column group c.
__host__ __device__ inline int wq_column(int c, int slot, int g, int gated)
{
    if (!gated) return c * 32 + slot * 8 + g;
    return 64 * (c >> 1) + 16 * (c & 1) + 8 * (slot >> 1) + g + 32 * (slot & 1);
}

// How a phase's work (tiles of n steps each along K) divides over at most `ctas`
// CTAs: every tile falls into U pieces of L steps (the last may be shorter), and
// range c of `parts` takes a contiguous run of the tiles·U pieces.
struct FtShare {
    int32_t n, L, U, parts;
    int64_t units;
};

// Cost of cutting tiles into pieces of L steps: the steps of the busiest CTA, each
// `step_ns`, and `join_ns` for the exchange of a cut tile.
__host__ __device__ inline int64_t ft_share_cost(int64_t tiles, int32_t n, int32_t L, int32_t ctas, int32_t step_ns,
                                                 int32_t join_ns)
{
    const int64_t units = tiles * ((n + L - 1) / L);
    return (units + ctas - 1) / ctas * L * step_ns + (L < n ? join_ns : 0);
}

__host__ __device__ inline FtShare ft_share_of(int64_t tiles, int32_t n, int32_t L, int32_t ctas)
{
    FtShare s;
    s.n = n;
    s.L = L;
    s.U = (n + L - 1) / L;
    s.units = tiles * s.U;
    s.parts = (int32_t)(s.units < ctas ? s.units : ctas);
    return s;
}
constexpr int kFtMostPieces = 32;   // pieces of a tile that are tried
constexpr int kFtMostCluster = 8;   // CTAs that may share a cluster

enum FtAct : int32_t { FT_ACT_NONE = 0, FT_ACT_RELU = 1, FT_ACT_GELU = 2, FT_ACT_SILU = 3 };

struct WqParams {
    int32_t T, N, t8;                  // t8: tokens padded to the fragment's 8
    int32_t nkb, ncg;                  // 256-K blocks, 32-column groups
    int32_t gpc, has_zeros, chunk_bytes;
    int32_t act, gated;
    int32_t tiles;                     // 128 columns each
    FtShare share;
    int32_t cluster;                   // CTAs of a cluster, the pieces of one tile (1: no cluster)
    int32_t stages;
    uint32_t off_ring, stage_bytes, off_x, off_meta, off_red;
    const uint8_t *packed;
    const uint8_t *prepared;           // converted activations, a piece for each 256 K
    uint32_t prepared_bytes;           // of a piece: T rows of 512 bytes, and the meta data
    const void *x;
    int32_t K;
    const void *bias, *residual;
    void *y;
    float *workspace;                  // partial tiles, two for each CTA
    int32_t *counters;                 // arrivals, one for each tile; zero between launches
    int32_t *status;
    int64_t timeout_ns;
    int32_t debug_stall;
    int32_t early_weights;             // weights are not written by the work before this launch
};

struct WqPackParams {
    const uint8_t *codes;
    const void *scales;
    const uint8_t *zeros;
    uint8_t *packed;
    int64_t mats;
    int32_t K, N, group, gated, nkb, ncg, gpc, chunk_bytes;
};

struct MoeParams {
    int32_t T, H, I, E, top_k, t8;
    int32_t act, normalize, routed;
    int32_t nkb_up, nkb_down;          // K steps of a tile
    int32_t x_spans, h_spans;          // bf16: maps view x and h in 64-K spans, one copy a step
    int32_t up_spans, down_spans;      // bf16: maps view the weight in 64-column spans
    int32_t tiles_up, tiles_down;      // 64 gated features / 128 columns each
    int32_t gpc, has_zeros, chunk_bytes;
    int32_t ncg_up, ncg_down;          // 4-bit: 32-column groups of a weight
    int32_t route_slices, route_rows;  // the router product's split of H
    int32_t route_reduce;              // the last slice of a token group chooses for all CTAs
    int32_t max_tiles_up;
    int32_t stages;
    uint32_t off_route, off_ring, stage_bytes, off_x, off_meta, off_powers, off_red, off_acc;
    const void *x, *router;
    const uint8_t *gate_up, *down;     // 4-bit: packed experts
    const int32_t *ids_in;             // routed by the caller
    const float *weights_in;
    int32_t *ids_out;                  // optional
    float *weights_out;
    const void *residual;
    void *y;
    // Workspace
    float *logits;                     // [slices][T][E] partial router products
    int32_t *ids;                      // [T][top_k]
    float *weights;
    // Activations between the products, T·top_k rows (+ padding: h_rows) by expert.  bf16
    // experts: [I] bf16, high parts, then (h_rows rows on) low parts.  4-bit experts: fp16,
    // [256 K][row][256], with powers of two for each 64 of a row, [256 K][row][4].
    void *h;
    float *h_powers;
    int32_t h_rows;
    float *partials;                   // two tiles for each CTA
    int32_t *ctl;                      // [0] status, [2..3] arrivals (64-bit), [8..15] router groups,
                                       // [16..] tile counters of the up and the down phase
    int64_t timeout_ns;
    int32_t debug_stall;
};
constexpr int kMoeCtlHead = 16;
constexpr int kMoeMaxExperts = 256;
constexpr int kMoeMaxTopK = 16;
constexpr int kMoeMaxSlices = 32;            // of H, in the router product
constexpr int kRouteWeightBytes = 32 * 1024; // of the router weight, staged at once,
constexpr int kRouteRows = 512;              // and at most so many of its rows
constexpr int kMoeMaxPairs = kFtMaxTokens * kMoeMaxTopK;
constexpr int kMoeMaxRuns = kMoeMaxExperts + kMoeMaxPairs / 32;   // of a down tile

struct WqPrepareParams {
    const void *x;
    uint8_t *out;
    int32_t T, K, t8, nkb, gpc;
    uint32_t piece_bytes;
};

struct WqQuantParams {
    const void *w;
    uint8_t *codes;
    void *scales;
    uint8_t *zeros;                    // null: symmetric
    int32_t K, N, group;
};

// Launches (wq.cu, moe.cu); nt: 8-token tiles, 1, 2, 4 or 8.
cudaError_t wq_set_smem_limit(int bytes);
cudaError_t launch_wq(int nt, const CUtensorMap &x, const WqParams &p, int grid, int smem, cudaStream_t stream);
cudaError_t launch_wq_prepare(const WqPrepareParams &p, cudaStream_t stream);
cudaError_t launch_wq_pack(const WqPackParams &p, cudaStream_t stream);
cudaError_t launch_wq_quantize(const WqQuantParams &p, cudaStream_t stream);
struct MoeMaps {
    CUtensorMap x, gate_up, down, h[4];
};
// K of one bf16 step (1 token, 2 of 8 experts of 4096x14336: 120.5 us, 122.6 with 64);
// above 16 tokens a step of 128, with both parts of h, would leave the ring two slots.
__host__ __device__ constexpr int moe_step_k(int nt) { return nt <= 2 ? 128 : 64; }
// Tokens of an expert that one run of the down phase takes.  bf16 experts read two parts
// of each row of h: with more than 32 tokens at once a stage would hold 16 KB of h beside
// 16 KB of weights and the ring three slots instead of four (64 tokens, 4 of 32 experts of
// 4096x2048: 336 us, 303 so); an expert with more has its down weights read twice instead.
constexpr int kMoeDownTokens = 32;
__host__ __device__ constexpr int moe_down_tokens(int kernel) { return kernel == FT_MOE_BF16 ? kMoeDownTokens : kFtMaxTokens; }
// Rows of a stage's tokens, in rows of step_k bf16.
__host__ __device__ constexpr int moe_stage_rows(int kernel, int t8)
{
    return kernel != FT_MOE_BF16 || t8 > kMoeDownTokens ? t8 : 2 * t8;
}
static_assert(moe_stage_rows(FT_MOE_BF16, kFtMaxTokens) >= 2 * kMoeDownTokens, "both parts of h");
cudaError_t moe_set_smem_limit(int bytes);
cudaError_t launch_moe(int nt, int wq, const MoeMaps &m, const MoeParams &p, int grid, int smem, cudaStream_t stream);

}  // namespace gemmgb
