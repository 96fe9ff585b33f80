// Host side of the few-token operators: argument checks, plans (workspace,
// shared-memory layout, how the grid divides the work) and launches.
#include <string.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <new>

#include "few_token.h"
#include "gemm_internal.h"

namespace gemmgb {

extern std::atomic<int64_t> g_timeout_ns;    // runtime.cpp
extern std::atomic<int32_t> g_debug_stall;   // runtime.cpp
extern std::atomic<int32_t> g_check;         // runtime.cpp
std::atomic<int32_t> g_wq_split{0};          // wq plans' grid: 0 by rule, 1 equal pieces without clusters, 2 whole tiles

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
uint32_t round_up(uint32_t v, uint32_t to) { return (v + to - 1) / to * to; }
int tiles_of_tokens(int64_t T) { return T <= 8 ? 1 : T <= 16 ? 2 : T <= 32 ? 4 : 8; }
bool valid_group(int group) { return group == 0 || group == 32 || group == 64 || group == 128 || group == 256; }
// The group as the kernels take it: one scale for a whole column reads like
// one for each chunk of 256.
int chunk_group(int group) { return group == 0 ? kWqChunkK : group; }

int act_of(int epi)
{
    switch (epi) {
    case GEMM_EPI_BIAS_RELU:
    case GEMM_EPI_BIAS_RELU_RESIDUAL:
    case GEMM_EPI_BIAS_REGLU: return FT_ACT_RELU;
    case GEMM_EPI_BIAS_GELU:
    case GEMM_EPI_BIAS_GELU_RESIDUAL:
    case GEMM_EPI_BIAS_GEGLU: return FT_ACT_GELU;
    case GEMM_EPI_BIAS_SWIGLU: return FT_ACT_SILU;
    default: return FT_ACT_NONE;
    }
}

int current_device(int plan_device)
{
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev != plan_device)
        return set_error(GEMM_ERR_INVALID_ARG, "plan was made on device %d, current device is %d", plan_device, dev);
    return GEMM_OK;
}

// Zeroes device memory before it returns: the work that reads it may come on a stream
// that does not wait for the default one, where the fill itself may have to queue.
cudaError_t clear_memory(void *p, size_t bytes)
{
    cudaError_t e = cudaMemset(p, 0, bytes);
    return e == cudaSuccess ? cudaStreamSynchronize(cudaStreamLegacy) : e;
}

// Status word of a few-token plan, after its work has finished; a part-way
// return leaves counts behind, so the whole control block starts afresh.
int read_word(int32_t *ctl, size_t bytes)
{
    int32_t st = 0;
    cudaError_t e = cudaMemcpy(&st, ctl, sizeof(st), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_err(e, "reading the status word");
    if (st == 0) return GEMM_OK;
    e = clear_memory(ctl, bytes);
    if (e != cudaSuccess) return cuda_err(e, "resetting the control block");
    return set_error(GEMM_ERR_TIMEOUT, "a device wait expired (site %d); the kernel returned early", st);
}

int finish_run(int32_t *ctl, size_t bytes, cudaStream_t stream)
{
    if (!g_check.load()) return GEMM_OK;
    cudaError_t e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return cuda_err(e, "cudaStreamSynchronize (checked run)");
    return read_word(ctl, bytes);
}

// Costs that divide the work (FtShare): a step's share of the memory's time (17 KB at
// 45 GB/s an SM), above 16 tokens its multiplications; and the exchange of a cut tile.
// Whole tiles against the cut that they choose: 1 token 8192x28672 31.5 and 25.5 us, 16
// tokens 4096x28672 28.0 and 25.1.
int step_ns(int nt) { return nt <= 2 ? 380 : nt == 4 ? 600 : 1100; }
constexpr int kJoinNs = 2500;

// The two buffers of the hand-over: K parts of sums, [token][row] each.  A call's
// widest buffer is the one for the most tokens, or (4-bit, above 32) as wide.
uint32_t red_bytes(int kernel, int nt) { return (uint32_t)(2 * ft_k_parts(kernel, nt, nt) * nt * 8 * (kFtTileRows + 4) * 4); }

// Powers of two and sums of a 4-bit stage's tokens (few_token.cuh).
uint32_t meta_bytes(int t8) { return 9u * (uint32_t)t8 * 4u; }

// Token rows [T, K] as a bf16 step copies them: `rows` of them and 64 K to a box, or
// `spans` times 64 where K is a whole number of spans.
int encode_tokens(CUtensorMap *m, const void *ptr, int64_t K, int64_t T, int rows, int spans)
{
    if (K % 64 == 0) return encode_spans(m, GEMM_BF16, ptr, (uint64_t)K, (uint64_t)T, 64, (uint32_t)rows, (uint32_t)spans);
    return encode_2d(m, GEMM_BF16, ptr, (uint64_t)K, (uint64_t)T, 64, (uint32_t)rows, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// Token rows [T, K] as a 4-bit step copies them: whole rows of 256 K, unswizzled.
int encode_rows(CUtensorMap *m, const void *ptr, int64_t K, int64_t T, int rows)
{
    return encode_2d(m, GEMM_BF16, ptr, (uint64_t)K, (uint64_t)T, kWqChunkK, (uint32_t)rows, CU_TENSOR_MAP_SWIZZLE_NONE,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

int check_weight(const char *who, int64_t mats, int64_t K, int64_t N, int group, int gated)
{
    const int64_t lim = (int64_t)1 << 24;
    if (mats < 0 || K < 1 || N < 0 || K >= lim || N >= lim)
        return set_error(GEMM_ERR_INVALID_ARG, "%s: extents must be K in [1, 2^24), N in [0, 2^24): K=%lld N=%lld", who,
                         (long long)K, (long long)N);
    if (!valid_group(group))
        return set_error(GEMM_ERR_INVALID_ARG, "%s: group must be 32, 64, 128, 256 or 0 (whole column), not %d", who, group);
    if (gated && N % 64)
        return set_error(GEMM_ERR_INVALID_ARG, "%s: a gated weight's N must be a multiple of 64, not %lld", who,
                         (long long)N);
    return GEMM_OK;
}

}  // namespace
}  // namespace gemmgb

using namespace gemmgb;

// ---------------------------------------------------------------------------
// 4-bit weights
// ---------------------------------------------------------------------------

struct gemm_wq_plan_s {
    int64_t K = 0, N = 0;
    int group = 0, zeros = 0, epi = 0, max_tokens = 0, device = 0, early = 0;
    int split = 0;                   // debug choice at the time of planning
    int sm_count = 0;
    int64_t smem_limit = 0;
    int32_t *ctl = nullptr;          // [0] status word, then one counter for each tile
    size_t ctl_bytes = 0;
    float *workspace = nullptr;
    uint8_t *prepared = nullptr;     // converted activations of a call
};

extern "C" int64_t gemm_wq_packed_bytes(int64_t mats, int64_t K, int64_t N, int32_t group, int32_t has_zeros)
{
    clear_error();
    if (check_weight("gemm_wq_packed_bytes", mats, K, N, group, 0)) return 0;
    return mats * cdiv(N, kWqChunkCols) * cdiv(K, kWqChunkK) * wq_chunk_bytes(chunk_group(group), has_zeros ? 1 : 0);
}

extern "C" int gemm_wq_pack(const void *codes, const void *scales, const void *zeros, int64_t mats, int64_t K,
                            int64_t N, int32_t group, int32_t gated, void *packed, gemm_stream_t stream)
{
    clear_error();
    int rc = check_weight("gemm_wq_pack", mats, K, N, group, gated);
    if (rc) return rc;
    if (mats == 0 || N == 0) return GEMM_OK;
    if (!codes || !scales || !packed) return set_error(GEMM_ERR_INVALID_ARG, "gemm_wq_pack: null codes, scales or packed");
    if (!aligned16(packed)) return set_error(GEMM_ERR_MISALIGNED, "gemm_wq_pack: packed must be 16-byte aligned");
    if ((uintptr_t)scales & 1u) return set_error(GEMM_ERR_MISALIGNED, "gemm_wq_pack: scales must be 2-byte aligned");
    rc = check_device_arch(nullptr);
    if (rc) return rc;
    WqPackParams p;
    memset(&p, 0, sizeof(p));
    p.codes = static_cast<const uint8_t *>(codes);
    p.scales = scales;
    p.zeros = static_cast<const uint8_t *>(zeros);
    p.packed = static_cast<uint8_t *>(packed);
    p.mats = mats;
    p.K = (int32_t)K;
    p.N = (int32_t)N;
    p.group = group;
    p.gated = gated ? 1 : 0;
    p.nkb = (int32_t)cdiv(K, kWqChunkK);
    p.ncg = (int32_t)cdiv(N, kWqChunkCols);
    p.gpc = wq_groups_per_chunk(chunk_group(group));
    p.chunk_bytes = wq_chunk_bytes(chunk_group(group), zeros ? 1 : 0);
    cudaError_t e = launch_wq_pack(p, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_err(e, "4-bit packing launch");
    return GEMM_OK;
}

extern "C" int gemm_wq_quantize(const void *W, int64_t K, int64_t N, int32_t group, void *codes, void *scales,
                                void *zeros, gemm_stream_t stream)
{
    clear_error();
    int rc = check_weight("gemm_wq_quantize", 1, K, N, group, 0);
    if (rc) return rc;
    if (N == 0) return GEMM_OK;
    if (!W || !codes || !scales) return set_error(GEMM_ERR_INVALID_ARG, "gemm_wq_quantize: null W, codes or scales");
    if (((uintptr_t)W & 1u) || ((uintptr_t)scales & 1u))
        return set_error(GEMM_ERR_MISALIGNED, "gemm_wq_quantize: W and scales must be 2-byte aligned");
    rc = check_device_arch(nullptr);
    if (rc) return rc;
    WqQuantParams p;
    memset(&p, 0, sizeof(p));
    p.w = W;
    p.codes = static_cast<uint8_t *>(codes);
    p.scales = scales;
    p.zeros = static_cast<uint8_t *>(zeros);
    p.K = (int32_t)K;
    p.N = (int32_t)N;
    p.group = group;
    cudaError_t e = launch_wq_quantize(p, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_err(e, "4-bit quantisation launch");
    return GEMM_OK;
}

extern "C" void gemm_wq_plan_destroy(gemm_wq_plan_t p)
{
    if (!p) return;
    cudaFree(p->ctl);
    cudaFree(p->workspace);
    cudaFree(p->prepared);
    delete p;
}

extern "C" int gemm_wq_plan(int64_t K, int64_t N, int32_t group, int32_t has_zeros, gemm_epilogue epi,
                            int32_t max_tokens, gemm_wq_plan_t *out)
{
    clear_error();
    if (!out) return set_error(GEMM_ERR_INVALID_ARG, "gemm_wq_plan: null out");
    *out = nullptr;
    if (epi < GEMM_EPI_NONE || epi > GEMM_EPI_BIAS_SWIGLU)
        return set_error(GEMM_ERR_INVALID_ARG, "unknown epilogue %d", (int)epi);
    int rc = check_weight("gemm_wq_plan", 1, K, N, group, is_glu(epi));
    if (rc) return rc;
    if (max_tokens < 1 || max_tokens > kFtMaxTokens)
        return set_error(GEMM_ERR_INVALID_ARG, "gemm_wq_plan: max_tokens must be 1..%d, not %d", kFtMaxTokens, max_tokens);
    if (K % 8) return set_error(GEMM_ERR_MISALIGNED, "gemm_wq_plan: K=%lld: x's rows must be multiples of 16 bytes", (long long)K);
    int dev = 0;
    rc = check_device_arch(&dev);
    if (rc) return rc;
    gemm_device_params d;
    rc = query_params(&d);
    if (rc) return rc;
    cudaError_t e = wq_set_smem_limit((int)d.smem_per_block);
    if (e != cudaSuccess) return cuda_err(e, "cudaFuncSetAttribute(wq kernel)");
    gemm_wq_plan_s *p = new (std::nothrow) gemm_wq_plan_s();
    if (!p) return set_error(GEMM_ERR_CUDA, "out of host memory");
    p->K = K;
    p->N = N;
    p->group = group;
    p->zeros = has_zeros ? 1 : 0;
    p->epi = epi;
    p->max_tokens = max_tokens;
    p->device = dev;
    p->split = g_wq_split.load();
    p->sm_count = d.sm_count;
    p->smem_limit = d.smem_per_block;
    p->ctl_bytes = (size_t)(1 + cdiv(N, kWqChunkCols)) * sizeof(int32_t);
    const size_t ws = (size_t)d.sm_count * 2 * (size_t)tiles_of_tokens(max_tokens) * 8 * kFtTileRows * sizeof(float);
    e = cudaMalloc(&p->ctl, p->ctl_bytes);
    if (e == cudaSuccess) e = clear_memory(p->ctl, p->ctl_bytes);
    if (e == cudaSuccess) e = cudaMalloc(&p->workspace, ws);
    if (e == cudaSuccess && wq_prepares(tiles_of_tokens(max_tokens)))
        e = cudaMalloc(&p->prepared, (size_t)cdiv(K, kWqChunkK) *
                                         ((size_t)max_tokens * 512 + meta_bytes(tiles_of_tokens(max_tokens) * 8)));
    if (e != cudaSuccess) {
        gemm_wq_plan_destroy(p);
        return cuda_err(e, "cudaMalloc(wq plan)");
    }
    *out = p;
    return GEMM_OK;
}

extern "C" int gemm_wq_plan_set_independent_weights(gemm_wq_plan_t p, int32_t independent)
{
    clear_error();
    if (!p) return set_error(GEMM_ERR_INVALID_ARG, "null plan");
    if (independent != 0 && independent != 1) return set_error(GEMM_ERR_INVALID_ARG, "independent must be 0 or 1");
    p->early = independent;
    return GEMM_OK;
}

extern "C" int gemm_wq_plan_status(gemm_wq_plan_t p)
{
    clear_error();
    if (!p) return set_error(GEMM_ERR_INVALID_ARG, "null plan");
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_err(e, "cudaDeviceSynchronize");
    return read_word(p->ctl, p->ctl_bytes);
}

extern "C" int gemm_wq_run(gemm_wq_plan_t p, int64_t tokens, const void *x, const void *packed, const void *bias,
                           const void *R, void *y, gemm_stream_t stream_)
{
    clear_error();
    if (!p) return set_error(GEMM_ERR_INVALID_ARG, "null plan");
    if (tokens < 0 || tokens > p->max_tokens)
        return set_error(GEMM_ERR_INVALID_ARG, "tokens must be 0..%d (the plan's max_tokens), not %lld", p->max_tokens,
                         (long long)tokens);
    if (is_residual(p->epi) && !R) return set_error(GEMM_ERR_INVALID_ARG, "the residual epilogue needs R");
    if (!is_residual(p->epi) && R)
        return set_error(GEMM_ERR_INVALID_ARG, "R given to a plan whose epilogue has no residual");
    if (tokens == 0 || p->N == 0) return GEMM_OK;
    if (!x || !packed || !y) return set_error(GEMM_ERR_INVALID_ARG, "null x, packed weight or y");
    if (p->epi != GEMM_EPI_NONE && !bias) return set_error(GEMM_ERR_INVALID_ARG, "bias is required by the epilogue");
    if (!aligned16(x) || !aligned16(packed) || !aligned16(y) || (p->epi != GEMM_EPI_NONE && !aligned16(bias)) ||
        (R && !aligned16(R)))
        return set_error(GEMM_ERR_MISALIGNED, "x, the packed weight, bias, R and y must be 16-byte aligned");
    int rc = current_device(p->device);
    if (rc) return rc;

    const int nt = tiles_of_tokens(tokens);
    WqParams k;
    memset(&k, 0, sizeof(k));
    k.T = (int32_t)tokens;
    k.N = (int32_t)p->N;
    k.t8 = nt * 8;
    k.nkb = (int32_t)cdiv(p->K, kWqChunkK);
    k.ncg = (int32_t)cdiv(p->N, kWqChunkCols);
    k.gpc = wq_groups_per_chunk(chunk_group(p->group));
    k.has_zeros = p->zeros;
    k.chunk_bytes = wq_chunk_bytes(chunk_group(p->group), p->zeros);
    k.act = act_of(p->epi);
    k.gated = is_glu(p->epi) ? 1 : 0;
    k.tiles = (int32_t)cdiv(k.ncg, 4);
    // Few tiles: one cluster of CTAs to a tile (64 tokens 14336x4096: 41 us, 78 with the
    // pieces through global memory, 149 uncut; 5 tokens 1000x1001: 5.3, 6.9 and 6.9; 1
    // token 4096x4096: 7.2, 7.4 and 9.7).  Else pieces as short as keeps the
    // busiest CTA's steps few, but not cut where that gains less than the exchange.
    int L = k.nkb;
    const int most = (int)std::min<int64_t>({kFtMostCluster, p->sm_count / k.tiles, k.nkb});
    k.cluster = 1;
    if (p->split == 0 && most > 1) {
        L = (k.nkb + most - 1) / most;
        k.cluster = (k.nkb + L - 1) / L;
    } else if (p->split != 2) {
        int64_t best = -1;
        for (int i = 0; i < kFtMostPieces && i < k.nkb; ++i) {
            const int len = (k.nkb + i) / (i + 1);
            const int64_t cost = ft_share_cost(k.tiles, k.nkb, len, p->sm_count, step_ns(nt), p->split == 1 ? 0 : kJoinNs);
            if (best < 0 || cost < best) best = cost, L = len;
        }
    }
    k.share = ft_share_of(k.tiles, k.nkb, L, p->sm_count);
    const int grid = k.share.parts;

    k.off_ring = kFtCtl;
    k.off_x = round_up(4u * (uint32_t)k.chunk_bytes, 1024);
    k.off_meta = k.off_x + (uint32_t)tokens * 512u;
    k.stage_bytes = round_up(k.off_meta + meta_bytes(k.t8), 1024);
    const uint32_t red = red_bytes(FT_PRODUCT, nt);
    const int64_t room = p->smem_limit - 1024 - kFtCtl - red;
    k.stages = (int32_t)std::min<int64_t>(kFtMaxStages, room / k.stage_bytes);
    k.stages -= k.stages % ft_k_parts(FT_PRODUCT, nt, nt);   // StepWalk
    if (k.stages < 2) return set_error(GEMM_ERR_UNSUPPORTED, "the device's shared memory holds too few stages");
    k.off_red = k.off_ring + (uint32_t)k.stages * k.stage_bytes;
    const int smem = (int)(k.off_red + red + 1024);

    k.packed = static_cast<const uint8_t *>(packed);
    k.x = x;
    k.K = (int32_t)p->K;
    k.bias = p->epi != GEMM_EPI_NONE ? bias : nullptr;
    k.residual = R;
    k.y = y;
    k.workspace = p->workspace;
    k.status = p->ctl;
    k.counters = p->ctl + 1;
    k.timeout_ns = g_timeout_ns.load();
    k.debug_stall = g_debug_stall.load();
    k.early_weights = p->early;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    cudaError_t e = cudaSuccess;
    CUtensorMap mx;
    if (wq_prepares(nt)) {
        memset(&mx, 0, sizeof(mx));
        WqPrepareParams q;
        q.x = x;
        q.out = p->prepared;
        q.T = k.T;
        q.K = (int32_t)p->K;
        q.t8 = k.t8;
        q.nkb = k.nkb;
        q.gpc = k.gpc;
        q.piece_bytes = (uint32_t)tokens * 512u + meta_bytes(k.t8);
        k.prepared = p->prepared;
        k.prepared_bytes = q.piece_bytes;
        e = launch_wq_prepare(q, stream);
        if (e != cudaSuccess) return cuda_err(e, "wq activation launch");
    } else {
        rc = encode_rows(&mx, x, p->K, tokens, (int)tokens);
        if (rc) return rc;
    }
    e = launch_wq(nt, mx, k, grid, smem, stream);
    if (e != cudaSuccess) return cuda_err(e, "wq kernel launch");
    return finish_run(p->ctl, p->ctl_bytes, stream);
}

// ---------------------------------------------------------------------------
// Mixture of experts
// ---------------------------------------------------------------------------

struct gemm_moe_plan_s {
    gemm_moe_desc d{};
    int device = 0, sm_count = 0;
    int64_t smem_limit = 0;
    int32_t *ctl = nullptr;
    size_t ctl_bytes = 0;
    int64_t max_tiles_up = 0;
    int64_t h_rows = 0;
    char *ws = nullptr;
    float *logits = nullptr, *weights = nullptr, *partials = nullptr;
    int32_t *ids = nullptr;
    void *h = nullptr;
    float *h_powers = nullptr;
};

extern "C" void gemm_moe_plan_destroy(gemm_moe_plan_t p)
{
    if (!p) return;
    cudaFree(p->ctl);
    cudaFree(p->ws);
    delete p;
}

extern "C" int gemm_moe_plan(const gemm_moe_desc *desc, gemm_moe_plan_t *out)
{
    clear_error();
    if (!desc || !out) return set_error(GEMM_ERR_INVALID_ARG, "gemm_moe_plan: null descriptor or out");
    *out = nullptr;
    const gemm_moe_desc &d = *desc;
    const int64_t lim = (int64_t)1 << 20;
    if (d.hidden < 1 || d.hidden >= lim || d.inter < 1 || d.inter >= lim)
        return set_error(GEMM_ERR_INVALID_ARG, "gemm_moe_plan: hidden and inter must be in [1, 2^20)");
    if (d.experts < 1 || d.experts > kMoeMaxExperts)
        return set_error(GEMM_ERR_INVALID_ARG, "gemm_moe_plan: experts must be 1..%d, not %d", kMoeMaxExperts, d.experts);
    if (d.top_k < 1 || d.top_k > std::min(d.experts, kMoeMaxTopK))
        return set_error(GEMM_ERR_INVALID_ARG, "gemm_moe_plan: top_k must be 1..min(experts, %d), not %d", kMoeMaxTopK,
                         d.top_k);
    if (d.max_tokens < 1 || d.max_tokens > kFtMaxTokens)
        return set_error(GEMM_ERR_INVALID_ARG, "gemm_moe_plan: max_tokens must be 1..%d, not %d", kFtMaxTokens, d.max_tokens);
    if (d.weights != GEMM_MOE_BF16 && d.weights != GEMM_MOE_WQ)
        return set_error(GEMM_ERR_INVALID_ARG, "gemm_moe_plan: unknown weight format %d", (int)d.weights);
    if (d.act != GEMM_EPI_BIAS_REGLU && d.act != GEMM_EPI_BIAS_GEGLU && d.act != GEMM_EPI_BIAS_SWIGLU)
        return set_error(GEMM_ERR_INVALID_ARG, "gemm_moe_plan: act must be one of the gated epilogues, not %d", (int)d.act);
    if (d.weights == GEMM_MOE_WQ && !valid_group(d.group))
        return set_error(GEMM_ERR_INVALID_ARG, "gemm_moe_plan: group must be 32, 64, 128, 256 or 0, not %d", d.group);
    if (d.hidden % 8 || d.inter % 32)
        return set_error(GEMM_ERR_MISALIGNED, "gemm_moe_plan: hidden must be a multiple of 8 and inter of 32");
    int dev = 0;
    int rc = check_device_arch(&dev);
    if (rc) return rc;
    gemm_device_params q;
    rc = query_params(&q);
    if (rc) return rc;
    cudaError_t e = moe_set_smem_limit((int)q.smem_per_block);
    if (e != cudaSuccess) return cuda_err(e, "cudaFuncSetAttribute(moe kernel)");
    gemm_moe_plan_s *p = new (std::nothrow) gemm_moe_plan_s();
    if (!p) return set_error(GEMM_ERR_CUDA, "out of host memory");
    p->d = d;
    p->device = dev;
    p->sm_count = q.sm_count;
    p->smem_limit = q.smem_per_block;
    const int64_t pairs = (int64_t)d.max_tokens * d.top_k;
    const bool wq = d.weights == GEMM_MOE_WQ;
    p->max_tiles_up = std::min<int64_t>(d.experts, pairs) * cdiv(d.inter, 64);
    p->ctl_bytes = (size_t)(kMoeCtlHead + p->max_tiles_up + cdiv(d.hidden, kFtTileRows)) * sizeof(int32_t);
    p->h_rows = pairs + 64;   // a box of rows may reach past the last one
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    const size_t n_logits = up((size_t)kMoeMaxSlices * d.max_tokens * d.experts * 4),
                 n_ids = up((size_t)pairs * 4),
                 n_h = up(wq ? (size_t)cdiv(d.inter, kWqChunkK) * p->h_rows * kWqChunkK * 2 : (size_t)p->h_rows * d.inter * 4),
                 n_powers = wq ? up((size_t)cdiv(d.inter, kWqChunkK) * p->h_rows * 16) : 0,
                 n_part = up((size_t)q.sm_count * 2 * tiles_of_tokens(d.max_tokens) * 8 * kFtTileRows * 4);
    e = cudaMalloc(&p->ctl, p->ctl_bytes);
    if (e == cudaSuccess) e = clear_memory(p->ctl, p->ctl_bytes);
    if (e == cudaSuccess) e = cudaMalloc(&p->ws, n_logits + 2 * n_ids + n_h + n_powers + n_part);
    // h past the last feature stays what it is here: zeros.
    if (e == cudaSuccess && wq) e = clear_memory(p->ws + n_logits + 2 * n_ids, n_h + n_powers);
    if (e != cudaSuccess) {
        gemm_moe_plan_destroy(p);
        return cuda_err(e, "cudaMalloc(moe plan)");
    }
    char *at = p->ws;
    p->logits = reinterpret_cast<float *>(at), at += n_logits;
    p->ids = reinterpret_cast<int32_t *>(at), at += n_ids;
    p->weights = reinterpret_cast<float *>(at), at += n_ids;
    p->h = at, at += n_h;
    p->h_powers = reinterpret_cast<float *>(at), at += n_powers;
    p->partials = reinterpret_cast<float *>(at);
    *out = p;
    return GEMM_OK;
}

extern "C" int gemm_moe_plan_status(gemm_moe_plan_t p)
{
    clear_error();
    if (!p) return set_error(GEMM_ERR_INVALID_ARG, "null plan");
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_err(e, "cudaDeviceSynchronize");
    return read_word(p->ctl, p->ctl_bytes);
}

// Both entry points: routed by the layer (router) or by the caller (ids, w).
static int moe_run(gemm_moe_plan_t p, int64_t tokens, const void *x, const void *router, const int32_t *ids_in,
                   const float *w_in, const void *gate_up, const void *down, const void *R, void *y, int32_t *ids_out,
                   float *w_out, cudaStream_t stream)
{
    clear_error();
    if (!p) return set_error(GEMM_ERR_INVALID_ARG, "null plan");
    const gemm_moe_desc &d = p->d;
    if (tokens < 0 || tokens > d.max_tokens)
        return set_error(GEMM_ERR_INVALID_ARG, "tokens must be 0..%d (the plan's max_tokens), not %lld", d.max_tokens,
                         (long long)tokens);
    if (tokens == 0) return GEMM_OK;
    const bool routed = router == nullptr;
    if (!x || !gate_up || !down || !y || (routed && (!ids_in || !w_in)))
        return set_error(GEMM_ERR_INVALID_ARG, routed ? "null x, ids, weights, gate_up, down or y"
                                                      : "null x, router, gate_up, down or y");
    if (!aligned16(x) || !aligned16(router) || !aligned16(gate_up) || !aligned16(down) || !aligned16(y) || !aligned16(R))
        return set_error(GEMM_ERR_MISALIGNED, "x, router, gate_up, down, R and y must be 16-byte aligned");
    if (((uintptr_t)ids_in & 3u) || ((uintptr_t)w_in & 3u) || ((uintptr_t)ids_out & 3u) || ((uintptr_t)w_out & 3u))
        return set_error(GEMM_ERR_MISALIGNED, "ids and weights must be 4-byte aligned");
    int rc = current_device(p->device);
    if (rc) return rc;

    const int nt = tiles_of_tokens(tokens);
    const bool wq = d.weights == GEMM_MOE_WQ;
    const int step_k = wq ? kWqChunkK : moe_step_k(nt);
    MoeParams k;
    memset(&k, 0, sizeof(k));
    k.T = (int32_t)tokens;
    k.H = (int32_t)d.hidden;
    k.I = (int32_t)d.inter;
    k.E = d.experts;
    k.top_k = d.top_k;
    k.t8 = nt * 8;
    k.act = act_of(d.act);
    k.normalize = d.normalize ? 1 : 0;
    k.routed = routed ? 1 : 0;
    k.nkb_up = (int32_t)cdiv(d.hidden, step_k);
    k.nkb_down = (int32_t)cdiv(d.inter, step_k);
    k.tiles_up = (int32_t)cdiv(d.inter, 64);
    k.tiles_down = (int32_t)cdiv(d.hidden, kFtTileRows);
    if (wq) {
        k.gpc = wq_groups_per_chunk(chunk_group(d.group));
        k.has_zeros = d.has_zeros ? 1 : 0;
        k.chunk_bytes = wq_chunk_bytes(chunk_group(d.group), k.has_zeros);
        k.ncg_up = (int32_t)(2 * d.inter / kWqChunkCols);
        k.ncg_down = (int32_t)cdiv(d.hidden, kWqChunkCols);
    }
    // The router product: 8 tokens and 1/slices of H to a CTA, at least 32 of H.
    const int groups = (int)cdiv(tokens, 8);
    const int slices = (int)std::max<int64_t>(
        1, std::min<int64_t>({kMoeMaxSlices, p->sm_count / groups, cdiv(d.hidden, 32)}));
    k.route_rows = (int32_t)cdiv(cdiv(d.hidden, slices), 8) * 8;
    k.route_slices = (int32_t)cdiv(d.hidden, k.route_rows);
    // Few tokens: every CTA adds the slices and chooses for itself (7 tokens, 13 experts:
    // 23.7 us, 24.9 where the last CTA chooses for all).
    k.route_reduce = tokens > 8;
    k.max_tiles_up = (int32_t)p->max_tiles_up;

    // Tables of the routing need about 13 KB.
    constexpr uint32_t kTables = 16 * 1024;
    static_assert(kMoeMaxExperts * 20 + kMoeMaxPairs * 5 + kMoeMaxRuns * 8 + 64 <= (int)kTables, "routing tables");
    const uint32_t red = red_bytes(wq ? FT_MOE_W4 : FT_MOE_BF16, nt), acc = (uint32_t)k.t8 * (kFtTileRows + 4) * 4u;
    k.off_route = kFtCtl;
    k.off_ring = kFtCtl + kTables;
    k.off_x = wq ? round_up(4u * (uint32_t)k.chunk_bytes, 1024) : (uint32_t)step_k * 256u;
    k.off_meta = k.off_x + (uint32_t)(moe_stage_rows(wq ? FT_MOE_W4 : FT_MOE_BF16, k.t8) * step_k * 2);
    k.off_powers = k.off_meta + meta_bytes(k.t8);
    k.stage_bytes = wq ? round_up(k.off_powers + (uint32_t)k.t8 * 16u, 1024) : k.off_meta;
    static_assert(8 * (2 * kMoeMaxExperts + 2 * kMoeMaxTopK) * 4 <= kRouteWeightBytes, "a token group's choice");
    const int64_t room = p->smem_limit - 1024 - k.off_ring - red - acc;
    k.stages = (int32_t)std::min<int64_t>(kFtMaxStages, room / k.stage_bytes);
    if (wq && nt <= 2) k.stages -= k.stages % ft_k_parts(FT_MOE_W4, nt, nt);   // StepWalk
    k.off_red = k.off_ring + (uint32_t)k.stages * k.stage_bytes;
    k.off_acc = k.off_red + red;
    // What routing keeps where the ring will be: the router product's scratch, later
    // ids, weights and (few tokens) logits, their keys and a word a worker.
    const uint32_t workers = (uint32_t)ft_workers(wq ? FT_MOE_W4 : FT_MOE_BF16, nt);
    const uint32_t scratch = workers * 32u + (uint32_t)kRouteRows * 32u + kRouteWeightBytes;
    const uint32_t chosen = (uint32_t)tokens * (uint32_t)d.top_k * 8u +
                            (k.route_reduce ? 0u : (uint32_t)tokens * (uint32_t)d.experts * 8u + workers * 4u);
    if (k.stages < 2 || std::max(scratch, chosen) > (uint32_t)k.stages * k.stage_bytes)
        return set_error(GEMM_ERR_UNSUPPORTED, "the device's shared memory holds too few stages");
    const int smem = (int)(k.off_acc + acc + 1024);

    k.x = x;
    k.router = router;
    k.gate_up = static_cast<const uint8_t *>(gate_up);
    k.down = static_cast<const uint8_t *>(down);
    k.ids_in = ids_in;
    k.weights_in = w_in;
    k.ids_out = ids_out;
    k.weights_out = w_out;
    k.residual = R;
    k.y = y;
    k.logits = p->logits;
    k.ids = p->ids;
    k.weights = p->weights;
    k.h = p->h;
    k.h_powers = p->h_powers;
    k.h_rows = (int32_t)p->h_rows;
    k.partials = p->partials;
    k.ctl = p->ctl;
    k.timeout_ns = g_timeout_ns.load();
    k.debug_stall = g_debug_stall.load();

    MoeMaps m;
    memset(&m, 0, sizeof(m));
    k.x_spans = d.hidden % 64 == 0;
    k.h_spans = d.inter % 64 == 0;
    k.up_spans = 1;                     // 2·inter is a multiple of 64
    k.down_spans = d.hidden % 64 == 0;
    rc = wq ? encode_rows(&m.x, x, d.hidden, tokens, (int)tokens) : encode_tokens(&m.x, x, d.hidden, tokens, k.t8, step_k / 64);
    for (int i = 0; i < 4 && !rc && !wq && (1 << i) <= nt; ++i)
        rc = encode_tokens(&m.h[i], p->h, d.inter, 2 * p->h_rows, 8 << i, step_k / 64);
    if (!rc && !wq) {
        rc = encode_stack(&m.gate_up, gate_up, (uint64_t)d.inter * 2, (uint64_t)d.hidden, (uint64_t)d.experts,
                          (uint32_t)step_k, 2);
        if (!rc)
            rc = encode_stack(&m.down, down, (uint64_t)d.hidden, (uint64_t)d.inter, (uint64_t)d.experts, (uint32_t)step_k,
                              k.down_spans ? 2 : 0);
    }
    if (rc) return rc;
    cudaError_t e = launch_moe(nt, wq ? 1 : 0, m, k, p->sm_count, smem, stream);
    if (e != cudaSuccess) return cuda_err(e, "moe kernel launch");
    return finish_run(p->ctl, p->ctl_bytes, stream);
}

extern "C" int gemm_moe_run(gemm_moe_plan_t plan, int64_t tokens, const void *x, const void *router, const void *gate_up,
                            const void *down, const void *R, void *y, int32_t *ids, float *weights,
                            gemm_stream_t stream)
{
    if (tokens > 0 && !router) {
        clear_error();
        return set_error(GEMM_ERR_INVALID_ARG, "null router (gemm_moe_run_routed takes ids and weights)");
    }
    return moe_run(plan, tokens, x, router, nullptr, nullptr, gate_up, down, R, y, ids, weights,
                   reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int gemm_moe_run_routed(gemm_moe_plan_t plan, int64_t tokens, const void *x, const int32_t *ids,
                                   const float *weights, const void *gate_up, const void *down, const void *R, void *y,
                                   gemm_stream_t stream)
{
    return moe_run(plan, tokens, x, nullptr, ids, weights, gate_up, down, R, y, nullptr, nullptr,
                   reinterpret_cast<cudaStream_t>(stream));
}
