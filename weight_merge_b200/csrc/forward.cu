// forward.cu -- C ABI of the per-token forward: routing to experts, the
// product of a weight with a fused epilogue, and the product with every
// token's own experts.  See include/adafuse.h for each contract.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "adafuse.h"
#include "common.cuh"
#include "context.cuh"
#include "linear_common.cuh"
#include "linear_host.cuh"
#include "route_experts.cuh"

using namespace adafuse;

namespace {

bool slots_ok(int32_t slots) { return slots == 2 || slots == 4 || slots == 8; }

// The weight (layer, target) of the context, or null.
const PairDesc* find_pair(const adafuse_ctx* ctx, int32_t layer, int32_t target) {
    if (layer < 0 || layer >= ctx->n_layers || target < 0 || target >= ctx->n_targets) return nullptr;
    return &ctx->h_pairs[(size_t)((int64_t)layer * ctx->n_targets + target)];
}

// A [T, n] operand of `size`-byte elements with rows ld apart: 16-byte aligned
// base, rows whole multiples of 16 bytes, at least n long, less than 2^40 bytes
// apart (the reach of a tensor map).
bool rows_ok(const void* p, int64_t ld, int64_t n, int64_t size) {
    return p != nullptr && aligned16(p) && ld >= n && ld < ((int64_t)1 << 40) / size && ld * size % 16 == 0;
}

// Tokens of one launch: tile coordinates stay far inside 32 bits, and a routed
// product's second launch, whose waits are bounded, never waits long for its
// first.
constexpr int64_t kTokensPerLaunch = (int64_t)1 << 17;

// The parameters of n tokens from the t0-th on.
LinearParams token_range(const LinearParams& p, int64_t t0, int64_t n) {
    LinearParams q = p;
    const int64_t size = p.f32 ? 4 : 2;
    q.T = n;
    q.x = p.x + t0 * p.ldx;
    if (p.mul != nullptr) q.mul = static_cast<const char*>(p.mul) + t0 * p.ldmul * size;
    if (p.res != nullptr) q.res = static_cast<const char*>(p.res) + t0 * p.ldres * size;
    q.y = static_cast<char*>(p.y) + t0 * p.ldy * size;
    if (p.routes != nullptr) q.routes = p.routes + t0 * 2 * p.slots;
    return q;
}

// Checks of a product's arguments, and its launch parameters.
int linear_params(const adafuse_ctx* ctx, const adafuse_linear_args* a, LinearParams* p) {
    std::memset(p, 0, sizeof *p);
    if (ctx == nullptr || a == nullptr) return ADAFUSE_ERR_INVALID_ARG;
    const PairDesc* pd = find_pair(ctx, a->layer, a->target);
    if (pd == nullptr || a->T < 0) return ADAFUSE_ERR_INVALID_ARG;
    if (a->weight != ADAFUSE_WEIGHT_CURRENT && a->weight != ADAFUSE_WEIGHT_BASE)
        return ADAFUSE_ERR_INVALID_ARG;
    if (a->weight == ADAFUSE_WEIGHT_BASE && !ctx->has_base) return ADAFUSE_ERR_INVALID_ARG;
    if (a->activation < ADAFUSE_ACT_NONE || a->activation > ADAFUSE_ACT_SILU)
        return ADAFUSE_ERR_INVALID_ARG;
    if (a->io_dtype != ADAFUSE_DTYPE_BF16 && a->io_dtype != ADAFUSE_DTYPE_F32)
        return ADAFUSE_ERR_INVALID_ARG;
    p->T = a->T;
    if (a->T == 0) return ADAFUSE_OK;
    if (a->T > INT32_MAX) return ADAFUSE_ERR_UNSUPPORTED_SHAPE;
    const int64_t size = a->io_dtype == ADAFUSE_DTYPE_F32 ? 4 : 2;
    if (!rows_ok(a->x, a->ldx, pd->in, 2) || !rows_ok(a->y, a->ldy, pd->out, size))
        return ADAFUSE_ERR_INVALID_ARG;
    if (a->mul != nullptr && !rows_ok(a->mul, a->ldmul, pd->out, size)) return ADAFUSE_ERR_INVALID_ARG;
    if (a->residual != nullptr && !rows_ok(a->residual, a->ldres, pd->out, size))
        return ADAFUSE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a->bias) & 3u) return ADAFUSE_ERR_INVALID_ARG;
    p->x = static_cast<const uint16_t*>(a->x);
    p->W = a->weight == ADAFUSE_WEIGHT_BASE ? pd->W0 : pd->W;
    p->bias = a->bias;
    p->mul = a->mul;
    p->res = a->residual;
    p->y = a->y;
    p->ldx = a->ldx;
    p->ldmul = a->ldmul;
    p->ldres = a->ldres;
    p->ldy = a->ldy;
    p->out = pd->out;
    p->in = pd->in;
    p->act = a->activation;
    p->f32 = a->io_dtype == ADAFUSE_DTYPE_F32;
    p->status = ctx->d_status;
    return ADAFUSE_OK;
}

// The pending request of the test hook: which launch of this call stalls, 0 = none.
int take_stall(adafuse_ctx* ctx) {
    return ctx->stall_product.load(std::memory_order_relaxed) == 0 ? 0 : ctx->stall_product.exchange(0);
}

// One launch of the router: 32 tokens a CTA, their columns shared by a cluster
// of up to 8 CTAs while that keeps the grid resident at once (T = 1 4096 x 8, T =
// 4096 4096 x 16, T = 777 5120 x 64: 6.1, 31.4, 54.1 us; on one CTA a group 19, 39,
// 145).
template <int EMAX, typename H>
cudaError_t launch_route_as(const H* h, int64_t T, int64_t d, int64_t ldh, const float* Wr, const GateParams& g,
                            int32_t* route, const adafuse_ctx* ctx, cudaStream_t s) {
    const int64_t groups = ceil_div(T, kRouteTokens), chunks = ceil_div(d, kRouteDepth);
    int C = 1;
    const int64_t most = (EMAX <= 16 ? 2 : 1) * (int64_t)ctx->sm_count;   // resident CTAs
    while (C < 8 && groups * C * 2 <= most && chunks >= C * 2) C *= 2;
    if (groups * C > INT32_MAX) return cudaErrorInvalidConfiguration;
    const size_t smem = std::max<size_t>(kRouteStages * route_stage_bytes<H>(g.E), route_tail_bytes<EMAX>());
    auto kernel = route_experts_kernel<EMAX, H>;
    ensure_smem_attr(kernel, smem, ctx->device);
    const int h_piece = ldh * (int64_t)sizeof(H) % 16 == 0 ? 16 : 8;
    const int w_piece = (reinterpret_cast<uintptr_t>(Wr) & 15u) == 0 ? 16 : 4;
    return launch_clusters(kernel, groups * C, kRouteThreads, smem, C, s, h, T, d, ldh, Wr, g, route, C,
                           h_piece, w_piece);
}

template <typename H>
cudaError_t launch_route(const H* h, int64_t T, int64_t d, int64_t ldh, const float* Wr, const GateParams& g,
                         int32_t* route, const adafuse_ctx* ctx, cudaStream_t s) {
    const int E = g.E;
    if (E <= 8) return launch_route_as<8>(h, T, d, ldh, Wr, g, route, ctx, s);
    if (E <= 16) return launch_route_as<16>(h, T, d, ldh, Wr, g, route, ctx, s);
    if (E <= 32) return launch_route_as<32>(h, T, d, ldh, Wr, g, route, ctx, s);
    return launch_route_as<64>(h, T, d, ldh, Wr, g, route, ctx, s);
}

}  // namespace

extern "C" {

int adafuse_route_experts(adafuse_ctx* ctx, const void* h, int32_t h_dtype, int64_t T, int64_t d,
                          int64_t ldh, const float* Wr, const adafuse_gating* gating, int32_t slots,
                          void* route, void* stream) {
    if (ctx == nullptr || gating == nullptr) return ADAFUSE_ERR_INVALID_ARG;
    if (h_dtype != ADAFUSE_DTYPE_BF16 && h_dtype != ADAFUSE_DTYPE_F32) return ADAFUSE_ERR_INVALID_ARG;
    if (T < 0 || d < 4 || d > INT32_MAX || (d & 3) != 0 || (ldh & 3) != 0 || ldh < d || !slots_ok(slots))
        return ADAFUSE_ERR_INVALID_ARG;
    const adafuse_gating& q = *gating;
    const int E = ctx->n_experts;
    if (q.score != ADAFUSE_SCORE_SOFTMAX && q.score != ADAFUSE_SCORE_SIGMOID)
        return ADAFUSE_ERR_INVALID_ARG;
    if (q.k < 1 || q.k > slots || q.n_groups < 1 || q.n_groups > E || E % q.n_groups != 0)
        return ADAFUSE_ERR_INVALID_ARG;
    if (q.top_groups < 1 || q.top_groups > q.n_groups || q.group_top < 1 || q.group_top > 2)
        return ADAFUSE_ERR_INVALID_ARG;
    if (!std::isfinite(q.scale) || (reinterpret_cast<uintptr_t>(q.bias) & 3u))
        return ADAFUSE_ERR_INVALID_ARG;
    if (T == 0) return ADAFUSE_OK;
    if (h == nullptr || Wr == nullptr || route == nullptr || !aligned16(h) || !aligned16(route) ||
        (reinterpret_cast<uintptr_t>(Wr) & 3u))
        return ADAFUSE_ERR_INVALID_ARG;
    DeviceGuard guard(ctx->device);
    if (!guard.ok) return cuda_fail(cudaGetLastError(), "cudaSetDevice");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const GateParams g{q.score, q.k, q.n_groups, q.top_groups, q.group_top, q.renorm != 0,
                       q.scale, q.bias, E, slots};
    int32_t* rt = static_cast<int32_t*>(route);
    const cudaError_t e = h_dtype == ADAFUSE_DTYPE_F32
                              ? launch_route(static_cast<const float*>(h), T, d, ldh, Wr, g, rt, ctx, s)
                              : launch_route(static_cast<const __nv_bfloat16*>(h), T, d, ldh, Wr, g, rt, ctx, s);
    return e == cudaSuccess ? ADAFUSE_OK : cuda_fail(e, "route launch");
}

int adafuse_linear(adafuse_ctx* ctx, const adafuse_linear_args* args, void* stream) {
    LinearParams p;
    const int rc = linear_params(ctx, args, &p);
    if (rc != ADAFUSE_OK || p.T == 0) return rc;
    DeviceGuard guard(ctx->device);
    if (!guard.ok) return cuda_fail(cudaGetLastError(), "cudaSetDevice");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (p.T <= kStreamMaxTokens) {
        e = launch_stream<kProduct>(p, p.W, p.out, nullptr, ctx, s);
    } else {
        TcLinear L;
        std::memset(&L, 0, sizeof L);
        int stall = take_stall(ctx);
        for (int64_t t = 0; t < p.T && e == cudaSuccess; t += kTokensPerLaunch) {
            L.p = token_range(p, t, std::min(p.T - t, kTokensPerLaunch));
            L.stall = --stall == 0;
            e = launch_product(L, ctx, s);
        }
    }
    return e == cudaSuccess ? ADAFUSE_OK : cuda_fail(e, "linear launch");
}

int adafuse_linear_workspace(const adafuse_ctx* ctx, int32_t layer, int32_t target, int64_t T,
                             int32_t io_dtype, int64_t* bytes) {
    if (ctx == nullptr || bytes == nullptr || T < 0) return ADAFUSE_ERR_INVALID_ARG;
    const PairDesc* pd = find_pair(ctx, layer, target);
    if (pd == nullptr) return ADAFUSE_ERR_INVALID_ARG;
    if (io_dtype != ADAFUSE_DTYPE_BF16 && io_dtype != ADAFUSE_DTYPE_F32) return ADAFUSE_ERR_INVALID_ARG;
    if (T > INT32_MAX) return ADAFUSE_ERR_UNSUPPORTED_SHAPE;
    *bytes = routed_layout(ctx, *pd, std::min(T, kTokensPerLaunch), io_dtype == ADAFUSE_DTYPE_F32).bytes;
    return ADAFUSE_OK;
}

int adafuse_linear_routed(adafuse_ctx* ctx, const adafuse_linear_args* args, const void* routes,
                          int32_t slots, void* workspace, int64_t workspace_bytes, void* stream) {
    LinearParams p;
    const int rc = linear_params(ctx, args, &p);
    if (rc != ADAFUSE_OK) return rc;
    if (!slots_ok(slots)) return ADAFUSE_ERR_INVALID_ARG;
    if (p.T == 0) return ADAFUSE_OK;
    if (routes == nullptr || !aligned16(routes)) return ADAFUSE_ERR_INVALID_ARG;
    const PairDesc* pd = find_pair(ctx, args->layer, args->target);
    const RoutedLayout lay = routed_layout(ctx, *pd, std::min(p.T, kTokensPerLaunch), p.f32 != 0);
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < lay.bytes)
        return ADAFUSE_ERR_INVALID_ARG;
    p.A = pd->A;
    p.B = pd->B;
    p.routes = static_cast<const int32_t*>(routes);
    p.slots = slots;
    p.E = ctx->n_experts;
    p.r = ctx->rank;
    p.s = ctx->scale;
    DeviceGuard guard(ctx->device);
    if (!guard.ok) return cuda_fail(cudaGetLastError(), "cudaSetDevice");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.T <= kStreamMaxTokens) {
        float* u = static_cast<float*>(workspace);
        cudaError_t e = launch_stream<kDown>(p, p.A, p.E * p.r, u, ctx, s);
        if (e == cudaSuccess) e = launch_stream<kRouted>(p, p.W, p.out, u, ctx, s);
        return e == cudaSuccess ? ADAFUSE_OK : cuda_fail(e, "routed linear launch");
    }
    p.B = pd->Bk;   // rows of a multiple of 8 columns
    TcLinear L;
    std::memset(&L, 0, sizeof L);
    L.rp = lay.rp;
    L.terms = lay.terms;
    L.b_swizzled = lay.rp == 16 || lay.rp == 32 || lay.rp == 64;
    L.v = static_cast<uint16_t*>(workspace);
    cudaError_t e = cudaSuccess;
    if (lay.pad) {
        uint16_t* padded = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + lay.v_bytes);
        const int64_t nrows = (int64_t)p.E * p.out;
        const int64_t grid = std::min<int64_t>(ceil_div(nrows * lay.rp, 256), (int64_t)ctx->sm_count * 8);
        e = launch_clusters(pad_b_kernel, grid, 256, 0, 1, s, p.B, padded, nrows, p.r, lay.rp);
        p.B = padded;
    }
    L.bsteps = (int)ceil_div((int64_t)p.E * lay.rp, 64);
    int stall = take_stall(ctx);
    for (int64_t t = 0; t < p.T && e == cudaSuccess; t += kTokensPerLaunch) {
        L.p = token_range(p, t, std::min(p.T - t, kTokensPerLaunch));
        L.vsteps = 0;
        L.stall = --stall == 0;
        e = launch_down(L, ctx, s, &L);
        L.vsteps = L.terms * L.bsteps;
        L.stall = --stall == 0;
        if (e == cudaSuccess) e = launch_product(L, ctx, s);
    }
    return e == cudaSuccess ? ADAFUSE_OK : cuda_fail(e, "routed linear launch");
}

int adafuse_debug_stall_next_product(adafuse_ctx* ctx, int32_t launch) {
    if (ctx == nullptr || launch < 1) return ADAFUSE_ERR_INVALID_ARG;
    ctx->stall_product = launch;
    return ADAFUSE_OK;
}

}  // extern "C"
