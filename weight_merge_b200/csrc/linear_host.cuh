// linear_host.cuh -- host side of the product kernels: tensor maps, the split
// of the contraction, workspace layout and launches.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <mutex>
#include <vector>

#include "context.cuh"
#include "linear_pair.cuh"
#include "linear_skinny.cuh"
#include "linear_stream.cuh"

namespace adafuse {

inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

inline bool encode_map(CUtensorMap* m, int dims, const void* base, const cuuint64_t* dim,
                       const cuuint64_t* stride_bytes, const cuuint32_t* box, CUtensorMapSwizzle sw) {
    const EncodeTiledFn enc = encode_tiled_fn();
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return enc != nullptr &&
           enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)dims, const_cast<void*>(base), dim,
               stride_bytes, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [rows, cols] bf16, rows ld elements apart: boxes of 64 columns x box_rows,
// 128-byte swizzle.
inline bool encode_rows(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld,
                        int box_rows) {
    const cuuint64_t dim[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t stride[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    return encode_map(m, 2, base, dim, stride, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// V [terms][T][width]: boxes of 64 columns x box_rows tokens of one term;
// columns past the width read as zero.
inline bool encode_v(CUtensorMap* m, const TcLinear& L, int box_rows) {
    const int64_t width = (int64_t)L.p.E * L.rp;
    const cuuint64_t dim[3] = {(cuuint64_t)width, (cuuint64_t)L.p.T, (cuuint64_t)L.terms};
    // (one term: any legal stride, the third coordinate stays 0)
    const cuuint64_t stride[2] = {(cuuint64_t)width * 2, (cuuint64_t)((L.terms > 1 ? L.p.T : 1) * width * 2)};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    return encode_map(m, 3, L.v, dim, stride, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// The stacked B [E, out, rp] for load_b_step on nrow rows.
inline bool encode_b(CUtensorMap* m, const TcLinear& L, int nrow) {
    const cuuint64_t rp = (cuuint64_t)L.rp, out = (cuuint64_t)L.p.out, E = (cuuint64_t)L.p.E;
    if (L.b_swizzled) {
        const cuuint64_t dim[3] = {rp, out, E};
        const cuuint64_t stride[2] = {rp * 2, out * rp * 2};
        const cuuint32_t box[3] = {(cuuint32_t)rp, (cuuint32_t)nrow, (cuuint32_t)(64 / rp)};
        return encode_map(m, 3, L.p.B, dim, stride, box,
                          rp == 16 ? CU_TENSOR_MAP_SWIZZLE_32B
                                   : rp == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (rp == 8) {
        // [E, out, 8] seen as [E][out / 8][64]: lines of 128 bytes that land as
        // the same [8 experts][nrow][8]
        const cuuint64_t dim[3] = {64, out / 8, E};
        const cuuint64_t stride[2] = {128, out * 16};
        const cuuint32_t box[3] = {64, (cuuint32_t)(nrow / 8), 8};
        return encode_map(m, 3, L.p.B, dim, stride, box, CU_TENSOR_MAP_SWIZZLE_NONE);
    }
    const cuuint64_t dim[4] = {8, out, rp / 8, E};
    const cuuint64_t stride[3] = {rp * 2, 16, out * rp * 2};
    const cuuint32_t box[4] = {8, (cuuint32_t)nrow, 1, 1};
    return encode_map(m, 4, L.p.B, dim, stride, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Workspace of a routed product: V (or, for up to kStreamMaxTokens tokens, u = x A^T
// in fp32: four bytes a value cover either), then, where more tokens meet a rank above
// 8 that is no multiple of 8, a padded copy of B.  That copy is made by each call:
// B may change between calls, and a copy kept with the context (as for ranks below
// 8, where it is at most 8 columns an expert) would hold up to twice the adapters'
// memory for every weight.
struct RoutedLayout {
    int rp, terms;
    bool pad;          // B is padded per call
    int64_t v_bytes, bytes;
};

inline RoutedLayout routed_layout(const adafuse_ctx* ctx, const PairDesc& pd, int64_t T, bool f32) {
    RoutedLayout w;
    w.rp = (int)round_up(ctx->rank, 8);
    w.terms = f32 ? 2 : 1;
    w.pad = ctx->rank % 8 != 0 && pd.Bk == pd.B;
    w.v_bytes = round_up(T * ctx->n_experts * w.rp * 4, 256);
    w.bytes = w.v_bytes;
    if (w.pad && T > kStreamMaxTokens) w.bytes += round_up((int64_t)ctx->n_experts * pd.out * w.rp * 2, 256);
    return w;
}

// A launch on clusters that may be set up while the launch before it ends:
// every kernel launched here executes griddepcontrol.wait before it touches
// memory an earlier launch may write (or relies on one that did), and lets the
// launch after it be set up once all its own CTAs run (1 to 2 us a call where
// calls follow each other).  A launch is complete only after what it waited for,
// so waiting for the one before is waiting for all.
template <typename Kernel, typename... Args>
cudaError_t launch_clusters(Kernel kernel, int64_t grid, int threads, size_t smem, int cluster, cudaStream_t s,
                            const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Clusters of 2, 4 and 8 CTAs of the skinny kernel, one CTA an SM, that the device
// runs at once: fewer than its SMs, since a cluster stays within one group of
// them.  Asked once per device.
struct ClusterRoom {
    int device, of[4];   // of[i]: clusters of 1 << i
};
inline ClusterRoom cluster_room(const adafuse_ctx* ctx) {
    static std::mutex mu;
    static std::vector<ClusterRoom> known;
    std::lock_guard<std::mutex> lk(mu);
    for (const ClusterRoom& r : known)
        if (r.device == ctx->device) return r;
    using C = SkinnyConfig<128>;
    auto kernel = linear_skinny_kernel<128, kProduct>;
    ensure_smem_attr(kernel, C::smem_bytes(C::stages(1)), ctx->device);
    ClusterRoom r = {ctx->device, {ctx->sm_count, 0, 0, 0}};
    for (int i = 1; i < 4; ++i) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 1u << i;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3((unsigned)ctx->sm_count >> i << i, 1, 1);
        cfg.blockDim = dim3(kSkinnyThreads, 1, 1);
        cfg.dynamicSmemBytes = C::smem_bytes(C::stages(1));
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&r.of[i], kernel, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            r.of[i] = 0;   // the contraction is not split that far
        }
    }
    try {
        known.push_back(r);
    } catch (...) {
        // not remembered: asked again
    }
    return r;
}

// Cluster size of the skinny kernel: the contraction is split while all clusters
// run at once, beside the `busy` CTAs of the launch before, and every CTA keeps
// at least four steps.  Measured at T = 61 (4096 -> 1024, 4096 -> 4096, 11008 -> 4096,
// 4096 -> 11008): 10.2, 13.1, 21.6 and 21.5 us at the sizes this takes (8, 4, 4, 1),
// up to twice that at the others.  A cluster that
// finds no room runs in a second wave: T = 250, 4096 -> 1024 with 8 experts of rank 16
// took 34.9 us on clusters of 8 and 21.1 on clusters of 4.
inline int skinny_split(int64_t tiles, int nsteps, int busy, const ClusterRoom& room) {
    int i = 0;
    while (i < 3 && tiles <= room.of[i + 1] - (busy >> (i + 1)) - (busy > 0) && nsteps >> (i + 1) >= 4) ++i;
    return 1 << i;
}

template <int TN, int MODE>
cudaError_t launch_skinny(TcLinear L, const CUtensorMap& map_w, const CUtensorMap& map_b, const adafuse_ctx* ctx,
                          cudaStream_t s, int* ctas) {
    using C = SkinnyConfig<TN>;
    CUtensorMap map_x, map_v;
    std::memset(&map_v, 0, sizeof map_v);
    if (!encode_rows(&map_x, L.p.x, L.p.T, L.p.in, L.p.ldx, TN)) return cudaErrorInvalidValue;
    if (L.vsteps > 0 && !encode_v(&map_v, L, TN)) return cudaErrorInvalidValue;
    L.tok_tiles = (int)ceil_div(L.p.T, TN);
    const int64_t tiles = ceil_div(L.rows, L.tile_rows) * L.tok_tiles;
    const int S = skinny_split(tiles, L.xsteps + L.vsteps, L.busy, cluster_room(ctx));
    if (tiles * S > INT32_MAX) return cudaErrorInvalidConfiguration;
    *ctas = (int)(tiles * S);
    const int stages = C::stages(tiles * S <= ctx->sm_count ? 1 : 2);
    auto kernel = linear_skinny_kernel<TN, MODE>;
    ensure_smem_attr(kernel, C::smem_bytes(C::stages(1)), ctx->device);
    return launch_clusters(kernel, tiles * S, kSkinnyThreads, C::smem_bytes(stages), S, s, L, map_w,
                           map_x, map_b, map_v, S, stages);
}

// The smallest tile that holds the tokens, up to 128.
template <int MODE>
cudaError_t launch_skinny_any(const TcLinear& L, const CUtensorMap& map_w, const CUtensorMap& map_b,
                              const adafuse_ctx* ctx, cudaStream_t s, int* ctas) {
    const int64_t T = L.p.T;
    if (T <= 16) return launch_skinny<16, MODE>(L, map_w, map_b, ctx, s, ctas);
    if (T <= 32) return launch_skinny<32, MODE>(L, map_w, map_b, ctx, s, ctas);
    if (T <= 64) return launch_skinny<64, MODE>(L, map_w, map_b, ctx, s, ctas);
    return launch_skinny<128, MODE>(L, map_w, map_b, ctx, s, ctas);
}

// Grid of the stream kernel: two CTAs an SM less `reserve` CTAs, or, where
// there are few units, clusters of S <= 8 CTAs that share a unit's columns
// while every warp keeps a step.
inline int stream_grid(int rows, int in, int reserve, int sm_count, int* S) {
    const int units = (int)ceil_div(rows, kStreamRows);
    *S = 1;
    while (*S < 8 && units * *S * 2 <= 2 * sm_count && in >= 64 * kStreamWarps * 2 * *S) *S *= 2;
    if (*S > 1) return units * *S;
    return std::max(1, std::min((int)ceil_div(rows, 4), 2 * sm_count - reserve));
}

// At most kStreamMaxTokens tokens.  kRouted overlaps the kDown launch before
// it and leaves that launch's CTAs their places.
template <int MODE>
cudaError_t launch_stream(const LinearParams& p, const uint16_t* W, int rows, float* u, const adafuse_ctx* ctx,
                          cudaStream_t s) {
    int S = 1, reserve = 0;
    if (MODE == kRouted) reserve = std::min(stream_grid(p.E * p.r, p.in, 0, ctx->sm_count, &S), ctx->sm_count);
    const int grid = stream_grid(rows, p.in, reserve, ctx->sm_count, &S);
    const bool wide = p.in % 16 == 0 && (reinterpret_cast<uintptr_t>(W) & 31u) == 0;
    return wide ? launch_clusters(linear_stream_kernel<MODE, true>, grid, kStreamThreads, 0, S, s, p,
                                  W, rows, u, S)
                : launch_clusters(linear_stream_kernel<MODE, false>, grid, kStreamThreads, 0, S, s, p,
                                  W, rows, u, S);
}

// Tile width of the pair kernel: the multiple of 16 in [128, 256] with the least
// estimated time for the longest pair's share, the narrower among equals (their
// tiles finish sooner).  A 64-column step of a tile takes about (BN + 64) ns
// (T = 512 4096 -> 4096, one round: 18.4, 21.1, 25.6, 26.8 us at BN = 128, 192,
// 240, 256; T = 4096, 7, 5, 4 and 4 rounds: 109.7, 100.6, 93.7, 94.9 us).  *us:
// the estimate for nsteps.
inline int pair_width(int64_t tok_tiles, int rows, int64_t pairs, int nsteps, double* us) {
    int best = kPairMaxCols;
    int64_t least = INT64_MAX;
    for (int bn = kPairMaxCols; bn >= 128; bn -= 16) {
        const int64_t ns = ceil_div(tok_tiles * ceil_div(rows, bn), pairs) * (bn + 64);
        if (ns <= least) { least = ns; best = bn; }
    }
    *us = 6.0 + 1e-3 * (double)least * nsteps;
    return best;
}

// SMs for a product's CTA pairs: beside a launch before it that holds a quarter of
// them or fewer, those it leaves (T = 333, 4096 -> 4096, 4 experts of rank 4: 22.9 us
// on 62 pairs; on 74, of which 12 wait 9 us for their SMs, 29.0); otherwise all (T =
// 765, 1120 -> 14312 fp32, 16 experts of rank 16: 47 us; beside 72 CTAs 68).
inline int64_t pair_count(const TcLinear& L, const adafuse_ctx* ctx) {
    return (ctx->sm_count - (L.busy <= ctx->sm_count / 4 ? L.busy : 0)) / 2;
}

// More than 128 tokens: the skinny kernel (tiles of 128 x 128, contraction
// split) where its estimate is below the pair kernel's, that is where the pair
// kernel has too few tiles to occupy the SMs.  Measured at T = 333 4096 -> 1024:
// 13.8 against 17.6 us; T = 1037 4096 -> 1024: 15.4 against 17.4 us.
inline bool pair_is_faster(const TcLinear& L, const adafuse_ctx* ctx) {
    const int nsteps = L.xsteps + L.vsteps, sm_count = ctx->sm_count;
    double pair_us;
    pair_width(ceil_div(L.p.T, kPairTokens), L.rows, pair_count(L, ctx), nsteps, &pair_us);
    const int64_t tiles = ceil_div(L.rows, L.tile_rows) * ceil_div(L.p.T, 128);
    const int S = skinny_split(tiles, nsteps, L.busy, cluster_room(ctx));
    const double skinny_us = 7.0 + (double)(ceil_div(tiles * S, sm_count) * ceil_div(nsteps, S)) * 0.19;
    return pair_us <= skinny_us;
}

// W: the [L.rows, in] operand, the weight or (kDown) the stacked A.
template <bool F32, int MODE>
cudaError_t launch_pair(TcLinear L, const uint16_t* W, const adafuse_ctx* ctx, cudaStream_t s) {
    L.tok_tiles = (int)ceil_div(L.p.T, kPairTokens);
    const int64_t most = pair_count(L, ctx);
    double us;
    const int BN = pair_width(L.tok_tiles, L.rows, most, L.xsteps + L.vsteps, &us);
    CUtensorMap map_w, map_x, map_b, map_v;
    std::memset(&map_b, 0, sizeof map_b);
    std::memset(&map_v, 0, sizeof map_v);
    if (!encode_rows(&map_w, W, L.rows, L.p.in, L.p.in, BN / 2) ||
        !encode_rows(&map_x, L.p.x, L.p.T, L.p.in, L.p.ldx, 128))
        return cudaErrorInvalidValue;
    if (L.vsteps > 0 && (!encode_b(&map_b, L, BN / 2) || !encode_v(&map_v, L, 128)))
        return cudaErrorInvalidValue;
    const int64_t tiles = L.tok_tiles * ceil_div(L.rows, BN);
    auto kernel = linear_pair_kernel<F32, MODE>;
    ensure_smem_attr(kernel, kPairSmemBytes, ctx->device);
    return launch_clusters(kernel, 2 * std::min(tiles, most), kPairThreads, kPairSmemBytes, 2, s, L,
                           map_w, map_x, map_b, map_v, BN);
}

// y of one product; L carries V's geometry when the adapters are part of it.
inline cudaError_t launch_product(TcLinear L, const adafuse_ctx* ctx, cudaStream_t s) {
    L.rows = L.p.out;
    L.tile_rows = 128;
    L.xsteps = (int)ceil_div(L.p.in, 64);
    if (L.p.T > 128 && pair_is_faster(L, ctx))
        return L.p.f32 ? launch_pair<true, kProduct>(L, L.p.W, ctx, s) : launch_pair<false, kProduct>(L, L.p.W, ctx, s);
    CUtensorMap map_w, map_b;
    std::memset(&map_b, 0, sizeof map_b);
    if (!encode_rows(&map_w, L.p.W, L.p.out, L.p.in, L.p.in, 128)) return cudaErrorInvalidValue;
    if (L.vsteps > 0 && !encode_b(&map_b, L, 128)) return cudaErrorInvalidValue;
    int ctas;
    return launch_skinny_any<kProduct>(L, map_w, map_b, ctx, s, &ctas);
}

// V of a routed product.  Notes in *next the SMs that this launch holds, up to
// half of them: the product launched next is laid out to run beside it (beside a
// larger launch nothing would be left: it starts as that one ends).
inline cudaError_t launch_down(TcLinear L, const adafuse_ctx* ctx, cudaStream_t s, TcLinear* next) {
    CUtensorMap map_a, none;
    std::memset(&none, 0, sizeof none);
    L.rows = L.p.E * L.p.r;
    L.tile_rows = 128 / L.p.r * L.p.r;
    L.xsteps = (int)ceil_div(L.p.in, 64);
    L.vsteps = L.busy = 0;
    next->busy = 0;
    if (L.p.T > 128 && L.rp == L.p.r && pair_is_faster(L, ctx))
        return L.terms == 2 ? launch_pair<true, kDown>(L, L.p.A, ctx, s)
                            : launch_pair<false, kDown>(L, L.p.A, ctx, s);
    if (!encode_rows(&map_a, L.p.A, L.rows, L.p.in, L.p.in, 128)) return cudaErrorInvalidValue;
    int ctas = 0;
    const cudaError_t e = launch_skinny_any<kDown>(L, map_a, none, ctx, s, &ctas);
    if (ctas <= ctx->sm_count / 2) next->busy = ctas;
    return e;
}

}  // namespace adafuse
