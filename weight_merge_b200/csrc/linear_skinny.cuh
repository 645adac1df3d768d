// linear_skinny.cuh -- products of a weight with few tokens, bound by reading
// the weight: 128 rows of W on the tensor cores' M side, a tile of up to TN
// tokens on the N side, the contraction split over a cluster.
//
//   D[128 out rows, TN tokens] = W tile x (x tile)^T, fp32 in TMEM
//
// A cluster of S CTAs shares one output tile; CTA q takes the q-th part of the
// contraction, so a weight of few row tiles still keeps every SM loading.  The
// CTAs' partial tiles meet in distributed shared memory: each CTA adds one
// slice of the tile over the S partials in rank order (no atomics, so the same
// bits every time), applies the epilogue and stores it.
//
// A CTA spreads its part over several TMEM accumulators, one 16-deep piece after
// the other, and joins them in registers with fp32 additions, for two reasons:
// successive MMAs on one accumulator wait for each other (about 130 clocks,
// whatever the width: a 64-column step took 0.28 us on one), and accumulators
// drop low bits on every piece (1e-6 of the result after 64 pieces, more in
// proportion).  For fp32 outputs (and V of two terms) the accumulators are
// emptied and started again after at most kFinePieces pieces each: 7e-7 of the
// result instead of 6e-6 at T = 128, 11008 -> 11008, for 23.2 instead of 22.2 us
// at T = 61, 11008 -> 4096.  A bf16 output, rounded at 2^-9 of itself, is not
// worth it.
//
// Routed products append the adapters to the contraction: after the columns of
// x come those of V [T, E * rp] (every token's gated x A^T, zero for experts it
// did not choose) against the stacked B.  V comes from the launch before
// (MODE kDown of this kernel, on the stacked A), which this one overlaps: only
// a CTA whose part reaches V waits for it.
#pragma once

#include <cuda.h>

#include "linear_common.cuh"
#include "linear_stream.cuh"
#include "sm100_ptx.cuh"

namespace adafuse {

// The contraction of a product kernel: `xsteps` 64-column steps of x and W,
// then `vsteps` steps of V and the stacked B (terms * the steps of E * rp).
struct TcLinear {
    LinearParams p;
    int xsteps, vsteps;
    int bsteps;        // 64-column steps of E * rp (vsteps = terms * bsteps)
    int rp;            // rank padded to a multiple of 8
    int terms;         // bf16 terms of V
    int b_swizzled;    // rp is 16, 32 or 64: B arrives as [64 / rp][rows][rp] swizzled tiles;
                       // otherwise as eight [rows][8] groups
    uint16_t* v;       // [terms][T][E * rp]
    int rows;          // kDown: E * r; otherwise out
    int tile_rows;     // rows of a tile that are its own: 128, or whole experts of kDown
    int tok_tiles;     // token tiles
    int busy;          // SMs that the launch before holds (host only)
    int stall;         // test hook: the first CTA's (pair's) first stage never fills
};

constexpr int kSkinnyThreads = 384;
constexpr int kFinePieces = 48;    // see the file's head

// Wait, as a whole warp, for the phase with the given parity of the barrier at
// shared-memory address `bar`; gives up (for all lanes alike) after `limit`
// clocks or once *abort is set.  Bounded by the SM's own clock, read every few
// polls: the global timer costs enough per read to pace these short waits.
constexpr long long kWaitClocks = 2000000000ll;   // about 1 s
__device__ __forceinline__ bool try_phase(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int* abort,
                                           long long limit = kWaitClocks) {
    uint32_t polls = 0;
    long long t0 = 0;
    while (!__all_sync(0xffffffffu, try_phase(bar, parity))) {
        if ((++polls & 15u) != 0) continue;
        const long long now = clock64();
        if (t0 == 0) t0 = now;
        if (__any_sync(0xffffffffu, *abort != 0 || now - t0 > limit)) return false;
    }
    return true;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// The context's status word as it is now.
__device__ __forceinline__ int status_now(const LinearParams& p) {
    int v;
    asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p.status) : "memory");
    return v;
}

// TMA loads named by shared-memory addresses, in their single-CTA and their
// CTA-pair form (the pair's completion may be counted in either CTA).
template <bool PAIR>
struct Tma {
    static __device__ __forceinline__ void load2(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
        if constexpr (PAIR)
            asm volatile(
                "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
                "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(m), "r"(x), "r"(y), "r"(bar) : "memory");
        else
            asm volatile(
                "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
                "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(m), "r"(x), "r"(y), "r"(bar) : "memory");
    }
    static __device__ __forceinline__ void load3(uint32_t dst, const CUtensorMap* m, int x, int y, int z,
                                                 uint32_t bar) {
        if constexpr (PAIR)
            asm volatile(
                "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
                "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
                : "memory");
        else
            asm volatile(
                "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
                "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
                : "memory");
    }
    static __device__ __forceinline__ void load4(uint32_t dst, const CUtensorMap* m, int x, int y, int z, int w,
                                                 uint32_t bar) {
        if constexpr (PAIR)
            asm volatile(
                "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
                "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst), "l"(m), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
                : "memory");
        else
            asm volatile(
                "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
                "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst), "l"(m), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
                : "memory");
    }
    // arrive on a barrier, announcing `bytes` that will complete on it
    static __device__ __forceinline__ void expect(uint32_t bar, uint32_t bytes) {
        if constexpr (PAIR)
            asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                         : "memory");
        else
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                         : "memory");
    }
};

// Loads of one 64-column step of the stacked B for `nrow` out rows from row0:
// columns 64 * c .. of the E * rp stacked ones.  Experts past E read as zero.
template <bool PAIR>
__device__ __forceinline__ void load_b_step(const TcLinear& L, const CUtensorMap* m, int c, int row0, int nrow,
                                            uint32_t dst, uint32_t bar) {
    if (L.b_swizzled) {
        Tma<PAIR>::load3(dst, m, 0, row0, c * (64 / L.rp), bar);
    } else if (L.rp == 8) {
        // an expert's rows are 16 bytes and contiguous: eight of them a line
        Tma<PAIR>::load3(dst, m, 0, row0 >> 3, c * 8, bar);
    } else {
        const int per = L.rp >> 3;
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
            const int grp = c * 8 + j;
            Tma<PAIR>::load4(dst + (uint32_t)(j * 16 * nrow), m, 0, row0, grp % per, grp / per, bar);
        }
    }
}

// One loading warp's share of an output tile, steps [k0, k1): x and V (LEFT) or
// W and the stacked B, into slot `dst0 + stage * stage_bytes` of each stage.
// The whole warp walks the steps and an elected lane issues, so that addresses
// and coordinates stay in uniform registers: walked by one lane alone a step
// took about 530 clocks.  Returns false when a wait gave up.
template <bool PAIR, bool LEFT>
__device__ __forceinline__ bool load_steps(const TcLinear& L, const CUtensorMap* map_k, const CUtensorMap* map_a,
                                           int k0, int k1, int at, int nrow, uint32_t bytes, uint32_t dst0,
                                           uint32_t stage_bytes, uint32_t empty, uint32_t full0, int stages,
                                           int& st, uint32_t& ph, bool& waited, volatile int* abort) {
    const bool lead = sm100::elect_one();
    const int kx = k1 < L.xsteps ? k1 : L.xsteps;
#pragma unroll 1
    for (int i = k0; i < kx; ++i) {
        if (!wait_phase(empty + 8u * (uint32_t)st, ph ^ 1, abort)) return false;
        const uint32_t bar = full0 + 8u * (uint32_t)st;
        if (lead) {
            Tma<PAIR>::expect(bar, bytes);
            Tma<PAIR>::load2(dst0 + (uint32_t)st * stage_bytes, map_k, i * 64, at, bar);
        }
        if (++st == stages) { st = 0; ph ^= 1; }
    }
    if (k1 <= L.xsteps) return true;
    if (LEFT && !waited) {
        pdl_wait();   // V is written by the launch before
        waited = true;
    }
#pragma unroll 1
    for (int i = k0 > L.xsteps ? k0 : L.xsteps; i < k1; ++i) {
        if (!wait_phase(empty + 8u * (uint32_t)st, ph ^ 1, abort)) return false;
        const uint32_t bar = full0 + 8u * (uint32_t)st, dst = dst0 + (uint32_t)st * stage_bytes;
        const int vi = i - L.xsteps;
        if (lead) {
            Tma<PAIR>::expect(bar, bytes);
            if constexpr (LEFT)
                Tma<PAIR>::load3(dst, map_a, (vi % L.bsteps) * 64, at, vi / L.bsteps, bar);
            else
                load_b_step<PAIR>(L, map_a, vi % L.bsteps, at, nrow, dst, bar);
        }
        if (++st == stages) { st = 0; ph ^= 1; }
    }
    return true;
}

// Shared-memory descriptor of a step's first 16-column piece at address 0, and
// what to add for the other three; a stage's address is added in 16-byte units.
struct StepDesc {
    uint64_t base;
    uint32_t off[4];
};

// Rows of 64 columns, 128-byte swizzle (W, x, V).
__device__ __forceinline__ uint64_t row_desc(uint32_t addr) {
    return sm100::smem_desc(addr, 16, 1024, sm100::kSwizzle128B);
}

// A step of the stacked B as load_b_step leaves it.
__device__ __forceinline__ StepDesc b_desc(const TcLinear& L, uint32_t addr, uint32_t nrow) {
    using namespace sm100;
    StepDesc d;
    const uint32_t rp = (uint32_t)L.rp;
    d.base = !L.b_swizzled ? smem_desc(addr, 16u * nrow, 128, kSwizzleNone)
                           : smem_desc(addr, 16, 16u * rp,
                                       rp == 16 ? kSwizzle32B : rp == 32 ? kSwizzle64B : kSwizzle128B);
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
        const uint32_t sub = (16u * k) / rp, in = (16u * k) % rp;
        d.off[k] = (L.b_swizzled ? sub * 2u * nrow * rp + in * 2u : 32u * nrow * k) >> 4;
    }
    return d;
}

// The gate of expert e for token t times s: the sum over the record's slots
// that name it (0 when none does).  Bad slots count as empty and set *bad.
__device__ __forceinline__ float gate_of(const LinearParams& p, int64_t t, int e, int& bad) {
    float g = 0.f;
    for (int j = 0; j < p.slots; ++j) {
        int ej;
        float gj;
        if (route_slot(p.routes, p.slots, p.E, t, j, ej, gj, bad) && ej == e) g += gj;
    }
    return p.s * g;
}

// Eight columns of V for token t and expert e, from k (a multiple of 8): gate *
// (x A^T) as bf16 terms, the first the value rounded, the second what that
// rounding left; zeros past the rank.  A token that did not choose the expert
// gets exact zeros, whatever its x holds.
//
// bf16 outputs carry one term, as a bf16 product by B would round it: 2^-9 of the
// adapters' part beside 2^-9 of the result, an error's norm of 0.001666 instead of
// 0.001658 at T = 2048, 4096 -> 4096, 16 experts of rank 64, and 0.001667 instead of
// 0.001666 at T = 24, 5120 -> 13824, 8 of rank 16.  A second term takes 14% and 2%
// more time there.
__device__ __forceinline__ void finish_down8(const TcLinear& L, int64_t t, int e, int k, const float (&u)[8],
                                             int& bad) {
    const LinearParams& p = L.p;
    const float g = gate_of(p, t, e, bad);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = g != 0.f && k + 2 * i < p.r ? g * u[2 * i] : 0.f;
        const float b = g != 0.f && k + 2 * i + 1 < p.r ? g * u[2 * i + 1] : 0.f;
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        const __nv_bfloat162 l = __floats2bfloat162_rn(a - __low2float(h), b - __high2float(h));
        hi[i] = *reinterpret_cast<const uint32_t*>(&h);
        lo[i] = *reinterpret_cast<const uint32_t*>(&l);
    }
    const int64_t width = (int64_t)p.E * L.rp;
    uint16_t* dst = L.v + t * width + (int64_t)e * L.rp + k;   // 16-byte aligned: rp and k are multiples of 8
    *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if (L.terms == 2) *reinterpret_cast<uint4*>(dst + p.T * width) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

template <int TN>
struct SkinnyConfig {
    static_assert(TN == 16 || TN == 32 || TN == 64 || TN == 128, "TN");
    static constexpr uint32_t kWBytes = 128 * 128;          // 128 rows x 64 columns bf16
    static constexpr uint32_t kXBytes = TN * 128;
    static constexpr uint32_t kStageBytes = kWBytes + kXBytes;
    static constexpr int kAccs = TN == 128 ? 2 : TN == 64 ? 4 : 8;   // TMEM accumulators
    static constexpr uint32_t kTmemCols = kAccs * TN;                // 128 or 256: two CTAs fit
    static constexpr uint32_t stages_min() { return 108u * 1024u / kStageBytes; }
    // stages of a launch with `ctas` (1 or 2) CTAs an SM
    static constexpr int stages(int ctas) {
        return (int)((ctas == 1 ? 216u * 1024u : 108u * 1024u) / kStageBytes);
    }
    static constexpr uint32_t smem_bytes(int stages) { return 1024 + stages * kStageBytes + 8 * (2 * stages + 2) + 16; }
    static_assert(TN * 128 * 4 + 32 <= stages_min() * kStageBytes, "the partial tile reuses the ring");
    static_assert(kStageBytes % 1024 == 0, "swizzle atoms stay aligned");
};

template <int TN, int MODE>
__global__ void __launch_bounds__(kSkinnyThreads, 2)
linear_skinny_kernel(const __grid_constant__ TcLinear L, const __grid_constant__ CUtensorMap map_w,
                     const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_b,
                     const __grid_constant__ CUtensorMap map_v, const int S, const int stages) {
    using C = SkinnyConfig<TN>;
    using namespace sm100;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + stages * C::kStageBytes);
    uint64_t* empty = full + stages;
    uint64_t* acc_full = empty + stages;
    uint64_t* acc_empty = acc_full + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    const int q = (int)(blockIdx.x % (unsigned)S);
    const int64_t tile = blockIdx.x / (unsigned)S;
    const int row0 = (int)(tile / L.tok_tiles) * L.tile_rows;
    const int64_t tok0 = (tile % L.tok_tiles) * TN;
    const int nsteps = L.xsteps + L.vsteps;
    const int k0 = (int)((int64_t)q * nsteps / S), k1 = (int)((int64_t)(q + 1) * nsteps / S);
    const int n = k1 - k0;
    // even chunks of at most kFinePieces pieces an accumulator
    constexpr int kChunk = kFinePieces * C::kAccs / 4;
    const bool fine = MODE == kDown ? L.terms == 2 : L.p.f32 != 0;
    const int chunks = fine ? (n + kChunk - 1) / kChunk : 1;
    const int chunk_steps = (n + chunks - 1) / chunks;

    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            // one arrival, with its bytes, from each loading warp
            mbar_init(&full[i], i == 0 && L.stall && blockIdx.x == 0 ? 3 : 2);
            mbar_init(&empty[i], 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 8);        // the warps that read the accumulators
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 5) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // The set-up above overlaps the end of the launch before this one.  A routed
    // product goes on: its x, W and B were complete before the kDown launch let
    // it start, and only V is waited for.
    if (MODE == kDown || L.vsteps == 0) pdl_wait();
    pdl_launch_dependents();
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(L.p.status, ADAFUSE_STATUS_TIMEOUT);
    };

    if (warp == 4 || warp == 6) {
        // two loading warps: one thread's TMA operations start about 120 clocks apart
        int st = 0;
        uint32_t ph = 0;
        bool waited = false;
        const uint32_t ring_s = smem_u32(ring), full_s = smem_u32(full);
        const bool ok =
            warp == 4 ? load_steps<false, true>(L, &map_x, &map_v, k0, k1, (int)tok0, 0, C::kXBytes,
                                                ring_s + C::kWBytes, C::kStageBytes, smem_u32(empty), full_s, stages, st,
                                                ph, waited, abort_flag)
                      : load_steps<false, false>(L, &map_w, &map_b, k0, k1, row0, 128, C::kWBytes, ring_s,
                                                 C::kStageBytes, smem_u32(empty), full_s, stages, st, ph, waited,
                                                 abort_flag);
        if (!ok) fail();
    } else if (warp == 5) {
        // The whole warp walks the steps with the fewest possible operations
        // between the MMAs, and one elected lane issues: descriptors stay in
        // uniform registers and a step takes about 200 clocks instead of 520.
        constexpr uint32_t idesc = instr_desc_bf16(128, TN, 0);
        const uint32_t ring_s = smem_u32(ring), full_s = smem_u32(full), empty_s = smem_u32(empty);
        const uint64_t dw = row_desc(ring_s), dx = row_desc(ring_s + C::kWBytes);
        const StepDesc db = b_desc(L, ring_s, 128);
        int st = 0, i = 0;              // i: the step within its chunk
        uint32_t ph = 0, off = 0;       // off: the stage's offset in 16-byte units
        bool ok = true;
        // successive MMAs go to different accumulators (see the file's head)
        auto acc_of = [&](int k) {
            return tmem + (uint32_t)((k & (C::kAccs >= 4 ? 3 : 1)) * TN) +
                   (C::kAccs == 8 && (i & 1) ? 4u * TN : 0u);
        };
        auto fresh = [&](int k) { return C::kAccs == 8 ? i < 2 : C::kAccs == 4 ? i == 0 : i == 0 && k < 2; };
        auto next_stage = [&]() {
            __syncwarp();
            ++i;
            ++st;
            off += C::kStageBytes / 16;
            if (st == stages) { st = 0; off = 0; ph ^= 1; }
        };
        uint32_t aph = 0;
#pragma unroll 1
        for (int c0 = k0; c0 < k1; c0 += chunk_steps) {
            if (c0 > k0) {
                ok = wait_phase(smem_u32(acc_empty), aph, abort_flag);
                if (!ok) break;
                tc_fence_after();
                aph ^= 1;
            }
            const int c1 = c0 + chunk_steps < k1 ? c0 + chunk_steps : k1;
            const int nx = (c1 < L.xsteps ? c1 : L.xsteps) - c0;   // steps of x and W (<= 0: none)
            i = 0;
#pragma unroll 1
            while (i < nx) {
                ok = wait_phase(full_s + 8u * (uint32_t)st, ph, abort_flag);
                if (!ok) break;
                const uint64_t a = dw + off, b = dx + off;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) tc_mma_f16(acc_of(k), a + 2 * k, b + 2 * k, idesc, !fresh(k));
                    tc_commit_addr(empty_s + 8u * (uint32_t)st);
                }
                next_stage();
            }
#pragma unroll 1
            while (ok && i < c1 - c0) {
                ok = wait_phase(full_s + 8u * (uint32_t)st, ph, abort_flag);
                if (!ok) break;
                const uint64_t a = db.base + off, b = dx + off;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) tc_mma_f16(acc_of(k), a + db.off[k], b + 2 * k, idesc, !fresh(k));
                    tc_commit_addr(empty_s + 8u * (uint32_t)st);
                }
                next_stage();
            }
            if (!ok) break;
            if (elect_one()) tc_commit(acc_full);
            __syncwarp();
        }
        if (!ok) fail();
    }

    // ---- the CTA's partial tile into shared memory: part[token][128 rows]; four
    // warps take the first half of the tokens, four the second
    float* part = reinterpret_cast<float*>(ring);
    if (warp < 4 || warp >= 8) {
        constexpr int kCols = TN / 2, kPiece = TN == 32 || TN == 64 ? 16 : 8;
        const int half = warp < 4 ? 0 : kCols;
        const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)half;
        float sum[kCols];
#pragma unroll
        for (int i = 0; i < kCols; ++i) sum[i] = 0.f;
        bool ok = true;
        uint32_t aph = 0;
#pragma unroll 1
        for (int c0 = 0; c0 < n; c0 += chunk_steps) {
            ok = wait_phase(smem_u32(acc_full), aph, abort_flag, 4 * kWaitClocks);
            if (!ok) break;
            aph ^= 1;
            tc_fence_after();
            const int len = c0 + chunk_steps < n ? chunk_steps : n - c0;
            const int naccs = 4 * len < C::kAccs ? 4 * len : C::kAccs;
#pragma unroll 1
            for (int a = 0; a < naccs; ++a) {
#pragma unroll
                for (int c = 0; c < kCols; c += kPiece) {
                    float v[kPiece];
                    if constexpr (kPiece == 16) tmem_ld16(t_lane + (uint32_t)(a * TN + c), v);
                    else tmem_ld8(t_lane + (uint32_t)(a * TN + c), v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < kPiece; ++i) sum[c + i] += v[i];
                }
            }
            if (c0 + chunk_steps < n) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acc_empty);
            }
        }
        if (ok) {
            // V has landed, so the launch that wrote it is complete: did it give up?
            int down = 0;
            if (MODE == kProduct && L.vsteps > 0 && threadIdx.x == 0) down = status_now(L.p);
#pragma unroll
            for (int i = 0; i < kCols; ++i) part[(half + i) * 128 + (warp & 3) * 32 + lane] = sum[i];
            tc_fence_before();
            if (down & ADAFUSE_STATUS_TIMEOUT) *abort_flag = 1;
        } else {
            fail();
        }
    }
    // ---- this CTA's slice of the tile: sum over the cluster, epilogue, store
    const int ntok = (int)(L.p.T - tok0 < TN ? L.p.T - tok0 : TN);
    const int nrow = L.rows - row0 < L.tile_rows ? L.rows - row0 : L.tile_rows;
    // eight columns each: of y (16 groups a token), or of an expert's V
    const int per_expert = MODE == kDown ? L.rp >> 3 : 0;
    const int per_tok = MODE == kDown ? nrow / L.p.r * per_expert : 16;
    const int groups = ntok * per_tok;
    const int g0 = (int)((int64_t)q * groups / S), g1 = (int)((int64_t)(q + 1) * groups / S);
    SideCols<8> side;
    // what does not depend on the sums is requested before they are complete
    auto request = [&](int gi) {
        if (MODE == kProduct && gi < g1 && (gi & 15) * 8 < nrow)
            side.load(L.p, tok0 + (gi >> 4), row0 + (gi & 15) * 8);
    };
    request(g0 + (int)threadIdx.x);
    __syncthreads();
    // where any CTA of the cluster gave up there is no tile to store
    bool whole = !*abort_flag;
    if (S > 1) {
        cluster_sync();
        const uint32_t gave_up = lane < S ? ld_cluster_u32(cluster_addr((const void*)abort_flag, (uint32_t)lane)) : 0u;
        whole = !__any_sync(0xffffffffu, gave_up != 0);
    }
    if (whole) {
        const uint32_t part_s = smem_u32(part);
        int bad = 0;
#pragma unroll 1
        for (int gi = g0 + (int)threadIdx.x; gi < g1; gi += kSkinnyThreads) {
            const int tok = MODE == kDown ? gi / per_tok : gi >> 4, in_tok = gi - tok * per_tok;
            int r8 = in_tok * 8, e = 0, k = 0;
            if constexpr (MODE == kDown) {
                e = in_tok / per_expert;
                k = (in_tok - e * per_expert) * 8;
                r8 = e * L.p.r + k;
            }
            if (r8 < nrow) {
                // (kDown: reads past an expert's or the tile's last row stay inside the
                // ring and are left out later; rows that start anywhere are read as
                // the three aligned vectors around them: T = 371, 8376 -> 288, 16 experts
                // of rank 21 42 us, read one by one 60)
                const uint32_t off = part_s + (uint32_t)(tok * 128 + r8) * 4u;
                const bool anywhere = MODE == kDown && (L.p.r & 3) != 0;
                const uint32_t from = anywhere ? off & ~15u : off;
                float v[MODE == kDown ? 12 : 8];
#pragma unroll
                for (int i = 0; i < (MODE == kDown ? 12 : 8); ++i) v[i] = 0.f;
#pragma unroll 4
                for (int c = 0; c < S; ++c) {
                    uint32_t a = from;
                    if (S > 1) asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(from), "r"(c));
                    const float4 lo = ld_cluster_f4(a), hi = ld_cluster_f4(a + 16);
                    v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
                    v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
                    if constexpr (MODE == kDown) {
                        if (anywhere) {
                            const float4 end = ld_cluster_f4(a + 32);
                            v[8] += end.x; v[9] += end.y; v[10] += end.z; v[11] += end.w;
                        }
                    }
                }
                if constexpr (MODE == kDown) {
                    const uint32_t sh = (off >> 2 & 3u);
                    if (anywhere) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            v[i] = sh < 2 ? (sh == 0 ? v[i] : v[i + 1]) : (sh == 2 ? v[i + 2] : v[i + 3]);
                    }
                    const float u[8] = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
                    finish_down8(L, tok0 + tok, row0 / L.p.r + e, k, u, bad);
                } else {
                    finish_cols(L.p, tok0 + tok, row0 + r8, v, side);
                }
            }
            request(gi + kSkinnyThreads);
        }
        if (MODE == kDown && bad != 0) atomicOr(L.p.status, bad);
    } else {
        // copies and MMAs still in flight get time to land before the CTA's
        // shared memory and TMEM go
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 200000ull) { }
    }
    if (S > 1) cluster_sync();   // peers may still read this CTA's partial tile
    else __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// Ranks above 8 that are not multiples of 8: B [E, out, r] copied to rows of
// rp columns, zero past r (B rows of 2 * r bytes are no legal TMA stride).
__global__ void __launch_bounds__(256)
pad_b_kernel(const uint16_t* B, uint16_t* dst, int64_t nrows, int r, int rp) {
    const int64_t total = nrows * rp;
    pdl_wait();   // the launch before may still read dst
    pdl_launch_dependents();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / rp;
        const int k = (int)(i % rp);
        dst[i] = k < r ? B[row * r + k] : (uint16_t)0;
    }
}

}  // namespace adafuse
