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
// Tensor-core accumulators drop low bits on every 16-deep step (measured: 4e-6
// of the result after 4096 products, 1.2e-5 after 11008).  A CTA therefore
// spreads its part over several TMEM accumulators, each summing a run of it,
// and joins them in registers with fp32 additions.
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
    int tok_tiles;     // token tiles
};

constexpr int kSkinnyThreads = 224;

// Wait for the phase with the given parity; gives up after `limit` clocks or
// once *abort is set.  Bounded by the SM's own clock, read every few polls:
// the global timer costs enough per read to pace these short waits.
constexpr long long kWaitClocks = 2000000000ll;   // about 1 s
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort,
                                           long long limit = kWaitClocks) {
    if (sm100::mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 16; ++i)
            if (sm100::mbar_try_wait(bar, parity)) return true;
        if (*abort || clock64() - t0 > limit) return false;
    }
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

// Loads of one 64-column step of the stacked B for `nrow` (128 or 64) out rows
// from row0: columns 64 * c .. of the E * rp stacked ones.  Experts past E read
// as zero.
template <typename Load3, typename Load4>
__device__ __forceinline__ void load_b_step(const TcLinear& L, int c, int row0, int nrow, uint8_t* dst,
                                            Load3&& load3, Load4&& load4) {
    if (L.b_swizzled) {
        load3(dst, 0, row0, c * (64 / L.rp));
    } else if (L.rp == 8) {
        // an expert's rows are 16 bytes and contiguous: eight of them a line
        load3(dst, 0, row0 >> 3, c * 8);
    } else {
        const int per = L.rp >> 3;
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
            const int grp = c * 8 + j;
            load4(dst + j * 16 * nrow, 0, row0, grp % per, grp / per);
        }
    }
}

// Shared-memory descriptors of the four 16-column pieces of a step: fixed bits
// and the pieces' offsets, worked out once, so that the issuing thread adds the
// stage's address and nothing else (it has 512 clocks a step in the pair kernel).
struct StepDesc {
    uint64_t fixed;
    uint32_t off[4];   // in 16-byte units
    __device__ __forceinline__ uint64_t at(uint32_t base, int k) const {
        return fixed | (uint64_t)(((base >> 4) + off[k]) & 0x3FFFu);
    }
};

// Rows of 64 columns, 128-byte swizzle (W, x, V).
__device__ __forceinline__ StepDesc row_step_desc() {
    StepDesc d;
    d.fixed = sm100::smem_desc(0, 16, 1024, sm100::kSwizzle128B);
#pragma unroll
    for (int k = 0; k < 4; ++k) d.off[k] = 2u * k;
    return d;
}

// A step of the stacked B as load_b_step leaves it.
__device__ __forceinline__ StepDesc b_step_desc(const TcLinear& L, uint32_t nrow) {
    using namespace sm100;
    StepDesc d;
    const uint32_t rp = (uint32_t)L.rp;
    d.fixed = !L.b_swizzled ? smem_desc(0, 16u * nrow, 128, kSwizzleNone)
                            : smem_desc(0, 16, 16u * rp,
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

// Eight consecutive rows of the stacked A (from c, a multiple of 8) for token
// t: V = gate * (x A^T) as bf16 terms, the first the value rounded, the second
// what that rounding left.  A token that did not choose the expert gets exact
// zeros, whatever its x holds.
__device__ __forceinline__ void finish_down8(const TcLinear& L, int64_t t, int c, const float (&u)[8],
                                             int& bad) {
    const LinearParams& p = L.p;
    const int64_t width = (int64_t)p.E * L.rp;
    const int64_t plane = p.T * width;
    int last = -1;
    float g = 0.f;
    for (int i = 0; i < 8; ++i) {
        if (c + i >= L.rows) break;
        const int e = (c + i) / p.r, k = (c + i) % p.r;
        if (e != last) {
            g = gate_of(p, t, e, bad);
            last = e;
        }
        const float val = g != 0.f ? g * u[i] : 0.f;
        const __nv_bfloat16 hi = __float2bfloat16_rn(val);
        uint16_t* dst = L.v + t * width + (int64_t)e * L.rp + k;
        dst[0] = __bfloat16_as_ushort(hi);
        if (L.terms == 2) dst[plane] = __bfloat16_as_ushort(__float2bfloat16_rn(val - __bfloat162float(hi)));
        if (k == p.r - 1)
            for (int z = 1; z <= L.rp - p.r; ++z) {
                dst[z] = 0;
                if (L.terms == 2) dst[plane + z] = 0;
            }
    }
}

template <int TN>
struct SkinnyConfig {
    static_assert(TN == 16 || TN == 32 || TN == 64 || TN == 128, "TN");
    static constexpr uint32_t kWBytes = 128 * 128;          // 128 rows x 64 columns bf16
    static constexpr uint32_t kXBytes = TN * 128;
    static constexpr uint32_t kStageBytes = kWBytes + kXBytes;
    // two CTAs an SM: at most 113 KB each
    static constexpr int kStages = TN <= 32 ? 5 : TN == 64 ? 4 : 3;
    static constexpr int kAccs = TN == 128 ? 2 : TN == 64 ? 4 : 8;   // TMEM accumulators
    static constexpr uint32_t kTmemCols = kAccs * TN;                // 128 or 256
    static constexpr uint32_t kRingBytes = kStages * kStageBytes;
    static constexpr uint32_t kSmemBytes = 1024 + kRingBytes + 8 * (2 * kStages + 1) + 16;
    static_assert(TN * 128 * 4 <= kRingBytes, "the partial tile reuses the ring");
    static_assert(kStageBytes % 1024 == 0, "swizzle atoms stay aligned");
};

template <int TN, int MODE>
__global__ void __launch_bounds__(kSkinnyThreads, 2)
linear_skinny_kernel(const __grid_constant__ TcLinear L, const __grid_constant__ CUtensorMap map_w,
                     const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_b,
                     const __grid_constant__ CUtensorMap map_v, const int S) {
    using C = SkinnyConfig<TN>;
    using namespace sm100;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + C::kRingBytes);
    uint64_t* empty = full + C::kStages;
    uint64_t* acc_full = empty + C::kStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (MODE == kDown) pdl_launch_dependents();
    const int q = (int)(blockIdx.x % (unsigned)S);
    const int64_t tile = blockIdx.x / (unsigned)S;
    const int row0 = (int)(tile / L.tok_tiles) * 128;
    const int64_t tok0 = (tile % L.tok_tiles) * TN;
    const int nsteps = L.xsteps + L.vsteps;
    const int k0 = (int)((int64_t)q * nsteps / S), k1 = (int)((int64_t)(q + 1) * nsteps / S);
    const int n = k1 - k0;
    const int naccs = n < C::kAccs ? n : C::kAccs;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&full[i], 2);     // one arrival, with its bytes, from each loading warp
            mbar_init(&empty[i], 1);
        }
        mbar_init(acc_full, 1);
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
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(L.p.status, ADAFUSE_STATUS_TIMEOUT);
    };

    if (warp == 4 || warp == 6) {
        // two warps, since one thread's TMA operations start about 120 clocks
        // apart: x and V (warp 4), W and B (warp 6)
        if (lane == 0) {
            const bool left = warp == 4;
            bool waited = false;
            int st = 0;
            uint32_t ph = 0;
#pragma unroll 1
            for (int i = k0; i < k1; ++i) {
                if (!wait_phase(&empty[st], ph ^ 1, abort_flag)) { fail(); break; }
                uint8_t* dst = ring + (size_t)st * C::kStageBytes + (left ? C::kWBytes : 0u);
                uint64_t* bar = &full[st];
                const int vi = i - L.xsteps;
                if (left && vi >= 0 && !waited) {
                    pdl_wait();   // V is written by the launch before
                    waited = true;
                }
                mbar_arrive_expect_tx(bar, left ? C::kXBytes : C::kWBytes);
                if (vi < 0) {
                    if (left)
                        tma_load_2d(dst, &map_x, i * 64, (int)tok0, bar);
                    else
                        tma_load_2d(dst, &map_w, i * 64, row0, bar);
                } else if (left) {
                    tma_load_3d(dst, &map_v, (vi % L.bsteps) * 64, (int)tok0, vi / L.bsteps, bar);
                } else {
                    load_b_step(L, vi % L.bsteps, row0, 128, dst,
                                [&](void* d, int a, int b, int c) { tma_load_3d(d, &map_b, a, b, c, bar); },
                                [&](void* d, int a, int b, int c, int e) {
                                    tma_load_4d(d, &map_b, a, b, c, e, bar);
                                });
                }
                if (++st == C::kStages) { st = 0; ph ^= 1; }
            }
        }
        __syncwarp();
    } else if (warp == 5) {
        // the whole warp walks the steps, so that descriptors are warp-uniform,
        // and one elected lane issues
        constexpr uint32_t idesc = instr_desc_bf16(128, TN, 0);
        const StepDesc rows = row_step_desc(), stacked = b_step_desc(L, 128);
        const uint32_t ring_s = smem_u32(ring);
        int st = 0, acc = -1, next = 0;   // accumulator acc takes the steps before `next`
        uint32_t ph = 0;
        bool ok = true;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            ok = __all_sync(0xffffffffu, wait_phase(&full[st], ph, abort_flag));
            if (!ok) break;
            const bool first = i == next;
            if (first) {
                ++acc;
                next = (acc + 1) * n / naccs;
            }
            const uint32_t w_s = ring_s + (uint32_t)st * C::kStageBytes, x_s = w_s + C::kWBytes;
            const uint32_t d = tmem + (uint32_t)(acc * TN);
            if (elect_one()) {
                if (k0 + i < L.xsteps) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_f16(d, rows.at(w_s, k), rows.at(x_s, k), idesc, !(first && k == 0));
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_f16(d, stacked.at(w_s, k), rows.at(x_s, k), idesc, !(first && k == 0));
                }
                tc_commit(&empty[st]);
                if (i == n - 1) tc_commit(acc_full);
            }
            __syncwarp();
            if (++st == C::kStages) { st = 0; ph ^= 1; }
        }
        if (!ok) fail();
    }

    // ---- the CTA's partial tile into shared memory: part[token][128 rows]
    float* part = reinterpret_cast<float*>(ring);
    if (warp < 4) {
        const bool ok = wait_phase(acc_full, 0, abort_flag, 4 * kWaitClocks);
        if (__all_sync(0xffffffffu, ok)) {
            tc_fence_after();
            const uint32_t t_lane = tmem + ((uint32_t)(warp * 32) << 16);
            constexpr int kCols = TN < 32 ? 16 : 32;
#pragma unroll 1
            for (int c0 = 0; c0 < TN; c0 += kCols) {
                float v[32];
                if constexpr (TN == 16) {
                    // two accumulators at a time: 32 columns
                    float s16[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) s16[i] = 0.f;
#pragma unroll 1
                    for (int a = 0; a < naccs; a += 2) {
                        tmem_ld32(t_lane + (uint32_t)(a * 16), v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) s16[i] += v[i];
                        if (a + 1 < naccs) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) s16[i] += v[16 + i];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) part[i * 128 + warp * 32 + lane] = s16[i];
                } else {
                    float sum[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[i] = 0.f;
#pragma unroll 1
                    for (int a = 0; a < naccs; ++a) {
                        tmem_ld32(t_lane + (uint32_t)(a * TN + c0), v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) sum[i] += v[i];
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) part[(c0 + i) * 128 + warp * 32 + lane] = sum[i];
                }
            }
            tc_fence_before();
        } else {
            fail();
        }
    }
    __syncthreads();
    if (S > 1) cluster_sync();

    // ---- this CTA's slice of the tile: sum over the cluster, epilogue, store
    if (!*abort_flag) {
        const int ntok = (int)(L.p.T - tok0 < TN ? L.p.T - tok0 : TN);
        const int nrow = L.rows - row0 < 128 ? L.rows - row0 : 128;
        const int groups = ntok * 16;
        const int g0 = (int)((int64_t)q * groups / S), g1 = (int)((int64_t)(q + 1) * groups / S);
        const uint32_t part_s = smem_u32(part);
        int bad = 0;
#pragma unroll 1
        for (int gi = g0 + (int)threadIdx.x; gi < g1; gi += kSkinnyThreads) {
            const int tok = gi >> 4, r8 = (gi & 15) * 8;
            if (r8 >= nrow) continue;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
            const uint32_t off = part_s + (uint32_t)(tok * 128 + r8) * 4u;
            for (int c = 0; c < S; ++c) {
                uint32_t a = off;
                if (S > 1) asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(off), "r"(c));
                const float4 lo = ld_cluster_f4(a), hi = ld_cluster_f4(a + 16);
                v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
                v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
            }
            if constexpr (MODE == kDown)
                finish_down8(L, tok0 + tok, row0 + r8, v, bad);
            else
                finish_cols<8>(L.p, tok0 + tok, row0 + r8, v);
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
pad_b_kernel(const uint16_t* __restrict__ B, uint16_t* __restrict__ dst, int64_t nrows, int r, int rp) {
    const int64_t total = nrows * rp;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / rp;
        const int k = (int)(i % rp);
        dst[i] = k < r ? __ldg(B + row * r + k) : (uint16_t)0;
    }
}

}  // namespace adafuse
