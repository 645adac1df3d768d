// linear_pair.cuh -- products of a weight with many tokens, bound by the tensor
// cores: CTA pairs (tcgen05 cta_group::2) on tiles of 256 tokens x BN columns.
//
//   D[256 tokens, BN out columns] = x tile x (W tile)^T, fp32 in TMEM
//
// Each CTA of a pair holds 128 tokens of the tile: it stages 128 x 64 of x and
// BN/2 x 64 of W per step (the MMA reads both halves of W), so a step moves half
// of what two single CTAs would.  Two accumulators in TMEM: the epilogue warps
// of both CTAs empty one while the tensor cores fill the other.  Persistent
// pairs take tiles with the token tiles of a W tile next to each other, so W
// comes from memory once and x stays in L2.
//
// CHUNKED (fp32 outputs): tensor-core accumulators drop low bits on every
// 16-deep step (measured: 4e-6 of the result after 4096 products, 1.2e-5 after
// 11008), so the contraction is cut into chunks of kChunkSteps steps, each
// started from zero, and the epilogue adds them in registers in fp32.  A bf16
// output does not see the difference and takes one chunk.
//
// Routed products: after x and W come V and the stacked B, as in
// linear_skinny.cuh.
//
// Warps: 0 and 2 loads, 1 MMA (even CTA) and TMEM, 4..11 epilogue (token = 32 *
// (warp % 4) + lane, half of the columns each four warps).
#pragma once

#include <cuda.h>

#include "linear_skinny.cuh"

namespace adafuse {

constexpr int kPairThreads = 384;
constexpr int kPairEpiWarps = 8;
constexpr int kPairTokens = 256;
constexpr int kChunkSteps = 16;

template <int BN>
struct PairConfig {
    static_assert(BN == 128 || BN == 256, "BN");
    static constexpr uint32_t kXBytes = 128 * 128;
    static constexpr uint32_t kWBytes = (BN / 2) * 128;
    static constexpr uint32_t kStageBytes = kXBytes + kWBytes;
    static constexpr int kStages = BN == 256 ? 6 : 8;
    static constexpr uint32_t kTmemCols = 2 * BN;
    static constexpr uint32_t kSmemBytes = 1024 + kStages * kStageBytes + 8 * (2 * kStages + 4) + 16;
    static_assert(kSmemBytes <= 232448, "shared memory");
};

template <int BN, bool CHUNKED>
__global__ void __launch_bounds__(kPairThreads, 1)
linear_pair_kernel(const __grid_constant__ TcLinear L, const __grid_constant__ CUtensorMap map_w,
                   const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_v) {
    using C = PairConfig<BN>;
    using namespace sm100;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // the same offsets in both CTAs: MMA descriptors name one address for both
    uint8_t* ring = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + C::kStages * C::kStageBytes);   // even CTA's used
    uint64_t* empty = full + C::kStages;
    uint64_t* acc_full = empty + C::kStages;    // [2]
    uint64_t* acc_empty = acc_full + 2;         // [2], even CTA's used
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t q = cluster_ctarank();
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&full[i], 4);     // one arrival, with its bytes, from each loading warp
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 2 * kPairEpiWarps);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, C::kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t peer_abort = cluster_addr((const void*)abort_flag, q ^ 1u);
    auto fail = [&]() {
        if (!*abort_flag) {
            *abort_flag = 1;
            st_cluster_u32(peer_abort, 1u);
            atomicOr(L.p.status, ADAFUSE_STATUS_TIMEOUT);
        }
    };

    const int nsteps = L.xsteps + L.vsteps;
    const int col_tiles = (L.p.out + BN - 1) / BN;
    const int64_t tiles = (int64_t)L.tok_tiles * col_tiles;
    const int64_t t_first = cluster_id_x(), t_stride = cluster_count_x();

    if (warp == 0 || warp == 2) {
        // two warps, since one thread's TMA operations start about 120 clocks
        // apart: x and V (warp 0), W and B (warp 2)
        if (lane == 0) {
            const bool left = warp == 0;
            const uint32_t bytes = left ? C::kXBytes : C::kWBytes;
            const uint32_t full0 = cluster_addr(full, 0);
            bool waited = false, ok = true;
            int st = 0;
            uint32_t ph = 0;
            for (int64_t t = t_first; ok && t < tiles; t += t_stride) {
                const int tok0 = (int)(t % L.tok_tiles) * kPairTokens + (int)q * 128;
                const int row0 = (int)(t / L.tok_tiles) * BN + (int)q * (BN / 2);
#pragma unroll 1
                for (int i = 0; i < nsteps; ++i) {
                    if (!wait_phase(&empty[st], ph ^ 1, abort_flag)) { ok = false; break; }
                    uint8_t* dst = ring + (size_t)st * C::kStageBytes + (left ? 0u : C::kXBytes);
                    const uint32_t bar = full0 + 8u * (uint32_t)st;
                    const int vi = i - L.xsteps;
                    if (left && vi >= 0 && !waited) {
                        pdl_wait();   // V is written by the launch before
                        waited = true;
                    }
                    mbar_arrive_expect_tx_cluster(bar, bytes);
                    if (vi < 0) {
                        if (left)
                            tma_load_2d_pair(dst, &map_x, i * 64, tok0, bar);
                        else
                            tma_load_2d_pair(dst, &map_w, i * 64, row0, bar);
                    } else if (left) {
                        tma_load_3d_pair(dst, &map_v, (vi % L.bsteps) * 64, tok0, vi / L.bsteps, bar);
                    } else {
                        load_b_step(L, vi % L.bsteps, row0, BN / 2, dst,
                                    [&](void* d, int a, int b, int c) { tma_load_3d_pair(d, &map_b, a, b, c, bar); },
                                    [&](void* d, int a, int b, int c, int e) {
                                        tma_load_4d_pair(d, &map_b, a, b, c, e, bar);
                                    });
                    }
                    if (++st == C::kStages) { st = 0; ph ^= 1; }
                }
            }
            if (!ok) fail();
            // every stage filled here is released by an MMA completion that
            // arrives on this CTA's barrier: see the last ones land
            for (int j = 0; ok && !*abort_flag && j < C::kStages; ++j) {
                if (!wait_phase(&empty[st], ph ^ 1, abort_flag)) { fail(); break; }
                if (++st == C::kStages) { st = 0; ph ^= 1; }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // the whole warp walks the steps, so that descriptors are warp-uniform,
        // and one elected lane issues
        if (q == 0) {
            constexpr uint32_t idesc = instr_desc_bf16(kPairTokens, BN, 0);
            const StepDesc rows = row_step_desc(), stacked = b_step_desc(L, BN / 2);
            const uint32_t ring_s = smem_u32(ring);
            int st = 0, buf = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true;
            for (int64_t t = t_first; ok && t < tiles; t += t_stride) {
#pragma unroll 1
                for (int i = 0; i < nsteps; ++i) {
                    const bool begins = CHUNKED ? i % kChunkSteps == 0 : i == 0;
                    const bool ends = i == nsteps - 1 || (CHUNKED && i % kChunkSteps == kChunkSteps - 1);
                    if (begins) {
                        ok = __all_sync(0xffffffffu, wait_phase(&acc_empty[buf], aph ^ 1, abort_flag));
                        if (!ok) break;
                        tc_fence_after();
                    }
                    ok = __all_sync(0xffffffffu, wait_phase(&full[st], ph, abort_flag));
                    if (!ok) break;
                    const uint32_t x_s = ring_s + (uint32_t)st * C::kStageBytes, w_s = x_s + C::kXBytes;
                    const uint32_t d = tmem + (uint32_t)(buf * BN);
                    if (elect_one()) {
                        if (i < L.xsteps) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc_mma_f16_pair(d, rows.at(x_s, k), rows.at(w_s, k), idesc, !(begins && k == 0));
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc_mma_f16_pair(d, rows.at(x_s, k), stacked.at(w_s, k), idesc,
                                                !(begins && k == 0));
                        }
                        tc_commit_pair(&empty[st], 0x3);
                        if (ends) tc_commit_pair(&acc_full[buf], 0x3);
                    }
                    __syncwarp();
                    if (++st == C::kStages) { st = 0; ph ^= 1; }
                    if (ends) {
                        buf ^= 1;
                        if (buf == 0) aph ^= 1;
                    }
                }
            }
            if (!ok) fail();
        }
    } else if (warp >= 4) {
        const int half = (warp - 4) >> 2;                 // which BN/2 columns
        const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(half * (BN / 2));
        const uint32_t acc_empty0 = cluster_addr(acc_empty, 0);
        const int chunks = CHUNKED ? (nsteps + kChunkSteps - 1) / kChunkSteps : 1;
        int buf = 0;
        uint32_t aph = 0;
        bool ok = true;
        for (int64_t t = t_first; ok && t < tiles; t += t_stride) {
            const int64_t tok = (t % L.tok_tiles) * kPairTokens + q * 128 + (warp & 3) * 32 + lane;
            const int col0 = (int)(t / L.tok_tiles) * BN + half * (BN / 2);
            const bool mine = tok < L.p.T;
            float acc[CHUNKED ? BN / 2 : 1];   // sum of the finished chunks
            if constexpr (CHUNKED) {
#pragma unroll
                for (int i = 0; i < BN / 2; ++i) acc[i] = 0.f;
            }
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                ok = wait_phase(&acc_full[buf], aph, abort_flag, 4 * kWaitClocks);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                const uint32_t src = t_lane + (uint32_t)(buf * BN);
                const bool last = c == chunks - 1;
                if constexpr (CHUNKED) {
                    // add the chunk; the finished sums go back to TMEM, from
                    // where one short loop takes them
#pragma unroll
                    for (int b = 0; b < BN / 64; ++b) {
                        float v[32];
                        tmem_ld32(src + 32u * b, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) acc[32 * b + i] += v[i];
                        if (last && chunks > 1) tmem_st32(src + 32u * b, &acc[32 * b]);
                    }
                    tmem_wait_st();
                }
                if (last) {
#pragma unroll 1
                    for (int b = 0; b < BN / 64; ++b) {
                        float v[32];
                        tmem_ld32(src + 32u * b, v);
                        tmem_wait_ld();
                        if (mine) finish_cols<32>(L.p, tok, col0 + 32 * b, v);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(acc_empty0 + 8u * (uint32_t)buf);
                buf ^= 1;
                if (buf == 0) aph ^= 1;
            }
            if (!ok) { fail(); break; }
        }
    }

    // teardown: after an abort copies and MMAs in flight get time to land;
    // neither CTA leaves while the other may still touch its shared memory
    __syncwarp();
    __syncthreads();
    if (*abort_flag) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 200000ull) { }
    }
    tc_fence_before();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, C::kTmemCols);
    }
}

}  // namespace adafuse
