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
// comes from memory once and x stays in L2.  BN is a launch parameter (a
// multiple of 16): the host takes the width whose tiles fill whole rounds.
//
// F32 (fp32 outputs, V of two terms): tensor-core accumulators drop low bits on
// every 16-deep piece (1e-6 of the result after 64, more in proportion; 4e-6 where
// all products have one sign), so the contraction is cut into chunks of at most
// kChunkSteps steps, each started from zero, and the epilogue adds them in
// registers in fp32.  7e-7 of the result is left; chunks of 24 steps left 1.4e-6
// and took 301 instead of 308 us for T = 4096, 11008 -> 4096 with 8 experts of rank
// 8.  A bf16 output, rounded at 2^-9 of itself, takes one chunk: at 4096 columns one
// in 400 values is rounded the other way, and the error's norm stays 0.00166.
//
// Routed products: after x and W come V and the stacked B, as in
// linear_skinny.cuh; kDown writes V (F32: as two terms).
//
// Warps: 0 and 2 loads, 1 MMA (even CTA) and TMEM, 4..19 epilogue (token = 32 *
// (warp % 4) + lane, every fourth 16-column block each four warps).
#pragma once

#include <cuda.h>

#include "linear_skinny.cuh"

namespace adafuse {

constexpr int kPairThreads = 640;
constexpr int kPairEpiWarps = 16;
constexpr int kPairTokens = 256;
constexpr int kPairMaxCols = 256;
constexpr int kChunkSteps = 12;
constexpr int kPairStages = 6;
constexpr uint32_t kPairXBytes = 128 * 128;
constexpr uint32_t kPairStageBytes = 2 * kPairXBytes;   // x, then up to 128 rows of W
constexpr uint32_t kTurnBytes = 32 * 16 * 4;              // per epilogue warp, see finish_block
constexpr uint32_t kPairSmemBytes =
    1024 + kPairStages * kPairStageBytes + kPairEpiWarps * kTurnBytes + 8 * (2 * kPairStages + 4) + 16;
static_assert(kPairSmemBytes <= 232448, "shared memory");

// kDown: a warp's 32 tokens x 16 columns of V (ranks that are multiples of 8, so
// V's columns are the stacked A's rows) from the finished x A^T, turned as in
// finish_block: 2 lanes a token, 8 columns, twice 16 tokens.
__device__ __forceinline__ void finish_down_block(const TcLinear& L, int64_t tok0, int col0, int lane,
                                                  const float (&v)[16], uint8_t* turn, int& bad) {
    auto piece = [&](int row, int c) { return turn + row * 64 + ((c ^ (row >> 1 & 3)) << 4); };
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<float4*>(piece(lane, c)) = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    __syncwarp();
    const int col = col0 + (lane & 1) * 8;
    const int e = col / L.p.r;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int row = (lane >> 1) + 16 * j;
        const float4 a = *reinterpret_cast<const float4*>(piece(row, (lane & 1) * 2));
        const float4 b = *reinterpret_cast<const float4*>(piece(row, (lane & 1) * 2 + 1));
        const float u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (tok0 + row < L.p.T && col < L.rows) finish_down8(L, tok0 + row, e, col - e * L.p.r, u, bad);
    }
    __syncwarp();
}

template <bool F32, int MODE>
__global__ void __launch_bounds__(kPairThreads, 1)
linear_pair_kernel(const __grid_constant__ TcLinear L, const __grid_constant__ CUtensorMap map_w,
                   const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_v, const int BN) {
    using namespace sm100;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // the same offsets in both CTAs: MMA descriptors name one address for both
    uint8_t* ring = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* turns = ring + kPairStages * kPairStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(turns + kPairEpiWarps * kTurnBytes);   // even CTA's used
    uint64_t* empty = full + kPairStages;
    uint64_t* acc_full = empty + kPairStages;    // [2]
    uint64_t* acc_empty = acc_full + 2;         // [2], even CTA's used
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t q = cluster_ctarank();
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kPairStages; ++i) {
            // one arrival, with its bytes, from each loading warp
            mbar_init(&full[i], i == 0 && L.stall && blockIdx.x == 0 ? 5 : 4);
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
        tmem_alloc_pair(tmem_slot, 2 * kPairMaxCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (MODE == kDown || L.vsteps == 0) pdl_wait();   // as in the skinny kernel
    pdl_launch_dependents();
    const uint32_t peer_abort = cluster_addr((const void*)abort_flag, q ^ 1u);
    auto fail = [&]() {
        if (!*abort_flag) {
            *abort_flag = 1;
            st_cluster_u32(peer_abort, 1u);
            atomicOr(L.p.status, ADAFUSE_STATUS_TIMEOUT);
        }
    };

    const int nsteps = L.xsteps + L.vsteps;
    // even chunks of at most kChunkSteps
    const int chunks = F32 ? (nsteps + kChunkSteps - 1) / kChunkSteps : 1;
    const int chunk_steps = (nsteps + chunks - 1) / chunks;
    const int col_tiles = (L.rows + BN - 1) / BN;
    const int64_t tiles = (int64_t)L.tok_tiles * col_tiles;
    const int64_t t_first = cluster_id_x(), t_stride = cluster_count_x();

    if (warp == 0 || warp == 2) {
        // two loading warps: one thread's TMA operations start about 120 clocks apart
        const uint32_t ring_s = smem_u32(ring), full0 = cluster_addr(full, 0);
        bool waited = false, ok = true;
        int st = 0;
        uint32_t ph = 0;
        for (int64_t t = t_first; ok && t < tiles; t += t_stride) {
            const int tok0 = (int)(t % L.tok_tiles) * kPairTokens + (int)q * 128;
            const int row0 = (int)(t / L.tok_tiles) * BN + (int)q * (BN / 2);
            ok = warp == 0 ? load_steps<true, true>(L, &map_x, &map_v, 0, nsteps, tok0, 0, kPairXBytes, ring_s,
                                                    kPairStageBytes, smem_u32(empty), full0, kPairStages, st, ph, waited,
                                                    abort_flag)
                           : load_steps<true, false>(L, &map_w, &map_b, 0, nsteps, row0, BN / 2,
                                                     (uint32_t)BN * 64u, ring_s + kPairXBytes, kPairStageBytes,
                                                     smem_u32(empty), full0, kPairStages, st, ph, waited, abort_flag);
        }
        if (!ok) fail();
        // every stage filled here is released by an MMA completion that arrives
        // on this CTA's barrier: see the last ones land
        for (int j = 0; ok && j < kPairStages; ++j) {
            ok = wait_phase(smem_u32(&empty[st]), ph ^ 1, abort_flag);
            if (!ok) fail();
            if (++st == kPairStages) { st = 0; ph ^= 1; }
        }
        __syncwarp();
    } else if (warp == 1) {
        // as in the skinny kernel: the whole warp walks, an elected lane issues
        if (q == 0) {
            const uint32_t idesc = instr_desc_bf16(kPairTokens, BN, 0);
            const uint32_t ring_s = smem_u32(ring), full_s = smem_u32(full), empty_s = smem_u32(empty);
            const uint64_t dx = row_desc(ring_s), dw = row_desc(ring_s + kPairXBytes);
            const StepDesc db = b_desc(L, ring_s + kPairXBytes, BN / 2);
            int st = 0, buf = 0;
            uint32_t ph = 0, aph = 0, off = 0;   // off: the stage's offset in 16-byte units
            bool ok = true;
            auto next_stage = [&]() {
                __syncwarp();
                ++st;
                off += kPairStageBytes / 16;
                if (st == kPairStages) { st = 0; off = 0; ph ^= 1; }
            };
            for (int64_t t = t_first; ok && t < tiles; t += t_stride) {
#pragma unroll 1
                for (int c0 = 0; c0 < nsteps; c0 += chunk_steps) {
                    const int c1 = c0 + chunk_steps < nsteps ? c0 + chunk_steps : nsteps;
                    ok = wait_phase(smem_u32(&acc_empty[buf]), aph ^ 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + (uint32_t)(buf * kPairMaxCols);
                    const int cx = c1 < L.xsteps ? c1 : L.xsteps;
                    int i = c0;
#pragma unroll 1
                    for (; i < cx; ++i) {
                        ok = wait_phase(full_s + 8u * (uint32_t)st, ph, abort_flag);
                        if (!ok) break;
                        const uint64_t a = dx + off, b = dw + off;
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc_mma_f16_pair(d, a + 2 * k, b + 2 * k, idesc, i > c0 || k > 0);
                            tc_commit_pair_addr(empty_s + 8u * (uint32_t)st, 0x3);
                        }
                        next_stage();
                    }
#pragma unroll 1
                    for (; ok && i < c1; ++i) {
                        ok = wait_phase(full_s + 8u * (uint32_t)st, ph, abort_flag);
                        if (!ok) break;
                        const uint64_t a = dx + off, b = db.base + off;
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc_mma_f16_pair(d, a + 2 * k, b + db.off[k], idesc, i > c0 || k > 0);
                            tc_commit_pair_addr(empty_s + 8u * (uint32_t)st, 0x3);
                        }
                        next_stage();
                    }
                    if (!ok) break;
                    if (elect_one()) tc_commit_pair(&acc_full[buf], 0x3);
                    __syncwarp();
                    buf ^= 1;
                    if (buf == 0) aph ^= 1;
                }
            }
            if (!ok) fail();
        }
    } else if (warp >= 4) {
        const int group = (warp - 4) >> 2;
        uint8_t* turn = turns + (warp - 4) * kTurnBytes;
        const int blocks = BN / 16;                       // 16-column blocks: group, group + 4, ...
        const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t acc_empty0 = cluster_addr(acc_empty, 0);
        int buf = 0, bad = 0;
        uint32_t aph = 0;
        bool ok = true;
        for (int64_t t = t_first; ok && t < tiles; t += t_stride) {
            const int64_t tok0 = (t % L.tok_tiles) * kPairTokens + q * 128 + (warp & 3) * 32;
            const int col0 = (int)(t / L.tok_tiles) * BN;
            auto await_chunk = [&]() {
                ok = wait_phase(smem_u32(&acc_full[buf]), aph, abort_flag, 4 * kWaitClocks);
                tc_fence_after();
                return t_lane + (uint32_t)(buf * kPairMaxCols);
            };
            auto release_chunk = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(acc_empty0 + 8u * (uint32_t)buf);
                buf ^= 1;
                if (buf == 0) aph ^= 1;
            };
            uint32_t src = 0;
            if constexpr (F32) {
                // The chunks' sums in registers; with the last chunk they go
                // back to TMEM, from where the loop below takes them.  (Held in
                // registers through that loop they would spill, and with the
                // ring in shared memory L1 is too small for more than the 16
                // bytes a thread that are spilled as it is.)
                float acc[4][16];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[j][i] = 0.f;
#pragma unroll 1
                for (int c = 0; c < chunks; ++c) {
                    src = await_chunk();
                    if (!ok || chunks == 1) break;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int cb = group + 4 * j;
                        if (cb < blocks) {
#pragma unroll
                            for (int h = 0; h < 16; h += 8) {
                                float v[8];
                                tmem_ld8(src + 16u * cb + h, v);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 8; ++i) acc[j][h + i] += v[i];
                            }
                        }
                    }
                    if (c < chunks - 1) release_chunk();
                }
                if (ok && chunks > 1) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (group + 4 * j < blocks) tmem_st16(src + 16u * (group + 4 * j), acc[j]);
                    tmem_wait_st();
                }
            } else {
                src = await_chunk();
            }
            // V has landed, so the launch that wrote it is complete: did it give up?
            if (MODE == kProduct && ok && t == t_first && L.vsteps > 0)
                ok = (status_now(L.p) & ADAFUSE_STATUS_TIMEOUT) == 0;
            if (!ok) { fail(); break; }
#pragma unroll 1
            for (int cb = group; cb < blocks; cb += 4) {
                float v[16];
                if constexpr (MODE == kDown) {
                    tmem_ld16(src + 16u * cb, v);
                    tmem_wait_ld();
                    finish_down_block(L, tok0, col0 + 16 * cb, lane, v, turn, bad);
                } else {
                    BlockSide<F32> side;
                    load_block<F32>(L.p, tok0, col0 + 16 * cb, lane, side);
                    tmem_ld16(src + 16u * cb, v);
                    tmem_wait_ld();
                    finish_block<F32>(L.p, tok0, col0 + 16 * cb, lane, v, side, turn);
                }
            }
            release_chunk();
        }
        if (MODE == kDown && bad != 0) atomicOr(L.p.status, bad);
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
        tmem_dealloc_pair(tmem, 2 * kPairMaxCols);
    }
}

}  // namespace adafuse
