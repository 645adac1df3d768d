// linear_stream.cuh -- products of a weight with at most 8 tokens: the weight
// streamed once from memory past the tensor cores.
//
// Persistent CTAs of 16 warps take units of 16 rows of W; the warps (and, where
// there are few rows, the CTAs of a cluster) share a unit's columns in
// 64-column steps.  For a step a lane loads 32 bytes (one 256-bit load) of row
// lane / 4 and of row lane / 4 + 8 at column 16 * (lane % 4): whole 128-byte
// lines per row.  With the contraction index permuted the same way on both
// sides, those and the same columns of one token's x are the A and B fragments
// of four mma.m16n8k16 as they stand, so W goes from memory through registers
// to the tensor cores.  A warp's next kStreamDepth steps, the next unit's
// included, are requested as soon as the last ones are consumed.  x stays in L1.
// (Every operand comes by plain loads, in this file and the others: a launch set up
// while the one before it still writes must not read its output as constant data.)
//
// Every sum is fp32; the partial sums of the warps and of the cluster's CTAs
// are added in a fixed order.
//
// Routed products: the launch before this one (MODE kDown, on the stacked A)
// leaves u = x A^T in fp32 for the experts some token chose; the epilogue adds
// s * gate * (B u) for each token's own slots, in fp32.
#pragma once

#include "linear_common.cuh"
#include "sm100_ptx.cuh"

namespace adafuse {

enum : int { kProduct = 0, kDown = 1, kRouted = 2 };

using sm100::pdl_launch_dependents;
using sm100::pdl_wait;

constexpr int kStreamWarps = 16;
constexpr int kStreamThreads = 32 * kStreamWarps;
constexpr int kStreamRows = 16;
// As many tokens as an MMA has columns.  4096 -> 11008: T = 1 15.9 us, T = 8 18.7;
// on the tensor-core kernel for more tokens 20.0 and 19.5.
constexpr int kStreamMaxTokens = 8;
// Steps in flight per warp, 2 KB each (T = 1, 4096 -> 11008: 16.8, 16.2 and 24.8 us
// for one, two and three, which spill 0, 12 and 112 bytes a thread there).
constexpr int kStreamDepth = 2;

// 16 consecutive bf16 of a row (n = 16, 8 or 0 of them inside it), read past L1.
// WIDE: p is 32-byte aligned and n is 16 or 0.
template <bool WIDE>
__device__ __forceinline__ void ldg_stream16(const uint16_t* p, int n, uint32_t (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0u;
    if constexpr (WIDE) {
        if (n > 0)
            asm volatile("ld.global.L1::no_allocate.L2::256B.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                           "=r"(v[6]), "=r"(v[7])
                         : "l"(p));
    } else {
        if (n > 0)
            asm volatile("ld.global.L1::no_allocate.L2::256B.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "l"(p));
        if (n > 8)
            asm volatile("ld.global.L1::no_allocate.L2::256B.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                         : "l"(p + 8));
    }
}

__device__ __forceinline__ void mma_bf16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One token's used slots as the epilogue reads them.
struct StreamSlots {
    int e[kStreamMaxTokens * ADAFUSE_MAX_ROUTE_SLOTS];     // -1: empty or bad
    float g[kStreamMaxTokens * ADAFUSE_MAX_ROUTE_SLOTS];   // s * gate
};

// Sum over token t's slots of s * gate * (B_e[o] . u[t][e]).
__device__ __forceinline__ float adapters_of(const LinearParams& p, const StreamSlots& sl, const float* u,
                                             int t, int o) {
    float v = 0.f;
    for (int j = 0; j < p.slots; ++j) {
        const int e = sl.e[t * p.slots + j];
        if (e < 0) continue;
        const uint16_t* b = p.B + ((int64_t)e * p.out + o) * p.r;
        const float* ue = u + (int64_t)(t * p.E + e) * p.r;
        float d = 0.f;
        if ((p.r & 7) == 0) {
#pragma unroll 1
            for (int k = 0; k < p.r; k += 8) {
                const uint4 w = *reinterpret_cast<const uint4*>(b + k);
                const float4 u0 = __ldcg(reinterpret_cast<const float4*>(ue + k));
                const float4 u1 = __ldcg(reinterpret_cast<const float4*>(ue + k + 4));
                d = fmaf(__uint_as_float(w.x << 16), u0.x, d);
                d = fmaf(__uint_as_float(w.x & 0xffff0000u), u0.y, d);
                d = fmaf(__uint_as_float(w.y << 16), u0.z, d);
                d = fmaf(__uint_as_float(w.y & 0xffff0000u), u0.w, d);
                d = fmaf(__uint_as_float(w.z << 16), u1.x, d);
                d = fmaf(__uint_as_float(w.z & 0xffff0000u), u1.y, d);
                d = fmaf(__uint_as_float(w.w << 16), u1.z, d);
                d = fmaf(__uint_as_float(w.w & 0xffff0000u), u1.w, d);
            }
        } else {
            for (int k = 0; k < p.r; ++k) d = fmaf(bf16_bits_to_float(b[k]), __ldcg(ue + k), d);
        }
        v = fmaf(sl.g[t * p.slots + j], d, v);
    }
    return v;
}

// rows: of W (kProduct, kRouted: out; kDown: the stacked A's E * r).  u: [T][E * r].
// S > 1: the cluster's CTAs share one unit and the grid covers all units.
template <int MODE, bool WIDE>
__global__ void __launch_bounds__(kStreamThreads, 2)
linear_stream_kernel(const LinearParams p, const uint16_t* __restrict__ W, const int rows,
                     float* __restrict__ u, const int S) {
    __shared__ __align__(16) float part[2][kStreamWarps][kStreamRows * 8];
    __shared__ __align__(16) float total[kStreamRows * 8];   // [token][16 rows], S > 1
    __shared__ unsigned long long used_s;
    __shared__ StreamSlots slots_s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q = (int)(blockIdx.x % (unsigned)S);
    const int part_no = (int)(blockIdx.x / (unsigned)S), parts = (int)(gridDim.x / (unsigned)S);
    // this CTA's rows: an even share, cut into even units of at most 16 (lanes
    // of missing rows load nothing), so every SM moves the same bytes
    const int row_begin = (int)((int64_t)rows * part_no / parts);
    const int row_end = (int)((int64_t)rows * (part_no + 1) / parts);
    const int units = (row_end - row_begin + kStreamRows - 1) / kStreamRows;
    const int height = units > 0 ? (row_end - row_begin + units - 1) / units : kStreamRows;
    const int T = (int)p.T;

    // A routed product starts while the kDown launch before it runs: its x and W
    // were complete before that launch let it start, and u is waited for below.
    if constexpr (MODE != kRouted) pdl_wait();
    pdl_launch_dependents();
    if constexpr (MODE == kDown) {
        // experts that some token chose; a unit of rows none of them owns is
        // neither read nor written
        if (threadIdx.x == 0) used_s = 0;
        __syncthreads();
        int bad = 0;
        for (int i = threadIdx.x; i < T * p.slots; i += kStreamThreads) {
            int e;
            float g;
            if (route_slot(p.routes, p.slots, p.E, i / p.slots, i % p.slots, e, g, bad))
                atomicOr(&used_s, 1ull << e);
        }
        if (bad != 0 && blockIdx.x == 0) atomicOr(p.status, bad);
        __syncthreads();
    }
    // the first unit at or after `row` of this CTA that has work
    auto next_unit = [&](int row) {
        if constexpr (MODE == kDown) {
            for (; row < row_end; row += height) {
                const int e0 = row / p.r, e1 = (min(row + height, row_end) - 1) / p.r;
                if (used_s & (((1ull << (e1 - e0 + 1)) - 1) << e0)) break;   // e1 - e0 < 16
            }
        }
        return row;
    };

    const int g = lane >> 2, c16 = (lane & 3) * 16;
    const bool tok = g < T;
    const uint16_t* xt = p.x + (tok ? g : 0) * p.ldx + c16;
    const int step = 64 * kStreamWarps * S;              // columns between a warp's steps
    const int k_first = 64 * (q * kStreamWarps + warp);

    // loads run one batch of steps ahead of the arithmetic
    uint32_t a[kStreamDepth][8], b[kStreamDepth][8];
    int lrow = next_unit(row_begin), lk = k_first;
    auto load_batch = [&]() {
        if (lrow >= row_end || lk >= p.in) return;
        const uint16_t* w = W + (int64_t)(lrow + g) * p.in + c16;
        const int valid = min(height, row_end - lrow);
        const int na = g < valid ? p.in - c16 : 0, nb = g + 8 < valid ? p.in - c16 : 0;
#pragma unroll
        for (int d = 0; d < kStreamDepth; ++d) {
            const int k = lk + d * step;
            ldg_stream16<WIDE>(w + k, na - k, a[d]);
            ldg_stream16<WIDE>(w + k + 8 * (int64_t)p.in, nb - k, b[d]);
        }
        lk += step * kStreamDepth;
        if (lk >= p.in) {
            lk = k_first;
            lrow = next_unit(lrow + height);
        }
    };
    load_batch();

    if constexpr (MODE == kRouted) {
        if ((int)threadIdx.x < T * p.slots) {
            int e, bad = 0;   // bad slots are reported by the launch that writes u
            float gate;
            const bool used = route_slot(p.routes, p.slots, p.E, threadIdx.x / p.slots,
                                         threadIdx.x % p.slots, e, gate, bad);
            slots_s.e[threadIdx.x] = used ? e : -1;
            slots_s.g[threadIdx.x] = p.s * gate;
        }
    }

    bool waited = MODE != kRouted;
    int buf = 0;
    const int n_out = T * kStreamRows;
#pragma unroll 1
    for (int row0 = next_unit(row_begin); row0 < row_end; row0 = next_unit(row0 + height), buf ^= 1) {
        const int unit_end = min(row0 + height, row_end);
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
        for (int k0 = k_first; k0 < p.in; k0 += step * kStreamDepth) {
#pragma unroll
            for (int d = 0; d < kStreamDepth; ++d) {
                const int k = k0 + d * step, n = p.in - c16 - k;
                const uint4 x0 = tok && n > 0 ? *reinterpret_cast<const uint4*>(xt + k) : zero;
                const uint4 x1 = tok && n > 8 ? *reinterpret_cast<const uint4*>(xt + k + 8) : zero;
                mma_bf16_16816(acc, a[d][0], b[d][0], a[d][1], b[d][1], x0.x, x0.y);
                mma_bf16_16816(acc, a[d][2], b[d][2], a[d][3], b[d][3], x0.z, x0.w);
                mma_bf16_16816(acc, a[d][4], b[d][4], a[d][5], b[d][5], x1.x, x1.y);
                mma_bf16_16816(acc, a[d][6], b[d][6], a[d][7], b[d][7], x1.z, x1.w);
            }
            load_batch();
        }
        // part[warp][token][16 rows]
        float* mine = part[buf][warp];
        const int t2 = 2 * (lane & 3);
        mine[t2 * kStreamRows + g] = acc[0];
        mine[(t2 + 1) * kStreamRows + g] = acc[1];
        mine[t2 * kStreamRows + g + 8] = acc[2];
        mine[(t2 + 1) * kStreamRows + g + 8] = acc[3];
        __syncthreads();
        float v = 0.f;
        if ((int)threadIdx.x < n_out) {
#pragma unroll
            for (int w = 0; w < kStreamWarps; ++w) v += part[buf][w][threadIdx.x];
        }
        int i = threadIdx.x;
        bool mine_to_store = i < n_out;
        if (S > 1) {
            if (i < n_out) total[i] = v;
            sm100::cluster_sync();
            const int i0 = q * n_out / S, i1 = (q + 1) * n_out / S;
            i = i0 + (int)threadIdx.x;
            mine_to_store = i < i1;
            if (mine_to_store) {
                v = 0.f;
                for (int c = 0; c < S; ++c) {
                    float f;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(f)
                                 : "r"(sm100::cluster_addr(&total[i], (uint32_t)c)));
                    v += f;
                }
            }
        }
        if (!waited) {
            pdl_wait();   // u is written by the launch before
            waited = true;
        }
        const int t = i / kStreamRows, o = row0 + i % kStreamRows;
        if (mine_to_store && o < unit_end) {
            if constexpr (MODE == kDown) {
                u[(int64_t)t * rows + o] = v;
            } else {
                if constexpr (MODE == kRouted) v += adapters_of(p, slots_s, u, t, o);
                store_one(p, t, o, v);
            }
        }
    }
    if (S > 1) sm100::cluster_sync();   // peers may still read this CTA's sums
}

}  // namespace adafuse
