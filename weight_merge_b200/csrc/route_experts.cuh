// route_experts.cuh -- per-token routing to experts: softmax or sigmoid
// scores, a selection bias, groups of experts, top-k, renormalised gates.
#pragma once

#include <cuda_bf16.h>
#include <float.h>

#include "common.cuh"

namespace adafuse {

struct GateParams {
    int score, k, n_groups, top_groups, group_top, renorm;
    float scale;
    const float* bias;
    int E, slots;
};

constexpr int kMaxExperts = 64;

__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const double o = __shfl_xor_sync(0xffffffffu, v, off);
        v = o > v ? o : v;
    }
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// One token's decision by one warp, in 64 bits.  Lane l holds the logits of
// experts l (z0) and l + 32 (z1); scratch: kMaxExperts doubles of shared memory
// that belong to this warp.  Writes the record at route[t].
__device__ __forceinline__ void route_decide(double z0, double z1, const GateParams& g, int lane,
                                             double* scratch, int32_t* __restrict__ route,
                                             int64_t t) {
    const double kNone = -INFINITY;
    const bool in0 = lane < g.E, in1 = lane + 32 < g.E;
    int32_t* idx_out = route + t * 2 * g.slots;
    float* gate_out = reinterpret_cast<float*>(idx_out + g.slots);
    const bool fine = (!in0 || fabs(z0) <= (double)FLT_MAX) && (!in1 || fabs(z1) <= (double)FLT_MAX);
    if (!__all_sync(0xffffffffu, fine)) {
        if (lane < g.slots) { idx_out[lane] = -1; gate_out[lane] = 0.f; }
        return;
    }
    // scores: softmax over all E, or sigmoid (exp overflows to +inf for very
    // negative logits, and the score to 0)
    double s0 = 0.0, s1 = 0.0;
    if (g.score == ADAFUSE_SCORE_SOFTMAX) {
        const double m = warp_max(fmax(in0 ? z0 : kNone, in1 ? z1 : kNone));
        s0 = in0 ? exp(z0 - m) : 0.0;
        s1 = in1 ? exp(z1 - m) : 0.0;
        const double sum = warp_sum(s0 + s1);
        s0 /= sum;
        s1 /= sum;
    } else {
        if (in0) s0 = 1.0 / (1.0 + exp(-z0));
        if (in1) s1 = 1.0 / (1.0 + exp(-z1));
    }
    bool on0 = in0, on1 = in1;          // enabled experts
    double q0 = s0, q1 = s1;            // selection values
    double key0 = z0, key1 = z1;        // what picks are ordered by
    if (g.bias != nullptr) {
        if (in0) { const float b = __ldg(g.bias + lane); on0 = b > -INFINITY; q0 = s0 + (double)b; }
        if (in1) { const float b = __ldg(g.bias + lane + 32); on1 = b > -INFINITY; q1 = s1 + (double)b; }
        key0 = q0;
        key1 = q1;
    }
    if (g.n_groups > 1) {
        // worth of a group: the sum of its group_top highest enabled values
        const int per = g.E / g.n_groups;
        if (in0) scratch[lane] = on0 ? q0 : kNone;
        if (in1) scratch[lane + 32] = on1 ? q1 : kNone;
        __syncwarp();
        double w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int grp = lane + 32 * h;
            double a = kNone, b = kNone;   // highest, second highest
            if (grp < g.n_groups)
                for (int i = 0; i < per; ++i) {
                    const double v = scratch[grp * per + i];
                    if (v > a) { b = a; a = v; } else if (v > b) { b = v; }
                }
            w[h] = g.group_top == 2 && b > kNone ? a + b : a;
        }
        __syncwarp();
        scratch[lane] = w[0];
        scratch[lane + 32] = w[1];
        __syncwarp();
        // a group is kept if fewer than top_groups groups come before it
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bool& on = h == 0 ? on0 : on1;
            if (!on) continue;
            const int grp = (lane + 32 * h) / per;
            const double v = scratch[grp];
            int before = 0;
            for (int i = 0; i < g.n_groups; ++i) before += scratch[i] > v || (scratch[i] == v && i < grp);
            on = before < g.top_groups;
        }
        __syncwarp();
    }
    // k picks, the lower index first among equals; lane j keeps pick j
    int my_pick = -1;
    double my_z = 0.0, my_s = 0.0, zmax = kNone;
    int n = 0;
    for (int j = 0; j < g.k; ++j) {
        int best = on0 ? lane : on1 ? lane + 32 : kMaxExperts;
        double kb = on0 ? key0 : on1 ? key1 : 0.0;
        if (on0 && on1 && key1 > key0) { best = lane + 32; kb = key1; }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const int ob = __shfl_xor_sync(0xffffffffu, best, off);
            const double ok = __shfl_xor_sync(0xffffffffu, kb, off);
            if (ob < kMaxExperts && (best == kMaxExperts || ok > kb || (ok == kb && ob < best))) {
                best = ob;
                kb = ok;
            }
        }
        if (best == kMaxExperts) break;
        const int src = best & 31;
        const double zb = __shfl_sync(0xffffffffu, best < 32 ? z0 : z1, src);
        const double sb = __shfl_sync(0xffffffffu, best < 32 ? s0 : s1, src);
        if (lane == src) { if (best < 32) on0 = false; else on1 = false; }
        if (lane == j) { my_pick = best; my_z = zb; my_s = sb; }
        zmax = fmax(zmax, zb);
        n = j + 1;
    }
    double gate = lane < n ? my_s : 0.0;
    if (g.renorm && n > 0) {
        // scores divided by a factor common to the picks, so that the largest
        // stays near 1 where all of them underflow: exp(z - zmax) for softmax;
        // for sigmoid e^min(z,0) / (1 + e^-|z|) without e^min(zmax,0)
        double x = 0.0;
        if (lane < n)
            x = g.score == ADAFUSE_SCORE_SOFTMAX
                    ? exp(my_z - zmax)
                    : exp(fmin(my_z, 0.0) - fmin(zmax, 0.0)) / (1.0 + exp(-fabs(my_z)));
        gate = x / warp_sum(x);
    }
    if (lane < g.slots) {
        idx_out[lane] = lane < n ? my_pick : -1;
        gate_out[lane] = lane < n ? (float)(gate * (double)g.scale) : 0.f;
    }
}

__device__ __forceinline__ float route_load(const float* p) { return __ldg(p); }
__device__ __forceinline__ float route_load(const __nv_bfloat16* p) {
    return __bfloat162float(__ldg(p));
}

// One CTA per token, logits in 64 bits.
template <typename H>
__global__ void __launch_bounds__(256)
route_experts_kernel(const H* __restrict__ h, int64_t T, int64_t d, int64_t ldh,
                     const float* __restrict__ Wr, const GateParams g, int32_t* __restrict__ route) {
    __shared__ double zs[kMaxExperts];
    __shared__ double scratch[kMaxExperts];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        for (int e = warp; e < g.E; e += 8) {
            double acc = 0.0;
            for (int64_t i = lane; i < d; i += 32)
                acc = fma((double)route_load(h + t * ldh + i), (double)__ldg(Wr + i * g.E + e), acc);
            acc = warp_sum(acc);
            if (lane == 0) zs[e] = acc;
        }
        __syncthreads();
        if (warp == 0)
            route_decide(lane < g.E ? zs[lane] : 0.0, lane + 32 < g.E ? zs[lane + 32] : 0.0, g, lane,
                         scratch, route, t);
        __syncthreads();
    }
}

}  // namespace adafuse
