// route_experts.cuh -- per-token routing to experts: softmax or sigmoid
// scores, a selection bias, groups of experts, top-k, renormalised gates.
//
// The picks are those of logits and scores in 64 bits, at the cost of 32-bit
// ones: the logits are fp32 sums with an error bound, the decision compares
// every gap it depends on with the bound, and a token with a gap inside it has
// just the logits concerned summed again, in fp64, and is decided again.
//
// Bound: a thread adds 16 products, then chunks of kRouteDepth columns (n on
// each of C CTAs) in runs of kRouteRun, then runs, 8 warps and the CTAs, so
// every product passes at most m = 16 + kRouteRun + n / kRouteRun + 1 + 8 + C
// roundings (16 + n + 8 + C above 32 experts, without runs) and
//   |z - z64| <= m 2^-24 sum |h w| <= m 2^-24 |h| |w|   (Cauchy-Schwarz).
//
// Work: a CTA takes 32 tokens and a share of d.  Chunks of h (as stored) and Wr
// (rows of E floats are contiguous) come by cp.async into a ring; a warp takes
// 16 of a chunk's columns, a lane 4 tokens x EMAX / 4 experts of them.
#pragma once

#include <cuda_bf16.h>
#include <float.h>

#include "common.cuh"
#include "sm100_ptx.cuh"

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
__device__ __noinline__ void route_decide64(double z0, double z1, const GateParams g, int lane, double* scratch,
                                            int32_t* __restrict__ route, int64_t t) {
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
        auto kept = [&](int grp) {
            const double v = scratch[grp];
            int before = 0;
            for (int i = 0; i < g.n_groups; ++i) before += scratch[i] > v || (scratch[i] == v && i < grp);
            return before < g.top_groups;
        };
        if (on0) on0 = kept(lane / per);
        if (on1) on1 = kept((lane + 32) / per);
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

// The same decision in 32 bits for a warp's four tokens, eight lanes a token:
// lane `sub` holds the logits of experts sub * EPL ..  Every value that a
// comparison depends on carries a bound of its error, from the logits' (delta)
// and from its own arithmetic.  Returns the experts whose logits have to be
// known better before the decision stands (0: it stands, and the record is
// written).  lo / hi: EMAX floats each of shared memory per token.  All lanes
// of the warp call it; `valid` marks tokens that exist.
template <int EPL>
__device__ __forceinline__ uint64_t route_decide32(const float (&z)[EPL], float delta, const GateParams& g, int sub,
                                               bool valid, float* lo, float* hi, int32_t* __restrict__ route,
                                               int64_t t) {
    constexpr uint32_t kAll = 0xffffffffu;
    auto seg_max = [](float v) {
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, off));
        return v;
    };
    auto seg_sum = [](float v) {
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
        return v;
    };
    const int e0 = sub * EPL;
    bool all = !(delta < 0.25f);   // every expert is open
    uint32_t open = 0;             // open experts of this lane
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (e0 + i < g.E) {
            all = all || !(fabsf(z[i]) <= 1e30f);   // infinities, NaN, near overflow
            m = fmaxf(m, z[i]);
        }
    m = seg_max(m);
    const float grow = delta * (1.f + 4.f * delta);   // e^(2 delta) - 1 over 2, bounded
    float s[EPL], q[EPL], eq[EPL];
    float part = 0.f;
    // d softmax_e = p_e (dz_e - sum p dz): within 2 p_e delta; its own
    // arithmetic within 2e-6 + 2^-23 |z - m| of p.  d sigmoid = s (1 - s) dz;
    // its own arithmetic within 5e-7 of s.
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        s[i] = 0.f;
        eq[i] = 0.f;
        if (e0 + i < g.E) {
            if (g.score == ADAFUSE_SCORE_SOFTMAX) {
                s[i] = expf(z[i] - m);
                eq[i] = 2.f * grow + 2e-6f + 1.2e-7f * (m - z[i]);
            } else {
                const float u = expf(-fabsf(z[i])), den = 1.f + u;
                s[i] = z[i] >= 0.f ? 1.f / den : u / den;
                eq[i] = u / (den * den) * grow + 5e-7f * s[i];
            }
            part += s[i];
        }
    }
    if (g.score == ADAFUSE_SCORE_SOFTMAX) {
        const float sum = seg_sum(part);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            s[i] /= sum;
            eq[i] *= s[i];
        }
    }
    uint32_t on = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        q[i] = s[i];
        if (e0 + i < g.E) {
            const float b = g.bias != nullptr ? __ldg(g.bias + e0 + i) : 0.f;
            if (b > -INFINITY) on |= 1u << i;
            if (g.bias != nullptr) {
                q[i] = s[i] + b;
                eq[i] = isinf(b) ? 0.f : eq[i] + 1.2e-7f * fabsf(q[i]);
            }
        }
        eq[i] += 1e-37f;
    }
    if (g.n_groups > 1) {
        // a group's worth lies between the sums of its best values' lower and
        // upper ends
        const int per = g.E / g.n_groups;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (e0 + i < g.E) {
                lo[e0 + i] = on >> i & 1 ? q[i] - eq[i] : -INFINITY;
                hi[e0 + i] = on >> i & 1 ? q[i] + eq[i] : -INFINITY;
            }
        __syncwarp();
        float wl[8], wh[8];   // groups sub, sub + 8, ...
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            float a = -INFINITY, b = -INFINITY, c = -INFINITY, d = -INFINITY;
            if (sub + 8 * u < g.n_groups)
                for (int i = 0; i < per; ++i) {
                    const float v = lo[(sub + 8 * u) * per + i], w = hi[(sub + 8 * u) * per + i];
                    if (v > a) { b = a; a = v; } else if (v > b) { b = v; }
                    if (w > c) { d = c; c = w; } else if (w > d) { d = w; }
                }
            wl[u] = g.group_top == 2 && b > -INFINITY ? a + b : a;
            wh[u] = g.group_top == 2 && d > -INFINITY ? c + d : c;
            if (fabsf(wl[u]) < INFINITY) wl[u] -= 1.2e-7f * fabsf(wl[u]);
            if (fabsf(wh[u]) < INFINITY) wh[u] += 1.2e-7f * fabsf(wh[u]);
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (sub + 8 * u < g.n_groups) { lo[sub + 8 * u] = wl[u]; hi[sub + 8 * u] = wh[u]; }
        __syncwarp();
        // a group is kept if fewer than top_groups may come before it, dropped
        // if at least that many must; anything else is open
        uint64_t keep = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int grp = sub + 8 * u;
            if (grp >= g.n_groups) continue;
            int may = 0, must = 0;
            for (int i = 0; i < g.n_groups; ++i) {
                if (i == grp) continue;
                // a group with nothing enabled is worth -inf exactly
                may += hi[i] >= wl[u] && (hi[i] > -INFINITY || i < grp);
                must += lo[i] > wh[u] || (lo[i] == -INFINITY && wh[u] == -INFINITY && i < grp);
            }
            if (may < g.top_groups) keep |= 1ull << grp;
            else if (must < g.top_groups) all = true;
        }
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) keep |= __shfl_xor_sync(kAll, (unsigned long long)keep, off);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (e0 + i < g.E && !(keep >> ((e0 + i) / per) & 1)) on &= ~(1u << i);
        __syncwarp();
    }
    // k picks, the lower index first among equals (equal keys are open, infinite
    // ones apart); lane `sub` keeps pick number sub
    int my_pick = -1, n = 0;
    float my_z = 0.f, my_s = 0.f, zmax = -INFINITY;
    for (int j = 0; j < g.k; ++j) {
        int best = kMaxExperts;
        float kb = 0.f, zb = 0.f, sb = 0.f, eb = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float key = g.bias != nullptr ? q[i] : z[i];
            if ((on >> i & 1) && (best == kMaxExperts || key > kb)) {
                best = e0 + i;
                kb = key;
                zb = z[i];
                sb = s[i];
                eb = g.bias != nullptr ? eq[i] : delta;
            }
        }
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) {
            const int ob = __shfl_xor_sync(kAll, best, off);
            const float ok = __shfl_xor_sync(kAll, kb, off), oz = __shfl_xor_sync(kAll, zb, off);
            const float os = __shfl_xor_sync(kAll, sb, off), oe = __shfl_xor_sync(kAll, eb, off);
            if (ob < kMaxExperts && (best == kMaxExperts || ok > kb || (ok == kb && ob < best))) {
                best = ob;
                kb = ok;
                zb = oz;
                sb = os;
                eb = oe;
            }
        }
        const uint32_t mine = best / EPL == sub ? 1u << (best % EPL) : 0u;
        on &= ~mine;
        // who among the rest may really come before this pick
        uint32_t rivals = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if ((on >> i & 1) && (g.bias != nullptr ? q[i] + eq[i] : z[i] + delta) >= kb - eb) rivals |= 1u << i;
        if (best == kMaxExperts || isinf(kb)) rivals = 0;
        open |= rivals;
        if (__ballot_sync(kAll, rivals != 0) >> (threadIdx.x & 24) & 0xffu) open |= mine;
        if (best < kMaxExperts) {
            if (sub == j) { my_pick = best; my_z = zb; my_s = sb; }
            zmax = fmaxf(zmax, zb);
            n = j + 1;
        }
    }
    float gate = sub < n ? my_s : 0.f;
    float x = 0.f;
    if (sub < n)   // see route_decide64
        x = g.score == ADAFUSE_SCORE_SOFTMAX
                ? expf(my_z - zmax)
                : expf(fminf(my_z, 0.f) - fminf(zmax, 0.f)) / (1.f + expf(-fabsf(my_z)));
    const float sum = seg_sum(x);
    if (g.renorm && n > 0) gate = x / sum;
    // a score with a bias depends on every logit: known better all at once
    if (open != 0 && g.bias != nullptr && g.score == ADAFUSE_SCORE_SOFTMAX) all = true;
    unsigned long long mask = (unsigned long long)open << e0;
    if (all) mask = g.E == 64 ? ~0ull : (1ull << g.E) - 1;
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) mask |= __shfl_xor_sync(kAll, mask, off);
    if (valid && mask == 0 && sub < g.slots) {
        int32_t* rec = route + t * 2 * g.slots;
        rec[sub] = sub < n ? my_pick : -1;
        reinterpret_cast<float*>(rec)[g.slots + sub] = sub < n ? gate * g.scale : 0.f;
    }
    return mask;
}

constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = 8;
constexpr int kRouteTokens = 32;
constexpr int kRouteDepth = 128;      // columns of h per chunk, 16 a warp
constexpr int kRouteStages = 4;
constexpr int kRouteRun = 6;

// Shared memory of a stage: h rows padded by 16 bytes (their 16-byte pieces
// fall into different banks), then Wr's rows as they are, 256 bytes of slack for
// the reads past the last expert.
template <typename H>
__host__ __device__ constexpr uint32_t route_h_pitch() { return kRouteDepth * (uint32_t)sizeof(H) + 16; }
template <typename H>
__host__ __device__ constexpr uint32_t route_stage_bytes(int E) {
    return kRouteTokens * route_h_pitch<H>() + (((uint32_t)kRouteDepth * E * 4 + 256u));
}
// after the loop: warps' partial logits and squares, the CTA's sums, the
// groups' scratch, the logits in 64 bits; the fp64 pass reuses the start
template <int EMAX>
__host__ __device__ constexpr uint32_t route_tail_bytes() {
    return 4u * ((kRouteWarps + 1) * (kRouteTokens + 1) * (EMAX + 1) + 2 * kRouteTokens * EMAX) + 64u +
           8u * (kRouteTokens + kRouteWarps) * kMaxExperts;
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, int valid) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(valid)
                     : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Four consecutive values of a row in shared memory as floats.
__device__ __forceinline__ float4 route_h4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 route_h4(const __nv_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ float route_load(const float* p) { return __ldg(p); }
__device__ __forceinline__ float route_load(const __nv_bfloat16* p) {
    return __bfloat162float(__ldg(p));
}

// VEC: E is a multiple of EMAX / 4 (up to 4), so a lane's experts of a row are
// read as vectors.  h_piece / w_piece: bytes of a copy (16, or 8 / 4 where rows
// or Wr are aligned to no more).
template <int EMAX, bool VEC, typename H>
__global__ void __launch_bounds__(kRouteThreads, EMAX <= 16 ? 2 : 1)
route_experts_kernel(const H* __restrict__ h, const int64_t T, const int64_t d, const int64_t ldh,
                     const float* __restrict__ Wr, const GateParams g, int32_t* __restrict__ route, const int C,
                     const int h_piece, const int w_piece) {
    constexpr int TE = EMAX / 4;         // experts per lane
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q = (int)(blockIdx.x % (unsigned)C);
    const int64_t tok0 = (int64_t)(blockIdx.x / (unsigned)C) * kRouteTokens;
    const int ntok = (int)(T - tok0 < kRouteTokens ? T - tok0 : kRouteTokens);
    const uint32_t smem_s = (uint32_t)__cvta_generic_to_shared(smem);
    const uint32_t stage_bytes = route_stage_bytes<H>(g.E);
    constexpr uint32_t kPitch = route_h_pitch<H>();
    const int64_t chunks = (d + kRouteDepth - 1) / kRouteDepth;

    // Chunk c (of the CTA's: q, q + C, ...) into a stage; columns from d on read
    // as zero, rows of missing tokens are left alone.  A thread copies pieces
    // of one row, tid / 8, and every kRouteThreads-th piece of Wr.
    const int row = threadIdx.x >> 3;
    const bool row_in = row < ntok;
    const H* hrow = h + (tok0 + (row_in ? row : 0)) * ldh;
    const uint32_t h_dst = smem_s + (uint32_t)row * kPitch;
    const uint32_t w_dst = smem_s + kRouteTokens * kPitch;
    const int w_all = kRouteDepth * g.E * 4;
    auto load_chunk = [&](int64_t c, int stage) {
        if (c < chunks) {
            const int64_t k0 = c * kRouteDepth;
            const int cols = (int)(d - k0 < kRouteDepth ? d - k0 : kRouteDepth);
            const uint32_t so = (uint32_t)stage * stage_bytes;
            if (row_in) {
                if (h_piece == 16) {
                    constexpr int kPer = 16 / (int)sizeof(H);
#pragma unroll
                    for (int k = (threadIdx.x & 7) * kPer; k < kRouteDepth; k += 8 * kPer) {
                        const int left = (cols - k) * (int)sizeof(H);
                        cp_async<16>(h_dst + so + k * (uint32_t)sizeof(H), hrow + k0 + (left > 0 ? k : 0),
                                     left <= 0 ? 0 : left < 16 ? left : 16);
                    }
                } else {
                    constexpr int kPer = 8 / (int)sizeof(H);
#pragma unroll
                    for (int k = (threadIdx.x & 7) * kPer; k < kRouteDepth; k += 8 * kPer) {
                        const int left = (cols - k) * (int)sizeof(H);
                        cp_async<8>(h_dst + so + k * (uint32_t)sizeof(H), hrow + k0 + (left > 0 ? k : 0),
                                    left <= 0 ? 0 : 8);
                    }
                }
            }
            const char* wsrc = reinterpret_cast<const char*>(Wr + k0 * g.E);
            const int w_in = cols * g.E * 4;   // a multiple of 16
            if (w_piece == 16) {
                for (int o = threadIdx.x * 16; o < w_all; o += kRouteThreads * 16)
                    cp_async<16>(w_dst + so + o, wsrc + (o < w_in ? o : 0), o < w_in ? 16 : 0);
            } else {
                for (int o = threadIdx.x * 4; o < w_all; o += kRouteThreads * 4)
                    cp_async<4>(w_dst + so + o, wsrc + (o < w_in ? o : 0), o < w_in ? 4 : 0);
            }
        }
        cp_async_commit();
    };

    // lane: tokens tl, tl + 8, tl + 16, tl + 24; experts TE * eg .. + TE
    const int tl = lane >> 2, eg = lane & 3;
    // sums of a chunk, of kRouteRun chunks (where registers allow), of all
    constexpr bool kRuns = EMAX <= 32;
    float sum[4][TE], run[kRuns ? 4 : 1][TE], hh = 0.f, ww[EMAX > 32 ? 2 : 1];
    int in_run = 0;
#pragma unroll
    for (int i = 0; i < (kRuns ? 4 : 1); ++i)
#pragma unroll
        for (int e = 0; e < TE; ++e) run[i][e] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < TE; ++e) sum[i][e] = 0.f;
    ww[0] = 0.f;
    if (EMAX > 32) ww[EMAX > 32 ? 1 : 0] = 0.f;

    sm100::pdl_wait();   // set-up overlaps the end of the launch before this one
#pragma unroll
    for (int s = 0; s < kRouteStages - 1; ++s) load_chunk(q + (int64_t)s * C, s);
    int stage = 0;
#pragma unroll 1
    for (int64_t c = q; c < chunks; c += C) {
        cp_async_wait<kRouteStages - 2>();
        __syncthreads();   // the chunk has landed, and the stage before it is free
        load_chunk(c + (int64_t)(kRouteStages - 1) * C, stage == 0 ? kRouteStages - 1 : stage - 1);
        const uint8_t* base = smem + (size_t)stage * stage_bytes;
        const float* wt = reinterpret_cast<const float*>(base + kRouteTokens * kPitch);
        float acc[4][TE];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < TE; ++e) acc[i][e] = 0.f;
        // few warps an SM: independent loads in flight rather than short code
#pragma unroll(EMAX <= 32 ? 4 : 1)
        for (int k4 = 0; k4 < 16; k4 += 4) {
            const int k = 16 * warp + k4;
            float4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = route_h4(reinterpret_cast<const H*>(base + (size_t)(tl + 8 * i) * kPitch) + k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const float* wrow = wt + (k + kk) * g.E + TE * eg;
                float w[TE];
                if constexpr (VEC && TE == 2) {
                    const float2 v = *reinterpret_cast<const float2*>(wrow);
                    w[0] = v.x; w[1] = v.y;
                } else if constexpr (VEC) {
#pragma unroll
                    for (int e = 0; e < TE; e += 4) {
                        const float4 v = *reinterpret_cast<const float4*>(wrow + e);
                        w[e] = v.x; w[e + 1] = v.y; w[e + 2] = v.z; w[e + 3] = v.w;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < TE; ++e) w[e] = TE * eg + e < g.E ? wrow[e] : 0.f;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float xv = kk == 0 ? x[i].x : kk == 1 ? x[i].y : kk == 2 ? x[i].z : x[i].w;
#pragma unroll
                    for (int e = 0; e < TE; ++e) acc[i][e] = fmaf(xv, w[e], acc[i][e]);
                }
            }
        }
        if constexpr (kRuns) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < TE; ++e) run[i][e] += acc[i][e];
            if (++in_run == kRouteRun) {
                in_run = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < TE; ++e) {
                        sum[i][e] += run[i][e];
                        run[i][e] = 0.f;
                    }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < TE; ++e) sum[i][e] += acc[i][e];
        }
        // squares of the same columns, for the bound: lane = token, lane = expert
        {
            const H* hr = reinterpret_cast<const H*>(base + (size_t)lane * kPitch) + 16 * warp;
            float2 a = make_float2(0.f, 0.f), b = a;
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
                const float4 v = route_h4(hr + k);
                a.x = fmaf(v.x, v.x, a.x);
                a.y = fmaf(v.y, v.y, a.y);
                b.x = fmaf(v.z, v.z, b.x);
                b.y = fmaf(v.w, v.w, b.y);
            }
            hh += (a.x + a.y) + (b.x + b.y);
#pragma unroll
            for (int u = 0; u < (EMAX > 32 ? 2 : 1); ++u)
                if (lane + 32 * u < g.E) {
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float v = wt[(16 * warp + k) * g.E + lane + 32 * u];
                        c[k & 3] = fmaf(v, v, c[k & 3]);
                    }
                    ww[u] += (c[0] + c[1]) + (c[2] + c[3]);
                }
        }
        if (++stage == kRouteStages) stage = 0;
    }
    if constexpr (kRuns) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < TE; ++e) sum[i][e] += run[i][e];
    }
    cp_async_wait<0>();
    __syncthreads();   // the ring is free

    // ---- sums over the warps, then over the cluster: z[token][expert]; row 32
    // of a partial holds the experts' squares, column EMAX the tokens'
    constexpr int kRow = EMAX + 1, kPart = (kRouteTokens + 1) * kRow;
    float* part = reinterpret_cast<float*>(smem);
    float* total = part + kRouteWarps * kPart;
    float* ends = total + kPart;             // [32][2][EMAX], the groups' scratch
    // the logits in 64 bits [32][64], then the fp64 pass's sums and scratch
    double* fixed = reinterpret_cast<double*>(
        smem + ((4u * ((kRouteWarps + 1) * kPart + 2 * kRouteTokens * EMAX) + 15u) & ~15u));
    {
        float* mine = part + warp * kPart;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < TE; ++e) mine[(tl + 8 * i) * kRow + TE * eg + e] = sum[i][e];
        mine[lane * kRow + EMAX] = hh;
        if (lane < EMAX) mine[kRouteTokens * kRow + lane] = ww[0];
        if (EMAX > 32) mine[kRouteTokens * kRow + 32 + lane] = ww[EMAX > 32 ? 1 : 0];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kPart; i += kRouteThreads) {
        float v = part[i];
#pragma unroll
        for (int w = 1; w < kRouteWarps; ++w) v += part[w * kPart + i];
        total[i] = v;
    }
    if (C > 1) sm100::cluster_sync(); else __syncthreads();
    auto total_at = [&](int i) {
        if (C == 1) return total[i];
        float f[8];   // all requested before the first is added
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            f[c] = 0.f;
            if (c < C)
                asm volatile("ld.shared::cluster.f32 %0, [%1];"
                             : "=f"(f[c])
                             : "r"(sm100::cluster_addr(&total[i], (uint32_t)c)));
        }
        float v = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) v += f[c];
        return v;
    };

    // ---- decisions: CTA q takes tokens q, q + C, ...; eight lanes a token
    constexpr int EPL = EMAX / 8;
    __shared__ uint64_t open_s[kRouteTokens];
    const int sub = lane & 7;
    const int t = q + C * (int)(threadIdx.x >> 3);
    float wmax = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (sub * EPL + i < g.E) wmax = fmaxf(wmax, total_at(kRouteTokens * kRow + sub * EPL + i));
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) wmax = fmaxf(wmax, __shfl_xor_sync(0xffffffffu, wmax, off));
    const bool valid = t < ntok;
    const int tt = valid ? t : 0;
    float z[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) z[i] = sub * EPL + i < g.E ? total_at(tt * kRow + sub * EPL + i) : 0.f;
    // 1.02: the squares are fp32 sums themselves; terms below fp32's normal
    // range are off by up to 2^-149 each instead.  (A NaN in Wr shows in z.)
    const int mine_chunks = (int)((chunks + C - 1) / C);
    const float roundings = 16.f + kRouteWarps + (float)C +
                            (kRuns ? kRouteRun + (float)(mine_chunks / kRouteRun + 1) : (float)mine_chunks);
    const float delta = 1.02f * roundings * 0x1p-24f * sqrtf(total_at(tt * kRow + EMAX)) * sqrtf(wmax) +
                        (float)d * 0x1p-148f;
    const uint64_t open = route_decide32<EPL>(z, delta, g, sub, valid, ends + (tt * 2) * EMAX,
                                              ends + (tt * 2 + 1) * EMAX, route, tok0 + t);
    if (valid) {
        if (sub == 0) open_s[t] = open;
        if (open != 0) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (sub * EPL + i < g.E) fixed[t * kMaxExperts + sub * EPL + i] = (double)z[i];
        }
    }
    if (C > 1) sm100::cluster_sync();   // peers may still read this CTA's sums
    if (!__syncthreads_or(valid && open != 0)) return;

    // ---- what the bounds left open, in fp64: for each token the CTA sums the
    // logits of four neighbouring experts at a time, a thread every 256th
    // column (16 of them requested at once), then its warps decide again
    double* sums = reinterpret_cast<double*>(smem);   // [8 warps][4]
    const bool w_vec = w_piece == 16 && (g.E & 3) == 0;
    for (int u = q; u < ntok; u += C) {
        const uint64_t rest = open_s[u];
        const H* hu = h + (tok0 + u) * ldh;
        for (int e = 0; e < g.E; e += 4) {
            if ((rest >> e & 15u) == 0) continue;
            double a[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 1
            for (int64_t i = threadIdx.x; i < d; i += 16 * kRouteThreads) {
                float x[16];
                float4 w[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int64_t k = i + j * kRouteThreads;
                    const float* src = Wr + k * g.E + e;
                    x[j] = 0.f;
                    w[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (k < d) {
                        x[j] = route_load(hu + k);
                        if (w_vec) {
                            w[j] = __ldg(reinterpret_cast<const float4*>(src));
                        } else {
                            w[j].x = __ldg(src);
                            if (e + 1 < g.E) w[j].y = __ldg(src + 1);
                            if (e + 2 < g.E) w[j].z = __ldg(src + 2);
                            if (e + 3 < g.E) w[j].w = __ldg(src + 3);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const double xv = (double)x[j];
                    a[0] = fma(xv, (double)w[j].x, a[0]);
                    a[1] = fma(xv, (double)w[j].y, a[1]);
                    a[2] = fma(xv, (double)w[j].z, a[2]);
                    a[3] = fma(xv, (double)w[j].w, a[3]);
                }
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) a[v] = warp_sum(a[v]);
            if (lane < 4) sums[warp * 4 + lane] = lane == 0 ? a[0] : lane == 1 ? a[1] : lane == 2 ? a[2] : a[3];
            __syncthreads();
            if (threadIdx.x < 4 && e + (int)threadIdx.x < g.E) {
                double v = 0.0;
                for (int w = 0; w < kRouteWarps; ++w) v += sums[w * 4 + threadIdx.x];
                fixed[u * kMaxExperts + e + threadIdx.x] = v;
            }
            __syncthreads();
        }
    }
    for (int u = q + C * warp; u < ntok; u += C * kRouteWarps)
        if (open_s[u] != 0)
            route_decide64(fixed[u * kMaxExperts + lane], fixed[u * kMaxExperts + 32 + lane], g, lane,
                           fixed + (kRouteTokens + warp) * kMaxExperts, route, tok0 + u);
}

}  // namespace adafuse
