// route_experts.cuh -- per-token routing to experts: softmax or sigmoid
// scores, a selection bias, groups of experts, top-k, renormalised gates.
//
// The picks are those of logits and scores in 64 bits, at the cost of 32-bit
// ones: the logits are fp32 sums with an error bound, the decision compares
// every gap it depends on with the bound, and a token with a gap inside it has
// just the logits concerned summed again, in fp64, and is decided again.
//
// Work: a CTA takes 32 tokens and a share of d; chunks of h (as stored) and of
// Wr come by cp.async into a ring, and each of 8 warps takes 16 of a chunk's
// columns: one step of mma.m16n8k16 for two token tiles and every 8 experts.
// Both factors are split into bf16 terms that add up to them (h: one if it is
// bf16, else three; Wr: three), so every product is exact, and products below
// 2^-25 of |h w| are left out.  (On the FP32 units the same sums took twice the
// instructions, which is what bounds this kernel.)
//
// Bound: a step's 16 products are summed by the tensor core, which may cut each
// of 17 addends and the sum at 2^-23 of the largest: 36 units of 2^-24 of the
// products' magnitude; the smaller terms, the left-out ones and joining them
// add less than 4.  Steps are added in runs of kRouteRun chunks (n chunks on
// each of C CTAs), then runs, 8 warps and the CTAs, so with
// m = 40 + kRouteRun + n / kRouteRun + 1 + 8 + C
//   |z - z64| <= m 2^-24 sum |h w| <= m 2^-24 |h| |w|   (Cauchy-Schwarz).
// |h| and |w| come from fp32 sums of squares, which say nothing where the squares
// underflow: a sum with any nonzero value in it is kept above zero, so that 0
// means a row (or a router) of zeros, whose logits are exact; below kRouteTiny
// nothing is bounded and every logit is open.  Above it |h| and |w| are at least
// 2^-40, and what terms below the normal range 2^-126 lose is no more than
//   in a sum of squares     d 2^-126                     (2^-15 of it for any d);
//   in splitting h and w    2^-126 sqrt(d) (|h| + |w|)   (2^-45 |h| |w| 2^-24);
//   in products and sums    2^-126 each, 16 a column     (d 2^-122).
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
constexpr float kRouteTiny = 0x1p-80f;   // of a sum of squares, see the file's head

// h, Wr and the bias may come from the launch before, under whose end this one is
// set up: they are no constant data.
__device__ __forceinline__ float route_load(const float* p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ float route_load(const __nv_bfloat16* p) {
    uint16_t v;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return __uint_as_float((uint32_t)v << 16);
}

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

// One decision by one warp, in 64 bits.  Lane l holds the logits of experts l
// (z0) and l + 32 (z1); scratch: kMaxExperts doubles of shared memory that belong
// to this warp.  Writes the record of every token in `tokens` (bit i: i-th record
// from `route` on), whose logits these are.
__device__ __noinline__ void route_decide64(double z0, double z1, const GateParams g, int lane, double* scratch,
                                            int32_t* __restrict__ route, uint32_t tokens) {
    const double kNone = -INFINITY;
    const bool in0 = lane < g.E, in1 = lane + 32 < g.E;
    auto write = [&](int idx, float gate) {
        for (uint32_t rest = tokens; rest != 0; rest &= rest - 1) {
            int32_t* rec = route + (__ffs((int)rest) - 1) * 2 * g.slots;
            if (lane < g.slots) {
                rec[lane] = idx;
                reinterpret_cast<float*>(rec)[g.slots + lane] = gate;
            }
        }
    };
    const bool fine = (!in0 || fabs(z0) <= (double)FLT_MAX) && (!in1 || fabs(z1) <= (double)FLT_MAX);
    if (!__all_sync(0xffffffffu, fine)) {
        write(-1, 0.f);
        return;
    }
    // scores: softmax over all E, or sigmoid (exp overflows to +inf for very
    // negative logits, and the score to 0); in 32 bits where only gates read them
    double s0 = 0.0, s1 = 0.0;
    if (g.bias == nullptr && g.n_groups == 1) {
        const float f0 = (float)z0, f1 = (float)z1;
        if (g.score == ADAFUSE_SCORE_SOFTMAX) {
            const double m = warp_max(fmax(in0 ? z0 : kNone, in1 ? z1 : kNone));
            const float e0 = in0 ? expf((float)(z0 - m)) : 0.f, e1 = in1 ? expf((float)(z1 - m)) : 0.f;
            const float sum = (float)warp_sum((double)(e0 + e1));
            s0 = e0 / sum;
            s1 = e1 / sum;
        } else {
            s0 = 1.f / (1.f + expf(-f0));
            s1 = 1.f / (1.f + expf(-f1));
        }
    } else if (g.score == ADAFUSE_SCORE_SOFTMAX) {
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
        if (in0) { const float b = route_load(g.bias + lane); on0 = b > -INFINITY; q0 = s0 + (double)b; }
        if (in1) { const float b = route_load(g.bias + lane + 32); on1 = b > -INFINITY; q1 = s1 + (double)b; }
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
        float x = 0.f;
        if (lane < n)
            x = g.score == ADAFUSE_SCORE_SOFTMAX
                    ? expf((float)(my_z - zmax))
                    : expf((float)(fmin(my_z, 0.0) - fmin(zmax, 0.0))) / (1.f + expf((float)-fabs(my_z)));
        gate = x / warp_sum((double)x);
    }
    write(lane < n ? my_pick : -1, lane < n ? (float)(gate * (double)g.scale) : 0.f);
}

// The same decision in 32 bits, LPT lanes a token and EPL <= 2 experts a lane:
// lane `sub` of the token holds the logits of experts sub + LPT * i.  Every value
// that a comparison depends on carries a bound of its error, from the logits'
// (delta) and from its own arithmetic.  Returns the experts whose logits have to
// be known better before the decision stands (0: it stands, and the record is
// written).  seg0: the token's first lane; ends: 4 * LPT * EPL floats of shared
// memory per token.  All lanes of the warp call it; `valid` marks tokens that
// exist.  What it costs is fetching its code, which every CTA runs once or a few
// times: eight experts a lane, unrolled, took 30 us longer at E = 64.
template <int LPT, int EPL>
__device__ __forceinline__ uint64_t route_decide32(const float (&z)[EPL], float delta, const GateParams& g, int sub,
                                                   int seg0, bool valid, float* ends,
                                                   int32_t* __restrict__ route, int64_t t) {
    constexpr uint32_t kAll = 0xffffffffu;
    constexpr uint32_t kSeg = LPT == 32 ? kAll : (1u << LPT) - 1;
    auto seg_max = [](float v) {
#pragma unroll
        for (int off = LPT / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, off));
        return v;
    };
    auto seg_sum = [](float v) {
#pragma unroll
        for (int off = LPT / 2; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
        return v;
    };
    // one bit for every lane of the token, and for every expert
    auto seg_bits = [&](bool p) { return __ballot_sync(kAll, p) >> seg0 & kSeg; };
    auto expert_bits = [&](const bool (&p)[EPL]) {
        uint64_t m = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) m |= (uint64_t)seg_bits(p[i]) << (LPT * i);
        return m;
    };
    bool all = !(delta < 0.25f);   // every expert is open
    bool in[EPL], on[EPL], open[EPL];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        in[i] = sub + LPT * i < g.E;
        open[i] = false;
        if (in[i]) {
            all = all || !(fabsf(z[i]) <= 1e30f);   // infinities, NaN, near overflow
            m = fmaxf(m, z[i]);
        }
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
        if (in[i]) {
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
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        q[i] = s[i];
        on[i] = false;
        if (in[i]) {
            const float b = g.bias != nullptr ? route_load(g.bias + sub + LPT * i) : 0.f;
            on[i] = b > -INFINITY;
            if (g.bias != nullptr) {
                q[i] = s[i] + b;
                eq[i] = isinf(b) ? 0.f : eq[i] + 1.2e-7f * fabsf(q[i]);
            }
        }
        eq[i] += 1e-37f;
    }
    // what picks are ordered by, and how far off it may be
    float key[EPL], ekey[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        key[i] = g.bias != nullptr ? q[i] : z[i];
        ekey[i] = g.bias != nullptr ? eq[i] : delta;
    }
    if (g.n_groups > 1) {
        // a group's worth lies between the sums of its best values' lower and
        // upper ends
        const int per = g.E / g.n_groups;
        float *lo = ends, *hi = ends + LPT * EPL, *glo = hi + LPT * EPL, *ghi = glo + LPT * EPL;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (in[i]) {
                lo[sub + LPT * i] = on[i] ? q[i] - eq[i] : -INFINITY;
                hi[sub + LPT * i] = on[i] ? q[i] + eq[i] : -INFINITY;
            }
        __syncwarp();
#pragma unroll 1
        for (int grp = sub; grp < g.n_groups; grp += LPT) {
            float a = -INFINITY, b = -INFINITY, c = -INFINITY, d = -INFINITY;
#pragma unroll 1
            for (int i = grp * per; i < (grp + 1) * per; ++i) {
                const float v = lo[i], w = hi[i];
                b = fmaxf(b, fminf(a, v));
                a = fmaxf(a, v);
                d = fmaxf(d, fminf(c, w));
                c = fmaxf(c, w);
            }
            float wl = g.group_top == 2 && b > -INFINITY ? a + b : a;
            float wh = g.group_top == 2 && d > -INFINITY ? c + d : c;
            if (fabsf(wl) < INFINITY) wl -= 1.2e-7f * fabsf(wl);
            if (fabsf(wh) < INFINITY) wh += 1.2e-7f * fabsf(wh);
            glo[grp] = wl;
            ghi[grp] = wh;
        }
        __syncwarp();
        // a group is kept if fewer than top_groups may come before it, dropped
        // if at least that many must; anything else is open
        bool keep[EPL], unsure[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int grp = sub + LPT * i;
            int may = 0, must = 0;
            if (grp < g.n_groups) {
                const float wl = glo[grp], wh = ghi[grp];
#pragma unroll 1
                for (int u = 0; u < g.n_groups; ++u) {
                    // a group with nothing enabled is worth -inf exactly
                    const float ul = glo[u], uh = ghi[u];
                    may += u != grp && uh >= wl && (uh > -INFINITY || u < grp);
                    must += u != grp && (ul > wh || (ul == -INFINITY && wh == -INFINITY && u < grp));
                }
            }
            keep[i] = grp < g.n_groups && may < g.top_groups;
            unsure[i] = grp < g.n_groups && !keep[i] && must < g.top_groups;
        }
        const uint64_t kept = expert_bits(keep), doubt = expert_bits(unsure);
        // of an unsure group, the experts that may be among its best are open
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (!in[i]) continue;
            const int grp = (sub + LPT * i) / per;
            if (doubt >> grp & 1) {
                int above = 0;   // experts of the group surely before this one
#pragma unroll 1
                for (int u = grp * per; u < (grp + 1) * per; ++u) above += lo[u] > q[i] + eq[i];
                open[i] = on[i] && above < g.group_top;
            } else if (!(kept >> grp & 1)) {
                on[i] = false;
            }
        }
        if (__any_sync(kAll, doubt != 0)) {
            // which experts the picks choose from depends on the groups: any
            // two of the kept and unsure groups' that are too close are open
            const uint64_t cand = expert_bits(on);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (in[i]) {
                    lo[sub + LPT * i] = key[i] - ekey[i];
                    hi[sub + LPT * i] = key[i] + ekey[i];
                }
            __syncwarp();
            uint64_t rest = doubt != 0 ? cand : 0;
#pragma unroll 1
            while (rest != 0) {
                const int u = __ffsll((long long)rest) - 1;
                rest &= rest - 1;
                const float l = lo[u], h = hi[u];
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (on[i] && u != sub + LPT * i && key[i] - ekey[i] <= h && l <= key[i] + ekey[i]) open[i] = true;
            }
        }
        __syncwarp();
    }
    // k picks, the lower index first among equals (equal keys are open, infinite
    // ones apart); lane `sub` keeps pick number sub
    int my_pick = -1, n = 0;
    float my_z = 0.f, my_s = 0.f, zmax = -INFINITY;
#pragma unroll 1
    for (int j = 0; j < g.k; ++j) {
        float kb = -INFINITY;   // no enabled key is this low
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (on[i]) kb = fmaxf(kb, key[i]);
        kb = seg_max(kb);
        bool hit[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) hit[i] = on[i] && key[i] == kb;
        const uint64_t hits = expert_bits(hit);
        const int best = hits != 0 ? __ffsll((long long)hits) - 1 : -1;
        const int src = seg0 + (best >= 0 ? best % LPT : 0);
        const bool second = EPL == 2 && best >= LPT;
        const float zb = __shfl_sync(kAll, second ? z[EPL - 1] : z[0], src);
        const float sb = __shfl_sync(kAll, second ? s[EPL - 1] : s[0], src);
        const float eb = __shfl_sync(kAll, second ? ekey[EPL - 1] : ekey[0], src);
        // who among the rest may really come before this pick; equal keys that
        // are exact are settled by the index
        const bool settled = best < 0 || isinf(kb) || (g.bias == nullptr && delta == 0.f);
        bool rivals = false;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (best == sub + LPT * i) on[i] = false;
            const bool rival = !settled && on[i] && key[i] + ekey[i] >= kb - eb;
            open[i] = open[i] || rival;
            rivals = rivals || rival;
        }
        const bool disputed = seg_bits(rivals) != 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (disputed && best == sub + LPT * i) open[i] = true;
        if (best >= 0) {
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
    uint64_t mask = expert_bits(open);
    // a score with a bias depends on every logit: known better all at once
    if (mask != 0 && g.bias != nullptr && g.score == ADAFUSE_SCORE_SOFTMAX) all = true;
    if (seg_bits(all) != 0) mask = g.E == 64 ? ~0ull : (1ull << g.E) - 1;
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

// Shared memory of a stage: h rows padded by 16 bytes, then rows of Wr padded to
// 4 or 12 floats past a multiple of 16, so that fragment reads fall into
// different banks (rows that no 16-byte copy divides are not padded: the chunk is
// copied as it lies.  T = 2376 5072 x 62: 125 us, in copies of 4 bytes to padded rows
// 219); 256 bytes of slack for the reads past the last expert.
template <typename H>
__host__ __device__ constexpr uint32_t route_h_pitch() { return kRouteDepth * (uint32_t)sizeof(H) + 16; }
__host__ __device__ constexpr int route_w_pitch(int E) {   // in floats
    return (E + 3) / 4 * 4 + ((E + 3) / 4 % 2 == 0 ? 4 : 0);
}
template <typename H>
__host__ __device__ constexpr uint32_t route_stage_bytes(int E) {
    return kRouteTokens * route_h_pitch<H>() + (uint32_t)kRouteDepth * route_w_pitch(E) * 4u + 256u;
}
// lanes that decide on a token, and the floats of shared memory they need
template <int EMAX>
__host__ __device__ constexpr int route_lanes() { return EMAX < 32 ? EMAX : 32; }
template <int EMAX>
__host__ __device__ constexpr int route_ends() { return kRouteThreads / route_lanes<EMAX>() * 4 * EMAX; }
// after the loop: warps' partial logits and squares, the CTA's sums, the
// groups' scratch, the logits in 64 bits; the fp64 pass reuses the start
template <int EMAX>
__host__ __device__ constexpr uint32_t route_tail_bytes() {
    return 4u * ((kRouteWarps + 1) * (kRouteTokens + 1) * (EMAX + 1) + route_ends<EMAX>()) + 64u +
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

// Two floats as the sum of packed bf16 terms, largest first (24 bits: exact up
// to 2^-27 of the value).
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void split3(float x, float y, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = pack_bf16(x, y);
    x -= __uint_as_float(hi << 16);
    y -= __uint_as_float(hi & 0xffff0000u);
    mid = pack_bf16(x, y);
    lo = pack_bf16(x - __uint_as_float(mid << 16), y - __uint_as_float(mid & 0xffff0000u));
}
// d = a b, and d += a b
__device__ __forceinline__ void route_mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void route_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A token tile's 16 columns as A fragments, one plane per term; the squares of
// its values added to the lane's two rows, their bits to the rows' (s, b).
__device__ __forceinline__ void route_h_frag(const float* r0, const float* r1, uint32_t (&a)[3][4], float (&s)[2],
                                             uint32_t (&b)[2]) {
    const float2 v[4] = {*reinterpret_cast<const float2*>(r0), *reinterpret_cast<const float2*>(r1),
                         *reinterpret_cast<const float2*>(r0 + 8), *reinterpret_cast<const float2*>(r1 + 8)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        split3(v[i].x, v[i].y, a[0][i], a[1][i], a[2][i]);
        s[i & 1] = fmaf(v[i].x, v[i].x, fmaf(v[i].y, v[i].y, s[i & 1]));
        b[i & 1] |= __float_as_uint(v[i].x) | __float_as_uint(v[i].y);
    }
}
__device__ __forceinline__ void route_h_frag(const __nv_bfloat16* r0, const __nv_bfloat16* r1,
                                             uint32_t (&a)[1][4], float (&s)[2], uint32_t (&b)[2]) {
    a[0][0] = *reinterpret_cast<const uint32_t*>(r0);
    a[0][1] = *reinterpret_cast<const uint32_t*>(r1);
    a[0][2] = *reinterpret_cast<const uint32_t*>(r0 + 8);
    a[0][3] = *reinterpret_cast<const uint32_t*>(r1 + 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = __uint_as_float(a[0][i] << 16), y = __uint_as_float(a[0][i] & 0xffff0000u);
        s[i & 1] = fmaf(x, x, fmaf(y, y, s[i & 1]));
    }
    b[0] |= a[0][0] | a[0][2];
    b[1] |= a[0][1] | a[0][3];
}
// A sum of squares above zero wherever one of its values is (bits: theirs, all
// taken together; `signs` are left out).
__device__ __forceinline__ float keep_nonzero(float s, uint32_t bits, uint32_t signs) {
    return (bits & ~signs) != 0 && s < FLT_MIN ? FLT_MIN : s;
}
// h_piece / w_piece: bytes of a copy (16, or 8 / 4 where rows or Wr are aligned
// to no more).
template <int EMAX, typename H>
__global__ void __launch_bounds__(kRouteThreads, EMAX <= 16 ? 2 : 1)
route_experts_kernel(const H* __restrict__ h, const int64_t T, const int64_t d, const int64_t ldh,
                     const float* __restrict__ Wr, const GateParams g, int32_t* __restrict__ route, const int C,
                     const int h_piece, const int w_piece) {
    constexpr int NT = EMAX / 8;                              // expert tiles
    constexpr int kTerms = sizeof(H) == 2 ? 1 : 3;            // of h
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q = (int)(blockIdx.x % (unsigned)C);
    const int64_t tok0 = (int64_t)(blockIdx.x / (unsigned)C) * kRouteTokens;
    const int ntok = (int)(T - tok0 < kRouteTokens ? T - tok0 : kRouteTokens);
    const uint32_t smem_s = (uint32_t)__cvta_generic_to_shared(smem);
    const uint32_t stage_bytes = route_stage_bytes<H>(g.E);
    constexpr uint32_t kPitch = route_h_pitch<H>();
    const int chunks = (int)((d + kRouteDepth - 1) / kRouteDepth);

    // Chunk c (of the CTA's: q, q + C, ...) into a stage; columns from d on read
    // as zero, rows of missing tokens are left alone.  A thread copies pieces of
    // one row, tid / 8, and every kRouteThreads-th piece of Wr, whose places in
    // the padded rows it works out once.
    const int row = threadIdx.x >> 3;
    const bool row_in = row < ntok;
    const H* hrow = h + (tok0 + (row_in ? row : 0)) * ldh;
    const uint32_t h_dst = smem_s + (uint32_t)row * kPitch;
    const uint32_t w_dst = smem_s + kRouteTokens * kPitch;
    const bool padded = w_piece == 16 && (g.E & 3) == 0;
    const int w_pitch = padded ? route_w_pitch(g.E) : g.E;
    const bool vec = h_piece == 16 && padded;
    const uint32_t w_row = (uint32_t)w_pitch * 4u;
    const int whole = (int)(d / kRouteDepth);
    const char* h_src = reinterpret_cast<const char*>(hrow) + (threadIdx.x & 7) * 16;
    const char* w_src = reinterpret_cast<const char*>(Wr) + threadIdx.x * 16;
    const int w_chunk = kRouteDepth * g.E * 4;
    uint32_t w_at[NT];   // piece tid + 256 j: E / 4 pieces a row
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int per = max(g.E >> 2, 1), i = (int)threadIdx.x + j * kRouteThreads;
        w_at[j] = w_dst + (uint32_t)(i / per) * w_row + (uint32_t)(i % per) * 16u;
    }
    auto load_chunk = [&](int c, int stage) {
        const uint32_t so = (uint32_t)stage * stage_bytes;
        if (c < whole && vec) {
            if (row_in) {
                const char* src = h_src + (int64_t)c * (kRouteDepth * (int)sizeof(H));
                const uint32_t dst = h_dst + so + (threadIdx.x & 7) * 16;
#pragma unroll
                for (int j = 0; j < kRouteDepth * (int)sizeof(H) / 128; ++j) cp_async<16>(dst + 128 * j, src + 128 * j, 16);
            }
            const char* src = w_src + (int64_t)c * w_chunk;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if ((int)threadIdx.x * 16 + j * (kRouteThreads * 16) < w_chunk)
                    cp_async<16>(w_at[j] + so, src + j * (kRouteThreads * 16), 16);
        } else if (c < chunks) {
            // pieces in the order they lie; what is past the last column reads as zero
            const int64_t k0 = (int64_t)c * kRouteDepth;
            const int cols = (int)(d - k0 < kRouteDepth ? d - k0 : kRouteDepth);
            if (row_in) {
                const int there = cols * (int)sizeof(H);
                const char* src = reinterpret_cast<const char*>(hrow + k0);
#pragma unroll 1
                for (int at = (threadIdx.x & 7) * h_piece; at < kRouteDepth * (int)sizeof(H); at += 8 * h_piece) {
                    const int valid = at >= there ? 0 : there - at < h_piece ? there - at : h_piece;
                    const char* from = src + (valid > 0 ? at : 0);
                    if (h_piece == 16) cp_async<16>(h_dst + so + at, from, valid);
                    else cp_async<8>(h_dst + so + at, from, valid);
                }
            }
            const char* src = reinterpret_cast<const char*>(Wr + k0 * g.E);
            const int there = cols * g.E * 4, per_row = g.E >> 2;
#pragma unroll 1
            for (int i = threadIdx.x; i * w_piece < w_chunk; i += kRouteThreads) {
                const int at = i * w_piece;
                const int valid = at >= there ? 0 : there - at < w_piece ? there - at : w_piece;
                const uint32_t dst = w_dst + so + (padded ? (i / per_row) * w_row + (i % per_row) * 16u : (uint32_t)at);
                const char* from = src + (valid > 0 ? at : 0);
                if (w_piece == 16) cp_async<16>(dst, from, valid); else cp_async<4>(dst, from, valid);
            }
        }
        cp_async_commit();
    };

    // fragments: lane = 4 * g8 + tig holds tokens 16 m + g8 and + 8, experts
    // 8 n + 2 tig and + 1
    const int g8 = lane >> 2, tig = lane & 3;
    float sum[2][NT][4], run[2][NT][4], hh[2][2], ww[NT];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        hh[m][0] = hh[m][1] = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[m][n][i] = run[m][n][i] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) ww[n] = 0.f;
    int in_run = 0;
    uint32_t w_bits = 0, h_bits[2][2] = {{0, 0}, {0, 0}};
    // what fragment reads past the last expert meet, row padding and slack, is zero
    {
        const uint32_t per = padded ? w_row - (uint32_t)g.E * 4u : 0u;   // 0 or 16 bytes a row
        const uint32_t tail = (uint32_t)kRouteDepth * w_row;
        for (int s = 0; s < kRouteStages; ++s) {
            uint8_t* w = smem + (size_t)s * stage_bytes + kRouteTokens * kPitch;
            if (per != 0 && threadIdx.x < kRouteDepth)
                *reinterpret_cast<uint4*>(w + threadIdx.x * w_row + g.E * 4) = make_uint4(0u, 0u, 0u, 0u);
            if (threadIdx.x >= kRouteThreads - 64)
                *reinterpret_cast<uint32_t*>(w + tail + (threadIdx.x - (kRouteThreads - 64)) * 4) = 0u;
        }
    }

    sm100::pdl_wait();   // set-up overlaps the end of the launch before this one
    sm100::pdl_launch_dependents();
#pragma unroll
    for (int s = 0; s < kRouteStages - 1; ++s) load_chunk(q + s * C, s);
    int stage = 0;
#pragma unroll 1
    for (int c = q; c < chunks; c += C) {
        cp_async_wait<kRouteStages - 2>();
        __syncthreads();   // the chunk has landed, and the stage before it is free
        load_chunk(c + (kRouteStages - 1) * C, stage == 0 ? kRouteStages - 1 : stage - 1);
        const uint8_t* base = smem + (size_t)stage * stage_bytes;
        const float* wt = reinterpret_cast<const float*>(base + kRouteTokens * kPitch) +
                          (16 * warp + 2 * tig) * w_pitch + g8;
        uint32_t a[2][kTerms][4];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const H* r0 = reinterpret_cast<const H*>(base + (size_t)(16 * m + g8) * kPitch) + 16 * warp + 2 * tig;
            const H* r1 = reinterpret_cast<const H*>(reinterpret_cast<const uint8_t*>(r0) + 8 * kPitch);
            route_h_frag(r0, r1, a[m], hh[m], h_bits[m]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float* w = wt + 8 * n;
            const float w0 = w[0], w1 = w[w_pitch], w2 = w[8 * w_pitch], w3 = w[9 * w_pitch];
            ww[n] = fmaf(w0, w0, fmaf(w1, w1, fmaf(w2, w2, fmaf(w3, w3, ww[n]))));
            w_bits |= __float_as_uint(w0) | __float_as_uint(w1);
            w_bits |= __float_as_uint(w2) | __float_as_uint(w3);
            uint32_t b[3][2];
            split3(w0, w1, b[0][0], b[1][0], b[2][0]);
            split3(w2, w3, b[0][1], b[1][1], b[2][1]);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float z[4];   // the smallest products first
                route_mma0(z, a[m][0], b[2][0], b[2][1]);
                if constexpr (kTerms == 3) {
                    route_mma(z, a[m][2], b[0][0], b[0][1]);
                    route_mma(z, a[m][1], b[1][0], b[1][1]);
                    route_mma(z, a[m][1], b[0][0], b[0][1]);
                }
                route_mma(z, a[m][0], b[1][0], b[1][1]);
                route_mma(z, a[m][0], b[0][0], b[0][1]);
#pragma unroll
                for (int i = 0; i < 4; ++i) run[m][n][i] += z[i];
            }
        }
        if (++in_run == kRouteRun) {
            in_run = 0;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        sum[m][n][i] += run[m][n][i];
                        run[m][n][i] = 0.f;
                    }
        }
        if (++stage == kRouteStages) stage = 0;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) ww[n] = keep_nonzero(ww[n], w_bits, 0x80000000u);
#pragma unroll
    for (int m = 0; m < 4; ++m)
        hh[m >> 1][m & 1] = keep_nonzero(hh[m >> 1][m & 1], h_bits[m >> 1][m & 1],
                                         sizeof(H) == 2 ? 0x80008000u : 0x80000000u);
    __shared__ uint32_t zeros_s;   // tokens whose logits are all 0 and whose ties the fp64 decision settles
    if (threadIdx.x == 0) zeros_s = 0;
    cp_async_wait<0>();
    __syncthreads();   // the ring is free

    // ---- sums over the warps, then over the cluster: z[token][expert]; row 32
    // of a partial holds the experts' squares, column EMAX the tokens'
    constexpr int kRow = EMAX + 1, kPart = (kRouteTokens + 1) * kRow;
    float* part = reinterpret_cast<float*>(smem);
    float* total = part + kRouteWarps * kPart;
    float* ends = total + kPart;             // the groups' scratch
    // the logits in 64 bits [32][64], then the fp64 pass's sums and scratch
    double* fixed = reinterpret_cast<double*>(
        smem + ((4u * ((kRouteWarps + 1) * kPart + route_ends<EMAX>()) + 15u) & ~15u));
    {
        float* mine = part + warp * kPart;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int t0 = 16 * m + g8;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mine[(t0 + (i >> 1) * 8) * kRow + 8 * n + 2 * tig + (i & 1)] = sum[m][n][i] + run[m][n][i];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v = hh[m][i];
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                if (tig == 0) mine[(t0 + 8 * i) * kRow + EMAX] = v;
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float v = ww[n];
            v += __shfl_xor_sync(0xffffffffu, v, 1);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
            if (tig == 0) mine[kRouteTokens * kRow + 8 * n + g8] = v;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kPart; i += kRouteThreads) {
        float v = part[i];
#pragma unroll
        for (int w = 1; w < kRouteWarps; ++w) v += part[w * kPart + i];
        total[i] = v;
    }
    // CTA q decides tokens q, q + C, ...: row t / C of zt, then the experts' squares
    float* zt = total;
    if (C > 1) {
        sm100::cluster_sync();
        zt = part;   // the warps' sums are done with
        const int rows = kRouteTokens / C, n = (rows + 1) * kRow;
        for (int i = threadIdx.x; i < n; i += kRouteThreads) {
            const int r = i / kRow, src = (r < rows ? q + C * r : kRouteTokens) * kRow + i - r * kRow;
            float f[8];   // all requested before the first is added
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                f[c] = 0.f;
                if (c < C)
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(f[c])
                                 : "r"(sm100::cluster_addr(&total[src], (uint32_t)c)));
            }
            float v = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) v += f[c];
            zt[i] = v;
        }
        sm100::cluster_sync();   // peers are done with this CTA's sums
    } else {
        __syncthreads();
    }
    const float* squares = zt + kRouteTokens / C * kRow;

    // ---- decisions: CTA q takes tokens q, q + C, ...
    constexpr int LPT = route_lanes<EMAX>(), EPL = EMAX / LPT;
    __shared__ uint64_t open_s[kRouteTokens];   // logits to be summed in fp64
    const int sub = lane % LPT, slot = (int)threadIdx.x / LPT;
    float wmax = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (sub + LPT * i < g.E) wmax = fmaxf(wmax, squares[sub + LPT * i]);
#pragma unroll
    for (int off = LPT / 2; off > 0; off >>= 1) wmax = fmaxf(wmax, __shfl_xor_sync(0xffffffffu, wmax, off));
    const int mine_chunks = (chunks + C - 1) / C;
    const float roundings = 49.f + kRouteRun + (float)(mine_chunks / kRouteRun) + (float)C;
    bool some_open = false;
#pragma unroll 1
    for (int r = slot; r - slot < kRouteTokens / C; r += kRouteThreads / LPT) {
        const int t = q + C * r;
        const bool valid = r < kRouteTokens / C && t < ntok;
        const float* zrow = zt + (valid ? r : 0) * kRow;
        float z[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) z[i] = sub + LPT * i < g.E ? zrow[sub + LPT * i] : 0.f;
        // the squares are sums of fp32 themselves: 4 additions a chunk, and 1.02 for
        // joining them and for what underflows.  (A NaN in Wr shows in z.)
        const float hh = zrow[EMAX];
        float delta = INFINITY;   // every logit is open
        if (hh == 0.f || wmax == 0.f)
            delta = 0.f;
        else if (hh >= kRouteTiny && wmax >= kRouteTiny)
            delta = (1.02f + (float)mine_chunks * 0x1p-22f) * roundings * 0x1p-24f * sqrtf(hh) * sqrtf(wmax) +
                    (float)d * 0x1p-122f;
        uint64_t open = route_decide32<LPT, EPL>(z, delta, g, sub, lane - sub, valid, ends + slot * 4 * EMAX,
                                                 route, tok0 + t);
        // A row (or a router) of zeros has nothing to sum: its logits are 0 as they
        // stand, and all such tokens share one decision.
        bool nonzero = delta != 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) nonzero = nonzero || z[i] != 0.f;   // a NaN is
        const uint32_t seg = LPT == 32 ? 0xffffffffu : ((1u << LPT) - 1) << (lane - sub);
        const bool zeros = (__ballot_sync(0xffffffffu, nonzero) & seg) == 0;
        if (valid) {
            if (zeros && open != 0) {
                if (sub == 0) atomicOr(&zeros_s, 1u << t);
                some_open = true;
                open = 0;
            }
            if (sub == 0) open_s[t] = open;
            if (open != 0) {
                some_open = true;
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (sub + LPT * i < g.E) fixed[t * kMaxExperts + sub + LPT * i] = (double)z[i];
            }
        }
    }
    if (!__syncthreads_or(some_open)) return;

    // ---- what the bounds left open, in fp64: for each token the CTA sums two open
    // logits at a time (most often there are two); then its warps decide again.
    // Two neighbouring lanes take the two experts of a row, 16 rows a warp: what
    // bounds this is the number of lines that a load touches.  (A lane for both
    // experts of a row, 32 rows a warp: 32.5 us instead of 30.2 at T = 4096 4096 x 16, 57.2
    // instead of 53.6 at T = 777 5120 x 64.)
    constexpr int kCols = 16, kRows = kRouteThreads / 2;
    double* sums = reinterpret_cast<double*>(smem);   // [8 warps][2], or one a thread
    const int which = threadIdx.x & 1, row0 = (int)threadIdx.x >> 1, w_step = kRows * g.E;
#pragma unroll 1
    for (int u = q; u < ntok; u += C) {
        uint64_t rest = open_s[u];
        // many at once (all, where a softmax score with a bias is open): a thread an
        // expert, whole rows of Wr.  Both ways' time, in tenths of a microsecond (T =
        // 777 4096 x 64, softmax and bias: 108 us, two at a time 345; T = 616 648 x 64:
        // 17 and 59).
        if (__popcll(rest) * (5 + 4 * (int)((d + 2047) >> 11)) > 7 * (int)((d * EMAX + 4095) >> 12)) {
            constexpr int kStep = kRouteThreads / EMAX;   // rows at a time
            const int e = threadIdx.x % EMAX, r0 = threadIdx.x / EMAX;
            const H* px = h + (tok0 + u) * ldh + r0;
            const float* pw = Wr + (int64_t)r0 * g.E + (e < g.E ? e : 0);
            double v = 0.0;
#pragma unroll 1
            for (int left = (int)((d - r0 + kStep - 1) / kStep); left > 0; left -= kCols) {
                float x[kCols], w[kCols];
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    x[c] = w[c] = 0.f;
                    if (c < left) {
                        x[c] = route_load(px + c * kStep);
                        w[c] = route_load(pw);
                    }
                    pw += kStep * g.E;
                }
                px += kCols * kStep;
#pragma unroll
                for (int c = 0; c < kCols; ++c) v = fma((double)x[c], (double)w[c], v);
            }
            sums[threadIdx.x] = v;
            __syncthreads();
            if ((int)threadIdx.x < g.E) {
                double t = 0.0;
#pragma unroll 1
                for (int r = 0; r < kStep; ++r) t += sums[r * EMAX + threadIdx.x];
                fixed[u * kMaxExperts + threadIdx.x] = t;
            }
            __syncthreads();
            continue;
        }
#pragma unroll 1
        while (rest != 0) {
            const int ea = __ffsll((long long)rest) - 1;
            rest &= rest - 1;
            const int eb = rest != 0 ? __ffsll((long long)rest) - 1 : ea;
            rest &= rest - 1;
            const int e = which ? eb : ea;
            const H* px = h + (tok0 + u) * ldh + row0;
            const float* pw = Wr + (int64_t)row0 * g.E + e;
            double v = 0.0;
            // the columns of this thread, kCols of them requested at once
#pragma unroll 1
            for (int left = (int)((d - row0 + kRows - 1) / kRows); left > 0; left -= kCols) {
                float x[kCols], w[kCols];
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    x[c] = w[c] = 0.f;
                    if (c < left) {
                        x[c] = route_load(px + c * kRows);
                        w[c] = route_load(pw);
                    }
                    pw += w_step;
                }
                px += kCols * kRows;
#pragma unroll
                for (int c = 0; c < kCols; ++c) v = fma((double)x[c], (double)w[c], v);
            }
#pragma unroll
            for (int off = 16; off > 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            if (lane < 2) sums[warp * 2 + lane] = v;
            __syncthreads();
            if (threadIdx.x < 2) {
                double t = 0.0;
#pragma unroll
                for (int w = 0; w < kRouteWarps; ++w) t += sums[w * 2 + threadIdx.x];
                fixed[u * kMaxExperts + e] = t;
            }
            __syncthreads();
        }
    }
    for (int u = q + C * warp; u < ntok; u += C * kRouteWarps)
        if (open_s[u] != 0)
            route_decide64(fixed[u * kMaxExperts + lane], fixed[u * kMaxExperts + 32 + lane], g, lane,
                           fixed + (kRouteTokens + warp) * kMaxExperts, route + tok0 * 2 * g.slots, 1u << u);
    // (by the warp that has the fewest of them)
    if (warp == kRouteWarps - 1 && zeros_s != 0)
        route_decide64(0.0, 0.0, g, lane, fixed + (kRouteTokens + warp) * kMaxExperts, route + tok0 * 2 * g.slots,
                       zeros_s);
}

}  // namespace adafuse
