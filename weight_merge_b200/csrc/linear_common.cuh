// linear_common.cuh -- what the product kernels share: launch parameters, the
// epilogue y = residual + mul * act(v + bias), and route records of 2, 4 or 8
// slots.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace adafuse {

struct LinearParams {
    const uint16_t* x;    // [T, in] bf16, rows ldx apart
    const uint16_t* W;    // [out, in] bf16
    const float* bias;    // [out] or null
    const void* mul;      // [T, out] io type or null
    const void* res;      // [T, out] io type or null
    void* y;              // [T, out] io type
    int64_t T, ldx, ldmul, ldres, ldy;
    int out, in;
    int act;
    int f32;              // io type: 1 fp32, 0 bf16
    // routed products only
    const uint16_t* A;    // [E, r, in]
    const uint16_t* B;    // [E, out, r]
    const int32_t* routes;
    int slots, E, r;
    float s;
    int32_t* status;
};

__device__ __forceinline__ float bf16_bits_to_float(uint32_t b) { return __uint_as_float(b << 16); }

// GELU in forms that keep their digits where it is small: 1 + erf and 1 + tanh
// cancel for negative v (three digits left at -4, none from -5.5 on).
//
// erf form: v (1 - h) for v >= 0 and v h below, h = erfc(|v| / sqrt 2) / 2.  h =
// e^(-v^2 / 2) t p(t) with t = 1 / (1 + 0.3 |v|): h e^(v^2 / 2) falls like 1 / |v|,
// so t takes [0, inf) to (0, 1] and p is smooth there.  p: least squares on the
// relative error, reweighted until its peaks were level (1.5e-7; over |v| <= 14).
// In all 1.5 v^2 + 16 units of 2^-24, most of it from rounding v^2.  (erfcf: T = 4096,
// 4096 -> 14336 fp32 9% more time.)
__device__ __forceinline__ float act_gelu(float v) {
    const float t = __fdividef(1.f, fmaf(0.3f, fabsf(v), 1.f));
    float p = 0.0356770121f;
    p = fmaf(p, t, -0.157212824f);
    p = fmaf(p, t, 0.206370935f);
    p = fmaf(p, t, -0.0537002124f);
    p = fmaf(p, t, 0.128570631f);
    p = fmaf(p, t, 0.0999106988f);
    p = fmaf(p, t, 0.120754413f);
    p = fmaf(p, t, 0.119629271f);
    const float h = p * t * exp2f(v * v * -0.721347520f);
    return v * (v < 0.f ? h : 1.f - h);
}
// tanh form: v / (1 + e^w), w = -2 sqrt(2 / pi) (v + 0.044715 v^3).
__device__ __forceinline__ float act_gelu_tanh(float v) {
    return __fdividef(v, 1.f + exp2f(v * fmaf(v * v, -0.102943240f, -2.30220820f)));
}
__device__ __forceinline__ float act_silu(float v) { return v / (1.f + expf(-v)); }

// The activation on N values, the choice made once: a choice per value would
// lay out every activation N times, and the epilogues would run from a cold
// instruction cache (34 us for one 256 x 256 tile).
template <int N>
__device__ __forceinline__ void apply_act(float (&v)[N], int act) {
    switch (act) {
        case ADAFUSE_ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];   // keeps NaN
            break;
        case ADAFUSE_ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = act_gelu(v[i]);
            break;
        case ADAFUSE_ACT_GELU_TANH:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = act_gelu_tanh(v[i]);
            break;
        case ADAFUSE_ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = act_silu(v[i]);
            break;
        default: break;
    }
}

// One element of y: v is the finished product (bias not yet added).
__device__ __forceinline__ void store_one(const LinearParams& p, int64_t t, int o, float v) {
    if (p.bias != nullptr) v += p.bias[o];
    float one[1] = {v};
    apply_act(one, p.act);
    v = one[0];
    if (p.f32) {
        if (p.mul != nullptr) v *= static_cast<const float*>(p.mul)[t * p.ldmul + o];
        if (p.res != nullptr) v += static_cast<const float*>(p.res)[t * p.ldres + o];
        static_cast<float*>(p.y)[t * p.ldy + o] = v;
    } else {
        if (p.mul != nullptr)
            v *= bf16_bits_to_float(static_cast<const uint16_t*>(p.mul)[t * p.ldmul + o]);
        if (p.res != nullptr)
            v += bf16_bits_to_float(static_cast<const uint16_t*>(p.res)[t * p.ldres + o]);
        static_cast<__nv_bfloat16*>(p.y)[t * p.ldy + o] = __float2bfloat16_rn(v);
    }
}

// Eight consecutive values of a [T, out] operand from o (a multiple of 8).
__device__ __forceinline__ void load8(const void* base, int64_t at, int f32, float* w) {
    if (f32) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
        const float4 a = q[0], b = q[1];
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[2 * i] = __uint_as_float(u[i] << 16);
            w[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
}

// The factor and the residual of N consecutive columns from o for token t, as
// 16-byte vectors (columns from p.out on are left out; o and N multiples of 8).
template <int N>
struct SideCols {
    float mul[N], res[N];
    __device__ __forceinline__ void load(const LinearParams& p, int64_t t, int o) {
        if (p.mul != nullptr) {
#pragma unroll
            for (int j = 0; j < N; j += 8)
                if (o + j < p.out) load8(p.mul, t * p.ldmul + o + j, p.f32, &mul[j]);
        }
        if (p.res != nullptr) {
#pragma unroll
            for (int j = 0; j < N; j += 8)
                if (o + j < p.out) load8(p.res, t * p.ldres + o + j, p.f32, &res[j]);
        }
    }
};

// Those columns of y from the finished product v: one rounding, 16-byte stores.
template <int N>
__device__ __forceinline__ void finish_cols(const LinearParams& p, int64_t t, int o, float (&v)[N],
                                            const SideCols<N>& side) {
    if (p.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (o + i < p.out) v[i] += p.bias[o + i];
    }
    apply_act(v, p.act);
    if (p.mul != nullptr) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= side.mul[i];
    }
    if (p.res != nullptr) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += side.res[i];
    }
    if (p.f32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p.y) + t * p.ldy + o);
#pragma unroll
        for (int j = 0; j < N; j += 8)
            if (o + j < p.out) {
                q[j / 4] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                q[j / 4 + 1] = make_float4(v[j + 4], v[j + 5], v[j + 6], v[j + 7]);
            }
    } else {
        uint4* q = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y) + t * p.ldy + o);
#pragma unroll
        for (int j = 0; j < N; j += 8)
            if (o + j < p.out) {
                uint32_t u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(v[j + 2 * i], v[j + 2 * i + 1]);
                    u[i] = *reinterpret_cast<const uint32_t*>(&b);
                }
                q[j / 8] = make_uint4(u[0], u[1], u[2], u[3]);
            }
    }
}

// A warp's 32 tokens x 16 columns of y from the finished products.  v: lane =
// token.  Stored from there, a warp's 16-byte pieces would fall into 32 rows and
// half of each 32-byte sector (a 256 x 240 fp32 tile took 10 us longer); so the
// block turns through `turn`, 2 KB of the warp's own shared memory whose 16-byte
// pieces are permuted against bank conflicts, and leaves in pieces that lie next
// to each other: F32: 4 lanes a token, 4 columns each, 4 times 8 tokens;
// otherwise 2 lanes, 8 columns, twice 16 tokens.
template <bool F32>
struct BlockSide {
    static constexpr int kIters = F32 ? 4 : 2, kCols = F32 ? 4 : 8;
    // the factor ahead of its use for bf16 only: in fp32, the rarer case, its
    // registers would spill
    float mul[F32 ? 1 : kIters][kCols], res[kIters][kCols];
};

__device__ __forceinline__ void load_cols(const void* base, int64_t at, float (&w)[4]) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
}
__device__ __forceinline__ void load_cols(const void* base, int64_t at, float (&w)[8]) {
    load8(base, at, 0, w);
}

// Requests the factor and the residual of the block at token tok0, column col0.
template <bool F32>
__device__ __forceinline__ void load_block(const LinearParams& p, int64_t tok0, int col0, int lane,
                                           BlockSide<F32>& side) {
    using S = BlockSide<F32>;
    constexpr int kLanes = 16 / S::kCols;
    const int col = col0 + lane % kLanes * S::kCols;
#pragma unroll
    for (int j = 0; j < S::kIters; ++j) {
        const int64_t t = tok0 + lane / kLanes + j * (32 / kLanes);
        if (t < p.T && col < p.out) {
            if (!F32 && p.mul != nullptr) load_cols(p.mul, t * p.ldmul + col, side.mul[F32 ? 0 : j]);
            if (p.res != nullptr) load_cols(p.res, t * p.ldres + col, side.res[j]);
        }
    }
}

template <bool F32>
__device__ __forceinline__ void finish_block(const LinearParams& p, int64_t tok0, int col0, int lane,
                                             const float (&v)[16], const BlockSide<F32>& side, uint8_t* turn) {
    using S = BlockSide<F32>;
    constexpr int kLanes = 16 / S::kCols;
    auto piece = [&](int row, int c) {   // the 16-byte piece of columns 4c .. 4c + 3
        return turn + row * 64 + ((c ^ (row >> 1 & 3)) << 4);
    };
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<float4*>(piece(lane, c)) = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    __syncwarp();
    const int col = col0 + lane % kLanes * S::kCols;
    float bias[S::kCols];
    if (p.bias != nullptr && col < p.out) {
#pragma unroll
        for (int i = 0; i < S::kCols; ++i) bias[i] = p.bias[col + i];
    }
    float w[S::kIters * S::kCols];
#pragma unroll
    for (int j = 0; j < S::kIters; ++j)
#pragma unroll
        for (int c = 0; c < S::kCols / 4; ++c) {
            const float4 f = *reinterpret_cast<const float4*>(
                piece(lane / kLanes + j * (32 / kLanes), lane % kLanes * (S::kCols / 4) + c));
            w[j * S::kCols + 4 * c] = f.x;
            w[j * S::kCols + 4 * c + 1] = f.y;
            w[j * S::kCols + 4 * c + 2] = f.z;
            w[j * S::kCols + 4 * c + 3] = f.w;
        }
    __syncwarp();
    if (p.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < S::kIters * S::kCols; ++i) w[i] += bias[i % S::kCols];
    }
    apply_act(w, p.act);
#pragma unroll
    for (int j = 0; j < S::kIters; ++j) {
        const int64_t t = tok0 + lane / kLanes + j * (32 / kLanes);
        if (t >= p.T || col >= p.out) continue;
        float* o = &w[j * S::kCols];
        if (p.mul != nullptr) {
            float m[S::kCols];
            if constexpr (F32) load_cols(p.mul, t * p.ldmul + col, m);
#pragma unroll
            for (int i = 0; i < S::kCols; ++i) o[i] *= F32 ? m[i] : side.mul[F32 ? 0 : j][i];
        }
        if (p.res != nullptr) {
#pragma unroll
            for (int i = 0; i < S::kCols; ++i) o[i] += side.res[j][i];
        }
        if constexpr (F32) {
            *reinterpret_cast<float4*>(static_cast<float*>(p.y) + t * p.ldy + col) =
                make_float4(o[0], o[1], o[2], o[3]);
        } else {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y) + t * p.ldy + col) =
                make_uint4(u[0], u[1], u[2], u[3]);
        }
    }
}

// Slot j of token t's record: false for an empty or bad slot; a bad one sets
// its bits in *bad.
__device__ __forceinline__ bool route_slot(const int32_t* routes, int slots, int E, int64_t t, int j,
                                           int& e, float& gate, int& bad) {
    const int32_t* rec = routes + t * 2 * slots;
    e = rec[j];
    gate = __int_as_float(rec[slots + j]);
    if (e == -1) return false;
    if (e < -1 || e >= E) { bad |= ADAFUSE_STATUS_BAD_EXPERT; return false; }
    if (!isfinite(gate)) { bad |= ADAFUSE_STATUS_BAD_GATE; return false; }
    return true;
}

}  // namespace adafuse
