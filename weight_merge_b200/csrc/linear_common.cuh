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

__device__ __forceinline__ float apply_act(float v, int act) {
    switch (act) {
        case ADAFUSE_ACT_RELU: return v < 0.f ? 0.f : v;   // keeps NaN
        case ADAFUSE_ACT_GELU: return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
        case ADAFUSE_ACT_GELU_TANH:
            return 0.5f * v * (1.f + tanhf(0.79788456080286536f * (v + 0.044715f * v * v * v)));
        case ADAFUSE_ACT_SILU: return v / (1.f + expf(-v));
        default: return v;
    }
}

// One element of y: v is the finished product (bias not yet added).
__device__ __forceinline__ void store_one(const LinearParams& p, int64_t t, int o, float v) {
    if (p.bias != nullptr) v += __ldg(p.bias + o);
    v = apply_act(v, p.act);
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

// Slot j of token t's record: false for an empty or bad slot; a bad one sets
// its bits in *bad.
__device__ __forceinline__ bool route_slot(const int32_t* routes, int slots, int E, int64_t t, int j,
                                           int& e, float& gate, int& bad) {
    const int32_t* rec = routes + t * 2 * slots;
    e = __ldg(rec + j);
    gate = __int_as_float(__ldg(rec + slots + j));
    if (e == -1) return false;
    if (e < -1 || e >= E) { bad |= ADAFUSE_STATUS_BAD_EXPERT; return false; }
    if (!isfinite(gate)) { bad |= ADAFUSE_STATUS_BAD_GATE; return false; }
    return true;
}

}  // namespace adafuse
