// linear_simple.cuh -- the products as plain shared-memory tiles in fp32.
#pragma once

#include "linear_common.cuh"

namespace adafuse {

constexpr int kSimpleTile = 64;
constexpr int kSimpleDepth = 32;

// acc[i][j] = sum_k x[t0 + 4 * ty + i][k] * w[o0 + 4 * tx + j][k]
__device__ __forceinline__ void simple_product(const uint16_t* x, int64_t ldx, int64_t T,
                                               const uint16_t* w, int64_t rows, int in, int64_t t0,
                                               int64_t o0, float (&acc)[4][4]) {
    __shared__ float xs[kSimpleDepth][kSimpleTile + 1], ws[kSimpleDepth][kSimpleTile + 1];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    for (int k0 = 0; k0 < in; k0 += kSimpleDepth) {
        for (int i = threadIdx.x; i < kSimpleTile * kSimpleDepth; i += 256) {
            const int k = i % kSimpleDepth, row = i / kSimpleDepth;
            const bool kin = k0 + k < in;
            xs[k][row] = kin && t0 + row < T ? bf16_bits_to_float(x[(t0 + row) * ldx + k0 + k]) : 0.f;
            ws[k][row] = kin && o0 + row < rows ? bf16_bits_to_float(w[(o0 + row) * in + k0 + k]) : 0.f;
        }
        __syncthreads();
#pragma unroll 8
        for (int k = 0; k < kSimpleDepth; ++k) {
            float a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) { a[i] = xs[k][4 * ty + i]; b[i] = ws[k][4 * tx + i]; }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
    }
}

// z = x A^T over all E * r rows of the stacked A.
__global__ void __launch_bounds__(256) simple_down_kernel(const LinearParams p) {
    const int64_t t0 = (int64_t)blockIdx.y * kSimpleTile, o0 = (int64_t)blockIdx.x * kSimpleTile;
    const int64_t rows = (int64_t)p.E * p.r;
    float acc[4][4];
    simple_product(p.x, p.ldx, p.T, p.A, rows, p.in, t0, o0, acc);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t t = t0 + 4 * ty + i, o = o0 + 4 * tx + j;
            if (t < p.T && o < rows) p.z[t * rows + o] = acc[i][j];
        }
}

__global__ void __launch_bounds__(256) simple_linear_kernel(const LinearParams p) {
    const int64_t t0 = (int64_t)blockIdx.y * kSimpleTile, o0 = (int64_t)blockIdx.x * kSimpleTile;
    float acc[4][4];
    simple_product(p.x, p.ldx, p.T, p.W, p.out, p.in, t0, o0, acc);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int bad = 0;
    for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + 4 * ty + i;
        if (t >= p.T) continue;
        for (int j = 0; j < 4; ++j) {
            const int64_t o = o0 + 4 * tx + j;
            if (o >= p.out) continue;
            float v = acc[i][j];
            if (p.routes != nullptr)
                for (int q = 0; q < p.slots; ++q) {
                    int e;
                    float g;
                    if (!route_slot(p.routes, p.slots, p.E, t, q, e, g, bad)) continue;
                    float u = 0.f;
                    for (int k = 0; k < p.r; ++k)
                        u = fmaf(p.z[t * p.E * p.r + e * p.r + k],
                                 bf16_bits_to_float(p.B[((int64_t)e * p.out + o) * p.r + k]), u);
                    v = fmaf(p.s * g, u, v);
                }
            store_one(p, t, (int)o, v);
        }
    }
    if (bad != 0) atomicOr(p.status, bad);
}

}  // namespace adafuse
