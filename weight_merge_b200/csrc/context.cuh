// context.cuh -- the context behind the C ABI and the host helpers its
// translation units share: error text, device guard, alignment, launch limits.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>
#include <vector>

#include "adafuse.h"
#include "common.cuh"

struct adafuse_ctx {
    int device = 0;
    int sm_count = 0;
    int32_t n_layers = 0, n_targets = 0, n_experts = 0, rank = 0;
    float alpha = 0.f, scale = 0.f;
    int64_t n_tiles = 0;
    std::vector<int64_t> layer_tile_begin;  // [n_layers + 1]
    adafuse::PairDesc* d_pairs = nullptr;
    adafuse::TileEntry* d_tiles = nullptr;
    int32_t* d_status = nullptr;
    CUtensorMap* d_maps = nullptr;  // kMapsPerPair per pair when the tensor-core kernel can run
    bool blk = false;               // those maps are blocked (every weight's in % 64 == 0)
    int tc_kp = 0;                  // its padded rank (16, 32, 64), 0 = not eligible
    int kernel = ADAFUSE_KERNEL_AUTO;
    std::vector<adafuse::PairDesc> h_pairs;  // host copy of d_pairs (re-base pointers are patched in)
    CUtensorMap* d_w0_maps = nullptr;  // 1 per pair on the re-base source W0
    bool has_base = false;
    int stall_at = 0;  // test hook: the next tensor-core launch stalls at each CTA's n-th tile
    std::atomic<int> stall_product{0};  // test hook: the n-th launch of the next product stalls
    // pair kernel: 256 x 128 blocks, layer-major like the tile table
    adafuse::TileEntry* d_blocks = nullptr;
    uint16_t* d_bpad = nullptr;              // rank < 8: B with rows zero-padded to 8
    uint16_t* d_fold = nullptr;              // rank <= 8: folded-coefficient operands
                                             // (allocated on first use, see ensure_fold)
    bool fold_failed = false;                // that allocation failed: the kernel is off
    float* d_logits = nullptr;               // [kMaxBatchTokens, E] batch pre-gate scratch
    unsigned long long* d_sched = nullptr;   // [2] ticket counter of the dynamic tile schedule
    int schedule = ADAFUSE_SCHEDULE_AUTO;
    std::vector<int64_t> layer_block_begin;  // [n_layers + 1]
    int pair_clusters = 0;                   // co-resident CTA pairs (0 = not queried yet)
    int max_ctas = 0;                        // cap on a switch's persistent grid (0 = none)
};

namespace adafuse {

// Records the CUDA error for adafuse_last_error and returns ADAFUSE_ERR_CUDA.
int cuda_fail(cudaError_t e, const char* what);

// Restores the caller's current device on scope exit.
struct DeviceGuard {
    int prev = -1;
    bool ok = false, moved = false;
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
        if (prev == dev) {
            ok = true;
        } else {
            ok = cudaSetDevice(dev) == cudaSuccess;
            moved = prev >= 0;
        }
    }
    ~DeviceGuard() {
        if (moved) cudaSetDevice(prev);
    }
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The driver's tensor-map encoder, looked up once (null when it is missing).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled_fn() {
    static const EncodeTiledFn fn = []() -> EncodeTiledFn {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(ptr);
        return nullptr;
    }();
    return fn;
}

// Raise a kernel's dynamic shared-memory limit only when this device has not
// been given at least `bytes` for that kernel yet (the host call is not free,
// and the decode-time pre-gate launches are short).  Keyed by the kernel's
// address and the device: kernels of one signature are different entries.
struct SmemAttrEntry {
    const void* fn;
    int device;
    size_t bytes;
};

template <typename Kernel>
void ensure_smem_attr(Kernel kernel, size_t bytes, int device) {
    static std::mutex mu;
    static std::vector<SmemAttrEntry> done;
    const void* fn = reinterpret_cast<const void*>(kernel);
    std::lock_guard<std::mutex> lk(mu);
    for (const SmemAttrEntry& en : done)
        if (en.fn == fn && en.device == device && en.bytes >= bytes) return;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) !=
        cudaSuccess)
        return;   // the launch reports the error
    for (SmemAttrEntry& en : done)
        if (en.fn == fn && en.device == device) {
            en.bytes = bytes;
            return;
        }
    try {
        done.push_back({fn, device, bytes});
    } catch (...) {
        // not remembered: the next launch sets the attribute again
    }
}

}  // namespace adafuse
