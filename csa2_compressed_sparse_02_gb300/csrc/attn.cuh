// What the attention kernels over pages share: the schedule's ranges, operand layouts and
// roundings, and the tensor map of a layer's rows.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include <atomic>

#include "pages.cuh"
#include "sm100.cuh"

namespace csa2 {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;

// The ranges: n = min(CTAs, items) of them, the first `total % n` one item longer.
struct Cut {
    int64_t base;
    int n, rem;
    __device__ __forceinline__ Cut(int64_t total, int ctas) {
        n = (int)min((int64_t)ctas, total);
        base = n ? total / n : 0;
        rem = n ? (int)(total - base * n) : 0;
    }
    __device__ __forceinline__ int64_t at(int c) const { return c * base + min(c, rem); }  // c = 0 .. n
    __device__ __forceinline__ int holder(int64_t item) const {
        const int64_t big = rem * (base + 1);
        return (int)(item < big ? item / (base + 1) : rem + (item - big) / base);
    }
};

// Sum over the warp, and with it the sum over the lanes before this one.
__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane) {
    uint32_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    return inc - v;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t sw128(int row, int unit) { return (uint32_t)(row * 128 + ((unit ^ (row & 7)) << 4)); }

__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"((uint16_t)v));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ uint32_t h2_sub(uint32_t x, uint32_t y) {
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
    return *reinterpret_cast<const uint32_t*>(&d);
}
// Four E5M2 of halves (x.lo, x.hi, y.lo, y.hi); E5M2 is the upper byte of f16.
__device__ __forceinline__ uint32_t h2x2_to_e5m2x4(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e5m2x2.f16x2 lo, %1;\n cvt.rn.satfinite.e5m2x2.f16x2 hi, %2;\n"
        " mov.b32 %0, {lo, hi};\n}"
        : "=r"(r)
        : "r"(x), "r"(y));
    return r;
}

// SMs of the current device, asked for once a device. 0: no device.
inline int sm_count() {
    static std::atomic<int> sms[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
    int n = dev < 64 ? sms[dev].load(std::memory_order_relaxed) : 0;
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        if (dev < 64) sms[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// The layer's rows as a 2-d tensor map, whose boxes are box_rows rows x 128 bytes, laid out in
// the 128-byte swizzle of the MMA operands. The driver's encoder is looked up once.
inline int encode_rows(const char* name, const Pages& g, const uint8_t* base, int box_rows, CUtensorMap* m) {
    using Encode = decltype(&cuTensorMapEncodeTiled);
    static Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return fail(CSA2_ERR_CUDA, std::string(name) + ": the driver has no cuTensorMapEncodeTiled");
    const bool bf16 = g.row_bytes == 2 * kD;
    const cuuint64_t dims[2] = {kD, (cuuint64_t)g.n_pages * g.page_size};
    const cuuint64_t strides[1] = {(cuuint64_t)g.row_bytes};
    const cuuint32_t box[2] = {bf16 ? 64u : 128u, (cuuint32_t)box_rows}, steps[2] = {1, 1};
    if (encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
               const_cast<uint8_t*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return fail(CSA2_ERR_CUDA, std::string(name) + ": tensor map of the pool");
    return CSA2_OK;
}

}  // namespace attn
}  // namespace csa2
