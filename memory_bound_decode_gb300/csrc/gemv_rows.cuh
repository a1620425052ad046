// Groups of neighbouring values of a row: loads of FP32 and BF16 rows, stores as
// BF16 and as E4M3 codes.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "gemv_common.cuh"

namespace gemv {

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two values to E4M3 codes, to nearest, values past 448 to 448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// N values from column c of a row in FP32 or BF16, as they come.
template <int N, bool F32>
struct Cols {
    static constexpr int kWords = N == 1 ? 1 : 4;         // N values of a wide load take 16 bytes
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const char* row, int c) {
        if constexpr (N > 1) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + c * (F32 ? 4 : 2));
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (F32) {
            w[0] = reinterpret_cast<const uint32_t*>(row)[c];
        } else {
            w[0] = reinterpret_cast<const uint16_t*>(row)[c];
        }
    }
    __device__ __forceinline__ void values(float (&f)[N]) const {
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = __uint_as_float(w[i]);
        } else if constexpr (N > 1) {
            unpack8(make_uint4(w[0], w[1], w[2], w[3]), f);
        } else {
            f[0] = bf16_lo(w[0]);
        }
    }
};

template <int N>
__device__ __forceinline__ void store_bf16(void* row, int c, const float (&f)[N]) {
    uint16_t* d = static_cast<uint16_t*>(row) + c;
    if constexpr (N == 8)
        *reinterpret_cast<uint4*>(d) = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    else if constexpr (N == 4)
        *reinterpret_cast<uint2*>(d) = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
    else
        *d = static_cast<uint16_t>(pack2(f[0], 0.f));
}

// Codes of value / scale, the quotient in FP32: times the reciprocal where that is exact (a scale that is a power of
// two, the usual choice), else (inv = 0) by division.
template <int N>
__device__ __forceinline__ void store_fp8(void* row, int c, const float (&f)[N], float scale, float inv) {
    unsigned char* d = static_cast<unsigned char*>(row) + c;
    float x[N];
    if (inv != 0.f) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = f[i] * inv;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = __fdiv_rn(f[i], scale);
    }
    if constexpr (N == 8)
        *reinterpret_cast<uint2*>(d) = make_uint2(e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16,
                                                  e4m3x2(x[4], x[5]) | e4m3x2(x[6], x[7]) << 16);
    else if constexpr (N == 4)
        *reinterpret_cast<uint32_t*>(d) = e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16;
    else
        *d = static_cast<unsigned char>(e4m3x2(x[0], 0.f));
}

}  // namespace gemv
