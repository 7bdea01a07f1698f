// Runs of 8 columns of a bf16 or binary32 row, as binary32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.hpp"

namespace tsl {

typedef float f32x8 __attribute__((ext_vector_type(8)));

// 8 consecutive columns col .. col + 7 of a row (element type by `bf`),
// zero past n.  VEC: the run is 16-byte aligned, so a whole one takes wide
// loads; otherwise, and for the run that crosses n, one element at a time.
template <bool VEC>
__device__ __forceinline__ f32x8 load8(const void *row, bool bf, int64_t col, int64_t n) {
    f32x8 v = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (col >= n)
        return v;
    if (VEC && col + 8 <= n) {
        if (bf) {
            const u32x4 w = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(row) + col);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = bf16_lo(w[i]);
                v[2 * i + 1] = bf16_hi(w[i]);
            }
        } else {
            const f32x4 *p = reinterpret_cast<const f32x4 *>(static_cast<const float *>(row) + col);
            const f32x4 a = p[0], b = p[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = a[i];
                v[4 + i] = b[i];
            }
        }
        return v;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (col + i < n)
            v[i] = bf ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(row)[col + i] << 16)
                      : static_cast<const float *>(row)[col + i];
    return v;
}

template <bool VEC>
__device__ __forceinline__ void store8(void *row, bool bf, int64_t col, int64_t n, f32x8 v) {
    if (col >= n)
        return;
    if (VEC && col + 8 <= n) {
        if (bf) {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(row) + col) = w;
        } else {
            f32x4 *p = reinterpret_cast<f32x4 *>(static_cast<float *>(row) + col);
            p[0] = f32x4{v[0], v[1], v[2], v[3]};
            p[1] = f32x4{v[4], v[5], v[6], v[7]};
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (col + i < n) {
            if (bf) {
                __bf16 h = (__bf16)v[i];
                static_cast<uint16_t *>(row)[col + i] = __builtin_bit_cast(uint16_t, h);
            } else {
                static_cast<float *>(row)[col + i] = v[i];
            }
        }
}

} // namespace tsl
