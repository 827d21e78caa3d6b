// types.h -- reading and writing elements of a runtime type (sl_dtype).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sparseloco_ops.h"

namespace sl {

__host__ __device__ inline int type_bytes(int32_t type) { return type == SL_F32 ? 4 : 2; }

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// Nearest bf16, ties to even; a NaN stays a (quiet) NaN.
__device__ __forceinline__ uint16_t to_bf16(float v) {
    const uint32_t u = __float_as_uint(v);
    if ((u & 0x7fffffffu) > 0x7f800000u) return (uint16_t)((u >> 16) | 0x40u);
    return (uint16_t)((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

__device__ __forceinline__ float load_value(const void* p, int32_t type, int64_t i) {
    if (type == SL_F32) return static_cast<const float*>(p)[i];
    if (type == SL_BF16) return bf16_value(static_cast<const uint16_t*>(p)[i]);
    return (float)static_cast<const _Float16*>(p)[i];
}

__device__ __forceinline__ void store_value(void* p, int32_t type, int64_t i, float v) {
    if (type == SL_F32)
        static_cast<float*>(p)[i] = v;
    else if (type == SL_BF16)
        static_cast<uint16_t*>(p)[i] = to_bf16(v);
    else
        static_cast<_Float16*>(p)[i] = (_Float16)v;
}

}  // namespace sl
