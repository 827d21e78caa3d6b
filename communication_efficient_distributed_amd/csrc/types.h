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

// Four elements from i on, one aligned access.
__device__ __forceinline__ void load_values4(const void* p, int32_t type, int64_t i, float* v) {
    if (type == SL_F32) {
        const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        return;
    }
    const ushort4 q = *reinterpret_cast<const ushort4*>(static_cast<const uint16_t*>(p) + i);
    const uint16_t w[4] = {q.x, q.y, q.z, q.w};
    for (int e = 0; e < 4; ++e) v[e] = type == SL_BF16 ? bf16_value(w[e]) : (float)__builtin_bit_cast(_Float16, w[e]);
}

// Eight elements from i on, 16-byte aligned.
__device__ __forceinline__ void load_values8(const void* p, int32_t type, int64_t i, float* v) {
    if (type == SL_F32) {
        load_values4(p, type, i, v);
        load_values4(p, type, i + 4, v + 4);
        return;
    }
    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    for (int e = 0; e < 8; ++e) {
        const uint16_t h = (uint16_t)(w[e / 2] >> (e % 2 * 16));
        v[e] = type == SL_BF16 ? bf16_value(h) : (float)__builtin_bit_cast(_Float16, h);
    }
}

__device__ __forceinline__ void store_values4(void* p, int32_t type, int64_t i, const float* v) {
    if (type == SL_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
        return;
    }
    uint16_t w[4];
    for (int e = 0; e < 4; ++e) w[e] = type == SL_BF16 ? to_bf16(v[e]) : __builtin_bit_cast(uint16_t, (_Float16)v[e]);
    *reinterpret_cast<ushort4*>(static_cast<uint16_t*>(p) + i) = make_ushort4(w[0], w[1], w[2], w[3]);
}

}  // namespace sl
