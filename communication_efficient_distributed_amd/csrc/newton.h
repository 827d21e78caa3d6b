// newton.h -- what the two ways of the matrix update share: values of the
// matrix that is orthogonalised, its norm, fp16 pairs.
#pragma once

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_internal.h"
#include "types.h"
#include "wave.h"

namespace sl {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef _Float16 half2 __attribute__((ext_vector_type(2)));
typedef float float16v __attribute__((ext_vector_type(16)));

// u of one element, before normalisation.
struct Source {
    const void* x;
    int32_t type;
    int64_t ld, stride;
    float* momentum;  // null: u = x
    float grad_scale, decay;
    bool nesterov;
};

__device__ __forceinline__ float momentum_next(float g, float m, float decay) { return __builtin_fmaf(decay, m, g); }

__device__ __forceinline__ double block_sum(double v, double* lds) {
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    if (lane_id() == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0;
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) s += lds[w];
    __syncthreads();
    return s;
}

// Multiplies by a factor that may itself be beyond fp32's range.
struct Scale {
    float mantissa;
    int exponent;
    __device__ __forceinline__ float operator()(float v) const { return ldexpf(v, exponent) * mantissa; }
};

// to / (|u|_F + eps) of matrix i from its partial sums of squares, 0 if that
// would divide by zero.  Called by every thread of a block; lds: one double
// for each wavefront.
__device__ __forceinline__ Scale start_scale(float to, const double* partial, int n_partial, int64_t i, float eps, double* lds) {
    double acc = 0;
    for (int k = threadIdx.x; k < n_partial; k += blockDim.x) acc += partial[i * n_partial + k];
    const double norm = sqrt(block_sum(acc, lds)) + (double)eps;
    const double scale = norm > 0 ? (double)to / norm : 0;
    const int e = scale > 0 ? ilogb(scale) : 0;
    return {(float)ldexp(scale, -e), e};
}

// Copies 16 bytes per lane from global memory to LDS, lane l's to lds + 16 l.
// In assembler because the compiler makes later LDS reads wait for such copies
// where it cannot tell the stages apart; arrive() waits for those that matter.
// No register is written, and m0 (the LDS address) needs one wait state before
// its use.
__device__ __forceinline__ void load_to_lds(const _Float16* src, _Float16* lds) {
    const uint32_t to = uniform((uint32_t)(uintptr_t)(__attribute__((address_space(3))) _Float16*)lds);
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(to) : "memory", "m0");
}

// Waits until the wavefront's loads have landed and its LDS reads are done,
// then for the other wavefronts of the block.
__device__ __forceinline__ void arrive() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ __forceinline__ void split_half(float v, _Float16* hi, _Float16* lo) {
    *hi = (_Float16)v;
    *lo = (_Float16)(v - (float)*hi);
}

// The update of long matrices whose shorter side is at most kNarrow, by way of
// the Gram matrix alone; false products only.  partial: n_partial partial sums of
// squares for each matrix.
constexpr int64_t kNarrow = 128;
bool is_narrow(const UpdateArgs& u);
size_t narrow_workspace_bytes(int64_t rows, int64_t cols, int64_t count);
hipError_t launch_narrow(const UpdateArgs& u, const Source& s, const double* partial, int n_partial, void* workspace,
                         hipStream_t stream);

}  // namespace sl
