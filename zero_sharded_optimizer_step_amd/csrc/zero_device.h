// zero_device.h -- device helpers shared by the HIP sources: the 16-bit
// formats, the block reduction and AdamW's arithmetic on one element.  Not
// part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include "zero_internal.h"

namespace zero {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------- formats
// bf16 is the upper half of an fp32; fp16 goes through the hardware convert,
// which is exact (every fp16 value, subnormals included, is an fp32 value).
template <int DT>
__device__ __forceinline__ float lo_to_f32(unsigned w) {
    if constexpr (DT == ZERO_BF16) return __uint_as_float(w << 16);
    else return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<unsigned short>(w & 0xffffu)));
}
template <int DT>
__device__ __forceinline__ float hi_to_f32(unsigned w) {
    if constexpr (DT == ZERO_BF16) return __uint_as_float(w & 0xffff0000u);
    else return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<unsigned short>(w >> 16)));
}
template <int DT>
__device__ __forceinline__ void decode4(const u32x2 v, float o[4]) {
    o[0] = lo_to_f32<DT>(v.x); o[1] = hi_to_f32<DT>(v.x);
    o[2] = lo_to_f32<DT>(v.y); o[3] = hi_to_f32<DT>(v.y);
}

// Round to nearest even with the gfx950 packed converts (v_cvt_pk_bf16_f32,
// v_cvt_pk_f16_f32).
template <int DT>
__device__ __forceinline__ unsigned pack2(float a, float b) {
    f32x2 v = {a, b};
    if constexpr (DT == ZERO_BF16) return __builtin_bit_cast(unsigned, __builtin_convertvector(v, bf16x2));
    else return __builtin_bit_cast(unsigned, __builtin_convertvector(v, f16x2));
}
template <int DT>
__device__ __forceinline__ unsigned short pack1(float a) {
    return static_cast<unsigned short>(pack2<DT>(a, 0.0f) & 0xffffu);
}

__device__ __forceinline__ bool finite(float x) { return __builtin_isfinite(x); }

// ------------------------------------------------------- block reduction
// Fixed shuffle pattern and fixed wave order: the block's result depends
// only on which values its threads hold, never on timing.  Thread 0 ends
// with the block's total.
template <int THREADS>
__device__ __forceinline__ void block_reduce(double& ss, int& bad) {
    #pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        ss += __shfl_xor(ss, off, 64);
        bad |= __shfl_xor(bad, off, 64);
    }
    if constexpr (THREADS > 64) {
        __shared__ double s_ss[THREADS / 64];
        __shared__ int s_bad[THREADS / 64];
        const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
        if (lane == 0) { s_ss[wave] = ss; s_bad[wave] = bad; }
        __syncthreads();
        if (threadIdx.x == 0) {
            ss = s_ss[0];
            bad = s_bad[0];
            for (int w = 1; w < THREADS / 64; ++w) { ss += s_ss[w]; bad |= s_bad[w]; }
        }
    }
}

// One element, in fp32 with one rounding per operation (no contraction):
//   m' = b1 m + c1 g;  v' = b2 v + c2 g^2;  d = sqrt(v') * inv_sqrt_bc2 + eps;
//   p' = p * decay - step_size * (m' / d),
// with the per-step constants inv_sqrt_bc2 = 1 / sqrt(1 - b2^t),
// decay = 1 - lr wd and step_size = lr / (1 - b1^t), each rounded once to
// fp32 on the host.
__device__ __forceinline__ void adamw1(float g, float& p, float& m, float& v, const AdamConsts& k) {
    m = k.b1 * m + k.c1 * g;
    v = k.b2 * v + k.c2 * (g * g);
    const float d = __builtin_sqrtf(v) * k.inv_sqrt_bc2 + k.eps;
    p = p * k.decay - k.step_size * (m / d);
}

}  // namespace
}  // namespace zero
