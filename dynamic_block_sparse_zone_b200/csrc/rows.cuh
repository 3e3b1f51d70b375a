// rows.cuh -- what the row kernels (layer norm, 8-bit checkpoints) share: row
// addressing, element types, and the 8-bit code of a group of 32 channels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "prism_internal.cuh"

namespace prism {
namespace rows {

constexpr int kGroup = 32;  // channels that share one scale of a checkpoint

// Row r of a prism_rows: group r / group, row r % group in it.
struct RowPtr {
    char *data;
    long long stride, group_stride;  // bytes
    unsigned group;                  // 0: one group
    __device__ __forceinline__ char *operator()(long long r) const {
        if (group == 0) return data + r * stride;
        const unsigned q = (unsigned)r / group;  // with groups, rows < 2^31 (checked on the host)
        return data + (long long)q * group_stride + (long long)((unsigned)r - q * group) * stride;
    }
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

// VEC elements moved as one access (16 bytes, or 1 element).
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

// A weight of type prism_dtype `dt` as fp32.
__device__ __forceinline__ float weight_at(const void *p, int dt, long long c) {
    if (dt == PRISM_FP32) return static_cast<const float *>(p)[c];
    if (dt == PRISM_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[c]);
    return __half2float(static_cast<const __half *>(p)[c]);
}
__device__ __forceinline__ void weight_store(void *p, int dt, long long c, float x) {
    if (dt == PRISM_FP32) static_cast<float *>(p)[c] = x;
    else if (dt == PRISM_BF16) static_cast<__nv_bfloat16 *>(p)[c] = __float2bfloat16_rn(x);
    else static_cast<__half *>(p)[c] = __float2half_rn(x);
}

// ---- the 8-bit code ----
// A group's values are q * 2^k, k the least integer >= -127 with max|x| <=
// qmax * 2^k (qmax = 127 for int8, 448 for e4m3), q = x * 2^-k to the nearest
// code, ties to even.  Scaling by a power of two is exact, so the code does
// not depend on how it is computed, and q * 2^k (at most 7 significant bits)
// is a bf16 value down to bf16's smallest.  The scale byte is k + 127; 255
// marks a group that holds an infinity or a NaN (it reads back as NaN).
__device__ __forceinline__ int code_exponent(float amax, int fmt) {
    const uint32_t u = __float_as_uint(amax);  // amax >= 0
    if (u >= 0x7f800000u) return 128;
    const int ex = (int)(u >> 23) - 127;
    const uint32_t mant = u & 0x7fffffu;
    // 127 = 1.984375 * 2^6, 448 = 1.75 * 2^8
    const int k = fmt == PRISM_CKPT_INT8 ? ex - 6 + (mant > 0x7e0000u) : ex - 8 + (mant > 0x600000u);
    return k < -127 ? -127 : k;
}
// 2^-k for k in [-127, 126]
__device__ __forceinline__ float code_inv_scale(int k) { return __uint_as_float((uint32_t)(127 - k) << 23); }
// 2^k of a scale byte
__device__ __forceinline__ float code_scale(uint32_t byte) {
    if (byte == 255u) return __uint_as_float(0x7fc00000u);
    return byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}
// The largest finite value: a code may stand for a little more than it.
template <typename T>
__device__ __forceinline__ float largest();
template <>
__device__ __forceinline__ float largest<float>() { return 3.402823466e38f; }
template <>
__device__ __forceinline__ float largest<__nv_bfloat16>() { return __uint_as_float(0x7f7f0000u); }
template <>
__device__ __forceinline__ float largest<__half>() { return 65504.f; }
template <typename T>
__device__ __forceinline__ float saturate_to(float v) {  // NaN stays NaN
    return fabsf(v) > largest<T>() ? copysignf(largest<T>(), v) : v;
}
// A group with k = 128 (not finite) is given codes of 0.
__device__ __forceinline__ uint8_t encode1(float x, float inv, int fmt) {
    const float y = x * inv;
    if (fmt == PRISM_CKPT_INT8) return (uint8_t)(int8_t)__float2int_rn(y);
    return (uint8_t)__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float decode1(uint8_t code, int fmt) {
    if (fmt == PRISM_CKPT_INT8) return (float)(int8_t)code;
    const __half_raw h = __nv_cvt_fp8_to_halfraw(code, __NV_E4M3);
    return __half2float(__half(h));
}

// ---- launchers (arguments checked by the caller) ----
struct NormFwd {
    RowPtr x, y;
    const void *gamma, *beta;  // may be NULL
    int wdt;
    float *mean, *rstd;
    uint8_t *codes, *scales;  // x's checkpoint; may be NULL
    int fmt;
    long long nrows;
    int C;
    float eps;
};
struct NormBwd {
    RowPtr x;                       // or the checkpoint of x:
    const uint8_t *codes, *scales;  // non-NULL
    int fmt;
    RowPtr dy, dx;
    const void *gamma;  // may be NULL
    int wdt;
    const float *mean, *rstd;
    void *dgamma, *dbeta;  // may be NULL
    float *part;           // norm_bwd_workspace bytes
    long long nrows;
    int C;
};

}  // namespace rows

prism_status launch_norm_fwd(const rows::NormFwd &a, int dtype, cudaStream_t st);
prism_status launch_norm_bwd(const rows::NormBwd &a, int dtype, cudaStream_t st);
size_t norm_bwd_workspace(long long nrows, int C);
prism_status launch_ckpt_pack(const rows::RowPtr &x, int dtype, long long nrows, int C, const prism_ckpt &k,
                              cudaStream_t st);
prism_status launch_ckpt_unpack(const prism_ckpt &k, const rows::RowPtr &y, int dtype, long long nrows, int C,
                                cudaStream_t st);

}  // namespace prism
