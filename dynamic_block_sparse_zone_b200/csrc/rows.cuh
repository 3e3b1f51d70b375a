// rows.cuh -- what the row kernels (layer norm, 8-bit checkpoints) share: row
// addressing, element types, and the 8-bit code of a group of 32 channels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include <type_traits>

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
// 2^-k for k in [-127, 126]; 0 for k = 128 (a group that is not finite: its
// codes say nothing)
__device__ __forceinline__ float code_inv_scale(int k) { return k == 128 ? 0.f : __uint_as_float((uint32_t)(127 - k) << 23); }
// 2^k of a scale byte
__device__ __forceinline__ float code_scale(uint32_t byte) {
    const uint32_t u = max(byte << 23, 0x00400000u);  // 2^-127 is no normal number
    return __uint_as_float(byte == 255u ? 0x7fc00000u : u);
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

// ---- packed fp32 pairs (f32x2 arithmetic): one instruction for two values ----
// The row kernels would be bound by instruction issue before HBM with one
// instruction per value; with VEC = 1 the upper half idles.
using f2 = uint64_t;
__device__ __forceinline__ f2 make2(float lo, float hi) {
    return (f2)__float_as_uint(lo) | ((f2)__float_as_uint(hi) << 32);
}
__device__ __forceinline__ f2 both(float v) { return make2(v, v); }
__device__ __forceinline__ float low(f2 v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float high(f2 v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// two neighbouring elements in one word <-> a pair
template <typename T>
__device__ __forceinline__ f2 widen(uint32_t w);
template <>
__device__ __forceinline__ f2 widen<__nv_bfloat16>(uint32_t w) { return (f2)(w << 16) | ((f2)(w & 0xffff0000u) << 32); }
template <>
__device__ __forceinline__ f2 widen<__half>(uint32_t w) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return make2(f.x, f.y);
}
template <typename T>
__device__ __forceinline__ uint32_t narrow(f2 v);
template <>
__device__ __forceinline__ uint32_t narrow<__nv_bfloat16>(f2 v) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(low(v), high(v));
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t narrow<__half>(f2 v) {
    const __half2 h = __floats2half2_rn(low(v), high(v));
    return *reinterpret_cast<const uint32_t *>(&h);
}

// cp.async of a thread's own bytes into its own shared-memory slot (N = 4, 8 or
// 16, both sides aligned to N); a thread that has waited may read its slots.
template <int N>
__device__ __forceinline__ void copy_async(void *smem, const void *g) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(d), "l"(g) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(d), "l"(g), "n"(N) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
// all but the last N groups of this thread have landed
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

// A thread's piece of a row, VEC elements as VEC / 2 pairs: one 16-byte access,
// or (VEC = 2: rows of any alignment and length) two elements fetched one by
// one, of which the second may lie past the row's C channels.
template <typename T, int VEC>
struct Vec {
    static_assert(VEC * sizeof(T) == 16 || VEC == 2, "16-byte accesses, or pairs");
    // the two single elements stay apart until they are used: a fetch ahead must not wait for its data
    static constexpr int VP = VEC / 2, W = VEC == 2 ? 2 : VEC * sizeof(T) / 4;
    uint32_t w[W];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void set(const uint4 &u) { w[0] = u.x, w[1 % W] = u.y, w[2 % W] = u.z, w[3 % W] = u.w; }
    __device__ __forceinline__ void load(const char *row, long long v, long long C) {
        if constexpr (VEC == 2) {
            using E = typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type;
            const E *p = reinterpret_cast<const E *>(row) + 2 * v;
            w[0] = p[0];
            w[1] = 2 * v + 1 < C ? p[1] : 0;
        } else {
            set(reinterpret_cast<const uint4 *>(row)[v]);
        }
    }
    __device__ __forceinline__ void store(char *row, long long v, long long C) const {
        if constexpr (VEC == 2) {
            using E = typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type;
            E *p = reinterpret_cast<E *>(row) + 2 * v;
            p[0] = (E)w[0];
            if (2 * v + 1 < C) p[1] = (E)w[1];
        } else {
            reinterpret_cast<uint4 *>(row)[v] = make_uint4(w[0], w[1 % W], w[2 % W], w[3 % W]);
        }
    }
    __device__ __forceinline__ f2 pair(int i) const {
        if constexpr (sizeof(T) == 4) return (f2)w[2 * i] | (f2)w[2 * i + 1] << 32;
        else return widen<T>(VEC == 2 ? w[0] | w[1 % W] << 16 : w[i]);
    }
    __device__ __forceinline__ void set_pair(int i, f2 v) {
        if constexpr (sizeof(T) == 4) {
            w[2 * i] = (uint32_t)v;
            w[2 * i + 1] = (uint32_t)(v >> 32);
        } else {
            w[i] = narrow<T>(v);
            if (VEC == 2) w[1 % W] = w[i] >> 16;
        }
    }
};

// The 8-bit codes of such a piece, one byte each.
template <int VEC>
struct Codes {
    static constexpr int VP = VEC / 2, W = (VEC + 3) / 4;
    uint32_t w[W], second = 0;  // VEC = 2: the second code apart, as above
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const uint8_t *row, long long v, long long C) {
        if constexpr (VEC == 2) {
            w[0] = row[2 * v];
            second = 2 * v + 1 < C ? row[2 * v + 1] : 0;
        }
        else if constexpr (VEC == 4) w[0] = reinterpret_cast<const uint32_t *>(row)[v];
        else {
            const uint2 u = reinterpret_cast<const uint2 *>(row)[v];
            w[0] = u.x, w[1 % W] = u.y;
        }
    }
    __device__ __forceinline__ void store(uint8_t *row, long long v, long long C) const {
        if constexpr (VEC == 2) {
            row[2 * v] = (uint8_t)w[0];
            if (2 * v + 1 < C) row[2 * v + 1] = (uint8_t)(w[0] >> 8);
        } else if constexpr (VEC == 4) {
            reinterpret_cast<uint32_t *>(row)[v] = w[0];
        } else {
            reinterpret_cast<uint2 *>(row)[v] = make_uint2(w[0], w[1 % W]);
        }
    }
    // x * inv to the nearest codes.  int8: adding 1.5 * 2^23 rounds to a whole
    // number (|x inv| <= 127) and leaves its two's complement in the low byte.
    __device__ __forceinline__ void encode(const f2 (&x)[VP], float inv, int fmt) {
        if (fmt == PRISM_CKPT_INT8) {
            f2 y[VP];
#pragma unroll
            for (int i = 0; i < VP; ++i) y[i] = fma2(x[i], both(inv), both(12582912.f));
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const f2 a = y[2 * i], b = y[(2 * i + 1) % VP];
                const uint32_t lo = __byte_perm((uint32_t)a, (uint32_t)(a >> 32), 0x0040);
                const uint32_t hi = __byte_perm((uint32_t)b, (uint32_t)(b >> 32), 0x0040);
                w[i] = __byte_perm(lo, hi, 0x5410);
            }
        } else {
            uint32_t h[VP];
#pragma unroll
            for (int i = 0; i < VP; ++i) {
                const f2 y = mul2(x[i], both(inv));
                h[i] = __nv_cvt_float2_to_fp8x2(make_float2(low(y), high(y)), __NV_SATFINITE, __NV_E4M3);
            }
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = h[2 * i] | (h[(2 * i + 1) % VP] << 16);
        }
    }
    // (q 2^k - mean) rstd of the codes, scale byte sb: q 2^k - mean is one
    // multiply-add, rounded once.
    __device__ __forceinline__ void decode_norm(uint32_t sb, int fmt, float mean, float rstd, f2 (&x)[VP]) const {
        const f2 sc = both(code_scale(sb)), m2 = both(-mean), r2 = both(rstd);
        if (fmt == PRISM_CKPT_INT8) {
#pragma unroll
            for (int i = 0; i < VP; ++i) x[i] = mul2(fma2(whole(i), sc, m2), r2);
        } else {
#pragma unroll
            for (int i = 0; i < VP; ++i) x[i] = mul2(fma2(small_float(i), sc, m2), r2);
        }
    }
    // pair i's codes as int8 (byte + 128 in the mantissa of 2^23) and as e4m3
    __device__ __forceinline__ f2 whole(int i) const {
        const uint32_t u = (VEC == 2 ? w[0] | second << 8 : w[i / 2]) ^ 0x80808080u;
        const uint32_t lo = __byte_perm(u, 0x4b000000u, i & 1 ? 0x7542 : 0x7540);
        const uint32_t hi = __byte_perm(u, 0x4b000000u, i & 1 ? 0x7543 : 0x7541);
        return add2((f2)lo | ((f2)hi << 32), both(-8388736.f));
    }
    __device__ __forceinline__ f2 small_float(int i) const {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(VEC == 2 ? w[0] | second << 8 : w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        return make2(f.x, f.y);
    }
    // the values q 2^k of the codes, scale byte sb, held within T's range
    template <typename T>
    __device__ __forceinline__ void decode(uint32_t sb, int fmt, f2 (&x)[VP]) const {
        const f2 sc = both(code_scale(sb));
        if (fmt == PRISM_CKPT_INT8) {
#pragma unroll
            for (int i = 0; i < VP; ++i) x[i] = mul2(whole(i), sc);
        } else {
#pragma unroll
            for (int i = 0; i < VP; ++i) x[i] = mul2(small_float(i), sc);
        }
        // 127 * 2^119 and 448 * 2^119 are finite; fp16 ends sooner
        if (sb >= (sizeof(T) == 2 && largest<T>() < 1e5f ? 128u : 247u) && sb != 255u) {
#pragma unroll
            for (int i = 0; i < VP; ++i) x[i] = make2(saturate_to<T>(low(x[i])), saturate_to<T>(high(x[i])));
        }
    }
};

// The largest magnitude of a vector's pairs, NaN if any is (max.NaN, three inputs).
template <int VP>
__device__ __forceinline__ float top_of(const f2 (&x)[VP]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < VP; ++i)
        asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(low(x[i])), "f"(high(x[i])));
    return m;
}
// A scale group's exponent from the 32 / VEC neighbouring lanes that hold it
template <int VEC>
__device__ __forceinline__ int group_exponent(float m, int fmt) {
    uint32_t top = __float_as_uint(m) & 0x7fffffffu;  // orders like the value; NaN above all
#pragma unroll
    for (int o = 16 / VEC; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    return code_exponent(__uint_as_float(top), fmt);
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
// four dense, 16-byte aligned bf16 tensors of whole scale groups
prism_status launch_ckpt_pack4(const void *const (&x)[4], const prism_ckpt *const (&k)[4], long long nrows, int C,
                               cudaStream_t st);
prism_status launch_ckpt_unpack(const prism_ckpt &k, const rows::RowPtr &y, int dtype, long long nrows, int C,
                                cudaStream_t st);

}  // namespace prism
