// layer_norm.cu -- layer norm over the channels of each row, forward and
// backward, with the weight gradients' reduction over the rows.
//
//   mean = sum x / C, rstd = (sum (x - mean)^2 / C + eps)^-1/2,
//   xhat = (x - mean) rstd, y = xhat gamma + beta
//   g = dy gamma, dx = rstd (g - mean(g) - xhat mean(g xhat)),
//   dgamma = sum_rows dy xhat, dbeta = sum_rows dy
//
// Statistics and sums are fp32.  The variance is summed from x - mean (a
// second look at the row), not from squares, so an offset costs no digits.
// The weight gradients are summed in a fixed order: every run gives the same
// bits.
#include "rows.cuh"

namespace prism {

using namespace rows;

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// the sum over the CTA's kThreads threads, in every thread
__device__ __forceinline__ float cta_sum(float v, float *red) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += red[w];
    return s;
}

// One CTA per row, any channel count and alignment: three passes over the row
// (the second and third find it in L1 / L2).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_fwd_any(RowPtr x, RowPtr y, const void *gamma, const void *beta,
                                                           int wdt, float *mean_out, float *rstd_out, uint8_t *codes,
                                                           uint8_t *scales, int fmt, long long nrows, int C,
                                                           float eps) {
    __shared__ float red[kThreads / 32];
    for (long long r = blockIdx.x; r < nrows; r += gridDim.x) {
        const T *xr = reinterpret_cast<const T *>(x(r));
        T *yr = reinterpret_cast<T *>(y(r));
        float s = 0.f;
        for (int c = threadIdx.x; c < C; c += kThreads) s += to_f(xr[c]);
        const float mean = cta_sum(s, red) / (float)C;
        float q = 0.f;
        for (int c = threadIdx.x; c < C; c += kThreads) {
            const float d = to_f(xr[c]) - mean;
            q = fmaf(d, d, q);
        }
        const float rstd = rsqrtf(cta_sum(q, red) / (float)C + eps);
        for (int c0 = 0; c0 < C; c0 += kThreads) {
            const int c = c0 + threadIdx.x;
            const float v = c < C ? to_f(xr[c]) : 0.f;
            if (c < C) {
                float o = (v - mean) * rstd;
                if (gamma) o *= weight_at(gamma, wdt, c);
                if (beta) o += weight_at(beta, wdt, c);
                yr[c] = from_f<T>(o);
            }
            if (codes) {  // 32 consecutive channels per warp: one scale group
                uint32_t top = __float_as_uint(fabsf(v));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                const int k = code_exponent(__uint_as_float(top), fmt);
                if (c < C) codes[r * C + c] = k == 128 ? 0 : encode1(v, code_inv_scale(k), fmt);
                if (c < C && (threadIdx.x & 31) == 0)
                    scales[r * ((C + kGroup - 1) / kGroup) + c / kGroup] = (uint8_t)(k + 127);
            }
        }
        if (threadIdx.x == 0) {
            mean_out[r] = mean;
            rstd_out[r] = rstd;
        }
    }
}

// x of row r, channel c: an element, or the value of an 8-bit code
template <typename T>
struct Source {
    RowPtr x;
    const uint8_t *codes, *scales;  // codes == NULL: x
    int fmt, C;
    __device__ __forceinline__ float operator()(long long r, int c) const {
        if (!codes) return to_f(reinterpret_cast<const T *>(x(r))[c]);
        return saturate_to<float>(decode1(codes[r * C + c], fmt) *
                                  code_scale(scales[r * ((C + kGroup - 1) / kGroup) + c / kGroup]));
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_dx_any(Source<T> x, RowPtr dy, RowPtr dx, const void *gamma, int wdt,
                                                          const float *mean_in, const float *rstd_in, long long nrows,
                                                          int C) {
    __shared__ float red[kThreads / 32];
    for (long long r = blockIdx.x; r < nrows; r += gridDim.x) {
        const T *dyr = reinterpret_cast<const T *>(dy(r));
        T *dxr = reinterpret_cast<T *>(dx(r));
        const float mean = mean_in[r], rstd = rstd_in[r];
        float a = 0.f, b = 0.f;
        for (int c = threadIdx.x; c < C; c += kThreads) {
            const float g = to_f(dyr[c]) * (gamma ? weight_at(gamma, wdt, c) : 1.f);
            a += g;
            b = fmaf(g, (x(r, c) - mean) * rstd, b);
        }
        a = cta_sum(a, red) / (float)C;
        b = cta_sum(b, red) / (float)C;
        for (int c = threadIdx.x; c < C; c += kThreads) {
            const float g = to_f(dyr[c]) * (gamma ? weight_at(gamma, wdt, c) : 1.f);
            dxr[c] = from_f<T>((g - a - (x(r, c) - mean) * rstd * b) * rstd);
        }
    }
}

// Column sums of a slice of the rows: part[p][0][c] = sum dy xhat, part[p][1][c] = sum dy.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_dw_any(Source<T> x, RowPtr dy, const float *mean_in,
                                                          const float *rstd_in, float *part, long long nrows, int C) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= C) return;
    const long long r0 = nrows * blockIdx.y / gridDim.y, r1 = nrows * (blockIdx.y + 1) / gridDim.y;
    float a = 0.f, b = 0.f;
    for (long long r = r0; r < r1; ++r) {
        const float d = to_f(reinterpret_cast<const T *>(dy(r))[c]);
        a = fmaf(d, (x(r, c) - mean_in[r]) * rstd_in[r], a);
        b += d;
    }
    part[((size_t)blockIdx.y * 2) * C + c] = a;
    part[((size_t)blockIdx.y * 2 + 1) * C + c] = b;
}

// dgamma, dbeta = the P partials summed in order; 32 columns per CTA.
__global__ void __launch_bounds__(kThreads) k_norm_dw_sum(const float *__restrict__ part, int P, void *dgamma,
                                                          void *dbeta, int wdt, int C) {
    __shared__ float red[2][kThreads / 32][32];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    float a = 0.f, b = 0.f;
    if (c < C)
        for (int p = w; p < P; p += kThreads / 32) {
            a += part[((size_t)p * 2) * C + c];
            b += part[((size_t)p * 2 + 1) * C + c];
        }
    red[0][w][threadIdx.x & 31] = a;
    red[1][w][threadIdx.x & 31] = b;
    __syncthreads();
    if (w < 2 && c < C) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) s += red[w][k][threadIdx.x & 31];
        void *dst = w == 0 ? dgamma : dbeta;
        if (dst) weight_store(dst, wdt, c, s);
    }
}

// Partial weight gradients of the backward: one per CTA, at most 64 MB.
int partials(long long nrows, int C) {
    long long p = (64ll << 20) / (8ll * C);
    if (p > 592) p = 592;
    if (p > nrows) p = nrows;
    return p < 1 ? 1 : (int)p;
}

template <typename T>
prism_status fwd_impl(const NormFwd &a, cudaStream_t st) {
    const int grid = (int)(a.nrows < 148 * 8 ? a.nrows : 148 * 8);
    k_norm_fwd_any<T><<<grid, kThreads, 0, st>>>(a.x, a.y, a.gamma, a.beta, a.wdt, a.mean, a.rstd, a.codes, a.scales,
                                                 a.fmt, a.nrows, a.C, a.eps);
    PRISM_CUDA_OK(cudaGetLastError());
    return PRISM_OK;
}

template <typename T>
prism_status bwd_impl(const NormBwd &a, cudaStream_t st) {
    const Source<T> src{a.x, a.codes, a.scales, a.fmt, a.C};
    const int P = partials(a.nrows, a.C);
    if (a.nrows > 0) {
        const int grid = (int)(a.nrows < 148 * 8 ? a.nrows : 148 * 8);
        k_norm_dx_any<T><<<grid, kThreads, 0, st>>>(src, a.dy, a.dx, a.gamma, a.wdt, a.mean, a.rstd, a.nrows, a.C);
        PRISM_CUDA_OK(cudaGetLastError());
    }
    if (a.dgamma || a.dbeta) {
        k_norm_dw_any<T><<<dim3((a.C + kThreads - 1) / kThreads, P), kThreads, 0, st>>>(src, a.dy, a.mean, a.rstd,
                                                                                        a.part, a.nrows, a.C);
        PRISM_CUDA_OK(cudaGetLastError());
        k_norm_dw_sum<<<(a.C + 31) / 32, kThreads, 0, st>>>(a.part, P, a.dgamma, a.dbeta, a.wdt, a.C);
        PRISM_CUDA_OK(cudaGetLastError());
    }
    return PRISM_OK;
}

}  // namespace

size_t norm_bwd_workspace(long long nrows, int C) { return (size_t)partials(nrows, C) * 2 * C * sizeof(float); }

prism_status launch_norm_fwd(const NormFwd &a, int dtype, cudaStream_t st) {
    if (a.nrows == 0) return PRISM_OK;
    if (dtype == PRISM_BF16) return fwd_impl<__nv_bfloat16>(a, st);
    if (dtype == PRISM_FP16) return fwd_impl<__half>(a, st);
    return fwd_impl<float>(a, st);
}

prism_status launch_norm_bwd(const NormBwd &a, int dtype, cudaStream_t st) {
    if (dtype == PRISM_BF16) return bwd_impl<__nv_bfloat16>(a, st);
    if (dtype == PRISM_FP16) return bwd_impl<__half>(a, st);
    return bwd_impl<float>(a, st);
}

}  // namespace prism
