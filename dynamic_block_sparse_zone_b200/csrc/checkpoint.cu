// checkpoint.cu -- activations in 8 bits between the forward and the backward
// pass: codes and one power-of-two scale per 32 channels (rows.cuh has the
// code's definition).
#include "rows.cuh"

namespace prism {

using namespace rows;

namespace {

constexpr int kThreads = 256;

// One warp per group of 32 channels of a row, one channel per lane.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_ckpt_pack(RowPtr x, long long nrows, int C, uint8_t *__restrict__ codes,
                                                        uint8_t *__restrict__ scales, int fmt) {
    const int lane = threadIdx.x & 31, ng = (C + kGroup - 1) / kGroup;
    const long long total = nrows * ng, step = (long long)gridDim.x * (kThreads / 32);
    for (long long it = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); it < total; it += step) {
        const long long r = it / ng;
        const int grp = (int)(it - r * ng), c = grp * kGroup + lane;
        const float v = c < C ? to_f(reinterpret_cast<const T *>(x(r))[c]) : 0.f;
        uint32_t top = __float_as_uint(fabsf(v));  // orders like the value; NaN above all
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int k = code_exponent(__uint_as_float(top), fmt);
        if (c < C) codes[r * C + c] = k == 128 ? 0 : encode1(v, code_inv_scale(k), fmt);
        if (lane == 0) scales[r * ng + grp] = (uint8_t)(k + 127);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_ckpt_unpack(const uint8_t *__restrict__ codes,
                                                          const uint8_t *__restrict__ scales, RowPtr y, long long nrows,
                                                          int C, int fmt) {
    const int lane = threadIdx.x & 31, ng = (C + kGroup - 1) / kGroup;
    const long long total = nrows * ng, step = (long long)gridDim.x * (kThreads / 32);
    for (long long it = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); it < total; it += step) {
        const long long r = it / ng;
        const int grp = (int)(it - r * ng), c = grp * kGroup + lane;
        if (c < C)
            reinterpret_cast<T *>(y(r))[c] =
                from_f<T>(saturate_to<T>(decode1(codes[r * C + c], fmt) * code_scale(scales[r * ng + grp])));
    }
}

int grid_for(long long warps) {
    const long long b = (warps + kThreads / 32 - 1) / (kThreads / 32);
    return (int)(b < 148 * 8 ? b : 148 * 8);
}

}  // namespace

prism_status launch_ckpt_pack(const RowPtr &x, int dtype, long long nrows, int C, const prism_ckpt &k, cudaStream_t st) {
    if (nrows == 0) return PRISM_OK;
    auto *codes = static_cast<uint8_t *>(k.codes), *scales = static_cast<uint8_t *>(k.scales);
    const int grid = grid_for(nrows * ((C + kGroup - 1) / kGroup));
    if (dtype == PRISM_BF16) k_ckpt_pack<__nv_bfloat16><<<grid, kThreads, 0, st>>>(x, nrows, C, codes, scales, k.format);
    else if (dtype == PRISM_FP16) k_ckpt_pack<__half><<<grid, kThreads, 0, st>>>(x, nrows, C, codes, scales, k.format);
    else k_ckpt_pack<float><<<grid, kThreads, 0, st>>>(x, nrows, C, codes, scales, k.format);
    PRISM_CUDA_OK(cudaGetLastError());
    return PRISM_OK;
}

prism_status launch_ckpt_unpack(const prism_ckpt &k, const RowPtr &y, int dtype, long long nrows, int C,
                                cudaStream_t st) {
    if (nrows == 0) return PRISM_OK;
    const auto *codes = static_cast<const uint8_t *>(k.codes), *scales = static_cast<const uint8_t *>(k.scales);
    const int grid = grid_for(nrows * ((C + kGroup - 1) / kGroup));
    if (dtype == PRISM_BF16) k_ckpt_unpack<__nv_bfloat16><<<grid, kThreads, 0, st>>>(codes, scales, y, nrows, C, k.format);
    else if (dtype == PRISM_FP16) k_ckpt_unpack<__half><<<grid, kThreads, 0, st>>>(codes, scales, y, nrows, C, k.format);
    else k_ckpt_unpack<float><<<grid, kThreads, 0, st>>>(codes, scales, y, nrows, C, k.format);
    PRISM_CUDA_OK(cudaGetLastError());
    return PRISM_OK;
}

}  // namespace prism
