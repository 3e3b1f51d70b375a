// attn_bwd_aux.cu -- the memory-bound steps around the tensor-core backward:
//   k_attn_bwd_pre   Delta_q = rowsum(dO_q * O_q) from the forward's bf16 O (or its 8-bit form) and
//                    the block-contiguous, head-major copy of dO
//   k_dq_finalize    fp32 dQ accumulator (block-contiguous) -> bf16 dQ in the
//                    caller's raster layout
// and the launcher of the whole backward [Prism guide, Method section 3; the
// standard softmax-attention gradient through the selected block pairs].
#include "rows.cuh"

namespace prism {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}

// ---------------------------------------------------------------------------
// backward, part 1: Delta = rowsum(dO * O) and the permuted copy of dO
// ---------------------------------------------------------------------------
// (doc, scored attention: a padding token's row counts as dO = 0, whatever it holds.)
// kO8: O is a checkpoint's codes, with their scales and format.  Olo, if not
// NULL (scored attention), is what the bf16 O leaves of the forward's fp32 O: in
// rows with few visible keys dP and Delta nearly cancel, and O's rounding would
// be the largest error of dS.
template <int D, bool kO8>
__global__ void __launch_bounds__(256) k_attn_bwd_pre(Geo g, const void *__restrict__ Ov,
                                                      const uint8_t *__restrict__ Os, int fmt,
                                                      const __nv_bfloat16 *__restrict__ dO,
                                                      const int *__restrict__ perm, const int *__restrict__ doc,
                                                      const __nv_bfloat16 *__restrict__ Olo,
                                                      __nv_bfloat16 *__restrict__ dOp, float *__restrict__ delta) {
    constexpr int L = D / 8;  // lanes per (token, head)
    const int b = blockIdx.y;
    const int G = g.C / 8;
    const size_t items = (size_t)kTile * G;
    for (size_t it = threadIdx.x; it < items; it += blockDim.x) {
        const int nl = (int)(it / G), grp = (int)(it % G);
        const int n = blockIdx.x * kTile + nl;
        const int tok = perm[(size_t)b * g.N + n];
        const size_t src = ((size_t)b * g.N + tok) * g.C + grp * 8;
        uint4 dv = *reinterpret_cast<const uint4 *>(dO + src);
        uint4 ov;
        if constexpr (kO8) {
            rows::Codes<8> c;
            c.load(static_cast<const uint8_t *>(Ov) + src, 0, 8);
            const uint32_t sb = Os[((size_t)b * g.N + tok) * (g.C / rows::kGroup) + grp / (rows::kGroup / 8)];
            rows::f2 x[4];
            c.decode<__nv_bfloat16>(sb, fmt, x);
            ov.x = rows::narrow<__nv_bfloat16>(x[0]), ov.y = rows::narrow<__nv_bfloat16>(x[1]);
            ov.z = rows::narrow<__nv_bfloat16>(x[2]), ov.w = rows::narrow<__nv_bfloat16>(x[3]);
        } else {
            ov = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(Ov) + src);
        }
        if (doc && doc[(size_t)b * g.N + n] < 0) ov = dv = make_uint4(0, 0, 0, 0);
        const int hd = grp * 8 / D, d0 = grp * 8 % D;
        const size_t bh = (size_t)b * g.heads + hd;
        *reinterpret_cast<uint4 *>(dOp + (bh * g.N + n) * D + d0) = dv;
        const uint32_t ow[4] = {ov.x, ov.y, ov.z, ov.w}, dw[4] = {dv.x, dv.y, dv.z, dv.w};
        float acc = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            acc += __uint_as_float(ow[k] << 16) * __uint_as_float(dw[k] << 16);
            acc += __uint_as_float(ow[k] & 0xffff0000u) * __uint_as_float(dw[k] & 0xffff0000u);
        }
        if (Olo) {
            const uint4 lv = *reinterpret_cast<const uint4 *>(Olo + (bh * g.N + n) * D + d0);
            const uint32_t lw[4] = {lv.x, lv.y, lv.z, lv.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc += __uint_as_float(lw[k] << 16) * __uint_as_float(dw[k] << 16);
                acc += __uint_as_float(lw[k] & 0xffff0000u) * __uint_as_float(dw[k] & 0xffff0000u);
            }
        }
#pragma unroll
        for (int o2 = L / 2; o2 > 0; o2 >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o2, L);
        if ((threadIdx.x & (L - 1)) == 0) delta[bh * g.N + n] = acc;
    }
}

// dQ (fp32, permuted, head-major) -> bf16 user layout
template <int D>
__global__ void __launch_bounds__(256) k_dq_finalize(Geo g, const float *__restrict__ dQacc,
                                                     const int *__restrict__ perm, __nv_bfloat16 *__restrict__ dQ) {
    const int b = blockIdx.y;
    const int G = g.C / 8;
    const size_t items = (size_t)kTile * G;
    for (size_t it = threadIdx.x; it < items; it += blockDim.x) {
        const int nl = (int)(it / G), grp = (int)(it % G);
        const int n = blockIdx.x * kTile + nl;
        const int hd = grp * 8 / D, d0 = grp * 8 % D;
        const size_t bh = (size_t)b * g.heads + hd;
        const float4 *src = reinterpret_cast<const float4 *>(dQacc + (bh * g.N + n) * D + d0);
        const float4 x = src[0], y = src[1];
        uint4 v;
        v.x = pack_bf16(x.x, x.y);
        v.y = pack_bf16(x.z, x.w);
        v.z = pack_bf16(y.x, y.y);
        v.w = pack_bf16(y.z, y.w);
        const int tok = perm[(size_t)b * g.N + n];
        *reinterpret_cast<uint4 *>(dQ + ((size_t)b * g.N + tok) * g.C + grp * 8) = v;
    }
}

// ---------------------------------------------------------------------------
// launcher
// ---------------------------------------------------------------------------
// O: bf16, or (o8) its checkpoint
template <int D>
static prism_status bwd_impl(Plan &pl, const void *O, const prism_ckpt *o8, const void *dO, void *dQ, void *dK, void *dV,
                             bool scored, cudaStream_t st) {
    const Geo &g = pl.g;
    PRISM_CUDA_OK(cudaMemsetAsync(pl.dQacc, 0, (size_t)g.batch * g.heads * g.N * D * sizeof(float), st));
    {
        TimerScope ts(pl, kTBwdPre, st);
        const int *doc = scored && pl.score.has_doc ? pl.score.doc : nullptr;
        const auto *dOb = static_cast<const __nv_bfloat16 *>(dO);
        if (o8)
            k_attn_bwd_pre<D, true><<<dim3(g.nbmax, g.batch), 256, 0, st>>>(
                g, o8->codes, static_cast<const uint8_t *>(o8->scales), o8->format, dOb, pl.perm, doc, nullptr, pl.dOp,
                pl.delta);
        else
            k_attn_bwd_pre<D, false>
                <<<dim3(g.nbmax, g.batch), 256, 0, st>>>(g, O, nullptr, 0, dOb, pl.perm, doc,
                                                         scored ? pl.score.Olo : nullptr, pl.dOp, pl.delta);
        PRISM_CUDA_OK(cudaGetLastError());
    }
    prism_status s = scored ? launch_attn_bwd_tc_scored(pl, dK, dV, st) : launch_attn_bwd_tc_main(pl, dK, dV, st);
    if (s != PRISM_OK) return s;
    TimerScope ts(pl, kTDqFinal, st);
    k_dq_finalize<D><<<dim3(g.nbmax, g.batch), 256, 0, st>>>(g, pl.dQacc, pl.perm,
                                                            static_cast<__nv_bfloat16 *>(dQ));
    PRISM_CUDA_OK(cudaGetLastError());
    return PRISM_OK;
}

prism_status launch_attn_bwd(Plan &pl, const void *O, const void *dO, void *dQ, void *dK, void *dV, bool scored,
                             cudaStream_t st) {
    return pl.g.D == 64 ? bwd_impl<64>(pl, O, nullptr, dO, dQ, dK, dV, scored, st)
                        : bwd_impl<128>(pl, O, nullptr, dO, dQ, dK, dV, scored, st);
}

prism_status launch_attn_bwd_o8(Plan &pl, const prism_ckpt &O, const void *dO, void *dQ, void *dK, void *dV, bool scored,
                                cudaStream_t st) {
    return pl.g.D == 64 ? bwd_impl<64>(pl, nullptr, &O, dO, dQ, dK, dV, scored, st)
                        : bwd_impl<128>(pl, nullptr, &O, dO, dQ, dK, dV, scored, st);
}

}  // namespace prism
