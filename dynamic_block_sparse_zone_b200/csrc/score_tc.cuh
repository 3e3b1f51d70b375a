// score_tc.cuh -- what the two scored forwards share: a group of 32 raw scores
// of one query row turned into logits.
#pragma once

#include "tc_common.cuh"

namespace prism {
namespace tc {

template <bool kNan>
__device__ __forceinline__ void logistic32(uint32_t (&sr)[32], float cap_in) {
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        float *x = reinterpret_cast<float *>(&sr[e]);
        uint64_t q02, q13;
        logistic4<kNan>(x[0], x[1], x[2], x[3], cap_in, q02, q13);
        x[0] = plo(q02), x[1] = plo(q13), x[2] = phi(q02), x[3] = phi(q13);
    }
}

// x becomes the logit in log2 units (without cap and bias: stays the raw score),
// -inf where the key is hidden.  pos, vis and doc: shared-window addresses of
// the 32 keys' positions, visibilities and documents (vis and doc only read
// where the pair of blocks is partly visible).  Warp-uniform: part.
template <int kScore>
__device__ __forceinline__ void logits32(uint32_t (&sr)[32], const ScoreArgs &sc, float scale_log2, float slope2, float pq,
                                         int dq, uint32_t pos, uint32_t vis, uint32_t doc, bool part) {
    float k = scale_log2, a = 0.f;  // the logit is what is in place times k, plus a and the bias
    if constexpr ((kScore & kCap) != 0) {
        float ma = 0.f, mb = 0.f;
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            const float *x = reinterpret_cast<const float *>(&sr[e]);
            ma = fmax3_abs(ma, x[0], x[1]);
            mb = fmax3_abs(mb, x[2], x[3]);
        }
        if (__all_sync(0xffffffffu, fmaxf(ma, mb) <= sc.cap_one)) {  // tanh in place
            const uint64_t ku = splat2(sc.cap_u);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                float *x = reinterpret_cast<float *>(&sr[e]);
                const uint64_t t = tanh_small2(x[0], x[1], ku);
                x[0] = plo(t), x[1] = phi(t);
            }
            k = sc.cap_out;
        } else {  // q of every score in place
            if (any_nan(sr)) logistic32<true>(sr, sc.cap_in);
            else logistic32<false>(sr, sc.cap_in);
            k = -2.f * sc.cap_out;
            a = sc.cap_out;
        }
    }
    if constexpr ((kScore & (kCap | kBias)) != 0) {
        const uint64_t k2 = splat2(k);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            float *x = reinterpret_cast<float *>(&sr[e]);
            uint64_t a01 = splat2(a), a23 = splat2(a);
            if constexpr ((kScore & kBias) != 0) {
                const float4 pk = lds_f4(pos + e * 4);
                a01 = pair2(fmaf(-slope2, fabsf(pq - pk.x), a), fmaf(-slope2, fabsf(pq - pk.y), a));
                a23 = pair2(fmaf(-slope2, fabsf(pq - pk.z), a), fmaf(-slope2, fabsf(pq - pk.w), a));
            }
            const uint64_t y01 = pfma(pair2(x[0], x[1]), k2, a01), y23 = pfma(pair2(x[2], x[3]), k2, a23);
            x[0] = plo(y01), x[1] = phi(y01), x[2] = plo(y23), x[3] = phi(y23);
        }
    }
    if (part) {
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            const float4 vk = lds_f4(vis + e * 4);
            const float4 dk = lds_f4(doc + e * 4);
            const uint32_t ninf = 0xff800000u;
            if (!(vk.x <= pq && __float_as_int(dk.x) == dq)) sr[e] = ninf;
            if (!(vk.y <= pq && __float_as_int(dk.y) == dq)) sr[e + 1] = ninf;
            if (!(vk.z <= pq && __float_as_int(dk.z) == dq)) sr[e + 2] = ninf;
            if (!(vk.w <= pq && __float_as_int(dk.w) == dq)) sr[e + 3] = ninf;
        }
    }
}

// P = exp2(x * s2 + c2) of 32 scores as two bf16 numbers each: hi, P's upper 16
// bits, and lo, the rest (pairs packed); adds P to acc2.
__device__ __forceinline__ void split_exp32(const uint32_t (&sr)[32], uint64_t s2, uint64_t c2, uint64_t &acc2,
                                            uint32_t (&hi)[16], uint32_t (&lo)[16]) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        float x0, x1;
        fma2(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]), s2, c2, x0, x1);
        const float p0 = ex2(x0), p1 = ex2(x1);
        add2(acc2, p0, p1);
        const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
        hi[e] = __byte_perm(u0, u1, 0x7632);
        const uint64_t d = psub(pair2(p0, p1), (uint64_t)(u0 & 0xffff0000u) | (uint64_t)(u1 & 0xffff0000u) << 32);
        lo[e] = pack_bf16x2(plo(d), phi(d));
    }
}

}  // namespace tc
}  // namespace prism
