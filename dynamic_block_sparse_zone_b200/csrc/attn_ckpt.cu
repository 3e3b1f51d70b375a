// attn_ckpt.cu -- the attention's side of 8-bit checkpoints: Q, K and V from
// codes straight into the plan's block-contiguous bf16 copies (a code times its
// power of two is a bf16 value, so nothing is rounded again), and the forward's
// log-sum-exp into the order in which the backward reads it.
//
// HBM-bound by its bytes (1 + 1/32 read and 2 written per value), on small grids
// by the walk over a block's tokens: a thread owns four channels of Q, K or V
// and has 16 tokens' loads in flight; the eight threads of a scale group share
// its scale byte's cache line.  16 x 32 x 32 tokens of 1024 channels, with the
// launch from Python: 68 us (a floor of 24 us; eight tokens at a time with the
// three tensors in one thread took 102 us, the next 16 fetched ahead of the
// current 67 us, not kept).
#include "rows.cuh"

namespace prism {

using namespace rows;

namespace {

constexpr int kThreads = 128;
constexpr int kRows = 16;  // blocks are multiples of 64 tokens

struct Codes8 {
    const uint8_t *codes, *scales;
    int fmt;
};

struct Restore {  // of Q, K, V: the checkpoint, the plan's copy and the block means (V has none)
    Codes8 from[3];
    __nv_bfloat16 *to[3];
    double *mean[3];
};

__global__ void __launch_bounds__(kThreads) k_permute_pool_ckpt(Restore a, Geo g, const int *__restrict__ nb,
                                                                const int *__restrict__ blk_off,
                                                                const int *__restrict__ perm) {
    const int nslice = (g.C / 4 + kThreads - 1) / kThreads;
    const int j = blockIdx.x / nslice, slice = blockIdx.x % nslice, b = blockIdx.y;
    if (j >= nb[b]) return;
    const int *bo = blk_off + (size_t)b * (g.nbmax + 1);
    const int off = bo[j], B = bo[j + 1] - off, ng = g.C / kGroup;
    const int *pb = perm + (size_t)b * g.N + off;
    const int c = 4 * (slice * kThreads + threadIdx.x);
    if (c >= g.C) return;
    const Codes8 from = a.from[blockIdx.z];
    __nv_bfloat16 *to = a.to[blockIdx.z];
    const int hd = c / g.D, d0 = c % g.D;
    const size_t bh = (size_t)b * g.heads + hd, dst0 = (bh * g.N + off) * g.D + d0;
    double sum[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 1
    for (int r0 = 0; r0 < B; r0 += kRows) {
        Codes<4> k[kRows];
        uint32_t ks[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const size_t row = (size_t)b * g.N + pb[r0 + i];
            k[i].w[0] = __ldg(reinterpret_cast<const uint32_t *>(from.codes + row * g.C + c));
            ks[i] = __ldg(from.scales + row * ng + c / kGroup);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            f2 x[2];
            k[i].decode<__nv_bfloat16>(ks[i], from.fmt, x);
            *reinterpret_cast<uint2 *>(to + dst0 + (size_t)(r0 + i) * g.D) =
                make_uint2(narrow<__nv_bfloat16>(x[0]), narrow<__nv_bfloat16>(x[1]));
            sum[0] += (double)low(x[0]), sum[1] += (double)high(x[0]);
            sum[2] += (double)low(x[1]), sum[3] += (double)high(x[1]);
        }
    }
    if (a.mean[blockIdx.z]) {
        const double inv = 1.0 / (double)B;
        double *o = a.mean[blockIdx.z] + (bh * g.nbmax + j) * g.D + d0;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = sum[e] * inv;
    }
}

// nlse_p = -log2(e) lse in block-contiguous order; a row without a key keeps -inf (P = 0).
__global__ void __launch_bounds__(256) k_restore_lse(Geo g, const int *__restrict__ perm, const float *__restrict__ lse,
                                                     float *__restrict__ nlse_p) {
    const int n = blockIdx.x * 256 + threadIdx.x, bh = blockIdx.y, b = bh / g.heads;
    if (n >= g.N) return;
    const float v = lse[(size_t)bh * g.N + perm[(size_t)b * g.N + n]];
    nlse_p[(size_t)bh * g.N + n] = v == -INFINITY ? v : -v * 1.4426950408889634f;
}

Codes8 codes_of(const prism_ckpt &k) {
    return Codes8{static_cast<const uint8_t *>(k.codes), static_cast<const uint8_t *>(k.scales), k.format};
}

}  // namespace

prism_status launch_regather_ckpt(Plan &pl, const prism_attn_ckpt &c, cudaStream_t st) {
    const Geo &g = pl.g;
    {
        TimerScope ts(pl, kTPermutePool, st);
        const Restore r{{codes_of(c.Q), codes_of(c.K), codes_of(c.V)}, {pl.Qp, pl.Kp, pl.Vp}, {pl.Qbar, pl.Kbar, nullptr}};
        k_permute_pool_ckpt<<<dim3((g.C / 4 + kThreads - 1) / kThreads * g.nbmax, g.batch, 3), kThreads, 0, st>>>(
            r, g, pl.nb, pl.blk_off, pl.perm);
    }
    PRISM_CUDA_OK(cudaGetLastError());
    pl.score.zeroed = false;
    return PRISM_OK;
}

prism_status launch_attn_bwd_ckpt(Plan &pl, const prism_attn_ckpt &c, const void *dO, void *dQ, void *dK, void *dV,
                                  bool scored, cudaStream_t st) {
    prism_status s = launch_regather_ckpt(pl, c, st);
    if (s == PRISM_OK && scored) s = launch_zero_padding(pl, st);
    if (s != PRISM_OK) return s;
    const Geo &g = pl.g;
    k_restore_lse<<<dim3((g.N + 255) / 256, g.batch * g.heads), 256, 0, st>>>(g, pl.perm, c.lse, pl.nlse_p);
    PRISM_CUDA_OK(cudaGetLastError());
    return launch_attn_bwd_o8(pl, c.O, dO, dQ, dK, dV, scored, st);
}

}  // namespace prism
