// checkpoint.cu -- activations in 8 bits between the forward and the backward
// pass: codes and one power-of-two scale per 32 channels (rows.cuh has the
// code's definition).
//
// HBM-bound: one read and one write of each value.  Every lane moves vectors
// of 16 bytes (two single elements where rows are not aligned to that); the 32 / VEC
// neighbouring lanes that hold a scale group agree on its exponent by
// shuffles.  Four vectors per lane are in flight.  Rows that follow each other
// without a gap, with whole groups in each, are taken as one long row.
// Measured, 92160 x 2048 bf16: pack 102 us, 0.87 of what a copy reaches, unpack
// 111 us, 0.80; 40000 rows of 1001 channels (element-wise, bound by the byte
// stores): 178 us and 118 us, 0.11 and 0.16.
#include "rows.cuh"

namespace prism {

using namespace rows;

namespace {

constexpr int kThreads = 256;
constexpr int kU = 4;  // vectors in flight per lane

struct CkptArgs {
    RowPtr x;
    uint8_t *codes, *scales;
    int fmt;
    long long nrows, nvec;  // rows, vectors per row
    long long C;
    int lanes;              // lanes per row (a power of two; 32: a warp walks along a row)
};

// The row and the vector in it of this lane's u-th access in warp item `it`.
struct Place {
    long long r, v;
    bool in;
};
__device__ __forceinline__ Place place(const CkptArgs &a, long long it, long long per_row, int u) {
    const int lane = threadIdx.x & 31;
    Place p;
    if (a.lanes == 32) {
        p.r = per_row == 1 ? it : it / per_row;
        p.v = (it - p.r * per_row) * (32 * kU) + u * 32 + lane;
    } else {
        p.r = (it * kU + u) * (32 / a.lanes) + lane / a.lanes;
        p.v = lane & (a.lanes - 1);
    }
    p.in = p.r < a.nrows && p.v < a.nvec;
    return p;
}
__device__ __forceinline__ long long items(const CkptArgs &a, long long &per_row) {
    per_row = (a.nvec + 32 * kU - 1) / (32 * kU);
    const long long rows_per_item = (long long)kU * (32 / a.lanes);
    return a.lanes == 32 ? a.nrows * per_row : (a.nrows + rows_per_item - 1) / rows_per_item;
}

// Tensors of one shape packed by one launch, one grid row each.
template <int N>
struct CkptBatch {
    CkptArgs a[N];
};

template <typename T, int VEC, int N>
__global__ void __launch_bounds__(kThreads) k_ckpt_pack(CkptBatch<N> batch) {
    const CkptArgs &a = batch.a[N == 1 ? 0 : blockIdx.y];
    constexpr int VP = VEC / 2, kPer = kGroup / VEC;
    long long per_row;
    const long long n = items(a, per_row), ng = (a.C + kGroup - 1) / kGroup;
    for (long long it = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); it < n;
         it += (long long)gridDim.x * (kThreads / 32)) {
        Vec<T, VEC> raw[kU];
        Place p[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            p[u] = place(a, it, per_row, u);
            if (p[u].in) raw[u].load(a.x(p[u].r), p[u].v, a.C);
            else raw[u].zero();
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            f2 x[VP];
#pragma unroll
            for (int e = 0; e < VP; ++e) x[e] = raw[u].pair(e);
            const int k = group_exponent<VEC>(top_of(x), a.fmt);
            if (p[u].in) {
                Codes<VEC> c;
                c.encode(x, code_inv_scale(k), a.fmt);
                c.store(a.codes + p[u].r * a.C, p[u].v, a.C);
                if (p[u].v % kPer == 0) a.scales[p[u].r * ng + p[u].v / kPer] = (uint8_t)(k + 127);
            }
        }
    }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) k_ckpt_unpack(CkptArgs a) {
    constexpr int VP = VEC / 2, kPer = kGroup / VEC;
    long long per_row;
    const long long n = items(a, per_row), ng = (a.C + kGroup - 1) / kGroup;
    for (long long it = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); it < n;
         it += (long long)gridDim.x * (kThreads / 32)) {
        Codes<VEC> c[kU];
        uint32_t sb[kU];
        Place p[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            p[u] = place(a, it, per_row, u);
            if (p[u].in) {
                c[u].load(a.codes + p[u].r * a.C, p[u].v, a.C);
                sb[u] = a.scales[p[u].r * ng + p[u].v / kPer];
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (p[u].in) {
                f2 x[VP];
                c[u].template decode<T>(sb[u], a.fmt, x);
                Vec<T, VEC> o;
#pragma unroll
                for (int e = 0; e < VP; ++e) o.set_pair(e, x[e]);
                o.store(a.x(p[u].r), p[u].v, a.C);
            }
    }
}

// How a's rows are laid over lanes, and the CTAs that takes.
template <int VEC>
int lay_out(CkptArgs &a, bool dense) {
    if (dense && a.C % kGroup == 0) {
        a.C *= a.nrows;
        a.nrows = 1;
    }
    a.nvec = (a.C + VEC - 1) / VEC;
    a.lanes = kGroup / VEC;
    while (a.lanes < 32 && a.lanes < a.nvec) a.lanes *= 2;
    const long long per = (long long)kU * (32 / a.lanes);
    const long long n = a.lanes == 32 ? a.nrows * ((a.nvec + 32 * kU - 1) / (32 * kU)) : (a.nrows + per - 1) / per;
    const long long ctas = (n + kThreads / 32 - 1) / (kThreads / 32), most = 148 * 16;
    return (int)(ctas < most ? ctas : most);
}

template <typename T, int VEC, bool kPack>
prism_status run(CkptArgs a, bool dense, cudaStream_t st) {
    const int grid = lay_out<VEC>(a, dense);
    if constexpr (kPack) k_ckpt_pack<T, VEC, 1><<<grid, kThreads, 0, st>>>(CkptBatch<1>{{a}});
    else k_ckpt_unpack<T, VEC><<<grid, kThreads, 0, st>>>(a);
    PRISM_CUDA_OK(cudaGetLastError());
    return PRISM_OK;
}

template <typename T, bool kPack>
prism_status run_type(const RowPtr &x, long long nrows, int C, const prism_ckpt &k, cudaStream_t st) {
    constexpr int VEC = 16 / sizeof(T);
    const CkptArgs a{x, static_cast<uint8_t *>(k.codes), static_cast<uint8_t *>(k.scales), k.format, nrows, 0, C, 0};
    const long long row = (long long)C * sizeof(T);
    const bool dense = nrows == 1 || (x.stride == row && (x.group == 0 || x.group >= nrows));
    // a dense tensor of whole groups needs only its first element aligned
    const bool vec = dense && C % kGroup == 0 ? ((uintptr_t)x.data & 15) == 0
                                              : (((uintptr_t)x.data | x.stride | x.group_stride | row) & 15) == 0;
    return vec ? run<T, VEC, kPack>(a, dense, st) : run<T, 2, kPack>(a, dense, st);
}

template <bool kPack>
prism_status run_any(const RowPtr &x, int dtype, long long nrows, int C, const prism_ckpt &k, cudaStream_t st) {
    if (nrows == 0) return PRISM_OK;
    if (dtype == PRISM_BF16) return run_type<__nv_bfloat16, kPack>(x, nrows, C, k, st);
    if (dtype == PRISM_FP16) return run_type<__half, kPack>(x, nrows, C, k, st);
    return run_type<float, kPack>(x, nrows, C, k, st);
}

}  // namespace

prism_status launch_ckpt_pack4(const void *const (&x)[4], const prism_ckpt *const (&k)[4], long long nrows, int C,
                               cudaStream_t st) {
    CkptBatch<4> b;
    int grid = 0;
    for (int i = 0; i < 4; ++i) {
        b.a[i] = CkptArgs{RowPtr{(char *)x[i], C * 2ll, 0, 0}, static_cast<uint8_t *>(k[i]->codes),
                          static_cast<uint8_t *>(k[i]->scales), k[i]->format, nrows, 0, C, 0};
        grid = lay_out<8>(b.a[i], true);
    }
    k_ckpt_pack<__nv_bfloat16, 8, 4><<<dim3(grid, 4), kThreads, 0, st>>>(b);
    PRISM_CUDA_OK(cudaGetLastError());
    return PRISM_OK;
}

prism_status launch_ckpt_pack(const RowPtr &x, int dtype, long long nrows, int C, const prism_ckpt &k, cudaStream_t st) {
    return run_any<true>(x, dtype, nrows, C, k, st);
}

prism_status launch_ckpt_unpack(const prism_ckpt &k, const RowPtr &y, int dtype, long long nrows, int C,
                                cudaStream_t st) {
    return run_any<false>(y, dtype, nrows, C, k, st);
}

}  // namespace prism
