// checkpoint.cu -- activations in 8 bits between the forward and the backward
// pass: codes and one power-of-two scale per 32 channels (rows.cuh has the
// code's definition).
//
// HBM-bound: one read and one write of each value.  Every lane moves vectors
// of 16 bytes (two single elements where rows are not aligned to that); the 32 / VEC
// neighbouring lanes that hold a scale group agree on its exponent by
// shuffles.  Four vectors per lane are in flight.  Rows that follow each other
// without a gap, with whole groups in each, are taken as one long row.
// A lane's vectors lie at constant distances from its first, which is found
// once: with a row, a vector and 64-bit addresses worked out for each, twice the
// registers halved the warps (92160 x 2048 bf16: pack 102 us, unpack 111 us).
// Measured: 94 us each, 0.94 of what a copy reaches; 40000 rows of 1001 channels
// (element-wise, bound by instructions): 71 us and 64 us, 0.27 and 0.30.
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

// Where a lane's kU vectors of warp item `it` are.  kLong: side by side in one
// row, 32 apart, at constant distances from the first; otherwise one each in kU
// rows that lie 32 / lanes apart.
template <bool kLong, int VEC, int kBytes>
struct Place {
    const char *x;    // kLong: this lane's first vector, else NULL
    long long at, g;  // kLong: its first code and scale
    int left, c;      // kLong: vectors of 32 lanes' steps left, channels left
    long long r0, v;
    __device__ __forceinline__ void init(const CkptArgs &a, long long it, long long per_row, long long ng) {
        const int lane = threadIdx.x & 31;
        if constexpr (kLong) {
            long long r = it, v0 = lane;
            if (per_row > 1) {
                r = (it | per_row) >> 32 ? it / per_row : (long long)((unsigned)it / (unsigned)per_row);
                v0 += (it - r * per_row) * (32 * kU);
            }
            x = a.x(r) + v0 * kBytes;
            at = r * a.C + v0 * VEC;
            g = r * ng + v0 / (kGroup / VEC);
            const long long l = a.nvec - v0, cl = a.C - v0 * VEC;
            left = l < 32 * kU ? (int)l : 32 * kU;
            c = cl < 32 * kU * VEC ? (int)cl : 32 * kU * VEC;
        } else {
            r0 = it * kU * (32 / a.lanes) + lane / a.lanes;
            v = lane & (a.lanes - 1);
        }
    }
    __device__ __forceinline__ bool in(const CkptArgs &a, int u) const {
        return kLong ? u * 32 < left : v < a.nvec && row(a, u) < a.nrows;
    }
    __device__ __forceinline__ long long row(const CkptArgs &a, int u) const { return r0 + u * (32 / a.lanes); }
    // the u-th vector is number vec(u) from data() on, of channels() channels
    __device__ __forceinline__ char *data(const CkptArgs &a, int u) const {
        return kLong ? const_cast<char *>(x) : a.x(row(a, u));
    }
    __device__ __forceinline__ uint8_t *codes(const CkptArgs &a, int u) const {
        return a.codes + (kLong ? at : row(a, u) * a.C);
    }
    __device__ __forceinline__ uint8_t *scale(const CkptArgs &a, int u, long long ng) const {
        return a.scales + (kLong ? g + u * (VEC * 32 / kGroup) : row(a, u) * ng + v / (kGroup / VEC));
    }
    __device__ __forceinline__ long long vec(int u) const { return kLong ? u * 32 : v; }
    __device__ __forceinline__ long long channels(const CkptArgs &a) const { return kLong ? c : a.C; }
    // lanes per row are a multiple of those that share a scale
    __device__ __forceinline__ bool first() const { return (threadIdx.x & (kGroup / VEC - 1)) == 0; }
};
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

template <typename T, int VEC, int N, bool kLong>
__global__ void __launch_bounds__(kThreads) k_ckpt_pack(CkptBatch<N> batch) {
    const CkptArgs &a = batch.a[N == 1 ? 0 : blockIdx.y];
    constexpr int VP = VEC / 2;
    long long per_row;
    const long long n = items(a, per_row), ng = (a.C + kGroup - 1) / kGroup;
    for (long long it = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); it < n;
         it += (long long)gridDim.x * (kThreads / 32)) {
        Vec<T, VEC> raw[kU];
        Place<kLong, VEC, VEC * sizeof(T)> p;
        p.init(a, it, per_row, ng);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            raw[u].zero();
            if (p.in(a, u)) raw[u].load(p.data(a, u), p.vec(u), p.channels(a));
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            f2 x[VP];
#pragma unroll
            for (int e = 0; e < VP; ++e) x[e] = raw[u].pair(e);
            const int k = group_exponent<VEC>(top_of(x), a.fmt);
            if (p.in(a, u)) {
                Codes<VEC> c;
                c.encode(x, code_inv_scale(k), a.fmt);
                c.store(p.codes(a, u), p.vec(u), p.channels(a));
                if (p.first()) *p.scale(a, u, ng) = (uint8_t)(k + 127);
            }
        }
    }
}

template <typename T, int VEC, bool kLong>
__global__ void __launch_bounds__(kThreads) k_ckpt_unpack(CkptArgs a) {
    constexpr int VP = VEC / 2;
    long long per_row;
    const long long n = items(a, per_row), ng = (a.C + kGroup - 1) / kGroup;
    for (long long it = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); it < n;
         it += (long long)gridDim.x * (kThreads / 32)) {
        Codes<VEC> c[kU];
        uint32_t sb[kU];
        Place<kLong, VEC, VEC * sizeof(T)> p;
        p.init(a, it, per_row, ng);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (p.in(a, u)) {
                c[u].load(p.codes(a, u), p.vec(u), p.channels(a));
                sb[u] = *p.scale(a, u, ng);
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (p.in(a, u)) {
                f2 x[VP];
                c[u].template decode<T>(sb[u], a.fmt, x);
                Vec<T, VEC> o;
#pragma unroll
                for (int e = 0; e < VP; ++e) o.set_pair(e, x[e]);
                o.store(p.data(a, u), p.vec(u), p.channels(a));
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
    const bool wide = a.lanes == 32;
    if constexpr (kPack) {
        if (wide) k_ckpt_pack<T, VEC, 1, true><<<grid, kThreads, 0, st>>>(CkptBatch<1>{{a}});
        else k_ckpt_pack<T, VEC, 1, false><<<grid, kThreads, 0, st>>>(CkptBatch<1>{{a}});
    } else {
        if (wide) k_ckpt_unpack<T, VEC, true><<<grid, kThreads, 0, st>>>(a);
        else k_ckpt_unpack<T, VEC, false><<<grid, kThreads, 0, st>>>(a);
    }
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
    // (heads * head_dim is a multiple of 32: one long row each)
    k_ckpt_pack<__nv_bfloat16, 8, 4, true><<<dim3(grid, 4), kThreads, 0, st>>>(b);
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
