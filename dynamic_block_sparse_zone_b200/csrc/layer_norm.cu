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
//
// Bound: HBM, by a read of each input and a write of each output.  Measured,
// bf16 with fp32 weights, as a share of the 6456 GB/s that a copy reaches:
//   rows x channels   forward       with checkpoint  backward      from 8 bits
//   1048576 x 128     103 us 0.81   163 us 0.64      157 us 0.79   170 us 0.62
//   92160 x 1536      108 us 0.81   123 us 0.90      147 us 0.90   167 us 0.66
//   92160 x 2048      140 us 0.83   162 us 0.91      190 us 0.92   222 us 0.66
//   40000 x 5120      157 us 0.81   239 us 0.67      281 us 0.68   456 us 0.35
//   40000 x 1001       72 us 0.34   127 us 0.24       87 us 0.43   100 us 0.31
// What holds the others: from 8 bits, latency (168 registers leave 12 warps per
// SM, which issue 0.50 instructions per cycle and scheduler; the decoding adds a
// byte permute, a multiply-add and a multiply per pair to their chains); rows of
// more than 4096 channels backward, one CTA per SM, whose barrier is not hidden by
// another's work; odd rows, element-wise loads and stores.
#include <atomic>

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

// dgamma, dbeta = the P partials, 32 columns per CTA: warp w sums the partials
// p = w mod 32, then the warps' sums are added in order.
__global__ void __launch_bounds__(1024) k_norm_dw_sum(const float *__restrict__ part, int P, void *dgamma, void *dbeta,
                                                      int wdt, int C) {
    __shared__ float red[2][32][33];
    const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, w = threadIdx.x >> 5;
    float a = 0.f, b = 0.f;
    if (c < C) {
#pragma unroll 8
        for (int p = w; p < P; p += 32) {
            a += part[((size_t)p * 2) * C + c];
            b += part[((size_t)p * 2 + 1) * C + c];
        }
    }
    red[0][w][lane] = a;
    red[1][w][lane] = b;
    __syncthreads();
    if (w < 2 && c < C) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) s += red[w][k][lane];
        void *dst = w == 0 ? dgamma : dbeta;
        if (dst) weight_store(dst, wdt, c, s);
    }
}

// ---------------------------------------------------------------------------
// Rows held in registers: one read of each input, one write of each output
// (the floor of these HBM-bound operators).  A row's nvec pieces of VEC
// elements are spread over `tpr` threads, NV each: lanes of one warp (tpr <=
// 32, a power of two, 256 / tpr rows per CTA; only shuffles between the lanes)
// or the whole CTA (one row at a time).  Every thread keeps its channels over
// all of the rows that it takes, so weights and their gradients stay put.
//
// The grid is resident and walks the rows.  A row's chain (fetch, one or two
// reductions, write) is long against its share of the bandwidth, so the rows
// to come are fetched kS - 1 ahead by cp.async, each thread into slots of its
// own (no barrier): what is in flight does not cost registers.
// ---------------------------------------------------------------------------

// N sums over tpr lanes, in each of them
template <int N>
__device__ __forceinline__ void lanes_sum(float (&v)[N], int tpr) {
    for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
}
// N sums over the CTA's threads (at most 512, red zeroed past its warps), one barrier
template <int N>
__device__ __forceinline__ void rows_cta_sum(float (&v)[N], float (&red)[N][16]) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = warp_sum(v[k]);
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) red[k][threadIdx.x >> 5] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = 0.f;
    for (int q = 0; q < (int)(blockDim.x + 127) / 128; ++q)
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float4 f = reinterpret_cast<const float4 *>(red[k])[q];
            v[k] += (f.x + f.y) + (f.z + f.w);
        }
}

// VEC weights from channel c0 on (NULL: `none` each); `vec`: 16-byte aligned
template <int VEC>
__device__ __forceinline__ void load_weights(const void *p, int dt, int c0, int C, bool vec, float none,
                                             f2 (&w)[VEC / 2]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) w[i] = both(none);
    } else if (VEC > 2 && vec && dt == PRISM_FP32) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + c0) + i);
            w[2 * i] = make2(f.x, f.y);
            w[2 * i + 1] = make2(f.z, f.w);
        }
    } else if (VEC == 8 && vec) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __half *>(p) + c0));
        const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
            w[i] = dt == PRISM_BF16 ? widen<__nv_bfloat16>(a[i % 4]) : widen<__half>(a[i % 4]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const int c = c0 + 2 * i;
            w[i] = make2(weight_at(p, dt, c), c + 1 < C ? weight_at(p, dt, c + 1) : 0.f);
        }
    }
}

// kS: steps in a thread's ring, by what a thread holds per step (bytes); at 512
// to 1280 threads per SM this keeps 64 to 128 KB in flight.
constexpr int ring(int bytes) { return bytes <= 64 ? 4 : bytes <= 96 ? 3 : 2; }
constexpr int bwd_ring(int bytes) { return bytes <= 64 ? 4 : 3; }
// NR: rows that a group of threads takes at once, so that short rows share the
// cost of a step and their reductions overlap.
constexpr int fwd_rows(int channels, bool cta) { return cta || channels > 16 ? 1 : channels > 8 ? 2 : 4; }
// (cta: 0 lanes of a warp, 1 a CTA of up to 192 threads, 2 of up to 512)
constexpr int bwd_rows(int channels, int cta) { return cta == 1 ? 2 : cta == 2 || channels > 8 ? 1 : 2; }

// A CTA's walk over the rows: step `it` takes rows it * step + j * per + sub
// (j < NR) past its first; all of them exist except in the last step.
struct Walk {
    long long first, step;
    int steps, last, per, sub;  // last: rows from the last step's first row on
    __device__ __forceinline__ void init(long long nrows, int per_, int nr, int sub_) {
        per = per_;
        sub = sub_;
        step = (long long)gridDim.x * per * nr;
        first = (long long)blockIdx.x * per * nr;
        steps = (int)((nrows - first + step - 1) / step);  // >= 1: the grid has no CTA without rows
        const long long left = nrows - first - (steps - 1) * step;
        last = left < per * nr ? (int)left : per * nr;
    }
    __device__ __forceinline__ bool live(int it, int j) const { return it < steps - 1 || (it < steps && j * per + sub < last); }
    __device__ __forceinline__ long long row(int it, int j) const { return first + it * step + j * per + sub; }
};
// The address of a step's rows: one addition per step where rows are evenly spaced.
struct RowWalk {
    char *p;
    long long inc, jinc;
    __device__ __forceinline__ void start(const RowPtr &q, const Walk &w) {
        inc = w.step * q.stride;
        jinc = (long long)w.per * q.stride;
        p = q.data + (w.first + w.sub) * q.stride;
    }
    __device__ __forceinline__ char *at(const RowPtr &q, const Walk &w, int it, int j) const {
        return q.group == 0 ? p + j * jinc : q(w.row(it, j));
    }
    __device__ __forceinline__ void next() { p += inc; }
};

struct FwdArgs {
    RowPtr x, y;
    const void *gamma, *beta;
    int wdt;
    bool wvec;
    float *mean, *rstd;
    uint8_t *codes, *scales;
    int fmt;
    long long nrows;
    int C, nvec, tpr;
    float eps, invC;
};

template <typename T, int VEC, int NV, bool kCta, bool kCkpt>
__global__ void __launch_bounds__(kCta ? 512 : 256, kCta ? 1 : 2) k_norm_fwd(FwdArgs a) {
    constexpr int VP = VEC / 2, NR = fwd_rows(NV * VEC, kCta), NP = NR * NV, kS = ring(NP * 16);
    constexpr bool kRing = VEC * sizeof(T) == 16;
    // weights stay in registers, or (more than 16 channels per thread) in shared memory as fp32
    constexpr bool kKeep = NV * VEC <= 16;
    extern __shared__ uint4 slots[];  // [kS][NP][threads] if kRing, then gamma and beta unless kKeep
    __shared__ __align__(16) float red[2][2][1][16];  // [row's parity][which sum]
    if (kCta && threadIdx.x < 64) (&red[0][0][0][0])[threadIdx.x] = 0.f;
    const int tpr = kCta ? blockDim.x : a.tpr, t = kCta ? threadIdx.x : (threadIdx.x & (tpr - 1));
    Walk w;
    w.init(a.nrows, kCta ? 1 : 256 / tpr, NR, kCta ? 0 : threadIdx.x / tpr);
    RowWalk xw, yw;
    xw.start(a.x, w);
    yw.start(a.y, w);
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) in[i] = i * tpr + t < a.nvec;
    auto slot = [&](int s, int p) -> uint4 & { return slots[(s * NP + p) * blockDim.x + threadIdx.x]; };
    Vec<T, VEC> ahead[kRing ? 1 : NP];  // without a ring: one step ahead in registers
    int fit = 0;                        // the step to fetch
    auto fetch = [&](int s) {
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            const bool live = w.live(fit, j);
            const char *xr = xw.at(a.x, w, fit, j);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int p = j * NV + i;
                if constexpr (kRing) {
                    if (live && in[i]) copy_async<16>(&slot(s, p), xr + (i * tpr + t) * 16);
                } else {
                    ahead[p].zero();
                    if (live && in[i]) ahead[p].load(xr, i * tpr + t, a.C);
                }
            }
        }
        if constexpr (kRing) copy_commit();
        xw.next();
        ++fit;
    };
    if constexpr (kRing) {  // slots that are not fetched into hold zeros
#pragma unroll
        for (int p = 0; p < kS * NP; ++p) slot(0, p) = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int s = 0; s < kS - 1; ++s) fetch(s);
    } else {
        fetch(0);
    }
    f2 gw[kKeep ? NV : 1][VP], bw[kKeep ? NV : 1][VP];
    // [gamma, beta][VP / 2][nvec] quadruples (VEC = 2: [gamma, beta][nvec] pairs): neighbouring
    // lanes read neighbouring 16 bytes, without bank conflicts
    f2 *wsm = reinterpret_cast<f2 *>(slots + (kRing ? kS * NP * blockDim.x : 0));
    auto weight_slot = [&](int which, int v, int e) {
        return VEC == 2 ? which * a.nvec + v : ((which * (VP / 2) + e / 2) * a.nvec + v) * 2 + (e & 1);
    };
    if constexpr (kKeep) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i]) {
                load_weights<VEC>(a.gamma, a.wdt, (i * tpr + t) * VEC, a.C, a.wvec, 1.f, gw[i]);
                load_weights<VEC>(a.beta, a.wdt, (i * tpr + t) * VEC, a.C, a.wvec, 0.f, bw[i]);
            }
    } else {
        for (int v = threadIdx.x; v < a.nvec; v += blockDim.x) {
            f2 u[VP];
            load_weights<VEC>(a.gamma, a.wdt, v * VEC, a.C, a.wvec, 1.f, u);
#pragma unroll
            for (int e = 0; e < VP; ++e) wsm[weight_slot(0, v, e)] = u[e];
            load_weights<VEC>(a.beta, a.wdt, v * VEC, a.C, a.wvec, 0.f, u);
#pragma unroll
            for (int e = 0; e < VP; ++e) wsm[weight_slot(1, v, e)] = u[e];
        }
        __syncthreads();
    }
    int par = 0, cur = 0;
    // a slot of red is written again two rows on, behind the barriers of the row between
    auto row_sums = [&](float (&v)[NR], int which) {
        if constexpr (kCta) rows_cta_sum(v, red[par][which]);
        else lanes_sum(v, tpr);
    };
    if (kCta) __syncthreads();
    const int ng = (a.C + kGroup - 1) / kGroup;
    uint8_t *cw = a.codes + (w.first + w.sub) * a.C, *sw = a.scales + (w.first + w.sub) * ng;
    const long long cinc = w.step * a.C, sinc = w.step * ng;
    for (int it = 0; it < w.steps; ++it) {
        f2 x[NP][VP];
        if constexpr (kRing) copy_wait<kS - 2>();
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            Vec<T, VEC> raw;
            if constexpr (kRing) raw.set(slot(cur, p));
            else raw = ahead[p];
#pragma unroll
            for (int e = 0; e < VP; ++e) x[p][e] = raw.pair(e);
        }
        if constexpr (kRing) {  // into the slots that the step before has been read from
            fetch(cur == 0 ? kS - 1 : cur - 1);
            cur = cur == kS - 1 ? 0 : cur + 1;
        } else {
            fetch(0);
        }
        float mean[NR], rstd[NR];
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            f2 s = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VP; ++e) s = add2(s, x[j * NV + i][e]);
            mean[j] = low(s) + high(s);
        }
        row_sums(mean, 0);
#pragma unroll
        for (int j = 0; j < NR; ++j) mean[j] *= a.invC;
        if constexpr (kCkpt) {
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                const bool live = w.live(it, j);
                uint8_t *cr = cw + j * w.per * (long long)a.C, *sr = sw + j * w.per * (long long)ng;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int v = i * tpr + t, k = group_exponent<VEC>(top_of(x[j * NV + i]), a.fmt);
                    if (in[i] && live) {
                        Codes<VEC> c;
                        c.encode(x[j * NV + i], code_inv_scale(k), a.fmt);
                        c.store(cr, v, a.C);
                        if (v % (kGroup / VEC) == 0) sr[v / (kGroup / VEC)] = (uint8_t)(k + 127);
                    }
                }
            }
            cw += cinc;
            sw += sinc;
        }
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            f2 q = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {  // x becomes x - mean; what lies past the row stays 0
                const float m0 = in[i] ? -mean[j] : 0.f;
                const f2 m = make2(m0, VEC == 2 && 2 * (i * tpr + t) + 1 >= a.C ? 0.f : m0);
#pragma unroll
                for (int e = 0; e < VP; ++e) {
                    x[j * NV + i][e] = add2(x[j * NV + i][e], m);
                    q = fma2(x[j * NV + i][e], x[j * NV + i][e], q);
                }
            }
            rstd[j] = low(q) + high(q);
        }
        row_sums(rstd, 1);
#pragma unroll
        for (int j = 0; j < NR; ++j) rstd[j] = rsqrtf(rstd[j] * a.invC + a.eps);
        par ^= 1;
#pragma unroll
        for (int j = 0; j < NR; ++j)
            if (w.live(it, j)) {
                const f2 rs = both(rstd[j]);
                char *yr = yw.at(a.y, w, it, j);
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (in[i]) {
                        const int v = i * tpr + t;
                        Vec<T, VEC> o;
                        f2 gs[VP], bs[VP];
                        if constexpr (!kKeep) {
                            if constexpr (VEC == 2) {
                                gs[0] = wsm[weight_slot(0, v, 0)];
                                bs[0] = wsm[weight_slot(1, v, 0)];
                            } else {
#pragma unroll
                                for (int e = 0; e < VP; e += 2) {
                                    const ulonglong2 g2 = *reinterpret_cast<const ulonglong2 *>(wsm + weight_slot(0, v, e));
                                    const ulonglong2 b2 = *reinterpret_cast<const ulonglong2 *>(wsm + weight_slot(1, v, e));
                                    gs[e] = g2.x, gs[e + 1] = g2.y, bs[e] = b2.x, bs[e + 1] = b2.y;
                                }
                            }
                        }
#pragma unroll
                        for (int e = 0; e < VP; ++e) {
                            const f2 g = kKeep ? gw[kKeep ? i : 0][e] : gs[e];
                            const f2 b = kKeep ? bw[kKeep ? i : 0][e] : bs[e];
                            o.set_pair(e, fma2(x[j * NV + i][e], mul2(g, rs), b));
                        }
                        o.store(yr, v, a.C);
                    }
                if (t == 0) {
                    a.mean[w.row(it, j)] = mean[j];
                    a.rstd[w.row(it, j)] = rstd[j];
                }
            }
        yw.next();
    }
    if constexpr (kRing) copy_wait<0>();
}

struct BwdArgs {
    RowPtr x, dy, dx;  // with a checkpoint, x walks its codes
    const uint8_t *scales;
    int fmt;
    const void *gamma;
    int wdt;
    bool wvec;
    const float *mean, *rstd;
    float *part;  // [gridDim.x][2][C]; NULL: no weight gradients
    long long nrows;
    int C, nvec, tpr;
    float invC;
};

// Each thread adds up dgamma and dbeta of its own channels over the CTA's rows
// in registers; the CTA writes one partial.  Rows past the last one, and
// channels past C, count as dy = 0.
// kCkpt: 0 x, 1 x's checkpoint, 2 the same with rows of scales that are whole
// 32-bit words: a piece's word then travels behind its codes in their slot.
template <typename T, int VEC, int NV, int kCta, int kCkpt>
__global__ void __launch_bounds__(kCta == 2 ? 512 : kCta ? 192 : 256, kCta == 2 ? 1 : 2) k_norm_bwd(BwdArgs a) {
    constexpr int VP = VEC / 2, NR = bwd_rows(NV * VEC, kCta), NP = NR * NV, kS = bwd_ring(NP * 32);
    constexpr bool kRing = VEC * sizeof(T) == 16;
    extern __shared__ uint4 slots[];  // [kS][dy, x or its codes][NP][threads]
    __shared__ __align__(16) float red[2][2 * NR][16];  // [step's parity]
    __shared__ float fold[kCta ? 1 : 256 * NV * VEC];
    if (kCta)
        for (int k = threadIdx.x; k < 64 * NR; k += blockDim.x) (&red[0][0][0])[k] = 0.f;
    const int tpr = kCta ? blockDim.x : a.tpr, t = kCta ? threadIdx.x : (threadIdx.x & (tpr - 1));
    Walk w;
    w.init(a.nrows, kCta ? 1 : 256 / tpr, NR, kCta ? 0 : threadIdx.x / tpr);
    RowWalk dyw, xw, dxw;
    dyw.start(a.dy, w);
    xw.start(a.x, w);
    dxw.start(a.dx, w);
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) in[i] = i * tpr + t < a.nvec;
    auto slot = [&](int s, int p) -> uint4 & { return slots[(s * 2 * NP + p) * blockDim.x + threadIdx.x]; };
    // without a ring: one step ahead in registers
    Vec<T, VEC> ndy[kRing ? 1 : NP], nx[kRing || kCkpt ? 1 : NP];
    Codes<VEC> nc[kRing || !kCkpt ? 1 : NP];
    const int ng = (a.C + kGroup - 1) / kGroup;
    int sbit[NV];  // where a piece's scale lies in its word
#pragma unroll
    for (int i = 0; i < NV; ++i) sbit[i] = 8 * ((i * tpr + t) / (kGroup / VEC) & 3);
    int fit = 0;  // the step to fetch
    auto fetch = [&](int s) {
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            const bool live = w.live(fit, j);
            const char *dyr = dyw.at(a.dy, w, fit, j), *xr = xw.at(a.x, w, fit, j);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int p = j * NV + i, v = i * tpr + t;
                if constexpr (kRing) {
                    if (live && in[i]) {
                        copy_async<16>(&slot(s, p), dyr + v * 16);
                        if constexpr (kCkpt) copy_async<VEC>(&slot(s, NP + p), xr + v * VEC);
                        if constexpr (kCkpt == 2)
                            copy_async<4>(reinterpret_cast<char *>(&slot(s, NP + p)) + VEC,
                                          a.scales + w.row(fit, j) * ng + v / (kGroup / VEC) / 4 * 4);
                        if constexpr (!kCkpt) copy_async<16>(&slot(s, NP + p), xr + v * 16);
                    } else if (kCta != 2) {  // rows past the last: zeros over what an earlier step left
                        slot(s, p) = make_uint4(0, 0, 0, 0);
                    }
                } else {
                    ndy[p].zero();
                    if constexpr (kCkpt) nc[p].zero();
                    else nx[p].zero();
                    if (live && in[i]) {
                        ndy[p].load(dyr, v, a.C);
                        if constexpr (kCkpt) nc[p].load((const uint8_t *)xr, v, a.C);
                        else nx[p].load(xr, v, a.C);
                    }
                }
            }
        }
        if constexpr (kRing) copy_commit();
        dyw.next();
        xw.next();
        ++fit;
    };
    if constexpr (kRing) {
#pragma unroll
        for (int p = 0; p < kS * 2 * NP; ++p) slot(0, p) = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int s = 0; s < kS - 1; ++s) fetch(s);
    } else {
        fetch(0);
    }
    uint32_t xs[NP];
    float mean[NR], rstd[NR];
    auto ahead = [&](int it) {  // what is small: one step ahead in registers
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            const bool live = w.live(it, j);
            const long long r = w.row(it, j);
            mean[j] = live ? a.mean[r] : 0.f;
            rstd[j] = live ? a.rstd[r] : 0.f;
            if constexpr (kCkpt == 1) {
                const uint8_t *sr = a.scales + r * ng;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    xs[j * NV + i] = live && in[i] ? sr[(i * tpr + t) / (kGroup / VEC)] : 0u;
            }
        }
    };
    ahead(0);
    f2 gw[NV][VP], dg[NV][VP], db[NV][VP];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int e = 0; e < VP; ++e) gw[i][e] = dg[i][e] = db[i][e] = 0;
        if (in[i]) load_weights<VEC>(a.gamma, a.wdt, (i * tpr + t) * VEC, a.C, a.wvec, 1.f, gw[i]);
    }
    int par = 0, cur = 0;
    if (kCta) __syncthreads();
    for (int it = 0; it < w.steps; ++it) {
        f2 xh[NP][VP], g[NP][VP];
        float sum[2 * NR], rs[NR];  // of g and of g xhat
        if constexpr (kRing) copy_wait<kS - 2>();
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            rs[j] = rstd[j];
            const f2 r2 = both(rs[j]), mm = both(-mean[j]);
            f2 sa2 = 0, sb2 = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int p = j * NV + i;
                Vec<T, VEC> dy;
                if constexpr (kRing) dy.set(slot(cur, p));
                else dy = ndy[p];
                if constexpr (kCkpt) {
                    Codes<VEC> c;
                    if constexpr (kRing) c.load(reinterpret_cast<const uint8_t *>(&slot(cur, NP + p)), 0, VEC);
                    else c = nc[p];
                    uint32_t sb = xs[p];
                    if constexpr (kCkpt == 2) {
                        const uint32_t word = *reinterpret_cast<const uint32_t *>(reinterpret_cast<const char *>(&slot(cur, NP + p)) + VEC);
                        sb = (word >> sbit[i]) & 0xffu;
                    }
                    c.decode_norm(sb, a.fmt, mean[j], rs[j], xh[p]);
                } else {
                    Vec<T, VEC> x;
                    if constexpr (kRing) x.set(slot(cur, NP + p));
                    else x = nx[p];
#pragma unroll
                    for (int e = 0; e < VP; ++e) xh[p][e] = x.pair(e);
                }
#pragma unroll
                for (int e = 0; e < VP; ++e) {
                    if constexpr (!kCkpt) xh[p][e] = mul2(add2(xh[p][e], mm), r2);
                    const f2 d = dy.pair(e);
                    dg[i][e] = fma2(d, xh[p][e], dg[i][e]);
                    db[i][e] = add2(db[i][e], d);
                    g[p][e] = mul2(d, gw[i][e]);
                    sa2 = add2(sa2, g[p][e]);
                    sb2 = fma2(g[p][e], xh[p][e], sb2);
                }
            }
            sum[2 * j] = low(sa2) + high(sa2);
            sum[2 * j + 1] = low(sb2) + high(sb2);
        }
        if constexpr (kRing) {  // into the slots that the step before has been read from
            fetch(cur == 0 ? kS - 1 : cur - 1);
            cur = cur == kS - 1 ? 0 : cur + 1;
        } else {
            fetch(0);
        }
        ahead(it + 1);
        if constexpr (kCta) {  // a slot is written again two rows on, behind the barrier of the row between
            rows_cta_sum(sum, red[par]);
            par ^= 1;
        } else {
            lanes_sum(sum, tpr);
        }
#pragma unroll
        for (int j = 0; j < NR; ++j)
            if (w.live(it, j)) {
                const f2 ma = both(-sum[2 * j] * a.invC), mb = both(-sum[2 * j + 1] * a.invC), r2 = both(rs[j]);
                char *dxr = dxw.at(a.dx, w, it, j);
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (in[i]) {
                        const int p = j * NV + i;
                        Vec<T, VEC> o;
#pragma unroll
                        for (int e = 0; e < VP; ++e)
                            o.set_pair(e, mul2(fma2(xh[p][e], mb, add2(g[p][e], ma)), r2));
                        o.store(dxr, i * tpr + t, a.C);
                    }
            }
        dxw.next();
    }
    if constexpr (kRing) copy_wait<0>();
    if (!a.part) return;
    float *pg = a.part + (size_t)blockIdx.x * 2 * a.C;
    if constexpr (kCta) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int c = (i * tpr + t) * VEC + e;
                if (c < a.C) {
                    pg[c] = e & 1 ? high(dg[i][e / 2]) : low(dg[i][e / 2]);
                    pg[a.C + c] = e & 1 ? high(db[i][e / 2]) : low(db[i][e / 2]);
                }
            }
    } else {  // the CTA's rows side by side: fold[row of the CTA][channel], summed in row order
        const int width = tpr * NV * VEC;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const f2 p = which ? db[i][e / 2] : dg[i][e / 2];
                    fold[w.sub * width + (i * tpr + t) * VEC + e] = e & 1 ? high(p) : low(p);
                }
            __syncthreads();
            for (int c = threadIdx.x; c < a.C; c += 256) {
                float s = 0.f;
                for (int p = 0; p < w.per; ++p) s += fold[p * width + c];
                pg[which * a.C + c] = s;
            }
        }
    }
}

// How a row is laid over one warp's lanes: NV pieces per lane, tpr lanes (nv =
// 0: it does not fit).  nvs: the NV to choose from, ascending.
struct Spread {
    int nvec, nv, tpr;
};
template <int VEC, int N>
Spread spread(int C, const int (&nvs)[N]) {
    Spread s{(C + VEC - 1) / VEC, 0, 0};
    for (int i = 0; i < N && !s.nv; ++i)
        if (s.nvec <= 32 * nvs[i]) {
            s.nv = nvs[i];
            s.tpr = kGroup / VEC;  // a scale group never leaves its row's lanes
            while (s.tpr * s.nv < s.nvec) s.tpr *= 2;
        }
    return s;
}

// Dynamic shared memory that every kernel here may be given beside its static
// part (at most 16.5 KB) of an SM's 227 KB.
constexpr size_t kMostSmem = 208 * 1024;

// Launches with dynamic shared memory; above 48 KB it has to be asked for,
// once per kernel and device.
template <typename Args>
prism_status launch(void (*kernel)(Args), const Args &a, int grid, int threads, size_t smem,
                    std::atomic<unsigned long long> &asked, cudaStream_t st) {
    if (smem > 31 * 1024) {  // the static part counts towards the 48 KB too
        int dev = 0;
        PRISM_CUDA_OK(cudaGetDevice(&dev));
        const unsigned long long bit = 1ull << (dev & 63);
        if (!(asked.load(std::memory_order_relaxed) & bit)) {
            PRISM_CUDA_OK(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostSmem));
            asked.fetch_or(bit, std::memory_order_relaxed);
        }
    }
    kernel<<<grid, threads, smem, st>>>(a);
    PRISM_CUDA_OK(cudaGetLastError());
    return PRISM_OK;
}

bool aligned16(const RowPtr &p, size_t row_bytes) {
    return (((uintptr_t)p.data | (uintptr_t)p.stride | (uintptr_t)p.group_stride | row_bytes) & 15) == 0;
}

// Partial weight gradients of the backward: one per CTA, at most 64 MB.
int partials(long long nrows, int C) {
    long long p = (64ll << 20) / (8ll * C);
    if (p > 592) p = 592;
    if (p > nrows) p = nrows;
    return p < 1 ? 1 : (int)p;
}

// ---- forward ----
template <typename T, int VEC, int NV, bool kCta, bool kCkpt>
prism_status run_fwd(const FwdArgs &a, cudaStream_t st) {
    // CTAs of 256 threads per SM by what NV costs in registers; with one row
    // per CTA, 512 threads' worth.  (Rows without a ring: what fits, and more.)
    constexpr bool kRing = VEC * sizeof(T) == 16;
    constexpr int kNR = fwd_rows(NV * VEC, kCta);
    constexpr int kPerSm = !kRing ? 8 : NV * VEC <= 16 ? 3 : 2;
    static std::atomic<unsigned long long> asked{0};
    const int per = (kCta ? 1 : 256 / a.tpr) * kNR, threads = kCta ? a.tpr : 256;
    const long long need = (a.nrows + per - 1) / per, most = 148ll * (kCta ? (kRing ? 768 : 2048) / a.tpr : kPerSm);
    size_t smem = kRing ? (size_t)ring(kNR * NV * 16) * kNR * NV * 16 * threads : 0;
    if (NV * VEC > 16) smem += (size_t)a.nvec * VEC * 8;  // gamma and beta
    return launch(k_norm_fwd<T, VEC, NV, kCta, kCkpt>, a, (int)(need < most ? need : most), threads, smem, asked, st);
}
// Whether a row's ring and its weights (fp32) fit: about 12500 channels of 16 bits, 8192 to 13000 of 32.
template <typename T, int VEC>
bool fwd_fits(int C) {
    const int nvec = (C + VEC - 1) / VEC;
    if (nvec <= 32 * 8) return true;
    const int nv = nvec <= 512 * 4 ? 4 : 8, threads = ((nvec + nv - 1) / nv + 31) / 32 * 32;
    const size_t slots = VEC * sizeof(T) == 16 ? (size_t)ring(nv * 16) * nv * 16 * threads : 0;
    return threads <= 512 && slots + (size_t)nvec * VEC * 8 <= kMostSmem;
}
template <typename T, int VEC, bool kCkpt>
prism_status fwd_spread(FwdArgs &a, cudaStream_t st) {
    static const int nvs[] = {1, 2, 3, 4, 6, 8, VEC == 2 ? 16 : 8};
    const Spread s = spread<VEC>(a.C, nvs);
    a.nvec = s.nvec;
    a.tpr = s.tpr;
    switch (s.nv) {
        case 1: return run_fwd<T, VEC, 1, false, kCkpt>(a, st);
        case 2: return run_fwd<T, VEC, 2, false, kCkpt>(a, st);
        case 3: return run_fwd<T, VEC, 3, false, kCkpt>(a, st);
        case 4: return run_fwd<T, VEC, 4, false, kCkpt>(a, st);
        case 6: return run_fwd<T, VEC, 6, false, kCkpt>(a, st);
        case 8: return run_fwd<T, VEC, 8, false, kCkpt>(a, st);
        case 16:
            if constexpr (VEC == 2) return run_fwd<T, VEC, 16, false, kCkpt>(a, st);
    }
    // one row per CTA of up to 512 threads
    const int nv = a.nvec <= 512 * 4 ? 4 : 8;
    a.tpr = ((a.nvec + nv - 1) / nv + 31) / 32 * 32;
    return nv == 4 ? run_fwd<T, VEC, 4, true, kCkpt>(a, st) : run_fwd<T, VEC, 8, true, kCkpt>(a, st);
}

template <typename T>
prism_status fwd_impl(const NormFwd &n, cudaStream_t st) {
    constexpr int VEC = 16 / sizeof(T);
    const size_t row = (size_t)n.C * sizeof(T);
    const bool vec = aligned16(n.x, row) && aligned16(n.y, row);
    if (vec ? fwd_fits<T, VEC>(n.C) : fwd_fits<T, 2>(n.C)) {
        FwdArgs a{n.x, n.y, n.gamma, n.beta, n.wdt, (((uintptr_t)n.gamma | (uintptr_t)n.beta) & 15) == 0,
                  n.mean, n.rstd, n.codes, n.scales, n.fmt, n.nrows, n.C, 0, 0, n.eps, 1.f / (float)n.C};
        if (vec) return n.codes ? fwd_spread<T, VEC, true>(a, st) : fwd_spread<T, VEC, false>(a, st);
        return n.codes ? fwd_spread<T, 2, true>(a, st) : fwd_spread<T, 2, false>(a, st);
    }
    const int grid = (int)(n.nrows < 148 * 8 ? n.nrows : 148 * 8);
    k_norm_fwd_any<T><<<grid, kThreads, 0, st>>>(n.x, n.y, n.gamma, n.beta, n.wdt, n.mean, n.rstd, n.codes, n.scales,
                                                 n.fmt, n.nrows, n.C, n.eps);
    PRISM_CUDA_OK(cudaGetLastError());
    return PRISM_OK;
}

// ---- backward ----
// Pieces per thread at most: 16 channels (dgamma, dbeta and gamma of each stay
// in registers), 8 where the next row waits in registers too.
template <int VEC>
constexpr int kBwdNV = VEC == 8 ? 2 : 4;

template <typename T, int VEC, int NV, int kCta, int kCkpt>
prism_status run_bwd(const BwdArgs &a, int &P, cudaStream_t st) {
    constexpr bool kRing = VEC * sizeof(T) == 16;
    constexpr int kNR = bwd_rows(NV * VEC, kCta);
    static std::atomic<unsigned long long> asked{0};
    const int per = (kCta ? 1 : 256 / a.tpr) * kNR, threads = kCta ? a.tpr : 256;
    const int per_sm = kCta == 0 ? 2 : kCta == 1 ? 384 / a.tpr : (kRing ? 512 : 768) / a.tpr;
    const long long need = (a.nrows + per - 1) / per, most = 148ll * per_sm;
    if (P > need) P = (int)need;
    if (P > most) P = (int)most;
    const size_t smem = kRing ? (size_t)bwd_ring(kNR * NV * 32) * kNR * NV * 32 * threads : 0;
    return launch(k_norm_bwd<T, VEC, NV, kCta, kCkpt>, a, P, threads, smem, asked, st);
}
// P: partials allowed; on return the partials written
template <typename T, int VEC, int kCkpt>
prism_status bwd_spread(BwdArgs &a, int &P, cudaStream_t st) {
    constexpr int kMost = kBwdNV<VEC>;
    static const int nvs[] = {kMost / 2, kMost};
    const Spread s = spread<VEC>(a.C, nvs);
    a.nvec = s.nvec;
    a.tpr = s.tpr;
    if (s.nv) return s.nv == kMost ? run_bwd<T, VEC, kMost, 0, kCkpt>(a, P, st)
                                   : run_bwd<T, VEC, kMost / 2, 0, kCkpt>(a, P, st);
    a.tpr = ((a.nvec + kMost - 1) / kMost + 31) / 32 * 32;
    if constexpr (VEC != 2)
        if (a.tpr <= 192) return run_bwd<T, VEC, kMost, 1, kCkpt>(a, P, st);
    return run_bwd<T, VEC, kMost, 2, kCkpt>(a, P, st);
}

template <typename T>
prism_status bwd_impl(const NormBwd &n, cudaStream_t st) {
    constexpr int VEC = 16 / sizeof(T);
    int P = partials(n.nrows, n.C);
    float *part = n.dgamma || n.dbeta ? n.part : nullptr;
    const size_t row = (size_t)n.C * sizeof(T);
    // codes and scales are 16-byte aligned and packed: a row of a multiple of VEC codes is aligned to VEC
    const bool vec = (n.codes ? n.C % VEC == 0 : aligned16(n.x, row)) && aligned16(n.dy, row) && aligned16(n.dx, row);
    if (n.nrows > 0 && n.C <= 512 * (vec ? 16 : 8)) {
        RowPtr x = n.x;
        if (n.codes) x = RowPtr{(char *)n.codes, n.C, 0, 0};
        BwdArgs a{x, n.dy, n.dx, n.scales, n.fmt, n.gamma, n.wdt, ((uintptr_t)n.gamma & 15) == 0,
                  n.mean, n.rstd, part, n.nrows, n.C, 0, 0, 1.f / (float)n.C};
        prism_status s;
        const bool words = (n.C + kGroup - 1) / kGroup % 4 == 0;
        if (vec) s = !n.codes ? bwd_spread<T, VEC, 0>(a, P, st)
                     : words  ? bwd_spread<T, VEC, 2>(a, P, st)
                              : bwd_spread<T, VEC, 1>(a, P, st);
        else s = n.codes ? bwd_spread<T, 2, 1>(a, P, st) : bwd_spread<T, 2, 0>(a, P, st);
        if (s != PRISM_OK) return s;
    } else {
        const Source<T> src{n.x, n.codes, n.scales, n.fmt, n.C};
        if (n.nrows > 0) {
            const int grid = (int)(n.nrows < 148 * 8 ? n.nrows : 148 * 8);
            k_norm_dx_any<T><<<grid, kThreads, 0, st>>>(src, n.dy, n.dx, n.gamma, n.wdt, n.mean, n.rstd, n.nrows, n.C);
            PRISM_CUDA_OK(cudaGetLastError());
        }
        if (part) {
            k_norm_dw_any<T><<<dim3((n.C + kThreads - 1) / kThreads, P), kThreads, 0, st>>>(src, n.dy, n.mean, n.rstd,
                                                                                            part, n.nrows, n.C);
            PRISM_CUDA_OK(cudaGetLastError());
        }
    }
    if (part) {
        k_norm_dw_sum<<<(n.C + 31) / 32, 1024, 0, st>>>(part, P, n.dgamma, n.dbeta, n.wdt, n.C);
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
