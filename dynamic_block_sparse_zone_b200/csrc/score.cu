// score.cu -- the scores and masks of a plan's scored attention: the caller's
// per-token positions, documents and visibility in block-contiguous order, and
// the plan's selection without the block pairs that the mask hides.
//
// A pair of blocks is hidden when no query of the one may see a key of the
// other (their documents do not meet, or every key lies behind every query),
// whole when every query sees every key, and partly visible otherwise.  The
// decision reads only each block's ranges, so it can call a pair partly visible
// that is hidden or whole; such a pair is looked at again by the kernels' units
// of work, 128 rows of its own block by 64 of the other, and by the kernels in
// groups of 32 keys by 32 or 16 queries, and only what is left token by token.
// Hidden units, most of a selection over packed clips, cost nothing after this
// (24 x 32 x 40 tokens in three causal clips: 65% of the selected pairs are in
// block pairs that are not hidden, 56% in such units, 22% are visible).
#include "tc_common.cuh"

namespace prism {

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) k_score_tokens(Geo g, const int *__restrict__ perm,
                                                           const float *__restrict__ pos, const int *__restrict__ doc,
                                                           bool causal, const float *__restrict__ prefix,
                                                           const float *__restrict__ slopes,
                                                           float *__restrict__ pos_p, float *__restrict__ vis_p,
                                                           int *__restrict__ doc_p, float *__restrict__ slopes_p,
                                                           GroupRange *__restrict__ qgrp, GroupRange *__restrict__ kgrp) {
    const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x;
    if (slopes && i < (size_t)g.heads) slopes_p[i] = slopes[i];
    if (i >= (size_t)g.batch * g.N) return;  // N is a multiple of 64: whole warps
    const int b = (int)(i / g.N), tok = perm[i];
    const size_t src = (size_t)b * g.N + tok;
    const float p = pos ? pos[src] : (float)(tok / (g.H * g.W));
    const int d = doc ? doc[src] : 0;
    pos_p[i] = p;
    doc_p[i] = d < 0 ? -1 : d;
    const float v = d < 0 ? INFINITY : !causal || (prefix && p < prefix[b]) ? -INFINITY : p;
    vis_p[i] = v;
    GroupRange q{d < 0 ? INFINITY : p, d < 0 ? -INFINITY : p, max(d, -1), max(d, -1)}, k{v, v, q.dmin, q.dmax};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        if (o == 16 && (i & 15) == 0) qgrp[i / 16] = q;
        q.lo = fminf(q.lo, __shfl_xor_sync(0xffffffffu, q.lo, o));
        q.hi = fmaxf(q.hi, __shfl_xor_sync(0xffffffffu, q.hi, o));
        k.lo = fminf(k.lo, __shfl_xor_sync(0xffffffffu, k.lo, o));
        k.hi = fmaxf(k.hi, __shfl_xor_sync(0xffffffffu, k.hi, o));
        q.dmin = min(q.dmin, __shfl_xor_sync(0xffffffffu, q.dmin, o));
        q.dmax = max(q.dmax, __shfl_xor_sync(0xffffffffu, q.dmax, o));
    }
    if ((i & 31) == 0) kgrp[i / 32] = GroupRange{k.lo, k.hi, q.dmin, q.dmax};
}

// One warp per block.
__global__ void __launch_bounds__(kThreads) k_score_blocks(Geo g, const int *__restrict__ nb, const int *__restrict__ blk_off,
                                                           const float *__restrict__ pos, const float *__restrict__ vis,
                                                           const int *__restrict__ doc, BlockRange *__restrict__ out) {
    const int b = blockIdx.y, j = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (j >= nb[b]) return;
    const int *bo = blk_off + (size_t)b * (g.nbmax + 1);
    BlockRange r{INFINITY, -INFINITY, INFINITY, -INFINITY, 0x7fffffff, -1, 0, 0};
    for (int n = bo[j] + lane; n < bo[j + 1]; n += 32) {
        const size_t i = (size_t)b * g.N + n;
        if (doc[i] < 0) {
            ++r.pads;
            continue;
        }
        ++r.tokens;
        r.pmin = fminf(r.pmin, pos[i]);
        r.pmax = fmaxf(r.pmax, pos[i]);
        r.kmin = fminf(r.kmin, vis[i]);
        r.kmax = fmaxf(r.kmax, vis[i]);
        r.dmin = min(r.dmin, doc[i]);
        r.dmax = max(r.dmax, doc[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        r.pmin = fminf(r.pmin, __shfl_xor_sync(0xffffffffu, r.pmin, o));
        r.pmax = fmaxf(r.pmax, __shfl_xor_sync(0xffffffffu, r.pmax, o));
        r.kmin = fminf(r.kmin, __shfl_xor_sync(0xffffffffu, r.kmin, o));
        r.kmax = fmaxf(r.kmax, __shfl_xor_sync(0xffffffffu, r.kmax, o));
        r.dmin = min(r.dmin, __shfl_xor_sync(0xffffffffu, r.dmin, o));
        r.dmax = max(r.dmax, __shfl_xor_sync(0xffffffffu, r.dmax, o));
        r.tokens += __shfl_xor_sync(0xffffffffu, r.tokens, o);
        r.pads += __shfl_xor_sync(0xffffffffu, r.pads, o);
    }
    if (lane == 0) out[(size_t)b * g.nbmax + j] = r;
}

// 0 hidden, 1 whole, 2 partly visible
__device__ __forceinline__ int pair_class(const BlockRange &q, const BlockRange &k) {
    if (q.tokens == 0 || k.tokens == 0 || q.dmax < k.dmin || k.dmax < q.dmin || k.kmin > q.pmax) return 0;
    const bool one = q.dmin == q.dmax && k.dmin == k.dmax && q.dmin == k.dmin;
    return one && q.pads == 0 && k.pads == 0 && k.kmax <= q.pmin ? 1 : 2;
}

__device__ __forceinline__ GroupRange both_ranges(const GroupRange &a, const GroupRange &b) {
    return GroupRange{fminf(a.lo, b.lo), fmaxf(a.hi, b.hi), min(a.dmin, b.dmin), max(a.dmax, b.dmax)};
}
// seg[0]: of 64 queries each, seg[1]: of 64 keys.
__global__ void __launch_bounds__(kThreads) k_score_segments(size_t segs, const GroupRange *__restrict__ qgrp,
                                                             const GroupRange *__restrict__ kgrp,
                                                             GroupRange *__restrict__ seg) {
    const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= segs) return;
    seg[i] = both_ranges(both_ranges(qgrp[4 * i], qgrp[4 * i + 1]), both_ranges(qgrp[4 * i + 2], qgrp[4 * i + 3]));
    seg[segs + i] = both_ranges(kgrp[2 * i], kgrp[2 * i + 1]);
}

// A list's entry for block j (see list_block) beside its own block; -1: hidden.
// own, other: the ranges of their segments.
template <bool kCols>
__device__ __forceinline__ int list_entry(int j, int cls, int own_rows, int rows, const GroupRange *__restrict__ own,
                                          const GroupRange *__restrict__ other) {
    const int segs = rows >> 6, tiles = (own_rows + 127) >> 7;
    if (cls != 2) return cls == 0 ? -1 : j << 9 | ((1 << segs) - 1) * (tiles == 2 ? 17 : 1) << 1;
    int seen = 0, partly = 0;
    for (int t = 0; t < tiles; ++t) {
        GroupRange a = own[2 * t];
        if (own_rows > 64) a = both_ranges(a, own[2 * t + 1]);
        for (int s = 0; s < segs; ++s) {
            const GroupRange x = other[s];
            const GroupRange &q = kCols ? x : a, &k = kCols ? a : x;
            const int c = tc::group_class(q.lo, q.hi, q.dmin, q.dmax, k.lo, k.hi, k.dmin, k.dmax);
            seen |= (c != 0) << (4 * t + s);
            partly |= c == 2;
        }
    }
    return seen ? j << 9 | seen << 1 | partly : -1;
}

// One warp per list: the entries that are not hidden, in order, at the list's
// own place; a list's end is written beside.  kCols: the list of a key block
// holds query blocks.
template <bool kCols>
__global__ void __launch_bounds__(kThreads) k_score_filter(Geo g, const int *__restrict__ ptr, const int *__restrict__ list,
                                                           const int *__restrict__ blk_off,
                                                           const BlockRange *__restrict__ blk,
                                                           const GroupRange *__restrict__ seg, int *__restrict__ end,
                                                           int *__restrict__ out) {
    const size_t lists = (size_t)g.batch * g.heads * g.nbmax;
    const int lane = threadIdx.x & 31;
    for (size_t r = (size_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < lists;
         r += (size_t)gridDim.x * (kThreads / 32)) {
        const int p0 = ptr[r], p1 = ptr[r + 1];
        const size_t b = r / g.nbmax / g.heads, per = g.N / 64, segs = g.batch * per;
        const BlockRange *bb = blk + b * g.nbmax;
        const int *bo = blk_off + b * (g.nbmax + 1);
        const GroupRange *so = seg + (kCols ? segs : 0) + b * per, *sx = seg + (kCols ? 0 : segs) + b * per;
        int w = p0;
        if (p0 < p1) {
            const BlockRange own = bb[r % g.nbmax];
            const int o0 = bo[r % g.nbmax], o1 = bo[r % g.nbmax + 1];
            for (int u0 = p0; u0 < p1; u0 += 32) {
                const int u = u0 + lane;
                const int j = u < p1 ? list[u] : 0;
                const int c = u < p1 ? (kCols ? pair_class(bb[j], own) : pair_class(own, bb[j])) : 0;
                const int x0 = bo[j], e = list_entry<kCols>(j, c, o1 - o0, bo[j + 1] - x0, so + o0 / 64, sx + x0 / 64);
                const unsigned kept = __ballot_sync(0xffffffffu, e >= 0);
                if (e >= 0) out[w + __popc(kept & ((1u << lane) - 1))] = e;
                w += __popc(kept);
            }
        }
        if (lane == 0) end[r] = w;
    }
}

// Segments that each tile streams (one warp per tile; y: forward, backward).
__global__ void __launch_bounds__(kThreads) k_score_work(Geo g, const int *__restrict__ nqt, const int *__restrict__ qt_row,
                                                         const int *__restrict__ qt_blk,
                                                         const int *__restrict__ blk_off, const int *__restrict__ row_ptr,
                                                         const int *__restrict__ row_end, const int *__restrict__ col,
                                                         const int *__restrict__ colT_ptr, const int *__restrict__ colT_end,
                                                         const int *__restrict__ rowT, int *__restrict__ work) {
    const size_t tiles = (size_t)g.batch * g.heads * g.nbmax;
    const size_t t = (size_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (t >= tiles) return;
    const int lane = threadIdx.x & 31, tile = (int)(t % g.nbmax), b = (int)(t / g.nbmax / g.heads);
    int n = -1;
    if (tile < nqt[b]) {
        const bool back = blockIdx.y;
        const int *ptr = back ? colT_ptr : row_ptr, *end = back ? colT_end : row_end, *list = back ? rowT : col;
        int j1, j2;
        tc::tile_blocks(qt_blk[(size_t)b * g.nbmax + tile], j1, j2);
        const size_t l = t - tile + j1;
        const int a0 = ptr[l], a1 = end[l], b0 = j2 >= 0 ? ptr[l + 1] : 0, b1 = j2 >= 0 ? end[l + 1] : 0;
        const int *bo = blk_off + (size_t)b * (g.nbmax + 1);
        n = tc::union_segments<true>(list + a0, a1 - a0, list + b0, b1 - b0, bo,
                                     (qt_row[(size_t)b * g.nbmax + tile] - bo[j1]) >> 7, lane);
    }
    if (lane == 0) work[blockIdx.y * tiles + t] = n;
}

// Launch order of all tiles (one CTA per direction): the ones with the most
// segments first, or as they are.  Masks leave tiles of very different lengths;
// started last, a long one runs alone at the end.  Tiles of equal length come in
// no fixed order: no result depends on it but the order in which dQ's partial
// sums arrive.
constexpr int kBins = 1024;
__global__ void __launch_bounds__(kBins) k_score_order(Geo g, bool sort_f, bool sort_b, const int *__restrict__ work,
                                                       int *__restrict__ order, int *__restrict__ status, int kind,
                                                       float cap) {
    if (blockIdx.y == 0 && threadIdx.x == 0) {  // the last kernel of a set_score: from here on the lists are these
        status[kStKind] = kind;
        status[kStCap] = __float_as_int(cap);
    }
    __shared__ int cursor[kBins];
    __shared__ int sums[kBins / 32];
    const size_t tiles = (size_t)g.batch * g.heads * g.nbmax;
    const int n = (int)tiles, tid = threadIdx.x, lane = tid & 31;
    const int *w = work + blockIdx.y * tiles;
    int *out = order + blockIdx.y * tiles;
    if (!(blockIdx.y ? sort_b : sort_f)) {
        for (int i = tid; i < n; i += kBins) out[i] = w[i] >= 0 ? i : -1;
        return;
    }
    auto bin = [](int v) { return kBins - 1 - min(v, kBins - 1); };  // longest first
    cursor[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kBins) {
        out[i] = -1;
        if (w[i] >= 0) atomicAdd(&cursor[bin(w[i])], 1);
    }
    __syncthreads();
    const int mine = cursor[tid];  // exclusive scan of the counts
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[tid >> 5] = x;
    __syncthreads();
    int before = 0;
    for (int k = 0; k < (tid >> 5); ++k) before += sums[k];
    __syncthreads();
    cursor[tid] = before + x - mine;
    __syncthreads();
    for (int i = tid; i < n; i += kBins)
        if (w[i] >= 0) out[atomicAdd(&cursor[bin(w[i])], 1)] = i;
}

// Rows of padding tokens become zero: what they hold (infinities, NaN) would
// reach other rows through products with P = 0.  A thread looks at one token;
// CTAs without padding are done then.
__global__ void __launch_bounds__(kThreads) k_zero_padding(Geo g, const int *__restrict__ doc, __nv_bfloat16 *__restrict__ Qp,
                                                           __nv_bfloat16 *__restrict__ Kp, __nv_bfloat16 *__restrict__ Vp,
                                                           int *__restrict__ status, ScoreArgs sc) {
    if (!tc::own_scores(status, sc)) return;
    const int b = blockIdx.y, n0 = blockIdx.x * kThreads + (threadIdx.x & ~31), lane = threadIdx.x & 31;
    const bool pad = n0 + lane < g.N && doc[(size_t)b * g.N + n0 + lane] < 0;
    const int per = g.D / 8;
    for (unsigned left = __ballot_sync(0xffffffffu, pad); left; left &= left - 1) {
        const int n = n0 + __ffs(left) - 1;
        for (int i = lane; i < g.heads * per; i += 32) {
            const size_t at = (((size_t)b * g.heads + i / per) * g.N + n) * g.D + i % per * 8;
            *reinterpret_cast<uint4 *>(Qp + at) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(Kp + at) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(Vp + at) = make_uint4(0, 0, 0, 0);
        }
    }
}

struct Buf {
    void **p;
    size_t bytes;
};
constexpr int kBuffers = 17;
int buffers(Plan &pl, Buf *out) {
    const Geo &g = pl.g;
    Score &s = pl.score;
    const size_t lists = (size_t)g.batch * g.heads * g.nbmax, nnz = lists * (size_t)pl.cap_stride;
    const size_t tokens = (size_t)g.batch * g.N;
    int n = 0;
    out[n++] = {(void **)&s.slopes, (size_t)g.heads * sizeof(float)};
    out[n++] = {(void **)&s.pos, tokens * sizeof(float)};
    out[n++] = {(void **)&s.vis, tokens * sizeof(float)};
    out[n++] = {(void **)&s.doc, tokens * sizeof(int)};
    out[n++] = {(void **)&s.blk, (size_t)g.batch * g.nbmax * sizeof(BlockRange)};
    out[n++] = {(void **)&s.qgrp, tokens / 16 * sizeof(GroupRange)};
    out[n++] = {(void **)&s.kgrp, tokens / 32 * sizeof(GroupRange)};
    out[n++] = {(void **)&s.seg, 2 * (tokens / 64) * sizeof(GroupRange)};
    out[n++] = {(void **)&s.row_end, lists * sizeof(int)};
    out[n++] = {(void **)&s.colT_end, lists * sizeof(int)};
    out[n++] = {(void **)&s.order, 2 * lists * sizeof(int)};
    out[n++] = {(void **)&s.work, 2 * lists * sizeof(int)};
    out[n++] = {(void **)&s.redo, (1 + lists) * sizeof(int)};
    out[n++] = {(void **)&s.Olo, (size_t)g.heads * tokens * g.D * 2};
    out[n++] = {(void **)&s.col, nnz * sizeof(int)};
    out[n++] = {(void **)&s.rowT, nnz * sizeof(int)};
    return n;
}

}  // namespace

void release_score(Plan &pl) {
    Buf b[kBuffers];
    const int n = buffers(pl, b);
    for (int k = 0; k < n; ++k)
        if (*b[k].p) {
            cudaFree(*b[k].p);
            *b[k].p = nullptr;
        }
    pl.score.set = false;
}

// Before every scored pass over the plan's copies (not once for all: a captured
// forward may be replayed behind an update that was not captured).
prism_status launch_zero_padding(Plan &pl, cudaStream_t st) {
    const Geo &g = pl.g;
    if (!pl.score.has_doc) return PRISM_OK;
    pl.score.zeroed = true;
    k_zero_padding<<<dim3((g.N + kThreads - 1) / kThreads, g.batch), kThreads, 0, st>>>(g, pl.score.doc, pl.Qp, pl.Kp, pl.Vp,
                                                                                           pl.status, score_args(pl, false));
    PRISM_CUDA_OK(cudaGetLastError());
    return PRISM_OK;
}

prism_status set_score(Plan &pl, const prism_score &in, cudaStream_t st) {
    const Geo &g = pl.g;
    Score &s = pl.score;
    if (s.zeroed)
        return fail(PRISM_ERR_STATE, "a scored forward has zeroed padding tokens in the plan's Q, K, V: bring them in again "
                                     "(build or update_qkv) before other scores");
    s.set = false;
    if (!s.rowT) {
        cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
        PRISM_CUDA_OK(cudaStreamIsCapturing(st, &cap));
        if (cap != cudaStreamCaptureStatusNone)
            return fail(PRISM_ERR_STATE, "a plan's first prism_plan_set_score allocates: make it before the capture");
        Buf b[kBuffers];
        const int n = buffers(pl, b);
        for (int k = 0; k < n; ++k) {
            const cudaError_t e = cudaMalloc(b[k].p, b[k].bytes);
            if (e != cudaSuccess) {
                *b[k].p = nullptr;
                cudaGetLastError();  // the failed allocation is reported here, not by a later call
                release_score(pl);
                return fail_cuda(e, "cudaMalloc", __FILE__, __LINE__);
            }
        }
    }
    s.cap = in.cap;
    s.has_bias = in.slopes != nullptr;
    s.has_doc = in.doc != nullptr;
    s.causal = in.causal != 0;
    size_t n = (size_t)g.batch * g.N;
    if ((size_t)g.heads > n) n = g.heads;
    k_score_tokens<<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(
        g, pl.perm, in.pos, in.doc, in.causal != 0, in.prefix, in.slopes, s.pos, s.vis, s.doc, s.slopes, s.qgrp, s.kgrp);
    PRISM_CUDA_OK(cudaGetLastError());
    k_score_blocks<<<dim3((g.nbmax + kThreads / 32 - 1) / (kThreads / 32), g.batch), kThreads, 0, st>>>(
        g, pl.nb, pl.blk_off, s.pos, s.vis, s.doc, s.blk);
    PRISM_CUDA_OK(cudaGetLastError());
    const size_t segs = (size_t)g.batch * g.N / 64;
    k_score_segments<<<(unsigned)((segs + kThreads - 1) / kThreads), kThreads, 0, st>>>(segs, s.qgrp, s.kgrp, s.seg);
    PRISM_CUDA_OK(cudaGetLastError());
    k_score_filter<false><<<1184, kThreads, 0, st>>>(g, pl.row_ptr, pl.col, pl.blk_off, s.blk, s.seg, s.row_end, s.col);
    PRISM_CUDA_OK(cudaGetLastError());
    k_score_filter<true><<<1184, kThreads, 0, st>>>(g, pl.colT_ptr, pl.rowT, pl.blk_off, s.blk, s.seg, s.colT_end,
                                                        s.rowT);
    PRISM_CUDA_OK(cudaGetLastError());
    const size_t tiles = (size_t)g.batch * g.heads * g.nbmax;
    k_score_work<<<dim3((unsigned)((tiles + kThreads / 32 - 1) / (kThreads / 32)), 2), kThreads, 0, st>>>(
        g, pl.nqt, pl.qt_row, pl.qt_blk, pl.blk_off, pl.row_ptr, s.row_end, s.col, pl.colT_ptr, s.colT_end, s.rowT, s.work);
    PRISM_CUDA_OK(cudaGetLastError());
    // Sorted while the tail counts more than neighbouring tiles' common blocks in L2:
    // forward, K and V of all heads within L2 or nearly; backward, up to eight tiles
    // per SM.  Measured as they are -> sorted, in ms, cap and bias | packed causal clips,
    // heads of 128, random block shapes:
    //   tokens, heads   K and V  forward                   tiles per SM  backward
    //   16x32x32, 8      67 MB   0.63->0.52 | 0.44->0.32     6.9  1.40->1.24 | 0.92->0.75
    //   24x32x40, 8     126 MB   2.06->1.81 | 0.76->0.63    13    4.75->4.35 | 1.61->1.53
    //   24x48x80, 4     189 MB   1.94->1.79 | 0.75->0.67    19    5.49->5.00 | 1.95->1.86
    //   24x48x80, 24    1.1 GB   12.4->10.8 | 4.14->3.91   117    34.0->32.0 | 10.7->11.6
    //   24x96x160, 24   4.5 GB   193->199 | 58.2->57.0     467    564->586 | 162->198
    // Both limits are on the safe side: where they stop, the order still gains up to a
    // tenth; the largest packed backward loses a fifth.
    const int BH = g.batch * g.heads;
    const bool sort_f = (double)BH * g.N * g.D * 4 <= 160e6, sort_b = (long long)BH * (g.N / 128) <= 8 * 148;
    k_score_order<<<dim3(1, 2), kBins, 0, st>>>(g, sort_f, sort_b, s.work, s.order, pl.status, score_kind(s), s.cap);
    PRISM_CUDA_OK(cudaGetLastError());
    s.set = true;
    return PRISM_OK;
}

ScoreArgs score_args(const Plan &pl, bool backward) {
    const Score &s = pl.score;
    ScoreArgs a{};
    a.list_end = backward ? s.colT_end : s.row_end;
    a.order = s.order + (backward ? (size_t)pl.g.batch * pl.g.heads * pl.g.nbmax : 0);
    a.pos = s.pos;
    a.vis = s.vis;
    a.doc = s.doc;
    a.qgrp = s.qgrp;
    a.kgrp = s.kgrp;
    a.slopes = s.slopes;
    a.Olo = s.Olo;
    a.redo = s.redo;
    a.kind = score_kind(s);
    a.cap = s.cap;
    if (s.cap > 0.f) {
        a.cap_one = (float)(sqrt((double)pl.g.D) * (double)s.cap);
        a.cap_u = (float)(1.0 / (sqrt((double)pl.g.D) * (double)s.cap));
        a.cap_in = (float)(2.0 * 1.4426950408889634 / (sqrt((double)pl.g.D) * (double)s.cap));
        a.cap_out = (float)((double)s.cap * 1.4426950408889634);
    }
    return a;
}

}  // namespace prism
