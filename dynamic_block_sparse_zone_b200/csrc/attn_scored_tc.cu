// attn_scored_tc.cu -- block-sparse attention forward with scores and masks, on
// the tcgen05 tensor cores.
//
//   logit = cap tanh(s / cap) - slope_h |p_q - p_k|,  s = q.k / sqrt(D),
//   visible = doc_q == doc_k and vis_k <= p_q,  P = exp(logit) where visible,
//   O = P V / sum P, lse = log sum P.
//
// Work unit: one 128-row query tile of one head, as in the unscored forward; its
// selected key blocks, without the pairs that the mask hides (score.cu), are
// streamed as 64-row segments.  Tiles are launched longest first.
//
// What the score needs (13 instructions per score with everything on, against 4
// for a plain softmax) makes the softmax the longest stage, and the chain S ->
// softmax -> P V the loss: four softmax warps in the unscored forward's strictly
// ordered pipeline issued 0.32 instructions per cycle and scheduler.  Here
// nothing ties one segment to the next but the sum in O:
//   - the reference of the exponential is 0, not a running maximum: P and the
//     sums are floating point, so a row is right as long as its sum lies in
//     [2^-30, 2^80] (largest logits of -20 to 55) and O stays finite.  A tile with
//     a row outside is put on a list and done again by the variant with a running
//     maximum (attn_tc.cu), launched behind this kernel; the list is empty for
//     ordinary scores (16 x 32 x 32 tokens, 8 heads of 128, without scores: 393 us,
//     with every tile done again 1001 us);
//   - segments alternate between two independent chains, each with its own 64
//     columns of S / P in TMEM, K and V buffers, barriers and four softmax warps
//     (one query row per thread).  Two CTAs share an SM: four chains.
// Warp roles (320 threads):
//   warp 0       TMA producer: Q once; per segment K, V and the keys' positions,
//                visibilities and documents (64 each, only what is needed)
//   warp 1       MMA issuer: S_i = Q K_i^T (N = 64), O += P_i V_i, in segment order
//   warps 2..5   softmax of the even segments, 6..9 of the odd ones
// P goes to the tensor cores as hi + lo, two bf16 numbers and two products with
// V: an 8-bit O may be kept for the backward, and a P of 8 bits moves O by about
// half a step of bf16, enough for every tenth 8-bit code to fall on the other
// side and Delta with it (dQ off by up to 0.012 in relative norm, 0.0025 so).
// Measured on 24 x 32 x 40 tokens, 8 heads of 128, 9.7e11 FLOP of selected pairs
// (none, with the same selection unscored: 1.03 ms, 942 TFLOP/s): without scores
// 1.16 ms, cap 1.59, bias 1.25, both 1.75 ms; 16 x 32 x 32 tokens with both:
// 514 us, 510 TFLOP/s, where the tensor cores are busy 44% of the cycles, the
// FMA pipe 49% and 0.54 instructions are issued per cycle and scheduler: bound by
// the latency of the softmax's instructions, 14 per score.
// TMEM columns: S / P of the chains [0, 64) and [64, 128) (in each 32 of them, hi
// in the first 16 and lo in the second), O [128, 128 + D).
#include <cuda.h>

#include "score_tc.cuh"

namespace prism {

using namespace tc;

namespace segtc {

constexpr int kThreads = 320;
constexpr uint32_t kTmemCols = 256;
constexpr float kLeast = 9.31322575e-10f, kMost = 1.20892582e24f;  // 2^-30, 2^80

template <int D>
struct Layout {
    static constexpr int kHalves = D / 64;             // 64-column (128 B) swizzle atoms along D
    static constexpr uint32_t kTileBytes = 128 * 128;  // 128 rows x 128 B; a segment's 64 rows are half of it
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kK = kQ + kHalves * kTileBytes;
    static constexpr uint32_t kV = kK + kHalves * kTileBytes;
    static constexpr uint32_t kBars = kV + kHalves * kTileBytes;
    // q, o, then [2] of k_full, k_empty, v_full, v_empty, s, p, then [4] of meta
    static constexpr uint32_t kNumBars = 2 + 6 * 2 + 4;
    static constexpr uint32_t kWords = kBars + kNumBars * 8;  // tmem slot, abort, put-off flag, -, mask[4]
    static constexpr uint32_t kMeta = (kWords + 32 + 15) & ~15u;
    static constexpr uint32_t kMetaSlot = 3 * 256 + 32;       // positions, visibilities, documents of 64 keys, their ranges
    static constexpr uint32_t kExch = kMeta + 4 * kMetaSlot;  // [chain][row] sums, then "has seen a key"
    static constexpr uint32_t kAlloc = kExch + 4 * 512 + 1024;
};

enum { kSiteQ = 31, kSiteK, kSiteV, kSiteKEmpty, kSiteVEmpty, kSiteS, kSiteP, kSiteO, kSiteMeta };

template <int D, int kScore>
__global__ void __launch_bounds__(kThreads, 2)
    k_attn_fwd_scored(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, Geo g, const int *__restrict__ qt_row,
                      const int *__restrict__ qt_blk, const int *__restrict__ blk_off, const int *__restrict__ row_ptr,
                      const int *__restrict__ col, const int *__restrict__ perm, __nv_bfloat16 *__restrict__ O,
                      float *__restrict__ lse_user, float *__restrict__ nlse_p, float scale_log2,
                      int *__restrict__ status, ScoreArgs sc) {
    using L = Layout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_u32(smem);

    if (!own_scores(status, sc)) return;
    const int tid = sc.order[blockIdx.y * gridDim.x + blockIdx.x];
    if (tid < 0) return;
    const int bh = tid / g.nbmax, tile = tid - bh * g.nbmax, b = bh / g.heads, h = bh % g.heads;
    if (*reinterpret_cast<volatile int *>(status) != 0) return;  // an earlier CTA timed out: fail fast
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int *bo = blk_off + (size_t)b * (g.nbmax + 1);
    const int q0 = qt_row[(size_t)b * g.nbmax + tile];
    int iblk, iblk2;
    tile_blocks(qt_blk[(size_t)b * g.nbmax + tile], iblk, iblk2);
    const bool shared_tile = iblk2 >= 0;
    const int qvalid = min(128, bo[(shared_tile ? iblk2 : iblk) + 1] - q0);
    const size_t crow = (size_t)bh * g.nbmax + iblk;
    const int c_begin = row_ptr[crow], c_end = sc.list_end[crow];
    // the second query block's selection (empty unless the tile is shared)
    const int c2_begin = shared_tile ? row_ptr[crow + 1] : 0, c2_end = shared_tile ? sc.list_end[crow + 1] : 0;
    const int own = (q0 - bo[iblk]) >> 7;  // which 128 rows of its block the tile is
    const int nseg = union_segments<true>(col + c_begin, c_end - c_begin, col + c2_begin, c2_end - c2_begin, bo, own, lane);

    const uint32_t bar_q = sbase + L::kBars, bar_o = bar_q + 8;
    const uint32_t bar_kf = bar_q + 16, bar_ke = bar_kf + 16, bar_vf = bar_ke + 16, bar_ve = bar_vf + 16;
    const uint32_t bar_s = bar_ve + 16, bar_p = bar_s + 16, bar_m = bar_p + 16;
    uint32_t *words = reinterpret_cast<uint32_t *>(smem + L::kWords);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(words + 1);
    volatile int *put_off = reinterpret_cast<volatile int *>(words + 2);
    volatile uint32_t *mask_w = words + 4;

    if (warp == 0) {
        if (lane == 0) {
            mbar_init(bar_q, 1);
            mbar_init(bar_o, 1);
            for (int s = 0; s < 2; ++s) {
                mbar_init(bar_kf + 8 * s, 1);
                mbar_init(bar_ke + 8 * s, 1);
                mbar_init(bar_vf + 8 * s, 1);
                mbar_init(bar_ve + 8 * s, 1);
                mbar_init(bar_s + 8 * s, 1);
                mbar_init(bar_p + 8 * s, 128);
            }
            for (int s = 0; s < 4; ++s) mbar_init(bar_m + 8 * s, 1);
            *abort_flag = 0;
            *put_off = 0;
            mbar_fence_init();
            prefetch_map(&tmQ);
            prefetch_map(&tmK);
            prefetch_map(&tmV);
        }
        __syncwarp();
        tmem_alloc(smem_u32(words), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = words[0];
    const uint32_t tO = tmem + 128;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            const int rowbase = bh * g.N;
            mbar_expect_tx(bar_q, 128 * D * 2);
            for (int hf = 0; hf < L::kHalves; ++hf)
                for (int rh = 0; rh < 2; ++rh)
                    tma_load_2d(sbase + L::kQ + hf * L::kTileBytes + rh * 8192, &tmQ, bar_q, hf * 64,
                                rowbase + q0 + rh * 64);
            SegWalk<true> wk;
            wk.init(c_begin, c_end, c2_begin, c2_end, col, bo, own);
            int kissued = 0, vissued = 0;
            // K of segment i and its keys' data, once S_{i-2} has read the K buffer.  The
            // data's slot is free then too: S_{i-2} was issued behind P_{i-4} V_{i-4}, so
            // the softmax has published P_{i-4}.
            auto issue_k = [&](int i) -> bool {
                const int s = i & 1, ms = i & 3;
                if (i >= 2 && !mbar_wait(bar_ke + 8 * s, ((i >> 1) - 1) & 1, status, kSiteKEmpty, abort_flag)) return false;
                const bool part = (kScore & kMask) && wk.mask >> 2;
                const size_t n0 = (size_t)b * g.N + wk.r;
                const uint32_t meta = sbase + L::kMeta + ms * L::kMetaSlot, bm = bar_m + 8 * ms;
                mask_w[ms] = (uint32_t)wk.mask;  // published by the arrive below
                mbar_expect_tx(bm, ((kScore & kBias) ? 256 : 0) + (part ? 512 + 32 : 0));
                if (kScore & kBias) bulk_load(meta, sc.pos + n0, 256, bm);
                if (part) {
                    bulk_load(meta + 256, sc.vis + n0, 256, bm);
                    bulk_load(meta + 512, sc.doc + n0, 256, bm);
                    bulk_load(meta + 768, sc.kgrp + n0 / 32, 32, bm);
                }
                mbar_expect_tx(bar_kf + 8 * s, 64 * D * 2);
                for (int hf = 0; hf < L::kHalves; ++hf)
                    tma_load_2d(sbase + L::kK + hf * L::kTileBytes + s * 8192, &tmK, bar_kf + 8 * s, hf * 64, rowbase + wk.r);
                kissued = i + 1;
                return true;
            };
            int r0 = 0, r1 = 0;  // rows of the next two segments of V
            bool ok = true;
            if (nseg > 0) {
                r0 = wk.r;
                ok = issue_k(0);
                wk.advance(col, bo);
            }
            if (ok && nseg > 1) {
                r1 = wk.r;
                ok = issue_k(1);
                wk.advance(col, bo);
            }
            for (int i = 0; ok && i < nseg; ++i) {
                const int s = i & 1;
                // V_i once P_{i-2} V_{i-2} has read the V buffer
                if (i >= 2 && !mbar_wait(bar_ve + 8 * s, ((i >> 1) - 1) & 1, status, kSiteVEmpty, abort_flag)) break;
                mbar_expect_tx(bar_vf + 8 * s, 64 * D * 2);
                for (int hf = 0; hf < L::kHalves; ++hf)
                    tma_load_2d(sbase + L::kV + hf * L::kTileBytes + s * 8192, &tmV, bar_vf + 8 * s, hf * 64, rowbase + r0);
                vissued = i + 1;
                r0 = r1;
                if (i + 2 < nseg) {
                    r1 = wk.r;
                    ok = issue_k(i + 2);
                    wk.advance(col, bo);
                }
            }
            // drain: every issued load must land before the CTA may exit
            for (int i = max(0, kissued - 2); i < kissued; ++i)
                mbar_wait(bar_kf + 8 * (i & 1), (i >> 1) & 1, status, kSiteK, abort_flag);
            for (int i = max(0, kissued - 4); i < kissued; ++i)
                mbar_wait(bar_m + 8 * (i & 3), (i >> 2) & 1, status, kSiteMeta, abort_flag);
            for (int i = max(0, vissued - 2); i < vissued; ++i)
                mbar_wait(bar_vf + 8 * (i & 1), (i >> 1) & 1, status, kSiteV, abort_flag);
            mbar_wait(bar_q, 0, status, kSiteQ, abort_flag);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        constexpr uint32_t idS = idesc_bf16(128, 64, false), idPV = idesc_bf16(128, D, true);
        const uint64_t aQ = sdesc(sbase + L::kQ, 16, 1024), bK = sdesc(sbase + L::kK, 16, 1024);
        const uint64_t bV = sdesc(sbase + L::kV, L::kTileBytes, 1024);
        // S_i; a segment's 64 rows are 512 descriptor units (8192 B) into the buffer
        auto issue_s = [&](int i) -> bool {
            const int s = i & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(bar_kf + 8 * s, (i >> 1) & 1, status, kSiteK, abort_flag))) return false;
            tc_fence_after();
            if constexpr (D == 128)
                mma_ss8<2, 4, 6, 1024, 1026, 1028, 1030, 2, 4, 6, 1024, 1026, 1028, 1030>(tmem + 64 * s, aQ, bK + 512 * s,
                                                                                          idS, 0u);
            else
                mma_ss4<2, 4, 6, 2, 4, 6>(tmem + 64 * s, aQ, bK + 512 * s, idS, 0u);
            mma_commit(bar_s + 8 * s);
            mma_commit(bar_ke + 8 * s);
            return true;
        };
        bool ok = __all_sync(0xffffffffu, mbar_wait(bar_q, 0, status, kSiteQ, abort_flag));
        if (ok && nseg > 0) ok = issue_s(0);
        if (ok && nseg > 1) ok = issue_s(1);
        for (int i = 0; ok && i < nseg; ++i) {
            const int s = i & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(bar_p + 8 * s, (i >> 1) & 1, status, kSiteP, abort_flag))) break;
            if (!__all_sync(0xffffffffu, mbar_wait(bar_vf + 8 * s, (i >> 1) & 1, status, kSiteV, abort_flag))) break;
            tc_fence_after();
            // k-step kk (16 keys): P columns 0, 8, 32, 40, V rows 2048 B (128 descriptor units) further
            mma_ts4<8, 32, 40, 128, 256, 384>(tO, tmem + 64 * s, bV + 512 * s, idPV, i > 0);
            mma_ts4<8, 32, 40, 128, 256, 384>(tO, tmem + 64 * s + 16, bV + 512 * s, idPV, 1u);
            mma_commit(bar_ve + 8 * s);
            // S_{i+2} over P_i: the tensor cores run a CTA's products in issue order
            if (i + 2 < nseg) ok = issue_s(i + 2);
        }
        mma_commit(bar_o);
    } else {
        // ------------------------------------------------------------ softmax
        const int quad = warp & 3, s = (warp - 2) >> 2;
        const int rowid = quad * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const uint32_t tS = tmem + 64 * s + lane_off;
        const int half = shared_tile ? (quad >> 1) : 0;  // which query block's rows (warp-uniform)
        // this row's position, document (no key has -2) and slope in log2 units
        float pq = 0.f, slope2 = 0.f;
        int dq = -2;
        if (rowid < qvalid) {
            pq = sc.pos[(size_t)b * g.N + q0 + rowid];
            dq = sc.doc[(size_t)b * g.N + q0 + rowid];
        }
        if (kScore & kBias) slope2 = sc.slopes[h] * 1.4426950408889634f;
        // of the warp's 32 queries (all or none of them are valid)
        GroupRange qr{INFINITY, -INFINITY, -2, -2};
        if ((kScore & kMask) && quad * 32 < qvalid) {
            const GroupRange *p = sc.qgrp + ((size_t)b * g.N + q0 + quad * 32) / 16;
            const GroupRange r0 = p[0], r1 = p[1];
            qr = GroupRange{fminf(r0.lo, r1.lo), fmaxf(r0.hi, r1.hi), min(r0.dmin, r1.dmin), max(r0.dmax, r1.dmax)};
        }
        const uint64_t s2 = splat2((kScore & (kCap | kBias)) ? 1.0f : scale_log2);
        float l = 0.f;
        bool ok = true, seen = false;  // seen: a key is visible to this row
        for (int i = s; i < nseg; i += 2) {
            ok = __all_sync(0xffffffffu, mbar_wait(bar_m + 8 * (i & 3), (i >> 2) & 1, status, kSiteMeta, abort_flag) &&
                                             mbar_wait(bar_s + 8 * s, (i >> 1) & 1, status, kSiteS, abort_flag));
            if (!ok) break;
            tc_fence_after();
            const uint32_t mw = mask_w[i & 3];
            if ((mw >> half) & 1u) {  // the segment is in this query block's selection
                const bool part = (kScore & kMask) && ((mw >> (2 + half)) & 1u);
                const uint32_t meta = sbase + L::kMeta + (i & 3) * L::kMetaSlot;
                uint64_t acc2 = 0;
#pragma unroll 1
                for (int q = 0; q < 2; ++q) {  // 32 keys at a time, P over their own scores
                    uint32_t sr[32];
                    int cls = 1;
                    if (part) {
                        const float4 kr = lds_f4(meta + 768 + 16 * q);
                        cls = group_class(qr.lo, qr.hi, qr.dmin, qr.dmax, kr.x, kr.y, __float_as_int(kr.z),
                                          __float_as_int(kr.w));
                    }
                    if (cls == 0) {  // none of these queries sees any of these keys
#pragma unroll
                        for (int e = 0; e < 32; ++e) sr[e] = 0u;
                        tmem_st32(tS + 32 * q, sr);
                        continue;
                    }
                    tmem_ld32(tS + 32 * q, sr);
                    tmem_wait_ld();
                    logits32<kScore>(sr, sc, scale_log2, slope2, pq, dq, meta + 128 * q, meta + 256 + 128 * q,
                                     meta + 512 + 128 * q, cls == 2);
                    seen = seen || cls == 1;
                    if (cls == 2) {  // a score that is NaN is not hidden either
                        float mx = -INFINITY;
#pragma unroll
                        for (int e = 0; e < 32; e += 2) mx = fmax3_nan(mx, __uint_as_float(sr[e]), __uint_as_float(sr[e + 1]));
                        seen = seen || mx != -INFINITY;
                    }
                    uint32_t hi[16], lo[16];
                    split_exp32(sr, s2, 0, acc2, hi, lo);
                    tmem_st16(tS + 32 * q, hi);
                    tmem_st16(tS + 32 * q + 16, lo);
                }
                l += sum2(acc2);
            } else {
                uint32_t z[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) z[e] = 0u;
                tmem_st32(tS, z);
                tmem_st32(tS + 32, z);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar_p + 8 * s);
        }
        // epilogue: the row's sum over both chains (every warp passes this barrier once,
        // on every path), then each thread one half of O's columns
        volatile float *sums = reinterpret_cast<volatile float *>(smem + L::kExch);
        volatile int *flags = reinterpret_cast<volatile int *>(smem + L::kExch + 1024);
        sums[s * 128 + rowid] = l;
        flags[s * 128 + rowid] = (seen ? 1 : 0) | (ok ? 0 : 2);
        named_bar_sync(1 + quad, 64);
        l = sums[rowid] + sums[128 + rowid];
        const int fl = flags[rowid] | flags[128 + rowid];
        if (__any_sync(0xffffffffu, fl & 2)) ok = false;
        if (ok)  // the last product P V must have landed
            ok = __all_sync(0xffffffffu, mbar_wait(bar_o, 0, status, kSiteO, abort_flag));
        if (ok) {
            tc_fence_after();
            const bool empty = !(fl & 1);  // no key is visible: O = 0, log-sum-exp -inf
            const float inv = 1.f / l;
            const int n = q0 + rowid;
            const bool write = rowid < qvalid;
            const int tok = write ? perm[(size_t)b * g.N + n] : 0;
            float past = 0.f;  // NaN once an O is past fp32: values near bf16's largest times a large P
            __nv_bfloat16 *dst = O + (((size_t)b * g.N + tok) * g.heads + h) * D + s * (D / 2);
#pragma unroll 1
            for (int q = 0; q < D / 64; ++q) {
                uint32_t orr[32];
                tmem_ld32(tO + lane_off + s * (D / 2) + q * 32, orr);
                tmem_wait_ld();
                uint4 pkt[4], low[4];
                uint32_t *pw = reinterpret_cast<uint32_t *>(pkt), *lw = reinterpret_cast<uint32_t *>(low);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float o0 = empty ? 0.f : __uint_as_float(orr[2 * e]) * inv;
                    const float o1 = empty ? 0.f : __uint_as_float(orr[2 * e + 1]) * inv;
                    past = fmaf(o0, 0.f, fmaf(o1, 0.f, past));
                    pw[e] = pack_bf16x2(o0, o1);
                    lw[e] = pack_bf16x2(o0 - __uint_as_float(pw[e] << 16), o1 - __uint_as_float(pw[e] & 0xffff0000u));
                }
                if (write) {
                    uint4 *d4 = reinterpret_cast<uint4 *>(dst + q * 32);
                    uint4 *l4 = reinterpret_cast<uint4 *>(sc.Olo + ((size_t)bh * g.N + n) * D + s * (D / 2) + q * 32);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        d4[e] = pkt[e];
                        l4[e] = low[e];
                    }
                }
            }
            if (__any_sync(0xffffffffu, write && !empty && !(l >= kLeast && l <= kMost && past == 0.f)) && lane == 0)
                *put_off = 1;
            if (write && s == 0) {
                const float lse2 = empty ? -INFINITY : __log2f(l);
                // negated: the backward's exp2 addend; an empty row's is -inf (P = 0)
                nlse_p[(size_t)bh * g.N + n] = empty ? -INFINITY : -lse2;
                if (lse_user) lse_user[(size_t)bh * g.N + tok] = lse2 * 0.69314718055994531f;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
        if (lane == 0 && *put_off) sc.redo[1 + atomicAdd(&sc.redo[0], 1)] = tid;
    }
}

}  // namespace segtc

template <int D>
static prism_status configure() {
    constexpr int bytes = (int)segtc::Layout<D>::kAlloc;
    const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    PRISM_CUDA_OK(cudaFuncSetAttribute(segtc::k_attn_fwd_scored<D, kScored>, attr, bytes));
    PRISM_CUDA_OK(cudaFuncSetAttribute(segtc::k_attn_fwd_scored<D, kScored | kCap>, attr, bytes));
    PRISM_CUDA_OK(cudaFuncSetAttribute(segtc::k_attn_fwd_scored<D, kScored | kBias>, attr, bytes));
    PRISM_CUDA_OK(cudaFuncSetAttribute(segtc::k_attn_fwd_scored<D, kScored | kCap | kBias>, attr, bytes));
    PRISM_CUDA_OK(cudaFuncSetAttribute(segtc::k_attn_fwd_scored<D, kScored | kMask>, attr, bytes));
    PRISM_CUDA_OK(cudaFuncSetAttribute(segtc::k_attn_fwd_scored<D, kScored | kCap | kMask>, attr, bytes));
    PRISM_CUDA_OK(cudaFuncSetAttribute(segtc::k_attn_fwd_scored<D, kScored | kBias | kMask>, attr, bytes));
    PRISM_CUDA_OK(cudaFuncSetAttribute(segtc::k_attn_fwd_scored<D, kScored | kCap | kBias | kMask>, attr, bytes));
    return PRISM_OK;
}

prism_status configure_attn_scored_kernels() {
    prism_status s = configure<64>();
    return s == PRISM_OK ? configure<128>() : s;
}

template <int D, int kScore>
static prism_status run(Plan &pl, void *O, float *lse, cudaStream_t st) {
    const Geo &g = pl.g;
    segtc::k_attn_fwd_scored<D, kScore>
        <<<dim3(g.nbmax, g.batch * g.heads), segtc::kThreads, segtc::Layout<D>::kAlloc, st>>>(
            pl.tmQ, pl.tmK, pl.tmV, g, pl.qt_row, pl.qt_blk, pl.blk_off, pl.row_ptr, pl.score.col, pl.perm,
            static_cast<__nv_bfloat16 *>(O), lse, pl.nlse_p, (float)(1.4426950408889634 / sqrt((double)D)), pl.status,
            score_args(pl, false));
    PRISM_CUDA_OK(cudaGetLastError());
    return PRISM_OK;
}

template <int D>
static prism_status run_any(Plan &pl, void *O, float *lse, cudaStream_t st) {
    // without a mask the kernel carries no code for one: the registers it takes cost a capped
    // forward (16 x 32 x 32, 8 heads of 128) 3 to 6%
    switch (score_flags(pl.score) | (score_masks(pl.score) ? kMask : 0)) {
        case kScored: return run<D, kScored>(pl, O, lse, st);
        case kScored | kCap: return run<D, kScored | kCap>(pl, O, lse, st);
        case kScored | kBias: return run<D, kScored | kBias>(pl, O, lse, st);
        case kScored | kCap | kBias: return run<D, kScored | kCap | kBias>(pl, O, lse, st);
        case kScored | kMask: return run<D, kScored | kMask>(pl, O, lse, st);
        case kScored | kCap | kMask: return run<D, kScored | kCap | kMask>(pl, O, lse, st);
        case kScored | kBias | kMask: return run<D, kScored | kBias | kMask>(pl, O, lse, st);
        default: return run<D, kScored | kCap | kBias | kMask>(pl, O, lse, st);
    }
}

prism_status launch_attn_fwd_scored(Plan &pl, void *O, float *lse, cudaStream_t st) {
    prism_status s = launch_zero_padding(pl, st);
    if (s != PRISM_OK) return s;
    PRISM_CUDA_OK(cudaMemsetAsync(pl.score.redo, 0, sizeof(int), st));
    TimerScope ts(pl, kTAttnFwd, st);  // one record for the tiles and those of them that are done again
    s = pl.g.D == 64 ? run_any<64>(pl, O, lse, st) : run_any<128>(pl, O, lse, st);
    return s == PRISM_OK ? launch_attn_fwd_scored_redo(pl, O, lse, st) : s;
}

}  // namespace prism
