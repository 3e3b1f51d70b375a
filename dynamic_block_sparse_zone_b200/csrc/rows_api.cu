// rows_api.cu -- the C entry points of the row operators (layer norm, 8-bit
// checkpoints) declared in include/prism.h: argument checks, then the launch.
#include <math.h>

#include "rows.cuh"

using namespace prism;
using rows::RowPtr;

namespace {

size_t dtype_size(int dt) { return dt == PRISM_FP32 ? 4 : 2; }

prism_status check_size(long long nrows, int C, int dtype) {
    if (nrows < 0 || nrows > (1ll << 40)) return fail(PRISM_ERR_INVALID_ARG, "rows must be in [0, 2^40]");
    if (C < 1 || C > (1 << 20)) return fail(PRISM_ERR_INVALID_ARG, "channels must be in [1, 2^20]");
    if (dtype != PRISM_BF16 && dtype != PRISM_FP16 && dtype != PRISM_FP32)
        return fail(PRISM_ERR_INVALID_ARG, "dtype %d is not bf16, fp16 or fp32", dtype);
    return PRISM_OK;
}

prism_status check_weights(int dtype, int wdt) {
    if (wdt != PRISM_FP32 && wdt != dtype)
        return fail(PRISM_ERR_INVALID_ARG, "weight_dtype %d must be fp32 or the rows' dtype", wdt);
    return PRISM_OK;
}

prism_status check_ptr(const void *p, const char *name, size_t align) {
    if ((uintptr_t)p % align) return fail(PRISM_ERR_INVALID_ARG, "%s must be %zu-byte aligned", name, align);
    return PRISM_OK;
}

// What a tensor covers: `groups` spans of bytes, `gstride` apart.
prism_status check_rows(const prism_rows *t, const char *name, long long nrows, int C, int dtype, RowPtr *out) {
    if (!t || (!t->data && nrows > 0)) return fail(PRISM_ERR_INVALID_ARG, "%s is NULL", name);
    const size_t es = dtype_size(dtype);
    prism_status s = check_ptr(t->data, name, es);
    if (s != PRISM_OK) return s;
    if (t->group < 0) return fail(PRISM_ERR_INVALID_ARG, "%s: group is negative", name);
    const long long lim = 1ll << 40, per = t->group > 0 ? t->group : nrows;
    if (t->stride > lim || t->group_stride > lim) return fail(PRISM_ERR_INVALID_ARG, "%s: stride too large", name);
    if (per > 1 && nrows > 1 && t->stride < C)
        return fail(PRISM_ERR_INVALID_ARG, "%s: stride %lld is less than %d channels", name, t->stride, C);
    if (t->group > 0) {
        if (nrows >= (1ll << 31)) return fail(PRISM_ERR_INVALID_ARG, "%s: grouped rows must be below 2^31", name);
        // groups may interleave (heads of one token between heads of another) or follow each other
        if (nrows > t->group && t->group_stride < C)
            return fail(PRISM_ERR_INVALID_ARG, "%s: group_stride %lld is less than %d channels", name, t->group_stride, C);
    }
    // (in doubles: the products below must stay far from 2^63)
    const double far = t->group > 0 ? (double)(nrows / t->group) * (double)t->group_stride + (double)(t->group - 1) * (double)t->stride
                                    : (double)nrows * (double)t->stride;
    if (far > 1e17) return fail(PRISM_ERR_INVALID_ARG, "%s reaches past any address space", name);
    *out = RowPtr{static_cast<char *>(t->data), t->stride * (long long)es, t->group_stride * (long long)es,
                  (unsigned)t->group};
    return PRISM_OK;
}

// An output's rows are apart when its groups follow one another, or when all
// groups' k-th rows lie before any group's k+1-th.
prism_status check_output(const RowPtr &p, const char *name, long long nrows, int C, size_t es) {
    if (!p.group || nrows <= p.group || p.group == 1) return PRISM_OK;  // evenly spaced, at least C apart
    const long long row = (long long)C * es, groups = (nrows + p.group - 1) / p.group;
    if (p.group_stride >= (long long)(p.group - 1) * p.stride + row || p.stride >= (groups - 1) * p.group_stride + row)
        return PRISM_OK;
    return fail(PRISM_ERR_INVALID_ARG, "%s: rows of one group reach into another's", name);
}

// First and one-past-last byte.
void span(const RowPtr &p, long long nrows, int C, size_t es, uintptr_t *lo, uintptr_t *hi) {
    *lo = (uintptr_t)p.data;
    long long last = (nrows - 1) * p.stride;
    if (p.group) {
        const long long q = (nrows - 1) / p.group;
        last = q * p.group_stride + (nrows - 1 - q * p.group) * p.stride;
        if (q > 0) {
            const long long full = (q - 1) * p.group_stride + (long long)(p.group - 1) * p.stride;
            if (full > last) last = full;
        }
    }
    *hi = *lo + (uintptr_t)last + (uintptr_t)C * es;
}

// Refuses tensors that share elements.  Two whose byte ranges cross are taken
// as apart only when both repeat with one period (the same stride, or the same
// group and strides) and their rows miss each other within it.
prism_status check_apart(const RowPtr &a, size_t ea, const char *na, const RowPtr &b, size_t eb, const char *nb,
                         long long nrows, int C) {
    if (nrows == 0) return PRISM_OK;
    uintptr_t a0, a1, b0, b1;
    span(a, nrows, C, ea, &a0, &a1);
    span(b, nrows, C, eb, &b0, &b1);
    if (a1 <= b0 || b1 <= a0) return PRISM_OK;
    const long long per_a = a.group ? a.group : nrows, per_b = b.group ? b.group : nrows;
    auto miss = [&](long long period, long long la, long long lb) {
        if (period <= 0) return false;
        long long d = (long long)(b0 - a0) % period;
        if (d < 0) d += period;
        return d >= la && period - d >= lb;
    };
    const long long ra = (long long)C * ea, rb = (long long)C * eb;
    if ((per_a >= nrows || a.group_stride == per_a * a.stride) && (per_b >= nrows || b.group_stride == per_b * b.stride) &&
        a.stride == b.stride && miss(a.stride, ra, rb))
        return PRISM_OK;
    if (per_a < nrows && per_a == per_b && a.group_stride == b.group_stride &&
        miss(a.group_stride, (per_a - 1) * a.stride + ra, (per_b - 1) * b.stride + rb))
        return PRISM_OK;
    return fail(PRISM_ERR_INVALID_ARG, "%s and %s overlap", na, nb);
}

prism_status check_ckpt(const prism_ckpt *k, long long nrows) {
    if (!k || ((!k->codes || !k->scales) && nrows > 0)) return fail(PRISM_ERR_INVALID_ARG, "checkpoint is NULL");
    if (k->format != PRISM_CKPT_INT8 && k->format != PRISM_CKPT_E4M3)
        return fail(PRISM_ERR_INVALID_ARG, "checkpoint format %d is not int8 or e4m3", k->format);
    prism_status s = check_ptr(k->codes, "checkpoint codes", 16);
    return s == PRISM_OK ? check_ptr(k->scales, "checkpoint scales", 16) : s;
}

}  // namespace

#define TRY(call)                                   \
    do {                                            \
        const prism_status s_ = (call);             \
        if (s_ != PRISM_OK) return s_;              \
    } while (0)

extern "C" {

prism_status prism_ckpt_bytes(long long nrows, int channels, size_t *codes, size_t *scales) {
    clear_error();
    if (!codes || !scales) return fail(PRISM_ERR_INVALID_ARG, "NULL argument to prism_ckpt_bytes");
    TRY(check_size(nrows, channels, PRISM_FP32));
    *codes = (size_t)nrows * channels;
    *scales = (size_t)nrows * ((channels + 31) / 32);
    return PRISM_OK;
}

prism_status prism_ckpt_pack(const prism_rows *x, int dtype, long long nrows, int channels, const prism_ckpt *out,
                             void *stream) {
    clear_error();
    RowPtr px;
    TRY(check_size(nrows, channels, dtype));
    TRY(check_rows(x, "x", nrows, channels, dtype, &px));
    TRY(check_ckpt(out, nrows));
    return launch_ckpt_pack(px, dtype, nrows, channels, *out, static_cast<cudaStream_t>(stream));
}

prism_status prism_ckpt_unpack(const prism_ckpt *in, const prism_rows *y, int dtype, long long nrows, int channels,
                               void *stream) {
    clear_error();
    RowPtr py;
    TRY(check_size(nrows, channels, dtype));
    TRY(check_ckpt(in, nrows));
    TRY(check_rows(y, "y", nrows, channels, dtype, &py));
    TRY(check_output(py, "y", nrows, channels, dtype_size(dtype)));
    return launch_ckpt_unpack(*in, py, dtype, nrows, channels, static_cast<cudaStream_t>(stream));
}

prism_status prism_layer_norm_fwd(const prism_rows *x, const void *gamma, const void *beta, const prism_rows *y,
                                  float *mean, float *rstd, const prism_ckpt *ckpt, long long nrows, int channels,
                                  float eps, int dtype, int weight_dtype, void *stream) {
    clear_error();
    rows::NormFwd a{};
    TRY(check_size(nrows, channels, dtype));
    TRY(check_weights(dtype, weight_dtype));
    if (!(eps >= 0.f) || isinf(eps)) return fail(PRISM_ERR_INVALID_ARG, "eps must be finite and not negative");
    TRY(check_rows(x, "x", nrows, channels, dtype, &a.x));
    TRY(check_rows(y, "y", nrows, channels, dtype, &a.y));
    if ((!mean || !rstd) && nrows > 0) return fail(PRISM_ERR_INVALID_ARG, "mean or rstd is NULL");
    TRY(check_ptr(mean, "mean", 4));
    TRY(check_ptr(rstd, "rstd", 4));
    TRY(check_ptr(gamma, "gamma", dtype_size(weight_dtype)));
    TRY(check_ptr(beta, "beta", dtype_size(weight_dtype)));
    const size_t es = dtype_size(dtype);
    TRY(check_output(a.y, "y", nrows, channels, es));
    TRY(check_apart(a.x, es, "x", a.y, es, "y", nrows, channels));
    if (ckpt) {
        TRY(check_ckpt(ckpt, nrows));
        a.codes = static_cast<uint8_t *>(ckpt->codes);
        a.scales = static_cast<uint8_t *>(ckpt->scales);
        a.fmt = ckpt->format;
    }
    a.gamma = gamma;
    a.beta = beta;
    a.wdt = weight_dtype;
    a.mean = mean;
    a.rstd = rstd;
    a.nrows = nrows;
    a.C = channels;
    a.eps = eps;
    return launch_norm_fwd(a, dtype, static_cast<cudaStream_t>(stream));
}

size_t prism_layer_norm_bwd_workspace(long long nrows, int channels) {
    clear_error();
    if (check_size(nrows, channels, PRISM_FP32) != PRISM_OK) return 0;
    return norm_bwd_workspace(nrows, channels);
}

prism_status prism_layer_norm_bwd(const prism_rows *x, const prism_ckpt *ckpt, const prism_rows *dy, const void *gamma,
                                  const float *mean, const float *rstd, const prism_rows *dx, void *dgamma, void *dbeta,
                                  void *workspace, size_t workspace_bytes, long long nrows, int channels, int dtype,
                                  int weight_dtype, void *stream) {
    clear_error();
    rows::NormBwd a{};
    TRY(check_size(nrows, channels, dtype));
    TRY(check_weights(dtype, weight_dtype));
    if ((x != nullptr) == (ckpt != nullptr))
        return fail(PRISM_ERR_INVALID_ARG, "exactly one of x and its checkpoint is needed");
    if (x) TRY(check_rows(x, "x", nrows, channels, dtype, &a.x));
    TRY(check_rows(dy, "dy", nrows, channels, dtype, &a.dy));
    TRY(check_rows(dx, "dx", nrows, channels, dtype, &a.dx));
    if ((!mean || !rstd) && nrows > 0) return fail(PRISM_ERR_INVALID_ARG, "mean or rstd is NULL");
    TRY(check_ptr(mean, "mean", 4));
    TRY(check_ptr(rstd, "rstd", 4));
    TRY(check_ptr(gamma, "gamma", dtype_size(weight_dtype)));
    TRY(check_ptr(dgamma, "dgamma", dtype_size(weight_dtype)));
    TRY(check_ptr(dbeta, "dbeta", dtype_size(weight_dtype)));
    const size_t es = dtype_size(dtype);
    TRY(check_output(a.dx, "dx", nrows, channels, es));
    TRY(check_apart(a.dy, es, "dy", a.dx, es, "dx", nrows, channels));
    if (x) {
        TRY(check_apart(a.x, es, "x", a.dx, es, "dx", nrows, channels));
    } else {
        TRY(check_ckpt(ckpt, nrows));
        a.codes = static_cast<const uint8_t *>(ckpt->codes);
        a.scales = static_cast<const uint8_t *>(ckpt->scales);
        a.fmt = ckpt->format;
    }
    if (dgamma || dbeta) {
        const size_t need = norm_bwd_workspace(nrows, channels);
        if (!workspace || workspace_bytes < need)
            return fail(PRISM_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
        TRY(check_ptr(workspace, "workspace", 16));
    }
    a.gamma = gamma;
    a.wdt = weight_dtype;
    a.mean = mean;
    a.rstd = rstd;
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.part = static_cast<float *>(workspace);
    a.nrows = nrows;
    a.C = channels;
    return launch_norm_bwd(a, dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
