// Host side of the layer operators: argument validation, workspace sizes and
// launches.  The entry points are declared in include/lags.h.
#include "lags.h"
#include "lags_args.h"
#include "lags_layer.h"

#include <algorithm>
#include <cmath>
#include <initializer_list>

using namespace lags;

static_assert(kActGelu == LAGS_ACT_GELU && kLnMax == LAGS_LN_MAX, "one numbering");

namespace {

int edge_of(const void *p, int64_t ld, int64_t cols, int32_t dtype)
{
    const uint32_t e = elem_bytes(dtype);
    if (!p) return kWhole;
    return (((uintptr_t)p | (uint64_t)ld * e) & 3) ? kShifted : cols % (16 / e) ? kRagged : kWhole;
}

int check_ln(const lags_ln *ln)
{
    if (!ln || !known_dtype(ln->dtype)) return LAGS_EINVAL;
    if (!(ln->eps >= 0) || !std::isfinite(ln->eps)) return LAGS_EINVAL;
    if (ln->rows < 0 || ln->channels < 1) return LAGS_EINVAL;
    if (ln->rows > kMaxDim || ln->channels > LAGS_LN_MAX) return LAGS_ERANGE;
    return LAGS_OK;
}

LnArgs ln_args(const lags_ln *ln)
{
    LnArgs a = {};
    const CkptShape cs = ckpt_shape(0, ln->channels);
    a.eps = ln->eps, a.inv_c = (float)(1.0 / (double)ln->channels);
    a.rows = ln->rows, a.C = (uint32_t)ln->channels, a.pitch = cs.pitch, a.nrun = cs.nrun;
    return a;
}

size_t ln_need(const lags_ln *ln)
{
    // of any alignment
    const uint32_t C = (uint32_t)ln->channels;
    const uint32_t groups = std::max(ln_plan(ln->dtype, true, kWhole, ln->rows, C).groups,
                                     ln_plan(ln->dtype, true, kShifted, ln->rows, C).groups);
    const size_t need = ln->rows ? (size_t)groups * 2 * C * 4 : 0;
    return std::max<size_t>((need + 15) / 16 * 16, 16);
}

// A checkpoint argument of [rows, cols]: null, or its region, or a status.
int checkpoint(const void *p, size_t bytes, int64_t rows, int64_t cols, Region &r)
{
    r = flat(nullptr, 0);
    if (!p) return LAGS_OK;
    const size_t need = ckpt_size(ckpt_shape(rows, cols));
    if (!aligned(p, 16) || bytes < need) return LAGS_EWORKSPACE;
    r = flat(p, need);
    return LAGS_OK;
}

bool embed_dims(int64_t tokens, int64_t vocab, int64_t cols)
{
    return tokens >= 0 && tokens <= kMaxDim && vocab >= 1 && vocab <= LAGS_VOCAB_MAX && cols >= 1 &&
           cols <= LAGS_WGRAD_MAX;
}

// Where a gradient's workspace keeps its parts.
struct EmbedSpace {
    size_t order, keys, start, part, bytes;
};
EmbedSpace embed_space(int64_t tokens, int64_t vocab, int64_t cols)
{
    auto up = [](size_t n) { return (n + 15) / 16 * 16; };
    EmbedSpace w;
    w.order = 0;
    w.keys = up((size_t)tokens * 4);
    w.start = w.keys + up((size_t)tokens * 4);
    w.part = w.start + up(((size_t)vocab + 1) * 4);
    w.bytes = w.part + up((size_t)embed_plan(LAGS_F32, tokens, vocab, cols).nchunk * 2 * cols * 4);
    return w;
}

}  // namespace

extern "C" {

size_t lags_ln_workspace_bytes(const lags_ln *ln) { return check_ln(ln) == LAGS_OK ? ln_need(ln) : 0; }

int lags_ln_forward(const lags_ln *ln, const void *x, int64_t ldx, const void *res, int64_t ldr, const float *gamma,
                    const float *beta, void *sum, int64_t lds, void *y, int64_t ldy, float *mean, float *rstd,
                    void *ckpt, size_t ckpt_bytes, void *yckpt, size_t yckpt_bytes, void *stream)
{
    if (int rc = check_ln(ln); rc != LAGS_OK) return rc;
    const int64_t R = ln->rows, C = ln->channels;
    if (sum && !res) return LAGS_EINVAL;
    enum { X, RES, SUM, Y, GAMMA, BETA, MEAN, RSTD, CK, YCK, N };
    Region r[N] = {};
    if (int rc = matrix(x, R, C, ldx, ln->dtype, r[X]); rc != LAGS_OK) return rc;
    if (res)
        if (int rc = matrix(res, R, C, ldr, ln->dtype, r[RES]); rc != LAGS_OK) return rc;
    if (sum)
        if (int rc = matrix(sum, R, C, lds, ln->dtype, r[SUM]); rc != LAGS_OK) return rc;
    if (int rc = matrix(y, R, C, ldy, ln->dtype, r[Y]); rc != LAGS_OK) return rc;
    if (ldx > LAGS_GN_MAX || ldy > LAGS_GN_MAX || (res && ldr > LAGS_GN_MAX) || (sum && lds > LAGS_GN_MAX))
        return LAGS_ERANGE;
    if (!gamma != !beta || !aligned(gamma, 4) || !aligned(beta, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
        return LAGS_EINVAL;
    r[GAMMA] = flat(gamma, C * 4), r[BETA] = flat(beta, C * 4), r[MEAN] = flat(mean, R * 4), r[RSTD] = flat(rstd, R * 4);
    if (int rc = checkpoint(ckpt, ckpt_bytes, R, C, r[CK]); rc != LAGS_OK) return rc;
    if (int rc = checkpoint(yckpt, yckpt_bytes, R, C, r[YCK]); rc != LAGS_OK) return rc;
    for (int out : {MEAN, RSTD, CK, YCK})
        if (!clear_of(r, N, out)) return LAGS_EINVAL;
    // y and sum may each be x or res itself
    for (int out : {SUM, Y}) {
        for (int in : {X, RES})
            if (overlap(r[out], r[in]) && !same(r[out], r[in])) return LAGS_EINVAL;
        if (overlap(r[out], r[GAMMA]) || overlap(r[out], r[BETA])) return LAGS_EINVAL;
    }
    if (overlap(r[SUM], r[Y])) return LAGS_EINVAL;
    if (!R) return LAGS_OK;
    LnArgs a = ln_args(ln);
    a.x = x, a.ldx = ldx, a.res = res, a.ldr = ldr, a.sum = sum, a.lds = lds, a.y = y, a.ldy = ldy;
    a.gamma = gamma, a.beta = beta, a.mean = mean, a.rstd = rstd;
    if (ckpt) a.wcodes = (uint8_t *)ckpt, a.wscales = (uint8_t *)ckpt + (size_t)R * a.pitch;
    if (yckpt) a.ycodes = (uint8_t *)yckpt, a.yscales = (uint8_t *)yckpt + (size_t)R * a.pitch;
    const int edge = std::max(edge_of(x, ldx, C, ln->dtype), edge_of(res, ldr, C, ln->dtype));
    const LnPlan p = ln_plan(ln->dtype, false, edge, R, (uint32_t)C);
    return hip(launch_ln_forward(p, a, ln->dtype, edge, (hipStream_t)stream));
}

int lags_ln_backward(const lags_ln *ln, const void *dy, int64_t lddy, const void *x, int64_t ldx, const void *ckpt,
                     size_t ckpt_bytes, const float *gamma, const float *mean, const float *rstd, const void *dsum,
                     int64_t ldds, void *dx, int64_t lddx, float *dgamma, float *dbeta, uint32_t flags, void *ws,
                     size_t ws_bytes, void *stream)
{
    if (int rc = check_ln(ln); rc != LAGS_OK) return rc;
    const int64_t R = ln->rows, C = ln->channels;
    if ((flags & ~LAGS_GRAD_ADD) || !x == !ckpt) return LAGS_EINVAL;
    enum { DY, X, DSUM, DX, GAMMA, MEAN, RSTD, DGAMMA, DBETA, CK, WS, N };
    Region r[N] = {};
    if (int rc = matrix(dy, R, C, lddy, ln->dtype, r[DY]); rc != LAGS_OK) return rc;
    if (x)
        if (int rc = matrix(x, R, C, ldx, ln->dtype, r[X]); rc != LAGS_OK) return rc;
    if (dsum)
        if (int rc = matrix(dsum, R, C, ldds, ln->dtype, r[DSUM]); rc != LAGS_OK) return rc;
    if (int rc = matrix(dx, R, C, lddx, ln->dtype, r[DX]); rc != LAGS_OK) return rc;
    if (lddy > LAGS_GN_MAX || lddx > LAGS_GN_MAX || (x && ldx > LAGS_GN_MAX) || (dsum && ldds > LAGS_GN_MAX))
        return LAGS_ERANGE;
    if (!mean || !rstd || !aligned(gamma, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dgamma, 4) ||
        !aligned(dbeta, 4))
        return LAGS_EINVAL;
    if (int rc = checkpoint(ckpt, ckpt_bytes, R, C, r[CK]); rc != LAGS_OK) return rc;
    const size_t need = ln_need(ln);
    if (!ws || !aligned(ws, 16) || ws_bytes < need) return LAGS_EWORKSPACE;
    r[GAMMA] = flat(gamma, C * 4), r[MEAN] = flat(mean, R * 4), r[RSTD] = flat(rstd, R * 4);
    r[DGAMMA] = flat(dgamma, C * 4), r[DBETA] = flat(dbeta, C * 4), r[WS] = flat(ws, need);
    for (int out : {DGAMMA, DBETA, WS})
        if (!clear_of(r, N, out)) return LAGS_EINVAL;
    // dx may be dy or dsum itself
    for (int in : {X, GAMMA, MEAN, RSTD, CK})
        if (overlap(r[DX], r[in])) return LAGS_EINVAL;
    for (int in : {DY, DSUM})
        if (overlap(r[DX], r[in]) && !same(r[DX], r[in])) return LAGS_EINVAL;
    LnArgs a = ln_args(ln);
    a.dy = dy, a.lddy = lddy, a.x = x, a.ldx = ldx, a.dsum = dsum, a.ldds = ldds, a.dx = dx, a.lddx = lddx;
    if (ckpt) a.rcodes = (const uint8_t *)ckpt, a.rscales = (const uint8_t *)ckpt + (size_t)R * a.pitch;
    a.gamma = gamma, a.mean = (float *)mean, a.rstd = (float *)rstd;
    a.dgamma = dgamma, a.dbeta = dbeta, a.add = flags & LAGS_GRAD_ADD;
    a.part = dgamma || dbeta ? (float *)ws : nullptr;
    const int edge = std::max({edge_of(dy, lddy, C, ln->dtype), edge_of(x, ldx, C, ln->dtype),
                               edge_of(dsum, ldds, C, ln->dtype)});
    const LnPlan p = ln_plan(ln->dtype, true, edge, R, (uint32_t)C);
    return hip(launch_ln_backward(p, a, ln->dtype, edge, (hipStream_t)stream));
}

size_t lags_embed_workspace_bytes(int64_t tokens, int64_t vocab, int64_t cols)
{
    return embed_dims(tokens, vocab, cols) ? embed_space(tokens, vocab, cols).bytes : 0;
}

int lags_embed_forward(int64_t tokens, int64_t vocab, int64_t cols, const void *ids, const void *table,
                       int32_t table_dtype, float scale, void *y, int64_t ldy, int32_t dtype, uint32_t flags,
                       void *stream)
{
    if (!known_dtype(dtype) || (table_dtype != LAGS_F32 && table_dtype != dtype)) return LAGS_EINVAL;
    if ((flags & ~LAGS_IDS64) || !std::isfinite(scale)) return LAGS_EINVAL;
    if (!embed_dims(tokens, vocab, cols)) return LAGS_ERANGE;
    const bool wide = flags & LAGS_IDS64;
    if (!ids || !aligned(ids, wide ? 8 : 4)) return LAGS_EINVAL;
    Region t, m;
    if (int rc = matrix(table, vocab, cols, cols, table_dtype, t); rc != LAGS_OK) return rc;
    if (int rc = matrix(y, tokens, cols, ldy, dtype, m); rc != LAGS_OK) return rc;
    if (overlap(m, t) || overlap(m, flat(ids, (size_t)tokens * (wide ? 8 : 4)))) return LAGS_EINVAL;
    if (!tokens) return LAGS_OK;
    EmbedArgs a = {};
    a.ids = ids, a.table = table, a.y = y, a.ldy = ldy;
    a.tokens = tokens, a.vocab = (uint32_t)vocab, a.cols = (uint32_t)cols, a.scale = scale;
    return hip(launch_embed(a, table_dtype, dtype, wide, (hipStream_t)stream));
}

int lags_embed_grad(int64_t tokens, int64_t vocab, int64_t cols, const void *ids, const void *dy, int64_t lddy,
                    int32_t dtype, float scale, float *dtable, uint32_t flags, void *ws, size_t ws_bytes, void *stream)
{
    if (!known_dtype(dtype) || (flags & ~(LAGS_IDS64 | LAGS_GRAD_ADD)) || !std::isfinite(scale)) return LAGS_EINVAL;
    if (!embed_dims(tokens, vocab, cols)) return LAGS_ERANGE;
    const bool wide = flags & LAGS_IDS64;
    if (!ids || !aligned(ids, wide ? 8 : 4) || !dtable || !aligned(dtable, 4)) return LAGS_EINVAL;
    Region r[4];
    if (int rc = matrix(dy, tokens, cols, lddy, dtype, r[0]); rc != LAGS_OK) return rc;
    const EmbedPlan p = embed_plan(dtype, tokens, vocab, cols);
    // threads of one launch
    if ((u128)(p.sumwgs + vocab / 64 + 1) * 256 > kMostThreads || (u128)p.nchunk * p.njoin * 256 > kMostThreads)
        return LAGS_ERANGE;
    const EmbedSpace w = embed_space(tokens, vocab, cols);
    if (!ws || !aligned(ws, 16) || ws_bytes < w.bytes) return LAGS_EWORKSPACE;
    r[1] = flat(ids, (size_t)tokens * (wide ? 8 : 4)), r[2] = flat(dtable, (size_t)vocab * cols * 4), r[3] = flat(ws, w.bytes);
    if (!clear_of(r, 4, 2) || !clear_of(r, 4, 3)) return LAGS_EINVAL;
    if (!tokens && (flags & LAGS_GRAD_ADD)) return LAGS_OK;
    EmbedArgs a = {};
    a.ids = ids, a.dy = dy, a.lddy = lddy, a.dtable = dtable;
    a.tokens = tokens, a.vocab = (uint32_t)vocab, a.cols = (uint32_t)cols, a.scale = scale;
    a.add = flags & LAGS_GRAD_ADD;
    char *b = (char *)ws;
    a.order = (uint32_t *)(b + w.order), a.keys = (uint32_t *)(b + w.keys), a.start = (uint32_t *)(b + w.start);
    a.part = (float *)(b + w.part);
    return hip(launch_embed_grad(p, a, dtype, wide, (hipStream_t)stream));
}

}  // extern "C"
