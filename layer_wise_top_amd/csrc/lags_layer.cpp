// Host side of the layer operators: argument validation, workspace sizes and
// launches.  The entry points are declared in include/lags.h.
#include "lags.h"
#include "lags_args.h"
#include "lags_layer.h"

#include <algorithm>
#include <cmath>
#include <initializer_list>

using namespace lags;

static_assert(kActGelu == LAGS_ACT_GELU && kLnMax == LAGS_LN_MAX && kLinearMax == LAGS_LINEAR_MAX, "one numbering");

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
    w.order = 0;                     // read a chunk at a time: what follows is the workspace's too
    w.keys = up((size_t)tokens * 4);
    w.start = w.keys + up((size_t)tokens * 4);
    w.part = w.start + up(((size_t)vocab + 1) * 4);
    w.bytes = w.part + up((size_t)embed_plan(LAGS_F32, tokens, vocab, cols).nchunk * 2 * cols * 4);
    return w;
}

int check_linear(const lags_linear *l)
{
    if (!l || !known_dtype(l->dtype) || l->act < LAGS_ACT_NONE || l->act > LAGS_ACT_GELU) return LAGS_EINVAL;
    if (l->rows < 0 || l->cols < 1 || l->outs < 1) return LAGS_EINVAL;
    if (l->rows > kMaxDim || l->cols > LAGS_LINEAR_MAX || l->outs > LAGS_LINEAR_MAX) return LAGS_ERANGE;
    return LAGS_OK;
}

struct LinearCall {
    LinPlan fwd, bwd;
    DzPlan dz;
    size_t need, turned;             // workspace, of both directions; where W turned round is in it
};
int plan_anew(const lags_linear *l, LinearCall &c)
{
    const int64_t M = std::max<int64_t>(l->rows, 1);
    c.fwd = linear_plan(l->dtype, false, M, l->outs, l->cols);
    c.bwd = linear_plan(l->dtype, true, M, l->cols, l->outs);
    c.dz = dz_plan(l->dtype, M, l->outs);
    // Tiles are counted in 32 bits; outputs of so many fit no memory.
    for (const LinPlan *p : {&c.fwd, &c.bwd})
        if ((u128)p->tm * p->tn * p->split > 0xffffffffu) return LAGS_ERANGE;
    const u128 f = c.fwd.split > 1 ? (u128)c.fwd.split * M * l->outs * 4 : 0;
    const u128 b = c.bwd.split > 1 ? (u128)c.bwd.split * M * l->cols * 4 : 0;
    // dbias is done before the product's sums are written
    const u128 d = (u128)c.dz.chunks * l->outs * 4;
    const u128 most = std::max(std::max(f, b), d);
    c.turned = (size_t)((most + 15) / 16 * 16);
    c.need = l->rows ? std::max<size_t>(c.turned + (c.bwd.turn ? (size_t)l->outs * l->cols * 2 : 0), 16) : 16;
    return LAGS_OK;
}

// The plan is a function of the shape alone; what it weighs takes the host a microsecond, as much as a
// fifth of a small call, so each thread keeps the last shapes'.
int plan(const lags_linear *l, LinearCall &c)
{
    if (int rc = check_linear(l); rc != LAGS_OK) return rc;
    struct Kept {
        lags_linear of;
        LinearCall call;
        int rc;
    };
    thread_local Kept kept[32];      // rows 0, cols 0 at first: no shape that is looked for
    const uint64_t h = ((uint64_t)l->rows * 31 + l->cols) * 31 + l->outs * 7 + l->dtype;
    Kept &k = kept[(h ^ h >> 17) % 32];
    if (k.of.rows != l->rows || k.of.cols != l->cols || k.of.outs != l->outs || k.of.dtype != l->dtype) {
        k.rc = plan_anew(l, k.call);
        k.of = *l;
    }
    c = k.call;
    return k.rc;
}

// How a product's operands get into LDS (lags_linear.h).
int how_of(std::initializer_list<std::pair<const void *, int64_t>> operands, int64_t inner, int32_t dtype)
{
    const uint32_t e = elem_bytes(dtype);
    uintptr_t bits = (uint64_t)inner * e;
    for (auto &o : operands) bits |= (uintptr_t)o.first | (uint64_t)o.second * e;
    return bits & 3 ? 2 : bits & 15 ? 1 : 0;
}

// How a product's results are stored.  Outputs above 64 MB go past the caches, which they would only
// pass through: 16384 x 2048 -> 8192 bf16 with gelu and z 550 -> 519 us.
void results(LinArgs &a, int32_t dtype)
{
    a.whole = !edge_of(a.y, a.ldy, a.N, dtype) && !edge_of(a.z, a.ldz, a.N, dtype) && !edge_of(a.res, a.ldr, a.N, dtype);
    a.past = (u128)a.M * a.N * elem_bytes(dtype) > ((u128)64 << 20);
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
    // threads of the sums' launch
    if ((u128)p.sumwgs * 256 > kMostThreads) return LAGS_ERANGE;
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

size_t lags_linear_workspace_bytes(const lags_linear *lin)
{
    LinearCall c;
    return plan(lin, c) == LAGS_OK ? c.need : 0;
}

int lags_linear_forward(const lags_linear *lin, const void *x, int64_t ldx, const void *w, int64_t ldw,
                        const float *bias, const void *res, int64_t ldr, void *z, int64_t ldz, void *y, int64_t ldy,
                        void *ws, size_t ws_bytes, void *stream)
{
    LinearCall c;
    if (int rc = plan(lin, c); rc != LAGS_OK) return rc;
    const int64_t M = lin->rows, K = lin->cols, N = lin->outs;
    enum { X, W, BIAS, RES, Z, Y, WS, COUNT };
    Region r[COUNT] = {};
    if (int rc = matrix(x, M, K, ldx, lin->dtype, r[X]); rc != LAGS_OK) return rc;
    if (int rc = matrix(w, N, K, ldw, lin->dtype, r[W]); rc != LAGS_OK) return rc;
    if (res)
        if (int rc = matrix(res, M, N, ldr, lin->dtype, r[RES]); rc != LAGS_OK) return rc;
    if (z)
        if (int rc = matrix(z, M, N, ldz, lin->dtype, r[Z]); rc != LAGS_OK) return rc;
    if (int rc = matrix(y, M, N, ldy, lin->dtype, r[Y]); rc != LAGS_OK) return rc;
    if (ldx > LAGS_LINEAR_MAX || ldw > LAGS_LINEAR_MAX || ldy > LAGS_LINEAR_MAX || (res && ldr > LAGS_LINEAR_MAX) ||
        (z && ldz > LAGS_LINEAR_MAX))
        return LAGS_ERANGE;
    if (!aligned(bias, 4)) return LAGS_EINVAL;
    if (!ws || !aligned(ws, 16) || ws_bytes < c.need) return LAGS_EWORKSPACE;
    r[BIAS] = flat(bias, N * 4), r[WS] = flat(ws, c.need);
    for (int out : {Z, WS})
        if (!clear_of(r, COUNT, out)) return LAGS_EINVAL;
    // y may be res itself
    for (int in : {X, W, BIAS})
        if (overlap(r[Y], r[in])) return LAGS_EINVAL;
    if (overlap(r[Y], r[RES]) && !same(r[Y], r[RES])) return LAGS_EINVAL;
    if (!M) return LAGS_OK;
    LinArgs a = {};
    a.a = x, a.lda = ldx, a.b = w, a.ldb = ldw, a.M = M, a.N = (uint32_t)N, a.K = (uint32_t)K;
    a.act = lin->act, a.bias = bias, a.res = res, a.ldr = ldr, a.z = z, a.ldz = ldz, a.y = y, a.ldy = ldy;
    a.part = (float *)ws;
    results(a, lin->dtype);
    const int how = how_of({{x, ldx}, {w, ldw}}, K, lin->dtype);
    return hip(launch_linear(c.fwd, a, false, how, lin->dtype, (hipStream_t)stream));
}

int lags_linear_backward(const lags_linear *lin, const void *dy, int64_t lddy, const void *z, int64_t ldz,
                         const void *w, int64_t ldw, void *dz, int64_t lddz, float *dbias, void *dx, int64_t lddx,
                         uint32_t flags, void *ws, size_t ws_bytes, void *stream)
{
    LinearCall c;
    if (int rc = plan(lin, c); rc != LAGS_OK) return rc;
    const int64_t M = lin->rows, K = lin->cols, N = lin->outs;
    const bool act = lin->act != LAGS_ACT_NONE;
    if (flags & ~LAGS_GRAD_ADD) return LAGS_EINVAL;
    if (!z != !act || !dz != !act || !w != !dx) return LAGS_EINVAL;
    enum { DY, Z, W, DZ, DBIAS, DX, WS, COUNT };
    Region r[COUNT] = {};
    if (int rc = matrix(dy, M, N, lddy, lin->dtype, r[DY]); rc != LAGS_OK) return rc;
    if (act) {
        if (int rc = matrix(z, M, N, ldz, lin->dtype, r[Z]); rc != LAGS_OK) return rc;
        if (int rc = matrix(dz, M, N, lddz, lin->dtype, r[DZ]); rc != LAGS_OK) return rc;
    }
    if (dx) {
        if (int rc = matrix(w, N, K, ldw, lin->dtype, r[W]); rc != LAGS_OK) return rc;
        if (int rc = matrix(dx, M, K, lddx, lin->dtype, r[DX]); rc != LAGS_OK) return rc;
    }
    if (lddy > LAGS_LINEAR_MAX || (act && (ldz > LAGS_LINEAR_MAX || lddz > LAGS_LINEAR_MAX)) ||
        (dx && (ldw > LAGS_LINEAR_MAX || lddx > LAGS_LINEAR_MAX)))
        return LAGS_ERANGE;
    if (!aligned(dbias, 4)) return LAGS_EINVAL;
    if (!ws || !aligned(ws, 16) || ws_bytes < c.need) return LAGS_EWORKSPACE;
    r[DBIAS] = flat(dbias, N * 4), r[WS] = flat(ws, c.need);
    for (int out : {DBIAS, DX, WS})
        if (!clear_of(r, COUNT, out)) return LAGS_EINVAL;
    // dz may be dy or z itself
    if (overlap(r[DZ], r[W])) return LAGS_EINVAL;
    for (int in : {DY, Z})
        if (overlap(r[DZ], r[in]) && !same(r[DZ], r[in])) return LAGS_EINVAL;
    const bool add = flags & LAGS_GRAD_ADD;
    const hipStream_t s = (hipStream_t)stream;
    LinArgs a = {};
    a.M = M, a.act = lin->act;
    if (M && (act || dbias)) {
        a.N = (uint32_t)N, a.dy = dy, a.lddy = lddy, a.zin = z, a.ldz = ldz, a.dz = dz, a.lddz = lddz;
        if (c.dz.chunks == 1)
            a.dbias = dbias, a.add = add;
        else
            a.part = dbias ? (float *)ws : nullptr;
        if (int rc = hip(launch_slopes(c.dz, a, lin->dtype, s)); rc != LAGS_OK) return rc;
    }
    if (dbias && (!M || c.dz.chunks > 1))
        if (int rc = hip(launch_dbias((const float *)ws, M ? c.dz.chunks : 0, (uint32_t)N, dbias, add, s)); rc != LAGS_OK)
            return rc;
    if (!M || !dx) return LAGS_OK;
    a = {};
    a.a = act ? dz : dy, a.lda = act ? lddz : lddy, a.b = w, a.ldb = ldw;
    a.M = M, a.N = (uint32_t)K, a.K = (uint32_t)N, a.act = LAGS_ACT_NONE, a.y = dx, a.ldy = lddx;
    a.part = (float *)ws, a.turned = (char *)ws + c.turned;
    results(a, lin->dtype);
    // W's rows run along the product's columns; turned round, along the outs
    const int how = c.bwd.turn && !how_of({{a.a, a.lda}}, N, lin->dtype) ? 0 : how_of({{a.a, a.lda}, {w, ldw}}, N | K, lin->dtype);
    return hip(launch_linear(c.bwd, a, true, how, lin->dtype, s));
}

}  // extern "C"
