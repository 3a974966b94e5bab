// Host side of the activation operators: argument validation, workspace sizes
// and launches.  The entry points are declared in include/lags.h.
#include "lags.h"
#include "lags_act.h"

#include <cmath>

using namespace lags;

static_assert(kF32 == LAGS_F32 && kBF16 == LAGS_BF16 && kF16 == LAGS_F16, "one numbering");
static_assert(kActNone == LAGS_ACT_NONE && kActRelu == LAGS_ACT_RELU && kActSilu == LAGS_ACT_SILU,
              "one numbering");
static_assert(kRun == LAGS_CKPT_RUN && kSlabMax == LAGS_SLAB_MAX, "one size");

namespace {

typedef unsigned __int128 u128;
constexpr int64_t kMaxDim = 0x7fffffff;
constexpr u128 kMaxBytes = (u128)1 << 62;

bool aligned(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool known_dtype(int32_t d) { return d == LAGS_F32 || d == LAGS_BF16 || d == LAGS_F16; }

// A strided region of device memory: `rows` runs of `width` bytes, `pitch` bytes apart.
struct Region {
    const void *p;
    u128 rows, width, pitch;
    u128 bytes() const { return rows ? (rows - 1) * pitch + width : 0; }
};

Region flat(const void *p, size_t bytes) { return {p, 1, bytes, bytes}; }

// Columns of one buffer taken at the same pitch do not overlap where their
// columns do not; regions of unlike pitch count as overlapping where their
// address ranges meet.
bool overlap(const Region &a, const Region &b)
{
    if (!a.p || !b.p || !a.bytes() || !b.bytes()) return false;
    const u128 x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    if (x + a.bytes() <= y || y + b.bytes() <= x) return false;
    if (a.pitch != b.pitch || a.rows < 2 || b.rows < 2) return true;
    // the later column's distance past the earlier one, within a row
    const u128 d = x <= y ? (y - x) % a.pitch : (a.pitch - (x - y) % a.pitch) % a.pitch;
    return d < a.width || d + b.width > a.pitch;
}

// A [rows, cols] matrix argument: its region, or a status.
int matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int32_t dtype, Region &r)
{
    const uint32_t e = elem_bytes(dtype);
    if (!p || !aligned(p, e) || ld < cols) return LAGS_EINVAL;
    if ((u128)rows * (u128)ld * e > kMaxBytes) return LAGS_ERANGE;
    r = {p, (u128)rows, (u128)cols * e, (u128)ld * e};
    return LAGS_OK;
}

bool ckpt_dims(int64_t rows, int64_t cols)
{
    return rows >= 0 && cols >= 1 && cols <= kMaxDim && (u128)rows * (u128)(cols + 64) * 2 <= kMaxBytes;
}

bool wgrad_dims(int64_t rows, int64_t outs, int64_t cols)
{
    return ckpt_dims(rows, cols) && cols <= LAGS_WGRAD_MAX && outs >= 1 && outs <= LAGS_WGRAD_MAX;
}

int hip(hipError_t e) { return e == hipSuccess ? LAGS_OK : LAGS_EHIP; }

int check_pack(int64_t rows, int64_t cols, const void *x, int64_t ldx, int32_t dtype, const void *ckpt,
               size_t ckpt_bytes)
{
    if (!known_dtype(dtype)) return LAGS_EINVAL;
    if (!ckpt_dims(rows, cols)) return LAGS_ERANGE;
    Region m;
    if (int rc = matrix(x, rows, cols, ldx, dtype, m); rc != LAGS_OK) return rc;
    const size_t need = ckpt_size(ckpt_shape(rows, cols));
    if (!ckpt || !aligned(ckpt, 16) || ckpt_bytes < need) return LAGS_EWORKSPACE;
    return overlap(m, flat(ckpt, need)) ? LAGS_EINVAL : LAGS_OK;
}

struct GnCall {
    GnPlan fwd, bwd;
    size_t need;                     // workspace, of both directions
    int64_t rows;
};

int check_shape(const lags_gn *gn)
{
    if (!gn || !known_dtype(gn->dtype)) return LAGS_EINVAL;
    if (gn->act != LAGS_ACT_NONE && gn->act != LAGS_ACT_RELU && gn->act != LAGS_ACT_SILU) return LAGS_EINVAL;
    if (!(gn->eps >= 0) || !std::isfinite(gn->eps)) return LAGS_EINVAL;
    if (gn->samples < 0 || gn->spatial < 0 || gn->channels < 1 || gn->groups < 1) return LAGS_EINVAL;
    if (gn->samples > kMaxDim || gn->spatial > kMaxDim || gn->channels > kMaxDim) return LAGS_ERANGE;
    if (gn->channels % gn->groups) return LAGS_EINVAL;
    return LAGS_OK;
}

int plan(const lags_gn *gn, GnCall &c)
{
    if (int rc = check_shape(gn); rc != LAGS_OK) return rc;
    c.rows = gn->samples * gn->spatial;
    // an empty call is planned as one of one row, whose limits are the same
    const uint64_t N = gn->samples ? gn->samples : 1, S = gn->spatial ? gn->spatial : 1;
    const uint32_t C = (uint32_t)gn->channels, G = (uint32_t)gn->groups;
    c.fwd = gn_plan(gn->dtype, false, N, S, C, G);
    c.bwd = gn_plan(gn->dtype, true, N, S, C, G);
    if (!c.fwd.threads || !c.bwd.threads) return LAGS_ERANGE;
    const size_t f = gn_part_floats(c.fwd, false, N, C, G) * 4, b = gn_part_floats(c.bwd, true, N, C, G) * 4;
    c.need = c.rows ? ((f > b ? f : b) + 15) / 16 * 16 : 0;
    if (c.need < 16) c.need = 16;
    return LAGS_OK;
}

void fill(const lags_gn *gn, GnArgs &a)
{
    const CkptShape cs = ckpt_shape(0, gn->channels);
    a.eps = gn->eps;
    a.N = (uint32_t)gn->samples, a.S = (uint32_t)gn->spatial;
    a.C = (uint32_t)gn->channels, a.G = (uint32_t)gn->groups, a.cg = a.C / a.G;
    a.pitch = cs.pitch, a.nrun = cs.nrun;
}

// `out` must not overlap any of the n regions of `all` but itself.
bool clear_of(const Region *all, int n, int out)
{
    for (int i = 0; i < n; ++i)
        if (i != out && overlap(all[i], all[out])) return false;
    return true;
}

bool same(const Region &a, const Region &b) { return a.p == b.p && a.pitch == b.pitch; }

}  // namespace

extern "C" {

size_t lags_ckpt_bytes(int64_t rows, int64_t cols)
{
    return ckpt_dims(rows, cols) ? ckpt_size(ckpt_shape(rows, cols)) : 0;
}

int lags_ckpt_pack(int64_t rows, int64_t cols, const void *x, int64_t ldx, int32_t dtype, void *ckpt,
                   size_t ckpt_bytes, void *stream)
{
    if (int rc = check_pack(rows, cols, x, ldx, dtype, ckpt, ckpt_bytes); rc != LAGS_OK) return rc;
    if (!rows) return LAGS_OK;
    PackArgs a = {};
    a.s = ckpt_shape(rows, cols);
    a.src = x, a.ld = ldx;
    a.dst = ckpt;
    a.wscale = (uint8_t *)ckpt + (size_t)rows * a.s.pitch;
    return hip(launch_pack(a, dtype, (hipStream_t)stream));
}

int lags_ckpt_unpack(int64_t rows, int64_t cols, const void *ckpt, size_t ckpt_bytes, void *x, int64_t ldx,
                     int32_t dtype, void *stream)
{
    if (int rc = check_pack(rows, cols, x, ldx, dtype, ckpt, ckpt_bytes); rc != LAGS_OK) return rc;
    if (!rows) return LAGS_OK;
    PackArgs a = {};
    a.s = ckpt_shape(rows, cols);
    a.src = ckpt, a.ld = ldx;
    a.dst = x;
    a.rscale = (const uint8_t *)ckpt + (size_t)rows * a.s.pitch;
    return hip(launch_unpack(a, dtype, (hipStream_t)stream));
}

size_t lags_gn_workspace_bytes(const lags_gn *gn)
{
    GnCall c;
    return plan(gn, c) == LAGS_OK ? c.need : 0;
}

int lags_gn_forward(const lags_gn *gn, const void *x, int64_t ldx, const float *gamma, const float *beta, void *y,
                    int64_t ldy, float *mean, float *rstd, void *ckpt, size_t ckpt_bytes, void *ws, size_t ws_bytes,
                    void *stream)
{
    GnCall c;
    if (int rc = plan(gn, c); rc != LAGS_OK) return rc;
    Region r[8];
    if (int rc = matrix(x, c.rows, gn->channels, ldx, gn->dtype, r[0]); rc != LAGS_OK) return rc;
    if (int rc = matrix(y, c.rows, gn->channels, ldy, gn->dtype, r[1]); rc != LAGS_OK) return rc;
    if (!gamma != !beta || !aligned(gamma, 4) || !aligned(beta, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
        return LAGS_EINVAL;
    const size_t cb = (size_t)gn->channels * 4, sb = (size_t)gn->samples * gn->groups * 4;
    r[2] = flat(gamma, cb), r[3] = flat(beta, cb), r[4] = flat(mean, sb), r[5] = flat(rstd, sb);
    size_t need_ck = 0;
    if (ckpt) {
        if (!ckpt_dims(c.rows, gn->channels)) return LAGS_ERANGE;
        need_ck = ckpt_size(ckpt_shape(c.rows, gn->channels));
        if (!aligned(ckpt, 16) || ckpt_bytes < need_ck) return LAGS_EWORKSPACE;
    }
    if (!ws || !aligned(ws, 16) || ws_bytes < c.need) return LAGS_EWORKSPACE;
    r[6] = flat(ckpt, need_ck), r[7] = flat(ws, c.need);
    for (int out : {4, 5, 6, 7})
        if (!clear_of(r, 8, out)) return LAGS_EINVAL;
    if (overlap(r[1], r[2]) || overlap(r[1], r[3]) || (overlap(r[0], r[1]) && !same(r[0], r[1]))) return LAGS_EINVAL;
    if (!c.rows) return LAGS_OK;
    GnArgs a = {};
    fill(gn, a);
    a.x = x, a.ldx = ldx, a.y = y, a.ldy = ldy;
    a.gamma = gamma, a.beta = beta, a.mean = mean, a.rstd = rstd;
    if (ckpt) a.wcodes = (uint8_t *)ckpt, a.wscales = (uint8_t *)ckpt + (size_t)c.rows * a.pitch;
    a.part = (float *)ws;
    return hip(launch_gn_forward(c.fwd, a, gn->dtype, gn->act, (hipStream_t)stream));
}

int lags_gn_backward(const lags_gn *gn, const void *dy, int64_t lddy, const void *x, int64_t ldx, const void *ckpt,
                     size_t ckpt_bytes, const float *gamma, const float *beta, const float *mean, const float *rstd,
                     void *dx, int64_t lddx, float *dgamma, float *dbeta, uint32_t flags, void *ws, size_t ws_bytes,
                     void *stream)
{
    GnCall c;
    if (int rc = plan(gn, c); rc != LAGS_OK) return rc;
    if (flags & ~LAGS_GRAD_ADD) return LAGS_EINVAL;
    if (!x == !ckpt) return LAGS_EINVAL;
    Region r[11];
    if (int rc = matrix(dy, c.rows, gn->channels, lddy, gn->dtype, r[0]); rc != LAGS_OK) return rc;
    if (int rc = matrix(dx, c.rows, gn->channels, lddx, gn->dtype, r[1]); rc != LAGS_OK) return rc;
    size_t need_ck = 0;
    r[2] = flat(nullptr, 0);
    if (x) {
        if (int rc = matrix(x, c.rows, gn->channels, ldx, gn->dtype, r[2]); rc != LAGS_OK) return rc;
    } else {
        if (!ckpt_dims(c.rows, gn->channels)) return LAGS_ERANGE;
        need_ck = ckpt_size(ckpt_shape(c.rows, gn->channels));
        if (!aligned(ckpt, 16) || ckpt_bytes < need_ck) return LAGS_EWORKSPACE;
    }
    if (!gamma != !beta || !mean || !rstd || !aligned(gamma, 4) || !aligned(beta, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4) || !aligned(dgamma, 4) || !aligned(dbeta, 4))
        return LAGS_EINVAL;
    if (!ws || !aligned(ws, 16) || ws_bytes < c.need) return LAGS_EWORKSPACE;
    const size_t cb = (size_t)gn->channels * 4, sb = (size_t)gn->samples * gn->groups * 4;
    r[3] = flat(ckpt, need_ck);
    r[4] = flat(gamma, cb), r[5] = flat(beta, cb), r[6] = flat(mean, sb), r[7] = flat(rstd, sb);
    r[8] = flat(dgamma, cb), r[9] = flat(dbeta, cb), r[10] = flat(ws, c.need);
    for (int out : {8, 9, 10})
        if (!clear_of(r, 11, out)) return LAGS_EINVAL;
    for (int in = 2; in < 8; ++in)
        if (overlap(r[1], r[in])) return LAGS_EINVAL;
    if (overlap(r[0], r[1]) && !same(r[0], r[1])) return LAGS_EINVAL;
    GnArgs a = {};
    fill(gn, a);
    a.dy = dy, a.lddy = lddy, a.dx = dx, a.lddx = lddx, a.x = x, a.ldx = ldx;
    if (ckpt) a.rcodes = (const uint8_t *)ckpt, a.rscales = (const uint8_t *)ckpt + (size_t)c.rows * a.pitch;
    a.gamma = gamma, a.beta = beta, a.mean = (float *)mean, a.rstd = (float *)rstd;
    a.dgamma = dgamma, a.dbeta = dbeta, a.add = flags & LAGS_GRAD_ADD;
    a.part = (float *)ws;
    return hip(launch_gn_backward(c.bwd, a, gn->dtype, gn->act, (hipStream_t)stream));
}

size_t lags_ckpt_wgrad_workspace_bytes(int64_t rows, int64_t outs, int64_t cols, int32_t dtype)
{
    if (!known_dtype(dtype) || !wgrad_dims(rows, outs, cols)) return 0;
    const WgradPlan p = wgrad_plan(dtype, rows, outs, cols);
    const u128 n = p.split > 1 ? (u128)p.split * (u128)outs * (u128)cols * 4 : 16;
    return n > kMaxBytes ? 0 : (size_t)((n + 15) / 16 * 16);
}

int lags_ckpt_wgrad(int64_t rows, int64_t outs, int64_t cols, const void *dy, int64_t lddy, int32_t dtype,
                    const void *ckpt, size_t ckpt_bytes, float *dw, uint32_t flags, void *ws, size_t ws_bytes,
                    void *stream)
{
    if (!known_dtype(dtype) || (flags & ~LAGS_GRAD_ADD)) return LAGS_EINVAL;
    if (!wgrad_dims(rows, outs, cols)) return LAGS_ERANGE;
    Region r[4];
    if (int rc = matrix(dy, rows, outs, lddy, dtype, r[0]); rc != LAGS_OK) return rc;
    if (lddy > LAGS_WGRAD_MAX) return LAGS_ERANGE;
    if (!dw || !aligned(dw, 4)) return LAGS_EINVAL;
    const size_t need_ck = ckpt_size(ckpt_shape(rows, cols));
    if (!ckpt || !aligned(ckpt, 16) || ckpt_bytes < need_ck) return LAGS_EWORKSPACE;
    const size_t need = lags_ckpt_wgrad_workspace_bytes(rows, outs, cols, dtype);
    const WgradPlan p = wgrad_plan(dtype, rows, outs, cols);
    if (!need || (u128)p.to * p.tc * p.split > kMaxDim) return LAGS_ERANGE;
    if (!ws || !aligned(ws, 16) || ws_bytes < need) return LAGS_EWORKSPACE;
    r[1] = flat(ckpt, need_ck), r[2] = flat(dw, (size_t)outs * cols * 4), r[3] = flat(ws, need);
    if (!clear_of(r, 4, 2) || !clear_of(r, 4, 3)) return LAGS_EINVAL;
    WgradArgs a = {};
    const CkptShape cs = ckpt_shape(rows, cols);
    a.dy = dy, a.lddy = lddy;
    a.codes = (const uint8_t *)ckpt, a.scales = (const uint8_t *)ckpt + (size_t)rows * cs.pitch;
    a.dw = dw, a.part = (float *)ws;
    a.M = rows, a.O = (uint32_t)outs, a.C = (uint32_t)cols, a.pitch = cs.pitch, a.nrun = cs.nrun;
    a.add = flags & LAGS_GRAD_ADD;
    return hip(launch_wgrad(p, a, dtype, (hipStream_t)stream));
}

}  // extern "C"
