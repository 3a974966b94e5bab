// Host side of the activation operators: argument validation, workspace sizes
// and launches.  The entry points are declared in include/lags.h.
#include "lags.h"
#include "lags_args.h"
#include "lags_gn.h"

#include <algorithm>
#include <cmath>
#include <initializer_list>

using namespace lags;

static_assert(kF32 == LAGS_F32 && kBF16 == LAGS_BF16 && kF16 == LAGS_F16, "one numbering");
static_assert(kActNone == LAGS_ACT_NONE && kActRelu == LAGS_ACT_RELU && kActSilu == LAGS_ACT_SILU,
              "one numbering");
static_assert(kRun == LAGS_CKPT_RUN && kSlabMax == LAGS_SLAB_MAX, "one size");
// A resident workgroup reaches its rows by 32-bit offsets: its lanes span 32 columns at least (8 lanes
// of fp32, 4 of 16-bit values), the others take kMostRows rows each, of LAGS_GN_MAX elements at most.
static_assert((uint64_t)kResident * kMostRows / 2 * LAGS_GN_MAX < 0x7fffffffull, "32-bit offsets");

namespace {
uint32_t gcd(uint32_t a, uint32_t b) { return b ? gcd(b, a % b) : a; }
}  // namespace

namespace lags {
// Register rows a thread of a resident workgroup aims at.  Forward 13: 28 x 28
// positions by 64 bf16 channels in 512 threads, two workgroups a compute unit
// (26 us for 64 x 784 x 512; 8 rows in 1024 threads: 28 us).  Backward 8, but 13
// with silu: by time, since both spill a few registers (64 x 784 x 512 bf16, 8
// and 13 rows: relu from the checkpoint 41.1 and 42.1 us, from x 50.6 and 50.7;
// silu from the checkpoint 56.7 and 51.0, from x 61.8 and 59.5).
static uint32_t rows_aimed_at(bool backward, int act) { return backward && act != kActSilu ? 8 : kMostRows; }

GnPlan gn_plan(int dtype, int act, bool backward, uint64_t N, uint64_t S, uint32_t C, uint32_t G)
{
    GnPlan p = {};
    const uint32_t E = elem_bytes(dtype), V = 16 / E, cg = C / G;
    // a slab is whole groups and whole runs
    const uint64_t whole = (uint64_t)(cg / gcd(cg, kRun)) * kRun;
    const uint32_t unit = whole < C ? (uint32_t)whole : C;
    if (unit > kSlabMax) return p;
    auto slab = [&](uint32_t bytes) {
        uint32_t w = unit;
        while (w < C && w * E < bytes && w + unit <= kSlabMax) w += unit;
        if (w > C) w = C;
        p.tcl = 0;
        while ((V << p.tcl) < w || (V << p.tcl) < kRun) ++p.tcl;
        p.w = w;
        p.nslab = (C + w - 1) / w;
        return S << p.tcl;                         // vectors of a slab's lanes
    };
    const uint32_t most = backward ? kResidentBwd : kResident;
    // the widest slab, up to 256 bytes of a row (forward: 128), that the registers aimed at hold and
    // that leaves two workgroups a compute unit; else 64 bytes, as long as they fit at all.
    // 64 x 196 x 1024 backward: 256 bytes 20 us, 64 bytes 23 us.
    uint64_t vecs = 0;
    for (uint32_t bytes = backward ? 256 : 128; bytes >= 64; bytes /= 2) {
        vecs = slab(bytes);
        if (vecs <= (uint64_t)most * (backward ? 8 : kMostRows) && N * p.nslab >= 512) break;
    }
    // A backward slab of 2049 to 4096 fp32 channels has more lanes than other workgroups and takes fewer
    // rows: in the split form a sample of one position leaves two sums for every value it has (16384 x 1 x
    // 4096: 537 MB of workspace beside 268 MB of data).
    const uint32_t lanes = 1u << p.tcl;
    const bool wide = lanes > most;
    // too few slabs to fill the GPU: split, unless the work is so small that one launch is what counts
    const uint64_t room = wide ? (uint64_t)lanes * kWideRows : (uint64_t)most * kMostRows;
    p.resident = lanes <= kResident && (vecs <= 2048 || (vecs <= room && N * p.nslab >= 128));
    if (p.resident) {
        const uint32_t rows = rows_aimed_at(backward, act);
        p.threads = lanes < 64 ? 64 : lanes;
        while (p.threads < 256 && (uint64_t)p.threads * 2 < vecs) p.threads *= 2;
        while (p.threads < most && (uint64_t)p.threads * rows < vecs) p.threads *= 2;
        p.rows = (uint32_t)((vecs + p.threads - 1) / p.threads);
        // backward: several samples a workgroup where there are far more than fill the GPU, or
        // where their channel sums, eight bytes a channel, would be more than the samples
        // themselves (8192 x 1 x 2048, one group: their sum takes 26 us for 8192 rows, 8 for 1024)
        uint64_t nper = 1;
        while (backward && nper < N &&
               (N * p.nslab / nper > 4096 || (N * p.nslab / nper > 1024 && S * nper < 32)))
            nper *= 2;
        p.nper = (uint32_t)nper;
        p.nparts = (uint32_t)((N + nper - 1) / nper);
    }
    if (!p.resident) {
        // 64 channels: 64 x 3136 x 256 backward 92 us (32: 97, 128: 95, 512: 99)
        slab(64 * E);
        p.threads = 1u << p.tcl;
        if (p.threads < 512) p.threads = 512;
        // chunks: about 1024 workgroups (256 to 4096 differ by 3 %)
        const uint64_t rows = p.threads >> p.tcl;
        uint64_t want = 1024 / (N * p.nslab);
        // but no more than sqrt(S) a sample: every workgroup joins the sums of its sample's chunks.
        // 1 x 11719 x 180 bf16 backward: at most sqrt(S) chunks 23 us, 2 sqrt(S) 26, no
        // limit 116; 3 x 6199 x 1178 fp32: 113, 175 and 180 us
        while (want > 1 && want * want > S) want -= want / 8 + 1;
        if (want < 1) want = 1;
        uint64_t chunk = (S + want - 1) / want;
        chunk = (chunk + rows - 1) / rows * rows;
        if (chunk > S) chunk = S;
        p.chunk = (uint32_t)chunk;
        p.nchunk = (uint32_t)((S + chunk - 1) / chunk);
        if (N * p.nchunk > kMostThreads) return GnPlan{};
        p.nparts = (uint32_t)(N * p.nchunk);
    }
    // a resident forward has as many launches as its samples need
    const uint64_t grid = (!p.resident ? N * p.nchunk : backward ? p.nparts : 1) * p.nslab;
    return grid * p.threads <= kMostThreads ? p : GnPlan{};
}

size_t gn_part_floats(const GnPlan &p, bool backward, uint64_t N, uint32_t C, uint32_t G)
{
    if (backward) return (size_t)p.nparts * 2 * C;
    return p.resident ? 0 : (size_t)N * G * p.nchunk * 2;
}

}  // namespace lags

namespace {

bool wgrad_dims(int64_t rows, int64_t outs, int64_t cols)
{
    return ckpt_dims(rows, cols) && cols <= LAGS_WGRAD_MAX && outs >= 1 && outs <= LAGS_WGRAD_MAX;
}

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
    size_t need;                     // workspace, of both
    int64_t rows;
};

int check_shape(const lags_gn *gn)
{
    if (!gn || !known_dtype(gn->dtype)) return LAGS_EINVAL;
    if (gn->act != LAGS_ACT_NONE && gn->act != LAGS_ACT_RELU && gn->act != LAGS_ACT_SILU) return LAGS_EINVAL;
    if (!(gn->eps >= 0) || !std::isfinite(gn->eps)) return LAGS_EINVAL;
    if (gn->samples < 0 || gn->spatial < 0 || gn->channels < 1 || gn->groups < 1) return LAGS_EINVAL;
    if (gn->samples > kMaxDim || gn->spatial > kMaxDim || gn->channels > LAGS_GN_MAX) return LAGS_ERANGE;
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
    c.fwd = gn_plan(gn->dtype, gn->act, false, N, S, C, G);
    c.bwd = gn_plan(gn->dtype, gn->act, true, N, S, C, G);
    if (!c.fwd.threads || !c.bwd.threads) return LAGS_ERANGE;
    const size_t f = gn_part_floats(c.fwd, false, N, C, G), b = gn_part_floats(c.bwd, true, N, C, G);
    const size_t floats = f > b ? f : b;
    c.need = c.rows ? (floats * 4 + 15) / 16 * 16 : 0;
    if (c.need < 16) c.need = 16;
    return LAGS_OK;
}

void fill(const lags_gn *gn, const GnPlan &p, GnArgs &a)
{
    const CkptShape cs = ckpt_shape(0, gn->channels);
    a.eps = gn->eps;
    a.N = (uint32_t)gn->samples, a.S = (uint32_t)gn->spatial;
    a.C = (uint32_t)gn->channels, a.G = (uint32_t)gn->groups, a.cg = a.C / a.G;
    a.pitch = cs.pitch, a.nrun = cs.nrun;
    a.act = gn->act, a.inv_cg = 1.0f / (float)a.cg;
    a.w = p.w, a.nslab = p.nslab, a.tcl = p.tcl, a.nchunk = p.nchunk, a.chunk = p.chunk;
    a.nper = p.nper, a.nparts = p.nparts;
}

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
    PackArgs a = {};
    a.s = ckpt_shape(rows, cols), a.ld = ldx;
    uint8_t *codes = (uint8_t *)ckpt, *scales = codes + (size_t)rows * a.s.pitch;
    for (int64_t r = 0, most = pack_rows(a.s, dtype); r < rows; r += most) {
        a.s.rows = std::min(most, rows - r);
        a.src = (const char *)x + r * ldx * elem_bytes(dtype);
        a.dst = codes + r * a.s.pitch, a.wscale = scales + r * a.s.nrun;
        if (int rc = hip(launch_pack(a, dtype, (hipStream_t)stream)); rc != LAGS_OK) return rc;
    }
    return LAGS_OK;
}

int lags_ckpt_unpack(int64_t rows, int64_t cols, const void *ckpt, size_t ckpt_bytes, void *x, int64_t ldx,
                     int32_t dtype, void *stream)
{
    if (int rc = check_pack(rows, cols, x, ldx, dtype, ckpt, ckpt_bytes); rc != LAGS_OK) return rc;
    PackArgs a = {};
    a.s = ckpt_shape(rows, cols), a.ld = ldx;
    const uint8_t *codes = (const uint8_t *)ckpt, *scales = codes + (size_t)rows * a.s.pitch;
    for (int64_t r = 0, most = pack_rows(a.s, dtype); r < rows; r += most) {
        a.s.rows = std::min(most, rows - r);
        a.src = codes + r * a.s.pitch, a.rscale = scales + r * a.s.nrun;
        a.dst = (char *)x + r * ldx * elem_bytes(dtype);
        if (int rc = hip(launch_unpack(a, dtype, (hipStream_t)stream)); rc != LAGS_OK) return rc;
    }
    return LAGS_OK;
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
    if (ldx > LAGS_GN_MAX || ldy > LAGS_GN_MAX) return LAGS_ERANGE;
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
    fill(gn, c.fwd, a);
    a.x = x, a.ldx = ldx, a.y = y, a.ldy = ldy;
    a.gamma = gamma, a.beta = beta, a.mean = mean, a.rstd = rstd;
    if (ckpt) a.wcodes = (uint8_t *)ckpt, a.wscales = (uint8_t *)ckpt + (size_t)c.rows * a.pitch;
    // A large y is stored past the caches: it would not stay there until it is read, and drives out x,
    // which a split forward reads twice.  With the operation before and after it in the loop: 103 MB 118
    // -> 107 us, 206 MB 219 -> 216, 51 MB 56.5 -> 57.7 (and no gain at any size for the backward's dx).
    a.past = (u128)c.rows * gn->channels * elem_bytes(gn->dtype) > ((u128)64 << 20);
    a.part = (float *)ws;
    return hip(launch_gn_forward(c.fwd, a, gn->dtype, (hipStream_t)stream));
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
    if (lddy > LAGS_GN_MAX || lddx > LAGS_GN_MAX || (x && ldx > LAGS_GN_MAX)) return LAGS_ERANGE;
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
    fill(gn, c.bwd, a);
    a.dy = dy, a.lddy = lddy, a.dx = dx, a.lddx = lddx, a.x = x, a.ldx = ldx;
    if (ckpt) a.rcodes = (const uint8_t *)ckpt, a.rscales = (const uint8_t *)ckpt + (size_t)c.rows * a.pitch;
    a.gamma = gamma, a.beta = beta, a.mean = (float *)mean, a.rstd = (float *)rstd;
    a.dgamma = dgamma, a.dbeta = dbeta, a.add = flags & LAGS_GRAD_ADD;
    a.part = (float *)ws;
    return hip(launch_gn_backward(c.bwd, a, gn->dtype, (hipStream_t)stream));
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
    if (!need || (u128)p.to * p.tc * p.split * 512 > kMostThreads) return LAGS_ERANGE;
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
