// Argument blocks and launches of the layer operators (layer normalisation,
// linear layers, embeddings).  Not part of the public ABI.
#pragma once

#include "lags_act.h"

namespace lags {

enum : int { kActGelu = 3 };                 // LAGS_ACT_GELU

// ---- layer normalisation ---------------------------------------------------
struct LnArgs {
    const void *x, *res, *dy, *dsum;
    void *sum, *y, *dx;
    int64_t ldx, ldr, lddy, ldds, lds, ldy, lddx;
    const uint8_t *rcodes, *rscales;         // checkpoint read (backward)
    uint8_t *wcodes, *wscales;               // checkpoint of the normalised rows, written (forward)
    uint8_t *ycodes, *yscales;               // checkpoint of y, written (forward)
    const float *gamma, *beta;
    float *mean, *rstd, *dgamma, *dbeta, *part;
    float eps, inv_c;
    int64_t rows;
    uint32_t C, pitch, nrun;
    uint32_t add;
    uint32_t tl;                             // 2^tl lanes a row
};
struct LnPlan {
    uint32_t tl, nv;                         // 2^tl lanes a row, vectors a lane
    uint32_t threads, groups;                // threads a workgroup, workgroups
};
constexpr int64_t kLnMax = 16384;            // channels, at most: 1024 threads of 16 values
// What the edges of rows ask for: nothing (whole vectors from whole words), columns past the last
// one to be cleared, or also words to be shifted into place (rows of 16-bit values that start inside one).
enum : int { kWhole = 0, kRagged = 1, kShifted = 2 };
LnPlan ln_plan(int dtype, bool backward, int edge, int64_t rows, uint32_t C);
hipError_t launch_ln_forward(const LnPlan &p, LnArgs a, int dtype, int edge, hipStream_t s);
hipError_t launch_ln_backward(const LnPlan &p, LnArgs a, int dtype, int edge, hipStream_t s);

// ---- embeddings ------------------------------------------------------------
struct EmbedArgs {
    const void *ids, *table, *dy;
    void *y;
    int64_t ldy, lddy, tokens;
    uint32_t vocab, cols;
    float scale;
    uint32_t add;
    float *dtable;
    // workspace: tokens by id, their ids, the ids' first places, chunks' sums [nchunk][2][cols]
    uint32_t *order, *keys, *start;
    float *part;
    uint32_t w;                              // ids a workgroup of the sort
    uint32_t chunk, nchunk, tl, nslab;       // tokens a chunk, chunks, 2^tl lanes a slab, slabs a row
    uint32_t zl, njoin, first;               // 2^zl lanes a row of zeros; 256-channel parts; a join's first chunk
    uint32_t past;                           // zeros go past the caches
};
constexpr int kFew = 256;                    // tokens of a gradient in one launch, at most
struct EmbedPlan {
    bool few;
    uint32_t w, chunk, nchunk, tl, nslab, njoin;
    uint64_t sumwgs, fewwgs;                 // workgroups of the sums; of the gradient in one launch
};
EmbedPlan embed_plan(int dtype, int64_t tokens, int64_t vocab, int64_t cols);
hipError_t launch_embed(EmbedArgs a, int table, int dtype, bool wide, hipStream_t s);
hipError_t launch_embed_grad(const EmbedPlan &p, EmbedArgs a, int dtype, bool wide, hipStream_t s);

// ---- linear layers ---------------------------------------------------------
struct LinArgs {
    // the product C = A B': a [M][K]; b forward W [N][K], backward W [K][N]
    const void *a, *b;
    int64_t lda, ldb, M;
    uint32_t N, K;
    int act;
    const float *bias;
    const void *res;
    void *z, *y;                             // C + bias; act of it + res
    int64_t ldr, ldz, ldy;
    float *part;                             // slices' sums [split][M][N]; column sums [chunks][N]
    void *turned;                            // W turned round
    uint32_t whole, past;                    // y, z and res have rows of whole vectors from whole words; they are
                                             // stored past the caches
    uint32_t tm, tn, split, k_per;           // tiles, slices of k, what a slice has of it (whole steps)
    // dz = dy act'(zin) over M x N
    const void *dy, *zin;
    void *dz;
    int64_t lddy, lddz, rows_per;
    uint32_t tl, nslab;
    float *dbias;                            // one chunk of rows: written, or added to, at once
    uint32_t add;
};
// Tiles of the product (rows, columns) and their waves.
struct LinTile {
    int bm, bn, wm, wn;
};
constexpr LinTile kLinTiles[] = {{256, 256, 2, 4}, {128, 128, 2, 2}, {64, 64, 2, 2}, {32, 128, 1, 4}};
struct LinPlan {
    uint32_t tile, tm, tn, split, k_per;
    bool turn;                               // backward: W is turned round first, where that can be used
};
struct DzPlan {
    uint32_t tl, nslab, chunks;
    int64_t rows_per;
};
constexpr int64_t kLinearMax = 1 << 20;      // cols, outs and every ld: 256 rows stay within 32-bit offsets
LinPlan linear_plan(int dtype, bool backward, int64_t M, int64_t N, int64_t K);
DzPlan dz_plan(int dtype, int64_t M, int64_t N);
template <int D> hipError_t product(const LinPlan &p, LinArgs a, bool nn, int how, hipStream_t s);
template <int D> hipError_t slopes(const DzPlan &p, LinArgs a, hipStream_t s);
// how: 0 operands of whole 16-byte vectors, 1 of rows that start on words, 2 on halves of them
hipError_t launch_linear(const LinPlan &p, const LinArgs &a, bool nn, int how, int dtype, hipStream_t s);
hipError_t launch_slopes(const DzPlan &p, const LinArgs &a, int dtype, hipStream_t s);
hipError_t launch_dbias(const float *part, uint32_t rows, uint32_t N, float *dbias, uint32_t add, hipStream_t s);

// dgamma, dbeta: sums over `rows` rows of part [rows][2][C] (dbeta's sums
// first), in a fixed order; either may be null (lags_gn.hip).
hipError_t launch_params(const float *part, uint32_t rows, uint32_t C, float *dgamma, float *dbeta, uint32_t add,
                         hipStream_t s);

}  // namespace lags
