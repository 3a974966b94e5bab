// Embeddings: y[t] = scale * table[ids[t]], and the table's gradient, whose row v
// is scale times the sum of dy over the tokens t with ids[t] = v, in the order of
// t.  An id outside [0, vocab) gives a row of zeros and adds to no gradient.
//
// Forward: a gather bound by memory; a thread has four tokens' vectors in flight.
// Gradient: the tokens are sorted by id (their order within an id kept), and
// the sorted list is cut into chunks of 8 or 16 tokens, so that a frequent id is
// the work of many workgroups.  A chunk adds up each id's rows in registers; an
// id that lies within one chunk is written to the table's gradient, the others
// leave a sum for each chunk, which are then added up in the order of the chunks.
// No atomics on floats: results repeat bit for bit.
//   lookup, 16384 tokens of 50304 x 2048, fp32 to bf16   26 us (3.4 TB/s with each row read once)
//   gradient of the same                                 113 to 122 us (4 TB/s): 85 sorting beside 368 MB
//                                                        of zeros, 23 the sums, 6 joining them
//   gradient, 700 tokens of 10000 x 1500 fp32            21 us: 14, 4, 3
// Many more tokens are bound by the sort, in which each workgroup reads all ids and one ranks the most frequent: of
// 50304 x 512 bf16 32768 take 65 us (27 at the rate of a copy), 65536 105 (33), 200000 310 to 333 (60).
#include "lags_gn.h"
#include "lags_layer.h"

#include <algorithm>

namespace lags {
namespace {

// The id of token t; `none` (never below vocab) where it is outside the vocabulary.
constexpr uint32_t kNone = 0xffffffffu;
typedef float f32x4 __attribute__((ext_vector_type(4)));
template <bool WIDE> __device__ inline uint32_t id_of(const EmbedArgs &a, int64_t t)
{
    if constexpr (WIDE) {
        const uint64_t v = ((const uint64_t *)a.ids)[t];
        return v < a.vocab ? (uint32_t)v : kNone;
    } else {
        const uint32_t v = ((const uint32_t *)a.ids)[t];
        return v < a.vocab ? v : kNone;
    }
}

// V values of a table row from channel c on, as fp32 (n of them count).
template <int TD, int V> __device__ inline void row_values(const void *p, int n, float (&f)[V])
{
    constexpr int TV = Elem<TD>::V;
#pragma unroll
    for (int i = 0; i < V / TV; ++i) {
        float g[TV];
        Elem<TD>::unpack(load_vec<TD>((const char *)p + i * 16, n - i * TV), g);
        for (int j = 0; j < TV; ++j) f[i * TV + j] = g[j];
    }
}

template <int TD, int D, bool WIDE, int U> __global__ __launch_bounds__(256) void k_embed(EmbedArgs a)
{
    constexpr int V = Elem<D>::V, E = Elem<D>::E, TE = Elem<TD>::E;
    const uint32_t T = 1u << a.tl, R = 256 >> a.tl;
    const uint32_t col = threadIdx.x & (T - 1);
    const int64_t t0 = (int64_t)blockIdx.x * (R * U) + (threadIdx.x >> a.tl);
    uint32_t id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = t0 + u * R < a.tokens ? id_of<WIDE>(a, t0 + u * R) : kNone;
    for (uint32_t c = col * V; c < a.cols; c += T * V) {
        const int n = (int)(a.cols - c);
        float f[U][V] = {};
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (id[u] != kNone) row_values<TD>((const char *)a.table + ((size_t)id[u] * a.cols + c) * TE, n, f[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = t0 + u * R;
            for (int j = 0; j < V; ++j) f[u][j] *= a.scale;
            if (t < a.tokens) store_vec<D>((char *)a.y + (t * a.ldy + c) * E, Elem<D>::pack(f[u]), n);
        }
    }
}

// n zeros from p on, by T lanes.  Rows of a flat buffer's slice start anywhere: vectors from the first whole line
// of 128 bytes on, single values before and behind them.  `past`: zeros of more than 128 MB, which the cache would
// only have to write back, go past it: 700 tokens of 60000 x 1501 fp32 121 -> 92 us, 16384 of 50304 x 2048 bf16 one
// value off 136 -> 122 (rows of whole lines 120 -> 117), 256 of 50304 x 2001 96 -> 79; 700 of 10000 x 1500 (60 MB) stays at 21, past the
// cache 26.
__device__ inline void zeros(float *p, uint32_t n, uint32_t lane, uint32_t T, uint32_t past)
{
    const f32x4 zero = {0, 0, 0, 0};
    const uint32_t head = min(n, (uint32_t)(-(uintptr_t)p >> 2) & 31), body = head + ((n - head) & ~3u);
    for (uint32_t c = lane; c < head; c += T) p[c] = 0;
    if (past)
        for (uint32_t c = head + lane * 4; c < body; c += T * 4) __builtin_nontemporal_store(zero, (f32x4 *)(p + c));
    else
        for (uint32_t c = head + lane * 4; c < body; c += T * 4) *(f32x4 *)(p + c) = zero;
    if (body + lane < n) p[body + lane] = 0;
}

// Tokens sorted by id: order[], their ids keys[], and start[v], the first place
// of id v (start[vocab]: how many tokens have an id); and (not adding) zeros in the
// rows of ids without tokens.  A workgroup owns a.w ids.  Its 16 waves each read a
// section of all tokens; within 64 of them a token's place among those of its id
// comes from comparing ids across the wave, and the section's count so far from
// LDS.  What ids and sections before it hold is added last.  The zeros, most of
// the memory that a gradient writes, are written while workgroups with frequent
// ids still sort (16384 tokens whose frequencies fall as 1 / rank: half of them in the first
// of 256 workgroups).
constexpr int kSortWaves = 16, kHeld = 16;
template <bool WIDE> __global__ __launch_bounds__(64 * kSortWaves) void k_embed_sort(EmbedArgs a)
{
    extern __shared__ uint32_t cnt[];               // [wave][a.w], then each id's count
    __shared__ uint32_t sum[kSortWaves], low[kSortWaves];
    uint32_t *count = cnt + kSortWaves * a.w;
    const uint32_t lo = blockIdx.x * a.w, w = min(a.w, a.vocab - lo);
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (uint32_t i = threadIdx.x; i < kSortWaves * a.w; i += 64 * kSortWaves) cnt[i] = 0;
    __syncthreads();
    const int64_t per = (a.tokens + 64 * kSortWaves - 1) / (64 * kSortWaves) * 64;
    const int64_t s0 = min(a.tokens, per * wave), s1 = min(a.tokens, s0 + per);
    uint32_t *mine = cnt + wave * a.w;
    uint32_t id[kHeld], place[kHeld];
    auto load = [&](int64_t s) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const int64_t t = s + k * 64 + lane;
            id[k] = t < s1 ? id_of<WIDE>(a, t) : kNone;
        }
    };
    const int bits = 32 - __builtin_clz(a.w);
    // A token's place among its id's, counted on from what `mine` holds.
    auto rank = [&](uint32_t key, bool in) -> uint32_t {
        const uint64_t all = __ballot(in);
        uint32_t same0 = (uint32_t)all, same1 = (uint32_t)(all >> 32);
        for (int b = 0; b < bits; ++b) {
            const uint64_t m = __ballot(key >> b & 1);
            const uint32_t mine1 = (uint32_t)((int)(key << (31 - b)) >> 31);          // all ones where the bit is set
            same0 &= ~((uint32_t)m ^ mine1), same1 &= ~((uint32_t)(m >> 32) ^ mine1);
        }
        uint32_t at = 0;
        if (in) {
            const int first = same0 ? __builtin_ctz(same0) : 32 + __builtin_ctz(same1);
            const uint32_t before = __builtin_amdgcn_mbcnt_hi(same1, __builtin_amdgcn_mbcnt_lo(same0, 0));
            if ((int)lane == first) at = atomicAdd(mine + key, (uint32_t)(__builtin_popcount(same0) + __builtin_popcount(same1)));
            at = __shfl(at, first) + before;
        }
        return at;
    };
    const bool held = per <= 64 * kHeld;             // a section stays in registers
    uint32_t below = 0;
    for (int64_t s = s0; s < s1; s += 64 * kHeld) {
        load(s);
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const uint32_t key = id[k] - lo;
            const bool in = key < w;
            below += id[k] < lo;
            if (!__ballot(in)) continue;
            if (held)
                place[k] = rank(key, in);
            else if (in)
                atomicAdd(mine + key, 1u);
        }
    }
    for (int o = 32; o; o >>= 1) below += __shfl_xor(below, o);
    if (lane == 0) low[wave] = below;
    __syncthreads();
    // ids' counts, their exclusive sum over the range, and each wave's first place
    const uint32_t i = threadIdx.x;
    uint32_t total = 0;
    if (i < w)
        for (int k = 0; k < kSortWaves; ++k) total += cnt[k * a.w + i];
    uint32_t run = total;
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t v = __shfl_up(run, o);
        if ((int)lane >= o) run += v;
    }
    if (lane == 63) sum[wave] = run;
    __syncthreads();
    uint32_t at = run - total;
    for (uint32_t k = 0; k < kSortWaves; ++k) at += low[k] + (k < wave ? sum[k] : 0);
    if (i < w) {
        a.start[lo + i] = at;
        count[i] = total;
        if (lo + i + 1 == a.vocab) a.start[a.vocab] = at + total;
        for (int k = 0; k < kSortWaves; ++k) {
            const uint32_t c = cnt[k * a.w + i];
            cnt[k * a.w + i] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int64_t s = s0; s < s1; s += 64 * kHeld) {
        if (!held) load(s);
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const uint32_t key = id[k] - lo;
            const bool in = key < w;
            if (!__ballot(in)) continue;
            uint32_t p = held ? place[k] : rank(key, in);
            if (in) {
                if (held) p += mine[key];
                a.order[p] = (uint32_t)(s + k * 64 + lane);
                a.keys[p] = id[k];
            }
        }
    }
    if (a.add) return;
    const uint32_t T = 1u << a.zl;
    for (uint32_t v = threadIdx.x >> a.zl; v < w; v += 64 * kSortWaves >> a.zl)
        if (!count[v]) zeros(a.dtable + (size_t)(lo + v) * a.cols, a.cols, threadIdx.x & (T - 1), T, a.past);
}

// Sums of one chunk's C tokens for each id in it.  2^tl lanes span a slab of a row's
// vectors, 64 of them at most.
template <int D, uint32_t C> __global__ __launch_bounds__(256) void k_embed_sum(EmbedArgs a)
{
    constexpr int V = Elem<D>::V, E = Elem<D>::E;
    const uint32_t T = 1u << a.tl;
    const uint64_t unit = (uint64_t)blockIdx.x * (256 >> a.tl) + (threadIdx.x >> a.tl);
    const uint32_t chunk = (uint32_t)(unit / a.nslab), slab = (uint32_t)(unit % a.nslab);
    const uint32_t c = (slab * T + (threadIdx.x & (T - 1))) * V;
    const int n = (int)a.cols - (int)c;
    if (chunk >= a.nchunk || n <= 0) return;
    // All places of the chunk and its neighbours' at once, not one after the other; those past the
    // last token's are read (the workspace goes on behind them) and not looked at.
    const uint32_t p0 = chunk * C, total = a.start[a.vocab];
    u32x4 v[C / 8][8], t[C / 4], key[C / 4];
#pragma unroll
    for (uint32_t h = 0; h < C / 4; ++h) t[h] = *(const u32x4 *)(a.order + p0 + 4 * h), key[h] = *(const u32x4 *)(a.keys + p0 + 4 * h);
    const uint32_t before = p0 ? a.keys[p0 - 1] : kNone, next = a.keys[p0 + C];
    if (p0 >= total) return;
    const uint32_t p1 = min(p0 + C, total), after = p1 < total ? next : kNone;
#pragma unroll
    for (uint32_t k = 0; k < C; ++k) {
        const uint32_t token = p0 + k < p1 ? t[k / 4][k % 4] : t[0][0];
        v[k / 8][k % 8] = load_vec<D>((const char *)a.dy + ((size_t)token * a.lddy + c) * E, n);
    }
    float acc[V] = {};
    uint32_t cur = key[0][0];
    bool first = cur == before;                    // the id began in an earlier chunk
    auto leave = [&](bool goes_on) {
        float *out = first ? a.part + (size_t)chunk * 2 * a.cols
                     : goes_on ? a.part + ((size_t)chunk * 2 + 1) * a.cols
                               : a.dtable + (size_t)cur * a.cols;
        out += c;
        const bool last = !first && !goes_on, add = last && a.add;
        if (last)
            for (int j = 0; j < V; ++j) acc[j] *= a.scale;
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            if (i + 4 <= n) {
                f32x4_u4 s = {acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
                if (add) s += *(f32x4_u4 *)(out + i);
                *(f32x4_u4 *)(out + i) = s;
            } else {
                for (int j = i; j < i + 4; ++j)
                    if (j < n) out[j] = add ? out[j] + acc[j] : acc[j];
            }
        }
    };
    auto take = [&](const u32x4(&w)[8], uint32_t k0) __attribute__((always_inline)) {
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
            const uint32_t k = k0 + i;
            if (p0 + k >= p1) break;
            if (key[k / 4][k % 4] != cur) {
                leave(false);
                cur = key[k / 4][k % 4], first = false;
                for (int j = 0; j < V; ++j) acc[j] = 0;
            }
            float f[V];
            Elem<D>::unpack(w[i], f);
            for (int j = 0; j < V; ++j) acc[j] += f[j];
        }
    };
    take(v[0], 0);
    if constexpr (C > 8) take(v[1], 8);
    leave(cur == after);
}

// The ids that began in a chunk and went on past it: their chunks' sums, four
// waves a run of them each.
__global__ __launch_bounds__(256) void k_embed_join(EmbedArgs a)
{
    __shared__ float4 sh[4][64];
    const uint32_t chunk = a.first + blockIdx.x / a.njoin, c = (blockIdx.x % a.njoin * 64 + (threadIdx.x & 63)) * 4;
    const uint32_t total = a.start[a.vocab], p0 = chunk * a.chunk, p1 = p0 + a.chunk;
    if (p1 >= total) return;
    const uint32_t v = a.keys[p1 - 1];
    if (a.keys[p1] != v || a.start[v] < p0) return;
    const uint32_t n = (a.start[v + 1] - 1) / a.chunk - chunk + 1;       // chunks with this id: this one's second sum, the others' first
    const uint32_t wave = threadIdx.x >> 6, k0 = (uint32_t)((uint64_t)n * wave / 4), k1 = (uint32_t)((uint64_t)n * (wave + 1) / 4);
    const int left = (int)a.cols - (int)c;
    float4 s = {0, 0, 0, 0};
    auto piece = [&](uint32_t k) { return a.part + ((size_t)(chunk + k) * 2 + (k == 0)) * a.cols + c; };
    if (left >= 4) {
#pragma unroll 8
        for (uint32_t k = k0; k < k1; ++k) {
            const f32x4_u4 t = *(const f32x4_u4 *)piece(k);
            s.x += t[0], s.y += t[1], s.z += t[2], s.w += t[3];
        }
    } else if (left > 0) {
        for (uint32_t k = k0; k < k1; ++k) {
            const float *p = piece(k);
            s.x += p[0];
            if (left > 1) s.y += p[1];
            if (left > 2) s.z += p[2];
        }
    }
    sh[wave][threadIdx.x & 63] = s;
    __syncthreads();
    if (wave || left <= 0) return;
    float f[4];
    for (int j = 0; j < 4; ++j) {
        const float *p = &sh[0][threadIdx.x].x + j;
        f[j] = a.scale * ((p[0] + p[64 * 4]) + (p[128 * 4] + p[192 * 4]));
    }
    float *out = a.dtable + (size_t)v * a.cols + c;
    for (int j = 0; j < 4; ++j)
        if (j < left) out[j] = a.add ? out[j] + f[j] : f[j];
}

// Few tokens: one launch.  Every wave holds all ids, kFew / 64 a lane; comparing
// them with an id of its own gives that id's tokens as bits, in order, and the
// wave adds up their rows, 64 vectors of them, or writes zeros.
constexpr int kFewIds = 4;                           // a wave's ids
template <int D, bool WIDE> __global__ __launch_bounds__(256) void k_embed_few(EmbedArgs a)
{
    constexpr int V = Elem<D>::V, E = Elem<D>::E, Q = kFew / 64, U = 8;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    uint32_t id[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) id[q] = q * 64 + lane < a.tokens ? id_of<WIDE>(a, q * 64 + lane) : kNone;
    const uint32_t unit = blockIdx.x * 4 + wave, v0 = unit / a.nslab * kFewIds;
    const uint32_t c = (unit % a.nslab * 64 + lane) * V;
    const int n = (int)a.cols - (int)c;
    for (uint32_t v = v0; v < min(a.vocab, v0 + kFewIds); ++v) {
        uint64_t m[Q], any = 0;
#pragma unroll
        for (int q = 0; q < Q; ++q) any |= m[q] = __ballot(id[q] == v);
        if (!any) {
            const uint32_t s0 = unit % a.nslab * 64 * V;
            if (!a.add) zeros(a.dtable + (size_t)v * a.cols + s0, min(64u * V, a.cols - s0), lane, 64, a.past);
            continue;
        }
        if (n <= 0) continue;
        float *out = a.dtable + (size_t)v * a.cols + c;
        float acc[V] = {};
#pragma unroll
        for (int q = 0; q < Q; ++q)
            for (uint64_t left = m[q]; left;) {
                u32x4 x[U];
                int k = 0;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int t = left ? __builtin_ctzll(left) : 0;
                    if (left) x[u] = load_vec<D>((const char *)a.dy + ((q * 64 + t) * a.lddy + c) * E, n), ++k;
                    left &= left - 1;
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (u >= k) break;
                    float f[V];
                    Elem<D>::unpack(x[u], f);
                    for (int j = 0; j < V; ++j) acc[j] += f[j];
                }
            }
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            if (i + 4 <= n) {
                f32x4_u4 s = {acc[i] * a.scale, acc[i + 1] * a.scale, acc[i + 2] * a.scale, acc[i + 3] * a.scale};
                if (a.add) s += *(f32x4_u4 *)(out + i);
                *(f32x4_u4 *)(out + i) = s;
            } else {
                for (int j = i; j < i + 4; ++j)
                    if (j < n) out[j] = a.add ? out[j] + acc[j] * a.scale : acc[j] * a.scale;
            }
        }
    }
}

uint32_t log2_up(uint64_t n, uint32_t lo, uint32_t hi)
{
    uint32_t l = lo;
    while (l < hi && (1ull << l) < n) ++l;
    return l;
}

}  // namespace

EmbedPlan embed_plan(int dtype, int64_t tokens, int64_t vocab, int64_t cols)
{
    EmbedPlan p = {};
    // One launch for a few tokens.  us in one and in three: 100 tokens of 100 x 100 fp32 6.5 and 12.2, 200 of 10000
    // x 1500 13 and 21, 256 of 50304 x 2048 bf16 75 and 93; but 700 of 10000 x 1500 57 and 21, where the rows of a
    // frequent id come 64 tokens at a time.
    // (a wave writes 64 vectors of four ids' rows; a table that needs more threads than a launch has takes three)
    const uint32_t V = 16 / elem_bytes(dtype);
    const uint64_t vecs = (cols + V - 1) / V;
    p.fewwgs = ((uint64_t)((vocab + kFewIds - 1) / kFewIds) * ((vecs + 63) / 64) + 3) / 4;
    p.few = tokens <= kFew && p.fewwgs * 256 <= kMostThreads;
    // ids a workgroup of the sort: 256 workgroups if the counts of 16 waves then stay within 32 KiB
    p.w = (uint32_t)std::min<int64_t>(512, (vocab + 255) / 256);
    // Tokens a chunk: short ones fill the card where there are few.  us for 8, 16 and 32: 700 tokens of 1500
    // fp32 22, 24, 28; 16384 of 2048 bf16 124, 118, 118 (1000 ids: 44, 40, 39).
    p.chunk = tokens < 8192 ? 8 : 16;
    p.nchunk = (uint32_t)((tokens + p.chunk - 1) / p.chunk);
    p.tl = log2_up(vecs, 2, 6);
    p.nslab = (uint32_t)((vecs + (1u << p.tl) - 1) >> p.tl);
    const uint64_t units = (uint64_t)p.nchunk * p.nslab, per = 256 >> p.tl;
    p.sumwgs = (units + per - 1) / per;
    p.njoin = (uint32_t)((cols + 255) / 256);
    return p;
}

hipError_t launch_embed(EmbedArgs a, int table, int dtype, bool wide, hipStream_t s)
{
    const uint32_t V = 16 / elem_bytes(dtype);
    a.tl = log2_up(((uint64_t)a.cols + V - 1) / V, 2, 8);
    const uint64_t rows = 256 >> a.tl;
    // four tokens a thread where that leaves enough workgroups
    const bool many = (uint64_t)a.tokens / (rows * 4) >= 1024;
    const uint64_t per = rows * (many ? 4 : 1);
    const int64_t most = (int64_t)(kMostThreads / 256 * per);
    for (int64_t t = 0, all = a.tokens; t < all; t += most) {
        EmbedArgs b = a;
        b.tokens = std::min(most, all - t);
        b.ids = (const char *)a.ids + t * (wide ? 8 : 4);
        b.y = (char *)a.y + t * a.ldy * elem_bytes(dtype);
        const uint32_t g = (uint32_t)((b.tokens + per - 1) / per);
        auto go = [&](auto td, auto d) {
            return by_bool(wide, [&](auto w) {
                return by_bool(many, [&](auto m) {
                    k_embed<td, d, w, m ? 4 : 1><<<g, 256, 0, s>>>(b);
                    return hipGetLastError();
                });
            });
        };
        const std::integral_constant<int, kF32> f32;
        const std::integral_constant<int, kBF16> bf16;
        const std::integral_constant<int, kF16> f16;
        const hipError_t e = dtype == kF32    ? go(f32, f32)
                             : dtype == kBF16 ? (table == kF32 ? go(f32, bf16) : go(bf16, bf16))
                                              : (table == kF32 ? go(f32, f16) : go(f16, f16));
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_embed_grad(const EmbedPlan &p, EmbedArgs a, int dtype, bool wide, hipStream_t s)
{
    a.w = p.w, a.chunk = p.chunk, a.nchunk = p.nchunk, a.tl = p.tl, a.nslab = p.nslab, a.njoin = p.njoin;
    a.past = (uint64_t)a.vocab * a.cols * 4 > (uint64_t)128 << 20;
    if (p.few) {
        const uint32_t V = 16 / elem_bytes(dtype), g = (uint32_t)p.fewwgs;
        a.nslab = ((a.cols + V - 1) / V + 63) / 64;
        return by_bool(wide, [&](auto w) {
            switch (dtype) {
            case kF32: k_embed_few<kF32, w><<<g, 256, 0, s>>>(a); break;
            case kBF16: k_embed_few<kBF16, w><<<g, 256, 0, s>>>(a); break;
            default: k_embed_few<kF16, w><<<g, 256, 0, s>>>(a); break;
            }
            return hipGetLastError();
        });
    }
    a.zl = log2_up(((uint64_t)a.cols + 3) / 4, 2, 10);
    const uint32_t groups = (a.vocab + a.w - 1) / a.w, lds = (kSortWaves + 1) * a.w * 4;
    if (wide)
        k_embed_sort<true><<<groups, 64 * kSortWaves, lds, s>>>(a);
    else
        k_embed_sort<false><<<groups, 64 * kSortWaves, lds, s>>>(a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (!a.nchunk) return hipSuccess;
    const uint32_t sums = (uint32_t)p.sumwgs;
    const hipError_t e = by_bool(p.chunk == 8, [&](auto few) {
        constexpr uint32_t C = few ? 8 : 16;
        switch (dtype) {
        case kF32: k_embed_sum<kF32, C><<<sums, 256, 0, s>>>(a); break;
        case kBF16: k_embed_sum<kBF16, C><<<sums, 256, 0, s>>>(a); break;
        default: k_embed_sum<kF16, C><<<sums, 256, 0, s>>>(a); break;
        }
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    // chunks of one launch, at most
    const uint32_t most = (uint32_t)(kMostThreads / 256 / a.njoin);
    for (a.first = 0; a.first < a.nchunk; a.first += most) {
        k_embed_join<<<std::min(most, a.nchunk - a.first) * a.njoin, 256, 0, s>>>(a);
        if (hipError_t j = hipGetLastError(); j != hipSuccess) return j;
    }
    return hipSuccess;
}

}  // namespace lags
