// Embeddings: y[t] = scale * table[ids[t]], and the table's gradient, whose row v
// is scale times the sum of dy over the tokens t with ids[t] = v, in the order of
// t.  An id outside [0, vocab) gives a row of zeros and adds to no gradient.
//
// Forward: a gather bound by memory; a thread has four tokens' vectors in flight.
// Gradient: the tokens are sorted by id (their order within an id kept), and
// the sorted list is cut into chunks of kChunk tokens, so that a frequent id is
// the work of many workgroups.  A chunk adds up each id's rows in registers; an
// id that lies within one chunk is written to the table's gradient, the others
// leave a sum for each chunk, which are then added up in the order of the chunks.
// No atomics on floats: results repeat bit for bit.
#include "lags_gn.h"
#include "lags_layer.h"

#include <algorithm>

namespace lags {
namespace {

// The id of token t; `none` (never below vocab) where it is outside the vocabulary.
constexpr uint32_t kNone = 0xffffffffu;
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

// Tokens sorted by id: order[], their ids keys[], and start[v], the first place
// of id v (start[vocab]: how many tokens have an id).  A workgroup owns a.w ids;
// its 16 waves each read a section of all tokens, count the ids of its range,
// and then place them: where an id's tokens of a section go follows from the
// counts, the place within 64 tokens from comparing ids across the wave.
//   16384 tokens of 50304 ids: see k_embed_sum
constexpr int kSortWaves = 16, kHeld = 16;
template <bool WIDE> __global__ __launch_bounds__(64 * kSortWaves) void k_embed_sort(EmbedArgs a)
{
    extern __shared__ uint32_t cnt[];               // [wave][a.w]
    __shared__ uint32_t sum[kSortWaves], low[kSortWaves];
    const uint32_t lo = blockIdx.x * a.w, w = min(a.w, a.vocab - lo);
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (uint32_t i = threadIdx.x; i < kSortWaves * a.w; i += 64 * kSortWaves) cnt[i] = 0;
    __syncthreads();
    const int64_t per = (a.tokens + 64 * kSortWaves - 1) / (64 * kSortWaves) * 64;
    const int64_t s0 = min(a.tokens, per * wave), s1 = min(a.tokens, s0 + per);
    uint32_t *mine = cnt + wave * a.w;
    uint32_t id[kHeld], below = 0;
    auto load = [&](int64_t s) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const int64_t t = s + k * 64 + lane;
            id[k] = t < s1 ? id_of<WIDE>(a, t) : kNone;
        }
    };
    for (int64_t s = s0; s < s1; s += 64 * kHeld) {
        load(s);
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            below += id[k] < lo;
            if (id[k] - lo < w) atomicAdd(mine + (id[k] - lo), 1u);
        }
    }
    for (int o = 32; o; o >>= 1) below += __shfl_xor(below, o);
    if (lane == 0) low[wave] = below;
    __syncthreads();
    // ids' totals, their exclusive sum over the range, and each wave's first place
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
        if (lo + i + 1 == a.vocab) a.start[a.vocab] = at + total;
        for (int k = 0; k < kSortWaves; ++k) {
            const uint32_t c = cnt[k * a.w + i];
            cnt[k * a.w + i] = at;
            at += c;
        }
    }
    __syncthreads();
    const int bits = 32 - __builtin_clz(a.w);
    for (int64_t s = s0; s < s1; s += 64 * kHeld) {
        if (s1 - s0 > 64 * kHeld) load(s);           // else they are still held
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const uint32_t key = id[k] - lo;
            const bool in = key < w;
            uint64_t same = __ballot(in);
            if (!same) continue;
            for (int b = 0; b < bits; ++b) {
                const uint64_t m = __ballot(key >> b & 1);
                same &= key >> b & 1 ? m : ~m;
            }
            if (in) {
                const int first = __builtin_ctzll(same);
                const uint32_t rank = __builtin_popcountll(same & ((1ull << lane) - 1));
                uint32_t place = 0;
                if ((int)lane == first) place = atomicAdd(mine + key, (uint32_t)__builtin_popcountll(same));
                place = __shfl(place, first) + rank;
                a.order[place] = (uint32_t)(s + k * 64 + lane);
                a.keys[place] = id[k];
            }
        }
    }
}

// Sums of one chunk's tokens for each id in it, and (not adding) zeros for ids
// without tokens.  2^tl lanes span a slab of a row's vectors, 64 of them at most; the
// workgroups after the chunks' take rows of the table.
constexpr uint32_t kChunk = 32, kAhead = 8, kZeroRows = 64;
template <int D> __global__ __launch_bounds__(256) void k_embed_sum(EmbedArgs a)
{
    constexpr int V = Elem<D>::V, E = Elem<D>::E;
    if (blockIdx.x >= a.sumwgs) {
        const uint32_t T = 1u << a.zl, v0 = (blockIdx.x - a.sumwgs) * kZeroRows;
        const f32x4_u4 zero = {0, 0, 0, 0};
        for (uint32_t v = v0 + (threadIdx.x >> a.zl); v < min(a.vocab, v0 + kZeroRows); v += 256 >> a.zl) {
            if (a.start[v] != a.start[v + 1]) continue;
            float *p = a.dtable + (size_t)v * a.cols;
            for (uint32_t c = (threadIdx.x & (T - 1)) * 4; c < a.cols; c += T * 4) {
                if (c + 4 <= a.cols)
                    *(f32x4_u4 *)(p + c) = zero;
                else
                    for (uint32_t j = c; j < a.cols; ++j) p[j] = 0;
            }
        }
        return;
    }
    const uint32_t T = 1u << a.tl;
    const uint64_t unit = (uint64_t)blockIdx.x * (256 >> a.tl) + (threadIdx.x >> a.tl);
    const uint32_t chunk = (uint32_t)(unit / a.nslab), slab = (uint32_t)(unit % a.nslab);
    const uint32_t c = (slab * T + (threadIdx.x & (T - 1))) * V;
    const int n = (int)a.cols - (int)c;
    const uint32_t total = a.start[a.vocab], p0 = chunk * kChunk;
    if (chunk >= a.nchunk || p0 >= total || n <= 0) return;
    const uint32_t p1 = min(p0 + kChunk, total);
    const uint32_t before = p0 ? a.keys[p0 - 1] : kNone, after = p1 < total ? a.keys[p1] : kNone;
    float acc[V] = {};
    uint32_t cur = a.keys[p0];
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
    for (uint32_t p = p0; p < p1; p += kAhead) {
        u32x4 v[kAhead];
        uint32_t key[kAhead];
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k) {
            const uint32_t q = min(p + k, p1 - 1);
            key[k] = a.keys[q];
            v[k] = load_vec<D>((const char *)a.dy + ((size_t)a.order[q] * a.lddy + c) * E, n);
        }
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k) {
            if (p + k >= p1) break;
            if (key[k] != cur) {
                leave(false);
                cur = key[k], first = false;
                for (int j = 0; j < V; ++j) acc[j] = 0;
            }
            float f[V];
            Elem<D>::unpack(v[k], f);
            for (int j = 0; j < V; ++j) acc[j] += f[j];
        }
    }
    leave(cur == after);
}

// The ids that began in a chunk and went on past it: their chunks' sums, four
// waves a run of them each.
__global__ __launch_bounds__(256) void k_embed_join(EmbedArgs a)
{
    __shared__ float4 sh[4][64];
    const uint32_t chunk = blockIdx.x / a.njoin, c = (blockIdx.x % a.njoin * 64 + (threadIdx.x & 63)) * 4;
    const uint32_t total = a.start[a.vocab], p0 = chunk * kChunk, p1 = p0 + kChunk;
    if (p1 >= total) return;
    const uint32_t v = a.keys[p1 - 1];
    if (a.keys[p1] != v || a.start[v] < p0) return;
    const uint32_t n = (a.start[v + 1] - 1) / kChunk - chunk + 1;       // chunks with this id: this one's second sum, the others' first
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
    // ids a workgroup of the sort: 256 workgroups if the counts of 16 waves then stay within 32 KiB
    p.w = (uint32_t)std::min<int64_t>(512, (vocab + 255) / 256);
    p.nchunk = (uint32_t)((tokens + kChunk - 1) / kChunk);
    const uint32_t V = 16 / elem_bytes(dtype);
    const uint64_t vecs = (cols + V - 1) / V;
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
    a.w = p.w, a.nchunk = p.nchunk, a.tl = p.tl, a.nslab = p.nslab, a.njoin = p.njoin;
    a.sumwgs = (uint32_t)p.sumwgs;
    a.zl = log2_up(((uint64_t)a.cols + 3) / 4, 2, 8);
    const uint32_t groups = (a.vocab + a.w - 1) / a.w, lds = kSortWaves * a.w * 4;
    if (wide)
        k_embed_sort<true><<<groups, 64 * kSortWaves, lds, s>>>(a);
    else
        k_embed_sort<false><<<groups, 64 * kSortWaves, lds, s>>>(a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const uint32_t zero = a.add ? 0 : (a.vocab + kZeroRows - 1) / kZeroRows;
    if (a.sumwgs + zero) {
        switch (dtype) {
        case kF32: k_embed_sum<kF32><<<a.sumwgs + zero, 256, 0, s>>>(a); break;
        case kBF16: k_embed_sum<kBF16><<<a.sumwgs + zero, 256, 0, s>>>(a); break;
        default: k_embed_sum<kF16><<<a.sumwgs + zero, 256, 0, s>>>(a); break;
        }
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    if (a.nchunk < 2) return hipSuccess;
    k_embed_join<<<(uint32_t)((uint64_t)a.nchunk * a.njoin), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace lags
