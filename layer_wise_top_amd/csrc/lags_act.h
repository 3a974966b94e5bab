// Shared by the activation operators (8-bit checkpoints, group normalisation,
// weight gradient): argument blocks, element types and the checkpoint format.
// Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

namespace lags {

enum : int { kF32 = 0, kBF16 = 1, kF16 = 2 };            // LAGS_F32, LAGS_BF16, LAGS_F16
enum : int { kActNone = 0, kActRelu = 1, kActSilu = 2 }; // LAGS_ACT_*
constexpr uint32_t kRun = 32;                            // columns that share a scale (LAGS_CKPT_RUN)

__host__ __device__ inline uint32_t elem_bytes(int dtype) { return dtype == kF32 ? 4 : 2; }

// Where a checkpoint of [rows, cols] keeps its parts.
struct CkptShape {
    int64_t rows;
    uint32_t cols, pitch, nrun;      // code bytes and scale bytes per row
};
inline CkptShape ckpt_shape(int64_t rows, int64_t cols)
{
    return {rows, (uint32_t)cols, (uint32_t)((cols + 15) / 16 * 16), (uint32_t)((cols + kRun - 1) / kRun)};
}
inline size_t ckpt_size(const CkptShape &s)
{
    return ((size_t)s.rows * (s.pitch + s.nrun) + 15) / 16 * 16;
}

struct PackArgs {
    CkptShape s;
    const void *src;                 // matrix (pack) or codes (unpack)
    void *dst;                       // codes (pack) or matrix (unpack)
    const uint8_t *rscale;           // unpack
    uint8_t *wscale;                 // pack
    int64_t ld;                      // elements between rows of the matrix
    uint32_t nvp;                    // 16-byte vectors a row, rounded up to whole runs
    uint32_t magic, shift;           // division by nvp
};

struct GnArgs {
    const void *x, *dy;
    void *y, *dx;
    int64_t ldx, lddy, ldy, lddx;
    const uint8_t *rcodes, *rscales; // checkpoint read (backward)
    uint8_t *wcodes, *wscales;       // checkpoint written (forward)
    const float *gamma, *beta;       // both null: 1 and 0
    float *mean, *rstd;              // forward: written where not null; backward: read
    float *dgamma, *dbeta;
    float *part;                     // workspace
    float eps, inv_cg;
    int act;
    uint32_t add;                    // dgamma, dbeta are added to
    uint32_t past;                   // y is stored past the caches
    uint32_t N, S, C, G, cg;         // samples, positions, channels, groups, channels per group
    uint32_t pitch, nrun;
    // geometry: a workgroup takes `w` channels (whole groups, whole runs) of
    // one sample; 2^tcl lanes span them, the others take rows
    uint32_t w, nslab, tcl;
    uint32_t nchunk, chunk;          // split form: row chunks a sample, rows each
    uint32_t nper, nparts;           // resident backward: samples a workgroup, rows of `part`
};

// One launch of the weight gradient.
struct WgradArgs {
    const void *dy;
    const uint8_t *codes, *scales;
    float *dw, *part;
    int64_t M, lddy;
    uint32_t O, C, pitch, nrun;
    uint32_t to, tc;                 // tiles over O and C
    uint32_t split;                  // slices of the rows
    int64_t rows_per;                // rows of a slice (a multiple of the k step)
    uint32_t add;
};

// Threads of one launch, at most: the runtime takes more and starts that number modulo 2^32.
constexpr uint64_t kMostThreads = 0xffffffffull;

int64_t pack_rows(const CkptShape &s, int dtype);    // rows of one launch, at most
hipError_t launch_pack(const PackArgs &a, int dtype, hipStream_t s);
hipError_t launch_unpack(const PackArgs &a, int dtype, hipStream_t s);

// Group normalisation: the plan chooses the form and the geometry for a shape.
struct GnPlan {
    bool resident;
    uint32_t threads, rows;          // threads a workgroup, register rows a thread
    uint32_t w, nslab, tcl, nchunk, chunk, nper, nparts;
};
constexpr uint32_t kSlabMax = 4096;  // channels a workgroup spans, at most
// .threads == 0: the shape is not supported
GnPlan gn_plan(int dtype, int act, bool backward, uint64_t N, uint64_t S, uint32_t C, uint32_t G);
size_t gn_part_floats(const GnPlan &p, bool backward, uint64_t N, uint32_t C, uint32_t G);
template <int D> hipError_t launch_gn_forward(const GnPlan &p, const GnArgs &a, hipStream_t s);
template <int D> hipError_t launch_gn_backward(const GnPlan &p, const GnArgs &a, hipStream_t s);
hipError_t launch_gn_forward(const GnPlan &p, const GnArgs &a, int dtype, hipStream_t s);
hipError_t launch_gn_backward(const GnPlan &p, const GnArgs &a, int dtype, hipStream_t s);
constexpr int kSweep = 4;          // rows a thread requests at a time (split form)

struct WgradPlan {
    uint32_t tile, to, tc, split;
    int64_t rows_per;
};
WgradPlan wgrad_plan(int dtype, int64_t M, int64_t O, int64_t C);
hipError_t launch_wgrad(const WgradPlan &p, WgradArgs a, int dtype, hipStream_t s);

// Dynamic LDS above 64 KiB has to be asked for.
inline hipError_t allow_lds(const void *kernel, size_t bytes)
{
    if (bytes <= 65536) return hipSuccess;
    return hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

#if defined(__HIPCC__)
// ---- device side: 16-byte vectors of any element type ----------------------
// Global vectors are only element-aligned: rows of odd pitch and slices start
// anywhere, and the hardware takes such accesses whole.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_u2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_u4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ inline float asf(uint32_t x) { return __builtin_bit_cast(float, x); }
__device__ inline uint32_t asu(float x) { return __builtin_bit_cast(uint32_t, x); }

template <int D> struct Elem;
template <> struct Elem<kF32> {
    static constexpr int E = 4, V = 4;
    __device__ static void unpack(u32x4 v, float (&f)[4])
    {
        for (int i = 0; i < 4; ++i) f[i] = asf(v[i]);
    }
    __device__ static u32x4 pack(const float (&f)[4])
    {
        return u32x4{asu(f[0]), asu(f[1]), asu(f[2]), asu(f[3])};
    }
    // largest magnitude of the vector, as fp32 bits (an infinity or NaN gives
    // 0x7f800000 or more)
    __device__ static uint32_t top(u32x4 v)
    {
        uint32_t m = 0;
        for (int i = 0; i < 4; ++i) m = max(m, v[i] & 0x7fffffffu);
        return m;
    }
};
template <> struct Elem<kBF16> {
    static constexpr int E = 2, V = 8;
    __device__ static void unpack(u32x4 v, float (&f)[8])
    {
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = asf(v[i] << 16);
            f[2 * i + 1] = asf(v[i] & 0xffff0000u);
        }
    }
    __device__ static u32x4 pack(const float (&f)[8])
    {
        typedef float f2 __attribute__((ext_vector_type(2)));
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        u32x4 r;
        for (int i = 0; i < 4; ++i)
            r[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{f[2 * i], f[2 * i + 1]}, b2));
        return r;
    }
    __device__ static uint32_t top(u32x4 v)
    {
        uint32_t lo = 0, hi = 0;
        for (int i = 0; i < 4; ++i) {
            lo = max(lo, v[i] & 0x7fffu);
            hi = max(hi, v[i] & 0x7fff0000u);
        }
        return max(lo << 16, hi);
    }
};
template <> struct Elem<kF16> {
    static constexpr int E = 2, V = 8;
    __device__ static void unpack(u32x4 v, float (&f)[8])
    {
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)v[i]);
            f[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(v[i] >> 16));
        }
    }
    // rounded to fp32 first, then to fp16: the compiler joins some conversions
    // with the operation before them, which rounds once, and which ones it joins
    // differs between kernels that are to agree bit for bit
    __device__ static u32x4 pack(const float (&f)[8])
    {
        u32x4 r;
        for (int i = 0; i < 4; ++i) {
            float a = f[2 * i], b = f[2 * i + 1];
            asm("" : "+v"(a), "+v"(b));
            r[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)a) |
                   (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)b) << 16;
        }
        return r;
    }
    __device__ static uint32_t top(u32x4 v)
    {
        uint32_t m = 0;                               // order of the bits is the order of the values
        for (int i = 0; i < 4; ++i) m = max(m, max(v[i] & 0x7fffu, v[i] >> 16 & 0x7fffu));
        return asu((float)__builtin_bit_cast(_Float16, (uint16_t)m)) & 0x7fffffffu;
    }
};

// `n` elements at p (n >= V: a whole vector; the rest reads as zero).
template <int D> __device__ inline u32x4 load_vec(const void *p, int n)
{
    constexpr int V = Elem<D>::V;
    if (n >= V) return *(const u32x4_u2 *)p;
    u32x4 r = {0, 0, 0, 0};
    for (int i = 0; i < V - 1; ++i)
        if (i < n) {
            if constexpr (Elem<D>::E == 4)
                r[i] = ((const uint32_t *)p)[i];
            else
                r[i / 2] |= (uint32_t)((const uint16_t *)p)[i] << (i % 2 * 16);
        }
    return r;
}
template <int D> __device__ inline void store_vec(void *p, u32x4 v, int n)
{
    constexpr int V = Elem<D>::V;
    if (n >= V) {
        *(u32x4_u2 *)p = v;
        return;
    }
    if (n <= 0) return;
    if constexpr (V == 8) {
        typedef uint32_t u32_u2 __attribute__((aligned(2)));
        typedef uint32_t u32x2_u2 __attribute__((ext_vector_type(2), aligned(2)));
        uint16_t *q = (uint16_t *)p;
        if (n & 4) {
            *(u32x2_u2 *)q = u32x2_u2{v[0], v[1]};
            q += 4, v[0] = v[2], v[1] = v[3];
        }
        if (n & 2) {
            *(u32_u2 *)q = v[0];
            q += 2, v[0] = v[1];
        }
        if (n & 1) *q = (uint16_t)v[0];
    } else {
        for (int i = 0; i < V - 1; ++i)
            if (i < n) ((uint32_t *)p)[i] = v[i];
    }
}

// A buffer descriptor for `left` bytes at p: reads past them give zeros, so a
// loop needs no branch between its loads.
__device__ inline __amdgpu_buffer_rsrc_t window(const void *p, int64_t left)
{
    const int n = left > 0x7ffffffc ? 0x7ffffffc : left < 0 ? 0 : (int)left;
    return __builtin_amdgcn_make_buffer_rsrc((void *)p, 0, n, 0x00020000);
}

// One column of vectors over `rows` rows of a matrix, through a window of
// them.  Values of columns past the window's width are whatever lies there;
// rows past its end read as zeros.  ODD: 16-bit rows that may start inside a
// word (odd pitch, odd slice): five words are read for a vector's four and
// shifted into place.
template <int D, bool ODD> struct Reader {
    __amdgpu_buffer_rsrc_t r;
    uint32_t at, pitch, rows;
    __device__ Reader(const void *base, int64_t row0, uint32_t n, int64_t ld, uint32_t c0, uint32_t w, uint32_t col)
    {
        constexpr int V = Elem<D>::V, E = Elem<D>::E;
        const char *p = (const char *)base + (row0 * ld + c0) * E;
        const uint32_t into = ODD ? (uint32_t)((uintptr_t)p & 3) : 0;
        // whole words: what a last one holds beside the last value is a column past the width or
        // (ODD) the next row's first, which load() drops
        r = window(p - into, n ? (((int64_t)(n - 1) * ld + w) * E + into + 3) & ~(int64_t)3 : 0);
        at = col * V < w ? into + col * V * E : 0x80000000u;       // idle lanes read nothing
        pitch = (uint32_t)(ld * E);
        rows = n;
    }
    __device__ u32x4 load(uint32_t row) const
    {
        const uint32_t o = at + row * pitch;
        if constexpr (!ODD) return __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0);
        u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, o & ~3u, 0, 0);
        const uint32_t e = __builtin_amdgcn_raw_buffer_load_b32(r, (o & ~3u) + 16, 0, 0), sh = (o & 2) * 8;
        for (int i = 0; i < 3; ++i) v[i] = __builtin_amdgcn_alignbit(v[i + 1], v[i], sh);
        v[3] = __builtin_amdgcn_alignbit(e, v[3], sh);
        return row < rows ? v : u32x4{0, 0, 0, 0};
    }
};

// ---- the 8-bit format ------------------------------------------------------
// Largest magnitude of a run of 32 columns from each lane's vector: the run is
// 4 (16-bit) or 8 (fp32) consecutive lanes, which must all be active.
template <int V> __device__ inline uint32_t run_top(uint32_t m)
{
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xb1, 0xf, 0xf, false));   // lanes 1 0 3 2
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4e, 0xf, 0xf, false));   // lanes 2 3 0 1
    if constexpr (V == 4)
        m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xf, 0xf, false));  // 7 - lane
    return m;
}
// Scale byte of a run: the step 2^(s - 127) is the power of two that takes
// the largest magnitude into [63.75, 127.5), so it rounds to at most 127 (adding
// 2^16 to the bits carries into the exponent exactly from 127.5/64 up); at
// least 2^-126, so steps are never subnormal.  255 where the run holds an
// infinity or NaN.
__device__ inline uint32_t run_scale(uint32_t top)
{
    if (top >= 0x7f800000u) return 255;
    return (uint32_t)max((int)((top + 0x10000u) >> 23) - 6, 1);
}
// Codes: round to nearest even of f / step, four to a word.  f / step is at
// most 127.5 in magnitude, so adding 1.5 * 2^23 in one rounded operation (the
// product by a power of two is exact, or far below 1/2) leaves the integer in
// the low byte.  A run marked 255 gets zeros: 0 times its step (infinity) is NaN.
template <int V> __device__ inline void run_codes(const float (&f)[V], uint32_t s, uint32_t (&q)[V / 4])
{
    const float inv = asf((254u - s) << 23);
    for (int i = 0; i < V / 4; ++i) {
        uint32_t b[4];
        for (int j = 0; j < 4; ++j) b[j] = asu(__builtin_fmaf(f[4 * i + j], inv, 12582912.0f));
        const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u);
        q[i] = s == 255 ? 0u : lo | hi << 16;
    }
}
// The four codes of a word as numbers.  One instruction each: written out
// because the compiler extracts the byte first where the word comes out of a
// vector.
__device__ inline void code_values(uint32_t q, float *f)
{
    asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0" : "=v"(f[0]) : "v"(q));
    asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1" : "=v"(f[1]) : "v"(q));
    asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2" : "=v"(f[2]) : "v"(q));
    asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3" : "=v"(f[3]) : "v"(q));
}
// The four values that a word of codes stands for.
__device__ inline void run_values(uint32_t q, float step, float *f)
{
    code_values(q, f);
    for (int j = 0; j < 4; ++j) f[j] *= step;
}
__device__ inline float run_step(uint32_t s) { return asf(s << 23); }

// ---- output ----------------------------------------------------------------
// One column of vectors over `rows` rows of a matrix.  Whole vectors go
// through a window that ends with the last row, so rows past it are dropped
// by the hardware; the last vector of a row of odd length, and rows that
// start inside a word (ODD), are stored piece by piece.
// `past`: whole vectors are stored past the caches.
template <int D, bool ODD> struct Writer {
    __amdgpu_buffer_rsrc_t r;
    char *p;
    uint32_t at, pitch, rows;
    int nv;
    bool past;
    __device__ Writer(void *base, int64_t row0, uint32_t n, int64_t ld, uint32_t c0, uint32_t w, uint32_t col,
                      bool past_caches = false)
        : past(past_caches)
    {
        constexpr int V = Elem<D>::V, E = Elem<D>::E;
        p = (char *)base + (row0 * ld + c0) * E;
        r = window(p, n ? ((int64_t)(n - 1) * ld + w) * E : 0);
        at = col * V * E, pitch = (uint32_t)(ld * E), rows = n;
        nv = (int)w - (int)(col * V);
    }
    __device__ void store(uint32_t row, u32x4 v) const
    {
        constexpr int V = Elem<D>::V;
        const uint32_t o = at + row * pitch;
        if constexpr (!ODD) {
            if (past)
                __builtin_amdgcn_raw_buffer_store_b128(v, r, nv >= V ? o : 0x80000000u, 0, 2);
            else
                __builtin_amdgcn_raw_buffer_store_b128(v, r, nv >= V ? o : 0x80000000u, 0, 0);
            if (nv > 0 && nv < V && row < rows) store_vec<D>(p + o, v, nv);
        } else {
            if (row < rows) store_vec<D>(p + o, v, nv);
        }
    }
};

// The same of a checkpoint: codes of whole vectors (a row's pad up to its
// pitch gets zeros), and a scale byte for each run.
template <int D> struct CodeWriter {
    __amdgpu_buffer_rsrc_t rq, rs;
    uint32_t q_at, s_at, pitch, nrun;
    __device__ CodeWriter(uint8_t *codes, uint8_t *scales, int64_t row0, uint32_t n, uint32_t pitch_, uint32_t nrun_,
                          uint32_t C, uint32_t c0, uint32_t w, uint32_t col)
    {
        constexpr uint32_t V = Elem<D>::V;
        pitch = pitch_, nrun = nrun_;
        rq = window(codes + row0 * pitch + c0, (int64_t)n * pitch - c0);
        rs = window(scales + row0 * nrun + c0 / kRun, (int64_t)n * nrun - c0 / kRun);
        const uint32_t c = c0 + col * V;
        // lanes past the slab write nothing unless they are past the last channel too
        q_at = c < pitch && (col * V < w || c >= C) ? col * V : 0x80000000u;
        s_at = col * V < w && c % kRun == 0 ? col * V / kRun : 0x80000000u;
    }
    // f: the values of `raw`, of which nv count
    __device__ void store(uint32_t row, u32x4 raw, float (&f)[Elem<D>::V], int nv) const
    {
        constexpr int V = Elem<D>::V;
        if (nv < V) {
            for (int j = 0; j < V; ++j) f[j] = j < nv ? f[j] : 0.0f;
            raw = Elem<D>::pack(f);
        }
        const uint32_t s = run_scale(run_top<V>(Elem<D>::top(raw)));
        uint32_t q[V / 4];
        run_codes<V>(f, s, q);
        if constexpr (V == 8)
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{q[0], q[V / 4 - 1]}, rq, q_at + row * pitch, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b32(q[0], rq, q_at + row * pitch, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b8((uint8_t)s, rs, s_at + row * nrun, 0, 0);
    }
};
#endif

}  // namespace lags
