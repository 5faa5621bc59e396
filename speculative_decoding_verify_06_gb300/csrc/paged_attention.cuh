// paged_attention.cuh -- what the attention kernels over paged caches share: the requests' row tiles and
// their split over CTAs, bounded waits, tcgen05 and paired fp32 helpers, and the checks of a call's arguments.
#pragma once

#include "paged.cuh"

namespace svd {

constexpr int kPaTile = 128;
constexpr int kPaTileUnits = kPaTile / kPgUnitPos;
constexpr float kPaOver = 15.f;      // a score this far above the reference moves it ...
constexpr float kPaUnder = 7.f;      // ... to this far below the new maximum
constexpr int kPaHeader = 256;       // workspace: status word, tile count, then the prefix sums

struct PaArgs {
    const __nv_bfloat16 *q;
    const int32_t *kv_len, *q_start, *table;
    const uint8_t *pages;
    void *out;
    uint32_t *status;
    int32_t *prefix;  // [R + 1] tiles before each request
    float *part;      // [2 CTAs][RP][128]
    float2 *part_ml;  // [2 CTAs][RP] (reference, sum)
    int64_t n_pages;
    int T, R, max_new, width, page, Hq, Hkv, G, stages;
    uint32_t upp_magic;  // ceil(2^32 / units of a page)
    uint32_t g_magic;    // x / G = x g_magic / 2^32 for x < 2^13, G > 1
    float c;          // scale * log2(e), over what K is scaled by
    int q_down;       // 8 bits: rows of queries are held over 2^q_down, which c makes up for
};

// ---- geometry shared by the two kernels -----------------------------------------------------
struct PaReq {
    int q0, n, base, len, rows;  // first token, tokens, position of token 0, positions, query rows
};
__device__ __forceinline__ PaReq pa_req(const PaArgs &A, int r) {
    PaReq x;
    const int a = A.q_start[r], b = A.q_start[r + 1], kv = A.kv_len[r];
    x.q0 = min(max(a, 0), A.T);
    const int n = max(b - a, 0);
    x.n = min(min(n, A.max_new), A.T - x.q0);
    x.base = kv - n;
    x.len = min(max(kv, 0), A.width * A.page);
    x.rows = x.n * A.G;
    return x;
}
// Tiles of row tile rt (one at least, so that every row gets written).
template <int RP>
__device__ __forceinline__ int pa_row_tiles(const PaArgs &A, const PaReq &x, int rt) {
    const int last = (min((rt + 1) * RP, x.rows) - 1) / A.G;
    const int see = min(x.base + last + 1, x.len);
    return max(1, (see + kPaTile - 1) / kPaTile);
}
template <int RP>
__device__ __forceinline__ int pa_head_tiles(const PaArgs &A, const PaReq &x) {
    int s = 0;
    for (int rt = 0; rt * RP < x.rows; ++rt) s += pa_row_tiles<RP>(A, x, rt);
    return s;
}
// CTA b's range of n tiles, and the CTA of tile u (G CTAs, those past n idle).
__device__ __forceinline__ int pa_lo(int n, int G, int b) {
    const int g = min(G, n);
    return b >= g ? n : (int)((int64_t)b * n / g);
}
__device__ __forceinline__ int pa_cta_of(int n, int G, int u) {
    const int g = min(G, n);
    return (int)((((int64_t)u + 1) * g - 1) / n);
}

// ---- tcgen05, TMEM, waits -------------------------------------------------------------------
constexpr uint32_t kPaPolls = 1u << 18;  // blocking polls, about a second
struct PaCtl {
    uint32_t stop;
    uint32_t limit;
    uint32_t *status;
};
__device__ __forceinline__ bool pa_stopped(const PaCtl *c) {
    return *reinterpret_cast<const volatile uint32_t *>(&c->stop) != 0u;
}
// Bounded wait; one that gives up stops the CTA (every later wait returns soon) and is recorded.
__device__ __forceinline__ bool pa_wait(uint32_t bar, uint32_t parity, PaCtl *c) {
    bool ok = mbar_poll(bar, parity, true);
    if (!ok) {
        const uint32_t limit = c->limit;
#pragma unroll 1
        for (uint32_t it = 0; it < limit; ++it) {
            ok = mbar_poll(bar, parity, true);
            if (ok || pa_stopped(c)) break;
        }
        if (!ok && !pa_stopped(c)) {
            *reinterpret_cast<volatile uint32_t *>(&c->stop) = 1u;
            atomicOr(c->status, 1u);
        }
    }
    return __all_sync(~0u, ok);  // one answer for the warp, which stays together
}
__device__ __forceinline__ void pa_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void pa_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void pa_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void pa_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void pa_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void pa_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// D[tmem] (+)= A[tmem] B[smem]^T, fp16 operands, fp32 accumulators.
__device__ __forceinline__ void pa_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; "
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void pa_st8(uint32_t t, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void pa_ld8(uint32_t t, float *f) {
    uint32_t *v = reinterpret_cast<uint32_t *>(f);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(t)
                 : "memory");
}
// Pairs of fp32.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pa_f2(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 pa_un2(f2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ f2 pa_fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 pa_add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 pa_mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint32_t pa_h2mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t pa_h2fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ float pa_ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pa_pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Nibbles moved to fraction bits 6..9 under the exponent of 16: 16 + c in each half, exactly.
__device__ __forceinline__ uint32_t pa_16plus(uint32_t moved) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(moved), "r"(0x03C003C0u), "r"(0x4C004C00u));
    return r;
}
// Ordered integers of floats (NaN above +inf), for a warp-wide maximum.
__device__ __forceinline__ int pa_order(float x) {
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float pa_unorder(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF)); }

// Shared-memory descriptors: Q, K-major with the 128-byte swizzle (rows of 64 fp16, 8-row groups
// 1024 bytes apart); P, row-major in positions (MN-major, no swizzle: 8 x 8 blocks of 16-byte lines
// of eight rows, the next eight positions 128 bytes on, the next eight rows 2048).
__device__ __forceinline__ uint64_t pa_desc_q(uint32_t a) {
    return (uint64_t)((a & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t pa_desc_p(uint32_t a) {
    return (uint64_t)((a & 0x3FFFFu) >> 4) | ((uint64_t)(128u >> 4) << 16) | ((uint64_t)(2048u >> 4) << 32) | (1ull << 46);
}

struct PaTileInfo {
    uint32_t mask;    // units present, one bit each
    int n_pos;        // positions of the request in the tile (may exceed 128)
    int tile;         // index along the cache
    uint32_t flags;   // 1 first, 2 last tile of the segment; segment ring entry above
};
struct PaSeg {
    int token0, head0, row0, rows;  // first token of the request, first query head, rows of the tile
    int base, len, slot;            // position of token 0; workspace slot, or -1: write the output
    int tok, off;                   // token of row 0, and row 0 among its heads
};

// Rows per tile: the fewest that hold a window's rows, 128 for longer ones (32 for fp32 outputs,
// whose sums live in registers beside the scores).
inline int pa_rows(int G, int max_new, bool f32) {
    const int64_t rows = (int64_t)G * max_new;
    return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 24 ? 24 : rows <= 32 || f32 ? 32 : rows <= 64 ? 64 : 128;
}
inline int pa_ctas(int rp, int sms) { return (rp <= 24 ? 2 : 1) * sms; }  // at most
inline size_t pa_prefix_bytes(int R) { return align_up(kPaHeader + ((size_t)R + 1) * 4, 256); }
// (sms is asked for once a call: the question costs a twentieth of a launch.)
inline size_t pa_ws_bytes(int Hq, int Hkv, int R, int max_new, int sms) {
    if (Hq < 1 || Hq > 4096 || Hkv < 1 || Hq % Hkv || R < 1 || R > SVD_PAGED_MAX_REQUESTS || max_new < 1 || sms < 1)
        return 0;
    // enough for every variant up to the one that max_new takes, so that shorter windows fit too
    const int most = pa_rows(Hq / Hkv, max_new, false);
    size_t parts = 0;
    for (int rp : {8, 16, 24, 32, 64, 128})
        if (rp <= most && parts < (size_t)pa_ctas(rp, sms) * rp) parts = (size_t)pa_ctas(rp, sms) * rp;
    return pa_prefix_bytes(R) + 2 * parts * (kPgDim + 2) * 4;
}

// The arguments of an attention call, checked and laid out; *rp: the rows of its row tiles.  (Nothing is set for T = 0.)
inline int pa_arguments(PaArgs *args, int *rp, const uint16_t *q, int T, const int32_t *kv_len, const int32_t *q_start, int R,
                        int max_new, const int32_t *table, int width, const void *pages, int page, int64_t n_pages, int Hq,
                        int Hkv, float scale, void *out, int out_dtype, void *ws, size_t ws_bytes, int sms) {
    if (!q || !kv_len || !q_start || !table || !pages || !out || !aligned16(q) || !aligned16(pages) ||
        !aligned16(out) || !aligned16(ws) || (out_dtype != SVD_F32 && out_dtype != SVD_BF16))
        return SVD_ERR_INVALID_ARG;
    if (T < 0 || R < 1 || R > SVD_PAGED_MAX_REQUESTS || max_new < 1 || max_new > 1 << 20 || width < 1 ||
        !pg_pool_ok(Hkv, page, n_pages) || (int64_t)width * page > INT32_MAX - kPaTile || Hq < 1 || Hq > 4096 ||
        Hq % Hkv || (int64_t)T * Hq > INT32_MAX || !(scale > 0.f) || scale > 3.4e38f)
        return SVD_ERR_INVALID_ARG;
    if (!ws || ws_bytes < pa_ws_bytes(Hq, Hkv, R, max_new, sms)) return SVD_ERR_WORKSPACE;
    if (T == 0) return SVD_OK;
    const int G = Hq / Hkv, rows_tile = pa_rows(G, max_new, out_dtype == SVD_F32);
    // the tiles of the largest call that these arguments allow are counted in 31 bits
    const int64_t row_tiles = ((int64_t)G * (max_new < T ? max_new : T) + rows_tile - 1) / rows_tile;
    const double most = (double)R * Hkv * row_tiles * (((int64_t)width * page + kPaTile - 1) / kPaTile);
    if (most > 2.0e9) return SVD_ERR_UNSUPPORTED;
    uint8_t *const w = (uint8_t *)ws + pa_prefix_bytes(R);
    PaArgs A = {};
    A.q = (const __nv_bfloat16 *)q;
    A.kv_len = kv_len;
    A.q_start = q_start;
    A.table = table;
    A.pages = (const uint8_t *)pages;
    A.out = out;
    A.status = (uint32_t *)ws;
    A.prefix = (int32_t *)((uint8_t *)ws + kPaHeader);
    A.part = (float *)w;
    A.part_ml = (float2 *)(w + (size_t)2 * pa_ctas(rows_tile, sms) * rows_tile * kPgDim * 4);
    A.n_pages = n_pages;
    A.T = T;
    A.R = R;
    A.max_new = max_new;
    A.width = width;
    A.page = page;
    A.upp_magic = (uint32_t)(((1ull << 32) + page / kPgUnitPos - 1) / (page / kPgUnitPos));
    A.Hq = Hq;
    A.Hkv = Hkv;
    A.G = G;
    A.g_magic = (uint32_t)(((1ull << 32) + G - 1) / G);
    A.c = scale * 1.4426950408889634f;
    *args = A;
    *rp = rows_tile;
    return SVD_OK;
}

}  // namespace svd
