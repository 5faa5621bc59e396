// paged_cache.cu -- the write side of the paged 4-bit cache: block tables and slot maps built from
// request lengths, rotary positions with several axes joined to the append, and the read-back.
//
// "100 tokens per second ..." ("Why a hiring company is writing this"): several sequences share a
// pass; "How speculative decoding gets past a per-token wall": each window keeps only its accepted
// prefix, so the lengths change on the GPU after every pass and the tables follow them there.
#include "paged.cuh"

#include <math.h>

namespace svd {

// ---- block tables and slot maps ------------------------------------------------------------
// Per request: keep = held - window + emitted positions stay, size = keep + new are wanted,
// p0 = ceil(held / page) pages are held and p1 = ceil(size / page) wanted.  Pages p1..p0-1 go back
// to the stack of free pages, then the missing ones are taken from its top; both in (request,
// page) order, so places follow from prefix sums over the requests.
//
// One launch: every CTA computes the sums over all requests for itself (up to 4096 of them, 16
// bytes each, from L2), keeps them in shared memory, and then fills its share of the outputs, each
// element a function of the sums and the inputs alone (no CTA waits for another).
constexpr int kTbThreads = 512;
constexpr int kTbWarps = kTbThreads / 32;
constexpr int kTbChunk = 1024;  // outputs per work item

struct TbArgs {
    const int32_t *held, *window, *emitted, *n_new, *table, *free_ids, *n_free;
    int32_t *table_out, *free_out, *n_free_out, *kv_len, *q_start, *positions, *status;
    int64_t *slots;
    int R, page, width, n_pages, tokens;
};

// Inclusive sum over the block of one 64-bit value per thread; *total gets the block's sum.
__device__ __forceinline__ unsigned long long tb_scan(unsigned long long v, unsigned long long *total,
                                                      unsigned long long *s_w) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long u = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();  // s_w may still be read from the scan before
    if (lane == 31) s_w[warp] = v;
    __syncthreads();
    unsigned long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kTbWarps; ++w) {
        const unsigned long long x = s_w[w];
        if (w < warp) before += x;
        all += x;
    }
    *total = all;
    return v + before;
}

// The last index r in [0, n) with a[r] <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int tb_last_le(const int *a, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kTbThreads) paged_tables_kernel(const TbArgs A) {
    extern __shared__ int sm[];
    __shared__ unsigned long long s_w[kTbWarps];
    const int R = A.R, tid = threadIdx.x;
    int *const s_keep = sm, *const s_p0 = sm + R, *const s_q1 = sm + 2 * R, *const s_take = sm + 3 * R;
    int *const s_give = sm + 4 * R, *const s_tok = sm + 5 * R;  // exclusive sums
    uint8_t *const s_st = reinterpret_cast<uint8_t *>(sm + 6 * R);
    griddep_wait();

    // What is asked for, and which requests are refused outright.
    unsigned long long tok_sum = 0, page_sum = 0, total;
    for (int base = 0; base < R; base += kTbThreads) {
        const int r = base + tid;
        long long keep = 0, add = 0, p0 = 0, p1 = 0;
        uint32_t st = 0;
        if (r < R) {
            const long long held = A.held[r], n = A.n_new[r];
            const long long win = A.window ? A.window[r] : 0, emi = A.window ? A.emitted[r] : 0;
            keep = held - win + emi;
            p0 = (held + A.page - 1) / A.page;
            p1 = (keep + n + A.page - 1) / A.page;
            add = n;
            if (win < 0 || emi < 0 || emi > win || win > held || n < 0 || p0 > A.width || p1 > A.width)
                st = SVD_ST_BAD_REQUEST;
        }
        const unsigned long long ask = st ? 0ull : (unsigned long long)add;
        const unsigned long long upto = tok_sum + tb_scan(ask, &total, s_w);
        tok_sum += total;
        if (!st && ask > 0 && upto > (unsigned long long)A.tokens) st = SVD_ST_NO_TOKENS;
        if (st) p1 = p0;
        const unsigned long long take = p1 > p0 ? p1 - p0 : 0, give = p0 > p1 ? p0 - p1 : 0;
        const unsigned long long pg = (give << 32) | take;
        const unsigned long long sum = page_sum + tb_scan(pg, &total, s_w);
        page_sum += total;
        if (r < R) {
            s_keep[r] = (int)keep;
            s_p0[r] = st == SVD_ST_BAD_REQUEST ? 0 : (int)p0;
            s_q1[r] = st == SVD_ST_BAD_REQUEST ? 0 : (int)p1;
            s_take[r] = (int)((uint32_t)sum - (uint32_t)take);
            s_give[r] = (int)((uint32_t)(sum >> 32) - (uint32_t)give);
            s_st[r] = (uint8_t)st;
        }
    }
    __syncthreads();
    const int n_free = min(max(*A.n_free, 0), A.n_pages);
    const int top = n_free + (int)(page_sum >> 32);
    // What is granted: a request that takes pages gets them if all that was asked before it and
    // its own fits.
    unsigned long long got = 0, took = 0;
    for (int base = 0; base < R; base += kTbThreads) {
        const int r = base + tid;
        int grant = 0, take = 0;
        if (r < R) {
            uint32_t st = s_st[r];
            take = max(s_q1[r] - s_p0[r], 0);
            if (take > 0 && s_take[r] + take > top) {
                st = SVD_ST_NO_PAGES;
                s_st[r] = (uint8_t)st;
                s_q1[r] = s_p0[r];
                take = 0;
            }
            if (!st) grant = A.n_new[r];
        }
        const unsigned long long v = ((unsigned long long)(uint32_t)take << 32) | (uint32_t)grant;
        const unsigned long long sum = tb_scan(v, &total, s_w);
        if (r < R) s_tok[r] = (int)((uint32_t)got + (uint32_t)sum) - grant;
        got += (uint32_t)total;
        took += total >> 32;
    }
    __syncthreads();
    const int n_tok = (int)got, left = top - (int)took;

    // The stack: the free ids, then the pages given back.
    auto stack = [&](int i) -> int {
        if (i < n_free) return A.free_ids[i];
        const int j = i - n_free, r = tb_last_le(s_give, R, j);
        return A.table[(int64_t)r * A.width + s_q1[r] + j - s_give[r]];
    };
    auto entry = [&](int r, int col) -> int {
        const int p0 = s_p0[r], q1 = s_q1[r];
        if (col < min(p0, q1) || s_st[r] == SVD_ST_BAD_REQUEST) return A.table[(int64_t)r * A.width + col];
        return col < q1 ? stack(top - 1 - s_take[r] - (col - p0)) : -1;
    };

    if (blockIdx.x == 0) {
        for (int r = tid; r < R; r += kTbThreads) {
            const uint32_t st = s_st[r];
            A.kv_len[r] = st == SVD_ST_BAD_REQUEST ? 0 : st ? s_keep[r] : s_keep[r] + A.n_new[r];
            A.q_start[r] = s_tok[r];
            A.status[r] = (int)st;
        }
        if (tid == 0) {
            A.q_start[R] = n_tok;
            *A.n_free_out = left;
        }
    }
    const int row_items = (A.width + kTbChunk - 1) / kTbChunk;
    const int64_t t_items = (int64_t)R * row_items;
    const int f_items = (A.n_pages + kTbChunk - 1) / kTbChunk, s_items = (A.tokens + kTbChunk - 1) / kTbChunk;
    for (int64_t it = blockIdx.x; it < t_items + f_items + s_items; it += gridDim.x) {
        if (it < t_items) {
            const int r = (int)(it / row_items), c0 = (int)(it % row_items) * kTbChunk;
            const int c1 = min(c0 + kTbChunk, A.width);
            for (int c = c0 + tid; c < c1; c += kTbThreads) A.table_out[(int64_t)r * A.width + c] = entry(r, c);
        } else if (it < t_items + f_items) {
            const int i0 = (int)(it - t_items) * kTbChunk, i1 = min(i0 + kTbChunk, A.n_pages);
            for (int i = i0 + tid; i < i1; i += kTbThreads) A.free_out[i] = i < left ? stack(i) : -1;
        } else {
            const int i0 = (int)(it - t_items - f_items) * kTbChunk, i1 = min(i0 + kTbChunk, A.tokens);
            for (int i = i0 + tid; i < i1; i += kTbThreads) {
                int64_t slot = -1;
                int pos = -1;
                if (i < n_tok) {
                    const int r = tb_last_le(s_tok, R, i);
                    pos = s_keep[r] + i - s_tok[r];
                    slot = (int64_t)entry(r, pos / A.page) * A.page + pos % A.page;
                }
                A.slots[i] = slot;
                A.positions[i] = pos;
            }
        }
    }
}

int paged_tables(const int32_t *held, const int32_t *window, const int32_t *emitted, const int32_t *n_new,
                 int R, int page, const int32_t *table, int width, const int32_t *free_ids,
                 const int32_t *n_free, int64_t n_pages, int32_t *table_out, int32_t *free_out,
                 int32_t *n_free_out, int32_t *kv_len, int32_t *q_start, int64_t *slots,
                 int32_t *positions, int64_t tokens, int32_t *status, cudaStream_t stream) {
    if (!held || !n_new || !table || !free_ids || !n_free || !table_out || !free_out || !n_free_out ||
        !kv_len || !q_start || !slots || !positions || !status || (!window) != (!emitted))
        return SVD_ERR_INVALID_ARG;
    if (R < 1 || R > SVD_PAGED_MAX_REQUESTS || !pg_page_size_ok(page) || width < 1 ||
        (int64_t)width * page > INT32_MAX || (int64_t)width * R > INT32_MAX || n_pages < 1 ||
        n_pages > (int64_t)1 << 30 || tokens < 1 || tokens > (int64_t)1 << 30)
        return SVD_ERR_INVALID_ARG;
    if (table_out == table || free_out == free_ids || n_free_out == n_free) return SVD_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms < 1) return SVD_ERR_CUDA;
    const TbArgs A = {held, window, emitted, n_new, table, free_ids, n_free, table_out, free_out, n_free_out,
                      kv_len, q_start, positions, status, slots, R, page, width, (int)n_pages, (int)tokens};
    const size_t smem = (size_t)R * 25 + 8;
    if (smem > 48 * 1024)
        SVD_CUDA_TRY(cudaFuncSetAttribute(paged_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          (int)smem));
    auto items = [](int64_t n) { return (n + kTbChunk - 1) / kTbChunk; };
    const int64_t work = (int64_t)R * items(width) + items(n_pages) + items(tokens);
    const int grid = (int)(work < 2 * sms ? work : 2 * sms);
    SVD_CUDA_TRY(launch(paged_tables_kernel, dim3(grid), dim3(kTbThreads), smem, stream, true, A));
    return SVD_OK;
}

// ---- rotary positions and the append -------------------------------------------------------
// q, k: (y_a, y_b) = (x_a cos - x_b sin, x_b cos + x_a sin) for every pair i of dimensions, the
// angle being position[axis(i)] * inv_freq(i); q is rounded to bf16, k and v to 4 bits per block of
// 32.
//
// Angles.  position * inv_freq reaches 10^6 radians; reduced in fp32 it would be off by 0.06.
// The host turns each frequency into turns per position as a 64-bit fraction, so that one 64-bit
// integer product gives the angle modulo a turn to 2^-33 turns for any 31-bit position, and cos
// and sin of the remaining eighth of a turn are cheap in fp32 (absolute error below 2^-22).
//
// Codes.  A key next to the border of two codes must get the code that exact arithmetic gives, or
// the cache would depend on how the angle was rounded.  Each fp32 key carries an error bound (0 for
// values and for unrotated dimensions); when a block's scale or one of its codes could change
// within it, the block's eight lanes redo it in fp64 with fp64 angles (about one block in 10^3).
// Borders are (n - 8.5) d, exact in fp32 because d has eight significant bits, so a code is
// settled by comparing against them and no division is rounded.
constexpr int kApWarps = 8;

struct RopeArgs {
    uint64_t phase[SVD_ROPE_MAX_PAIRS];  // turns per position, as a fraction of 2^64
    double inv[SVD_ROPE_MAX_PAIRS];      // radians per position (the fp64 path)
    uint8_t axis[SVD_ROPE_MAX_PAIRS];
    int pairs, interleaved;
};
struct ApArgs {
    const void *qkv;
    int64_t ld;
    const int32_t *positions;
    int64_t positions_ld;
    const int64_t *slots;
    uint8_t *pages;
    __nv_bfloat16 *q;
    int32_t *status;
    int64_t n_slots;
    int T, Hq, Hkv, page;
    RopeArgs rope;
};

__device__ __forceinline__ void ap_load4(const float *p, float x[4]) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void ap_load4(const __nv_bfloat16 *p, float x[4]) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xFFFF0000u);
}

// d = round8(m / -8) as fp16 bits.
__device__ __forceinline__ uint16_t ap_scale(float m) {
    return __half_as_ushort(__float2half_rn(__bfloat162float(__float2bfloat16_rn(m * -0.125f))));
}
__device__ __forceinline__ uint16_t ap_scale(double m) {
    unsigned long long u = (unsigned long long)__double_as_longlong(m * -0.125);
    u += 0xFFFFFFFFFFFull + ((u >> 45) & 1ull);  // to nearest even at seven fraction bits
    u &= ~0x1FFFFFFFFFFFull;
    return __half_as_ushort(__float2half_rn((float)__longlong_as_double((long long)u)));
}

// The value of largest magnitude among the block's eight lanes (the lowest dimension on ties).
template <typename F>
__device__ __forceinline__ F ap_extreme(const F y[4], int lane, uint32_t mask) {
    F m = y[0];
    int at = 0;
#pragma unroll
    for (int j = 1; j < 4; ++j)
        if (fabs(y[j]) > fabs(m)) { m = y[j]; at = j; }
    at += (lane & 7) * 4;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        const F om = __shfl_xor_sync(mask, m, o);
        const int oa = __shfl_xor_sync(mask, at, o);
        if (fabs(om) > fabs(m) || (fabs(om) == fabs(m) && oa < at)) { m = om; at = oa; }
    }
    return m;
}

// The four codes of a lane from keys in fp64, and the block's scale.
__device__ __noinline__ uint32_t ap_block_f64(const ApArgs &A, int t, int d0, const float *xa4,
                                              const float *xb4, int lane, uint32_t mask, uint16_t *scale) {
    double y[4];
    const int pairs = A.rope.pairs;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int d = d0 + j;
        double v = xa4[j];
        if (d < 2 * pairs) {
            const bool second = A.rope.interleaved ? (d & 1) : d >= pairs;
            const int i = A.rope.interleaved ? d >> 1 : second ? d - pairs : d;
            double s, c;
            sincos((double)A.positions[A.rope.axis[i] * A.positions_ld + t] * A.rope.inv[i], &s, &c);
            const double own = __dmul_rn(v, c), other = __dmul_rn((double)xb4[j], s);
            v = second ? __dadd_rn(own, other) : __dsub_rn(own, other);
        }
        y[j] = fmin(fmax(v, -kPgMaxAbs), kPgMaxAbs);
    }
    const uint16_t db = ap_scale(ap_extreme(y, lane, mask));
    const double d = (double)__half2float(__ushort_as_half(db));
    uint32_t codes = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const double c = d != 0.0 ? floor(y[j] / d + 8.5) : 8.0;
        codes |= (uint32_t)fmin(fmax(c, 0.0), 15.0) << (8 * j);
    }
    *scale = db;
    return codes;
}

template <typename T>
__global__ void __launch_bounds__(kApWarps * 32) paged_append_kernel(const __grid_constant__ ApArgs A) {
    __shared__ float2 s_cs[SVD_ROPE_MAX_PAIRS];
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pairs = A.rope.pairs;
    griddep_wait();
    if ((int)threadIdx.x < pairs) {
        const int i = threadIdx.x;
        const int64_t pos = A.positions[A.rope.axis[i] * A.positions_ld + t];
        const uint64_t ph = (uint64_t)pos * A.rope.phase[i];
        const uint64_t quad = (ph + (1ull << 61)) >> 62;  // nearest quarter turn
        const float r = __ll2float_rn((long long)(ph - (quad << 62))) * 0x1p-63f;  // half turns
        float s, c;
        sincospif(r, &s, &c);
        if (quad & 1) { const float x = s; s = c; c = -x; }
        if (quad & 2) { s = -s; c = -c; }
        s_cs[i] = make_float2(c, s);
    }
    __syncthreads();
    const int head = blockIdx.y * kApWarps + warp;
    if (head >= A.Hq + 2 * A.Hkv) return;
    const T *const row = reinterpret_cast<const T *>(A.qkv) + t * A.ld + (int64_t)head * kPgDim;
    const int d0 = 4 * lane;
    const bool is_v = head >= A.Hq + A.Hkv;
    float x[4], xb[4] = {0.f, 0.f, 0.f, 0.f}, y[4], err[4] = {0.f, 0.f, 0.f, 0.f};
    ap_load4(row + d0, x);
    if (!is_v && d0 < 2 * pairs) {  // pairs is a multiple of four: a lane's dimensions turn alike
        float2 cs[4];
        bool second[4];
        if (A.rope.interleaved) {
            const float2 c0 = s_cs[2 * lane], c1 = s_cs[2 * lane + 1];
            cs[0] = cs[1] = c0;
            cs[2] = cs[3] = c1;
            xb[0] = x[1]; xb[1] = x[0]; xb[2] = x[3]; xb[3] = x[2];
            second[0] = second[2] = false;
            second[1] = second[3] = true;
        } else {
            const bool up = d0 >= pairs;
            ap_load4(row + (up ? d0 - pairs : d0 + pairs), xb);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                cs[j] = s_cs[(up ? d0 - pairs : d0) + j];
                second[j] = up;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float own = __fmul_rn(x[j], cs[j].x), other = __fmul_rn(xb[j], cs[j].y);
            y[j] = second[j] ? __fadd_rn(own, other) : __fsub_rn(own, other);
            err[j] = (fabsf(x[j]) + fabsf(xb[j])) * 0x1p-20f;  // angle, products and sum
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = x[j];
    }
    if (head < A.Hq) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(y[0], y[1]), hi = __floats2bfloat162_rn(y[2], y[3]);
        uint2 o;
        o.x = reinterpret_cast<const uint32_t &>(lo);
        o.y = reinterpret_cast<const uint32_t &>(hi);
        *reinterpret_cast<uint2 *>(A.q + ((int64_t)t * A.Hq + head) * kPgDim + d0) = o;
        return;
    }
    const int64_t slot = A.slots[t];
    if (slot < 0 || slot >= A.n_slots) {
        if (slot >= 0 && A.status && lane == 0) atomicOr(A.status + t, SVD_ST_BAD_SLOT);
        return;
    }
    // What is not finite is noted and stored as 0 or the largest magnitude: a cache byte never
    // stands for a NaN that a masked position could spread.
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (!(fabsf(y[j]) <= 3.4028235e38f)) {
            odd = true;
            if (y[j] != y[j]) y[j] = 0.f;
            if (x[j] != x[j] || fabsf(x[j]) > 3.4028235e38f || xb[j] != xb[j] || fabsf(xb[j]) > 3.4028235e38f)
                err[j] = 0.f;
        }
        if (fabsf(y[j]) > (float)kPgMaxAbs && fabsf(y[j]) - err[j] > (float)kPgMaxAbs) err[j] = 0.f;
        y[j] = fminf(fmaxf(y[j], -(float)kPgMaxAbs), (float)kPgMaxAbs);
    }
    const uint32_t bad = __ballot_sync(~0u, odd);
    if (bad && A.status && lane == 0) atomicOr(A.status + t, SVD_ST_NONFINITE);

    // The block's scale, and whether another one lies within the keys' error.
    const uint32_t grp = 0xFFu << (lane & 24);
    float e = fmaxf(fmaxf(err[0], err[1]), fmaxf(err[2], err[3]));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) e = fmaxf(e, __shfl_xor_sync(~0u, e, o));
    const float m = ap_extreme(y, lane, ~0u);
    uint16_t db = ap_scale(m);
    const float d = __half2float(__ushort_as_half(db));
    bool unsure = false;
    if (e > 0.f) {
#pragma unroll
        for (int j = 0; j < 4; ++j)  // a value of the other sign that could be the larger one
            unsure |= (y[j] < 0.f) != (m < 0.f) && fabsf(y[j]) + 2.f * e >= fabsf(m);
        // m within its error of the border of two scales, or a scale among fp16's subnormals
        const float lo = __bfloat162float(__float2bfloat16_rn(fabsf(m) - e));
        const float hi = __bfloat162float(__float2bfloat16_rn(fabsf(m) + e));
        unsure |= lo != hi || fabsf(d) < 0x1p-14f;
    }
    uint32_t codes = 0x08080808u;
    if (d != 0.f) {
        const float inv = 1.f / d;
        const float s = d < 0.f ? -1.f : 1.f;
        codes = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            int n = (int)fminf(fmaxf(floorf(y[j] * inv + 8.5f), 0.f), 15.f);
            // below the border (n - 8.5) d, or on or above the next one (signs taken out by s)
            if (n > 0 && s * y[j] < s * ((float)n - 8.5f) * d) --n;
            else if (n < 15 && s * y[j] >= s * ((float)n - 7.5f) * d) ++n;
            if (err[j] > 0.f) {
                unsure |= n > 0 && fabsf(y[j] - ((float)n - 8.5f) * d) <= err[j];
                unsure |= n < 15 && fabsf(y[j] - ((float)n - 7.5f) * d) <= err[j];
            }
            codes |= (uint32_t)n << (8 * j);
        }
    }
    if (__ballot_sync(~0u, unsure && !bad) & grp) codes = ap_block_f64(A, t, d0, x, xb, lane, grp, &db);
    __syncwarp();

    const int64_t page = slot / A.page;
    const int off = (int)(slot - page * A.page), pos = off & 15;
    const int kvh = head - A.Hq - (is_v ? A.Hkv : 0);
    uint8_t *const unit =
        A.pages + ((page * A.Hkv + kvh) * (A.page >> 4) + (off >> 4)) * (int64_t)kPgUnitBytes;
    if (!is_v) {
        const uint32_t c2 = codes | (codes >> 4);  // nibbles of dims 0, 1 in byte 0, of 2, 3 in byte 2
        const uint16_t two = (uint16_t)((c2 & 0xFFu) | ((c2 >> 8) & 0xFF00u));
        *reinterpret_cast<uint16_t *>(unit + (lane >> 3) * 256 + pos * 16 + (lane & 7) * 2) = two;
        if ((lane & 7) == 0) *reinterpret_cast<uint16_t *>(unit + kPgKScales + pos * 8 + (lane >> 3) * 2) = db;
    } else {
        const uint32_t hi = __shfl_down_sync(~0u, codes, 16);  // dims + 64
        if (lane < 16) {
            const uint32_t both = codes | (hi << 4);
            uint8_t *const v = unit + kPgVCodes + d0 * 16 + pg_v_byte(pos);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j * 16] = (uint8_t)(both >> (8 * j));
        }
        if ((lane & 7) == 0) *reinterpret_cast<uint16_t *>(unit + kPgVScales + (lane >> 3) * 32 + pos * 2) = db;
    }
}

// Turns per position of a frequency in radians, as a fraction of 2^64 modulo a turn:
// |inv| = m 2^e with a 53-bit m, times 1 / (2 pi) to 2^-128, in integers.
static uint64_t rope_phase(double inv) {
    const uint64_t c_hi = 0x28BE60DB9391054Aull, c_lo = 0x7F09D5F47D4D3770ull;
    int e;
    const uint64_t m = (uint64_t)ldexp(frexp(fabs(inv), &e), 53);
    e -= 53;
    const unsigned __int128 lo = (unsigned __int128)m * c_lo;
    const unsigned __int128 hi = (unsigned __int128)m * c_hi + (uint64_t)(lo >> 64);
    const uint64_t w0 = (uint64_t)lo, w1 = (uint64_t)hi, w2 = (uint64_t)(hi >> 64);  // w2:w1:w0 / 2^128
    // times 2^e: the 64 bits from bit 64 - e on
    const uint64_t w[3] = {w0, w1, w2};
    const int k = (64 - e) >> 6, b = (64 - e) & 63;  // |inv| < 2^32, so e <= -21
    auto at = [&](int i) -> uint64_t { return i < 3 ? w[i] : 0; };
    uint64_t out = b ? (at(k) >> b) | (at(k + 1) << (64 - b)) : at(k);
    out += ((b ? at(k) >> (b - 1) : at(k - 1) >> 63) & 1);  // to nearest
    return inv < 0 ? 0 - out : out;
}

int paged_append(const void *qkv, int dtype, int64_t ld, int T, int Hq, int Hkv, const svd_rope *rope,
                 const int32_t *positions, int64_t positions_ld, const int64_t *slots, void *pages,
                 int page, int64_t n_pages, void *q, int32_t *status, cudaStream_t stream) {
    if (!qkv || !slots || !pages || (dtype != SVD_F32 && dtype != SVD_BF16) || T < 0 || Hq < 0 ||
        Hq > 4096 || !pg_pool_ok(Hkv, page, n_pages) || (Hq > 0 && !q))
        return SVD_ERR_INVALID_ARG;
    const int64_t heads = (int64_t)Hq + 2 * Hkv;
    const int lane_bytes = dtype == SVD_F32 ? 16 : 8;
    if (!aligned16(qkv) || !aligned16(pages) || !aligned16(q) || ld < heads * kPgDim ||
        (ld * (lane_bytes / 4)) % lane_bytes != 0)
        return SVD_ERR_INVALID_ARG;
    ApArgs A = {qkv, ld, positions, positions_ld, slots, (uint8_t *)pages, (__nv_bfloat16 *)q, status,
                n_pages * page, T, Hq, Hkv, page, {}};
    if (rope) {
        const svd_rope &r = *rope;
        if (!positions || r.n_pairs < 4 || r.n_pairs > SVD_ROPE_MAX_PAIRS || r.n_pairs % 4 || r.n_axes < 1 ||
            r.n_axes > SVD_ROPE_MAX_AXES || (r.n_axes > 1 && positions_ld < T))
            return SVD_ERR_INVALID_ARG;
        A.rope.pairs = r.n_pairs;
        A.rope.interleaved = r.interleaved != 0;
        for (int i = 0; i < r.n_pairs; ++i) {
            if (!(fabs(r.inv_freq[i]) < 4294967296.0) || r.axis[i] >= r.n_axes) return SVD_ERR_INVALID_ARG;
            A.rope.inv[i] = r.inv_freq[i];
            A.rope.phase[i] = rope_phase(r.inv_freq[i]);
            A.rope.axis[i] = r.axis[i];
        }
    }
    if (T == 0) return SVD_OK;
    const dim3 grid((unsigned)T, (unsigned)((heads + kApWarps - 1) / kApWarps));
    if (dtype == SVD_F32)
        SVD_CUDA_TRY(launch(paged_append_kernel<float>, grid, dim3(kApWarps * 32), 0, stream, true, A));
    else
        SVD_CUDA_TRY(launch(paged_append_kernel<__nv_bfloat16>, grid, dim3(kApWarps * 32), 0, stream, true, A));
    return SVD_OK;
}

// ---- read-back -----------------------------------------------------------------------------
// One warp per token and kv head; a lane's four dimensions of K and of V.
__global__ void __launch_bounds__(256) paged_read_kernel(const int64_t *__restrict__ slots, int T, int Hkv,
                                                         const uint8_t *__restrict__ pages, int page,
                                                         int64_t n_slots, float *__restrict__ k,
                                                         float *__restrict__ v) {
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    griddep_wait();
    if (w >= (int64_t)T * Hkv) return;
    const int64_t t = w / Hkv, slot = slots[t];
    const int h = (int)(w - t * Hkv);
    float4 ko = {0.f, 0.f, 0.f, 0.f}, vo = {0.f, 0.f, 0.f, 0.f};
    if (slot >= 0 && slot < n_slots) {
        const int64_t pg = slot / page;
        const int off = (int)(slot - pg * page), pos = off & 15, blk = lane >> 3;
        const uint8_t *const unit = pages + ((pg * Hkv + h) * (page >> 4) + (off >> 4)) * (int64_t)kPgUnitBytes;
        const uint32_t kc = *reinterpret_cast<const uint16_t *>(unit + blk * 256 + pos * 16 + (lane & 7) * 2);
        const float kd = __half2float(*reinterpret_cast<const __half *>(unit + kPgKScales + pos * 8 + blk * 2));
        const float vd = __half2float(*reinterpret_cast<const __half *>(unit + kPgVScales + blk * 32 + pos * 2));
        const uint8_t *const vr = unit + kPgVCodes + (4 * (lane & 15)) * 16 + pg_v_byte(pos);
        const int sh = lane < 16 ? 0 : 4;
        ko.x = kd * ((int)(kc & 15) - 8);
        ko.y = kd * ((int)((kc >> 4) & 15) - 8);
        ko.z = kd * ((int)((kc >> 8) & 15) - 8);
        ko.w = kd * ((int)(kc >> 12) - 8);
        vo.x = vd * (((vr[0] >> sh) & 15) - 8);
        vo.y = vd * (((vr[16] >> sh) & 15) - 8);
        vo.z = vd * (((vr[32] >> sh) & 15) - 8);
        vo.w = vd * (((vr[48] >> sh) & 15) - 8);
    }
    reinterpret_cast<float4 *>(k)[w * 32 + lane] = ko;
    reinterpret_cast<float4 *>(v)[w * 32 + lane] = vo;
}

int paged_read(const int64_t *slots, int T, int Hkv, const void *pages, int page, int64_t n_pages, float *k,
               float *v, cudaStream_t stream) {
    if (!slots || !pages || !k || !v || T < 0 || !pg_pool_ok(Hkv, page, n_pages) || !aligned16(pages) ||
        !aligned16(k) || !aligned16(v))
        return SVD_ERR_INVALID_ARG;
    if (T == 0) return SVD_OK;
    const int64_t grid = ((int64_t)T * Hkv + 7) / 8;
    if (grid > INT32_MAX) return SVD_ERR_INVALID_ARG;
    SVD_CUDA_TRY(launch(paged_read_kernel, dim3((unsigned)grid), dim3(256), 0, stream, true, slots, T, Hkv,
                        (const uint8_t *)pages, page, n_pages * page, k, v));
    return SVD_OK;
}

}  // namespace svd
