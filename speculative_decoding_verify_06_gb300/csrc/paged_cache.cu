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
// element a function of the sums and the inputs alone (no CTA waits for another).  What bounds it is
// latency, a launch and three block-wide sums one after the other: 3.8 us for 8 requests (95 KB moved), 5.9
// us for 256 with 131 K table entries, 6.5 us for 48 prompts with 49 K new tokens.  (With 64-bit divisions in
// the sums 4.1, 6.3 and 6.9.)
constexpr int kTbThreads = 512;
constexpr int kTbWarps = kTbThreads / 32;
constexpr int kTbChunk = 1024;  // outputs per work item

struct TbArgs {
    const int32_t *held, *window, *emitted, *n_new, *table, *free_ids, *n_free;
    int32_t *table_out, *free_out, *n_free_out, *kv_len, *q_start, *positions, *status;
    int64_t *slots;
    int R, page, width, n_pages, tokens;
    int32_t *held_out, *window_out;  // the state carried to the next call, or null: see tb_ask
    int max_new;                     // tokens of one request
};

// What request r asks for: the positions held, the tokens of the last window and how many of them
// stay.  Where the state is carried, a window of -d says that d positions go (its count is settled),
// and a request without a window has no count.
struct TbAsk {
    long long held, win, emi;
    __device__ bool in_order() const { return win >= 0 && emi >= 0 && emi <= win && win <= held; }
};
__device__ __forceinline__ TbAsk tb_ask(const TbArgs &A, int r) {
    TbAsk a = {A.held[r], A.window ? A.window[r] : 0, A.emitted ? A.emitted[r] : 0};
    if (A.held_out) {
        a.emi = a.win <= 0 ? 0 : A.emitted ? a.emi : a.win;
        a.win = a.win < 0 ? -a.win : a.win;
    }
    return a;
}

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
        long long keep = 0;
        uint32_t st = 0, ask = 0, p0 = 0, p1 = 0;
        if (r < R) {
            const TbAsk a = tb_ask(A, r);
            const long long n = A.n_new[r];
            const long long room = (long long)A.width * A.page;  // < 2^31
            keep = a.held - a.win + a.emi;
            if (!a.in_order() || n < 0 || a.held > room || keep + n > room) {
                st = SVD_ST_BAD_REQUEST;
            } else {
                p0 = ((uint32_t)a.held + A.page - 1) / (uint32_t)A.page;
                p1 = ((uint32_t)(keep + n) + A.page - 1) / (uint32_t)A.page;
                if (n > A.max_new) st = SVD_ST_NO_TOKENS;
                else ask = (uint32_t)n;
            }
        }
        const unsigned long long upto = tok_sum + tb_scan(ask, &total, s_w);
        tok_sum += total;
        if (!st && ask > 0 && upto > (unsigned long long)A.tokens) st = SVD_ST_NO_TOKENS;
        if (st) p1 = p0;
        const uint32_t take = p1 > p0 ? p1 - p0 : 0, give = p0 > p1 ? p0 - p1 : 0;
        const unsigned long long pg = ((unsigned long long)give << 32) | take;
        const unsigned long long sum = page_sum + tb_scan(pg, &total, s_w);
        page_sum += total;
        if (r < R) {
            s_keep[r] = (int)keep;
            s_p0[r] = (int)p0;
            s_q1[r] = (int)p1;
            s_take[r] = (int)((uint32_t)sum - take);
            s_give[r] = (int)((uint32_t)(sum >> 32) - give);
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
            const int n = st ? 0 : A.n_new[r];
            A.q_start[r] = s_tok[r];
            A.status[r] = (int)st;
            if (!A.held_out) {
                A.kv_len[r] = st == SVD_ST_BAD_REQUEST ? 0 : s_keep[r] + n;
            } else {
                // A refused request holds what it held; its count is settled if it was in order, and
                // else asked for again (what stays for certain is counted).
                const TbAsk a = tb_ask(A, r);
                const bool good = a.in_order();
                A.kv_len[r] = good ? s_keep[r] + n : (int)max(a.held - a.win, 0ll);
                A.held_out[r] = st ? (int)a.held : s_keep[r] + n;
                A.window_out[r] = !st ? n : good ? (int)(a.emi - a.win) : A.window[r];
            }
        }
        if (tid == 0) {
            A.q_start[R] = n_tok;
            *A.n_free_out = left;
        }
    }
    const uint32_t row_items = (A.width + kTbChunk - 1) / kTbChunk, t_items = (uint32_t)R * row_items;  // < 2^31
    const uint32_t f_items = (A.n_pages + kTbChunk - 1) / kTbChunk, s_items = (A.tokens + kTbChunk - 1) / kTbChunk;
    for (uint32_t it = blockIdx.x; it < t_items + f_items + s_items; it += gridDim.x) {
        if (it < t_items) {
            const int r = (int)(it / row_items), c0 = (int)(it - r * row_items) * kTbChunk;
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
                    const uint32_t col = (uint32_t)pos / (uint32_t)A.page;
                    slot = (int64_t)entry(r, (int)col) * A.page + (pos - (int)col * A.page);
                }
                A.slots[i] = slot;
                A.positions[i] = pos;
            }
        }
    }
}

static int tb_launch(TbArgs A, int64_t n_pages, int64_t tokens, cudaStream_t stream) {
    if (!A.held || !A.n_new || !A.table || !A.free_ids || !A.n_free || !A.table_out || !A.free_out || !A.n_free_out ||
        !A.kv_len || !A.q_start || !A.slots || !A.positions || !A.status)
        return SVD_ERR_INVALID_ARG;
    if (A.R < 1 || A.R > SVD_PAGED_MAX_REQUESTS || !pg_page_size_ok(A.page) || A.width < 1 ||
        (int64_t)A.width * A.page > INT32_MAX || (int64_t)A.width * A.R > INT32_MAX || n_pages < 1 ||
        n_pages > (int64_t)1 << 30 || tokens < 1 || tokens > (int64_t)1 << 30)
        return SVD_ERR_INVALID_ARG;
    if (A.table_out == A.table || A.free_out == A.free_ids || A.n_free_out == A.n_free) return SVD_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms < 1) return SVD_ERR_CUDA;
    A.n_pages = (int)n_pages;
    A.tokens = (int)tokens;
    const size_t smem = (size_t)A.R * 25 + 8;
    if (smem > 48 * 1024)
        SVD_CUDA_TRY(allow_smem<paged_tables_kernel>((size_t)SVD_PAGED_MAX_REQUESTS * 25 + 8));
    auto items = [](int64_t n) { return (n + kTbChunk - 1) / kTbChunk; };
    const int64_t work = (int64_t)A.R * items(A.width) + items(n_pages) + items(tokens);
    const int grid = (int)(work < 2 * sms ? work : 2 * sms);
    SVD_CUDA_TRY(launch(paged_tables_kernel, dim3(grid), dim3(kTbThreads), smem, stream, true, A));
    return SVD_OK;
}

int paged_tables(const int32_t *held, const int32_t *window, const int32_t *emitted, const int32_t *n_new,
                 int R, int page, const int32_t *table, int width, const int32_t *free_ids,
                 const int32_t *n_free, int64_t n_pages, int32_t *table_out, int32_t *free_out,
                 int32_t *n_free_out, int32_t *kv_len, int32_t *q_start, int64_t *slots,
                 int32_t *positions, int64_t tokens, int32_t *status, cudaStream_t stream) {
    if ((!window) != (!emitted)) return SVD_ERR_INVALID_ARG;
    return tb_launch({held, window, emitted, n_new, table, free_ids, n_free, table_out, free_out, n_free_out, kv_len,
                      q_start, positions, status, slots, R, page, width, 0, 0, nullptr, nullptr, INT32_MAX},
                     n_pages, tokens, stream);
}

int paged_advance(const int32_t *held, const int32_t *window, const int32_t *emitted, const int32_t *n_new,
                  int R, int max_new, int page, const int32_t *table, int width, const int32_t *free_ids,
                  const int32_t *n_free, int64_t n_pages, int32_t *held_out, int32_t *window_out,
                  int32_t *table_out, int32_t *free_out, int32_t *n_free_out, int32_t *kv_len,
                  int32_t *q_start, int64_t *slots, int32_t *positions, int64_t tokens, int32_t *status,
                  cudaStream_t stream) {
    if (!window || !held_out || !window_out || held_out == held || window_out == window || max_new < 1)
        return SVD_ERR_INVALID_ARG;
    return tb_launch({held, window, emitted, n_new, table, free_ids, n_free, table_out, free_out, n_free_out, kv_len,
                      q_start, positions, status, slots, R, page, width, 0, 0, held_out, window_out, max_new},
                     n_pages, tokens, stream);
}

// ---- rotary positions and the append -------------------------------------------------------
// q, k: (y_a, y_b) = (x_a cos - x_b sin, x_b cos + x_a sin) for every pair i of dimensions, the
// angle being position[axis(i)] * inv_freq(i); q is rounded to bf16, k and v to 4 bits per block of
// 32.
//
// Angles.  position * inv_freq reaches 10^6 radians; reduced in fp32 it would be off by 0.06.
// The host turns each frequency into turns per position as a 64-bit fraction, so that one 64-bit
// integer product gives the angle modulo a turn to 2^-33 turns for any 31-bit position; cos and sin of
// what is left come from a small table and one short turn, as sums of two floats.
//
// Codes.  A key next to the border of two codes must get the code that exact arithmetic gives, or
// the cache would depend on how the angle was rounded.  Keys are therefore carried as sums of two
// floats with an error bound of 2^-27 (|x_a| + |x_b|) (none for values and for unrotated dimensions);
// where a block's scale or one of its codes could still change within it (by the bound, about once in 10^4
// key heads; ten times as often with plain fp32 keys, for which a batch of 256 tokens took 16.5 us instead
// of 11.5 with the read-back), the warp redoes the head in fp64 from the same integer angle.  Borders are
// (n - 8.5) d, exact in fp32 because d has eight significant bits, so a code is settled by comparing
// against them and no division is rounded.
//
// Split.  A CTA of four warps takes a token, its warps every fourth head, four heads fetched ahead;
// calls of few tokens spread a token's heads over several CTAs.  4099 tokens of 32 + 2 x 8 heads in
// bf16 take 42 us (88 MB, 2.1 TB/s), 256 tokens of 40 + 2 x 8 in fp32 8.8 us: what bounds the first is issue
// (72 % at 173 warp instructions a head on average; before branches left the loops over dimensions, copies
// with a part taken out counted 24 for a query head, 248 for a value head and 529 for a key head).
// With the read-back 51.6 us.  Compared when that was 50.4 (before finite and other blocks of a head were
// told apart): eight warps to a CTA 51.4, two 52.0; six or seven CTAs to an SM 54.9 and 52.5 (and 10.2 and
// 10.4 for the 256 tokens, against 11.0); a warp a head and no loop 89.  The rare paths behind one call that
// makes both: 57.8, in a loop over them: 59.5.
constexpr int kApWarps = 4;

struct RopeArgs {
    uint64_t phase[SVD_ROPE_MAX_PAIRS];  // turns per position, as a fraction of 2^64
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

// Four values as they lie in memory, and as floats.
__device__ __forceinline__ float4 ap_raw(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ uint2 ap_raw(const __nv_bfloat16 *p) { return *reinterpret_cast<const uint2 *>(p); }
__device__ __forceinline__ void ap_floats(const float4 &v, float x[4]) {
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void ap_floats(const uint2 &v, float x[4]) {
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xFFFF0000u);
}

// Pair i's angle at token t, less the nearest multiple of a quarter turn (*quad): 2^-64 turns.
__device__ __forceinline__ int64_t ap_phase(const ApArgs &A, int t, int i, uint32_t *quad) {
    const int64_t pos = A.positions[A.rope.axis[i] * A.positions_ld + t];
    const uint64_t ph = (uint64_t)pos * A.rope.phase[i], q = (ph + (1ull << 61)) >> 62;
    *quad = (uint32_t)q;
    return (int64_t)(ph - (q << 62));
}

// cos and sin of k / 256 turns (high and low parts), k = 0..32.
__constant__ float4 kApTurn[33] = {
    {1.0f, 0.0f, 0.0f, 0.0f}, {0.999698818f, 9.66254299e-10f, 0.024541229f, -4.86716001e-10f},
    {0.99879545f, 6.47143805e-09f, 0.0490676761f, -1.73993431e-09f}, {0.997290432f, 2.42255354e-08f, 0.0735645667f, -3.07218095e-09f},
    {0.99518472f, 7.10966619e-09f, 0.0980171412f, -8.93393193e-10f}, {0.992479563f, -2.81606898e-08f, 0.122410677f, -2.17419305e-09f},
    {0.989176512f, -1.79974535e-09f, 0.146730468f, 6.77824552e-09f}, {0.985277653f, -1.03515374e-08f, 0.170961887f, 2.11593787e-09f},
    {0.980785251f, 2.97394731e-08f, 0.195090324f, -1.67047143e-09f}, {0.975702107f, 2.30858621e-08f, 0.219101235f, 4.88636953e-09f},
    {0.970031261f, -8.24954771e-09f, 0.242980182f, -2.2676041e-09f}, {0.963776052f, 1.37973011e-08f, 0.266712755f, 2.51006993e-09f},
    {0.956940353f, -1.7184508e-08f, 0.290284663f, 1.38156651e-08f}, {0.949528158f, 2.28820074e-08f, 0.313681751f, -1.10907479e-08f},
    {0.941544056f, 9.24430044e-09f, 0.336889863f, -9.62200097e-09f}, {0.932992816f, -1.71366352e-08f, 0.359895051f, -1.39906771e-08f},
    {0.923879504f, 2.83074897e-08f, 0.382683426f, 6.22335072e-09f}, {0.914209783f, -2.73737086e-08f, 0.405241311f, 3.40852391e-09f},
    {0.903989315f, -2.1909516e-08f, 0.427555084f, 9.20176646e-09f}, {0.893224299f, 2.2415052e-09f, 0.449611336f, -6.3382064e-09f},
    {0.881921291f, -2.70029634e-08f, 0.471396744f, -7.42525375e-09f}, {0.870086968f, 2.31636132e-08f, 0.492898196f, -3.75219544e-09f},
    {0.857728601f, 9.49825818e-09f, 0.514102757f, -1.27838593e-08f}, {0.84485358f, -1.47483092e-08f, 0.534997642f, -2.21531558e-08f},
    {0.831469595f, 1.68702634e-08f, 0.555570245f, -1.17695214e-08f}, {0.817584813f, 5.10439913e-10f, 0.575808167f, 2.39602649e-08f},
    {0.803207517f, 1.48104178e-08f, 0.59569931f, -5.81030113e-09f}, {0.78834641f, 1.78289383e-08f, 0.615231574f, 1.6998932e-08f},
    {0.773010433f, 2.06425526e-08f, 0.634393275f, 9.37955758e-09f}, {0.757208824f, 2.23487699e-08f, 0.653172851f, -7.65504904e-09f},
    {0.740951121f, 4.50153514e-09f, 0.671558976f, -2.13263824e-08f}, {0.724247098f, -1.5017589e-08f, 0.689540565f, -2.02768184e-08f},
    {0.707106769f, 1.21016175e-08f, 0.707106769f, 1.21016175e-08f},
};
// cos and sin of the pair's angle as sums of two floats, to 2^-28: an entry of the table, turned by what
// is left (at most a 512th of a turn), whose fp32 errors count for an 80th.
__device__ __forceinline__ float4 ap_cos_sin(const ApArgs &A, int t, int i) {
    uint32_t quad;
    const int64_t r = ap_phase(A, t, i, &quad);
    const int k = (int)((r + (1ll << 55)) >> 56);
    const float a = __ll2float_rn(r - ((int64_t)k << 56)) * (6.283185307f * 0x1p-64f), z = a * a;
    float4 e = kApTurn[k < 0 ? -k : k];
    if (k < 0) { e.z = -e.z; e.w = -e.w; }
    const float sa = a * fmaf(z, -1.f / 6.f, 1.f), ca = z * fmaf(z, 1.f / 24.f, -0.5f);  // sin a, cos a - 1
    const float dc = fmaf(e.x, ca, -e.z * sa) + e.y, ds = fmaf(e.z, ca, e.x * sa) + e.w;
    float4 o;
    o.x = e.x + dc;
    o.y = dc - (o.x - e.x);
    o.z = e.z + ds;
    o.w = fabsf(e.z) >= fabsf(ds) ? ds - (o.z - e.z) : e.z - (o.z - ds);
    if (quad & 1) o = make_float4(-o.z, -o.w, o.x, o.y);
    if (quad & 2) o = make_float4(-o.x, -o.y, -o.z, -o.w);
    return o;
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
__device__ __forceinline__ F ap_extreme(const F y[4], int lane) {
    F m = y[0];
    int at = 0;
#pragma unroll
    for (int j = 1; j < 4; ++j)
        if (fabs(y[j]) > fabs(m)) { m = y[j]; at = j; }
    at += (lane & 7) * 4;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        const F om = __shfl_xor_sync(~0u, m, o);
        const int oa = __shfl_xor_sync(~0u, at, o);
        if (fabs(om) > fabs(m) || (fabs(om) == fabs(m) && oa < at)) { m = om; at = oa; }
    }
    return m;
}

// (Arguments and results of the two rare paths go by value: an array whose address is passed would
// live in local memory on the common path too.)
struct ApOut {
    uint32_t codes, scale;
};

// Rotated keys in fp64, for a warp in which one is in doubt.  cos and sin of the reduced angle,
// |x| <= pi / 4, by their Taylor series (the first terms left out are below 2^-58); the four pairs side
// by side, since this GPU issues one fp64 instruction of a warp in sixteen cycles and what counts is
// that they follow each other closely.  The whole path takes about 2 us, and a batch waits for it.
__device__ __noinline__ ApOut ap_keys_f64(const ApArgs &A, int t, float4 xa, float4 xo, int lane) {
    const float xa4[4] = {xa.x, xa.y, xa.z, xa.w}, xb4[4] = {xo.x, xo.y, xo.z, xo.w};
    const int pairs = A.rope.pairs, d0 = 4 * lane;
    const bool on = d0 < 2 * pairs, up = !A.rope.interleaved && d0 >= pairs;
    double x[4], z[4], c[4], sn[4], y[4];
    uint32_t quad[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = A.rope.interleaved ? 2 * lane + (j >> 1) : d0 + j - (up ? pairs : 0);
        x[j] = (double)(on ? ap_phase(A, t, i, &quad[j]) : 0) * (3.14159265358979323846 * 0x1p-63);
        z[j] = x[j] * x[j];
        c[j] = 1.0 / 20922789888000.0;   // 1 / 16!
        sn[j] = 1.0 / 355687428096000.0;  // 1 / 17!
    }
    const double fc[8] = {-1.0 / 87178291200.0, 1.0 / 479001600.0, -1.0 / 3628800.0, 1.0 / 40320.0, -1.0 / 720.0, 1.0 / 24.0, -0.5, 1.0};
    const double fs[8] = {-1.0 / 1307674368000.0, 1.0 / 6227020800.0, -1.0 / 39916800.0, 1.0 / 362880.0, -1.0 / 5040.0,
                          1.0 / 120.0, -1.0 / 6.0, 1.0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c[j] = fma(c[j], z[j], fc[k]);
            sn[j] = fma(sn[j], z[j], fs[k]);
        }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        double cc = c[j], ss = sn[j] * x[j];
        if (on && (quad[j] & 1)) { const double w = ss; ss = cc; cc = -w; }
        if (on && (quad[j] & 2)) { ss = -ss; cc = -cc; }
        if (!(A.rope.interleaved ? (j & 1) : up)) ss = -ss;
        const double r = __dadd_rn(__dmul_rn((double)xa4[j], cc), __dmul_rn((double)xb4[j], ss));
        y[j] = on ? r : (double)xa4[j];
        if (fabs(y[j]) > kPgMaxAbs) y[j] = y[j] < 0.0 ? -kPgMaxAbs : kPgMaxAbs;
    }
    const uint16_t db = ap_scale(ap_extreme(y, lane));
    const float df = __half2float(__ushort_as_half((uint16_t)(db & 0x7FFFu)));
    const double d = (double)df;
    uint32_t codes = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const double v = (db & 0x8000u) ? -y[j] : y[j];
        float n = floorf(fminf(fmaxf((float)v * (1.f / df) + 8.5f, 0.f), 15.f));  // this or a neighbour
        const double gap = fma((double)(8.5f - n), d, v);                          // v - (n - 8.5) d
        if (gap < 0.0) n -= 1.f;
        else if (gap >= d) n += 1.f;
        codes |= (df == 0.f ? 8u : (uint32_t)fminf(fmaxf(n, 0.f), 15.f)) << (8 * j);
    }
    return {codes, db};
}

// Values as they came, with anything in them: not finite, too large, all zero, ties, scales among
// fp16's subnormals.  What came not finite (odd: in this lane) is noted and stored as 0 or the largest
// magnitude: a cache byte never stands for a NaN that a masked position could spread.
__device__ __noinline__ ApOut ap_general(int32_t *status, float4 y4, bool odd, int lane) {
    float y[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (y[j] != y[j]) y[j] = 0.f;
        y[j] = fminf(fmaxf(y[j], -(float)kPgMaxAbs), (float)kPgMaxAbs);
    }
    if (__any_sync(~0u, odd) && status && lane == 0) atomicOr(status, SVD_ST_NONFINITE);
    const uint16_t db = ap_scale(ap_extreme(y, lane));
    const float d = __half2float(__ushort_as_half((uint16_t)(db & 0x7FFFu)));
    uint32_t codes = 0x08080808u;
    if (d != 0.f) {
        codes = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float v = (db & 0x8000u) ? -y[j] : y[j];
            float n = floorf(fminf(fmaxf(v * (1.f / d) + 8.5f, 0.f), 15.f));
            if (v < (n - 8.5f) * d) n -= 1.f;  // borders are exact: eight bits and five
            else if (v >= (n - 7.5f) * d) n += 1.f;
            codes |= (uint32_t)fminf(fmaxf(n, 0.f), 15.f) << (8 * j);
        }
    }
    return {codes, db};
}

// The scale and codes of a lane's block where nothing is in doubt; false where something is.  With the
// sign of d taken out, z = v / |d| + 8 rounds to the code or to one more (its error is below 2^-18),
// and the exact distance v - (n - 8.5) |d| from the border decides; a rotated key is in doubt when it
// lies within its error of a border.
template <bool ROT>
__device__ __forceinline__ bool ap_quick(const float y[4], const float low[4], const float err[4], bool turned,
                                         uint16_t *scale, uint32_t *codes) {
    float hi = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])), lo = fminf(fminf(y[0], y[1]), fminf(y[2], y[3]));
    const float none = (y[0] + y[1]) * 0.f + (y[2] + y[3]) * 0.f;  // NaN if one is not finite
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, o));
        lo = fminf(lo, __shfl_xor_sync(~0u, lo, o));
    }
    const float m = hi > -lo ? hi : lo, big = fabsf(m);
    const uint16_t db = ap_scale(m);
    const float d = __half2float(__ushort_as_half((uint16_t)(db & 0x7FFFu)));
    // (& and not &&: no branches)
    bool sure = (none == 0.f) & (hi != -lo) & (big <= (float)kPgMaxAbs) & (d >= 0x1p-14f);
    if (ROT) {
        const float e4 = fmaxf(fmaxf(err[0], err[1]), fmaxf(err[2], err[3]));
        const float e = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(e4)));
        // the other extreme as large, or a scale next to a border: within the error, or m (which stands
        // for what rounds to it) on one
        const bool clear_m = (fabsf(hi + lo) > 2.f * e + 0x1p-22f * big) & ((__float_as_uint(m) & 0xFFFFu) != 0x8000u) &
                             (__bfloat16_as_ushort(__float2bfloat16_rn(big - e)) ==
                              __bfloat16_as_ushort(__float2bfloat16_rn(big + e)));
        sure &= clear_m | (e == 0.f);
    }
    const uint32_t flip = (uint32_t)(db & 0x8000u) << 16;
    const float inv = __fdividef(1.f, d), half = 0.5f * d, clear = half - 0x1p-23f * d;
    float room = 1.f;  // of the key that is nearest to a border
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float v = __uint_as_float(__float_as_uint(y[j]) ^ flip);
        float n = fmaf(v, inv, 8.f + 0x1p-18f) + 0x1p23f;  // to a whole number, in the low bits
        float gap = v - fmaf(n - 0x1p23f, d, -8.5f * d);   // (the border is exact: eight bits and five)
        if (ROT) gap += __uint_as_float(__float_as_uint(low[j]) ^ flip);
        const bool below = gap < 0.f;
        n -= below ? 1.f : 0.f;
        if (ROT) {
            gap += below ? d : 0.f;
            room = fminf(room, (clear - err[j]) - fabsf(gap - half));
        }
        c[j] = __float_as_uint(fminf(n, 0x1p23f + 15.f));
    }
    if (ROT) sure &= (room > 0.f) | !turned;
    *scale = db;
    *codes = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    return sure;
}

// What a lane's four dimensions turn by, the same for every head of a token.
struct ApTurn {
    float c[4], s[4];  // y = x c + xb s, xb the other dimension of the pair (s carries the sign)
    float cl[4], sl[4];  // their low parts
    bool on;           // the dimensions are rotated
    int mate;          // the lane of the other dimensions of half-split pairs; -1: interleaved
};

// One head of one token: a warp, four dimensions to a lane.  unit0, pos: the token's unit of kv head
// 0 and its place there; unit0 is null when it is not stored.
__device__ __forceinline__ void ap_head(const ApArgs &A, int t, int head, int lane, uint8_t *unit0, int pos,
                                        const ApTurn &turn, const float x[4]) {
    const int d0 = 4 * lane;
    const bool is_v = head >= A.Hq + A.Hkv;
    float xb[4] = {0.f, 0.f, 0.f, 0.f}, y[4], low[4] = {0.f, 0.f, 0.f, 0.f}, err[4] = {0.f, 0.f, 0.f, 0.f};
    // (branches around the loops, selects inside them)
    if (!is_v) {
        if (turn.mate < 0) {
            xb[0] = x[1]; xb[1] = x[0]; xb[2] = x[3]; xb[3] = x[2];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) xb[j] = __shfl_sync(~0u, x[j], turn.mate);
        }
    }
    if (head < A.Hq) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float r = __fadd_rn(__fmul_rn(x[j], turn.c[j]), __fmul_rn(xb[j], turn.s[j]));
            y[j] = turn.on ? r : x[j];
        }
    } else if (!is_v) {  // a key: with what the products and the sum dropped, and cos' and sin's low parts
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float p = __fmul_rn(x[j], turn.c[j]), q = __fmul_rn(xb[j], turn.s[j]), r = __fadd_rn(p, q);
            const float b = __fsub_rn(r, p), lost = __fadd_rn(__fsub_rn(p, __fsub_rn(r, b)), __fsub_rn(q, b));
            const float rest = fmaf(x[j], turn.c[j], -p) + fmaf(xb[j], turn.s[j], -q) + lost +
                               fmaf(x[j], turn.cl[j], xb[j] * turn.sl[j]);
            const float v = __fadd_rn(r, rest);
            y[j] = turn.on ? v : x[j];
            low[j] = turn.on ? __fsub_rn(rest, __fsub_rn(v, r)) : 0.f;
            err[j] = turn.on ? (fabsf(x[j]) + fabsf(xb[j])) * 0x1p-27f : 0.f;
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
    if (!unit0) return;
    // The common case; whatever it cannot settle goes the general way.
    uint16_t db;
    uint32_t codes;
    const bool sure = is_v ? ap_quick<false>(y, low, err, false, &db, &codes)
                           : ap_quick<true>(y, low, err, turn.on, &db, &codes);
    if (!__all_sync(~0u, sure)) {
        // Rotated blocks in doubt need the angle again; others, and those with a value that is not finite,
        // only their values (for the latter as the formula gives them: the parts that the products dropped
        // are not numbers there).
        const bool turned = !is_v && 4 * (lane & 24) < 2 * A.rope.pairs;
        bool odd = false, clean = true;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            odd |= !(fabsf(x[j]) <= 3.4028235e38f);
            clean &= fabsf(x[j]) <= 3.4028235e38f && (is_v || fabsf(xb[j]) <= 3.4028235e38f);
            if (!is_v && turn.on && !(fabsf(y[j]) <= 3.4028235e38f))
                y[j] = __fadd_rn(__fmul_rn(x[j], turn.c[j]), __fmul_rn(xb[j], turn.s[j]));
        }
        const uint32_t all_clean = __ballot_sync(~0u, clean);  // (a vote of all lanes: before anything that divides them)
        const bool again = turned && ((all_clean >> (lane & 24)) & 0xFFu) == 0xFFu;  // of the block
        if (__any_sync(~0u, !sure && again)) {
            const ApOut o =
                ap_keys_f64(A, t, make_float4(x[0], x[1], x[2], x[3]), make_float4(xb[0], xb[1], xb[2], xb[3]), lane);
            if (again) {
                codes = o.codes;
                db = (uint16_t)o.scale;
            }
        }
        if (__any_sync(~0u, !sure && !again)) {
            const ApOut o = ap_general(A.status ? A.status + t : nullptr, make_float4(y[0], y[1], y[2], y[3]), odd, lane);
            if (!again) {
                codes = o.codes;
                db = (uint16_t)o.scale;
            }
        }
    }

    uint8_t *const unit = unit0 + (int64_t)(head - A.Hq - (is_v ? A.Hkv : 0)) * ((A.page >> 4) * kPgUnitBytes);
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

template <typename T>
__global__ void __launch_bounds__(kApWarps * 32, 8) paged_append_kernel(const __grid_constant__ ApArgs A) {
    __shared__ float4 s_cs[SVD_ROPE_MAX_PAIRS];
    __shared__ uint8_t *s_unit;
    __shared__ int s_pos;
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pairs = A.rope.pairs, heads = A.Hq + 2 * A.Hkv, step = kApWarps * gridDim.y, d0 = 4 * lane;
    const T *const row = reinterpret_cast<const T *>(A.qkv) + t * A.ld + d0;
    int head = blockIdx.y * kApWarps + warp;
    griddep_wait();
    // A CTA lives for a few microseconds, most of them loads: four heads are fetched ahead, the
    // first ones before the angles.
    decltype(ap_raw(row)) ahead[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (head + k * step < heads) ahead[k] = ap_raw(row + (int64_t)(head + k * step) * kPgDim);
    if ((int)threadIdx.x < pairs) s_cs[threadIdx.x] = ap_cos_sin(A, t, threadIdx.x);
    if (threadIdx.x == kApWarps * 32 - 1) {
        const int64_t slot = A.slots[t];
        uint8_t *unit = nullptr;
        int pos = 0;
        if (slot >= 0 && slot < A.n_slots) {
            const int64_t page = slot / A.page;
            const int off = (int)(slot - page * A.page);
            pos = off & 15;
            unit = A.pages + (page * A.Hkv * (A.page >> 4) + (off >> 4)) * (int64_t)kPgUnitBytes;
        } else if (slot >= 0 && A.status && blockIdx.y == 0) {
            atomicOr(A.status + t, SVD_ST_BAD_SLOT);
        }
        s_unit = unit;
        s_pos = pos;
    }
    __syncthreads();
    uint8_t *const unit0 = s_unit;
    const int pos = s_pos;
    ApTurn turn;
    turn.on = d0 < 2 * pairs;  // pairs is a multiple of four: a lane's dimensions turn alike
    const bool up = !A.rope.interleaved && d0 >= pairs;
    turn.mate = A.rope.interleaved ? -1 : turn.on ? (up ? lane - (pairs >> 2) : lane + (pairs >> 2)) : lane;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = A.rope.interleaved ? 2 * lane + (j >> 1) : d0 + j - (up ? pairs : 0);
        const float4 cs = turn.on ? s_cs[i] : make_float4(1.f, 0.f, 0.f, 0.f);
        const bool plus = A.rope.interleaved ? (j & 1) : up;
        turn.c[j] = cs.x;
        turn.cl[j] = cs.y;
        turn.s[j] = plus ? cs.z : -cs.z;
        turn.sl[j] = plus ? cs.w : -cs.w;
    }
    for (; head < heads; head += step) {
        float x[4];
        ap_floats(ahead[0], x);
#pragma unroll
        for (int k = 0; k < 3; ++k) ahead[k] = ahead[k + 1];
        if (head + 4 * step < heads) ahead[3] = ap_raw(row + (int64_t)(head + 4 * step) * kPgDim);
        ap_head(A, t, head, lane, unit0, pos, turn, x);
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
            r.n_axes > SVD_ROPE_MAX_AXES || (r.n_axes > 1 && positions_ld != 0 && positions_ld < T))
            return SVD_ERR_INVALID_ARG;
        A.rope.pairs = r.n_pairs;
        A.rope.interleaved = r.interleaved != 0;
        for (int i = 0; i < r.n_pairs; ++i) {
            if (!(fabs(r.inv_freq[i]) < 4294967296.0) || r.axis[i] >= r.n_axes) return SVD_ERR_INVALID_ARG;
            A.rope.phase[i] = rope_phase(r.inv_freq[i]);
            A.rope.axis[i] = r.axis[i];
        }
    }
    if (T == 0) return SVD_OK;
    // One CTA to a token once there are several tokens to an SM; fewer tokens' heads are spread.
    const int sms = sm_count();
    if (sms < 1) return SVD_ERR_CUDA;
    const int most = (int)((heads + kApWarps - 1) / kApWarps), want = (4 * sms + T - 1) / T;
    const dim3 grid((unsigned)T, (unsigned)(want < most ? want : most));
    if (dtype == SVD_F32)
        SVD_CUDA_TRY(launch(paged_append_kernel<float>, grid, dim3(kApWarps * 32), 0, stream, true, A));
    else
        SVD_CUDA_TRY(launch(paged_append_kernel<__nv_bfloat16>, grid, dim3(kApWarps * 32), 0, stream, true, A));
    return SVD_OK;
}

// ---- read-back -----------------------------------------------------------------------------
// One warp per token and kv head; a lane's four dimensions of K and of V.  Bounded by its fp32 writes and
// by latency: 4099 tokens of 8 heads (38 MB) in 10.3 us, 3.7 TB/s; 4 tokens in 1.5 us.  Two heads to a
// warp, loads first: 9.7 and 1.9 us; four: 11.8 and 2.6; divisions in 32 bits: no change.
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
