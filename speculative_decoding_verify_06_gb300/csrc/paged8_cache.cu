// paged8_cache.cu -- the write side of the paged 8-bit cache: rotary positions with several axes joined to the
// append, and the read-back.
//
// "Decode is memory-bound ..." ("The ceiling"): the cache joins the weights on every pass; 8 bits a value stand
// between the 4.5 of the other paged cache and the 16 of none.
//
//   scale = 2^e, e the smallest with 448 2^e >= |y| over the new values of a unit (16 positions of one kv head; K and
//   V apart), and no smaller than the scale that earlier positions of the unit have;  code = e4m3(y / 2^e)
//
// Units.  A scale belongs to 16 positions, so a unit is written by one CTA: the tokens of a request that lie in
// one unit are a run, and the CTA of the run's first token handles all of it.  Warp w has positions 4w .. 4w + 3 of the
// unit, a lane four dimensions of each: four codes of a dimension then fill a word of V's row.  Where earlier
// positions keep a smaller scale, their codes are rounded again in place.
//
// Codes.  A key next to the border of two codes must get the code that exact arithmetic gives, or the cache
// would depend on how the angle was rounded.  Keys are carried as sums of two floats with an error bound, as in the
// 4-bit append: a code is settled where y +- bound round alike, else by the distance from the border
// between the two codes, and where that is within the bound the token's keys are worked out again in fp64.  The scale in
// the same way.  Values and dimensions that do not turn are exact as they come.
#include "paged8.cuh"
#include "paged_rope.cuh"

namespace svd {

constexpr int kA8Warps = 4;
constexpr int kA8Threads = 32 * kA8Warps;
constexpr int kA8VRow = 5;  // words of a V row in shared memory (four and one apart)

struct A8Args {
    const void *qkv;
    int64_t ld;
    const int32_t *kv_len, *q_start, *table;
    uint8_t *pages;
    __nv_bfloat16 *q;
    int32_t *status;
    int64_t n_pages;
    int T, R, width, Hq, Hkv, page;
    int block, q_heads, kv_heads, q_parts;  // tokens of a CTA; heads of one; CTAs of the query heads
    RopeArgs rope;
};

// What a lane's four dimensions turn by, and the largest error of cos and sin (0 where they are exact).
struct A8Turn {
    float c[4], s[4], cl[4], sl[4], err[4];
};
struct A8Lane {
    bool on, up;
    int mate, d0;
};
__device__ __forceinline__ A8Lane a8_lane(const RopeArgs &R, int lane) {
    A8Lane l;
    l.d0 = 4 * lane;
    l.on = l.d0 < 2 * R.pairs;  // pairs is a multiple of four: a lane's dimensions turn alike
    l.up = !R.interleaved && l.d0 >= R.pairs;
    l.mate = R.interleaved ? -1 : l.on ? (l.up ? lane - (R.pairs >> 2) : lane + (R.pairs >> 2)) : lane;
    return l;
}
__device__ __forceinline__ A8Turn a8_turn(const RopeArgs &R, const A8Lane &l, int lane, const float4 *cs_row) {
    A8Turn t;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = R.interleaved ? 2 * lane + (j >> 1) : l.d0 + j - (l.up ? R.pairs : 0);
        const float4 cs = l.on ? cs_row[i] : make_float4(1.f, 0.f, 0.f, 0.f);
        const bool plus = R.interleaved ? (j & 1) : l.up;
        t.c[j] = cs.x;
        t.cl[j] = cs.y;
        t.s[j] = plus ? cs.z : -cs.z;
        t.sl[j] = plus ? cs.w : -cs.w;
        // (a quarter turn or none: the products are exact)
        t.err[j] = (cs.x == 0.f || cs.z == 0.f) && cs.y == 0.f && cs.w == 0.f ? 0.f : 0x1p-27f;
    }
    return t;
}
__device__ __forceinline__ void a8_mates(const A8Lane &l, const float x[4], float xb[4]) {
    if (l.mate < 0) {
        xb[0] = x[1]; xb[1] = x[0]; xb[2] = x[3]; xb[3] = x[2];
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) xb[j] = __shfl_sync(~0u, x[j], l.mate);
    }
}

// The request of token t: the last one whose first token is not behind it (a count over all of them).
__device__ __forceinline__ int a8_request(const A8Args &A, int t, int *s_count) {
    int n = 0;
    for (int r = threadIdx.x; r < A.R; r += kA8Threads) n += A.q_start[r] <= t;
    n = __reduce_add_sync(~0u, n);
    if ((threadIdx.x & 31) == 0) s_count[threadIdx.x >> 5] = n;
    __syncthreads();
    n = s_count[0] + s_count[1] + s_count[2] + s_count[3];
    __syncthreads();
    return max(n - 1, 0);
}

// A token's keys in fp64, where one is in doubt.
__device__ __noinline__ uint32_t a8_codes_f64(const A8Args &A, int t, float4 x, float4 xb, int lane, int e) {
    double y[4];
    ap_turn_f64(A.rope, t, x, xb, lane, y);
    uint32_t codes = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const double z = fmin(fabs(y[j]) * __longlong_as_double((long long)(1023 - e) << 52), 448.0);
        const int ex = max((int)((unsigned long long)__double_as_longlong(z) >> 52) - 1023, -6);
        const int n = __double2int_rn(z * __longlong_as_double((long long)(1023 + 3 - ex) << 52));
        const uint32_t c = (uint32_t)min(n + 8 * (ex + 6), 0x7E) | (y[j] < 0.0 ? 0x80u : 0u);
        codes |= c << (8 * j);
    }
    return codes;
}
__device__ __noinline__ double a8_top_f64(const A8Args &A, int t, float4 x, float4 xb, int lane) {
    double y[4];
    ap_turn_f64(A.rope, t, x, xb, lane, y);
    const double top = fmax(fmax(fabs(y[0]), fabs(y[1])), fmax(fabs(y[2]), fabs(y[3])));
    return top > (double)kP8MaxAbs ? (double)kP8MaxAbs : top;  // (NaN stays one, and counts for nothing)
}

// Codes of earlier positions under a scale 2^down times as large.
__device__ __forceinline__ uint32_t a8_again(uint32_t codes, float down) {
    const float2 a = p8_floats2(codes & 0xFFFFu), b = p8_floats2(codes >> 16);
    return p8_encode2(a.x * down, a.y * down) | (p8_encode2(b.x * down, b.y * down) << 16);
}

template <typename T>
__global__ void __launch_bounds__(kA8Threads) paged8_append_kernel(const __grid_constant__ A8Args A) {
    __shared__ float4 s_cs[16 * SVD_ROPE_MAX_PAIRS];
    __shared__ uint32_t s_v[kPgDim * kA8VRow];
    __shared__ uint32_t s_top[3][kA8Warps];
    __shared__ double s_top64[kA8Warps];
    __shared__ int s_count[kA8Warps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pairs = A.rope.pairs;
    const T *const qkv = reinterpret_cast<const T *>(A.qkv);
    griddep_wait();
    const int t0 = blockIdx.x * A.block, t1 = min(min(t0 + A.block, A.T), A.q_start[A.R]);
    if (t0 >= t1) return;
    const A8Lane l = a8_lane(A.rope, lane);

    if ((int)blockIdx.y < A.q_parts) {
        // ---- queries: a warp takes a head of a token ----------------------------------------------
        const int h0 = blockIdx.y * A.q_heads, nh = min(A.q_heads, A.Hq - h0), items = (t1 - t0) * nh;
        auto raw = [&](int it) {
            const int t = it / nh;
            return ap_raw(qkv + (t0 + t) * A.ld + (int64_t)(h0 + it - t * nh) * kPgDim + l.d0);
        };
        decltype(ap_raw(qkv)) ahead[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (warp + k * kA8Warps < items) ahead[k] = raw(warp + k * kA8Warps);
        for (int i = tid; i < (t1 - t0) * pairs; i += kA8Threads) {
            const int t = i / pairs;
            s_cs[t * SVD_ROPE_MAX_PAIRS + i - t * pairs] = ap_cos_sin(A.rope, t0 + t, i - t * pairs);
        }
        __syncthreads();
        for (int it = warp; it < items; it += kA8Warps) {
            float x[4], xb[4], y[4];
            ap_floats(ahead[0], x);
#pragma unroll
            for (int k = 0; k < 3; ++k) ahead[k] = ahead[k + 1];
            if (it + 4 * kA8Warps < items) ahead[3] = raw(it + 4 * kA8Warps);
            const int t = it / nh;
            a8_mates(l, x, xb);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = A.rope.interleaved ? 2 * lane + (j >> 1) : l.d0 + j - (l.up ? pairs : 0);
                const float2 cs = l.on ? *reinterpret_cast<const float2 *>(&s_cs[t * SVD_ROPE_MAX_PAIRS + i].x) : make_float2(1.f, 0.f);
                const float sn = l.on ? s_cs[t * SVD_ROPE_MAX_PAIRS + i].z : 0.f;
                const bool plus = A.rope.interleaved ? (j & 1) : l.up;
                const float r = __fadd_rn(__fmul_rn(x[j], cs.x), __fmul_rn(xb[j], plus ? sn : -sn));
                y[j] = l.on ? r : x[j];
            }
            const __nv_bfloat162 a = __floats2bfloat162_rn(y[0], y[1]), b = __floats2bfloat162_rn(y[2], y[3]);
            uint2 o;
            o.x = reinterpret_cast<const uint32_t &>(a);
            o.y = reinterpret_cast<const uint32_t &>(b);
            *reinterpret_cast<uint2 *>(A.q + ((int64_t)(t0 + t) * A.Hq + h0 + it - t * nh) * kPgDim + l.d0) = o;
        }
        return;
    }

    // ---- keys and values: the runs that begin in this block of tokens --------------------------------
    const int h0 = ((int)blockIdx.y - A.q_parts) * A.kv_heads, h1 = min(h0 + A.kv_heads, A.Hkv);
    int r = a8_request(A, t0, s_count);
    for (int t = t0; t < t1;) {
        while (r + 1 < A.R && A.q_start[r + 1] <= t) ++r;
        if (A.q_start[r] > t) {  // (a token before the first request's)
            t = A.q_start[r];
            continue;
        }
        const int q0 = max(A.q_start[r], 0), q1 = min(A.q_start[r + 1], A.T);
        const int64_t at = (int64_t)A.kv_len[r] - (A.q_start[r + 1] - (int64_t)A.q_start[r]) + (t - q0);  // position of token t
        const int i0 = (int)(at & 15), end = min(t + 16 - i0, q1);
        if (end <= t) return;  // (a q_start that does not ascend)
        if (t != q0 && i0 != 0) {  // the run began in another block
            t = end;
            continue;
        }
        const int n = end - t;  // positions i0 .. i0 + n - 1 of the unit
        int64_t pg = -1;
        if (at >= 0 && at < (int64_t)A.width * A.page) pg = A.table[(int64_t)r * A.width + (uint32_t)at / (uint32_t)A.page];
        if (pg < 0 || pg >= A.n_pages) {
            if (A.status && h0 == 0 && tid < n) atomicOr(A.status + t + tid, SVD_ST_BAD_SLOT);
            t = end;
            continue;
        }
        const int upp = A.page >> 4, place = (int)((uint32_t)at % (uint32_t)A.page) >> 4;
        for (int h = h0; h < h1; ++h) {
            uint8_t *const unit = A.pages + ((pg * A.Hkv + h) * upp + place) * (int64_t)kP8UnitBytes;
            // Warp w's positions 4w + k: those of the run are tokens tw + k.
            const int tw = t + 4 * warp - i0;
            decltype(ap_raw(qkv)) kr[4], vr[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (tw + k >= t && tw + k < end) {
                    const T *const row = qkv + (tw + k) * A.ld + (int64_t)(A.Hq + h) * kPgDim + l.d0;
                    kr[k] = ap_raw(row);
                    vr[k] = ap_raw(row + (int64_t)A.Hkv * kPgDim);
                }
            // V's row of dimension tid and the scales, where they hold other positions
            uint4 old = {0u, 0u, 0u, 0u};
            int ek0 = kP8ExpLo, ev0 = kP8ExpLo;
            if (n < 16) old = *reinterpret_cast<const uint4 *>(unit + kP8VCodes + 16 * tid);
            if (i0 > 0) {
                const float2 sc = *reinterpret_cast<const float2 *>(unit + kP8Scales);
                ek0 = p8_exponent(sc.x);
                ev0 = p8_exponent(sc.y);
            }
            if (h == h0) {
                __syncthreads();  // (the angles of the run before are read)
                for (int i = tid; i < n * pairs; i += kA8Threads) {
                    const int k = i / pairs;
                    s_cs[k * SVD_ROPE_MAX_PAIRS + i - k * pairs] = ap_cos_sin(A.rope, t + k, i - k * pairs);
                }
                __syncthreads();
            }
            float y[4][4], low[4][4], err[4][4], v[4][4];
            float top_k = 0.f, top_v = 0.f, top_err = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool here = tw + k >= t && tw + k < end;  // the same for the warp
#pragma unroll
                for (int j = 0; j < 4; ++j) y[k][j] = low[k][j] = err[k][j] = v[k][j] = 0.f;
                if (!here) continue;
                float x[4], xb[4];
                ap_floats(kr[k], x);
                ap_floats(vr[k], v[k]);
                a8_mates(l, x, xb);
                bool odd = false;
                if (l.on) {
                    const A8Turn tn = a8_turn(A.rope, l, lane, s_cs + (tw + k - t) * SVD_ROPE_MAX_PAIRS);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {  // with what the products and the sum dropped, and cos' and sin's low parts
                        const float p = __fmul_rn(x[j], tn.c[j]), q = __fmul_rn(xb[j], tn.s[j]), s = __fadd_rn(p, q);
                        const float b = __fsub_rn(s, p), lost = __fadd_rn(__fsub_rn(p, __fsub_rn(s, b)), __fsub_rn(q, b));
                        const float rest = fmaf(x[j], tn.c[j], -p) + fmaf(xb[j], tn.s[j], -q) + lost +
                                           fmaf(x[j], tn.cl[j], xb[j] * tn.sl[j]);
                        const float w = __fadd_rn(s, rest);
                        y[k][j] = w;
                        low[k][j] = __fsub_rn(rest, __fsub_rn(w, s));
                        err[k][j] = (fabsf(x[j]) + fabsf(xb[j])) * tn.err[j];
                        if (!(fabsf(w) <= kP8MaxAbs)) {  // too large, or no number: as the formula gives it
                            y[k][j] = s;
                            low[k][j] = err[k][j] = 0.f;
                        }
                        odd |= !(fabsf(x[j]) <= 3.4028235e38f);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        y[k][j] = x[j];
                        odd |= !(fabsf(x[j]) <= 3.4028235e38f);
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    odd |= !(fabsf(v[k][j]) <= 3.4028235e38f);
                    // what is no number counts as 0, and magnitudes end at the largest
                    y[k][j] = y[k][j] == y[k][j] ? fminf(fmaxf(y[k][j], -kP8MaxAbs), kP8MaxAbs) : 0.f;
                    v[k][j] = v[k][j] == v[k][j] ? fminf(fmaxf(v[k][j], -kP8MaxAbs), kP8MaxAbs) : 0.f;
                    top_k = fmaxf(top_k, fabsf(y[k][j]));
                    top_v = fmaxf(top_v, fabsf(v[k][j]));
                    top_err = fmaxf(top_err, err[k][j]);
                }
                if (__any_sync(~0u, odd) && A.status && lane == 0) atomicOr(A.status + tw + k, SVD_ST_NONFINITE);
            }
            // (floats that are not negative are ordered as their bits)
            const uint32_t w_k = __reduce_max_sync(~0u, __float_as_uint(top_k)), w_v = __reduce_max_sync(~0u, __float_as_uint(top_v));
            const uint32_t w_e = __reduce_max_sync(~0u, __float_as_uint(top_err));
            if (lane == 0) {
                s_top[0][warp] = w_k;
                s_top[1][warp] = w_v;
                s_top[2][warp] = w_e;
            }
            __syncthreads();
            auto most = [&](int i) { return __uint_as_float(max(max(s_top[i][0], s_top[i][1]), max(s_top[i][2], s_top[i][3]))); };
            const float big_k = most(0), big_v = most(1), big_e = most(2);
            int ek = p8_need(big_k);
            if (big_e > 0.f) {
                // the largest key's exact magnitude lies between these
                const float d = big_e + 0x1p-23f * big_k;
                const int e_hi = p8_need(big_k + d);
                if (p8_need(fmaxf(big_k - d, 0.f)) != e_hi) {
                    double top = 0.0;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (tw + k >= t && tw + k < end) {
                            float x[4], xb[4];
                            ap_floats(kr[k], x);
                            a8_mates(l, x, xb);
                            const double one = a8_top_f64(A, tw + k, make_float4(x[0], x[1], x[2], x[3]), make_float4(xb[0], xb[1], xb[2], xb[3]), lane);
                            top = fmax(top, one);
                        }
#pragma unroll
                    for (int o = 16; o; o >>= 1) top = fmax(top, __shfl_xor_sync(~0u, top, o));
                    if (lane == 0) s_top64[warp] = top;
                    __syncthreads();
                    top = fmax(fmax(s_top64[0], s_top64[1]), fmax(s_top64[2], s_top64[3]));
                    const float low_e = p8_pow2(max(e_hi - 1, kP8ExpLo));
                    ek = top > 448.0 * (double)low_e ? e_hi : e_hi - 1;
                }
            }
            ek = max(min(max(ek, kP8ExpLo), kP8ExpHi), ek0);
            const int ev = max(min(max(p8_need(big_v), kP8ExpLo), kP8ExpHi), ev0);
            const float inv_k = p8_pow2(-ek), inv_v = p8_pow2(-ev);

            uint32_t kc[4], vw[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                // what the key's exact value lies between rounds alike, or the border between the two codes decides
                uint32_t hi2[2], lo2[2];
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    float a[2], b[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float z = y[k][j + i] * inv_k, e = err[k][j + i];
                        const float d = e > 0.f ? fmaf(e, inv_k, 0x1p-23f * fabsf(z)) : 0.f;
                        a[i] = z + d;
                        b[i] = z - d;
                    }
                    hi2[j >> 1] = p8_encode2(a[0], a[1]);
                    lo2[j >> 1] = p8_encode2(b[0], b[1]);
                }
                kc[k] = hi2[0] | (hi2[1] << 16);
                const uint32_t kd = lo2[0] | (lo2[1] << 16);
                if (__any_sync(~0u, kc[k] != kd) && tw + k >= t && tw + k < end) {
                    uint32_t out = 0, ask = 0;  // ask: the bytes still in doubt
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t c = (kc[k] >> (8 * j)) & 0xFFu;
                        const uint32_t c0 = (kd >> (8 * j)) & 0xFFu;
                        if (c != c0) {
                            const float border = 0.5f * (p8_floats2(c).x + p8_floats2(c0).x);  // exact
                            const float small = low[k][j] * inv_k, gap = fmaf(y[k][j], inv_k, -border) + small;
                            if (!(fabsf(gap) > fmaf(err[k][j], inv_k, 0x1p-22f * fabsf(small)))) ask |= 0xFFu << (8 * j);
                            c = gap > 0.f ? c : c0;
                        }
                        out |= c << (8 * j);
                    }
                    kc[k] = out;
                    if (__any_sync(~0u, ask != 0u)) {
                        float x[4], xb[4];
                        ap_floats(kr[k], x);
                        a8_mates(l, x, xb);
                        const uint32_t exact = a8_codes_f64(A, tw + k, make_float4(x[0], x[1], x[2], x[3]), make_float4(xb[0], xb[1], xb[2], xb[3]), lane, ek);
                        kc[k] = (out & ~ask) | (exact & ask);
                    }
                }
                if (tw + k >= t && tw + k < end) {
                    const int p = 4 * warp + k;
                    *reinterpret_cast<uint32_t *>(unit + p * kPgDim + (((lane >> 2) ^ (p & 7)) << 4) + (lane & 3) * 4) = kc[k];
                }
                const uint32_t va = p8_encode2(v[k][0] * inv_v, v[k][1] * inv_v), vb = p8_encode2(v[k][2] * inv_v, v[k][3] * inv_v);
                const int sh = 8 * k;
                vw[0] |= (va & 0xFFu) << sh;
                vw[1] |= (va >> 8) << sh;
                vw[2] |= (vb & 0xFFu) << sh;
                vw[3] |= (vb >> 8) << sh;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) s_v[(l.d0 + j) * kA8VRow + warp] = vw[j];
            __syncthreads();
            // V's row: new bytes i0 .. i0 + n - 1, earlier ones under the scale as it is now, later ones as they were
            uint32_t row[4], was[4] = {old.x, old.y, old.z, old.w};
            const float down_v = p8_pow2(ev0 - ev), down_k = p8_pow2(ek0 - ek);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int a = min(max(i0 - 4 * w, 0), 4), b = min(max(i0 + n - 4 * w, 0), 4);  // new bytes of the word
                const uint32_t ma = a < 4 ? ~0u << (8 * a) : 0u, mb = b < 4 ? ~0u << (8 * b) : 0u, fresh = ma & ~mb;
                uint32_t keep = was[w];
                if (i0 > 0 && ev > ev0 && a > 0) {
                    const uint32_t again = a8_again(keep, down_v);
                    keep = (again & ~ma) | (keep & ma);
                }
                row[w] = (s_v[tid * kA8VRow + w] & fresh) | (keep & ~fresh);
            }
            *reinterpret_cast<uint4 *>(unit + kP8VCodes + 16 * tid) = make_uint4(row[0], row[1], row[2], row[3]);
            if (i0 > 0 && ek > ek0)
                for (int i = tid; i < i0 * (kPgDim / 4); i += kA8Threads) {
                    uint32_t *const w = reinterpret_cast<uint32_t *>(unit) + i;
                    *w = a8_again(*w, down_k);
                }
            if (tid == 0) *reinterpret_cast<float2 *>(unit + kP8Scales) = make_float2(p8_pow2(ek), p8_pow2(ev));
            // (s_top is written again only behind the barrier above; s_v only behind that of the next head's s_top)
        }
        t = end;
    }
}

int paged8_append(const void *qkv, int dtype, int64_t ld, int T, int Hq, int Hkv, const svd_rope *rope,
                  const int32_t *positions, int64_t positions_ld, const int32_t *kv_len, const int32_t *q_start, int R,
                  const int32_t *table, int width, void *pages, int page, int64_t n_pages, void *q, int32_t *status,
                  cudaStream_t stream) {
    if (!qkv || !kv_len || !q_start || !table || !pages || (dtype != SVD_F32 && dtype != SVD_BF16) || T < 0 || Hq < 0 ||
        Hq > 4096 || !pg_pool_ok(Hkv, page, n_pages) || (Hq > 0 && !q) || R < 1 || R > SVD_PAGED_MAX_REQUESTS || width < 1 ||
        (int64_t)width * page > INT32_MAX)
        return SVD_ERR_INVALID_ARG;
    const int64_t heads = (int64_t)Hq + 2 * Hkv;
    const int lane_bytes = dtype == SVD_F32 ? 16 : 8;
    if (!aligned16(qkv) || !aligned16(pages) || !aligned16(q) || ld < heads * kPgDim ||
        (ld * (lane_bytes / 4)) % lane_bytes != 0)
        return SVD_ERR_INVALID_ARG;
    A8Args A = {};
    if (!rope_set(&A.rope, rope, positions, positions_ld, T)) return SVD_ERR_INVALID_ARG;
    if (T == 0) return SVD_OK;
    const int sms = sm_count();
    if (sms < 1) return SVD_ERR_CUDA;
    A.qkv = qkv;
    A.ld = ld;
    A.kv_len = kv_len;
    A.q_start = q_start;
    A.table = table;
    A.pages = (uint8_t *)pages;
    A.q = (__nv_bfloat16 *)q;
    A.status = status;
    A.n_pages = n_pages;
    A.T = T;
    A.R = R;
    A.width = width;
    A.Hq = Hq;
    A.Hkv = Hkv;
    A.page = page;
    // Few tokens: a CTA to each token and kv head, and to each four of its query heads.  Many: sixteen tokens share a
    // CTA, and two kv heads or eight query heads their angles.
    const bool many = (int64_t)T * Hkv > 24ll * sms;
    A.block = many ? 16 : 1;
    A.q_heads = many ? 8 : 4;
    A.kv_heads = many && Hkv > 1 ? 2 : 1;
    A.q_parts = (Hq + A.q_heads - 1) / A.q_heads;
    const dim3 grid((unsigned)((T + A.block - 1) / A.block), (unsigned)(A.q_parts + (Hkv + A.kv_heads - 1) / A.kv_heads));
    if (dtype == SVD_F32)
        SVD_CUDA_TRY(launch(paged8_append_kernel<float>, grid, dim3(kA8Threads), 0, stream, true, A));
    else
        SVD_CUDA_TRY(launch(paged8_append_kernel<__nv_bfloat16>, grid, dim3(kA8Threads), 0, stream, true, A));
    return SVD_OK;
}

// ---- read-back -----------------------------------------------------------------------------
// One warp per slot and kv head; a lane's four dimensions of K and of V.
__global__ void __launch_bounds__(256) paged8_read_kernel(const int64_t *__restrict__ slots, int T, int Hkv,
                                                          const uint8_t *__restrict__ pages, int page, int64_t n_slots,
                                                          float *__restrict__ k, float *__restrict__ v) {
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    griddep_wait();
    if (w >= (int64_t)T * Hkv) return;
    const int64_t t = w / Hkv, slot = slots[t];
    const int h = (int)(w - t * Hkv);
    float4 ko = {0.f, 0.f, 0.f, 0.f}, vo = {0.f, 0.f, 0.f, 0.f};
    if (slot >= 0 && slot < n_slots) {
        const int64_t pg = slot / page;
        const int off = (int)(slot - pg * page), pos = off & 15;
        const uint8_t *const unit = pages + ((pg * Hkv + h) * (page >> 4) + (off >> 4)) * (int64_t)kP8UnitBytes;
        const uint32_t kc = *reinterpret_cast<const uint32_t *>(unit + pos * kPgDim + (((lane >> 2) ^ (pos & 7)) << 4) + (lane & 3) * 4);
        const float2 sc = *reinterpret_cast<const float2 *>(unit + kP8Scales);
        const uint8_t *const vr = unit + kP8VCodes + 64 * lane + pos;
        const uint32_t v01 = vr[0] | (uint32_t)vr[16] << 8, v23 = vr[32] | (uint32_t)vr[48] << 8;
        const float2 k01 = p8_floats2(kc & 0xFFFFu), k23 = p8_floats2(kc >> 16), w01 = p8_floats2(v01), w23 = p8_floats2(v23);
        ko = make_float4(k01.x * sc.x, k01.y * sc.x, k23.x * sc.x, k23.y * sc.x);
        vo = make_float4(w01.x * sc.y, w01.y * sc.y, w23.x * sc.y, w23.y * sc.y);
    }
    reinterpret_cast<float4 *>(k)[w * 32 + lane] = ko;
    reinterpret_cast<float4 *>(v)[w * 32 + lane] = vo;
}

int paged8_read(const int64_t *slots, int T, int Hkv, const void *pages, int page, int64_t n_pages, float *k, float *v,
                cudaStream_t stream) {
    if (!slots || !pages || !k || !v || T < 0 || !pg_pool_ok(Hkv, page, n_pages) || !aligned16(pages) || !aligned16(k) ||
        !aligned16(v))
        return SVD_ERR_INVALID_ARG;
    if (T == 0) return SVD_OK;
    const int64_t grid = ((int64_t)T * Hkv + 7) / 8;
    if (grid > INT32_MAX) return SVD_ERR_INVALID_ARG;
    SVD_CUDA_TRY(launch(paged8_read_kernel, dim3((unsigned)grid), dim3(256), 0, stream, true, slots, T, Hkv,
                        (const uint8_t *)pages, page, n_pages * page, k, v));
    return SVD_OK;
}

}  // namespace svd
