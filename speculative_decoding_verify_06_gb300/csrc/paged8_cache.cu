// paged8_cache.cu -- the write side of the paged 8-bit cache: rotary positions with several axes joined to the
// append, and the read-back.
//
// "Decode is memory-bound ..." ("The ceiling"): the cache joins the weights on every pass; 8 bits a value stand
// between the 4.5 of the other paged cache and the 16 of none.
//
//   scale = 2^e, e the smallest with 448 2^e >= |y| over the new values of a unit (16 positions of one kv head; K and
//   V apart), and no smaller than the scale that earlier positions of the unit have;  code = e4m3(y / 2^e)
//
// Units.  A scale belongs to 16 positions, so a unit is written by one CTA: the tokens of a request that lie in one unit
// are a run, and the CTA of the run's first token handles all of it, for two kv heads, with four warps to a head that take turns at its
// tokens, keys and values alike.  A lane keeps four dimensions of them in shared memory, where the
// copies bring them while the angles are worked out (in registers, eight positions took 128 of them; cut down to 64, that
// spilled).  The largest magnitudes take one exchange.  Codes of values go through shared memory to whole rows of the
// page.  Where earlier positions keep a smaller scale, their codes are rounded again; what the unit held is fetched ahead of the angles.
//
// Codes.  A key next to the border of two codes must get the code that exact arithmetic gives, or the cache
// would depend on how the angle was rounded.  Rotated keys are worked out in plain fp32, with an error below
// 2.6 * 2^-24 (|x_a| + |x_b|) (cos and sin are off by 2^-25 and 2^-28, the product and the sum by 2^-24); a code is settled where the key plus and minus that bound (the largest of a lane) round alike.  Else (in
// about one of a hundred heads of a token) the warp works the key out as a sum of two floats good to 2^-27 (|x_a| + |x_b|), as the 4-bit append
// does for all, and decides by the distance from the border between the two codes; where that is within the
// bound still, in fp64.  The scale likewise.  Values and dimensions that do not turn are exact as they come.
//
// What bounds it (times in a graph).  4 tokens take 4.6 us, a launch and the chain of one unit: loads that follow from one
// another, angles, rotation, the exchange, the codes.  64 windows of 4 tokens take 8.4 us: every CTA has such a chain, some two, and all are there
// at once.  4099 tokens of 32 + 16 heads in bf16 take 27.5 us for 92 MB, 0.50 of the copy rate: issue at
// half, three CTAs to an SM (by registers), whose warps wait for copies, shared memory and each other (in fp32 43 us
// for 143 MB, 0.50 too).  On the way there, in us: a CTA
// to a unit with all of it in registers 112, halves of a unit 109, one maximum's border cases kept apart from
// the certain ones 60 (a maximum of 448 * 2^e itself, frequent in bf16, had gone the slow way), query heads one at a time 47,
// inputs in shared memory 40, a bound for a lane and not an element 35, angle tables in shared memory 30,
// fp64 for one element at a time 28.7; two warps for the keys of eight positions each and two for their values, of which the latter were done
// in a third of the time, until here.
#include "paged8.cuh"
#include "paged_rope.cuh"

namespace svd {

constexpr int kA8Warps = 8;
constexpr int kA8Threads = 32 * kA8Warps;
constexpr int kA8Pos = 4;                  // positions of a warp, of keys and of values
constexpr int kA8Low = 16 * SVD_ROPE_MAX_PAIRS;
constexpr float kA8Err = 3.f * 0x1p-24f;   // of a rotated key, against |x_a| + |x_b|

struct A8Args {
    const void *qkv;
    int64_t ld;
    const int32_t *kv_len, *q_start, *table;
    uint8_t *pages;
    __nv_bfloat16 *q;
    int32_t *status;
    int64_t n_pages;
    int T, R, width, Hq, Hkv, page;
    int block, kv_parts;  // tokens of a CTA; CTAs of the kv heads (which come first)
    int q_step;           // query heads of all CTAs that share a block of tokens: a warp takes every q_step-th
    int row_bits;         // the power of two that holds all pairs
    RopeArgs rope;
};

// A lane's four dimensions: whether they turn, and where the other ones of their pairs are.
struct A8Lane {
    bool on, up, inter;
    int mate, first;  // lane (-1: interleaved); first pair
};
__device__ __forceinline__ A8Lane a8_lane(const RopeArgs &R, int lane) {
    A8Lane l;
    l.inter = R.interleaved;
    l.on = 4 * lane < 2 * R.pairs;  // pairs is a multiple of four: a lane's dimensions turn alike
    l.up = !l.inter && 4 * lane >= R.pairs;
    l.mate = l.inter ? -1 : l.on ? (l.up ? lane - (R.pairs >> 2) : lane + (R.pairs >> 2)) : lane;
    l.first = !l.on ? 0 : l.inter ? 2 * lane : 4 * lane - (l.up ? R.pairs : 0);
    return l;
}
__device__ __forceinline__ void a8_mates(const A8Lane &l, const float x[4], float xb[4]) {
    if (l.inter) {
        xb[0] = x[1]; xb[1] = x[0]; xb[2] = x[3]; xb[3] = x[2];
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) xb[j] = __shfl_sync(~0u, x[j], l.mate);
    }
}
// cos and (signed) sin of the lane's dimensions, y = x c + xb s, from a token's row of them.
__device__ __forceinline__ void a8_turn(const A8Lane &l, const float2 *row, float c[4], float s[4]) {
    if (l.inter) {
        const float4 a = *reinterpret_cast<const float4 *>(row + l.first);
        c[0] = c[1] = a.x; c[2] = c[3] = a.z;
        s[0] = -a.y; s[1] = a.y; s[2] = -a.w; s[3] = a.w;
    } else {
        const float4 a = *reinterpret_cast<const float4 *>(row + l.first), b = *reinterpret_cast<const float4 *>(row + l.first + 2);
        c[0] = a.x; c[1] = a.z; c[2] = b.x; c[3] = b.z;
        s[0] = a.y; s[1] = a.w; s[2] = b.y; s[3] = b.w;
        if (!l.up) {
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] = -s[j];
        }
    }
}
// What every angle of a CTA needs, where lanes may read different entries at once (as kernel arguments and constants, an
// entry a time, they cost as much as the angles).
struct A8Tables {
    float4 turn[33];
    uint64_t phase[SVD_ROPE_MAX_PAIRS];
    uint8_t axis[SVD_ROPE_MAX_PAIRS];
};
__device__ __forceinline__ void a8_tables(const A8Args &A, A8Tables *s) {
    const int i = threadIdx.x;
    if (i < SVD_ROPE_MAX_PAIRS) {
        s->phase[i] = A.rope.phase[i];
        s->axis[i] = A.rope.axis[i];
    } else if (i < SVD_ROPE_MAX_PAIRS + 33) {
        s->turn[i - SVD_ROPE_MAX_PAIRS] = kApTurn[i - SVD_ROPE_MAX_PAIRS];
    }
}
__device__ __forceinline__ void a8_angles(const A8Args &A, int t, int n, float2 *s_cs, const A8Tables &S) {  // (low parts behind all high ones)
    for (int j = threadIdx.x; j < n << A.row_bits; j += kA8Threads) {
        const int k = j >> A.row_bits, i = j & ((1 << A.row_bits) - 1);
        if (i < A.rope.pairs) {
            uint32_t quad;
            const int64_t r = ap_reduce(A.rope.positions[S.axis[i] * A.rope.positions_ld + t + k], S.phase[i], &quad);
            const float4 cs = ap_cos_sin(r, quad, S.turn);
            s_cs[k * SVD_ROPE_MAX_PAIRS + i] = make_float2(cs.x, cs.z);
            s_cs[kA8Low + k * SVD_ROPE_MAX_PAIRS + i] = make_float2(cs.y, cs.w);
        }
    }
}

// A token's key once more, where plain fp32 leaves something open: as the sum y + low, good to err; what is no number
// counts as 0 and magnitudes end at the largest, as the plain formula gives them.
struct A8Key {
    float y[4], low[4], err[4];
};
__device__ __forceinline__ A8Key a8_key(const A8Args &A, const float x[4], const float xb[4], const float2 *cs_row, int lane) {
    const A8Lane l = a8_lane(A.rope, lane);
    A8Key k;
    float c[4], s[4], cl[4], sl[4];
    if (l.on) {
        a8_turn(l, cs_row, c, s);
        a8_turn(l, cs_row + kA8Low, cl, sl);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        k.y[j] = x[j];
        k.low[j] = k.err[j] = 0.f;
        if (l.on) {
            // what the products and the sum drop, and cos' and sin's low parts
            const float p = __fmul_rn(x[j], c[j]), q = __fmul_rn(xb[j], s[j]), r = __fadd_rn(p, q);
            const float b = __fsub_rn(r, p), lost = __fadd_rn(__fsub_rn(p, __fsub_rn(r, b)), __fsub_rn(q, b));
            const float rest = fmaf(x[j], c[j], -p) + fmaf(xb[j], s[j], -q) + lost + fmaf(x[j], cl[j], xb[j] * sl[j]);
            const float w = __fadd_rn(r, rest);
            k.y[j] = w;
            if (fabsf(w) <= kP8MaxAbs) {
                k.low[j] = __fsub_rn(rest, __fsub_rn(w, r));
                k.err[j] = c[j] == 0.f || s[j] == 0.f ? 0.f : (fabsf(x[j]) + fabsf(xb[j])) * 0x1p-27f;  // (0: exact)
            } else {
                k.y[j] = r;
            }
        }
        k.y[j] = k.y[j] == k.y[j] ? fminf(fmaxf(k.y[j], -kP8MaxAbs), kP8MaxAbs) : 0.f;
    }
    return k;
}
__device__ __forceinline__ float a8_pick(const float x[4], int j) { return j < 2 ? (j ? x[1] : x[0]) : j == 2 ? x[2] : x[3]; }
__device__ __forceinline__ int a8_order(uint32_t c) { return c & 0x80u ? -(int)(c & 0x7Fu) : (int)c; }

// The codes of a token's key under the scale 2^e, as exact arithmetic gives them.
template <typename T>
__device__ __forceinline__ uint32_t a8_codes(const A8Args &A, int t, const T *key, int lane, int e, const float2 *cs_row) {
    float x[4], xb[4];
    ap_floats(ap_raw(key + 4 * lane), x);
    a8_mates(a8_lane(A.rope, lane), x, xb);
    const A8Key k = a8_key(A, x, xb, cs_row, lane);
    const float inv = p8_pow2(-e);
    uint32_t out = 0, ask = 0;  // ask: bytes still in doubt
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float z = k.y[j] * inv, err = k.err[j] * inv, d = err > 0.f ? fmaf(0x1p-23f, fabsf(z), err) : 0.f;
        const uint32_t two = p8_encode2(z - d, z + d), c0 = two & 0xFFu;
        uint32_t c = two >> 8;
        if (c != c0) {
            const float border = 0.5f * (p8_floats2(c).x + p8_floats2(c0).x);  // exact
            const float small = k.low[j] * inv, gap = fmaf(k.y[j], inv, -border) + small;
            if (!(fabsf(gap) > fmaf(0x1p-22f, fabsf(small), err)) || a8_order(c) - a8_order(c0) > 1) ask |= 0xFFu << (8 * j);
            if (!(gap > 0.f)) c = c0;
        }
        out |= c << (8 * j);
    }
    if (!__any_sync(~0u, ask != 0u)) return out;
    uint32_t exact = 0;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {  // (one at a time: side by side they would take registers from what is not rare)
        const double y = ap_turn_f64(A.rope, t, a8_pick(x, j), a8_pick(xb, j), lane, j);
        const double z = fmin(fabs(y) * __longlong_as_double((long long)(1023 - e) << 52), 448.0);
        const int ex = max((int)((unsigned long long)__double_as_longlong(z) >> 52) - 1023, -6);
        const int n = __double2int_rn(z * __longlong_as_double((long long)(1023 + 3 - ex) << 52));
        exact |= ((uint32_t)min(n + 8 * (ex + 6), 0x7E) | (y < 0.0 ? 0x80u : 0u)) << (8 * j);
    }
    return (out & ~ask) | (exact & ask);
}
// Codes of earlier positions under a scale 1 / down times as large.
__device__ __forceinline__ uint32_t a8_again(uint32_t codes, float down) {
    const float2 a = p8_floats2(codes & 0xFFFFu), b = p8_floats2(codes >> 16);
    return p8_encode2(a.x * down, a.y * down) | (p8_encode2(b.x * down, b.y * down) << 16);
}
__device__ __forceinline__ int a8_clamp(int e) { return min(max(e, kP8ExpLo), kP8ExpHi); }
// The largest magnitude of a warp's values (0 where there is none; NaN counts for nothing).
__device__ __forceinline__ float a8_most(float top) { return __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(top))); }

// What the four warps of a head tell each other.
struct A8Head {
    uint4 top[4];        // the largest key, with and less what it may be off, and the largest value
    int need[4];         // exponents that keys ask for, where those leave it open
};
__device__ __forceinline__ void a8_sync(int warp) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + (warp >> 2)) : "memory"); }

// Sixteen or eight bytes into the front of a slot of shared memory.
__device__ __forceinline__ void a8_fetch(float4 *to, const float *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void a8_fetch(float4 *to, const __nv_bfloat16 *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void a8_fetched() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// The lane's four values of a slot as they were copied.
template <typename T>
__device__ __forceinline__ void a8_slot(const float4 *slot, float x[4]) {
    ap_floats(ap_raw(reinterpret_cast<const T *>(slot)), x);
}
template <typename T>
__device__ __forceinline__ void a8_put(float4 *slot, const float x[4]) {  // (values that T holds)
#pragma unroll
    for (int j = 0; j < 4; ++j) reinterpret_cast<T *>(slot)[j] = (T)x[j];
}
__device__ __forceinline__ bool a8_odd(const float x[4]) {  // one is not finite
    return !(fabsf(x[0]) <= 3.4028235e38f) || !(fabsf(x[1]) <= 3.4028235e38f) || !(fabsf(x[2]) <= 3.4028235e38f) ||
           !(fabsf(x[3]) <= 3.4028235e38f);
}

// The exponent (less the lowest) that a warp's part of a run asks for, from its keys in fp64; what is not finite is
// reported.
template <typename T>
__device__ __forceinline__ int a8_need_f64(const A8Args &A, const T *row, int t, int n, int lane) {  // n tokens, four apart
    double top = 0.0;
    for (; n > 0; --n, t += 4) {
        float x[4], xb[4];
        ap_floats(ap_raw(row + (int64_t)t * A.ld + 4 * lane), x);
        a8_mates(a8_lane(A.rope, lane), x, xb);
        if (__any_sync(~0u, a8_odd(x)) && A.status && lane == 0) atomicOr(A.status + t, SVD_ST_NONFINITE);
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
            const double y = ap_turn_f64(A.rope, t, a8_pick(x, j), a8_pick(xb, j), lane, j);
            top = fmax(top, y == y ? fmin(fabs(y), (double)kP8MaxAbs) : 0.0);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmax(top, __shfl_xor_sync(~0u, top, o));
    int e = kP8ExpLo;
    while (e < kP8ExpHi && 448.0 * (double)p8_pow2(e) < top) ++e;
    return e - kP8ExpLo;
}

// What a unit holds that a run in it may change or has to keep: its scales, a dimension's values, and the words of earlier
// positions' keys that the warp would round again.
struct A8Old {
    uint4 v;
    float2 scales;
    uint32_t k[4];
};
__device__ __forceinline__ void a8_old(A8Old *o, const uint8_t *unit, int i0, int n, int turn, int lane) {
    if (n < 16) o->v = *reinterpret_cast<const uint4 *>(unit + kP8VCodes + 16 * (32 * turn + lane));
    if (i0 > 0) o->scales = *reinterpret_cast<const float2 *>(unit + kP8Scales);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (turn + 4 * k < i0) o->k[k] = reinterpret_cast<const uint32_t *>(unit)[32 * (turn + 4 * k) + lane];
}

// A run in a unit: four warps take turns at its tokens, keys and values alike.  row: the head's key of token 0; i0, n: the run's first position and its
// length; t0: its first token, with the others' cos and sin in s_cs; slot, v_slot: the lane's, 32 apart.
template <typename T>
__device__ __forceinline__ void a8_unit(const A8Args &A, const T *row, int i0, int n, int t0, uint8_t *unit, const A8Old &old,
                                        const float2 *s_cs, A8Head *s, float4 *slot, float4 *v_slot, int warp, int lane) {
    const int turn = warp & 3, dim = 32 * turn + lane, mine = (n - turn + 3) >> 2;  // tokens turn, turn + 4 ... of the run
    const int e0 = i0 > 0 ? p8_exponent(old.scales.x) : kP8ExpLo, v0 = i0 > 0 ? p8_exponent(old.scales.y) : kP8ExpLo;
    const A8Lane l = a8_lane(A.rope, lane);
    float top = 0.f, none = 0.f, turned = 0.f;  // none: NaN where a value is not finite; turned: not 0 where an angle is no quarter turn
#pragma unroll 2
    for (int p = 0; p < mine; ++p) {
        float x[4];
        a8_slot<T>(slot + 32 * p, x);
        if (A.rope.pairs) {
            float xb[4];
            a8_mates(l, x, xb);
            if (l.on) {
                float c[4], s[4];
                a8_turn(l, s_cs + (turn + 4 * p) * SVD_ROPE_MAX_PAIRS, c, s);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    turned = fmaxf(turned, fminf(fabsf(c[j]), fabsf(s[j])));
                    x[j] = fmaf(x[j], c[j], xb[j] * s[j]);
                }
            }
            slot[32 * p] = make_float4(x[0], x[1], x[2], x[3]);
        } else if (sizeof(T) == 2) {
            slot[32 * p] = make_float4(x[0], x[1], x[2], x[3]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            top = fmaxf(top, fabsf(x[j]));
            none = fmaf(x[j], 0.f, none);
        }
    }
    // What the lane's keys may be off: a turn keeps the length of a pair, so |x_a| + |x_b| is at most twice the larger of
    // its two keys.
    const float pair = l.inter ? top : fmaxf(top, __shfl_sync(~0u, top, l.mate));
    const bool none_open = turned == 0.f;
    const float off = none_open ? 0.f : fmaf(2.f * kA8Err, pair, 0x1p-23f * top);
    // The largest key: of the exact ones, and of the others with what they may be off (bits of floats that are not negative
    // are ordered as they are).  All ones: something is not finite, or too large, and all of the run's keys are open.
    const float big = a8_most(top), sure = a8_most(none_open ? top : 0.f), near = a8_most(none_open ? 0.f : top), far = a8_most(off);
    const bool wild = __any_sync(~0u, none != 0.f) || big > kP8MaxAbs;
    // The largest value.
    float v_top = 0.f, v_none = 0.f;
#pragma unroll
    for (int p = 0; p < kA8Pos; ++p) {
        if (p >= mine) break;
        float x[4];
        a8_slot<T>(v_slot + 32 * p, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v_top = fmaxf(v_top, fabsf(x[j]));
            v_none = fmaf(x[j], 0.f, v_none);
        }
    }
    if (__any_sync(~0u, v_none != 0.f || v_top > kP8MaxAbs)) {  // what is no number counts as 0, and magnitudes end
        v_top = 0.f;
        for (int p = 0; p < mine; ++p) {
            float x[4];
            a8_slot<T>(v_slot + 32 * p, x);
            if (__any_sync(~0u, a8_odd(x)) && A.status && lane == 0) atomicOr(A.status + t0 + turn + 4 * p, SVD_ST_NONFINITE);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = x[j] == x[j] ? fminf(fmaxf(x[j], -kP8MaxAbs), kP8MaxAbs) : 0.f;
                v_top = fmaxf(v_top, fabsf(x[j]));
            }
            a8_put<T>(v_slot + 32 * p, x);
        }
    }
    v_top = a8_most(v_top);
    if (lane == 0)
        s->top[turn] = make_uint4(wild ? ~0u : __float_as_uint(fmaxf(sure, near > 0.f ? near + far : 0.f)),
                                     wild ? 0u : __float_as_uint(fmaxf(sure, near - far)), __float_as_uint(v_top), 0u);
    a8_sync(warp);
    uint32_t hi = 0, lo = 0, vb = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const uint4 m = s->top[w];
        hi = max(hi, m.x);
        lo = max(lo, m.y);
        vb = max(vb, m.z);
    }

    // Codes of values (slots of no token hold anything: their bytes are not used), and into the warp's slots with them: those of
    // dimension 4l + j at word 40 j + l, so that no two lanes meet in a bank, here or where rows are read.
    uint32_t *const v_codes = reinterpret_cast<uint32_t *>(v_slot - lane);
    const int ve = max(a8_clamp(p8_need(__uint_as_float(vb))), v0);
    {
        const float inv = p8_pow2(-ve);
        uint32_t w[4];
#pragma unroll
        for (int p = 0; p < kA8Pos; p += 2) {
            float a4[4], b4[4];
            a8_slot<T>(v_slot + 32 * p, a4);
            a8_slot<T>(v_slot + 32 * p + 32, b4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t two = p8_encode2(a4[j] * inv, b4[j] * inv);
                if (p) w[j] |= two << 16;
                else w[j] = two;
            }
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) v_codes[40 * j + lane] = w[j];
    }

    // Codes of keys.
    int e = a8_clamp(p8_need(__uint_as_float(hi)));
    uint32_t again = 0;  // positions whose codes are open
    if (hi == ~0u || a8_clamp(p8_need(__uint_as_float(lo))) != e) {
        const int need = a8_need_f64(A, row, t0 + turn, mine, lane);
        if (lane == 0) s->need[turn] = need;
        a8_sync(warp);
        e = max(max(max(s->need[0], s->need[1]), max(s->need[2], s->need[3])) + kP8ExpLo, e0);
        again = (1u << max(mine, 0)) - 1u;
    } else {
        e = max(e, e0);
        const float inv = p8_pow2(-e), d = off * inv;
#pragma unroll 2
        for (int p = 0; p < mine; ++p) {
            const float4 y = slot[32 * p];
            const float y4[4] = {y.x, y.y, y.z, y.w};
            float a[4], b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a[j] = fmaf(y4[j], inv, d);
                b[j] = fmaf(y4[j], inv, -d);
            }
            const uint32_t codes = p8_encode2(a[0], a[1]) | (p8_encode2(a[2], a[3]) << 16);
            const uint32_t other = p8_encode2(b[0], b[1]) | (p8_encode2(b[2], b[3]) << 16);
            if (__any_sync(~0u, codes != other)) again |= 1u << p;
            const int i = i0 + turn + 4 * p;
            *reinterpret_cast<uint32_t *>(unit + i * kPgDim + (((lane >> 2) ^ (i & 7)) << 4) + (lane & 3) * 4) = codes;
        }
    }
    for (; again; again &= again - 1u) {
        const int k = turn + 4 * (__ffs(again) - 1), t = t0 + k, i = i0 + k;
        const uint32_t codes = a8_codes(A, t, row + (int64_t)t * A.ld, lane, e, s_cs + k * SVD_ROPE_MAX_PAIRS);
        *reinterpret_cast<uint32_t *>(unit + i * kPgDim + (((lane >> 2) ^ (i & 7)) << 4) + (lane & 3) * 4) = codes;
    }
    if (e > e0 && i0 > 0) {
        const float down = p8_pow2(e0 - e);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (turn + 4 * k < i0) reinterpret_cast<uint32_t *>(unit)[32 * (turn + 4 * k) + lane] = a8_again(old.k[k], down);
    }

    // Rows of values, a dimension to a lane: new bytes i0 .. i0 + n - 1, earlier ones under the scale as it is now, later
    // ones as they were.
    a8_sync(warp);  // (also: every warp has read the scales)
    uint32_t v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = v_codes[(k - turn) * (2 * kA8Pos * 32 * 4) + 40 * (lane & 3) + (dim >> 2)];
    // in the order of tokens: byte k of the warps' four words is word k
    const uint32_t a01 = __byte_perm(v[0], v[1], 0x5140), a23 = __byte_perm(v[2], v[3], 0x5140);
    const uint32_t b01 = __byte_perm(v[0], v[1], 0x7362), b23 = __byte_perm(v[2], v[3], 0x7362);
    uint32_t w[4] = {__byte_perm(a01, a23, 0x5410), __byte_perm(a01, a23, 0x7632), __byte_perm(b01, b23, 0x5410),
                     __byte_perm(b01, b23, 0x7632)};
    if (i0 > 0) {  // token 0 goes to byte i0
        const int by = 8 * (i0 & 3);
        w[3] = __funnelshift_l(w[2], w[3], by);
        w[2] = __funnelshift_l(w[1], w[2], by);
        w[1] = __funnelshift_l(w[0], w[1], by);
        w[0] <<= by;
        if (i0 & 4) {
            w[3] = w[2];
            w[2] = w[1];
            w[1] = w[0];
        }
        if (i0 & 8) {
            w[3] = w[1];
            w[2] = w[0];
        }
    }
    uint32_t was[4] = {old.v.x, old.v.y, old.v.z, old.v.w};
    if (n < 16) {
        const float down = p8_pow2(v0 - ve);
        const bool grown = i0 > 0 && ve > v0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int a = min(max(i0 - 4 * q, 0), 4), b = min(max(i0 + n - 4 * q, 0), 4);  // new bytes of the word
            const uint32_t ma = a < 4 ? ~0u << (8 * a) : 0u, mb = b < 4 ? ~0u << (8 * b) : 0u, fresh = ma & ~mb;
            if (grown && a > 0) was[q] = (a8_again(was[q], down) & ~ma) | (was[q] & ma);
            w[q] = (w[q] & fresh) | (was[q] & ~fresh);
        }
    }
    reinterpret_cast<uint4 *>(unit + kP8VCodes)[dim] = make_uint4(w[0], w[1], w[2], w[3]);
    if (dim == 0) *reinterpret_cast<float2 *>(unit + kP8Scales) = make_float2(p8_pow2(e), p8_pow2(ve));
}

constexpr size_t kA8Smem = kA8Warps * 2 * kA8Pos * 32 * sizeof(float4) + 2 * kA8Low * sizeof(float2);

template <typename T>
__global__ void __launch_bounds__(kA8Threads, 3) paged8_append_kernel(const __grid_constant__ A8Args A) {
    extern __shared__ float4 s_x[];  // [warp][keys, values][position][lane], then the angles
    __shared__ __align__(16) A8Tables s_tab;
    __shared__ __align__(16) A8Head s_head[2];
    __shared__ int s_r;
    __shared__ int4 s_run;  // of the block's first token that a request has: where the request's tokens begin and end, and its length
    float2 *const s_cs = reinterpret_cast<float2 *>(s_x + kA8Warps * 2 * kA8Pos * 32);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const T *const qkv = reinterpret_cast<const T *>(A.qkv) + 4 * lane;
    const int t0 = blockIdx.x * A.block, t1 = min(t0 + A.block, A.T);
    a8_tables(A, &s_tab);
    if (tid == kA8Threads - 1) s_r = -1;
    __syncthreads();
    griddep_wait();

    if ((int)blockIdx.y >= A.kv_parts) {
        // ---- queries: a warp takes a head of the block's tokens -----------------------------------
        const int first = ((int)blockIdx.y - A.kv_parts) * kA8Warps + warp, end = A.q_start[A.R];
        constexpr int kAhead = sizeof(T) == 2 ? 8 : 4;
        decltype(ap_raw(qkv)) ahead[kAhead];
        auto fetch = [&](int head) {
            const T *const row = qkv + t0 * A.ld + (int64_t)head * kPgDim;
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (head < A.Hq && t0 + k < t1) ahead[k] = ap_raw(row + k * A.ld);
        };
        fetch(first);
        a8_angles(A, t0, t1 - t0, s_cs, s_tab);
        __syncthreads();
        const A8Lane l = a8_lane(A.rope, lane);
        const int n = min(t1, end) - t0;
#pragma unroll 1
        for (int head = first; head < A.Hq; head += A.q_step) {
            const T *const row = qkv + t0 * A.ld + (int64_t)head * kPgDim;
            __nv_bfloat16 *q = A.q + ((int64_t)t0 * A.Hq + head) * kPgDim + 4 * lane;
            for (int g = 0; g < n; g += kAhead) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int t = g + k;
                    if (t >= n) break;
                    float x[4], xb[4];
                    ap_floats(ahead[k], x);
                    if (t0 + t + kAhead < t1) ahead[k] = ap_raw(row + (int64_t)(t + kAhead) * A.ld);
                    if (A.rope.pairs) {
                        a8_mates(l, x, xb);
                        if (l.on) {
                            float c[4], s[4];
                            a8_turn(l, s_cs + t * SVD_ROPE_MAX_PAIRS, c, s);
#pragma unroll
                            for (int j = 0; j < 4; ++j) x[j] = fmaf(x[j], c[j], xb[j] * s[j]);
                        }
                    }
                    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
                    uint2 o;
                    o.x = reinterpret_cast<const uint32_t &>(a);
                    o.y = reinterpret_cast<const uint32_t &>(b);
                    *reinterpret_cast<uint2 *>(q) = o;
                    q += A.Hq * kPgDim;
                }
            }
            fetch(head + A.q_step);
        }
        return;
    }

    // ---- keys and values: the runs that begin in this block of tokens, two kv heads ------------------
    const int h = 2 * (int)blockIdx.y + (warp >> 2), turn = warp & 3;
    const int begin = max(t0, A.q_start[0]);  // (tokens before the first request's belong to none)
    for (int r = tid; r < A.R; r += kA8Threads) {
        const int a = A.q_start[r], b = A.q_start[r + 1];
        if (a <= begin && begin < b) {
            atomicMax(&s_r, r);
            s_run = make_int4(a, b, A.kv_len[r], 0);
        }
    }
    __syncthreads();
    int r = s_r;
    if (r < 0) return;  // behind the last request
    int q0 = s_run.x, q2 = s_run.y, len = s_run.z;
    for (int t = begin; t < t1;) {
        if (q2 <= t) {
            while (r + 1 < A.R && A.q_start[r + 1] <= t) ++r;
            q0 = A.q_start[r];
            q2 = A.q_start[r + 1];
            len = A.kv_len[r];
        }
        const int64_t at = (int64_t)len - ((int64_t)q2 - q0) + ((int64_t)t - q0);  // position of token t
        const int i0 = (int)(at & 15), end = min(t + 16 - i0, min(q2, A.T));
        if (end <= t || t < q0) return;  // (behind the last request, or a q_start that does not ascend)
        if (t != q0 && i0 != 0) {  // the run began in another block
            t = end;
            continue;
        }
        const int n = end - t;  // positions i0 .. i0 + n - 1 of the unit
        int64_t pg = -1;
        if (at >= 0 && at < (int64_t)A.width * A.page) pg = A.table[(int64_t)r * A.width + (uint32_t)at / (uint32_t)A.page];
        const T *const row = qkv + (int64_t)(A.Hq + h) * kPgDim;
        float4 *const slot = s_x + warp * (2 * kA8Pos * 32) + lane, *const v_slot = slot + kA8Pos * 32;
        __syncthreads();  // (of the run before, the angles are read, and the codes of values in all four warps' slots)
        if (h < A.Hkv)
            for (int k = turn, p = 0; k < n; k += 4, ++p) {
                const T *const from = row + (int64_t)(t + k) * A.ld;
                a8_fetch(slot + 32 * p, from);
                a8_fetch(v_slot + 32 * p, from + A.Hkv * kPgDim);
            }
        const bool stored = pg >= 0 && pg < A.n_pages;
        const int place = (int)((uint32_t)at % (uint32_t)A.page) >> 4;
        uint8_t *const unit = A.pages + ((pg * A.Hkv + h) * (A.page >> 4) + place) * (int64_t)kP8UnitBytes;
        A8Old old = {};
        if (stored && h < A.Hkv) a8_old(&old, unit, i0, n, turn, lane);  // (on its way while the angles are worked out)
        a8_angles(A, t, n, s_cs, s_tab);
        a8_fetched();
        __syncthreads();
        if (!stored) {
            if (A.status && h == 0 && warp == 0 && lane < n) atomicOr(A.status + t + lane, SVD_ST_BAD_SLOT);
        } else if (h < A.Hkv) {
            a8_unit(A, row - 4 * lane, i0, n, t, unit, old, s_cs, &s_head[warp >> 2], slot, v_slot, warp, lane);
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
    // As many tokens to a CTA, up to sixteen, as let nearly all CTAs be there at once.
    A.kv_parts = (Hkv + 1) / 2;
    while (1 << A.row_bits < A.rope.pairs) ++A.row_bits;
    int q_parts = (Hq + kA8Warps - 1) / kA8Warps;
    const int parts = A.kv_parts + q_parts;
    A.block = 1;
    while (A.block < 16 && (int64_t)T * parts > 4ll * sms * A.block) A.block *= 2;
    // Two query heads to a warp where that lets all CTAs be there at once, three to an SM (64 windows of 4 tokens, 40 + 16 heads: 9.5 -> 8.45 us;
    // chunks of 4099 tokens, far from that, gain nothing by it: 28.4 -> 28.5).
    const int blocks = (T + A.block - 1) / A.block, half = (q_parts + 1) / 2;
    if ((int64_t)blocks * (A.kv_parts + q_parts) > 3ll * sms && (int64_t)blocks * (A.kv_parts + half) <= 3ll * sms) q_parts = half;
    A.q_step = q_parts * kA8Warps;
    const dim3 grid((unsigned)blocks, (unsigned)(A.kv_parts + q_parts));
    if (dtype == SVD_F32) {
        SVD_CUDA_TRY((allow_smem<paged8_append_kernel<float>>(kA8Smem)));
        SVD_CUDA_TRY(launch(paged8_append_kernel<float>, grid, dim3(kA8Threads), kA8Smem, stream, true, A));
    } else {
        SVD_CUDA_TRY((allow_smem<paged8_append_kernel<__nv_bfloat16>>(kA8Smem)));
        SVD_CUDA_TRY(launch(paged8_append_kernel<__nv_bfloat16>, grid, dim3(kA8Threads), kA8Smem, stream, true, A));
    }
    return SVD_OK;
}

// ---- read-back -----------------------------------------------------------------------------
// One warp per slot and kv head; a lane's four dimensions of K and of V.  1.8 us for 4 tokens, 11.2 for 4099 (42 MB, 34 of them fp32
// written, which stay in L2).  Bounded by the latency of its loads, of which the slot comes first and then codes, scales and single
// bytes of 128 rows of values (long scoreboard 23 an instruction issued, in the profiler; issue 39 %).  More of them in flight did not
// help: two or four slots to a warp with consecutive tokens of one head to a CTA, whose lines of V L1 would then hold, took 12.1 and 12.2, one 11.2.
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
