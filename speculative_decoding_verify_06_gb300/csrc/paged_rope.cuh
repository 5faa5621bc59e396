// paged_rope.cuh -- what the appends to paged caches share: rotary angles of several axes, exactly reduced, and
// rows of activations as they lie in memory.
#pragma once

#include "paged.cuh"

#include <math.h>
#include <string.h>

namespace svd {

struct RopeArgs {
    uint64_t phase[SVD_ROPE_MAX_PAIRS];  // turns per position, as a fraction of 2^64
    uint8_t axis[SVD_ROPE_MAX_PAIRS];
    int pairs, interleaved;
    const int32_t *positions;
    int64_t positions_ld;
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
__device__ __forceinline__ int64_t ap_reduce(int64_t pos, uint64_t phase, uint32_t *quad) {
    const uint64_t ph = (uint64_t)pos * phase, q = (ph + (1ull << 61)) >> 62;
    *quad = (uint32_t)q;
    return (int64_t)(ph - (q << 62));
}
__device__ __forceinline__ int64_t ap_phase(const RopeArgs &A, int t, int i, uint32_t *quad) {
    return ap_reduce(A.positions[A.axis[i] * A.positions_ld + t], A.phase[i], quad);
}

// cos and sin of k / 256 turns (high and low parts), k = 0..32.
static __constant__ float4 kApTurn[33] = {
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
// is left (at most a 512th of a turn), whose fp32 errors count for an 80th.  turn: the table, here or copied to where
// lanes may read different entries at once.
__device__ __forceinline__ float4 ap_cos_sin(int64_t r, uint32_t quad, const float4 *turn) {
    const int k = (int)((r + (1ll << 55)) >> 56);
    const float a = __ll2float_rn(r - ((int64_t)k << 56)) * (6.283185307f * 0x1p-64f), z = a * a;
    float4 e = turn[k < 0 ? -k : k];
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

__device__ __forceinline__ float4 ap_cos_sin(const RopeArgs &A, int t, int i) {
    uint32_t quad;
    const int64_t r = ap_phase(A, t, i, &quad);
    return ap_cos_sin(r, quad, kApTurn);
}

// Four rotated dimensions of a lane in fp64: x (xa) with the other dimensions of their pairs (xo).  (The series are written out
// here and below: through a function for any number of angles, the 4-bit append spilled more.)
__device__ __forceinline__ void ap_turn_f64(const RopeArgs &A, int t, float4 xa, float4 xo, int lane, double y[4]) {
    const float xa4[4] = {xa.x, xa.y, xa.z, xa.w}, xb4[4] = {xo.x, xo.y, xo.z, xo.w};
    const int pairs = A.pairs, d0 = 4 * lane;
    const bool on = d0 < 2 * pairs, up = !A.interleaved && d0 >= pairs;
    double x[4], z[4], c[4], sn[4];
    uint32_t quad[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = A.interleaved ? 2 * lane + (j >> 1) : d0 + j - (up ? pairs : 0);
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
        if (!(A.interleaved ? (j & 1) : up)) ss = -ss;
        const double r = __dadd_rn(__dmul_rn((double)xa4[j], cc), __dmul_rn((double)xb4[j], ss));
        y[j] = on ? r : (double)xa4[j];
    }
}
// One of them, j.
__device__ __forceinline__ double ap_turn_f64(const RopeArgs &A, int t, float xa, float xo, int lane, int j) {
    const int pairs = A.pairs, d0 = 4 * lane;
    if (d0 >= 2 * pairs) return xa;
    const bool up = !A.interleaved && d0 >= pairs;
    uint32_t quad;
    const int64_t r = ap_phase(A, t, A.interleaved ? 2 * lane + (j >> 1) : d0 + j - (up ? pairs : 0), &quad);
    const double x = (double)r * (3.14159265358979323846 * 0x1p-63), z = x * x;
    const double fc[9] = {1.0 / 20922789888000.0, -1.0 / 87178291200.0, 1.0 / 479001600.0, -1.0 / 3628800.0, 1.0 / 40320.0,
                          -1.0 / 720.0, 1.0 / 24.0, -0.5, 1.0};
    const double fs[9] = {1.0 / 355687428096000.0, -1.0 / 1307674368000.0, 1.0 / 6227020800.0, -1.0 / 39916800.0,
                          1.0 / 362880.0, -1.0 / 5040.0, 1.0 / 120.0, -1.0 / 6.0, 1.0};
    double c = fc[0], s = fs[0];
#pragma unroll
    for (int k = 1; k < 9; ++k) {
        c = fma(c, z, fc[k]);
        s = fma(s, z, fs[k]);
    }
    s *= x;
    if (quad & 1) { const double w = s; s = c; c = -w; }
    if (quad & 2) { s = -s; c = -c; }
    if (!(A.interleaved ? (j & 1) : up)) s = -s;
    return __dadd_rn(__dmul_rn((double)xa, c), __dmul_rn((double)xo, s));
}

// Turns per position of a frequency in radians, as a fraction of 2^64 modulo a turn:
// |inv| = m 2^e with a 53-bit m, times 1 / (2 pi) to 2^-128, in integers.
inline uint64_t rope_phase(double inv) {
    const uint64_t c_hi = 0x28BE60DB9391054Aull, c_lo = 0x7F09D5F47D4D3770ull;
    uint64_t u;
    memcpy(&u, &inv, sizeof u);
    const int field = (int)(u >> 52) & 2047;
    if (field == 0) return 0;  // (below 2^-1022: no turn within any position)
    const uint64_t m = (u & ((1ull << 52) - 1)) | 1ull << 52;
    const int e = field - 1075;
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

// Rotary positions as the kernels take them; false where the arguments are out of range.
inline bool rope_set(RopeArgs *out, const svd_rope *rope, const int32_t *positions, int64_t positions_ld, int T) {
    out->positions = positions;
    out->positions_ld = positions_ld;
    if (rope) {
        const svd_rope &r = *rope;
        if (!positions || r.n_pairs < 4 || r.n_pairs > SVD_ROPE_MAX_PAIRS || r.n_pairs % 4 || r.n_axes < 1 ||
            r.n_axes > SVD_ROPE_MAX_AXES || (r.n_axes > 1 && positions_ld != 0 && positions_ld < T))
            return false;
        out->pairs = r.n_pairs;
        out->interleaved = r.interleaved != 0;
        for (int i = 0; i < r.n_pairs; ++i) {
            if (!(fabs(r.inv_freq[i]) < 4294967296.0) || r.axis[i] >= r.n_axes) return false;
            out->phase[i] = rope_phase(r.inv_freq[i]);
            out->axis[i] = r.axis[i];
        }
    }
    return true;
}

}  // namespace svd
