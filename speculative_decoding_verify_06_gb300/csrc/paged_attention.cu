// paged_attention.cu -- attention of ragged verify windows over the paged 4-bit cache.
//
// "Decode is memory-bound ..." ("The ceiling"): at long context the cache joins the weights on
// every pass; "100 tokens per second ..." ("Why a hiring company is writing this"): several
// sequences share the pass.
#include "paged.cuh"

namespace svd {

// One CTA per (token, query head), four warps over the positions in chunks of 32: a lane scores one
// position, then owns four dimensions of the weighted sum; the warps merge at the end.
struct PaArgs {
    const __nv_bfloat16 *q;
    const int32_t *kv_len, *q_start, *table;
    const uint8_t *pages;
    void *out;
    int64_t n_pages;
    int T, R, max_new, width, page, Hq, Hkv, out_bf16;
    float scale;
};

__global__ void __launch_bounds__(128) paged_attention_plain_kernel(const PaArgs A) {
    __shared__ float s_q[kPgDim], s_o[4][kPgDim], s_m[4], s_l[4];
    const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_wait();
    if (t >= A.q_start[A.R]) return;
    int lo = 0, hi = A.R;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (A.q_start[mid] <= t) lo = mid; else hi = mid;
    }
    const int r = lo, n = A.q_start[r + 1] - A.q_start[r], i = t - A.q_start[r];
    if (i < 0 || i >= n || i >= A.max_new) return;
    const int len = min(max(A.kv_len[r], 0), A.width * A.page);
    const int seen = len - n + i + 1;  // positions this token sees
    s_q[tid] = __bfloat162float(A.q[((int64_t)t * A.Hq + h) * kPgDim + tid]) * A.scale;
    __syncthreads();
    const int g = h / (A.Hq / A.Hkv);
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int base = warp * 32; base < seen; base += 128) {
        const int p = base + lane;
        float s = -INFINITY;
        int64_t unit_off = -1;
        if (p < seen) {
            const int pg = A.table[(int64_t)r * A.width + p / A.page];
            if (pg >= 0 && pg < A.n_pages)
                unit_off = (((int64_t)pg * A.Hkv + g) * (A.page >> 4) + ((p % A.page) >> 4)) * kPgUnitBytes;
        }
        if (unit_off >= 0) {
            const uint8_t *u = A.pages + unit_off;
            s = 0.f;
            for (int b = 0; b < 4; ++b) {
                float x = 0.f;
                for (int j = 0; j < 16; ++j) {
                    const int c = u[b * 256 + (p & 15) * 16 + j];
                    x += s_q[32 * b + 2 * j] * ((c & 15) - 8) + s_q[32 * b + 2 * j + 1] * ((c >> 4) - 8);
                }
                s += x * __half2float(*reinterpret_cast<const __half *>(u + kPgKScales + (p & 15) * 8 + 2 * b));
            }
        }
        float mx = s;
        for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, k));
        mx = fmaxf(mx, m);
        const float ref = mx == -INFINITY ? 0.f : mx;
        const float pr = expf(s - ref), f = expf(m - ref);
        float sum = pr;
        for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(~0u, sum, k);
        l = l * f + sum;
        m = mx;
        for (int k = 0; k < 4; ++k) o[k] *= f;
        for (int j = 0; j < 32; ++j) {
            const float pj = __shfl_sync(~0u, pr, j);
            const int64_t uj = __shfl_sync(~0u, unit_off, j);
            if (uj < 0) continue;
            const uint8_t *u = A.pages + uj;
            const int pos = (base + j) & 15;
            const float d = pj * __half2float(*reinterpret_cast<const __half *>(u + kPgVScales + (lane >> 3) * 32 + 2 * pos));
            for (int k = 0; k < 4; ++k) {
                const int c = u[kPgVCodes + ((4 * lane + k) & 63) * 16 + pg_v_byte(pos)];
                o[k] += d * ((lane < 16 ? c & 15 : c >> 4) - 8);
            }
        }
    }
    for (int k = 0; k < 4; ++k) s_o[warp][4 * lane + k] = o[k];
    if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
    __syncthreads();
    float mm = -INFINITY, ll = 0.f, oo = 0.f;
    for (int w = 0; w < 4; ++w) mm = fmaxf(mm, s_m[w]);
    for (int w = 0; w < 4; ++w) {
        const float f = s_m[w] == -INFINITY ? 0.f : expf(s_m[w] - mm);
        ll += s_l[w] * f;
        oo += s_o[w][tid] * f;
    }
    oo = ll > 0.f ? oo / ll : mm == -INFINITY ? 0.f : oo / ll;
    const int64_t at = ((int64_t)t * A.Hq + h) * kPgDim + tid;
    if (A.out_bf16) ((__nv_bfloat16 *)A.out)[at] = __float2bfloat16_rn(oo);
    else ((float *)A.out)[at] = oo;
}

size_t paged_attention_ws_bytes(int Hq, int Hkv, int R, int max_new) {
    if (Hq < 1 || Hkv < 1 || Hq % Hkv || R < 1 || R > SVD_PAGED_MAX_REQUESTS || max_new < 1) return 0;
    return 256;
}

int paged_attention(const uint16_t *q, int T, const int32_t *kv_len, const int32_t *q_start, int R,
                    int max_new, const int32_t *table, int width, const void *pages, int page,
                    int64_t n_pages, int Hq, int Hkv, float scale, void *out, int out_dtype, void *ws,
                    size_t ws_bytes, cudaStream_t stream) {
    if (!q || !kv_len || !q_start || !table || !pages || !out || !aligned16(q) || !aligned16(pages) ||
        !aligned16(out) || !aligned16(ws) || (out_dtype != SVD_F32 && out_dtype != SVD_BF16))
        return SVD_ERR_INVALID_ARG;
    if (T < 0 || R < 1 || R > SVD_PAGED_MAX_REQUESTS || max_new < 1 || width < 1 ||
        !pg_pool_ok(Hkv, page, n_pages) || (int64_t)width * page > INT32_MAX || Hq < 1 || Hq > 4096 ||
        Hq % Hkv || !(scale > 0.f) || scale > 3.4e38f)
        return SVD_ERR_INVALID_ARG;
    const size_t need = paged_attention_ws_bytes(Hq, Hkv, R, max_new);
    if (!ws || ws_bytes < need) return SVD_ERR_WORKSPACE;
    if (T == 0) return SVD_OK;
    const PaArgs A = {(const __nv_bfloat16 *)q, kv_len, q_start, table, (const uint8_t *)pages, out, n_pages,
                      T, R, max_new, width, page, Hq, Hkv, out_dtype == SVD_BF16, scale};
    SVD_CUDA_TRY(launch(paged_attention_plain_kernel, dim3(T, Hq), dim3(128), 0, stream, true, A));
    return SVD_OK;
}

}  // namespace svd
