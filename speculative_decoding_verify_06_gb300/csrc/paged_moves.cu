// paged_moves.cu -- pages on the move: forking requests, compacting a pool, and the copies of page contents that
// both ask for, whatever a page holds.
//
// A fork gives every child pages of its own, so appends of different requests never meet in a page and no page
// needs a count of its readers; the price is the copy, which runs at the rate of memory.
#include "paged.cuh"

namespace svd {

constexpr int kMvChunk = 1024;  // outputs per work item

// ---- forking ---------------------------------------------------------------------------------
// A child holds p0 = ceil(held / page) pages and gets p1 = ceil(keep of its parent / page): its own first, surplus ones go
// back to the stack of free pages, missing ones come from its top, both in (request, page) order as for the block
// tables.  One launch, every CTA with all sums for itself (up to 4096 requests), each output a function of
// the sums and the inputs.  What bounds it is latency: a launch and three block-wide sums; 3 us for two requests, 9 from cold
// caches for 64 requests of up to 64 pages.
struct FkArgs {
    const int32_t *held, *window, *emitted, *parent, *table, *free_ids, *n_free;
    int32_t *held_out, *window_out, *table_out, *free_out, *n_free_out, *from, *to, *n_copies, *status;
    int R, page, width, n_pages;
};
constexpr uint8_t kFkStays = 0xFF;  // in place of a status: the request is no child

// A request that becomes another's copy: any parent but itself and none.
__device__ __forceinline__ bool fk_child(int p, int r) { return p >= 0 && p != r; }

__global__ void __launch_bounds__(kTbThreads) paged_fork_kernel(const FkArgs A) {
    extern __shared__ int sm[];
    __shared__ unsigned long long s_w[kTbWarps];
    const int R = A.R, tid = threadIdx.x;
    int *const s_keep = sm, *const s_p0 = sm + R, *const s_p1 = sm + 2 * R, *const s_take = sm + 3 * R;
    int *const s_give = sm + 4 * R, *const s_copy = sm + 5 * R;  // exclusive sums
    uint8_t *const s_st = reinterpret_cast<uint8_t *>(sm + 6 * R);
    griddep_wait();

    unsigned long long page_sum = 0, total;
    const long long room = (long long)A.width * A.page;  // < 2^31
    for (int base = 0; base < R; base += kTbThreads) {
        const int r = base + tid;
        uint32_t p0 = 0, p1 = 0;
        if (r < R) {
            const int p = A.parent[r];
            uint32_t st = kFkStays;
            int keep = 0;
            if (fk_child(p, r)) {
                const int mine = A.held[r];
                bool ok = p < R && mine >= 0 && mine <= room;
                if (ok) {
                    // what the parent keeps: its last window's count, where it has one (a window of -d: d positions go)
                    const long long held = A.held[p], w = A.window ? A.window[p] : 0, win = w < 0 ? -w : w;
                    const long long emi = w <= 0 ? 0 : A.emitted ? A.emitted[p] : w;
                    ok = !fk_child(A.parent[p], p) && emi >= 0 && emi <= win && win <= held && held <= room;
                    keep = (int)(held - win + emi);
                }
                st = ok ? 0 : SVD_ST_BAD_REQUEST;
                if (ok) {
                    p0 = ((uint32_t)mine + A.page - 1) / (uint32_t)A.page;
                    p1 = ((uint32_t)keep + A.page - 1) / (uint32_t)A.page;
                }
            }
            s_keep[r] = keep;
            s_p0[r] = (int)p0;
            s_p1[r] = (int)p1;
            s_st[r] = (uint8_t)st;
        }
        const uint32_t take = p1 > p0 ? p1 - p0 : 0, give = p0 > p1 ? p0 - p1 : 0;
        const unsigned long long sum = page_sum + tb_scan(((unsigned long long)give << 32) | take, &total, s_w);
        page_sum += total;
        if (r < R) {
            s_take[r] = (int)((uint32_t)sum - take);
            s_give[r] = (int)((uint32_t)(sum >> 32) - give);
        }
    }
    __syncthreads();
    const int n_free = min(max(*A.n_free, 0), A.n_pages);
    const int top = n_free + (int)(page_sum >> 32);
    // A child that takes pages gets them if all that was asked before it and its own fits.
    unsigned long long copies = 0, took = 0;
    for (int base = 0; base < R; base += kTbThreads) {
        const int r = base + tid;
        int take = 0, mine = 0;
        if (r < R) {
            take = max(s_p1[r] - s_p0[r], 0);
            if (take > 0 && s_take[r] + take > top) {
                s_st[r] = SVD_ST_NO_PAGES;
                take = 0;
            }
            if (s_st[r] == 0) mine = s_p1[r];
        }
        const unsigned long long sum =
            tb_scan(((unsigned long long)(uint32_t)take << 32) | (uint32_t)mine, &total, s_w);
        if (r < R) s_copy[r] = (int)((uint32_t)copies + (uint32_t)sum) - mine;
        copies += (uint32_t)total;
        took += total >> 32;
    }
    __syncthreads();
    const int n_copies = (int)copies, left = top - (int)took;

    // The stack: the free ids, then the pages given back.
    auto stack = [&](int i) -> int {
        if (i < n_free) return A.free_ids[i];
        const int j = i - n_free, r = tb_last_le(s_give, R, j);
        return A.table[(int64_t)r * A.width + s_p1[r] + j - s_give[r]];
    };
    auto entry = [&](int r, int col) -> int {
        if (s_st[r]) return A.table[(int64_t)r * A.width + col];
        if (col >= s_p1[r]) return -1;
        return col < s_p0[r] ? A.table[(int64_t)r * A.width + col] : stack(top - 1 - s_take[r] - (col - s_p0[r]));
    };

    if (blockIdx.x == 0) {
        for (int r = tid; r < R; r += kTbThreads) {
            const uint32_t st = s_st[r];
            A.status[r] = st == kFkStays ? 0 : (int)st;
            A.held_out[r] = st ? A.held[r] : s_keep[r];
            A.window_out[r] = st ? (A.window ? A.window[r] : 0) : 0;
        }
        if (tid == 0) {
            *A.n_free_out = left;
            *A.n_copies = n_copies;
        }
    }
    const uint32_t row_items = (A.width + kMvChunk - 1) / kMvChunk, t_items = (uint32_t)R * row_items;  // < 2^31
    const uint32_t p_items = (A.n_pages + kMvChunk - 1) / kMvChunk;
    for (uint32_t it = blockIdx.x; it < t_items + 2 * p_items; it += gridDim.x) {
        if (it < t_items) {
            const int r = (int)(it / row_items), c0 = (int)(it - r * row_items) * kMvChunk, c1 = min(c0 + kMvChunk, A.width);
            for (int c = c0 + tid; c < c1; c += kTbThreads) A.table_out[(int64_t)r * A.width + c] = entry(r, c);
        } else if (it < t_items + p_items) {
            const int i0 = (int)(it - t_items) * kMvChunk, i1 = min(i0 + kMvChunk, A.n_pages);
            for (int i = i0 + tid; i < i1; i += kTbThreads) A.free_out[i] = i < left ? stack(i) : -1;
        } else {
            const int i0 = (int)(it - t_items - p_items) * kMvChunk, i1 = min(i0 + kMvChunk, A.n_pages);
            for (int i = i0 + tid; i < i1; i += kTbThreads) {
                int from = -1, to = -1;
                if (i < n_copies) {
                    const int r = tb_last_le(s_copy, R, i), col = i - s_copy[r];
                    from = A.table[(int64_t)A.parent[r] * A.width + col];
                    to = entry(r, col);
                }
                A.from[i] = from;
                A.to[i] = to;
            }
        }
    }
}

static bool mv_sizes_ok(int R, int page, int width, int64_t n_pages) {
    return R >= 1 && R <= SVD_PAGED_MAX_REQUESTS && pg_page_size_ok(page) && width >= 1 &&
           (int64_t)width * page <= INT32_MAX && (int64_t)width * R <= INT32_MAX && n_pages >= 1 &&
           n_pages <= (int64_t)1 << 30;
}
static int64_t mv_items(int64_t n) { return (n + kMvChunk - 1) / kMvChunk; }

int paged_fork(const int32_t *held, const int32_t *window, const int32_t *emitted, const int32_t *parent, int R,
               int page, const int32_t *table, int width, const int32_t *free_ids, const int32_t *n_free,
               int64_t n_pages, int32_t *held_out, int32_t *window_out, int32_t *table_out, int32_t *free_out,
               int32_t *n_free_out, int32_t *copy_from, int32_t *copy_to, int32_t *n_copies, int32_t *status,
               cudaStream_t stream) {
    if (!held || !parent || !table || !free_ids || !n_free || !held_out || !window_out || !table_out || !free_out ||
        !n_free_out || !copy_from || !copy_to || !n_copies || !status || !mv_sizes_ok(R, page, width, n_pages))
        return SVD_ERR_INVALID_ARG;
    if (held_out == held || window_out == window || table_out == table || free_out == free_ids || n_free_out == n_free ||
        copy_from == copy_to)
        return SVD_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms < 1) return SVD_ERR_CUDA;
    const FkArgs A = {held, window, emitted, parent, table, free_ids, n_free, held_out, window_out, table_out, free_out,
                      n_free_out, copy_from, copy_to, n_copies, status, R, page, width, (int)n_pages};
    const size_t smem = (size_t)R * 25 + 8;
    if (smem > kPlainSmem) SVD_CUDA_TRY(allow_smem<paged_fork_kernel>((size_t)SVD_PAGED_MAX_REQUESTS * 25 + 8));
    const int64_t work = (int64_t)R * mv_items(width) + 2 * mv_items(n_pages);
    const int grid = (int)(work < 2 * sms ? work : 2 * sms);
    SVD_CUDA_TRY(launch(paged_fork_kernel, dim3(grid), dim3(kTbThreads), smem, stream, true, A));
    return SVD_OK;
}

// ---- compacting ------------------------------------------------------------------------------
// U pages are in use.  The used ids from U on move, in ascending order, to the unused ids below U, in ascending
// order; as many as there are of the others.  One launch: every CTA marks the used ids of the whole table in a bit
// map in shared memory and sums it, and then answers for its share of the outputs by itself: the place of an id
// among its kind from the sums, and the unused id of a place by a search in them.  Nothing is handed from CTA to
// CTA; the table's entries are read by each, from L2.  What bounds it is latency, of those reads and of atomics on shared
// memory: 13 us for 48 requests of up to 512 pages, beside 190 for the copies.
struct CpArgs {
    const int32_t *held, *table;
    int32_t *table_out, *free_out, *n_free_out, *from, *to, *n_copies;
    int R, page, width, n_pages;
};

__global__ void __launch_bounds__(kTbThreads) paged_compact_kernel(const CpArgs A) {
    extern __shared__ uint32_t bits[];
    __shared__ unsigned long long s_w[kTbWarps];
    __shared__ int s_pre[kTbThreads + 1];  // used ids before each thread's words
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int words = (A.n_pages + 31) >> 5, per = (words + kTbThreads - 1) / kTbThreads;
    for (int i = tid; i < words; i += kTbThreads) bits[i] = 0u;
    __syncthreads();
    griddep_wait();
    auto pages_of = [&](int r) -> int {
        const int h = A.held[r];
        return h <= 0 ? 0 : min((int)(((uint32_t)h + A.page - 1) / (uint32_t)A.page), A.width);
    };
    // A row to a warp, or few rows to the whole CTA one after the other.
    const bool wide = A.R < kTbWarps;
    for (int r = wide ? 0 : warp; r < A.R; r += wide ? 1 : kTbWarps) {
        const int n = pages_of(r);
        const int32_t *const row = A.table + (int64_t)r * A.width;
#pragma unroll 8
        for (int c = wide ? tid : lane; c < n; c += wide ? kTbThreads : 32) {
            const int id = row[c];
            if (id >= 0 && id < A.n_pages) atomicOr(bits + (id >> 5), 1u << (id & 31));
        }
    }
    __syncthreads();
    int mine = 0;
    for (int i = tid * per; i < min((tid + 1) * per, words); ++i) mine += __popc(bits[i]);
    unsigned long long total;
    const unsigned long long upto = tb_scan((unsigned long long)mine, &total, s_w);
    s_pre[tid] = (int)upto - mine;
    if (tid == 0) s_pre[kTbThreads] = (int)total;
    __syncthreads();
    const int used = (int)total;
    // Used ids below id (id <= 32 words).
    auto before = [&](int id) -> int {
        const int w = id >> 5, t = min(w / per, kTbThreads - 1);
        int n = s_pre[t];
        for (int i = t * per; i < w; ++i) n += __popc(bits[i]);
        return (id & 31) ? n + __popc(bits[w] & ((1u << (id & 31)) - 1u)) : n;
    };
    const int low = before(used), moves = used - low;
    // The unused id with j unused ones before it.
    auto unused = [&](int j) -> int {
        int a = 0, b = kTbThreads;  // 32 per t - s_pre[t] unused ids lie before thread t's words
        while (b - a > 1) {
            const int mid = (a + b) >> 1;
            if (min(mid * per, words) * 32 - s_pre[mid] <= j) a = mid; else b = mid;
        }
        j -= a * per * 32 - s_pre[a];
        int w = a * per;
        for (; w < words - 1; ++w) {
            const int n = 32 - __popc(bits[w]);
            if (j < n) break;
            j -= n;
        }
        uint32_t m = ~bits[w];
        for (; j > 0; --j) m &= m - 1u;
        return w * 32 + __ffs(m) - 1;
    };

    if (blockIdx.x == 0 && tid == 0) {
        *A.n_free_out = A.n_pages - used;
        *A.n_copies = moves;
    }
    const uint32_t row_items = (A.width + kMvChunk - 1) / kMvChunk, t_items = (uint32_t)A.R * row_items;  // < 2^31
    const uint32_t p_items = (A.n_pages + kMvChunk - 1) / kMvChunk;
    for (uint32_t it = blockIdx.x; it < t_items + 2 * p_items; it += gridDim.x) {
        if (it < t_items) {
            const int r = (int)(it / row_items), c0 = (int)(it - r * row_items) * kMvChunk, c1 = min(c0 + kMvChunk, A.width);
            const int n = pages_of(r);
            for (int c = c0 + tid; c < c1; c += kTbThreads) {
                const int64_t at = (int64_t)r * A.width + c;
                int id = -1;
                if (c < n) {
                    id = A.table[at];
                    if (id >= used && id < A.n_pages) id = unused(before(id) - low);
                }
                A.table_out[at] = id;
            }
        } else if (it < t_items + p_items) {
            const int i0 = (int)(it - t_items) * kMvChunk, i1 = min(i0 + kMvChunk, A.n_pages);
            for (int i = i0 + tid; i < i1; i += kTbThreads) A.free_out[i] = i < A.n_pages - used ? A.n_pages - 1 - i : -1;
        } else {
            const int i0 = (int)(it - t_items - p_items) * kMvChunk, i1 = min(i0 + kMvChunk, A.n_pages);
            for (int i = i0 + tid; i < i1; i += kTbThreads) {
                const bool in = (bits[i >> 5] >> (i & 31)) & 1u;
                const int n = before(i);
                if (i >= used && in) A.from[n - low] = i;
                if (i < used && !in) A.to[i - n] = i;
                if (i >= moves) A.from[i] = A.to[i] = -1;
            }
        }
    }
}

int paged_compact(const int32_t *held, int R, int page, const int32_t *table, int width, int64_t n_pages,
                  int32_t *table_out, int32_t *free_out, int32_t *n_free_out, int32_t *copy_from, int32_t *copy_to,
                  int32_t *n_copies, cudaStream_t stream) {
    if (!held || !table || !table_out || !free_out || !n_free_out || !copy_from || !copy_to || !n_copies ||
        !mv_sizes_ok(R, page, width, n_pages) || table_out == table || copy_from == copy_to)
        return SVD_ERR_INVALID_ARG;
    if (n_pages > SVD_PAGED_COMPACT_MAX_PAGES) return SVD_ERR_UNSUPPORTED;
    const int sms = sm_count();
    if (sms < 1) return SVD_ERR_CUDA;
    const CpArgs A = {held, table, table_out, free_out, n_free_out, copy_from, copy_to, n_copies, R, page, width,
                      (int)n_pages};
    const size_t smem = ((size_t)n_pages + 31) / 32 * 4;
    if (smem > kPlainSmem) SVD_CUDA_TRY(allow_smem<paged_compact_kernel>((size_t)SVD_PAGED_COMPACT_MAX_PAGES / 8));
    const int64_t work = (int64_t)R * mv_items(width) + 2 * mv_items(n_pages);
    const int grid = (int)(work < sms ? work : sms);
    SVD_CUDA_TRY(launch(paged_compact_kernel, dim3(grid), dim3(kTbThreads), smem, stream, true, A));
    return SVD_OK;
}

// ---- copying ---------------------------------------------------------------------------------
// A page is cut into equal parts of up to 16 KB.  Work items, ordered by copy, pool and part; a CTA takes every
// grid-th.  A thread has four 16-byte loads in flight.  Bounded by memory: every byte is read once and written once, and a
// page that goes to several others is read from memory once if the parts in flight lie close together, so that more CTAs
// are not better: 64 requests forked from eight of up to 4K, 860 MB written, 172 us with four CTAs to an SM (0.85 of the copy
// peak), 164 with three, 195 with eight; a compaction of 640 MB 190 us (1.0), 203 and 207.  A CTA for every part
// that the list has room for: 151, but 276 for the compaction, whose list is two thirds empty.  Loads of the next part ahead of the stores
// of this one: 189 and 208.
constexpr int kPcThreads = 256;
constexpr int kPcDeep = 4;
constexpr int kPcPart = kPcThreads * 16 * kPcDeep;
constexpr int kPcCtas = 4;  // to an SM

struct PcArgs {
    void *pool[SVD_PAGED_MAX_POOLS];
    const int32_t *from, *to, *n_copies;
    int64_t page_bytes, n_pages;
    int pools, most, parts, part;  // parts of a page, bytes of one
};

__global__ void __launch_bounds__(kPcThreads) paged_copy_kernel(const __grid_constant__ PcArgs A) {
    griddep_wait();
    const int n = min(max(*A.n_copies, 0), A.most);
    const int64_t per = (int64_t)A.pools * A.parts, total = n * per;
    for (int64_t it = blockIdx.x; it < total; it += gridDim.x) {
        const int64_t copy = it / per;
        const int rest = (int)(it - copy * per), pool = rest / A.parts, part = rest - pool * A.parts;
        const int64_t from = A.from[copy], to = A.to[copy];
        if (from < 0 || from >= A.n_pages || to < 0 || to >= A.n_pages || from == to) continue;
        const int64_t at = (int64_t)part * A.part;
        const int left = (int)min((int64_t)A.part, A.page_bytes - at) - (int)threadIdx.x * 16;  // bytes from this thread's first
        uint8_t *const base = reinterpret_cast<uint8_t *>(A.pool[pool]) + at + threadIdx.x * 16;
        const uint8_t *const src = base + from * A.page_bytes;
        uint8_t *const dst = base + to * A.page_bytes;
        uint4 v[kPcDeep];
#pragma unroll
        for (int j = 0; j < kPcDeep; ++j)
            if (j * (kPcThreads * 16) < left) v[j] = *reinterpret_cast<const uint4 *>(src + j * (kPcThreads * 16));
#pragma unroll
        for (int j = 0; j < kPcDeep; ++j)
            if (j * (kPcThreads * 16) < left) __stcs(reinterpret_cast<uint4 *>(dst + j * (kPcThreads * 16)), v[j]);
    }
}

int paged_copy(void *const *pools, int n_pools, int64_t page_bytes, int64_t n_pages, const int32_t *from,
               const int32_t *to, const int32_t *n_copies, int64_t most, cudaStream_t stream) {
    if (!pools || !from || !to || !n_copies || n_pools < 1 || page_bytes < 16 || page_bytes % 16 ||
        page_bytes > (int64_t)1 << 30 || n_pages < 1 || n_pages > (int64_t)1 << 30 || most < 0 || most > (int64_t)1 << 30)
        return SVD_ERR_INVALID_ARG;
    for (int i = 0; i < n_pools; ++i)
        if (!pools[i] || !aligned16(pools[i])) return SVD_ERR_INVALID_ARG;
    if (most == 0) return SVD_OK;
    const int sms = sm_count();
    if (sms < 1) return SVD_ERR_CUDA;
    for (int p0 = 0; p0 < n_pools; p0 += SVD_PAGED_MAX_POOLS) {
        PcArgs A = {};
        A.pools = n_pools - p0 < SVD_PAGED_MAX_POOLS ? n_pools - p0 : SVD_PAGED_MAX_POOLS;
        for (int i = 0; i < A.pools; ++i) A.pool[i] = pools[p0 + i];
        A.from = from;
        A.to = to;
        A.n_copies = n_copies;
        A.page_bytes = page_bytes;
        A.n_pages = n_pages;
        A.most = (int)most;
        A.parts = (int)((page_bytes + kPcPart - 1) / kPcPart);
        A.part = (int)align_up((size_t)((page_bytes + A.parts - 1) / A.parts), 16);
        const int64_t work = most * A.pools * A.parts, fit = (int64_t)kPcCtas * sms;
        SVD_CUDA_TRY(launch(paged_copy_kernel, dim3((unsigned)(work < fit ? work : fit)), dim3(kPcThreads), 0, stream, true, A));
    }
    return SVD_OK;
}

}  // namespace svd
