// paged8_attention.cu -- attention of ragged verify windows over the paged 8-bit cache.
//
// "Decode is memory-bound ..." ("The ceiling"): at long context the cache joins the weights on every pass; "100
// tokens per second ..." ("Why a hiring company is writing this"): several sequences share the pass.
//
//   o = sum_j p_j v_j / sum_j p_j,   v_j = sv(j) cv_j,  k_j = sk(j) ck_j,   p_j = 2^(c sk(j) <q, ck_j>),  c = scale log2(e)
//
// with codes c in e4m3 and one power of two sk, sv for 16 positions.  Row tiles, their split over CTAs, segments
// and the join are those of the 4-bit cache's kernel (paged_attention.cuh).
//
// One tile of 128 positions.  Bulk copies bring up to eight units into a ring stage, K and V apart: K codes lie in the pages
// as the K-major operand that tcgen05 reads, 128-byte swizzle and all, so S^T = K Q^T (M = 128 positions) takes them from
// shared memory as they are (kind::f8f6f4).  A query row is split once a segment into two e4m3 parts,
// q = 2^e (hi + lo / 16), which stand side by side as columns of one product.  V becomes fp16 in tensor memory (a lane a
// dimension, two positions a column; four warps), exactly, and O^T += V^T P^T runs on fp16 operands: turning 128 x 128
// codes of V costs as much as splitting P of 24 rows into the three e4m3 parts that fp16's eleven bits fill, and less for
// more rows.  For 128 rows K goes the same way (a lane a position, two dimensions a column), against queries of one fp16
// part under a power of two: half the columns of S to load, and room for all of it (chunks 255 -> 233 us; 64 rows lose by it, 102 -> 119).
//
// Softmax.  A lane holds one position of S for all rows, as in the 4-bit kernel, and the reference of a row moves
// only when a score exceeds it by 15 (p <= 2^15 in between).  What is weighed is t = s + log2 sv(j): P = 2^(t - ref) then
// carries V's scale and O sums codes, whatever the scales of other blocks are, and the row's sum takes
// P / sv(j), in fp32.  Scales are powers of two, so both cost one addition or multiplication of exact numbers.
//
// Rows a mask leaves empty get zeros.  Positions past the length, or on a page outside the pool, are cut out
// of S, and their V codes are replaced by 0, whatever their bytes.
//
// What bounds it (8 kv heads, 40 query heads, times in a graph, of a measured copy rate of 6686 GB/s).  For windows,
// memory: 539 MB at 262K take 93.5 us (0.86; 6.4 TB/s once going), 64 ragged requests of up to 16K 215 us (0.89), 200 short ones with
// fp32 outputs 85 us (0.80).  Some 10 us do not depend on the length: a launch, the first tile's way through copy, products and
// softmax, and the join; one token behind 1500 positions takes 9.0 us, 32K positions 21.  Issue stands at 60 % there.  Where a
// request has few tiles, the borders between segments: 64 requests of up to 512 positions take 29 us for 43 MB.
// For chunks of 512 tokens (128-row tiles), 143 GFLOP in 235 us, 0.32 of the product rate: some 3400 cycles a tile of
// 128 x 128, in which four groups of softmax warps take turns with nothing but one another.  A first prompt, with nothing
// behind it, is furthest from what its products need: 2048 tokens take 334 us for 43 GFLOP (0.07 of the rate), eight of 300
// tokens 127 us for 54 MB.  A segment has 8.5 tiles there, some 60 us of them in all, and one warp brings and splits the 128 query rows of
// every segment but a CTA's first.  fp32 outputs, in tiles of 32 rows, take 548 us for the 2048 tokens.
// Tried and slower or no faster there: groups with barriers of their
// own (304 -> 335), scalar softmax (304 -> 346), row tiles of 96 (378), 64 rows to a lane (297 to 320), the queries' parts as two products
// into the same columns, the second in e5m2 (300), two buffers for P beside two stages in place of three (296 of 296; a prompt of 2048
// 391 -> 406), loads of S by fours.  Registers: 32 for V warps leave 64 to the one that walks the segments (40 and 56: 233 of 235, but
// a prompt of 2048 tokens 344 of 331).  One warp that heard of a segment when its copies began took long
// enough over its queries to hold all others up (281 -> 233): the segments are announced ahead.
#include "paged8.cuh"
#include "paged_attention.cuh"

namespace svd {

constexpr int kP8StageK = kPaTileUnits * 2048;
constexpr int kP8VUnit = kP8UnitBytes - kP8VCodes;  // codes of V and the scales
constexpr int kP8StageV = kPaTileUnits * kP8VUnit;
constexpr int kP8MaxStages = 5;
constexpr int kP8Ring = 16;  // tile and segment descriptors in flight (see the copies)

// S = K Q^T (+)= A[smem] B[smem]^T, e4m3 operands, fp32 accumulators.
__device__ __forceinline__ void p8_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; "
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// As pa_wait(), with all but the first look out of line: the kernel's loops are short of instruction cache (a larger V loop
// costs 200 requests of 2K a seventh).  (Not beside a register split, where the
// compiler takes no calls, nor for fp32 outputs, which lost by it: 91 -> 106 us; bf16 262K 94.6 -> 93.0.)
__device__ __noinline__ bool p8_wait_on(uint32_t bar, uint32_t parity, PaCtl *c) {
    for (uint32_t left = c->limit; left; --left) {
        if (mbar_poll(bar, parity, true)) return true;
        if (pa_stopped(c)) return false;
    }
    if (!pa_stopped(c)) {
        *reinterpret_cast<volatile uint32_t *>(&c->stop) = 1u;
        atomicOr(c->status, 1u);
    }
    return false;
}
template <bool kInline>
__device__ __forceinline__ bool p8_wait(uint32_t bar, uint32_t parity, PaCtl *c) {
    if (kInline) return pa_wait(bar, parity, c);
    bool ok = mbar_poll(bar, parity, true);
    if (!__all_sync(~0u, ok)) ok = __all_sync(~0u, ok || p8_wait_on(bar, parity, c));
    return ok;
}

// n (4 or 8) columns of a warp's lanes.
template <int n>
__device__ __forceinline__ void p8_ld(uint32_t t, float *f) {
    if (n == 8) {
        pa_ld8(t, f);
    } else {
        uint32_t *const v = reinterpret_cast<uint32_t *>(f);
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "r"(t)
                     : "memory");
    }
}
template <int n>
__device__ __forceinline__ void p8_st(uint32_t t, const float *f) {
    const uint32_t *const v = reinterpret_cast<const uint32_t *>(f);
    if (n == 8) pa_st8(t, v);
    else
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(t), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                     : "memory");
}

template <int n>
__device__ __forceinline__ void p8_line(uint8_t *to, const uint32_t *w) {  // n fp16
    if (n == 8) *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[n == 8 ? 2 : 0], w[n == 8 ? 3 : 0]);
    else *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
}

// What a CTA leaves to be joined: the row tile that begins among its tiles and goes on in the next CTAs, up to CTA last.
struct P8Split {
    int token0, head0, row0, rows;  // rows 0: none
    int last, pad[3];
};
struct P8Seg {
    int token0, head0, row0, rows;  // first token of the request, first query head, rows of the tile
    int base, len, slot;            // position of token 0; workspace slot, or -1: write the output
    int tok, off;                   // token of row 0, and row 0 among its heads
    int tiles;                      // of this segment
    int req, head, tile0;           // request, kv head, first tile along the cache
};

// Query rows row0 + step i + (0, 1), i < n, of a segment: fetched, split and laid out by a warp, sixteen lanes to a row; in two
// e4m3 parts, or (kTurned) as fp16, 64 dimensions after 64: below 448, exact down to 2^-16.
template <int RP, int n, bool kTurned>
__device__ __forceinline__ void p8_queries(const PaArgs &A, const P8Seg &g, int row0, int step, uint8_t *q, float *qs, int lane) {
    const int ch = lane & 15;
    uint4 w[n];
#pragma unroll
    for (int i = 0; i < n; ++i) {
        const int row = row0 + step * i + (lane >> 4);
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row < g.rows) {
            // row's token behind token g.tok: (g.off + row) / G, exact (below 2^13, by G <= 4096)
            const int rr = g.off + row, tok = A.G == 1 ? rr : (int)__umulhi((uint32_t)rr, A.g_magic);
            w[i] = *reinterpret_cast<const uint4 *>(A.q + ((int64_t)(g.token0 + g.tok + tok) * A.Hq + g.head0 + rr - tok * A.G) * kPgDim + ch * 8);
        }
    }
#pragma unroll
    for (int i = 0; i < n; ++i) {
        const int row = row0 + step * i + (lane >> 4);
        const uint32_t ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t top = 0u;  // magnitudes of bf16 are ordered as their bits
#pragma unroll
        for (int j = 0; j < 4; ++j) top = __vmaxu2(top, ww[j] & 0x7FFF7FFFu);
        top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
        for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
        const bool finite = top < 0x7F80u;
        const int e = max(p8_need(__uint_as_float(top << 16)), A.q_down - 126);
        const float inv = finite ? p8_pow2(-e) : 0.f;
        uint32_t hi4[2], lo4[2], half4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // (0 where the row is not finite: its factor makes it NaN)
            const float a = finite ? __uint_as_float(ww[j] << 16) * inv : 0.f;
            const float b = finite ? __uint_as_float(ww[j] & 0xFFFF0000u) * inv : 0.f;
            if (kTurned) {
                half4[j] = pa_pack(a, b);
                continue;
            }
            const uint32_t c = p8_encode2(a, b);
            const float2 f = p8_floats2(c);
            const uint32_t d = p8_encode2((a - f.x) * 16.f, (b - f.y) * 16.f);  // at most 256
            if (j & 1) {
                hi4[j >> 1] |= c << 16;
                lo4[j >> 1] |= d << 16;
            } else {
                hi4[j >> 1] = c;
                lo4[j >> 1] = d;
            }
        }
        if (kTurned) {
            *reinterpret_cast<uint4 *>(q + (ch >> 3) * (RP * 128) + row * 128 + (((ch & 7) ^ (row & 7)) * 16)) =
                make_uint4(half4[0], half4[1], half4[2], half4[3]);
        } else {
            uint8_t *const to = q + row * 128 + (((ch >> 1) ^ (row & 7)) * 16) + (ch & 1) * 8;
            *reinterpret_cast<uint2 *>(to) = make_uint2(hi4[0], hi4[1]);
            *reinterpret_cast<uint2 *>(to + RP * 128) = make_uint2(lo4[0], lo4[1]);
        }
        if (ch == 0) qs[row] = finite ? p8_pow2(e - A.q_down) : __int_as_float(0x7FC00000);
    }
}

// Warps: four for V (and K, where it is turned, and the next segment's queries for windows), four for each softmax group (two groups for
// up to 32 rows, four for more), one that copies, two that issue the MMAs of S and of O, one that walks the segments ahead of the copies
// and splits their queries where the V warps do not.  Two CTAs to an SM where registers and tensor memory allow.
template <int RP, bool F32>
struct P8Cfg {
    static constexpr int N = RP < 16 ? 16 : (RP + 15) / 16 * 16;
    static constexpr bool kTurned = RP == 128;   // K becomes fp16 in tensor memory, as V does
    static constexpr int NS = kTurned ? RP : 2 * RP;  // columns of S: both parts of the queries, or the one
    static constexpr int NO = F32 ? 2 * RP : N;  // columns of O: for fp32 outputs P's two parts, rows j and RP + j
    static constexpr int kGroups = RP == 8 ? 1 : RP <= 32 ? 2 : 4, RG = RP / kGroups;  // softmax groups, rows of each
    static constexpr int kThreads = (4 + 4 * kGroups + 4) * 32;
    static constexpr int kCtas = RP <= (F32 ? 16 : 24) ? 2 : 1;  // per SM
    static constexpr uint32_t kCols = kCtas == 2 ? 256 : 512;
    static constexpr int VB = 2, KB = kTurned ? 2 : 0, SB = 64 * (VB + KB) + 2 * NS + NO <= (int)kCols ? 2 : 1;
    static constexpr uint32_t kColV = 0, kColK = 64 * VB, kColS = kColK + 64 * KB, kColO = kColS + SB * NS;
    static_assert(kColO + NO <= kCols && NS % 16 == 0 && NO % 16 == 0, "tensor memory");
    static constexpr int PB = F32 || RP == 128 ? 1 : 2;  // P buffers
    // Queries of all segments but the first: for windows by the V warps, where a segment begins (one warp took 7 to 17 thousand
    // cycles for 24 rows, as long as four tiles: 64 requests of up to 512 positions 37 -> 29 us); long row tiles have more tiles to a
    // segment, and V warps of few registers; fp32 outputs in 8-row tiles lose by the larger V loop (200 short requests of one token 84 ->
    // 94).  Not measured: fp32 outputs in tiles of 16 to 32 rows, where the one warp is as slow (64 requests of up to 512 positions, windows of 4: 41 us,
    // and 29 for bf16), and 64 rows.
    static constexpr bool kVQueries = RP <= 32 && !F32;
    static constexpr int kQ = 2 * RP * 128, kP = NO * 256;
    static constexpr size_t smem(int stages, int R) {
        return 1024 + (size_t)stages * (kP8StageK + kP8StageV) + 2 * kQ + PB * kP + ((size_t)R + 1) * 4;
    }
    // Registers of a thread where softmax warps get some of the others' (24 warps of 80; see kSplit below).
    static constexpr int kRegs = RP == 128 ? 80 : 0;
    static constexpr bool kSplit = RP == 128;
    static constexpr int kRegsV = 32, kRegsRest = 64, kRegsS = 96;
    static_assert(!kSplit || 4 * kRegsV + 4 * kRegsRest + 4 * kGroups * kRegsS <= (8 + 4 * kGroups) * kRegs,
                  "a split may not ask for more than the launch has");
};

template <int RP, bool F32>
__global__ void __launch_bounds__(P8Cfg<RP, F32>::kThreads, P8Cfg<RP, F32>::kCtas)
paged8_attention_kernel(const __grid_constant__ PaArgs A, P8Split *__restrict__ splits) {
    using Cfg = P8Cfg<RP, F32>;
    constexpr int NS = Cfg::NS, VB = Cfg::VB, SB = Cfg::SB, RG = Cfg::RG, kThreads = Cfg::kThreads;
    constexpr int kCopyWarp = 4 + 4 * Cfg::kGroups, kSWarp = kCopyWarp + 1, kOWarp = kCopyWarp + 2;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t s_bar[2 * kP8MaxStages + 20 + kP8Ring];
    __shared__ PaTileInfo s_info[kP8Ring];
    __shared__ P8Seg s_seg[kP8Ring];
    __shared__ __align__(16) float s_nref[RP], s_del[RP], s_fac[RP], s_sum[4][RP], s_qs[4][RP];
    __shared__ int s_unset[Cfg::kGroups];  // whether a row has no reference yet (s_seen: each row's)
    __shared__ uint8_t s_seen[RP];
    __shared__ int s_quit[Cfg::kGroups][2];  // a wait of the group gave up (tile parity)
    __shared__ int s_max[4][RP];
    __shared__ int s_scan[kThreads / 32];
    __shared__ uint32_t s_tmem;
    __shared__ PaCtl s_ctl;
    uint8_t *const s_k = smem + ((1024u - (smem_u32(smem) & 1023u)) & 1023u);
    uint8_t *const s_q = s_k + A.stages * kP8StageK, *const s_p = s_q + 2 * Cfg::kQ;
    uint8_t *const s_v = s_p + Cfg::PB * Cfg::kP;
    int *const s_pre = reinterpret_cast<int *>(s_v + A.stages * kP8StageV);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t bar0 = smem_u32(s_bar);
    // Barriers come in pairs where what they guard has two buffers; tile t uses number t mod 2.
    const uint32_t b_full = bar0, b_empty = bar0 + 8 * kP8MaxStages;
    const uint32_t b_sf = bar0 + 16 * kP8MaxStages;             // the columns of S(t - SB) read
    const uint32_t b_o = b_sf + 16;                             // what O(t) waits for: V(t) and P(t)
    const uint32_t b_s = b_sf + 32, b_pv = b_sf + 48;           // S(t), O(t) complete
    const uint32_t b_vfree = b_sf + 64;                         // V's columns read
    const uint32_t b_q = b_sf + 80, b_qfree = b_sf + 96;        // queries of a segment there, read
    const uint32_t b_end = b_sf + 112, b_q0 = b_sf + 120;       // b_q0: those of the first segment
    const uint32_t b_seg = b_sf + 128;                          // segment descriptors (kP8Ring of them)
    const uint32_t b_k = b_seg + 8 * kP8Ring, b_kfree = b_k + 16;  // K in tensor memory, read

    if (tid == 0) {
        for (int i = 0; i < A.stages; ++i) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, (Cfg::kTurned ? 4 : 5) + 4 * Cfg::kGroups);  // K's and V's warps, S complete where it reads the stage, the softmax warps (scales)
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_sf + 8 * i, 4 * Cfg::kGroups);
            mbar_init(b_o + 8 * i, 4 + 4 * Cfg::kGroups);
            mbar_init(b_s + 8 * i, 1);
            mbar_init(b_pv + 8 * i, 1);
            mbar_init(b_vfree + 8 * i, 1);
            mbar_init(b_q + 8 * i, Cfg::kVQueries ? 5 : 1);
            mbar_init(b_qfree + 8 * i, 1);
            mbar_init(b_k + 8 * i, 4);
            mbar_init(b_kfree + 8 * i, 1);
        }
        mbar_init(b_end, 2);
        mbar_init(b_q0, kCopyWarp);
        for (int i = 0; i < kP8Ring; ++i) mbar_init(b_seg + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = tid; i < RP; i += kThreads) s_nref[i] = 0.f;
    if (tid < kP8Ring) {
        s_info[tid] = PaTileInfo{};
        s_seg[tid] = P8Seg{};
        if (tid < 2 * Cfg::kGroups) s_quit[tid >> 1][tid & 1] = 0;
    }
    griddep_wait();
    griddep_launch_dependents();
    // Not before the wait: a kernel ahead that lets this one start before it has its own tensor memory would wait for this
    // one's, and this one for its end.  By the warp that has nothing to do yet; with a register split by the first one, after the scan, where
    // it leaves the scan fewer spills (chunks 317 -> 295 us; windows lose by that: 32K 20.7 -> 22.1).
    constexpr int kTmemWarp = Cfg::kSplit ? 0 : kOWarp + 1;
    auto take_tmem = [&]() {
        if (warp != kTmemWarp) return;
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(Cfg::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    };
    if (!Cfg::kSplit) take_tmem();

    // Tiles before every request.
    const uint32_t lim = tid ? 0u : reinterpret_cast<volatile uint32_t *>(A.status)[1];
    int n_tiles = 0;
    for (int r0 = 0; r0 < A.R; r0 += kThreads) {
        const int r = r0 + tid;
        int mine = 0;
        if (r < A.R) {
            const PaReq x = pa_req(A, r);
            mine = A.Hkv * pa_head_tiles<RP>(A, x);
        }
        int v = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(~0u, v, o);
            if (lane >= o) v += u;
        }
        __syncthreads();
        if (lane == 31) s_scan[warp] = v;
        __syncthreads();
        int all = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const int y = s_scan[w];
            if (w < warp) v += y;
            all += y;
        }
        if (r < A.R) s_pre[r] = n_tiles + v - mine;
        n_tiles += all;
    }
    if (Cfg::kSplit) take_tmem();
    if (tid == 0) {
        s_pre[A.R] = n_tiles;
        s_ctl.stop = 0u;
        s_ctl.limit = lim ? lim - 1u : kPaPolls;
        s_ctl.status = A.status;
    }
    __syncthreads();
    const int lo = pa_lo(n_tiles, gridDim.x, blockIdx.x), hi = pa_lo(n_tiles, gridDim.x, blockIdx.x + 1);
    if (n_tiles == 0 || hi <= lo) {
        if (tid == 0) splits[blockIdx.x].rows = 0;
        if (warp == kTmemWarp)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(s_tmem), "r"(Cfg::kCols) : "memory");
        return;
    }
    const uint32_t count = hi - lo;

    pa_fence_before();
    __syncthreads();
    pa_fence_after();
    const uint32_t tmem = s_tmem;
    const uint32_t quarter = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes

    // S: NS columns of e4m3 or fp16 products, both operands K-major; O: NO columns, P's rows the fast index
    constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(NS >> 3) << 17) | (8u << 24);
    constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((uint32_t)(Cfg::NO >> 3) << 17) | (8u << 24);
    // Tile t's phase of a barrier that counts the tiles of one of two buffers, or of n.
    auto phase = [](uint32_t t, uint32_t n) { return (t / n) & 1u; };

    if (warp < kCopyWarp) {  // the first segment's queries: the V and the softmax warps, which have nothing to do yet
        if (p8_wait<Cfg::kSplit || F32>(b_seg, 0u, &s_ctl)) {
            const P8Seg g = s_seg[0];
            constexpr int kWarps = kCopyWarp, kEach = (RP / 2 + kWarps - 1) / kWarps;
            if (2 * warp + 2 * kWarps * (kEach - 1) < RP) p8_queries<RP, kEach, Cfg::kTurned>(A, g, 2 * warp, 2 * kWarps, s_q, s_qs[0], lane);
            else if (kEach > 1) p8_queries<RP, kEach - (kEach > 1), Cfg::kTurned>(A, g, 2 * warp, 2 * kWarps, s_q, s_qs[0], lane);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) pa_arrive(b_q0);
    }
    if (warp >= kCopyWarp && Cfg::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsRest));
    if (warp == kCopyWarp) {
        // ---- copies: lane j < 8 brings unit j of each tile ---------------------------------
        // Descriptors of tile t go into ring entry t mod 16.  A stage is refilled after V of its
        // tile is turned, and that runs at most two tiles ahead of O: the slowest reader, a softmax warp that ends a
        // segment, is at tile t - 8 at the earliest.
        const bool copies = s_ctl.limit != 0u;  // (a limit of no polls, the test hook: as if the copy engine had stopped)
        int u = lo, k = 0, n_seg = 0, st = 0;
        uint32_t st_phase = 0;
        while (u < hi) {
            const int si = n_seg % kP8Ring;
            if (!p8_wait<Cfg::kSplit || F32>(b_seg + 8 * si, phase(n_seg, kP8Ring), &s_ctl)) break;
            const int h = s_seg[si].head, len = s_seg[si].len, s0 = u - s_seg[si].tile0, r = s_seg[si].req;
            int end = u + s_seg[si].tiles;
            const int upp = A.page / kPgUnitPos;
            // j / upp for j < 2^28 (upp <= 16)
            auto page_of = [&](int j) { return upp == 1 ? j : (int)__umulhi((uint32_t)j, A.upp_magic); };
            const int32_t *const row = A.table + (int64_t)r * A.width;
            auto lookup = [&](int tile) -> int {
                const int j = tile * kPaTileUnits + lane;
                return lane < kPaTileUnits && j * kPgUnitPos < len ? row[page_of(j)] : -1;
            };
            int pg = lookup(u - s0);
            for (; u < end; ++u, ++k) {
                const int tile = u - s0;
                const int pg_next = u + 1 < end ? lookup(tile + 1) : -1;
                // a wait that gave up ends the copies: no descriptor in use is overwritten
                if (k >= A.stages && !p8_wait<Cfg::kSplit || F32>(b_empty + 8 * st, st_phase ^ 1u, &s_ctl)) {
                    end = u = hi;
                    break;
                }
                const bool ok = pg >= 0 && pg < A.n_pages;
                const uint32_t mask = __ballot_sync(~0u, ok);
                if (lane == 0) {
                    PaTileInfo t;
                    t.mask = mask;
                    t.n_pos = len - tile * kPaTile;
                    t.tile = tile;
                    const bool first = tile == 0 || u == lo;
                    t.flags = (first ? 1u : 0u) | (u + 1 == end ? 2u : 0u) | ((uint32_t)si << 2);
                    s_info[k % kP8Ring] = t;
                    if (copies) mbar_expect_tx(b_full + 8 * st, __popc(mask) * kP8UnitBytes);
                }
                __syncwarp();
                if (ok && copies) {
                    const int j = tile * kPaTileUnits + lane, unit = j - page_of(j) * upp;
                    const uint8_t *const src = A.pages + (((int64_t)pg * A.Hkv + h) * upp + unit) * kP8UnitBytes;
                    bulk_g2s(smem_u32(s_k + st * kP8StageK + lane * 2048), src, 2048, b_full + 8 * st);
                    bulk_g2s(smem_u32(s_v + st * kP8StageV + lane * kP8VUnit), src + kP8VCodes, kP8VUnit, b_full + 8 * st);
                }
                pg = pg_next;
                if (++st == A.stages) {
                    st = 0;
                    st_phase ^= 1u;
                }
            }
            ++n_seg;
        }
        // Whatever the other warps do (one may still give up a wait once this one has no more to copy), the
        // copies in flight land before the CTA ends.
        for (int j = max(0, k - A.stages); copies && j < k; ++j)
            mbar_wait_ok(b_full + 8 * (j % A.stages), (uint32_t)(j / A.stages) & 1u);
        __syncwarp();
    } else if (warp == kSWarp) {
        // ---- S = K Q^T ---------------------------------------------------------------------
        const uint64_t q0 = pa_desc_q(smem_u32(s_q)), k0 = pa_desc_q(smem_u32(s_k));
        int st = 0;
        uint32_t st_phase = 0, n_seg = 0;
        for (uint32_t t = 0; t < count; ++t) {
            if (Cfg::kTurned) p8_wait<Cfg::kSplit || F32>(b_k + 8 * (t & 1), phase(t, 2), &s_ctl);
            else p8_wait<Cfg::kSplit || F32>(b_full + 8 * st, st_phase, &s_ctl);
            const uint32_t flags = s_info[t % kP8Ring].flags;
            if (flags & 1u) p8_wait<Cfg::kSplit || F32>(n_seg ? b_q + 8 * (n_seg & 1) : b_q0, n_seg ? phase(n_seg - (~n_seg & 1u), 2) : 0u, &s_ctl);
            if (t >= SB) p8_wait<Cfg::kSplit || F32>(b_sf + 8 * (t % SB), phase(t - SB, SB), &s_ctl);
            if (lane == 0) {
                pa_fence_after();
                const uint64_t q = q0 + (n_seg & 1) * (Cfg::kQ / 16), ka = k0 + st * (kP8StageK / 16);
                const uint32_t d = tmem + Cfg::kColS + NS * (t % SB);
                if (Cfg::kTurned) {
                    const uint32_t kt = tmem + Cfg::kColK + 64 * (t & 1);
#pragma unroll
                    for (int s = 0; s < 8; ++s) pa_mma(d, kt + 8 * s, q + (s >> 2) * (RP * 128 / 16) + 2 * (s & 3), kIdescS, s ? 1u : 0u);
                    pa_commit(b_kfree + 8 * (t & 1));
                } else {
#pragma unroll
                    for (int s = 0; s < 4; ++s) p8_mma_ss(d, ka + 2 * s, q + 2 * s, kIdescS, s ? 1u : 0u);
                    pa_commit(b_empty + 8 * st);
                }
                pa_commit(b_s + 8 * (t % SB));
                if (flags & 2u) pa_commit(b_qfree + 8 * (n_seg & 1));
            }
            __syncwarp();
            n_seg += (flags >> 1) & 1u;
            if (++st == A.stages) {
                st = 0;
                st_phase ^= 1u;
            }
        }
        if (lane == 0) {
            pa_commit(b_end);
            mbar_wait_ok(b_end, 0u);
        }
        __syncwarp();
    } else if (warp == kOWarp) {
        // ---- O += V^T P^T ------------------------------------------------------------------
        const uint64_t p0 = pa_desc_p(smem_u32(s_p));
        for (uint32_t t = 0; t < count; ++t) {
            p8_wait<Cfg::kSplit || F32>(b_o + 8 * (t & 1), phase(t, 2), &s_ctl);
            const uint32_t first = s_info[t % kP8Ring].flags & 1u;
            if (lane == 0) {
                pa_fence_after();
                const uint32_t va = tmem + Cfg::kColV + 64 * (t % VB);
                const uint64_t pb = p0 + t % Cfg::PB * (Cfg::kP / 16);
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    pa_mma(tmem + Cfg::kColO, va + 8 * s, pb + 16 * s, kIdescO, s || (!F32 && !first) ? 1u : 0u);
                pa_commit(b_pv + 8 * (t & 1));
                pa_commit(b_vfree + 8 * (t % VB));
            }
            __syncwarp();
        }
        if (lane == 0) {
            pa_commit(b_end);
            mbar_wait_ok(b_end, 0u);
        }
        __syncwarp();
    } else if (warp == kOWarp + 1) {
        // ---- segments, and the queries of all but the first --------------------------------
        // Segment n + 1 is announced before the queries of n are fetched, so that copies and queries run ahead of one
        // another.  Segment n + 2 takes n's buffer once the last S of n is complete.  The rows' factors have four: that S
        // waited for softmax warps to have read S, and the factors with it, two tiles before.  (Descriptors have sixteen, and the slowest
        // reader is a few segments behind.)
        int r = 0;
        {
            int a = 0, b = A.R;
            while (b - a > 1) {
                const int mid = (a + b) >> 1;
                if (s_pre[mid] <= lo) a = mid; else b = mid;
            }
            r = a;
        }
        PaReq x = pa_req(A, r);
        int head_tiles = pa_head_tiles<RP>(A, x), u = lo, there = 0;
        P8Split split = {};
        for (int n = 0; n < there || u < hi; ++n) {
            // (twice for the first)
            while (u < hi && there < n + 2) {
                while (s_pre[r + 1] <= u) {
                    ++r;
                    if (s_pre[r + 1] > u) {
                        x = pa_req(A, r);
                        head_tiles = pa_head_tiles<RP>(A, x);
                    }
                }
                const int h = (u - s_pre[r]) / head_tiles;
                int s0 = s_pre[r] + h * head_tiles, rt = 0, nt = pa_row_tiles<RP>(A, x, 0);
                while (s0 + nt <= u) {
                    s0 += nt;
                    nt = pa_row_tiles<RP>(A, x, ++rt);
                }
                const int end = min(hi, s0 + nt), si = there % kP8Ring;
                if (lane == 0) {
                    P8Seg g;
                    g.token0 = x.q0;
                    g.head0 = h * A.G;
                    g.row0 = rt * RP;
                    g.rows = min(RP, x.rows - rt * RP);
                    g.base = x.base;
                    g.len = x.len;
                    g.slot = u == s0 && end == s0 + nt ? -1 : 2 * (int)blockIdx.x + (u == s0 ? 1 : 0);
                    g.tok = g.row0 / A.G;
                    g.off = g.row0 - g.tok * A.G;
                    g.tiles = end - u;
                    g.req = r;
                    g.head = h;
                    g.tile0 = u - s0;
                    s_seg[si] = g;
                    pa_arrive(b_seg + 8 * si);
                    if (u == s0 && end < s0 + nt) split = {g.token0, g.head0, g.row0, g.rows, pa_cta_of(n_tiles, gridDim.x, s0 + nt - 1), {}};
                }
                __syncwarp();
                u = end;
                ++there;
            }
            if (n == 0) continue;
            // a wait that gave up: what is in the buffer may still be read
            if (n >= 2 && !p8_wait<Cfg::kSplit || F32>(b_qfree + 8 * (n & 1), phase(n - 2, 2), &s_ctl)) break;
            if (!Cfg::kVQueries) {
                const P8Seg g = s_seg[n % kP8Ring];
                uint8_t *const q = s_q + (n & 1) * Cfg::kQ;
                constexpr int kDeep = RP == 24 ? 6 : RP == 128 ? 4 : RP / 2 < 8 ? RP / 2 : 8;  // pairs of rows in flight, by registers
                for (int i = 0; i < RP / 2; i += kDeep) p8_queries<RP, kDeep, Cfg::kTurned>(A, g, 2 * i, 2, q, s_qs[n & 3], lane);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }
            // (also where the V warps fetch them: no S of segment n before this warp has seen that of n - 2 complete, or the
            // wait above could miss it)
            if (lane == 0) pa_arrive(b_q + 8 * (n & 1));
        }
        if (lane == 0) splits[blockIdx.x] = split;
    } else if (warp < 4) {
        if (Cfg::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsV));
        // ---- V: lane = dimension, columns of two positions ---------------------------------
        const uint8_t *const vrow = s_v + tid * 16;
        int st = 0;
        uint32_t st_phase = 0, n_next = 1;
        for (uint32_t t = 0; t < count; ++t) {
            p8_wait<Cfg::kSplit || F32>(b_full + 8 * st, st_phase, &s_ctl);
            const uint32_t mask = s_info[t % kP8Ring].mask, flags = s_info[t % kP8Ring].flags;
            const int n_pos = s_info[t % kP8Ring].n_pos;
            const bool whole = mask == 0xFFu && n_pos >= kPaTile;
            if (Cfg::kTurned) {  // K: lane = position, columns of two dimensions (what is no position is cut out of S)
                if (t >= 2) p8_wait<Cfg::kSplit || F32>(b_kfree + 8 * (t & 1), phase(t - 2, 2), &s_ctl);
                pa_fence_after();
                const uint8_t *const krow = s_k + st * kP8StageK + tid * kPgDim;
#pragma unroll 2
                for (int c = 0; c < 8; ++c) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(krow + ((c ^ (tid & 7)) << 4));
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
                    uint32_t o[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        o[2 * i] = p8_decode2(ww[i] & 0xFFFFu);
                        o[2 * i + 1] = p8_decode2(ww[i] >> 16);
                    }
                    pa_st8(tmem + quarter + Cfg::kColK + 64 * (t & 1) + 8 * c, o);
                }
                pa_wait_st();
                pa_fence_before();
                __syncwarp();
                if (lane == 0) pa_arrive(b_k + 8 * (t & 1));
            }
            const int vb = t % VB;
            if (t >= VB) p8_wait<Cfg::kSplit || F32>(b_vfree + 8 * vb, phase(t - VB, VB), &s_ctl);
            pa_fence_after();
            const uint32_t col = tmem + quarter + Cfg::kColV + 64 * vb;
#pragma unroll 2
            for (int j = 0; j < kPaTileUnits; ++j) {
                const uint4 w = *reinterpret_cast<const uint4 *>(vrow + st * kP8StageV + j * kP8VUnit);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[2 * i] = p8_decode2(ww[i] & 0xFFFFu);
                    o[2 * i + 1] = p8_decode2(ww[i] >> 16);
                }
                if (!whole) {
                    const int left = (mask >> j) & 1u ? n_pos - j * kPgUnitPos : 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = 2 * i >= left ? 0u : 2 * i + 1 >= left ? o[i] & 0xFFFFu : o[i];
                }
                pa_st8(col + 8 * j, o);
            }
            pa_wait_st();
            pa_fence_before();
            __syncwarp();
            if (lane == 0) {
                pa_arrive(b_empty + 8 * st);
                pa_arrive(b_o + 8 * (t & 1));
            }
            if (Cfg::kVQueries && (flags & 1u)) {  // segment n_next - 1 begins: the queries of the next one
                if (t + s_seg[flags >> 2].tiles < count) {
                    const uint32_t b = n_next & 1;
                    if (p8_wait<Cfg::kSplit || F32>(b_seg + 8 * (n_next % kP8Ring), phase(n_next, kP8Ring), &s_ctl) &&
                        (n_next < 2 || p8_wait<Cfg::kSplit || F32>(b_qfree + 8 * b, phase(n_next - 2, 2), &s_ctl))) {
                        const P8Seg g = s_seg[n_next % kP8Ring];
                        p8_queries<RP, RP / 8, Cfg::kTurned>(A, g, 2 * warp, 8, s_q + b * Cfg::kQ, s_qs[n_next & 3], lane);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) pa_arrive(b_q + 8 * b);
                }
                ++n_next;
            }
            if (++st == A.stages) {
                st = 0;
                st_phase ^= 1u;
            }
        }
    } else {
        // ---- softmax: lane = position, rows rb .. rb + RG - 1 of the row tile --------------
        if (Cfg::kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsS));
        const int sg = (warp - 4) >> 2, rb = sg * RG, gt = (tid & 127), gw = warp & 3;
        auto group_sync = [&]() { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + sg) : "memory"); };

        // l: sums of p over this lane's positions.  acc (fp32 outputs): o, added up here tile by tile,
        // since the tensor core truncates what it adds to its accumulators (2^-24 a time).
        constexpr int kStep = RG % 8 ? 4 : 8;           // rows taken together
        int pos0 = 0, off0 = 0, whole_to = 0, len = 0;  // of the segment
        f2 l[RG / 2], acc[F32 ? RG / 2 : 1];
        const f2 lo_step = pa_f2(0x1p-11f, 0x1p-11f), q_step = pa_f2(0x1p-4f, 0x1p-4f);
        int st = 0;
        uint32_t st_phase = 0, n_seg = 0;
        for (uint32_t t = 0; t < count; ++t) {
            f2 s[RG / 2];
            // A wait that gave up must not let the group's threads disagree on what comes next: the
            // vote below carries it, and then all of them leave.
            // (Three questions at once, each as long as a whole wait; mostly all are answered.)
            uint32_t got = mbar_poll(b_s + 8 * (t % SB), phase(t, SB), true) ? 1u : 0u;
            if (mbar_poll(b_full + 8 * st, st_phase, true)) got |= 2u;
            if (t < Cfg::PB || mbar_poll(b_pv + 8 * ((t - Cfg::PB) & 1), phase(t - Cfg::PB, 2), false)) got |= 4u;  // P is read
            got = __reduce_and_sync(~0u, got);
            if ((got & 3u) != 3u && (!p8_wait<Cfg::kSplit || F32>(b_s + 8 * (t % SB), phase(t, SB), &s_ctl) || !p8_wait<Cfg::kSplit || F32>(b_full + 8 * st, st_phase, &s_ctl)))
                s_quit[sg][t & 1] = 1;
            const PaTileInfo ti = s_info[t % kP8Ring];
            const bool first = ti.flags & 1u, last = ti.flags & 2u;
            const P8Seg &g = s_seg[ti.flags >> 2];
            if (first) {
                pos0 = g.base + g.tok;
                off0 = g.off + rb;
                whole_to = min(pos0 + 1, g.len);
                len = g.len;
            }
            // the scales of the lane's unit (anything, where there is none)
            const float2 sc = *reinterpret_cast<const float2 *>(s_v + st * kP8StageV + (gt >> 4) * kP8VUnit + kP8Scales - kP8VCodes);
            const float ck = A.c * p8_pow2(p8_exponent(sc.x));
            const int ev = p8_exponent(sc.y);
            const float lv = (float)ev, iv = p8_pow2(-ev);
            const f2 c2 = pa_f2(ck, ck), lv2 = pa_f2(lv, lv), iv2 = pa_f2(iv, iv);
            pa_fence_after();
            {
                // the next columns are on their way while these are joined
                float h[2][kStep], f[2][kStep];
                const uint32_t col = tmem + quarter + Cfg::kColS + NS * (t % SB) + rb;
                p8_ld<kStep>(col, h[0]);
                if (!Cfg::kTurned) p8_ld<kStep>(col + RP, f[0]);
#pragma unroll
                for (int j = 0; j < RG; j += kStep) {
                    constexpr int kHalf = kStep / 2;
                    const int now = (j / kStep) & 1;
                    pa_wait_ld();
                    if (j + kStep < RG) {
                        p8_ld<kStep>(col + j + kStep, h[now ^ 1]);
                        if (!Cfg::kTurned) p8_ld<kStep>(col + RP + j + kStep, f[now ^ 1]);
                    }
#pragma unroll
                    for (int i = 0; i < kHalf; i += 2) {
                        const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(s_qs[n_seg & 3] + rb + j + 2 * i);
                        if (Cfg::kTurned) {
                            s[j / 2 + i] = pa_mul2(pa_f2(h[now][2 * i], h[now][2 * i + 1]), q.x);
                            s[j / 2 + i + 1] = pa_mul2(pa_f2(h[now][2 * i + 2], h[now][2 * i + 3]), q.y);
                            continue;
                        }
                        s[j / 2 + i] = pa_mul2(pa_fma2(pa_f2(f[now][2 * i], f[now][2 * i + 1]), q_step, pa_f2(h[now][2 * i], h[now][2 * i + 1])), q.x);
                        s[j / 2 + i + 1] =
                            pa_mul2(pa_fma2(pa_f2(f[now][2 * i + 2], f[now][2 * i + 3]), q_step, pa_f2(h[now][2 * i + 2], h[now][2 * i + 3])), q.y);
                    }
                }
            }
            pa_fence_before();
            __syncwarp();
            if (lane == 0) {
                pa_arrive(b_sf + 8 * (t % SB));
                pa_arrive(b_empty + 8 * st);
            }
            if (++st == A.stages) {
                st = 0;
                st_phase ^= 1u;
            }

            if (first) {
#pragma unroll
                for (int j = 0; j < RG / 2; ++j) l[j] = 0ull;
                if (F32) {
#pragma unroll
                    for (int j = 0; j < RG / 2; ++j) acc[j] = 0ull;
                }
            }
            // s = score + log2 of V's scale - reference, in powers of two.
#pragma unroll
            for (int j = 0; j < RG / 2; j += 2) {
                const ulonglong2 r = *reinterpret_cast<const ulonglong2 *>(s_nref + rb + 2 * j);  // (0 where a segment begins)
                s[j] = pa_fma2(s[j], c2, pa_add2(r.x, lv2));
                s[j + 1] = pa_fma2(s[j + 1], c2, pa_add2(r.y, lv2));
            }
            // What a row does not see is cut out (its first row sees the fewest positions).
            if (ti.mask != 0xFFu || (ti.tile + 1) * kPaTile > whole_to) {
                asm volatile("");  // (a branch, and not a selection for every score of every tile)
                const int pos = ti.tile * kPaTile + gt;
                const bool here = ((ti.mask >> (gt >> 4)) & 1u) && pos < len;
                // row j is token tok + (off + j) / G: it sees the position once j reaches this (a
                // position before the first token is seen by all rows, one RP + 1 past it by none; the
                // distance times G may pass 32 bits)
                const int from = here ? min(max(pos - pos0, 0), RP + 1) * A.G - off0 : RG;
#pragma unroll
                for (int j = 0; j < RG / 2; ++j) {
                    float2 v = pa_un2(s[j]);
                    if (2 * j < from) v.x = -INFINITY;
                    if (2 * j + 1 < from) v.y = -INFINITY;
                    s[j] = pa_f2(v.x, v.y);
                }
            }
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < RG / 2; ++j) {
                const float2 v = pa_un2(s[j]);
                top = fmaxf(fmaxf(top, v.x), v.y);
            }
            uint32_t any;
            asm volatile(
                "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.or.pred q, %2, 128, p; selp.u32 %0, 1, 0, q; }"
                : "=r"(any)
                : "r"((uint32_t)(first || top > kPaOver || s_unset[sg] != 0)), "r"(1 + sg)
                : "memory");
            if (s_quit[sg][t & 1]) break;
            if (any) {
                // New references, 7 below the largest score, for rows without one and for those that
                // a score exceeds by more than 15.
#pragma unroll
                for (int j = 0; j < RG / 2; ++j) {
                    const float2 v = pa_un2(s[j]);
                    const int m0 = __reduce_max_sync(~0u, pa_order(v.x)), m1 = __reduce_max_sync(~0u, pa_order(v.y));
                    if (lane == 0) {
                        s_max[gw][rb + 2 * j] = m0;
                        s_max[gw][rb + 2 * j + 1] = m1;
                    }
                }
                if (gt == 0) s_unset[sg] = 0;
                group_sync();
                if (gt < RG) {
                    const float m =
                        pa_unorder(max(max(s_max[0][rb + gt], s_max[1][rb + gt]), max(s_max[2][rb + gt], s_max[3][rb + gt])));
                    const bool set = !first && s_seen[rb + gt];
                    const float old = first ? 0.f : s_nref[rb + gt];
                    float del = 0.f, now = old;
                    bool seen = set;
                    if (m != -INFINITY && (!set || !(m <= kPaOver))) {
                        now = old + (kPaUnder - m);
                        del = now - old;
                        seen = true;
                    }
                    if (!seen) s_unset[sg] = 1;
                    s_nref[rb + gt] = now;
                    s_seen[rb + gt] = seen;
                    s_del[rb + gt] = del;
                    s_fac[rb + gt] = set ? pa_ex2(del) : 1.f;
                }
                group_sync();
#pragma unroll
                for (int j = 0; j < RG / 2; j += 2) {
                    const ulonglong2 r = *reinterpret_cast<const ulonglong2 *>(s_del + rb + 2 * j);
                    s[j] = pa_add2(s[j], r.x);
                    s[j + 1] = pa_add2(s[j + 1], r.y);
                }
                if (!first) {
#pragma unroll
                    for (int j = 0; j < RG / 2; ++j) {
                        const f2 f = *reinterpret_cast<const f2 *>(s_fac + rb + 2 * j);
                        l[j] = pa_mul2(l[j], f);
                    }
                    if (!F32) {
                        p8_wait<Cfg::kSplit || F32>(b_pv + 8 * ((t - 1) & 1), phase(t - 1, 2), &s_ctl);
                        pa_fence_after();
#pragma unroll
                        for (int j = 0; j < RG; j += kStep) {
                            float o[kStep];
                            p8_ld<kStep>(tmem + quarter + Cfg::kColO + rb + j, o);
                            pa_wait_ld();
#pragma unroll
                            for (int i = 0; i < kStep; ++i) o[i] *= s_fac[rb + j + i];
                            p8_st<kStep>(tmem + quarter + Cfg::kColO + rb + j, o);
                        }
                        pa_wait_st();
                        pa_fence_before();
                    }
                }
            }
            if (!(got & 4u)) p8_wait<Cfg::kSplit || F32>(b_pv + 8 * ((t - Cfg::PB) & 1), phase(t - Cfg::PB, 2), &s_ctl);  // P is read
            if (F32 && !first) {
                pa_fence_after();
#pragma unroll
                for (int j = 0; j < RG; j += kStep) {
                    float o[kStep], lo[kStep];
                    p8_ld<kStep>(tmem + quarter + Cfg::kColO + rb + j, o);
                    p8_ld<kStep>(tmem + quarter + Cfg::kColO + RP + rb + j, lo);
                    pa_wait_ld();
#pragma unroll
                    for (int i = 0; i < kStep / 2; ++i)
                        acc[j / 2 + i] = pa_add2(acc[j / 2 + i], pa_fma2(pa_f2(lo[2 * i], lo[2 * i + 1]), lo_step, pa_f2(o[2 * i], o[2 * i + 1])));
                }
                pa_fence_before();
                if (any) {
#pragma unroll
                    for (int j = 0; j < RG / 2; ++j) acc[j] = pa_mul2(acc[j], *reinterpret_cast<const f2 *>(s_fac + rb + 2 * j));
                }
            }
            uint8_t *const prow = s_p + t % Cfg::PB * Cfg::kP + (gt >> 3) * 128 + (gt & 7) * 16;
#pragma unroll
            for (int j = 0; j < RG; j += kStep) {
                float p[kStep];
                uint32_t w[kStep / 2];
#pragma unroll
                for (int i = 0; i < kStep / 2; ++i) {
                    const float2 v = pa_un2(s[j / 2 + i]);
                    p[2 * i] = pa_ex2(v.x);
                    p[2 * i + 1] = pa_ex2(v.y);
                    l[j / 2 + i] = pa_fma2(pa_f2(p[2 * i], p[2 * i + 1]), iv2, l[j / 2 + i]);
                    w[i] = pa_pack(p[2 * i], p[2 * i + 1]);
                }
                // rows in lines of eight
                p8_line<kStep>(prow + ((rb + j) >> 3) * 2048 + ((rb + j) & 7) * 2, w);
                if (F32) {
#pragma unroll
                    for (int i = 0; i < kStep / 2; ++i) {
                        const float2 f = __half22float2(reinterpret_cast<const __half2 &>(w[i]));
                        // 2^11 (p - f), exact before the rounding
                        w[i] = pa_pack(fmaf(f.x, -2048.f, p[2 * i] * 2048.f), fmaf(f.y, -2048.f, p[2 * i + 1] * 2048.f));
                    }
                    p8_line<kStep>(prow + ((RP + rb + j) >> 3) * 2048 + ((RP + rb + j) & 7) * 2, w);
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) pa_arrive(b_o + 8 * (t & 1));

            if (last) {
                // The segment's sums over positions (each step of the exchange halves the rows a lane
                // holds, so that lane i ends with row i), then o.
                constexpr int RX = RG == 12 ? 16 : RG;
                float v[RX];
#pragma unroll
                for (int j = 0; j < RX; j += 2) {
                    const float2 x = j < RG ? pa_un2(l[j / 2 < RG / 2 ? j / 2 : 0]) : make_float2(0.f, 0.f);
                    v[j] = x.x;
                    v[j + 1] = x.y;
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    if (o >= RX) {
#pragma unroll
                        for (int j = 0; j < RX; ++j) v[j] += __shfl_xor_sync(~0u, v[j], o);
                    } else {
                        const bool up = lane & o;
#pragma unroll
                        for (int j = 0; j < o; ++j) {
                            const float send = up ? v[j] : v[j + o], keep = up ? v[j + o] : v[j];
                            v[j] = keep + __shfl_xor_sync(~0u, send, o);
                        }
                    }
                }
                if (lane < RG) s_sum[gw][rb + lane] = v[0];
                group_sync();
                const int slot = g.slot, rows = g.rows;
                if (gt < RG) {
                    const int row = rb + gt, rr = g.row0 + row, tok = rr / A.G;
                    const float sum = s_sum[0][row] + s_sum[1][row] + s_sum[2][row] + s_sum[3][row];
                    const bool seen = s_seen[row];
                    s_fac[row] = seen ? 1.f / sum : 0.f;
                    s_max[0][row] = (g.token0 + tok) * A.Hq + g.head0 + rr - tok * A.G;
                    if (slot >= 0 && row < rows)
                        A.part_ml[(int64_t)slot * RP + row] = make_float2(seen ? -s_nref[row] : -INFINITY, sum);
                    s_nref[row] = 0.f;  // for the next segment
                }
                group_sync();
                p8_wait<Cfg::kSplit || F32>(b_pv + 8 * (t & 1), phase(t, 2), &s_ctl);
                pa_fence_after();
                float o[RG];
#pragma unroll
                for (int j = 0; j < RG; j += kStep) p8_ld<kStep>(tmem + quarter + Cfg::kColO + rb + j, o + j);
                pa_wait_ld();
                if (F32) {
#pragma unroll
                    for (int j = 0; j < RG; j += kStep) {
                        float lo[kStep];
                        p8_ld<kStep>(tmem + quarter + Cfg::kColO + RP + rb + j, lo);
                        pa_wait_ld();
#pragma unroll
                        for (int i = 0; i < kStep; ++i) {
                            const float2 x = pa_un2(acc[(j + i) / 2]);
                            o[j + i] = fmaf(lo[i], 0x1p-11f, o[j + i]) + (i & 1 ? x.y : x.x);
                        }
                    }
                }
                if (slot >= 0) {
                    float *const to = A.part + ((int64_t)slot * RP + rb) * kPgDim + gt;
#pragma unroll
                    for (int j = 0; j < RG; ++j)
                        if (rb + j < rows) to[j * kPgDim] = o[j];
                } else {
#pragma unroll
                    for (int j = 0; j < RG; ++j)
                        if (rb + j < rows) {
                            const int64_t at = (int64_t)s_max[0][rb + j] * kPgDim + gt;
                            const float f = s_fac[rb + j], y = f == 0.f ? 0.f : o[j] * f;
                            if (F32) reinterpret_cast<float *>(A.out)[at] = y;
                            else reinterpret_cast<__nv_bfloat16 *>(A.out)[at] = __float2bfloat16_rn(y);
                        }
                }
                ++n_seg;
                pa_fence_before();  // (the next tile's vote comes before anything read here is written again)
            }
        }
    }
    pa_fence_before();
    __syncthreads();
    pa_fence_after();
    if (warp == kTmemWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Cfg::kCols) : "memory");
}

// Joins the segments of a row that several CTAs hold.  CTA (i, j) takes the i-th row tile that was split, and of it 8 / W rows, W
// warps to each, every one over every W-th segment with all of its loads in flight together.
template <int RP, bool F32, int W>
__global__ void __launch_bounds__(256) paged8_join_kernel(const __grid_constant__ PaArgs A, const P8Split *__restrict__ splits, int ctas) {
    __shared__ float4 s_acc[8][32];
    __shared__ float2 s_ml[8];
    __shared__ P8Split s_split;
    __shared__ int s_first, s_count[16];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) s_first = -1;
    griddep_wait();
    griddep_launch_dependents();
    // (at most 512 CTAs)
    P8Split x[2] = {};
    uint32_t there[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (tid + 256 * i < ctas) x[i] = splits[tid + 256 * i];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        there[i] = __ballot_sync(~0u, x[i].rows > 0);
        if (lane == 0) s_count[warp + 8 * i] = __popc(there[i]);
    }
    __syncthreads();
    int before = 0;  // split tiles of the CTAs before
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        if ((w & 7) == warp && x[w >> 3].rows > 0 &&
            before + __popc(there[w >> 3] & ((1u << lane) - 1u)) == (int)blockIdx.x) {
            s_split = x[w >> 3];
            s_first = tid + 256 * (w >> 3);
        }
        before += s_count[w];
    }
    __syncthreads();
    const int f = s_first;
    if (f < 0) return;
    constexpr int kRows = 8 / W;
    const int row = blockIdx.y * kRows + warp / W, wj = warp % W, e = s_split.last;
    const bool mine = row < s_split.rows;
    // (ref, sum, acc) += (r, l, o), a part that saw nothing (r = -inf) left out.
    float ref = -INFINITY, sum = 0.f;
    float4 acc = {0.f, 0.f, 0.f, 0.f};
    auto join = [&](float r1, float l1, const float4 &o1) {
        if (r1 == -INFINITY) return;
        const float top = ref > r1 ? ref : r1;  // (NaN: r1)
        const float k0 = ref == -INFINITY ? 0.f : pa_ex2(ref - top), k1 = pa_ex2(r1 - top);
        sum = sum * k0 + l1 * k1;
        acc.x = acc.x * k0 + o1.x * k1;
        acc.y = acc.y * k0 + o1.y * k1;
        acc.z = acc.z * k0 + o1.z * k1;
        acc.w = acc.w * k0 + o1.w * k1;
        ref = top;
    };
    constexpr int kDeep = W == 1 ? 4 : 8;
    for (int c0 = f + wj; mine && c0 <= e; c0 += kDeep * W) {
        float4 o[kDeep];
        float2 ml[kDeep];
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            const int c = c0 + j * W;
            ml[j] = make_float2(-INFINITY, 0.f);
            if (c <= e) {
                const int64_t slot = (int64_t)(c == f ? 2 * f + 1 : 2 * c) * RP + row;
                ml[j] = A.part_ml[slot];
                o[j] = *reinterpret_cast<const float4 *>(A.part + slot * kPgDim + 4 * lane);
            }
        }
#pragma unroll
        for (int j = 0; j < kDeep; ++j) join(ml[j].x, ml[j].y, o[j]);
    }
    if (W > 1) {
        s_acc[warp][lane] = acc;
        if (lane == 0) s_ml[warp] = make_float2(ref, sum);
        __syncthreads();
        if (wj) return;
#pragma unroll
        for (int j = 1; j < W; ++j) join(s_ml[warp + j].x, s_ml[warp + j].y, s_acc[warp + j][lane]);
    }
    if (!mine) return;
    const float inv = ref == -INFINITY ? 0.f : 1.f / sum;
    const int rr = s_split.row0 + row, tok = rr / A.G;
    const int64_t at = ((int64_t)(s_split.token0 + tok) * A.Hq + s_split.head0 + rr - tok * A.G) * kPgDim + 4 * lane;
    if (F32) {
        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(A.out) + at) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    } else {
        const __nv_bfloat162 p = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
        const __nv_bfloat162 q = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
        uint2 v;
        v.x = reinterpret_cast<const uint32_t &>(p);
        v.y = reinterpret_cast<const uint32_t &>(q);
        *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(A.out) + at) = v;
    }
}

template <int RP, bool F32>
static int p8_launch(PaArgs A, P8Split *splits, int sms, cudaStream_t stream) {
    using Cfg = P8Cfg<RP, F32>;
    const size_t most = Cfg::kCtas == 2 ? 110 * 1024 : 216 * 1024;  // with the static part and 1 KB reserved a CTA
    A.stages = kP8MaxStages;
    while (A.stages > 2 && Cfg::smem(A.stages, A.R) > most) --A.stages;
    const size_t smem = Cfg::smem(A.stages, A.R);
    // No more row tiles than the windows allow, nor more tiles than the table's rows hold: short caches get a CTA to a tile
    // and none that has nothing to do (one token at 1500 positions: 9.8 -> 9.2 us).
    const int most_new = A.max_new < A.T ? A.max_new : A.T;
    const int64_t by_request = (int64_t)A.R * (((int64_t)most_new * A.G + RP - 1) / RP), by_rows = ((int64_t)A.T * A.G + RP - 1) / RP + A.R;
    const int64_t row_tiles = A.Hkv * (by_request < by_rows ? by_request : by_rows);
    const int64_t tiles = row_tiles * (((int64_t)A.width * A.page + kPaTile - 1) / kPaTile);
    const int most_ctas = Cfg::kCtas * sms < 512 ? Cfg::kCtas * sms : 512;  // (what the join looks through)
    const int grid = (int)(tiles < most_ctas ? tiles : most_ctas);
    SVD_CUDA_TRY((allow_smem<paged8_attention_kernel<RP, F32>>(most)));
    // A register split above what the launch has would wait forever: refuse to launch one.
    static std::atomic<int> regs{0};
    if (Cfg::kSplit && regs.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes at;
        SVD_CUDA_TRY(cudaFuncGetAttributes(&at, paged8_attention_kernel<RP, F32>));
        regs.store(at.numRegs, std::memory_order_relaxed);
    }
    if (Cfg::kSplit && regs.load(std::memory_order_relaxed) < Cfg::kRegs) return SVD_ERR_UNSUPPORTED;
    SVD_CUDA_TRY(launch(paged8_attention_kernel<RP, F32>, dim3(grid), dim3(Cfg::kThreads), smem, stream, true, A, splits));
    // No more row tiles are split than there are, nor more than there are borders between CTAs.  Few row tiles are split over
    // at least eight CTAs each, and then eight warps join a row (five parts to a tile, 8 requests of 4096 positions: 26 us with
    // eight warps, 20 with one; twelve, one token behind 1500: 9.1 and 9.7).
    const int n = (int)(row_tiles < grid ? row_tiles : grid);
    if (row_tiles * 8 <= grid)
        SVD_CUDA_TRY(launch(paged8_join_kernel<RP, F32, 8>, dim3(n, RP), dim3(256), 0, stream, true, A, (const P8Split *)splits, grid));
    else
        SVD_CUDA_TRY(launch(paged8_join_kernel<RP, F32, 1>, dim3(n, (RP + 7) / 8), dim3(256), 0, stream, true, A, (const P8Split *)splits, grid));
    return SVD_OK;
}

// The workspace of the 4-bit cache's attention, with the descriptions of what CTAs leave to be joined behind it.
static size_t p8_splits_at(int Hq, int Hkv, int R, int max_new, int sms) { return align_up(pa_ws_bytes(Hq, Hkv, R, max_new, sms), 256); }
size_t paged8_attention_ws_bytes(int Hq, int Hkv, int R, int max_new) {
    const int sms = sm_count();
    const size_t n = sms < 1 ? 0 : p8_splits_at(Hq, Hkv, R, max_new, sms);
    return n ? n + (size_t)2 * sms * sizeof(P8Split) : 0;
}

int paged8_attention(const uint16_t *q, int T, const int32_t *kv_len, const int32_t *q_start, int R,
                     int max_new, const int32_t *table, int width, const void *pages, int page,
                     int64_t n_pages, int Hq, int Hkv, float scale, void *out, int out_dtype, void *ws,
                     size_t ws_bytes, cudaStream_t stream) {
    PaArgs A;
    int rp;
    const int sms = sm_count();
    const int rc = pa_arguments(&A, &rp, q, T, kv_len, q_start, R, max_new, table, width, pages, page, n_pages, Hq, Hkv,
                                scale, out, out_dtype, ws, ws_bytes, sms);
    if (rc != SVD_OK) return rc;
    if (sms < 1) return SVD_ERR_CUDA;
    const size_t at = p8_splits_at(Hq, Hkv, R, max_new, sms);
    if (ws_bytes < at + (size_t)2 * sms * sizeof(P8Split)) return SVD_ERR_WORKSPACE;
    if (T == 0) return SVD_OK;
    // A sum of codes reaches 448^2 * 128 < 2^25 and a row's power of two 2^120: over 2^20, their product stays in fp32's range
    // whatever the scales of keys, so that a row is lost only where its scores leave that range.  (Scales from 2^64 on would take c
    // out of it in turn; there, a score leaves the range before that product does.)
    A.q_down = scale < 0x1p64f ? 20 : 0;
    A.c *= A.q_down ? 0x1p20f : 1.f;
    P8Split *const splits = (P8Split *)((uint8_t *)ws + at);
#define SVD_P8(RP) (out_dtype == SVD_F32 ? p8_launch<RP, true>(A, splits, sms, stream) : p8_launch<RP, false>(A, splits, sms, stream))
    switch (rp) {
        case 8: return SVD_P8(8);
        case 16: return SVD_P8(16);
        case 24: return SVD_P8(24);
        case 32: return SVD_P8(32);
        case 64: return p8_launch<64, false>(A, splits, sms, stream);
        default: return p8_launch<128, false>(A, splits, sms, stream);
    }
#undef SVD_P8
}

}  // namespace svd
