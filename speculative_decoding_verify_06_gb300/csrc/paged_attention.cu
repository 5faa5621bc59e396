// paged_attention.cu -- attention of ragged verify windows over the paged 4-bit cache.
//
// "Decode is memory-bound ..." ("The ceiling"): at long context the cache joins the weights on
// every pass; "100 tokens per second ..." ("Why a hiring company is writing this"): several
// sequences share the pass.
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c <q, k_j> - ref),   c = scale log2(e)
//
// Work.  Query rows of one request and kv head (token-major, then head in the group) form row tiles
// of up to RP rows; a row tile reads the cache positions its last token sees in tiles of 128.  All
// tiles, ordered by request, kv head, row tile and position, are split into equal contiguous
// ranges, one per CTA, so that ragged lengths balance without the host knowing them.  The part of a
// range within one row tile is a segment.  A segment that is a whole row tile writes the output;
// others leave (sums, reference, unnormalised o) in the workspace, at most two per CTA, and a
// second kernel joins them.
//
// One tile.  Bulk copies bring up to eight units into a ring stage.  Four warps turn K into fp16 in
// tensor memory (lane = position) and four others V (lane = dimension, two positions per column): codes
// to fp16 by a mask and an exponent, then d (c - 8), exact because d has eight significant bits (K as
// d / 4 (16 + c) - 6 d in one step: a quarter, since 24 d may leave fp16.  d / 4 is rounded to a multiple of
// 2^-24 below d = 2^-15, keys below 2.4e-4; the exact form, two steps where a warp finds a d above 2720, took
// 107 us instead of 102.5 for 200 requests of 2K).  S^T = K Q^T (M = 128
// positions, N = query rows) and O^T += V^T P^T (M = 128 dimensions) run on tcgen05 with A in tensor
// memory and fp32 accumulators, issued by a warp each; K is refilled by halves, so that its next tile
// starts while S still reads the second half.  The softmax warps turn S into P in shared memory.  A lane
// holds one position of S for all rows, so the softmax needs no lane exchange: the reference of a row
// changes only when a score exceeds it by 15 (p <= 2^15 in between), checked by one vote of the four
// warps, and starts 7 below the first tile's maximum.  p keeps fp16's eleven bits down to 2^-21 of the
// largest and loses them gradually to 2^-32.  For fp32 outputs P is split into two fp16 parts that
// stand side by side as columns of one product, the second times 2^11 so that it does not fall among fp16's
// subnormals (p to a relative 2^-22 and 2^-43 of the largest), and O is added up in registers
// tile by tile, because the tensor core truncates what it adds to its accumulators: 256 additions
// were 2.5e-6 off, so are 6e-7.
//
// Rows a mask leaves empty get zeros.  Positions past the length, or on a page outside the pool,
// are cut out of S, and their V scales are replaced by 0, whatever their bytes.
//
// What bounds it.  Every cache byte is read once, 144 per position and kv head, but each takes work that
// no pipe does at HBM's pace: a tile takes 4538 warp instructions at 20 rows, of
// which the SM issues 73 % of what it could, with instruction
// fetch and the chain copy - K - S - P - O behind the rest.  262144 positions of 8 kv heads, 20 rows: 91.4 us,
// 3.3 TB/s of cache; 64 ragged requests of up to 16K: 213 us, 3.35 TB/s; 200 requests of 2K, one
// token, fp32: 103 us, 2.5 TB/s; 32768 positions: 23.4 us, of which 11 to 14 do not depend on the
// length (lines through 8K and 16K, and through 32K and 262K); two chunks of 512 tokens behind 8K: 260 us, 550 TFLOP/s.
//
// What was measured on the way (262K / chunk of 512): K and softmax in the same four warps, 105 / 640 us;
// four roles with one MMA warp, 107 / 450; two MMA warps and halves, 103 / 422; queries fetched
// ahead and a join by eight warps, 93 / 356; row tiles of 128 instead of 64 rows for long windows, 261.  Not
// kept: two K and two V groups (355 with 64 rows), softmax groups of 16 rows (372), MMAs under
// elect.sync with uniform operands (359, 93.3), V's loop unrolled four or eight times (200 short requests:
// 117 and 125 us against 109), waits that poll without suspending, that sleep, or with a hint (no gain).
#include "paged_attention.cuh"

namespace svd {

constexpr int kPaStageBytes = kPaTileUnits * kPgUnitBytes;
constexpr int kPaMaxStages = 4;
constexpr int kPaRing = 8;           // tile and segment descriptors in flight (see producer)

// Warps: four for K, four for V, four for each softmax group (of up to 32 rows), one that copies and
// two that issue the MMAs of S and of O.  Two CTAs to an SM where registers and tensor memory allow, so that
// one's waits are filled by the other.
template <int RP, bool F32>
struct PaCfg {
    static constexpr int N = RP < 16 ? 16 : (RP + 15) / 16 * 16;
    // columns of O: for fp32 outputs P's two parts stand side by side, rows j and RP + j
    static constexpr int NO = F32 ? 2 * RP : N;
    static constexpr int kGroups = RP > 32 ? RP / 32 : 1, RG = RP / kGroups;  // softmax groups, rows of each
    static constexpr int kThreads = (8 + 4 * kGroups + 3) * 32;
    static constexpr int kCtas = RP <= (F32 ? 16 : 24) ? 2 : 1;  // per SM
    // operands and scores in flight, in tensor memory: 256 columns for each of two CTAs, or 512
    static constexpr int KB = kCtas == 2 || RP == 128 ? 1 : 2, VB = 2, SB = 64 * (KB + VB) + 2 * N + NO <= (kCtas == 2 ? 256 : 512) ? 2 : 1;
    static constexpr uint32_t kColK = 0, kColV = 64 * KB, kColS = kColV + 64 * VB, kColO = kColS + SB * N;
    static constexpr uint32_t kCols = kCtas == 2 ? 256 : 512;
    static_assert(kColO + NO <= kCols && NO % 16 == 0, "tensor memory");
    // (K(t + SB) may not arrive at the barrier of S(t) before S(t) is issued)
    static_assert(SB >= KB, "as many S buffers as K buffers");
    static constexpr int PB = F32 ? 1 : 2;  // P buffers
    static constexpr int kQ = N * 256, kP = NO * 256;
    static constexpr size_t smem(int stages, int R) {
        return 1024 + (size_t)stages * kPaStageBytes + 2 * kQ + PB * kP + ((size_t)R + 1) * 4;
    }
    // Registers of a thread: two CTAs of 15 warps leave 64, one of 27 warps 72; there the K and V warps
    // hand some of theirs to the softmax warps.
    static constexpr int kRegs = RP == 128 ? 72 : 64;
    static constexpr bool kSplit = RP == 128 || (kCtas == 2 && RP >= 16);
    static constexpr int kRegsKV = RP == 128 ? 40 : 48, kRegsS = RP == 128 ? 88 : 96;
    static_assert(!kSplit || 8 * kRegsKV + 4 * kGroups * kRegsS <= (8 + 4 * kGroups) * kRegs,
                  "a split may not ask for more than the launch has");
};

template <int RP, bool F32>
__global__ void __launch_bounds__(PaCfg<RP, F32>::kThreads, PaCfg<RP, F32>::kCtas)
paged_attention_kernel(const __grid_constant__ PaArgs A) {
    using Cfg = PaCfg<RP, F32>;
    constexpr int N = Cfg::N, KB = Cfg::KB, VB = Cfg::VB, SB = Cfg::SB, RG = Cfg::RG, kThreads = Cfg::kThreads;
    constexpr int kCopyWarp = 8 + 4 * Cfg::kGroups, kSWarp = kCopyWarp + 1, kOWarp = kCopyWarp + 2;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t s_bar[2 * kPaMaxStages + 17 + kPaRing];
    __shared__ PaTileInfo s_info[kPaRing];
    __shared__ PaSeg s_seg[kPaRing];
    __shared__ __align__(16) float s_nref[RP], s_del[RP], s_fac[RP], s_sum[4][RP];
    __shared__ int s_unset[Cfg::kGroups];  // whether a row has no reference yet (s_seen: each row's)
    __shared__ uint8_t s_seen[RP];
    __shared__ int s_quit[Cfg::kGroups][2];  // a wait of the group gave up (tile parity)
    __shared__ int s_max[4][RP];
    __shared__ int s_scan[kThreads / 32];
    __shared__ uint32_t s_tmem;
    __shared__ PaCtl s_ctl;
    uint8_t *const sm0 = smem + ((1024u - (smem_u32(smem) & 1023u)) & 1023u);
    uint8_t *const s_q = sm0 + A.stages * kPaStageBytes, *const s_p = s_q + 2 * Cfg::kQ;
    int *const s_pre = reinterpret_cast<int *>(s_p + Cfg::PB * Cfg::kP);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t bar0 = smem_u32(s_bar);
    // Barriers come in pairs where what they guard has two buffers; tile t uses number t mod 2.
    const uint32_t b_full = bar0, b_empty = bar0 + 8 * kPaMaxStages;
    // What S(t) waits for: the first half of K(t) and the columns of S(t - SB) read (b_s0), the second
    // half (b_s1); what O(t) waits for: V(t) and P(t) (b_o).
    const uint32_t b_s0 = bar0 + 16 * kPaMaxStages, b_s1 = b_s0 + 16, b_o = b_s0 + 32;
    const uint32_t b_s = b_s0 + 48, b_pv = b_s0 + 64;             // S(t), O(t) complete
    const uint32_t b_kfree = b_s0 + 80, b_vfree = b_s0 + 112;     // K (by buffer and half), V read
    const uint32_t b_end = b_s0 + 128, b_seg = b_s0 + 136;        // segment descriptors (kPaRing of them)

    if (tid == 0) {
        for (int i = 0; i < A.stages; ++i) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_s0 + 8 * i, 4 + 4 * Cfg::kGroups);
            mbar_init(b_s1 + 8 * i, 4);
            mbar_init(b_o + 8 * i, 4 + 4 * Cfg::kGroups);
            mbar_init(b_s + 8 * i, 1);
            mbar_init(b_pv + 8 * i, 1);
            mbar_init(b_kfree + 16 * i, 1);
            mbar_init(b_kfree + 16 * i + 8, 1);
            mbar_init(b_vfree + 8 * i, 1);
        }
        mbar_init(b_end, 2);
        for (int i = 0; i < kPaRing; ++i) mbar_init(b_seg + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid < kPaRing) {
        s_info[tid] = PaTileInfo{};
        s_seg[tid] = PaSeg{};
        if (tid < 2 * Cfg::kGroups) s_quit[tid >> 1][tid & 1] = 0;
    }
    griddep_wait();
    griddep_launch_dependents();

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
    if (tid == 0) {
        s_pre[A.R] = n_tiles;
        s_ctl.stop = 0u;
        s_ctl.limit = lim ? lim - 1u : kPaPolls;
        s_ctl.status = A.status;
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int r = tid; r <= A.R; r += kThreads) A.prefix[r] = s_pre[r];
    const int lo = pa_lo(n_tiles, gridDim.x, blockIdx.x), hi = pa_lo(n_tiles, gridDim.x, blockIdx.x + 1);
    if (n_tiles == 0 || hi <= lo) return;
    const uint32_t count = hi - lo;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(Cfg::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pa_fence_before();
    __syncthreads();
    pa_fence_after();
    const uint32_t tmem = s_tmem;
    const uint32_t quarter = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes

    // S: N columns, both operands K-major; O: NO columns, P's rows the fast index
    constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
    constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((uint32_t)(Cfg::NO >> 3) << 17) | (8u << 24);
    // Tile t's phase of a barrier that counts the tiles of one of two buffers, or of n.
    auto phase = [](uint32_t t, uint32_t n) { return (t / n) & 1u; };

    if (warp == kCopyWarp) {
        // ---- copies: lane j < 8 brings unit j of each tile ---------------------------------
        // Descriptors of tile t (and its segment) go into ring entry t mod 8.  The slowest reader
        // is at tile t - 6 at most: a stage is refilled after both dequantisations of its tile, and
        // those run at most two tiles ahead of the last use of a descriptor.
        int r = 0;
        {
            int a = 0, b = A.R;
            while (b - a > 1) {
                const int mid = (a + b) >> 1;
                if (s_pre[mid] <= lo) a = mid; else b = mid;
            }
            r = a;
        }
        int u = lo, k = 0, n_seg = 0, st = 0;
        uint32_t st_phase = 0;
        PaReq x = pa_req(A, r);
        int head_tiles = pa_head_tiles<RP>(A, x);
        while (u < hi) {
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
            int end = min(hi, s0 + nt);
            const int si = n_seg % kPaRing;
            if (lane == 0) {
                PaSeg g;
                g.token0 = x.q0;
                g.head0 = h * A.G;
                g.row0 = rt * RP;
                g.rows = min(RP, x.rows - rt * RP);
                g.base = x.base;
                g.len = x.len;
                g.slot = u == s0 && end == s0 + nt ? -1 : 2 * (int)blockIdx.x + (u == s0 ? 1 : 0);
                g.tok = g.row0 / A.G;
                g.off = g.row0 - g.tok * A.G;
                s_seg[si] = g;
                pa_arrive(b_seg + 8 * si);
            }
            const int upp = A.page / kPgUnitPos;
            // j / upp for j < 2^28 (upp <= 16)
            auto page_of = [&](int j) { return upp == 1 ? j : (int)__umulhi((uint32_t)j, A.upp_magic); };
            const int32_t *const row = A.table + (int64_t)r * A.width;
            auto lookup = [&](int tile) -> int {
                const int j = tile * kPaTileUnits + lane;
                return lane < kPaTileUnits && j * kPgUnitPos < x.len ? row[page_of(j)] : -1;
            };
            int pg = lookup(u - s0);
            for (; u < end; ++u, ++k) {
                const int tile = u - s0;
                const int pg_next = u + 1 < end ? lookup(tile + 1) : -1;
                // a wait that gave up ends the copies: no descriptor in use is overwritten
                if (k >= A.stages && !pa_wait(b_empty + 8 * st, st_phase ^ 1u, &s_ctl)) {
                    end = u = hi;
                    break;
                }
                const bool ok = pg >= 0 && pg < A.n_pages;
                const uint32_t mask = __ballot_sync(~0u, ok);
                if (lane == 0) {
                    PaTileInfo t;
                    t.mask = mask;
                    t.n_pos = x.len - tile * kPaTile;
                    t.tile = tile;
                    const bool first = tile == 0 || u == lo;
                    t.flags = (first ? 1u : 0u) | (u + 1 == end ? 2u : 0u) | ((uint32_t)si << 2);
                    s_info[k % kPaRing] = t;
                    mbar_expect_tx(b_full + 8 * st, __popc(mask) * kPgUnitBytes);
                }
                __syncwarp();
                if (ok) {
                    const int j = tile * kPaTileUnits + lane, unit = j - page_of(j) * upp;
                    bulk_g2s(smem_u32(sm0 + st * kPaStageBytes + lane * kPgUnitBytes),
                             A.pages + (((int64_t)pg * A.Hkv + h) * upp + unit) * kPgUnitBytes,
                             kPgUnitBytes, b_full + 8 * st);
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
        for (int j = max(0, k - A.stages); j < k; ++j)
            mbar_wait_ok(b_full + 8 * (j % A.stages), (uint32_t)(j / A.stages) & 1u);
        __syncwarp();
    } else if (warp == kSWarp) {
        // ---- S = K Q^T ---------------------------------------------------------------------
        const uint64_t q0 = pa_desc_q(smem_u32(s_q));
        for (uint32_t t = 0; t < count; ++t) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                pa_wait((half ? b_s1 : b_s0) + 8 * (t % SB), phase(t, SB), &s_ctl);
                const uint32_t qb = (s_info[t % kPaRing].flags >> 2) & 1u;
                if (lane == 0) {
                    pa_fence_after();
                    const uint64_t q = q0 + (qb * Cfg::kQ + half * (N * 128)) / 16;
                    const uint32_t d = tmem + Cfg::kColS + N * (t % SB);
                    const uint32_t ka = tmem + Cfg::kColK + 64 * (t % KB) + 32 * half;
#pragma unroll
                    for (int s = 0; s < 4; ++s) pa_mma(d, ka + 8 * s, q + 2 * s, kIdesc, s || half ? 1u : 0u);
                    pa_commit(b_kfree + 16 * (t % KB) + 8 * half);
                    if (half) pa_commit(b_s + 8 * (t % SB));
                }
                __syncwarp();
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
            pa_wait(b_o + 8 * (t & 1), phase(t, 2), &s_ctl);
            const uint32_t first = s_info[t % kPaRing].flags & 1u;
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
    } else if (warp >= 4 && warp < 8) {
        if (Cfg::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsKV));
        // ---- V: lane = dimension, columns of two positions ---------------------------------
        const int dim = tid - 128;
        // low nibbles: (1024 + c) - 1032; high ones: (1024 + 16 c) / 16 - 72; both c - 8 exactly
        const uint32_t nib = dim < 64 ? 0x000F000Fu : 0x00F000F0u;
        const uint32_t mul = dim < 64 ? 0x3C003C00u : 0x2C002C00u, add = dim < 64 ? 0xE408E408u : 0xD480D480u;
        const uint8_t *const vrow = sm0 + kPgVCodes + (dim & 63) * 16;
        const uint8_t *const vsc = sm0 + kPgVScales + (warp & 3) * 32;
        int st = 0;
        uint32_t st_phase = 0;
        for (uint32_t t = 0; t < count; ++t) {
            pa_wait(b_full + 8 * st, st_phase, &s_ctl);
            const uint32_t mask = s_info[t % kPaRing].mask;
            const int n_pos = s_info[t % kPaRing].n_pos;
            const bool whole = mask == 0xFFu && n_pos >= kPaTile;
            const int vb = t % VB;
            if (t >= VB) pa_wait(b_vfree + 8 * vb, phase(t - VB, VB), &s_ctl);
            pa_fence_after();
            const uint32_t col = tmem + quarter + Cfg::kColV + 64 * vb;
#pragma unroll 2
            for (int j = 0; j < kPaTileUnits; ++j) {
                const uint4 w = *reinterpret_cast<const uint4 *>(vrow + st * kPaStageBytes + j * kPgUnitBytes);
                uint32_t d[8];
                *reinterpret_cast<uint4 *>(d) = *reinterpret_cast<const uint4 *>(vsc + st * kPaStageBytes + j * kPgUnitBytes);
                *reinterpret_cast<uint4 *>(d + 4) =
                    *reinterpret_cast<const uint4 *>(vsc + st * kPaStageBytes + j * kPgUnitBytes + 16);
                if (!whole) {
                    const int left = (mask >> j) & 1u ? n_pos - j * kPgUnitPos : 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        d[i] = 2 * i >= left ? 0u : 2 * i + 1 >= left ? d[i] & 0xFFFFu : d[i];
                }
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[2 * i] = pa_h2mul(pa_h2fma((ww[i] & nib) | 0x64006400u, mul, add), d[2 * i]);
                    o[2 * i + 1] = pa_h2mul(pa_h2fma(((ww[i] >> 8) & nib) | 0x64006400u, mul, add), d[2 * i + 1]);
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
            if (++st == A.stages) {
                st = 0;
                st_phase ^= 1u;
            }
        }
    } else if (warp < 4) {
        // ---- K: lane = position, columns of two dimensions ---------------------------------
        if (Cfg::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsKV));
        int st = 0;
        uint32_t st_phase = 0, n_seg = 0;
        bool fresh = true;
        for (uint32_t t = 0; t < count; ++t) {
            const int kb = t % KB;
            if (t >= KB) pa_wait(b_kfree + 16 * kb, phase(t - KB, KB), &s_ctl);
            if (fresh) {  // a new segment: its query rows
                // (with S(t - KB) complete, and all before it, the buffer of the segment before the last
                // is free)
                if (t >= KB) pa_wait(b_kfree + 16 * kb + 8, phase(t - KB, KB), &s_ctl);
                const uint32_t si = n_seg % kPaRing;
                pa_wait(b_seg + 8 * si, phase(n_seg, kPaRing), &s_ctl);
                const PaSeg g = s_seg[si];
                uint8_t *const q = s_q + (si & 1u) * Cfg::kQ;
                ++n_seg;
                for (int i = tid; i < RP * 16; i += 128) {
                    const int row = i >> 4, ch = i & 15;
                    uint4 o = {0u, 0u, 0u, 0u};
                    if (row < g.rows) {
                        const int rr = g.row0 + row, tok = rr / A.G;
                        const uint4 w = *reinterpret_cast<const uint4 *>(
                            A.q + ((int64_t)(g.token0 + tok) * A.Hq + g.head0 + rr - tok * A.G) * kPgDim + ch * 8);
                        // dims 0 4 | 1 5 | 2 6 | 3 7, as the K words give them
                        const uint32_t lo4[2] = {w.x, w.y}, hi4[2] = {w.z, w.w};
                        uint32_t r4[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t a = lo4[j >> 1], b = hi4[j >> 1];
                            r4[j] = pa_pack(__uint_as_float(j & 1 ? a & 0xFFFF0000u : a << 16),
                                            __uint_as_float(j & 1 ? b & 0xFFFF0000u : b << 16));
                        }
                        o = make_uint4(r4[0], r4[1], r4[2], r4[3]);
                    }
                    *reinterpret_cast<uint4 *>(q + (ch >> 3) * (N * 128) + row * 128 + (((ch & 7) ^ (row & 7)) * 16)) = o;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            pa_wait(b_full + 8 * st, st_phase, &s_ctl);
            pa_fence_after();
            fresh = (s_info[t % kPaRing].flags & 2u) != 0u;
            const uint8_t *const unit = sm0 + st * kPaStageBytes + (tid >> 4) * kPgUnitBytes;
            const uint2 sc = *reinterpret_cast<const uint2 *>(unit + kPgKScales + (lane & 15) * 8);
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                if (h && t >= KB) {
                    pa_wait(b_kfree + 16 * kb + 8, phase(t - KB, KB), &s_ctl);
                    pa_fence_after();
                }
                const uint32_t s1 = h ? sc.y : sc.x;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(unit + h * 512 + b * 256 + (lane & 15) * 16);
                    const uint32_t d = __byte_perm(s1, s1, b ? 0x3232 : 0x1010);
                    const uint32_t d4 = pa_h2mul(d, 0x34003400u), d6 = pa_h2mul(d4, 0xCE00CE00u);  // d / 4, -24 times it
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t o[8];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t y = ww[2 * half + i];
                            o[4 * i + 0] = pa_h2fma(pa_16plus(y << 6), d4, d6);
                            o[4 * i + 1] = pa_h2fma(pa_16plus(y << 2), d4, d6);
                            o[4 * i + 2] = pa_h2fma(pa_16plus(y >> 2), d4, d6);
                            o[4 * i + 3] = pa_h2fma(pa_16plus(y >> 6), d4, d6);
                        }
                        pa_st8(tmem + quarter + Cfg::kColK + 64 * kb + 32 * h + 16 * b + 8 * half, o);
                    }
                }
                pa_wait_st();
                pa_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (h) pa_arrive(b_empty + 8 * st);
                    pa_arrive((h ? b_s1 : b_s0) + 8 * (t % SB));
                }
            }
            if (++st == A.stages) {
                st = 0;
                st_phase ^= 1u;
            }
        }
    } else {
        // ---- softmax: lane = position, rows rb .. rb + RG - 1 of the row tile --------------
        if (Cfg::kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsS));
        const int sg = (warp - 8) >> 2, rb = sg * RG, gt = (tid & 127), gw = warp & 3;
        const float c = A.c;
        auto group_sync = [&]() { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + sg) : "memory"); };

        // l: sums of p over this lane's positions.  acc (fp32 outputs): o, added up here tile by tile,
        // since the tensor core truncates what it adds to its accumulators (2^-24 a time).
        int pos0 = 0, off0 = 0, whole_to = 0, len = 0;  // of the segment
        f2 l[RG / 2], acc[F32 ? RG / 2 : 1];
        const f2 c2 = pa_f2(c, c);
        const f2 lo_step = pa_f2(0x1p-11f, 0x1p-11f);
        if (lane == 0)  // the first SB tiles find their S columns free
            for (int i = 0; i < SB; ++i) pa_arrive(b_s0 + 8 * i);
        for (uint32_t t = 0; t < count; ++t) {
            f2 s[RG / 2];
            // A wait that gave up must not let the group's threads disagree on what comes next: the
            // vote below carries it, and then all of them leave.
            if (!pa_wait(b_s + 8 * (t % SB), phase(t, SB), &s_ctl)) s_quit[sg][t & 1] = 1;
            const PaTileInfo ti = s_info[t % kPaRing];
            const bool first = ti.flags & 1u, last = ti.flags & 2u;
            const PaSeg &g = s_seg[ti.flags >> 2];
            if (first) {
                pos0 = g.base + g.tok;
                off0 = g.off + rb;
                whole_to = min(pos0 + 1, g.len);
                len = g.len;
            }
            pa_fence_after();
            {
                float f[RG];
#pragma unroll
                for (int j = 0; j < RG; j += 8) pa_ld8(tmem + quarter + Cfg::kColS + N * (t % SB) + rb + j, f + j);
                pa_wait_ld();
#pragma unroll
                for (int j = 0; j < RG / 2; ++j) s[j] = pa_f2(f[2 * j], f[2 * j + 1]);
            }
            pa_fence_before();
            __syncwarp();
            if (lane == 0) pa_arrive(b_s0 + 8 * (t % SB));

            if (first) {
#pragma unroll
                for (int j = 0; j < RG / 2; ++j) l[j] = 0ull;
                if (F32) {
#pragma unroll
                    for (int j = 0; j < RG / 2; ++j) acc[j] = 0ull;
                }
            }
            // s = score - reference, in powers of two.
#pragma unroll
            for (int j = 0; j < RG / 2; j += 2) {
                ulonglong2 r = *reinterpret_cast<const ulonglong2 *>(s_nref + rb + 2 * j);
                if (first) r.x = r.y = 0ull;
                s[j] = pa_fma2(s[j], c2, r.x);
                s[j + 1] = pa_fma2(s[j + 1], c2, r.y);
            }
            // What a row does not see is cut out (its first row sees the fewest positions).
            if (ti.mask != 0xFFu || (ti.tile + 1) * kPaTile > whole_to) {
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
                        pa_wait(b_pv + 8 * ((t - 1) & 1), phase(t - 1, 2), &s_ctl);
                        pa_fence_after();
#pragma unroll
                        for (int j = 0; j < RG; j += 8) {
                            float o[8];
                            pa_ld8(tmem + quarter + Cfg::kColO + rb + j, o);
                            pa_wait_ld();
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] *= s_fac[rb + j + i];
                            pa_st8(tmem + quarter + Cfg::kColO + rb + j, reinterpret_cast<const uint32_t *>(o));
                        }
                        pa_wait_st();
                        pa_fence_before();
                    }
                }
            }
            if (t >= Cfg::PB) pa_wait(b_pv + 8 * ((t - Cfg::PB) & 1), phase(t - Cfg::PB, 2), &s_ctl);  // P is read
            if (F32 && !first) {
                pa_fence_after();
#pragma unroll
                for (int j = 0; j < RG; j += 8) {
                    float o[8], lo[8];
                    pa_ld8(tmem + quarter + Cfg::kColO + rb + j, o);
                    pa_ld8(tmem + quarter + Cfg::kColO + RP + rb + j, lo);
                    pa_wait_ld();
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[j / 2 + i] = pa_add2(acc[j / 2 + i], pa_fma2(pa_f2(lo[2 * i], lo[2 * i + 1]), lo_step, pa_f2(o[2 * i], o[2 * i + 1])));
                }
                pa_fence_before();
                if (any) {
#pragma unroll
                    for (int j = 0; j < RG / 2; ++j) acc[j] = pa_mul2(acc[j], *reinterpret_cast<const f2 *>(s_fac + rb + 2 * j));
                }
            }
            uint8_t *const prow = s_p + t % Cfg::PB * Cfg::kP + (gt >> 3) * 128 + (gt & 7) * 16 + (rb >> 3) * 2048;
#pragma unroll
            for (int j = 0; j < RG; j += 8) {
                float p[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = pa_un2(s[j / 2 + i]);
                    p[2 * i] = pa_ex2(v.x);
                    p[2 * i + 1] = pa_ex2(v.y);
                    l[j / 2 + i] = pa_add2(l[j / 2 + i], pa_f2(p[2 * i], p[2 * i + 1]));
                }
                uint4 w = make_uint4(pa_pack(p[0], p[1]), pa_pack(p[2], p[3]), pa_pack(p[4], p[5]), pa_pack(p[6], p[7]));
                *reinterpret_cast<uint4 *>(prow + (j >> 3) * 2048) = w;
                if (F32) {
                    const uint32_t h[4] = {w.x, w.y, w.z, w.w};
                    uint32_t lo2[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = __half22float2(reinterpret_cast<const __half2 &>(h[i]));
                        // 2^11 (p - f), exact before the rounding
                        lo2[i] = pa_pack(fmaf(f.x, -2048.f, p[2 * i] * 2048.f), fmaf(f.y, -2048.f, p[2 * i + 1] * 2048.f));
                    }
                    *reinterpret_cast<uint4 *>(prow + (RP >> 3) * 2048 + (j >> 3) * 2048) = make_uint4(lo2[0], lo2[1], lo2[2], lo2[3]);
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) pa_arrive(b_o + 8 * (t & 1));

            if (last) {
                // The segment's sums over positions (each step of the exchange halves the rows a lane
                // holds, so that lane i ends with row i), then o.
                constexpr int RX = RG == 24 ? 32 : RG;
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
                }
                group_sync();
                pa_wait(b_pv + 8 * (t & 1), phase(t, 2), &s_ctl);
                pa_fence_after();
                float o[RG];
#pragma unroll
                for (int j = 0; j < RG; j += 8) pa_ld8(tmem + quarter + Cfg::kColO + rb + j, o + j);
                pa_wait_ld();
                if (F32) {
#pragma unroll
                    for (int j = 0; j < RG; j += 8) {
                        float lo[8];
                        pa_ld8(tmem + quarter + Cfg::kColO + RP + rb + j, lo);
                        pa_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
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
                pa_fence_before();  // (the next tile's vote comes before anything read here is written again)
            }
        }
    }
    pa_fence_before();
    __syncthreads();
    pa_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Cfg::kCols) : "memory");
}
// Joins the segments of a row that several CTAs hold: W warps per (token, query head), each over
// every W-th segment, all of its loads in flight together.  What the requests' lengths alone decide
// is worked out before the main kernel's end is waited for (the lengths were complete before it began).
template <int RP, bool F32, int W>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W) paged_merge_kernel(const __grid_constant__ PaArgs A, int ctas) {
    constexpr int kRows = W == 1 ? 4 : 1;  // rows of a CTA
    __shared__ float4 s_acc[W][32];
    __shared__ float2 s_ml[W];
    const int lane = threadIdx.x & 31, wj = W == 1 ? 0 : threadIdx.x >> 5;
    const int64_t w = (int64_t)blockIdx.x * kRows + (W == 1 ? threadIdx.x >> 5 : 0);
    const int t = (int)(w / A.Hq), head = (int)(w - (int64_t)t * A.Hq);
    int r = 0, b = A.R;
    const bool there = t < A.T && t < A.q_start[A.R];
    while (b - r > 1) {
        const int mid = (r + b) >> 1;
        if (A.q_start[mid] <= t) r = mid; else b = mid;
    }
    const PaReq x = pa_req(A, r);
    const int i = t - x.q0;
    const int h = head / A.G, rr = i * A.G + head - h * A.G, rt = rr / RP, row = rr - rt * RP;
    int before = 0, nt = 0;
    const bool mine = there && i >= 0 && i < x.n;
    if (mine) {
        for (int j = 0; j < rt; ++j) before += pa_row_tiles<RP>(A, x, j);
        nt = pa_row_tiles<RP>(A, x, rt);
    }
    // A finite query that fp16 does not hold makes its row NaN and is reported (here, where it costs nothing:
    // with the check at the main kernel's fetch of the queries, 262K took 94.7 us instead of 91.3).
    bool far = false;
    if (mine && wj == 0) {
        const uint2 q = *reinterpret_cast<const uint2 *>(A.q + w * kPgDim + 4 * lane);
        const uint32_t m = __vmaxu2(q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu), m1 = max(m & 0xFFFFu, m >> 16);
        far = m1 >= 0x4780u && m1 < 0x7F80u;  // 65536 .. the largest
    }
    griddep_wait();
    griddep_launch_dependents();
    if (far) atomicOr(A.status, 2u);
    if (!mine) return;  // (the same for all warps of a row)
    const int n_tiles = A.prefix[A.R], pre = A.prefix[r], per = (A.prefix[r + 1] - pre) / A.Hkv;
    if (n_tiles == 0) return;
    const int s0 = pre + h * per + before;
    const int f = pa_cta_of(n_tiles, ctas, s0), e = pa_cta_of(n_tiles, ctas, s0 + nt - 1);
    if (f == e) return;
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
    for (int c0 = f + wj; c0 <= e; c0 += 8 * W) {
        float4 o[8];
        float2 ml[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = c0 + j * W;
            ml[j] = make_float2(-INFINITY, 0.f);
            if (c <= e) {
                const int64_t slot = (int64_t)(c == f ? 2 * f + 1 : 2 * c) * RP + row;
                ml[j] = A.part_ml[slot];
                o[j] = *reinterpret_cast<const float4 *>(A.part + slot * kPgDim + 4 * lane);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) join(ml[j].x, ml[j].y, o[j]);
    }
    if (W > 1) {
        s_acc[wj][lane] = acc;
        if (lane == 0) s_ml[wj] = make_float2(ref, sum);
        __syncthreads();
        if (wj) return;
#pragma unroll
        for (int j = 1; j < W; ++j) join(s_ml[j].x, s_ml[j].y, s_acc[j][lane]);
    }
    const float inv = ref == -INFINITY ? 0.f : 1.f / sum;
    const int64_t at = w * kPgDim + 4 * lane;
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
static int pa_launch(PaArgs A, int sms, cudaStream_t stream) {
    using Cfg = PaCfg<RP, F32>;
    const size_t most = Cfg::kCtas == 2 ? 110 * 1024 : 220 * 1024;  // with the static part and 1 KB reserved a CTA
    A.stages = kPaMaxStages;
    while (A.stages > 2 && Cfg::smem(A.stages, A.R) > most) --A.stages;
    const size_t smem = Cfg::smem(A.stages, A.R);
    const int grid = Cfg::kCtas * sms;
    SVD_CUDA_TRY((allow_smem<paged_attention_kernel<RP, F32>>(most)));
    // A register split above what the launch has would wait forever: refuse to launch one.
    static std::atomic<int> regs{0};
    if (Cfg::kSplit && regs.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes at;
        SVD_CUDA_TRY(cudaFuncGetAttributes(&at, paged_attention_kernel<RP, F32>));
        regs.store(at.numRegs, std::memory_order_relaxed);
    }
    if (Cfg::kSplit && regs.load(std::memory_order_relaxed) < Cfg::kRegs) return SVD_ERR_UNSUPPORTED;
    SVD_CUDA_TRY(launch(paged_attention_kernel<RP, F32>, dim3(grid), dim3(Cfg::kThreads), smem, stream, true, A));
    // Few rows are split over many CTAs each, and then eight warps join one; many rows over few.
    const int64_t rows = (int64_t)A.T * A.Hq;
    if (rows <= 2048)
        SVD_CUDA_TRY(launch(paged_merge_kernel<RP, F32, 8>, dim3((unsigned)rows), dim3(256), 0, stream, true, A, grid));
    else
        SVD_CUDA_TRY(launch(paged_merge_kernel<RP, F32, 1>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, stream, true, A, grid));
    return SVD_OK;
}
size_t paged_attention_ws_bytes(int Hq, int Hkv, int R, int max_new) {
    return pa_ws_bytes(Hq, Hkv, R, max_new, sm_count());
}

int paged_attention(const uint16_t *q, int T, const int32_t *kv_len, const int32_t *q_start, int R,
                    int max_new, const int32_t *table, int width, const void *pages, int page,
                    int64_t n_pages, int Hq, int Hkv, float scale, void *out, int out_dtype, void *ws,
                    size_t ws_bytes, cudaStream_t stream) {
    PaArgs A;
    int rp;
    const int sms = sm_count();
    const int rc = pa_arguments(&A, &rp, q, T, kv_len, q_start, R, max_new, table, width, pages, page, n_pages, Hq, Hkv,
                                scale, out, out_dtype, ws, ws_bytes, sms);
    if (rc != SVD_OK || T == 0) return rc;
    A.c *= 4.f;  // (the K operand is K / 4)
#define SVD_PA(RP) (out_dtype == SVD_F32 ? pa_launch<RP, true>(A, sms, stream) : pa_launch<RP, false>(A, sms, stream))
    switch (rp) {
        case 8: return SVD_PA(8);
        case 16: return SVD_PA(16);
        case 24: return SVD_PA(24);
        case 32: return SVD_PA(32);
        case 64: return pa_launch<64, false>(A, sms, stream);
        default: return pa_launch<128, false>(A, sms, stream);
    }
#undef SVD_PA
}

}  // namespace svd
