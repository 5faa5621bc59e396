// paged.cuh -- the 4-bit page format shared by the paged-cache kernels.
//
// A page holds page_size positions (a multiple of 16) of every kv head as units of 16 positions,
// [page][kv head][page_size / 16][2304 bytes]:
//   bytes    0..1023  K codes  [4 blocks of 32 dims][16 positions][16 B]: dims 2b, 2b + 1 of the
//                     block in the low and high nibble of byte b
//   bytes 1024..2047  V codes  [64][16 B]: row d holds dim d in the low and dim d + 64 in the high
//                     nibbles; position 4k + j at byte 4k + (0, 2, 1, 3)[j]
//   bytes 2048..2175  K scales fp16 [16 positions][4 blocks]
//   bytes 2176..2303  V scales fp16 [4 blocks][16 positions]
// Every byte belongs to one position, so appends of different positions never meet in a byte.
// The value of code c is d (c - 8).  d has eight significant bits: d (c - 8) then needs at most
// eleven, so it is exact in fp16 and the attention kernel's operands carry no rounding (but for blocks
// of keys below 2^-12, whose d it holds to a multiple of 2^-22).
#pragma once

#include "svd_common.cuh"

#include <atomic>

namespace svd {

constexpr int kPgDim = 128;
constexpr int kPgUnitPos = 16;
constexpr int kPgUnitBytes = SVD_PAGED_UNIT_BYTES;
constexpr int kPgVCodes = 1024;
constexpr int kPgKScales = 2048;
constexpr int kPgVScales = 2176;
constexpr double kPgMaxAbs = 65280.0;  // magnitudes end here: d <= 8160, and -8 d still fits fp16

// Byte of position i (0..15) inside a V row: pairs of positions sit 16 bits apart, so that one
// mask of a 32-bit word yields two neighbouring positions as an fp16 pair.
__host__ __device__ __forceinline__ int pg_v_byte(int i) {
    return (i & 12) | ((i & 1) << 1) | ((i >> 1) & 1);
}

// Lets a kernel have `bytes` of dynamic shared memory: asked once for each kernel and device (the
// call costs as much as a tenth of a launch).
template <auto *kernel>
inline cudaError_t allow_smem(size_t bytes) {
    static std::atomic<uint64_t> asked{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (asked.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) asked.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

inline bool pg_page_size_ok(int ps) { return ps >= 16 && ps <= SVD_PAGED_PAGE_MAX && ps % 16 == 0; }
inline bool pg_pool_ok(int n_kv_heads, int page_size, int64_t n_pages) {
    return n_kv_heads >= 1 && n_kv_heads <= 1024 && pg_page_size_ok(page_size) && n_pages >= 1 &&
           n_pages <= (int64_t)1 << 30;
}

}  // namespace svd
