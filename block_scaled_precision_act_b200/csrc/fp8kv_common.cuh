// fp8kv_common.cuh -- what the kernels of the block-scaled 8-bit key/value cache share:
// the cache's geometry, the ragged batch, and the E4M3 / E8M0 arithmetic of one block.
//
// A cache holds E4M3 codes [pages][Hkv][page_size][D] and, for every block of 16 tokens and
// head, one E8M0 byte e (scale 2^(e - 127)) in [pages][Hkv][page_size / 16].  A power of two
// costs E4M3 no precision, leaves the decode exact, and lets a later token raise a block's
// scale: the earlier codes then only move their exponent (they are re-rounded where they
// become subnormal, below 2^-6 of the new scale).
#pragma once

#include <cstdint>

#include "bsp_internal.h"
#include "bsp_ptx.cuh"

namespace bsp {

// What an earlier kernel of the stream may write is read by plain loads, after griddep_wait(): this
// kernel may have begun before that one ended, so to it the data are not read-only.

constexpr int kKvBlock = 16;        // tokens that share one scale
constexpr int kKvMaxExp = 246;      // largest scale byte: 448 * 2^119 is the last finite multiple

struct KvCache {
    uint8_t* k;
    uint8_t* v;
    uint8_t* k_scale;
    uint8_t* v_scale;
    const int32_t* table;           // [B][max_pages] page numbers
    const int32_t* cu_new;          // [B + 1] rows of the new tokens
    const int32_t* kv_len;          // [B] lengths, the new tokens included
    int64_t max_pages;
    int32_t pages;
    int32_t page_blocks;            // page_size / 16
    int32_t B, T, Hq, Hkv, D;
};

// Rows [first, first + n) of sequence b; whatever cu_new holds, they lie in [0, T).
struct KvRows {
    int32_t first, n;
};

__device__ __forceinline__ int32_t kv_clamp_row(int32_t r, int32_t T)
{
    return r < 0 ? 0 : (r > T ? T : r);
}

__device__ __forceinline__ KvRows kv_rows(const KvCache& c, int b)
{
    const int32_t lo = kv_clamp_row(c.cu_new[b], c.T);
    const int32_t hi = kv_clamp_row(c.cu_new[b + 1], c.T);
    return {lo, hi > lo ? hi - lo : 0};
}

// Tokens that a row of the table can address.
__device__ __forceinline__ int32_t kv_capacity(const KvCache& c)
{
    return static_cast<int32_t>(c.max_pages) * c.page_blocks * kKvBlock;
}

// kv_len[b], cut to that.
__device__ __forceinline__ int32_t kv_length(const KvCache& c, int b)
{
    return min(max(c.kv_len[b], 0), kv_capacity(c));
}

// Smallest scale byte whose 448 multiples reach amax (bits of a non-negative fp32):
// e = ceil(log2(amax / 448)) + 127, within [0, kKvMaxExp].  448 = 1.75 * 2^8.
__device__ __forceinline__ int kv_scale_exp(uint32_t amax_bits)
{
    const int e = static_cast<int>(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u);
    return e < 0 ? 0 : (e > kKvMaxExp ? kKvMaxExp : e);
}

// 2^(e - 127) for e in [0, 254]; e == 0 is the subnormal 2^-127.
__device__ __forceinline__ float kv_pow2(int e)
{
    return __uint_as_float(e > 0 ? static_cast<uint32_t>(e) << 23 : 0x00400000u);
}

// The same down to the smallest subnormal, and 0 below it
__device__ __forceinline__ float kv_pow2_low(int e)
{
    return __int_as_float(e > 0 ? e << 23 : e > -23 ? 1 << (22 + e) : 0);
}

// Four E4M3 bytes -> two pairs of f16 (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ void f16x2_to_f32(uint32_t h, float& lo, float& hi)
{
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.f32.f16 %0, a;\n\t"
        "cvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
}

// Device status word: a page outside the pool, or a length that does not fit the new tokens or the
// table (first writer wins).
__device__ __forceinline__ void kv_report_bad_batch(int* status)
{
    if (atomicCAS(status, 0, BSP_ERR_INVALID_ARG) == 0) atomicCAS(status + 1, 0, 200);
}

}  // namespace bsp
