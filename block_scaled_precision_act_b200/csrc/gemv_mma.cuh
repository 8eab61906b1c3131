// gemv_mma.cuh -- what the kernels of nvfp4_gemv share: a warp's way through the weight.
//
// A warp takes 32 rows of a 128-row tile, r, r + 32, r + 64, r + 96 for 8 values of r, whose scales lie in
// the same 16-byte words, and 256 elements of K at a time: a lane reads 2 x 16 bytes of codes of each of
// its four rows and as many scales, all of which it uses.  Each weight becomes f16 (e2m1 * e4m3 has at
// most 6 significant bits and lies in [2^-10, 2688]: exact) on its way through
// mma.sync m16n8k16 with fp32 sums, 16 weight rows against 8 rows of x.  The products may run over k
// in any order, so the 64 consecutive codes of a lane's row are the k slots that it owns in 16 products.
// x is bf16, whose range f16 lacks: it is scaled by a power of two, so that its largest element is in
// [2^14, 2^15); f16 then holds elements down to 2^-28 of that exactly and rounds smaller ones by at
// most 2^-39 of it.
#pragma once

#include <cuda_bf16.h>

#include "bsp_ptx.cuh"

namespace bsp {
namespace {

constexpr int kTileRows = 128;
constexpr int kStepK = 256;
constexpr int kStepBytes = kStepK * 2;          // of one row of x in f16
constexpr int kThreads = 256;                   // four octets of rows r, two halves of the steps

__device__ __forceinline__ float pow2_biased(int e)     // 2^(e - 127), e in [0, 254]
{
    return __uint_as_float(e > 0 ? static_cast<uint32_t>(e) << 23 : 0x00400000u);
}

// Eight codes of w as f16.  (Half of them made of the codes' bits, with shifts and masks, instead of
// by conversions: 134 us for 131072 x 8192 where this takes 114.)
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// the E4M3 scale in byte i of w, twice in an f16 pair
__device__ __forceinline__ uint32_t scale_to_f16(uint32_t w, int i)
{
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
        : "=r"(r)
        : "r"(__byte_perm(w, 0, i * 0x11)));
    return r;
}

__device__ __forceinline__ uint32_t word_of(uint4 v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight bf16 of x times `up` in f16
__device__ __forceinline__ uint4 pack_x8(uint4 v, float up)
{
    return make_uint4(pack_f16(bf16lo_to_f32(v.x) * up, bf16hi_to_f32(v.x) * up),
                      pack_f16(bf16lo_to_f32(v.y) * up, bf16hi_to_f32(v.y) * up),
                      pack_f16(bf16lo_to_f32(v.z) * up, bf16hi_to_f32(v.z) * up),
                      pack_f16(bf16lo_to_f32(v.w) * up, bf16hi_to_f32(v.w) * up));
}

// A lane's loads of half a step (128 elements of K): 32 codes of each of its four rows, at t * 32
// of the half, so that four lanes read 64 bytes of a row side by side; and the 16 scales of those
// rows and the 64 elements that hold the lane's two blocks.  Rows past N and elements past K are
// read from the last ones instead: the results of such rows are not stored, and x is zero there.
struct HalfStep {
    uint4 c[4];
    uint4 s;                  // word q: row + 32 q
};

struct GemvWeight {
    const uint8_t* codes;
    const uint8_t* sf;
    int32_t N, K;
};

struct LaneRows {
    const uint8_t* codes;     // of the lane's first row
    const uint8_t* sf;
    uint32_t off[3];          // from there to the other rows' codes
};

// Not the read-only path: the weight may be an earlier kernel's output, and this kernel may have begun
// before that one ended.
__device__ __forceinline__ uint4 ld_once(const void* a)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(a));
    return v;
}

__device__ __forceinline__ LaneRows lane_rows(const GemvWeight& p, int tile, int row_in_tile)
{
    LaneRows r;
    const int row = min(tile * kTileRows + row_in_tile, p.N - 1);
    r.codes = p.codes + static_cast<int64_t>(row) * (p.K / 2);
#pragma unroll
    for (int q = 1; q < 4; ++q)
        r.off[q - 1] = static_cast<uint32_t>(min(row + 32 * q, p.N - 1) - row) * (p.K / 2);
    r.sf = p.sf + static_cast<int64_t>(tile) * (p.K / 64) * 512 + row_in_tile * 16;
    return r;
}

__device__ __forceinline__ void load_half(const GemvWeight& p, const LaneRows& r, int s, int t,
                                          int half, HalfStep& d)
{
    const uint32_t kt = min(s * 4 + 2 * half + (t >> 1), p.K / 64 - 1);
    const uint8_t* a = r.codes + (kt * 32 + (t & 1) * 16);
    d.c[0] = ld_once(a);
    d.c[1] = ld_once(a + r.off[0]);
    d.c[2] = ld_once(a + r.off[1]);
    d.c[3] = ld_once(a + r.off[2]);
    d.s = ld_once(r.sf + kt * 512);
}

// Biased exponent that a row of x goes by: the row is multiplied by 2^(14 - (e - 127)).
__device__ __forceinline__ int x_exponent(uint32_t amax_bits)
{
    return max(15, static_cast<int>(amax_bits >> 23));
}

// x in shared memory: rows of whole steps, a multiple of 128 bytes apart, whose 16-byte pieces c lie at
// c ^ x_key(m, c), so that the eight lanes of one read (four t, two g) are in different banks.
__device__ __forceinline__ int x_key(int m, int c) { return (m & 7) ^ ((c >> 3 & 1) << 1); }

// Where lane t's 16-byte pieces of row m begin (of piece j: that address ^ 16 j).
__device__ __forceinline__ uint32_t x_address(uint32_t row, int m, int t)
{
    return row + (t >> 1) * 128 + (((t & 1) << 2 ^ x_key(m, t << 2)) << 4);
}

__device__ __forceinline__ uint4 ld_shared(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

// The products of half a step: acc[16-row tile][8 rows of x], and xg[nt]: the lane's x_address of one
// row of each 8, in the half.
template <int NT>
__device__ __forceinline__ void mma_half(float (&acc)[2][NT][4], const HalfStep& w,
                                         const uint32_t (&xg)[NT], int offset, int t)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint4 b[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            b[nt] = ld_shared((xg[nt] + offset) ^ (j * 16));
        uint32_t h[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            // scale byte 2 (t % 2) + j / 2 of the row's word
            const uint32_t sc = scale_to_f16(word_of(w.s, q), (t & 1) * 2 + (j >> 1));
            e2m1x8_to_f16(word_of(w.c[q], j), h[q]);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[q][i] = mul_f16x2(h[q][i], sc);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mma_f16(acc[0][nt], h[0][0], h[1][0], h[0][1], h[1][1], b[nt].x, b[nt].y);
            mma_f16(acc[1][nt], h[2][0], h[3][0], h[2][1], h[3][1], b[nt].x, b[nt].y);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mma_f16(acc[0][nt], h[0][2], h[1][2], h[0][3], h[1][3], b[nt].z, b[nt].w);
            mma_f16(acc[1][nt], h[2][2], h[3][2], h[2][3], h[3][3], b[nt].z, b[nt].w);
        }
    }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(in ? 16 : 0)
                 : "memory");
}

}  // namespace
}  // namespace bsp
