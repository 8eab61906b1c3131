// gemv.cu -- nvfp4_gemv: y[m][n] = bf16(g * sum_k x[m][k] w[n][k] + bias[n]) for a few rows of
// bf16 x, w = e2m1(code) * e4m3(scale) in the layout of nvfp4_gemm.  The weight-only form:
// x is not quantized.
//
// What bounds it is reading the weight: 9/16 byte per weight.  Decoding 16 weights costs the
// CUDA cores 8 conversions and 8 products with the scale if the multiply-adds are left to the
// tensor cores, and several times the budget if they are not, so each weight becomes f16 (e2m1 *
// e4m3 has at most 6 significant bits and lies in [2^-10, 2688]: exact) and goes through
// m16n8k16 with fp32 sums, 16 weight rows against 8 rows of x.  x is bf16, whose range f16 lacks:
// it is scaled by a power of two per row of x and piece of K, so that its largest element is in
// [2^14, 2^15); f16 then holds elements down to 2^-28 of that exactly and rounds smaller ones by
// at most 2^-39 of it.
//
// One CTA takes a 128-row tile of the weight (the tile of the scale layout) and a piece of K.  A
// warp takes the 32 rows r, r + 32, r + 64, r + 96 for 8 values of r, whose scales lie in the same
// 16-byte words, and every other 256-element step of K: per step a lane reads 32 bytes of codes of
// each of its four rows and one 16-byte word of scales, all of which it uses.  The products may run
// over k in any order, so these 64 consecutive codes of a row are the k slots that the lane owns
// in 16 products.  The next step's loads are in flight while a step is computed.  The pieces of K
// are a cluster: the CTAs add their sums through distributed shared memory, in order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "bsp_internal.h"
#include "bsp_ptx.cuh"
#include "nvfp4_block.cuh"

namespace bsp {
namespace {

constexpr int kGemvMaxRows = 32;
constexpr int kThreads = 256;
constexpr int kTileRows = 128;
constexpr int kStepK = 256;
constexpr int kStepBytes = kStepK * 2;          // of one row of x in f16
constexpr int kMaxStage = 96 * 1024;            // shared memory for x: two CTAs fit an SM

struct GemvParams {
    const __nv_bfloat16* x;
    const uint8_t* codes;
    const uint8_t* sf;
    const float* scale;
    const __nv_bfloat16* bias;
    __nv_bfloat16* out;
    int32_t M, N, K;
    int32_t steps;            // of K in all
    int32_t cta_steps;        // of one CTA
    int32_t stage_steps;      // of x in shared memory at a time, even
    int32_t wide;             // codes are 32-byte aligned
};

struct StepData {
    uint4 c[4][2];            // 64 codes of each of four rows
    uint4 s;                  // 4 scales of each
};

__device__ __forceinline__ float pow2_biased(int e)     // 2^(e - 127), e in [0, 254]
{
    return __uint_as_float(e > 0 ? static_cast<uint32_t>(e) << 23 : 0x00400000u);
}

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

// four E4M3 scales -> each twice in an f16 pair
__device__ __forceinline__ void scales_to_f16(uint32_t w, uint32_t (&h)[4])
{
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    h[0] = __byte_perm(lo, lo, 0x1010);
    h[1] = __byte_perm(lo, lo, 0x3232);
    h[2] = __byte_perm(hi, hi, 0x1010);
    h[3] = __byte_perm(hi, hi, 0x3232);
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
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
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

// Codes and scales of step s for the warp's rows row0 + 32 q + g, q = 0 .. 3.
__device__ __forceinline__ void load_step(const GemvParams& p, int s, int row0, int g, int t,
                                          StepData& d)
{
    const int kt = s * 4 + t;
    const bool in = kt * 64 < p.K;
    const int64_t row_bytes = p.K / 2;
    const int row = row0 + g;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const bool ok = in && row + 32 * q < p.N;
        const uint8_t* a = p.codes + (row + 32 * q) * row_bytes + kt * 32;
        d.c[q][0] = d.c[q][1] = make_uint4(0, 0, 0, 0);
        if (ok && p.wide) {
            asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(d.c[q][0].x), "=r"(d.c[q][0].y), "=r"(d.c[q][0].z),
                           "=r"(d.c[q][0].w), "=r"(d.c[q][1].x), "=r"(d.c[q][1].y),
                           "=r"(d.c[q][1].z), "=r"(d.c[q][1].w)
                         : "l"(a));
        } else if (ok) {
            d.c[q][0] = __ldg(reinterpret_cast<const uint4*>(a));
            d.c[q][1] = __ldg(reinterpret_cast<const uint4*>(a) + 1);
        }
    }
    d.s = make_uint4(0, 0, 0, 0);
    if (in)
        d.s = __ldg(reinterpret_cast<const uint4*>(
            p.sf + (static_cast<int64_t>(row / kTileRows) * (p.K / 64) + kt) * 512 +
            (row & 31) * 16));
}

// NT: 8-row tiles of x.
template <int NT>
__global__ void __launch_bounds__(kThreads, 2) nvfp4_gemv_kernel(const GemvParams p)
{
    extern __shared__ uint4 xs[];               // x in f16: [nt][step][8][t][rows of the tile]
    __shared__ float part[kTileRows][NT * 8];
    __shared__ uint32_t amax[NT * 8];           // bits of the largest |x| of this piece so far
    griddep_wait();
    griddep_launch_dependents();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int oct = warp & 3, kw = warp >> 2;
    uint32_t rank, pieces;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(pieces));
    const int tile = blockIdx.x / pieces;
    const int row0 = tile * kTileRows + oct * 8;
    const int c0 = rank * p.cta_steps, c1 = min(c0 + p.cta_steps, p.steps);

    StepData cur;
    int s = c0 + kw;
    if (s < c1) load_step(p, s, row0, g, t, cur);

    const int mp = p.M < 8 ? p.M : 8;           // rows of an x tile in shared memory
    const int rows_pow2 = p.M <= 1 ? 1 : 1 << (32 - __clz(p.M - 1));
    const int xm = threadIdx.x & (rows_pow2 - 1), xc = threadIdx.x / rows_pow2;
    const int xstep = kThreads / rows_pow2;
    if (threadIdx.x < NT * 8) amax[threadIdx.x] = 0;

    float acc[2][NT][4] = {};
    int e_acc[NT][2];                           // biased exponents that the columns' sums go by
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) e_acc[nt][0] = e_acc[nt][1] = 15;

    for (int a0 = c0; a0 < c1; a0 += p.stage_steps) {
        const int a1 = min(a0 + p.stage_steps, c1);
        const int chunks = (a1 - a0) * (kStepK / 8), valid = p.K / 8 - a0 * (kStepK / 8);
        const uint4* xrow = reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(xm) * p.K +
                                                           static_cast<int64_t>(a0) * kStepK);
        __syncthreads();                        // amax is set, the last stage is read
        uint32_t top = 0;
        if (xm < p.M)
            for (int i = xc; i < min(chunks, valid); i += xstep) {
                const uint4 v = __ldg(xrow + i);
                const uint32_t a = max_bf16x2(max_bf16x2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                              max_bf16x2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
                top = max(top, max(a << 16, a & 0xFFFF0000u));
            }
        for (int o = 16; o >= rows_pow2; o >>= 1)
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        if (xm < p.M && lane < rows_pow2) atomicMax(&amax[xm], top);
        __syncthreads();
        if (xm < p.M) {
            const int e = max(15, static_cast<int>(amax[xm] >> 23));
            const float up = pow2_biased(268 - e);             // 2^(14 - (e - 127))
            for (int i = xc; i < chunks; i += xstep) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (i < valid) v = __ldg(xrow + i);
                uint4 h;
                h.x = pack_f16(bf16lo_to_f32(v.x) * up, bf16hi_to_f32(v.x) * up);
                h.y = pack_f16(bf16lo_to_f32(v.y) * up, bf16hi_to_f32(v.y) * up);
                h.z = pack_f16(bf16lo_to_f32(v.z) * up, bf16hi_to_f32(v.z) * up);
                h.w = pack_f16(bf16lo_to_f32(v.w) * up, bf16hi_to_f32(v.w) * up);
                // chunk i: step i / 32, lane quarter (i / 8) % 4, eighth i % 8
                const int at = (((xm >> 3) * p.stage_steps + (i >> 5)) * 8 + (i & 7)) * 4 +
                               ((i >> 3) & 3);
                xs[at * mp + (xm & 7)] = h;
            }
        }
        // the sums so far move to this stage's exponents
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int e = max(15, static_cast<int>(amax[nt * 8 + 2 * t + i] >> 23));
                const int d = e - e_acc[nt][i];
                e_acc[nt][i] = e;
                const float f = d < 127 ? pow2_biased(127 - d) : 0.0f;
                acc[0][nt][i] *= f;
                acc[0][nt][i + 2] *= f;
                acc[1][nt][i] *= f;
                acc[1][nt][i + 2] *= f;
            }
        __syncthreads();

        for (; s < a1; s += 2) {
            StepData next;
            if (s + 2 < c1) load_step(p, s + 2, row0, g, t, next);
            uint32_t sc[4][4];
            scales_to_f16(cur.s.x, sc[0]);
            scales_to_f16(cur.s.y, sc[1]);
            scales_to_f16(cur.s.z, sc[2]);
            scales_to_f16(cur.s.w, sc[3]);
#pragma unroll
            for (int jj = 0; jj < 8; ++jj) {
                uint4 b[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int at = ((nt * p.stage_steps + (s - a0)) * 8 + jj) * 4 + t;
                    b[nt] = make_uint4(0, 0, 0, 0);
                    if (nt * 8 + g < p.M) b[nt] = xs[at * mp + g];
                }
                uint32_t h[4][4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 c = cur.c[q][jj >> 2];
                    const uint32_t w = (jj & 3) == 0   ? c.x
                                       : (jj & 3) == 1 ? c.y
                                       : (jj & 3) == 2 ? c.z
                                                       : c.w;
                    e2m1x8_to_f16(w, h[q]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) h[q][i] = mul_f16x2(h[q][i], sc[q][jj >> 1]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_f16(acc[0][nt], h[0][0], h[1][0], h[0][1], h[1][1], b[nt].x, b[nt].y);
                    mma_f16(acc[1][nt], h[2][0], h[3][0], h[2][1], h[3][1], b[nt].x, b[nt].y);
                    mma_f16(acc[0][nt], h[0][2], h[1][2], h[0][3], h[1][3], b[nt].z, b[nt].w);
                    mma_f16(acc[1][nt], h[2][2], h[3][2], h[2][3], h[3][3], b[nt].z, b[nt].w);
                }
            }
            cur = next;
        }
    }

    // ---- sums of the two halves of the warps, then of the cluster's CTAs, in order
    const float gs = __ldg(p.scale);
#pragma unroll
    for (int half = 1; half >= 0; --half) {
        if (kw == half) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int ta = 0; ta < 2; ++ta)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = oct * 8 + g + 64 * ta + 32 * (i >> 1);
                        const int col = nt * 8 + 2 * t + (i & 1);
                        const float v = acc[ta][nt][i] * gs * pow2_biased(e_acc[nt][i & 1] - 14);
                        part[row][col] = half ? v : part[row][col] + v;
                    }
        }
        __syncthreads();
    }
    if (pieces > 1) cluster_sync();
    const int share = kTileRows / pieces;
    for (int i = threadIdx.x; i < share * p.M; i += kThreads) {
        const int m = i / share, row = rank * share + i - m * share;
        const int n = tile * kTileRows + row;
        if (n >= p.N) continue;
        float v = 0.0f;
        if (pieces == 1) {
            v = part[row][m];
        } else {
            const uint32_t at = smem_u32(&part[row][m]);
            for (uint32_t r = 0; r < pieces; ++r) {
                float y;
                asm volatile("ld.shared::cluster.f32 %0, [%1];"
                             : "=f"(y)
                             : "r"(mapa_shared(at, r)));
                v += y;
            }
        }
        if (p.bias) v += __bfloat162float(p.bias[n]);
        p.out[static_cast<int64_t>(m) * p.N + n] = __float2bfloat16_rn(v);
    }
    if (pieces > 1) cluster_sync();             // the others have read this CTA's sums
}

template <int NT>
int launch_gemv(GemvParams p, int dev, int sms, cudaStream_t stream)
{
    static std::atomic<bool> ready[kMaxDevices];
    if (!ready[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(nvfp4_gemv_kernel<NT>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kMaxStage) != cudaSuccess) {
            cudaGetLastError();
            return BSP_ERR_CUDA;
        }
        ready[dev].store(true, std::memory_order_release);
    }
    // pieces of K: as many as give every SM two CTAs, while each has a step for both warp halves
    const int tiles = (p.N + kTileRows - 1) / kTileRows;
    int pieces = 1;
    while (pieces < 8 && tiles * pieces < 2 * sms && pieces * 4 <= p.steps) pieces *= 2;
    p.cta_steps = (p.steps + pieces - 1) / pieces;
    const int step_bytes = kStepBytes * (p.M < 8 ? p.M : 8 * NT);
    p.stage_steps = std::min((p.cta_steps + 1) / 2 * 2, kMaxStage / step_bytes / 2 * 2);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = pieces;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(tiles) * pieces, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.stage_steps) * step_bytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, nvfp4_gemv_kernel<NT>, p) != cudaSuccess) {
        cudaGetLastError();
        return BSP_ERR_CUDA;
    }
    return launch_status();
}

}  // namespace
}  // namespace bsp

extern "C" int nvfp4_gemv(const void* x_bf16, const uint8_t* w_codes, const uint8_t* w_sf,
                          const float* w_scale, const void* bias_bf16, void* out_bf16, int64_t M,
                          int64_t N, int64_t K, bsp_stream_t stream)
{
    using namespace bsp;
    if (M < 0 || N < 0 || K < 0) return BSP_ERR_INVALID_ARG;
    if (M > kGemvMaxRows || K % 64 != 0 || K < 64 || N % 8 != 0 || N > (int64_t{1} << 30) ||
        K > (int64_t{1} << 24))
        return BSP_ERR_UNSUPPORTED_SHAPE;
    if (M == 0 || N == 0) return BSP_OK;
    if (!x_bf16 || !w_codes || !w_sf || !w_scale || !out_bf16) return BSP_ERR_INVALID_ARG;
    if (!aligned16(x_bf16) || !aligned16(w_codes) || !aligned16(w_sf) || !aligned16(bias_bf16) ||
        !aligned16(out_bf16) || (reinterpret_cast<uintptr_t>(w_scale) & 3u))
        return BSP_ERR_MISALIGNED;
    int dev = 0, sms = 0;
    int st = check_device(&dev, &sms);
    if (st != BSP_OK) return st;
    GemvParams p = {};
    p.x = static_cast<const __nv_bfloat16*>(x_bf16);
    p.codes = w_codes;
    p.sf = w_sf;
    p.scale = w_scale;
    p.bias = static_cast<const __nv_bfloat16*>(bias_bf16);
    p.out = static_cast<__nv_bfloat16*>(out_bf16);
    p.M = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.steps = static_cast<int32_t>((K + kStepK - 1) / kStepK);
    p.wide = (reinterpret_cast<uintptr_t>(w_codes) & 31u) == 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (M <= 8) return launch_gemv<1>(p, dev, sms, s);
    if (M <= 16) return launch_gemv<2>(p, dev, sms, s);
    if (M <= 24) return launch_gemv<3>(p, dev, sms, s);
    return launch_gemv<4>(p, dev, sms, s);
}
