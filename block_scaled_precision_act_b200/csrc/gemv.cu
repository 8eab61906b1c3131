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
    int32_t tiles, groups;    // row tiles, and clusters that share them
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

// the E4M3 scale in the low byte, twice in an f16 pair
__device__ __forceinline__ uint32_t scale_to_f16(uint32_t w)
{
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
        : "=r"(r)
        : "r"(__byte_perm(w, 0, 0x0000)));
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

// A lane's loads of a step: half 0 or 1 of its 64 codes of the rows row + 32 q, and the four
// scales of each.  Outside the weight they are zeros.
__device__ __forceinline__ void load_codes(const GemvParams& p, int s, int row, int t, int half,
                                           uint4 (&c)[4])
{
    const int kt = s * 4 + t;
    const uint8_t* a = p.codes + static_cast<int64_t>(row) * (p.K / 2) + kt * 32 + 16 * half;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        c[q] = make_uint4(0, 0, 0, 0);
        if (kt * 64 < p.K && row + 32 * q < p.N)
            c[q] = __ldg(reinterpret_cast<const uint4*>(a + static_cast<int64_t>(16 * q) * p.K));
    }
}

__device__ __forceinline__ uint4 load_scales(const GemvParams& p, int s, int row, int t)
{
    const int kt = s * 4 + t;
    if (kt * 64 >= p.K) return make_uint4(0, 0, 0, 0);
    return __ldg(reinterpret_cast<const uint4*>(
        p.sf + (static_cast<int64_t>(row / kTileRows) * (p.K / 64) + kt) * 512 + (row & 31) * 16));
}

// Biased exponent that a row of x goes by: the row is multiplied by 2^(14 - (e - 127)).
__device__ __forceinline__ int x_exponent(uint32_t amax_bits)
{
    return max(15, static_cast<int>(amax_bits >> 23));
}

// Steps [a0, a1) of x to shared memory in f16, in the order in which the products read them:
// [x tile][step][eighth of a lane's 64 elements][lane quarter t][row].  amax: bits of the largest
// |x| of each row so far.  Every thread calls; the stage is readable on return.
template <int NT>
__device__ __forceinline__ void stage_x(const GemvParams& p, int a0, int a1, int mp, uint4* xs,
                                        uint32_t* amax)
{
    constexpr int kBatch = 4;                   // loads of a thread in flight
    const int lane = threadIdx.x & 31;
    const int rows = p.M <= 1 ? 1 : 1 << (32 - __clz(p.M - 1));     // a power of two
    const int m = threadIdx.x & (rows - 1), first = threadIdx.x / rows, stride = kThreads / rows;
    const int chunks = (a1 - a0) * (kStepK / 8), valid = p.K / 8 - a0 * (kStepK / 8);
    const uint4* src = reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(m) * p.K +
                                                      static_cast<int64_t>(a0) * kStepK);
    uint4 v[kBatch];
    const auto load = [&](int i0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * stride;
            v[j] = make_uint4(0, 0, 0, 0);
            if (m < p.M && i < chunks && i < valid) v[j] = __ldg(src + i);
        }
    };
    uint32_t top = 0;
    for (int i0 = first; i0 < chunks; i0 += kBatch * stride) {
        load(i0);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const uint32_t a =
                max_bf16x2(max_bf16x2(v[j].x & 0x7FFF7FFFu, v[j].y & 0x7FFF7FFFu),
                           max_bf16x2(v[j].z & 0x7FFF7FFFu, v[j].w & 0x7FFF7FFFu));
            top = max(top, max(a << 16, a & 0xFFFF0000u));
        }
    }
    for (int o = 16; o >= rows; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (m < p.M && lane < rows) atomicMax(&amax[m], top);
    __syncthreads();
    if (m < p.M) {
        const int e = x_exponent(amax[m]);
        const float up = pow2_biased(268 - e);                 // 2^(14 - (e - 127))
        const bool once = chunks <= kBatch * stride;           // still in registers
        for (int i0 = first; i0 < chunks; i0 += kBatch * stride) {
            if (!once) load(i0);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int i = i0 + j * stride;
                if (i >= chunks) break;
                uint4 h;
                h.x = pack_f16(bf16lo_to_f32(v[j].x) * up, bf16hi_to_f32(v[j].x) * up);
                h.y = pack_f16(bf16lo_to_f32(v[j].y) * up, bf16hi_to_f32(v[j].y) * up);
                h.z = pack_f16(bf16lo_to_f32(v[j].z) * up, bf16hi_to_f32(v[j].z) * up);
                h.w = pack_f16(bf16lo_to_f32(v[j].w) * up, bf16hi_to_f32(v[j].w) * up);
                const int at = (((m >> 3) * p.stage_steps + (i >> 5)) * 8 + (i & 7)) * 4 +
                               ((i >> 3) & 3);
                xs[at * mp + (m & 7)] = h;
            }
        }
    }
    __syncthreads();
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
    int tile = blockIdx.x / pieces;
    const int c0 = rank * p.cta_steps, c1 = min(c0 + p.cta_steps, p.steps);

    // in registers: the codes of the step at hand in two halves, each replaced by the next
    // step's as soon as it is used, and the scales
    uint4 c[2][4], sf;
    if (c0 + kw < c1) {
        const int row = tile * kTileRows + oct * 8 + g;
        load_codes(p, c0 + kw, row, t, 0, c[0]);
        sf = load_scales(p, c0 + kw, row, t);
        load_codes(p, c0 + kw, row, t, 1, c[1]);
    }
    if (threadIdx.x < NT * 8) amax[threadIdx.x] = 0;
    __syncthreads();

    const int mp = p.M < 8 ? p.M : 8;           // rows of an x tile in shared memory
    const float gs = __ldg(p.scale);

  for (; tile < p.tiles; tile += p.groups) {
    const int row = tile * kTileRows + oct * 8 + g;
    int s = c0 + kw;
    float acc[2][NT][4] = {};
    for (int a0 = c0; a0 < c1; a0 += p.stage_steps) {
        const int a1 = min(a0 + p.stage_steps, c1);
        // x stays in shared memory from one tile to the next when its piece fits there
        if (tile == static_cast<int>(blockIdx.x / pieces) || c1 - c0 > p.stage_steps) {
            int e_old[NT][2];                   // biased exponents that the columns' sums go by
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    e_old[nt][i] = a0 == c0 ? 0 : x_exponent(amax[nt * 8 + 2 * t + i]);
            __syncthreads();                    // the last stage and its exponents are read
            if (a0 == c0 && tile != static_cast<int>(blockIdx.x / pieces)) {
                if (threadIdx.x < NT * 8) amax[threadIdx.x] = 0;
                __syncthreads();
            }
            stage_x<NT>(p, a0, a1, mp, xs, amax);
            if (a0 != c0) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int d = x_exponent(amax[nt * 8 + 2 * t + i]) - e_old[nt][i];
                        const float f = d < 127 ? pow2_biased(127 - d) : 0.0f;
                        acc[0][nt][i] *= f;
                        acc[0][nt][i + 2] *= f;
                        acc[1][nt][i] *= f;
                        acc[1][nt][i + 2] *= f;
                    }
            }
        }

        for (; s < a1; s += 2) {
            // the step after the last is the next tile's first
            const bool wrap = s + 2 >= c1;
            const int s_next = wrap ? c0 + kw : s + 2;
            const int row_next = row + (wrap ? p.groups * kTileRows : 0);
            const bool more = !wrap || tile + p.groups < p.tiles;
            uint4 sf_next;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int jj = 4 * half + j;
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
                        const uint32_t w = word_of(c[half][q], j);
                        const uint32_t sc = scale_to_f16(word_of(sf, q) >> (8 * (jj >> 1)));
                        e2m1x8_to_f16(w, h[q]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) h[q][i] = mul_f16x2(h[q][i], sc);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f16(acc[0][nt], h[0][0], h[1][0], h[0][1], h[1][1], b[nt].x, b[nt].y);
                        mma_f16(acc[1][nt], h[2][0], h[3][0], h[2][1], h[3][1], b[nt].x, b[nt].y);
                        mma_f16(acc[0][nt], h[0][2], h[1][2], h[0][3], h[1][3], b[nt].z, b[nt].w);
                        mma_f16(acc[1][nt], h[2][2], h[3][2], h[2][3], h[3][3], b[nt].z, b[nt].w);
                    }
                }
                if (more) {
                    load_codes(p, s_next, row_next, t, half, c[half]);
                    if (half == 0) sf_next = load_scales(p, s_next, row_next, t);
                }
            }
            sf = sf_next;
        }
    }

    // ---- sums of the two halves of the warps, then of the cluster's CTAs, in order
#pragma unroll
    for (int half = 1; half >= 0; --half) {
        if (kw == half) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int ta = 0; ta < 2; ++ta)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = oct * 8 + g + 64 * ta + 32 * (i >> 1);
                        const int col = nt * 8 + 2 * t + (i & 1);
                        const float v = acc[ta][nt][i] * gs *
                                        pow2_biased(x_exponent(amax[col]) - 14);
                        part[r][col] = half ? v : part[r][col] + v;
                    }
        }
        __syncthreads();
    }
    if (pieces > 1) cluster_sync();
    const int share = kTileRows / pieces;
    for (int i = threadIdx.x; i < share * p.M; i += kThreads) {
        const int m = i / share, r = rank * share + i - m * share;
        const int n = tile * kTileRows + r;
        if (n >= p.N) continue;
        float v = 0.0f;
        if (pieces == 1) {
            v = part[r][m];
        } else {
            const uint32_t at = smem_u32(&part[r][m]);
            for (uint32_t j = 0; j < pieces; ++j) {
                float y;
                asm volatile("ld.shared::cluster.f32 %0, [%1];"
                             : "=f"(y)
                             : "r"(mapa_shared(at, j)));
                v += y;
            }
        }
        if (p.bias) v += __bfloat162float(p.bias[n]);
        p.out[static_cast<int64_t>(m) * p.N + n] = __float2bfloat16_rn(v);
    }
    // the others have read this CTA's sums, before they are written again or the CTA ends
    if (pieces > 1)
        cluster_sync();
    else
        __syncthreads();
  }
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
    // Pieces of K, and clusters ("groups") that take the row tiles in turn, two CTAs to an SM:
    // the split whose busiest CTA has the least to do, counting one step for each tile's sums.
    p.tiles = (p.N + kTileRows - 1) / kTileRows;
    int pieces = 1;
    int64_t best = INT64_MAX;
    for (int c = 1; c <= 8 && (c == 1 || 2 * c <= p.steps); c *= 2) {
        const int groups = std::min(p.tiles, std::max(1, 2 * sms / c));
        const int64_t cost = static_cast<int64_t>((p.tiles + groups - 1) / groups) *
                             ((p.steps + c - 1) / c + 1);
        if (cost < best) {
            best = cost;
            pieces = c;
            p.groups = groups;
        }
    }
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
    cfg.gridDim = dim3(static_cast<unsigned>(p.groups) * pieces, 1, 1);
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
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (M <= 8) return launch_gemv<1>(p, dev, sms, s);
    if (M <= 16) return launch_gemv<2>(p, dev, sms, s);
    if (M <= 24) return launch_gemv<3>(p, dev, sms, s);
    return launch_gemv<4>(p, dev, sms, s);
}
