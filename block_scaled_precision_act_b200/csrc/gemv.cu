// gemv.cu -- nvfp4_gemv: y[m][n] = bf16(g * sum_k x[m][k] w[n][k] + bias[n]) for a few rows of
// bf16 x, w = e2m1(code) * e4m3(scale) in the layout of nvfp4_gemm.  The weight-only form:
// x is not quantized.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bsp_internal.h"
#include "bsp_ptx.cuh"
#include "nvfp4_block.cuh"

namespace bsp {
namespace {

constexpr int kGemvMaxRows = 32;
constexpr int kThreads = 256;

__device__ __forceinline__ void e2m1x2_decode(uint32_t byte, float& lo, float& hi)
{
    uint32_t h2;
    asm("{\n\t.reg .b8 c;\n\tcvt.u8.u32 c, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}"
        : "=r"(h2)
        : "r"(byte));
    const __half2 h = *reinterpret_cast<__half2*>(&h2);
    lo = __low2float(h);
    hi = __high2float(h);
}

// One warp per weight row; a lane takes 16-element blocks.  MT rows of x at a time.
template <int MT>
__global__ void __launch_bounds__(kThreads)
    nvfp4_gemv_kernel(const __nv_bfloat16* x, const uint8_t* codes, const uint8_t* sf,
                      const float* scale, const __nv_bfloat16* bias, __nv_bfloat16* out, int M,
                      int64_t N, int64_t K)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t n = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (n >= N) return;
    const int64_t kb4 = K / 64;
    const float g = __ldg(scale);
    for (int m0 = 0; m0 < M; m0 += MT) {
        float acc[MT] = {};
        for (int64_t kb = lane; kb < K / 16; kb += 32) {
            const uint2 c = __ldg(reinterpret_cast<const uint2*>(codes + n * (K / 2) + kb * 8));
            const float s = e4m3_to_f32(__ldg(sf + sf_mma_offset(n, kb, kb4)));
            float w[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t word = i < 4 ? c.x : c.y;
                e2m1x2_decode(word >> (8 * (i & 3)) & 0xFFu, w[2 * i], w[2 * i + 1]);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (m0 + m >= M) break;
                const uint4* xp = reinterpret_cast<const uint4*>(x + (m0 + m) * K + kb * 16);
                const uint4 a = __ldg(xp), b = __ldg(xp + 1);
                const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                float t = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    t = fmaf(w[2 * i], bf16lo_to_f32(u[i]), t);
                    t = fmaf(w[2 * i + 1], bf16hi_to_f32(u[i]), t);
                }
                acc[m] = fmaf(t, s, acc[m]);
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float v = acc[m];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            if (lane == 0 && m0 + m < M)
                out[(m0 + m) * N + n] =
                    __float2bfloat16_rn(v * g + (bias ? __bfloat162float(bias[n]) : 0.0f));
        }
    }
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
    const auto* x = static_cast<const __nv_bfloat16*>(x_bf16);
    const auto* bias = static_cast<const __nv_bfloat16*>(bias_bf16);
    auto* out = static_cast<__nv_bfloat16*>(out_bf16);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const unsigned grid = static_cast<unsigned>((N + kThreads / 32 - 1) / (kThreads / 32));
    const int m = static_cast<int>(M);
    cudaError_t e =
        M == 1 ? launch_kernel(nvfp4_gemv_kernel<1>, grid, kThreads, 0, s, true, x, w_codes, w_sf,
                               w_scale, bias, out, m, N, K)
               : launch_kernel(nvfp4_gemv_kernel<8>, grid, kThreads, 0, s, true, x, w_codes, w_sf,
                               w_scale, bias, out, m, N, K);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return BSP_ERR_CUDA;
    }
    return launch_status();
}
