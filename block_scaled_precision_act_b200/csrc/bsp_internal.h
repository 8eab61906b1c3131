// bsp_internal.h -- host-side helpers shared by the library's translation units.
#pragma once

#include <cstdint>
#include <utility>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "bsp.h"

namespace bsp {

// Devices the library keeps per-device state for (ids 0 .. kMaxDevices - 1; check_device
// refuses others before any of that state is touched).
constexpr int kMaxDevices = 64;

// Returns BSP_OK when the current device is compute capability 10.0; caches per device.
int check_device(int* device_out, int* num_sms_out);

// Device address of the current device's status word (int[2]: code, where).
int* device_status_ptr(int device);

// Bounded-wait limit for kernels, in nanoseconds.
uint64_t wait_limit_ns();

// Loads after which a CTA of the decode operators stops loading (bsp_testing_set_load_stall).
int32_t load_stall();

// Tensor map of a paged cache [groups][tokens][D] of bytes, with boxes of box_tokens x 128 bytes in
// the 128-byte swizzle (bytes past D are zeros).
int make_page_map(CUtensorMap* m, const void* base, uint64_t D, uint64_t tokens, uint64_t groups,
                  uint32_t box_tokens);

// nvfp4_gemv in one launch: the pieces of K that a tile is cut into and the CTAs of an SM, and the
// launch.  No pieces: for these sizes it is not the faster way.
struct GemvSplit {
    int pieces, per_sm;
};
GemvSplit gemv_one_launch(int64_t M, int64_t N, int64_t K, int sms);
int gemv_direct(const GemvSplit& split, const __nv_bfloat16* x, const uint8_t* w_codes,
                const uint8_t* w_sf, const float* w_scale, const __nv_bfloat16* bias,
                __nv_bfloat16* out, int64_t M, int64_t N, int64_t K, int dev, cudaStream_t stream);

// nvfp4_gemm (nvf4) / fp8r_gemm launched right after the library's activation quantizer
// wrote `a` (and `a_sf`): same results, but the weight operand's first stages are fetched
// while that quantizer finishes (the quantizer never writes the weights).
int gemm_after_quantizer(bool nvf4, const uint8_t* a, const uint8_t* a_sf, const float* a_scale,
                         const uint8_t* w, const uint8_t* w_sf, const float* w_scale,
                         const void* bias_bf16, void* out_bf16, int64_t M, int64_t N, int64_t K,
                         bsp_stream_t stream);

// nvfp4_quantize_act with an optional per-call global scale: when `partials` is not null,
// g is reduced from the `npartials` per-CTA maxima of |x| there (fp32 bit patterns) and
// published at `gout`; `global_scale` is then unused.
int quantize_act_impl(const void* x_bf16, int64_t M, int64_t K, const float* global_scale,
                      uint8_t* codes, uint8_t* scales, int layout, bsp_stream_t stream,
                      const uint32_t* partials, int npartials, float* gout);

// Slots of per-CTA maxima the dynamic path keeps in the linear workspace.
constexpr int kDynamicPartials = 2048;

// amax pass into `partials`, then the quantizer reducing them (MMA scale layout).
int dynamic_quantize_front(const void* x_bf16, int64_t M, int64_t K, uint32_t* partials,
                           float* g_out, uint8_t* codes, uint8_t* scales, bsp_stream_t stream);

// Launch `kernel`; with `pdl` the launch allows programmatic stream serialisation, so
// the grid may start (prologue: barriers, TMEM, tensor-map prefetch, or just being
// scheduled) while the preceding grid in the stream finishes.  Every kernel launched
// this way executes griddep_wait() before its first read of an input or write of an
// output.
template <typename... Params, typename... Args>
cudaError_t launch_kernel(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem,
                          cudaStream_t s, bool pdl, Args&&... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// A grid that waits for the one in front (griddep_wait) must not hold tensor memory which that one still
// asks for.  The GEMMs let their dependents begin before they have theirs: so a CTA of theirs leaves an SM
// no shared memory for a CTA of the other kernel that takes tensor memory before it waits,
// fp8kv_attention_kernel, which in turn lets its dependents begin only after it has its own.
constexpr int kSmemOfSm = 228 * 1024, kSmemOfCta = 1024;        // the latter: reserved for each CTA
constexpr int kLeastSmemWithTmem = 48 * 1024;
constexpr int kLeastSmemOfGemm = kSmemOfSm - 2 * kSmemOfCta - kLeastSmemWithTmem;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int launch_status()
{
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

}  // namespace bsp
