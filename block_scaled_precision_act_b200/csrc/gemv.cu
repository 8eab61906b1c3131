// gemv.cu -- nvfp4_gemv: y[m][n] = bf16(g * sum_k x[m][k] w[n][k] + bias[n]) for a few rows of
// bf16 x, w = e2m1(code) * e4m3(scale) in the layout of nvfp4_gemm.  The weight-only form.
//
// What bounds it is reading the weight, 9/16 byte for each, and next to it decoding what was read: 14
// instructions for 8 weights of a lane keep the schedulers busy in half of the cycles, and the loads
// that four warps on each can have in flight bring 5.4 TB/s (131072 x 8192, one row: 112 us at 1965 MHz, and
// 122 to 126 after a tenth of a second of such calls, when the power limit holds the SMs at 1.75 GHz).  With
// more rows the products come on top (16384 x 12288, 16 rows: 40 us, 2.9 TB/s; three CTAs on an SM, whose
// registers spill, took a quarter longer).  Where all CTAs run at once it goes another way (gemv_direct.cu).
//
// Two kernels.  nvfp4_gemv_rows_kernel writes x in f16, times a power of two for each row, to the
// workspace, in the order in which shared memory will hold it.  nvfp4_gemv_kernel: the 256-element K
// steps of all 128-row tiles in a row are cut into equal runs, one for each CTA, so that every SM
// reads the same number of bytes whatever N and K are; a tile that is cut leaves fp32 parts, and the
// last CTA to finish one adds them in order, when its own run has ended.  x comes to shared memory a few
// steps at a time, by one bulk copy and one such chunk ahead; a lane's codes are one step ahead in
// registers, across the ends of tiles too.  (Sums of parts at each end of a tile, with a fence of every
// thread, and 16-byte copies of x by all threads: 44 us for the 16 rows above.)
#include <algorithm>
#include <atomic>

#include "bsp_internal.h"
#include "bsp_ptx.cuh"
#include "gemv_mma.cuh"

namespace bsp {
namespace {

constexpr int kGemvMaxRows = 32;
constexpr int kMaxCtas = 320;
constexpr int kMinSteps = 4;                    // of a run
// Of x in shared memory, twice.  More of it takes from the L1, where loads under way wait: 8 rows of
// 16384 x 12288 took 34 us, 34 with 18 KB and 44 with 51 KB.
constexpr int kChunkBytes = 36 * 1024;
constexpr int kMaxChunk = 16;                   // steps
constexpr int kPoison = 0x7FFFFFFF;             // exponent of a row that is not finite

struct GemvArgs {
    GemvWeight w;
    const float* w_scale;
    const __nv_bfloat16* bias;
    __nv_bfloat16* out;
    const uint8_t* xh;           // [steps][M][512 bytes] f16
    const int32_t* exponent;     // [M] biased exponent that a row goes by, or kPoison
    float* parts;                // [2 * ctas][M][128]
    int32_t* done;               // [tiles] parts that have arrived, zeroed by the rows kernel
    int32_t M;
    int32_t steps;               // of K
    int32_t chunk;               // steps of x in shared memory at a time, even
    int64_t total;               // steps of all tiles
    int32_t stop_loads;          // a CTA's chunks end after that many (tests of the waits; else never)
    uint64_t wait_ns;
    int* status;
};

// One CTA per row of x; a thread takes 8-element pieces.  Also zeroes the counters of the tiles.
__global__ void __launch_bounds__(1024)
    nvfp4_gemv_rows_kernel(const __nv_bfloat16* x, int K, int steps, uint8_t* xh, int32_t* exponent,
                           int32_t* done, int tiles)
{
    __shared__ uint32_t warp_max[32];
    griddep_wait();
    griddep_launch_dependents();
    const int m = blockIdx.x, M = gridDim.x, pieces = steps * (kStepK / 8);
    const uint4* row = reinterpret_cast<const uint4*>(x + static_cast<int64_t>(m) * K);
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < tiles; i += gridDim.x * blockDim.x)
        done[i] = 0;
    uint4 v = make_uint4(0, 0, 0, 0);
    uint32_t top = 0;            // bits of the largest |x|; an infinity or NaN is the largest of all
    for (int i = threadIdx.x; i < pieces; i += blockDim.x) {
        v = i * 8 < K ? row[i] : make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max(u[j] << 16 & 0x7FFFFFFFu, u[j] & 0x7FFF0000u));
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = top;
    __syncthreads();
    top = threadIdx.x % 32 < blockDim.x / 32 ? warp_max[threadIdx.x & 31] : 0;
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    const int e = x_exponent(top);
    if (threadIdx.x == 0) exponent[m] = top < 0x7F800000u ? e : kPoison;
    const float up = pow2_biased(268 - e);       // 2^(14 - (e - 127))
    const bool held = pieces <= static_cast<int>(blockDim.x);      // v still has the piece
    for (int i = threadIdx.x; i < pieces; i += blockDim.x) {
        if (!held) v = i * 8 < K ? row[i] : make_uint4(0, 0, 0, 0);
        const int step = i >> 5, c = i & 31;
        *reinterpret_cast<uint4*>(xh + (static_cast<int64_t>(step) * M + m) * kStepBytes +
                                  (c ^ x_key(m, c)) * 16) = pack_x8(v, up);
    }
}

// First step of CTA i's run, and the CTA whose run holds step s.
__device__ __forceinline__ int64_t run_begin(int64_t total, int ctas, int i)
{
    return total * i / ctas;
}

__device__ __forceinline__ int run_owner(int64_t total, int ctas, int64_t s)
{
    return static_cast<int>(((s + 1) * ctas - 1) / total);
}

// NT: 8-row tiles of x.
template <int NT>
__global__ void __launch_bounds__(kThreads, 2) nvfp4_gemv_kernel(const GemvArgs p)
{
    extern __shared__ uint8_t raw[];            // two chunks of x: [step][M][kStepBytes]
    __shared__ float part[NT * 8][kTileRows + 4];   // the padding spreads a store over the banks
    __shared__ float2 factor[NT * 8];           // 2^e g of a row, in two parts
    __shared__ uint64_t full[2];
    __shared__ int abort_word, joins[2];
    volatile int* abort_flag = &abort_word;
    griddep_launch_dependents();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int oct = warp & 3, kw = warp >> 2;
    const int ctas = gridDim.x, steps = p.steps, M = p.M;
    const int64_t s0 = run_begin(p.total, ctas, blockIdx.x);
    const int run = static_cast<int>(run_begin(p.total, ctas, blockIdx.x + 1) - s0);
    const int tile0 = static_cast<int>(s0 / steps);
    const int k0 = static_cast<int>(s0 - static_cast<int64_t>(tile0) * steps);

    // The step of the run whose codes the warp holds: every other one is its own.  The first are on their
    // way before the rows kernel has ended, which begins only when everything before this call has.
    HalfStep w[2];
    int at_tile = tile0, at_k = k0 + kw;
    while (at_k >= steps) {
        at_k -= steps;
        ++at_tile;
    }
    LaneRows rows = lane_rows(p.w, at_tile, oct * 8 + g);
    if (kw < run) {
        load_half(p.w, rows, at_k, t, 0, w[0]);
        load_half(p.w, rows, at_k, t, 1, w[1]);
    }

    griddep_wait();
    // Chunk c of the run's steps to its buffer: steps follow one another in the workspace, up to the
    // last of K.  Thread 0.  Once a wait has run out no more are brought: the buffer's barrier may still
    // be in the phase of the chunk before, which takes no second arrival.
    const uint32_t pad = -smem_u32(raw) & 127u;
    uint8_t* xs = raw + pad;
    const int step_bytes = M * kStepBytes, buffer = p.chunk * step_bytes;
    int brought = 0;
    const auto bring = [&](int c) {
        if (c >= p.stop_loads || *abort_flag) return;
        brought = c + 1;
        int left = min(p.chunk, run - c * p.chunk);
        int k = static_cast<int>((k0 + static_cast<int64_t>(c) * p.chunk) % steps);
        uint8_t* to = xs + (c & 1) * buffer;
        mbar_arrive_expect_tx(full + (c & 1), left * step_bytes);
        while (left > 0) {
            const int n = min(left, steps - k);
            bulk_load(to, p.xh + static_cast<int64_t>(k) * step_bytes, n * step_bytes, full + (c & 1));
            to += n * step_bytes;
            left -= n;
            k = 0;
        }
    };
    if (threadIdx.x == 0) {
        mbar_init(full, 1);
        mbar_init(full + 1, 1);
        abort_word = 0;
        fence_mbar_init();
        bring(0);
    }
    if (threadIdx.x < NT * 8) {
        const int e = threadIdx.x < M ? p.exponent[threadIdx.x] : 127;
        const float gs = *p.w_scale;
        // x was multiplied by 2^(141 - e)
        factor[threadIdx.x] = e == kPoison ? make_float2(NAN, NAN)
                                           : make_float2(gs, pow2_biased(e - 14));
    }

    // rows of a tile past M read the last row; their columns are not stored
    uint32_t xg[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int m = min(nt * 8 + g, M - 1);
        xg[nt] = x_address(smem_u32(xs) + m * kStepBytes, m, t);
    }

    // thread 0: which of the (at most two) tiles that the run cuts are to be joined here
    int cuts = 0, arrived[2] = {};
    int mine = kw;                               // step of the run
    int r0 = 0;
    for (int tile = tile0; r0 < run; ++tile) {
        const int first = tile == tile0 ? k0 : 0;             // step of the tile that comes at r0
        const int r_end = min(run, r0 + steps - first);
        const bool begins = first == 0, whole = begins && r_end - r0 == steps;
        float acc[2][NT][4] = {};
        for (int r = r0; r < r_end;) {
            const int c = r / p.chunk, in_chunk = r - c * p.chunk;
            if (in_chunk == 0) {
                __syncthreads();                 // nobody reads the other buffer any more
                if (threadIdx.x == 0 && (c + 1) * p.chunk < run) bring(c + 1);
                // if that runs out it is reported, and the results are wrong
                mbar_wait(full + (c & 1), c >> 1 & 1, abort_flag, p.wait_ns, p.status, 130);
                __syncwarp();
            }
            const int r1 = min(r_end, (c + 1) * p.chunk);
            const int base = (c & 1) * buffer - c * buffer;
            for (; mine < r1; mine += 2) {
                const int xo = base + mine * step_bytes;
                const bool more = mine + 2 < run;
                at_k += 2;
                if (at_k >= steps) {             // the next one of the warp's is another tile's
                    do {
                        at_k -= steps;
                        ++at_tile;
                    } while (at_k >= steps);
                    if (more) rows = lane_rows(p.w, at_tile, oct * 8 + g);
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    mma_half<NT>(acc, w[half], xg, xo + half * 256, t);
                    if (more) load_half(p.w, rows, at_k, t, half, w[half]);
                }
            }
            r = r1;
        }
        r0 = r_end;

        // sums of the two halves of the warps
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
                            part[col][r] = half ? acc[ta][nt][i] : part[col][r] + acc[ta][nt][i];
                        }
            }
            __syncthreads();
        }
        const int r = threadIdx.x & (kTileRows - 1), m0 = threadIdx.x / kTileRows;
        constexpr int kSide = kThreads / kTileRows;
        const int n = tile * kTileRows + r;
        const bool in = n < p.w.N;
        const float bias = in && p.bias ? __bfloat162float(p.bias[n]) : 0.0f;
        const auto finish = [&](int m, float v) {
            const float2 f = factor[m];
            if (in) p.out[static_cast<int64_t>(m) * p.w.N + n] = __float2bfloat16_rn(v * f.x * f.y + bias);
        };
        if (whole) {
            for (int m = m0; m < M; m += kSide) finish(m, part[m][r]);
        } else {
            const int64_t step = static_cast<int64_t>(2) * M * kTileRows;
            float* own = p.parts + blockIdx.x * step + (begins ? step / 2 : 0) + r;
            for (int m = m0; m < M; m += kSide) own[m * kTileRows] = part[m][r];
            __syncthreads();
            if (threadIdx.x == 0) {              // what comes back is looked at when the run has ended
                __threadfence();
                const int n = atomicAdd(p.done + tile, 1);
                if (cuts == 0)
                    arrived[0] = n;
                else
                    arrived[1] = n;
                ++cuts;
            }
        }
        __syncthreads();                         // `part` is read
    }

    // The parts of the tiles whose last part was brought here.  Cut tiles of a run: its first, its last.
    const int tile1 = static_cast<int>((s0 + run - 1) / steps);
    const bool first_cut = k0 != 0 || run < steps, last_cut = (s0 + run) % steps != 0;
    if (threadIdx.x == 0) {
        int i = 0;
        for (int k = 0; k < 2; ++k) {
            const int tile = k ? tile1 : tile0;
            joins[k] = -1;
            if (k ? !last_cut || tile1 == tile0 : !first_cut) continue;
            const int64_t t0 = static_cast<int64_t>(tile) * steps;
            const int others = run_owner(p.total, ctas, t0 + steps - 1) - run_owner(p.total, ctas, t0);
            if ((i++ ? arrived[1] : arrived[0]) == others) joins[k] = tile;
        }
        __threadfence();
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
        const int tile = joins[k];
        if (tile < 0) continue;
        __threadfence();
        const int64_t t0 = static_cast<int64_t>(tile) * steps;
        const int o0 = run_owner(p.total, ctas, t0), o1 = run_owner(p.total, ctas, t0 + steps - 1);
        const int r = threadIdx.x & (kTileRows - 1), n = tile * kTileRows + r;
        const float bias = n < p.w.N && p.bias ? __bfloat162float(p.bias[n]) : 0.0f;
        // part 0 is the second slot of CTA o0, the others the first of theirs
        const int64_t step = static_cast<int64_t>(2) * M * kTileRows;
        const float* other = p.parts + o0 * step + r;
        for (int m = threadIdx.x / kTileRows; m < M; m += kThreads / kTileRows) {
            const float* of = other + m * kTileRows;
            float v = __ldcg(of + step / 2);
            for (int i0 = 1; i0 <= o1 - o0; i0 += 4) {
                float y[4];                      // four parts' loads in flight
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y[i] = i0 + i <= o1 - o0 ? __ldcg(of + (i0 + i) * step) : 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) v += y[i];
            }
            const float2 f = factor[m];
            if (n < p.w.N)
                p.out[static_cast<int64_t>(m) * p.w.N + n] = __float2bfloat16_rn(v * f.x * f.y + bias);
        }
    }
    // a load that was waited for in vain must land before shared memory is freed
    if (threadIdx.x == 0 && *abort_flag)
        for (int c = max(0, brought - 2); c < brought; ++c)
            drain_wait(full + (c & 1), c >> 1 & 1, p.wait_ns, p.status);
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// Workspace: x in f16, parts, exponents, counters.
struct GemvLayout {
    int64_t parts, exponent, done, bytes;
    int32_t steps, tiles;
};

GemvLayout gemv_layout(int64_t M, int64_t N, int64_t K)
{
    GemvLayout l;
    l.steps = static_cast<int32_t>((K + kStepK - 1) / kStepK);
    l.tiles = static_cast<int32_t>((N + kTileRows - 1) / kTileRows);
    l.parts = up256(static_cast<int64_t>(l.steps) * M * kStepBytes);
    l.exponent = l.parts + static_cast<int64_t>(2) * kMaxCtas * M * kTileRows * 4;
    l.done = up256(l.exponent + M * 4);
    l.bytes = up256(l.done + static_cast<int64_t>(l.tiles) * 4);
    return l;
}

int gemv_check(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0) return BSP_ERR_INVALID_ARG;
    if (M > kGemvMaxRows || K % 64 != 0 || K < 64 || N % 8 != 0 || N > (int64_t{1} << 30) ||
        K > (int64_t{1} << 24))
        return BSP_ERR_UNSUPPORTED_SHAPE;
    return BSP_OK;
}

template <int NT>
int launch_gemv(GemvArgs a, int dev, int sms, cudaStream_t s)
{
    static std::atomic<bool> ready[kMaxDevices];
    constexpr int kSmem = 2 * kChunkBytes + 128;
    if (!ready[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(nvfp4_gemv_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmem) != cudaSuccess) {
            cudaGetLastError();
            return BSP_ERR_CUDA;
        }
        ready[dev].store(true, std::memory_order_release);
    }
    a.chunk = std::clamp(kChunkBytes / (a.M * kStepBytes) / 2 * 2, 2, kMaxChunk);
    const int64_t ctas = std::min<int64_t>(std::min(kMaxCtas, 2 * sms),
                                           (a.total + kMinSteps - 1) / kMinSteps);
    const size_t smem = static_cast<size_t>(2) * a.chunk * a.M * kStepBytes + 128;
    if (launch_kernel(nvfp4_gemv_kernel<NT>, static_cast<unsigned>(ctas), kThreads, smem, s, true,
                      a) != cudaSuccess) {
        cudaGetLastError();
        return BSP_ERR_CUDA;
    }
    return launch_status();
}

static_assert(2 * kGemvMaxRows * kStepBytes <= kChunkBytes, "two steps of 32 rows fit a chunk");

}  // namespace
}  // namespace bsp

extern "C" {

int64_t nvfp4_gemv_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    const int st = bsp::gemv_check(M, N, K);
    return st != BSP_OK ? st : bsp::gemv_layout(M, N, K).bytes;
}

int nvfp4_gemv(const void* x_bf16, const uint8_t* w_codes, const uint8_t* w_sf,
               const float* w_scale, const void* bias_bf16, void* out_bf16, int64_t M, int64_t N,
               int64_t K, void* workspace, int64_t workspace_bytes, bsp_stream_t stream)
{
    using namespace bsp;
    int st = gemv_check(M, N, K);
    if (st != BSP_OK) return st;
    if (M == 0 || N == 0) return BSP_OK;
    if (!x_bf16 || !w_codes || !w_sf || !w_scale || !out_bf16) return BSP_ERR_INVALID_ARG;
    const GemvLayout l = gemv_layout(M, N, K);
    if (!workspace || workspace_bytes < l.bytes) return BSP_ERR_INVALID_ARG;
    if (!aligned16(x_bf16) || !aligned16(w_codes) || !aligned16(w_sf) || !aligned16(bias_bf16) ||
        !aligned16(out_bf16) || !aligned16(workspace) ||
        (reinterpret_cast<uintptr_t>(w_scale) & 3u))
        return BSP_ERR_MISALIGNED;
    int dev = 0, sms = 0;
    st = check_device(&dev, &sms);
    if (st != BSP_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const GemvSplit split = gemv_one_launch(M, N, K, sms);
    if (split.pieces > 0)
        return gemv_direct(split, static_cast<const __nv_bfloat16*>(x_bf16), w_codes, w_sf, w_scale,
                           static_cast<const __nv_bfloat16*>(bias_bf16),
                           static_cast<__nv_bfloat16*>(out_bf16), M, N, K, dev, s);
    auto* ws = static_cast<uint8_t*>(workspace);
    GemvArgs a = {};
    a.w.codes = w_codes;
    a.w.sf = w_sf;
    a.w.N = static_cast<int32_t>(N);
    a.w.K = static_cast<int32_t>(K);
    a.w_scale = w_scale;
    a.bias = static_cast<const __nv_bfloat16*>(bias_bf16);
    a.out = static_cast<__nv_bfloat16*>(out_bf16);
    a.xh = ws;
    a.exponent = reinterpret_cast<int32_t*>(ws + l.exponent);
    a.parts = reinterpret_cast<float*>(ws + l.parts);
    a.done = reinterpret_cast<int32_t*>(ws + l.done);
    a.M = static_cast<int32_t>(M);
    a.steps = l.steps;
    a.total = static_cast<int64_t>(l.tiles) * l.steps;
    a.stop_loads = load_stall();
    a.wait_ns = wait_limit_ns();
    a.status = device_status_ptr(dev);
    const int threads = std::min(1024, l.steps * (kStepK / 8));
    if (launch_kernel(nvfp4_gemv_rows_kernel, static_cast<unsigned>(M), static_cast<unsigned>(threads), 0,
                      s, true, static_cast<const __nv_bfloat16*>(x_bf16), a.w.K, a.steps, ws,
                      reinterpret_cast<int32_t*>(ws + l.exponent),
                      reinterpret_cast<int32_t*>(ws + l.done), l.tiles) != cudaSuccess) {
        cudaGetLastError();
        return BSP_ERR_CUDA;
    }
    if (M <= 8) return launch_gemv<1>(a, dev, sms, s);
    if (M <= 16) return launch_gemv<2>(a, dev, sms, s);
    if (M <= 24) return launch_gemv<3>(a, dev, sms, s);
    return launch_gemv<4>(a, dev, sms, s);
}

}  // extern "C"
