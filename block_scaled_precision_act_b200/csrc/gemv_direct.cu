// gemv_direct.cu -- nvfp4_gemv in one launch, where the row tiles' CTAs run at once (or K is short):
//     y[m][n] = bf16(g * sum_k x[m][k] w[n][k] + bias[n]),   w = e2m1(code) * e4m3(scale).
//
// A small weight is read in a microsecond or two, so what bounds the call is latency: a launch, one
// round to memory and one through the sums.  A cluster of up to eight CTAs takes a 128-row tile of
// the weight (the tile of the scale layout), each a piece of K, and adds its sums through distributed
// shared memory, in order.  Every other 256-element step of a piece belongs to one half of the warps
// (gemv_mma.cuh).  All of a warp's first step is asked for before x is staged, and each half of the
// next as soon as one is used.  x is scaled for each row and piece of K.
// 1024 x 1024, one row: 3.9 us; 4096 x 4096: 6.2 us (1.5 TB/s); 18944 x 2048: 8.3 us (2.6 TB/s).
#include <algorithm>
#include <atomic>

#include "bsp_internal.h"
#include "bsp_ptx.cuh"
#include "gemv_mma.cuh"
#include "nvfp4_block.cuh"

namespace bsp {
namespace {

constexpr int kMaxPieces = 8;
constexpr int kMaxStage = 96 * 1024;            // shared memory for x: two CTAs fit an SM
constexpr int kFewSteps = 6;
constexpr int kManySteps = 24;

struct DirectParams {
    GemvWeight w;
    const __nv_bfloat16* x;
    const float* scale;
    const __nv_bfloat16* bias;
    __nv_bfloat16* out;
    int32_t M;
    int32_t steps;            // of K in all
    int32_t row_bytes;        // of a row of x in shared memory
};

// Steps [a0, a1) of x, a1 > a0, to shared memory in f16; beyond K it is zeros.  amax: bits of the largest
// |x| of each row, 0 before.  A warp takes one step of one row at a time and copies all of its own first,
// so that their latencies overlap; a lane touches no other's.  Every thread calls; the stage is readable
// on return.
__device__ __forceinline__ void stage_x(const DirectParams& p, int a0, int a1, uint8_t* xs,
                                        uint32_t* amax)
{
    constexpr int kWarps = kThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int steps = a1 - a0;
    const auto piece = [&](int m, int s) {
        return reinterpret_cast<uint4*>(xs + m * p.row_bytes + s * kStepBytes) + (lane ^ x_key(m, lane));
    };
    // units (row m, step s) go to the warps in turn
    const int m0 = warp / steps, s0 = warp - m0 * steps;
    const int dm = kWarps / steps, ds = kWarps - dm * steps;
    for (int m = m0, s = s0; m < p.M;) {
        const int k = (a0 + s) * kStepK + lane * 8;
        const bool in = k < p.w.K;
        cp_async16(smem_u32(piece(m, s)),
                   p.x + (in ? static_cast<int64_t>(m) * p.w.K + k : 0), in);
        m += dm;
        s += ds;
        if (s >= steps) {
            s -= steps;
            ++m;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    for (int m = m0, s = s0; m < p.M;) {
        const uint4 v = *piece(m, s);
        const uint32_t a = max_bf16x2(max_bf16x2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                      max_bf16x2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, max(a << 16, a & 0xFFFF0000u));
        if (lane == 0) atomicMax(&amax[m], top);
        m += dm;
        s += ds;
        if (s >= steps) {
            s -= steps;
            ++m;
        }
    }
    __syncthreads();
    for (int m = m0, s = s0; m < p.M;) {
        uint4* at = piece(m, s);
        const float up = pow2_biased(268 - x_exponent(amax[m]));     // 2^(14 - (e - 127))
        const uint4 v = *at;
        *at = pack_x8(v, up);
        m += dm;
        s += ds;
        if (s >= steps) {
            s -= steps;
            ++m;
        }
    }
    __syncthreads();
}

// NT: 8-row tiles of x; PER: CTAs of an SM.  Grid: the row tiles' clusters.
template <int NT, int PER>
__global__ void __launch_bounds__(kThreads, PER) nvfp4_gemv_direct_kernel(const DirectParams p)
{
    extern __shared__ uint8_t raw[];            // x in f16, from the next multiple of 128
    __shared__ float part[NT * 8][kTileRows + 4];   // the padding spreads a store over the banks
    __shared__ uint32_t amax[NT * 8];           // bits of the largest |x| of this piece
    griddep_wait();
    griddep_launch_dependents();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int oct = warp & 3, kw = warp >> 2;
    uint32_t rank, pieces;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(pieces));
    const int tile = blockIdx.x / pieces;
    const int c0 = p.steps * rank / pieces, c1 = p.steps * (rank + 1) / pieces;

    // in registers: the two halves of the step at hand, each replaced by the next step's as soon
    // as it is used
    HalfStep w[2];
    const LaneRows rows = lane_rows(p.w, tile, oct * 8 + g);
    if (c0 + kw < c1) {
        load_half(p.w, rows, c0 + kw, t, 0, w[0]);
        load_half(p.w, rows, c0 + kw, t, 1, w[1]);
    }
    if (threadIdx.x < NT * 8) amax[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t pad = -smem_u32(raw) & 127u;
    stage_x(p, c0, c1, raw + pad, amax);

    // rows of a tile past M read the last row; their columns are not stored
    uint32_t xg[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int m = min(nt * 8 + g, p.M - 1);
        xg[nt] = x_address(smem_u32(raw) + pad + m * p.row_bytes, m, t);
    }
    float acc[2][NT][4] = {};
    for (int s = c0 + kw; s < c1; s += 2) {
        const int xo = (s - c0) * kStepBytes;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            mma_half<NT>(acc, w[half], xg, xo + half * 256, t);
            if (s + 2 < c1) load_half(p.w, rows, s + 2, t, half, w[half]);
        }
    }

    // sums of the two halves of the warps, then of the cluster's CTAs, in order
    const float gs = *p.scale;
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
                        // a row of x that is not finite gives NaN, whichever piece finds that
                        const float v = amax[col] < 0x7F800000u
                                            ? acc[ta][nt][i] * gs *
                                                  pow2_biased(x_exponent(amax[col]) - 14)
                                            : NAN;
                        part[col][r] = half ? v : part[col][r] + v;
                    }
        }
        __syncthreads();
    }
    if (pieces > 1) cluster_sync();
    // a thread keeps its row n: 128 / pieces rows, and every (kThreads / that)-th row of x
    const int share = kTileRows / pieces;
    const int r = rank * share + (threadIdx.x & (share - 1)), n = tile * kTileRows + r;
    const float bias = p.bias && n < p.w.N ? __bfloat162float(p.bias[n]) : 0.0f;
    for (int m = threadIdx.x / share; m < p.M; m += kThreads / share) {
        if (n >= p.w.N) break;
        float v;
        if (pieces == 1) {
            v = part[m][r];
        } else {
            const uint32_t at = smem_u32(&part[m][r]);
            float y[8];
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) {
                y[j] = 0.0f;
                if (j < pieces)
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(y[j])
                                 : "r"(mapa_shared(at, j)));
            }
            v = ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
        }
        p.out[static_cast<int64_t>(m) * p.w.N + n] = __float2bfloat16_rn(v + bias);
    }
    if (pieces > 1) cluster_sync();             // the others have read this CTA's sums before it ends
}

template <int NT, int PER>
int launch_direct(const DirectParams& p, int64_t ctas, int pieces, int dev, cudaStream_t stream)
{
    static std::atomic<bool> ready[kMaxDevices];
    if (!ready[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(nvfp4_gemv_direct_kernel<NT, PER>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kMaxStage) != cudaSuccess) {
            cudaGetLastError();
            return BSP_ERR_CUDA;
        }
        ready[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = pieces;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.M) * p.row_bytes + 128;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, nvfp4_gemv_direct_kernel<NT, PER>, p) != cudaSuccess) {
        cudaGetLastError();
        return BSP_ERR_CUDA;
    }
    return launch_status();
}

}  // namespace

// Pieces of K: as many as leave each half of the warps of a CTA a step and, of all tiles, keep to two
// CTAs an SM; or to three, which up to 8 rows of x leave registers for, where that makes it twice as
// many (10368 x 2560: 9.7 us and 10.7 for 4 and 8 rows, 11.7 and 13.9 with two; where two do, the third's
// registers cost 10 to 20 %).
//
// One launch does better than two where all CTAs run at once, or K is short, as long as a CTA's piece of
// x fits and is not long.  Measured, us, with one and with two launches:
//     4096 x 14336 (8 pieces of 7 steps):  8 rows 13.3, 21.9;   16 rows 17.9, 25.0
//     14336 x 4096 (2 pieces of 8 steps):  1 row 11.5, 13.9;    16 rows 19.0, 21.6
//     14336 x 8192 (2 pieces of 16 steps): 1 row 20.0, 20.2;    4 rows 21.9, 21.3
//     28672 x 8192 (1 piece of 32 steps):  4 rows 37.6, 33.6
//     128 x 65536 (8 pieces of 32 steps):  1 row 18.8, 14.2;    4 rows 22.5, 17.8
//     65536 x 1280 (1 piece, two waves):   1 row 15.3, 18.5;    16 rows 24.6, 27.2
//     131072 x 2048 (1 piece, four waves): 1 row 38.1, 38.5;    16 rows 60.9, 57.1
GemvSplit gemv_one_launch(int64_t M, int64_t N, int64_t K, int sms)
{
    const int64_t tiles = (N + kTileRows - 1) / kTileRows, steps = (K + kStepK - 1) / kStepK;
    const auto pieces = [&](int per) {
        int c = 1;
        while (c < kMaxPieces && 4 * c <= steps && 2 * c * tiles <= per * sms) c *= 2;
        return c;
    };
    GemvSplit s = {pieces(2), 2};
    if (M <= 8 && pieces(3) > s.pieces) s = {pieces(3), 3};
    const int64_t most = (steps + s.pieces - 1) / s.pieces;
    const int64_t room = s.per_sm == 2 ? kMaxStage : kMaxStage / 2;
    const int64_t ctas = tiles * s.pieces;
    if (M * most * kStepBytes + 128 > room || (ctas > s.per_sm * sms && steps > kFewSteps) ||
        most > kManySteps)
        s.pieces = 0;
    return s;
}

int gemv_direct(const GemvSplit& split, const __nv_bfloat16* x, const uint8_t* w_codes,
                const uint8_t* w_sf, const float* w_scale, const __nv_bfloat16* bias,
                __nv_bfloat16* out, int64_t M, int64_t N, int64_t K, int dev, cudaStream_t stream)
{
    const int64_t tiles = (N + kTileRows - 1) / kTileRows, steps = (K + kStepK - 1) / kStepK;
    const int c = split.pieces;
    DirectParams p = {};
    p.x = x;
    p.w.codes = w_codes;
    p.w.sf = w_sf;
    p.w.N = static_cast<int32_t>(N);
    p.w.K = static_cast<int32_t>(K);
    p.scale = w_scale;
    p.bias = bias;
    p.out = out;
    p.M = static_cast<int32_t>(M);
    p.steps = static_cast<int32_t>(steps);
    p.row_bytes = static_cast<int32_t>((steps + c - 1) / c) * kStepBytes;
    if (M <= 8)
        return split.per_sm == 3 ? launch_direct<1, 3>(p, tiles * c, c, dev, stream)
                                 : launch_direct<1, 2>(p, tiles * c, c, dev, stream);
    if (M <= 16) return launch_direct<2, 2>(p, tiles * c, c, dev, stream);
    if (M <= 24) return launch_direct<3, 2>(p, tiles * c, c, dev, stream);
    return launch_direct<4, 2>(p, tiles * c, c, dev, stream);
}

}  // namespace bsp
