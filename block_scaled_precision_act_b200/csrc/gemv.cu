// gemv.cu -- nvfp4_gemv: y[m][n] = bf16(g * sum_k x[m][k] w[n][k] + bias[n]) for a few rows of
// bf16 x, w = e2m1(code) * e4m3(scale) in the layout of nvfp4_gemm.  The weight-only form.
//
// What bounds it is reading the weight, 9/16 byte for each.  Decoded by the CUDA cores, a weight
// costs a conversion, a product with its scale and its share of the products with x: at 16 rows
// that took 2.7 times as long as the reading.  So no CUDA core touches the weight: it goes from
// global memory to shared memory and into tcgen05.mma kind::mxf4nvf4 as it is stored, as the M = 128
// operand, and x is made to fit the other operand instead, as a sum of seven E2M1 rows:
//     x[m][k] = rho_m * sum_i 2^(q_i) e2m1(c_i[m][k]),    q = 0, -2, -5, -8, -11, -14, -17,
// rho_m the smallest power of two with |x[m][.]| <= 6 rho_m.  A term takes the nearest code of what
// the terms before it left:
//     term 1: |r| <= 6 leaves at most 1 (codes are 2 apart above 4) = 4 * 2^-2;
//     term 2: |r| <= 4 units leaves at most half a unit (codes are at most 1 apart up to 4),
//             2^-3 = 4 * 2^-5, and so on: 2^-18 after term 7, while the row's largest is above 3.
// So x is held to 2^-19.5 of the largest of its row (bf16 has 2^-8 of the element).  The scale
// vector of that operand is 1 throughout (it is laid down in tensor memory once, where loading one for
// each stage cost the issuing thread 430 cycles of a budget of 790), and the epilogue adds the seven
// columns of a row with their powers of two, smallest first.
//
// Two kernels.  nvfp4_gemv_split_kernel writes the seven rows of each x row to the workspace, in the
// order in which shared memory will hold them.  nvfp4_gemv_kernel, one CTA per SM: the 256-element
// K stages of all 128-row tiles in a row are cut into equal runs, one for each CTA, so that every SM
// reads the same number of bytes whatever N and K are; a tile that is cut leaves fp32 parts, and the
// last CTA to finish one adds them in order.  Its producer fills the ring with weights before the
// split kernel has ended (that kernel begins only when everything before this call has).
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
constexpr int kTerms = 7;
constexpr int kTileRows = 128;
constexpr int kStageK = 256;
constexpr int kABytes = kTileRows * kStageK / 2;
constexpr int kSfBytes = 4 * 512;                // scales of 128 rows and one stage
constexpr int kMaxStages = 8;
constexpr int kMaxCtas = 160;
constexpr int kThreads = 224;                    // producer, MMA issuer, four epilogue warps, issuer
constexpr int kRingBytes = 224 * 1024;
constexpr uint32_t kTmemCols = 512;
constexpr int kAccCols = 448;                    // of the accumulators; then the scales
constexpr int kSfaCol = kAccCols, kSfbCol = kSfaCol + 32;
constexpr int kPoison = 0x7FFFFFFF;              // exponent of a row that is not finite

__host__ __device__ constexpr int term_exp(int i) { return i == 0 ? 0 : 1 - 3 * i; }

struct GemvArgs {
    const uint8_t* sfa;
    const float* w_scale;
    const __nv_bfloat16* bias;
    __nv_bfloat16* out;
    const uint8_t* xc;           // [stages of K][nb rows][128 bytes], swizzled
    const int32_t* rho;          // [M] exponent of a row's power of two, or kPoison
    float* parts;                // [2 * ctas][M][128]
    int32_t* done;               // [tiles][4] parts that have arrived, zeroed by the split kernel
    int32_t M, N, K;
    int32_t mp;                  // rows of x rounded up to 8
    int32_t nb;                  // 7 mp rounded up to 16: rows of the second operand
    int32_t num_kt;
    int32_t stages;              // of the ring
    int64_t total;               // K stages of all tiles
    uint64_t wait_ns;
    int* status;
};

__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr));
}

// 2^e as a float, e in [-126, 127]
__device__ __forceinline__ float exp2_int(int e)
{
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// ceil(log2(v / 6)) of a positive normal v
__device__ __forceinline__ int log2_over_6(float v)
{
    const uint32_t b = __float_as_uint(v);
    return static_cast<int>(b >> 23) - 127 - 2 + ((b & 0x7FFFFFu) > 0x400000u);
}

// Sixteen codes of r / 2^q (element 2j in the low nibble), and r minus what they stand for.
__device__ __forceinline__ uint2 take_term(float (&r)[16], int q)
{
    const float down = exp2_int(-q), up = exp2_int(q);
    uint2 w;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = r[8 * half + i] * down;
        const uint32_t c = cvt_e2m1x8(y);
        (half ? w.y : w.x) = c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h2;
            asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
                : "=r"(h2)
                : "r"(c >> (8 * i) & 0xFFu));
            const __half2 h = *reinterpret_cast<const __half2*>(&h2);
            r[8 * half + 2 * i] = fmaf(-up, __low2float(h), r[8 * half + 2 * i]);
            r[8 * half + 2 * i + 1] = fmaf(-up, __high2float(h), r[8 * half + 2 * i + 1]);
        }
    }
    return w;
}

// Largest |x| of sixteen bf16 as fp32 bits; an infinity or NaN is the largest of all.
__device__ __forceinline__ uint32_t max_bits(const uint4 (&v)[2])
{
    uint32_t m = 0;
    const uint32_t u[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, max(u[i] << 16 & 0x7FFFFFFFu, u[i] & 0x7FFF0000u));
    return m;
}

// One CTA per row of x; a thread takes 16-element blocks.  Also zeroes the counters of the tiles.
__global__ void __launch_bounds__(1024)
    nvfp4_gemv_split_kernel(const __nv_bfloat16* x, int K, int mp, int nb,
                            uint8_t* xc, int32_t* rho, int32_t* done, int counters)
{
    __shared__ uint32_t warp_max[32];
    griddep_wait();
    griddep_launch_dependents();
    const int m = blockIdx.x, blocks = K / 16;
    const uint4* row = reinterpret_cast<const uint4*>(x + static_cast<int64_t>(m) * K);
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < counters; i += gridDim.x * blockDim.x)
        done[i] = 0;
    uint4 v[2] = {};
    uint32_t top = 0;
    for (int b = threadIdx.x; b < blocks; b += blockDim.x) {
        v[0] = row[2 * b];
        v[1] = row[2 * b + 1];
        top = max(top, max_bits(v));
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = top;
    __syncthreads();
    top = threadIdx.x % 32 < blockDim.x / 32 ? warp_max[threadIdx.x & 31] : 0;
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    const bool finite = top < 0x7F800000u;
    const int e = finite ? max(log2_over_6(fmaxf(__uint_as_float(top), 0x1p-120f)), -120) : 0;
    if (threadIdx.x == 0) rho[m] = finite ? e : kPoison;
    const float n1 = exp2_int(-e / 2), n2 = exp2_int(-e - -e / 2);
    const bool held = blocks <= static_cast<int>(blockDim.x);      // v still has the block
    for (int b = threadIdx.x; b < blocks; b += blockDim.x) {
        if (!held) {
            v[0] = row[2 * b];
            v[1] = row[2 * b + 1];
        }
        const uint32_t u[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
        float r[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r[2 * i] = bf16lo_to_f32(u[i]) * n1 * n2;
            r[2 * i + 1] = bf16hi_to_f32(u[i]) * n1 * n2;
        }
#pragma unroll
        for (int i = 0; i < kTerms; ++i) {
            const int j = i * mp + m;
            const int64_t at = (static_cast<int64_t>(b >> 4) * nb + j) * 128;
            *reinterpret_cast<uint2*>(xc + at + (((b >> 1 & 7) ^ (j & 7)) << 4) + (b & 1) * 8) =
                take_term(r, term_exp(i));
        }
    }
}

// First K stage of CTA i's run, and the CTA whose run holds stage s.
__device__ __forceinline__ int64_t run_begin(int64_t total, int ctas, int i)
{
    return total * i / ctas;
}

__device__ __forceinline__ int run_owner(int64_t total, int ctas, int64_t s)
{
    return static_cast<int>(((s + 1) * ctas - 1) / total);
}

__global__ void __launch_bounds__(kThreads, 1)
    nvfp4_gemv_kernel(const __grid_constant__ CUtensorMap tm_w, const GemvArgs args)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2], ones_ready, fin[2];
    __shared__ float2 factor[kGemvMaxRows];                      // 2^e g of a row, in two parts
    __shared__ uint32_t tmem_holder;
    __shared__ int abort_word;
    __shared__ __align__(128) uint32_t ones[128];                // E4M3 1.0
    volatile int* abort_flag = &abort_word;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stages = args.stages, num_kt = args.num_kt, nb = args.nb;
    const int b_bytes = nb * 128, stage_bytes = kABytes + b_bytes + kSfBytes;
    const int ctas = gridDim.x;
    const int64_t s0 = run_begin(args.total, ctas, blockIdx.x);
    const int64_t s1 = run_begin(args.total, ctas, blockIdx.x + 1);
    const int mine = static_cast<int>(s1 - s0);
    // two issuers' accumulators, twice when they fit
    const int bufs = 4 * nb <= kAccCols ? 2 : 1, acc_cols = kAccCols / (2 * bufs);

    // a walk over the run's stages: K stage, tile, slot of the ring, and the slot's phase
    struct Walk {
        int tile, kt, slot;
        uint32_t phase;
    };
    const int kb_all = args.K / 64;
    const int tile0 = static_cast<int>(s0 / num_kt);
    const Walk begin = {tile0, static_cast<int>(s0 - static_cast<int64_t>(tile0) * num_kt),
                        0, 0};
    const auto next = [&](Walk& w) {
        if (++w.kt == num_kt) {
            w.kt = 0;
            ++w.tile;
        }
        if (++w.slot == stages) {
            w.slot = 0;
            w.phase ^= 1;
        }
    };
    const auto weight = [&](const Walk& w) {
        const int nkb = min(4, kb_all - 4 * w.kt);
        uint8_t* dst = ring + w.slot * stage_bytes;
        uint64_t* bar = full + w.slot;
        mbar_arrive_expect_tx(bar, kABytes + b_bytes + nkb * 512);
        tma_load_2d(dst, &tm_w, bar, w.kt * (kStageK / 2), w.tile * kTileRows);
        bulk_load(dst + kABytes + b_bytes,
                  args.sfa + (static_cast<int64_t>(w.tile) * kb_all + 4 * w.kt) * 512,
                  nkb * 512, bar);
    };
    const auto rows = [&](const Walk& w) {
        uint8_t* dst = ring + w.slot * stage_bytes;
        bulk_load(dst + kABytes, args.xc + static_cast<int64_t>(w.kt) * b_bytes, b_bytes,
                  full + w.slot);
    };
    const int early = min(mine, stages);
    if (warp == 0 && lane == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull + a, 2);
            mbar_init(tempty + a, 4);
        }
        mbar_init(&ones_ready, 1);
        mbar_init(fin, 1);
        mbar_init(fin + 1, 1);
        *abort_flag = 0;
        fence_mbar_init();
        // The first weights are on their way before the split kernel has ended, and before this CTA is
        // set up: nothing that this grid depends on writes them.
        Walk w = begin;
        for (int i = 0; i < early; ++i, next(w)) weight(w);
    }
    if (warp == 1) {
        tmem_alloc(&tmem_holder, kTmemCols);
        tmem_relinquish();
    }
    if (threadIdx.x < 128) ones[threadIdx.x] = 0x38383838u;
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();             // not before this CTA has its tensor memory
    const uint32_t tbase = tmem_holder;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            griddep_wait();                      // x is split
            Walk w = begin;
            for (int i = 0; i < early; ++i, next(w)) rows(w);
            int i = early;
            for (; i < mine; ++i, next(w)) {
                if (!mbar_wait(empty + w.slot, w.phase ^ 1u, abort_flag, args.wait_ns, args.status,
                               101))
                    break;
                weight(w);
                rows(w);
            }
            // the last loads must land before shared memory is freed
            for (int j = max(0, i - stages); j < i; ++j)
                drain_wait(full + j % stages, j / stages & 1, args.wait_ns, args.status);
        }
    } else if (warp == 1 || warp == 6) {
        // ------------------------------------------------------------ MMA issuers
        if (lane == 0) {
            const int own = warp == 6;               // stages i with i % 2 == own
            const uint32_t idesc = idesc_nvf4(kTileRows, nb);
            const uint32_t sfa = tbase + kSfaCol + 16 * own, sfb = tbase + kSfbCol;
            if (own == 0)
                for (int c = 0; c < 2; ++c)          // scales of up to 256 rows of the second operand
                    tmem_cp_32x128b_x4(sfb + 4 * c, sdesc_sf_block(smem_u32(ones)));
            if (own == 0) {
                tc_commit(&ones_ready);
            } else if (!mbar_wait(&ones_ready, 0, abort_flag, args.wait_ns, args.status, 105)) {
                *abort_flag = 1;
            }
            tc_fence_after();
            int seg = -1, kt = static_cast<int>(s0 % num_kt), s = 0;
            uint32_t phase = 0;
            bool fresh = true;                       // nothing of this segment is issued yet
            for (int i = 0; i < mine; ++i) {
                if (i == 0 || kt == 0) {
                    if (seg >= 0) tc_commit(tfull + seg % bufs);
                    ++seg;
                    fresh = true;
                    if (!mbar_wait(tempty + seg % bufs, (seg / bufs & 1) ^ 1u, abort_flag,
                                   args.wait_ns, args.status, 102)) {
                        seg = -1;
                        break;
                    }
                }
                if ((i & 1) == own) {
                    if (!mbar_wait(full + s, phase, abort_flag, args.wait_ns, args.status, 103)) {
                        seg = -1;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = smem_u32(ring + s * stage_bytes);
                    const uint64_t sf = sdesc_sf_block(a + kABytes + b_bytes);
                    const uint64_t ad = sdesc_kmajor_sw128(a);
                    const uint64_t bd = sdesc_kmajor_sw128(a + kABytes);
                    const uint32_t d = tbase + (2 * (seg % bufs) + own) * acc_cols;
                    const int nk = args.K / 64 - 4 * kt;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < nk) tmem_cp_32x128b_x4(sfa + 4 * k, sf + 32 * k);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < nk)
                            mma_nvf4(d, ad + 2 * k, bd + 2 * k, idesc, sfa + 4 * k, sfb,
                                     fresh && k == 0 ? 0u : 1u);
                    tc_commit(empty + s);
                    fresh = false;
                }
                if (++kt == num_kt) kt = 0;
                if (++s == stages) {
                    s = 0;
                    phase ^= 1;
                }
            }
            if (seg >= 0) tc_commit(tfull + seg % bufs);
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3, row = q * 32 + lane;
        griddep_wait();                          // the exponents and the counters are written
        const float g = *args.w_scale;
        if (lane < args.M) {                     // each warp writes them all: the same values
            const int e = __ldcg(args.rho + lane);
            factor[lane] = e == kPoison ? make_float2(NAN, NAN)
                                        : make_float2(exp2_int(e / 2) * g, exp2_int(e - e / 2));
        }
        __syncwarp();
        int seg = 0;
        for (int64_t at = s0; at < s1; ++seg) {
            const int tile = static_cast<int>(at / num_kt);
            const int64_t t0 = static_cast<int64_t>(tile) * num_kt, t1 = t0 + num_kt;
            const bool begins = at == t0, whole = begins && t1 <= s1;
            const int n = tile * kTileRows + row;
            const bool in = n < args.N;
            const float bias = in && args.bias ? __bfloat162float(args.bias[n]) : 0.0f;
            const int64_t end = min(t1, s1);
            const bool one = end - at == 1;      // then one of the issuers had nothing to do
            const int first_own = static_cast<int>(at - s0) & 1;
            const bool ok = mbar_wait(tfull + seg % bufs, seg / bufs & 1, abort_flag, args.wait_ns,
                                      args.status, 104);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc_fence_after();
            const uint32_t acc = tbase + (static_cast<uint32_t>(q * 32) << 16) +
                                 2 * (seg % bufs) * acc_cols;
            const auto finish = [&](int m, float v) {
                if (!in || m >= args.M) return;
                const float2 f = factor[m];
                args.out[static_cast<int64_t>(m) * args.N + n] =
                    __float2bfloat16_rn(v * f.x * f.y + bias);
            };
            float* part = args.parts +
                          static_cast<int64_t>(2 * blockIdx.x + begins) * args.M * kTileRows + row;
            for (int c = 0; c < args.mp; c += 8) {
                float v[8] = {};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (k == 1 && one) break;
                    const uint32_t from = acc + (first_own ^ k) * acc_cols + c;
                    uint32_t r[kTerms][8];
#pragma unroll
                    for (int i = 0; i < kTerms; ++i) tmem_ld_x8(from + i * args.mp, r[i]);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float y = 0.0f;          // the smallest terms first
#pragma unroll
                        for (int i = kTerms - 1; i >= 0; --i)
                            y = fmaf(__uint_as_float(r[i][j]), 1.0f / (1 << -term_exp(i)), y);
                        v[j] += y;
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (whole)
                        finish(c + j, v[j]);
                    else if (c + j < args.M)
                        part[(c + j) * kTileRows] = v[j];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty + seg % bufs);
            if (!whole) {
                // each of the four epilogue warps adds its own 32 rows when it is the last of the
                // CTAs' warps to bring them
                const int o0 = run_owner(args.total, ctas, t0), o1 = run_owner(args.total, ctas, t1 - 1);
                __threadfence();
                __syncwarp();
                int before = 0;
                if (lane == 0) before = atomicAdd(args.done + 4 * tile + q, 1);
                before = __shfl_sync(0xFFFFFFFFu, before, 0);
                if (before == o1 - o0) {
                    __threadfence();
                    const int64_t step = static_cast<int64_t>(2) * args.M * kTileRows;
                    const float* first = args.parts + o0 * step + step / 2 + row;
                    const float* rest = args.parts + o0 * step + row;
                    for (int m = 0; m < args.M; m += 8) {
                        float v[8];
                        const int rows = min(8, args.M - m);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            v[j] = j < rows ? __ldcg(first + (m + j) * kTileRows) : 0.0f;
                        for (int i0 = 1; i0 <= o1 - o0; i0 += 4) {
                            float y[4][8];       // four parts' loads in flight
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    y[i][j] = i0 + i <= o1 - o0 && j < rows
                                                  ? __ldcg(rest + (i0 + i) * step +
                                                           (m + j) * kTileRows)
                                                  : 0.0f;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int j = 0; j < 8; ++j) v[j] += y[i][j];
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j) finish(m + j, v[j]);
                    }
                }
            }
            at = end;
        }
    }

    // ---------------------------------------------------------------- teardown
    __syncwarp();
    if ((warp == 1 || warp == 6) && lane == 0) {
        tc_commit(fin + (warp == 6));
        drain_wait(fin + (warp == 6), 0, args.wait_ns, args.status);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tbase, kTmemCols);
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// Workspace: codes of the split x, parts, exponents, counters.
struct GemvLayout {
    int64_t parts, rho, done, bytes;
    int32_t mp, nb, num_kt, tiles;
};

GemvLayout gemv_layout(int64_t M, int64_t N, int64_t K)
{
    GemvLayout l;
    l.mp = static_cast<int32_t>((M + 7) / 8 * 8);
    l.nb = (kTerms * l.mp + 15) / 16 * 16;
    l.num_kt = static_cast<int32_t>((K + kStageK - 1) / kStageK);
    l.tiles = static_cast<int32_t>((N + kTileRows - 1) / kTileRows);
    l.parts = up256(static_cast<int64_t>(l.num_kt) * l.nb * 128);
    l.rho = l.parts + static_cast<int64_t>(2) * kMaxCtas * M * kTileRows * 4;
    l.done = up256(l.rho + M * 4);
    l.bytes = up256(l.done + static_cast<int64_t>(l.tiles) * 16);
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
    if (gemv_is_small(M, N, K, sms))
        return gemv_direct(static_cast<const __nv_bfloat16*>(x_bf16), w_codes, w_sf, w_scale,
                           static_cast<const __nv_bfloat16*>(bias_bf16),
                           static_cast<__nv_bfloat16*>(out_bf16), M, N, K, dev, sms,
                           reinterpret_cast<cudaStream_t>(stream));
    static std::atomic<bool> ready[kMaxDevices];
    constexpr int kSmem = kRingBytes + 1024;
    if (!ready[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(nvfp4_gemv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmem) != cudaSuccess) {
            cudaGetLastError();
            return BSP_ERR_CUDA;
        }
        ready[dev].store(true, std::memory_order_release);
    }
    CUtensorMap tm;
    st = make_code_map(&tm, w_codes, static_cast<uint64_t>(K) / 2, static_cast<uint64_t>(N),
                       kTileRows);
    if (st != BSP_OK) return st;
    auto* ws = static_cast<uint8_t*>(workspace);
    GemvArgs a = {};
    a.sfa = w_sf;
    a.w_scale = w_scale;
    a.bias = static_cast<const __nv_bfloat16*>(bias_bf16);
    a.out = static_cast<__nv_bfloat16*>(out_bf16);
    a.xc = ws;
    a.rho = reinterpret_cast<int32_t*>(ws + l.rho);
    a.parts = reinterpret_cast<float*>(ws + l.parts);
    a.done = reinterpret_cast<int32_t*>(ws + l.done);
    a.M = static_cast<int32_t>(M);
    a.N = static_cast<int32_t>(N);
    a.K = static_cast<int32_t>(K);
    a.mp = l.mp;
    a.nb = l.nb;
    a.num_kt = l.num_kt;
    const int stage_bytes = kABytes + l.nb * 128 + kSfBytes;
    a.stages = std::min(kMaxStages, kRingBytes / stage_bytes);
    a.total = static_cast<int64_t>(l.tiles) * l.num_kt;
    a.wait_ns = wait_limit_ns();
    a.status = device_status_ptr(dev);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const unsigned threads = static_cast<unsigned>(std::min<int64_t>(1024, (K / 16 + 31) / 32 * 32));
    // CTAs.  At least sqrt(num_kt M / 20) stages to each: fewer leave more parts of a tile to its
    // last CTA than they save in stages (about 0.4 us each, against 0.6 us for 32 rows of parts).
    // Where the tiles are fewer than that many CTAs, a multiple of the tiles gives every CTA one whole
    // tile or one even part of one; it is taken unless its runs are over 7 stages (3 us, what a
    // second part in a run costs) longer than equal runs over all SMs.
    int per = 1;
    while (per * per * 20 < l.num_kt * M) ++per;
    int64_t ctas = std::min<int64_t>(std::min(sms, kMaxCtas), (a.total + per - 1) / per);
    if (l.tiles <= ctas) {
        const int64_t even = ctas / l.tiles;
        if ((l.num_kt + even - 1) / even <= (a.total + ctas - 1) / ctas + 7) ctas = even * l.tiles;
    }
    if (launch_kernel(nvfp4_gemv_split_kernel, static_cast<unsigned>(M), threads, 0, s, true,
                      static_cast<const __nv_bfloat16*>(x_bf16), a.K, a.mp, a.nb, ws,
                      reinterpret_cast<int32_t*>(ws + l.rho),
                      reinterpret_cast<int32_t*>(ws + l.done), 4 * l.tiles) != cudaSuccess ||
        launch_kernel(nvfp4_gemv_kernel, static_cast<unsigned>(ctas), kThreads,
                      static_cast<size_t>(a.stages) * stage_bytes + 1024, s, true, tm,
                      a) != cudaSuccess) {
        cudaGetLastError();
        return BSP_ERR_CUDA;
    }
    return launch_status();
}

}  // extern "C"
