// fp8kv_attention.cu -- attention of the new tokens over the paged block-scaled E4M3 cache.
//
//   out[r] = sum_t p_rt v_t / sum_t p_rt,  p_rt = exp(sm_scale q_r . k_t), over the tokens t that
//   row r sees: t <= pos(r), and t > pos(r) - window when a window is given.
//
// Rows: the query heads that share a key head and the new tokens of a sequence, 16 to a tile
// (row = token * G + head in group).  A step is one 16-token block of the cache, taken by one
// warp with m16n8k16 f16 products accumulated in fp32; the block's two scales are one number
// each, so they never touch the elements:
//   * E4M3 -> f16 is exact.  K goes from global memory into the B fragments without shared
//     memory: the products may run over d in any order, so a lane takes the 16-byte chunks of its
//     token row that it loads as the k slots that it owns.  q is scaled by a power of two per row
//     so that its largest element is in [2^14, 2^15): f16 then holds every bf16 element of the
//     row down to 2^-28 of the largest exactly, and rounds smaller ones by at most 2^-39 of it.
//   * V: a lane loads a chunk of each of the four tokens whose k slots it owns; a byte permute
//     pairs tokens.  The softmax weights (in [0, 1], fp32) are rounded once, to f16 with 11 bits,
//     after a factor 2^(13 + e_V - e_ref), which keeps them normal down to 2^-27 of the largest;
//     e_ref follows the V scales when they leave [e_ref - 10, e_ref + 2].
//   * running maximum and sum in fp32; the output is rescaled only when a maximum moves.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <mutex>

#include "fp8kv_common.cuh"

namespace bsp {

int kv_check_cache(KvCache& c, const void* k_cache, const void* v_cache, const void* k_scale,
                   const void* v_scale, int64_t pages, int64_t page_size, const int32_t* table,
                   int64_t max_pages, const int32_t* cu_new, const int32_t* kv_len, int64_t B,
                   int64_t T, int64_t Hq, int64_t Hkv, int64_t D);
int kv_check_pointers(const KvCache& c);

namespace {

struct AttnParams {
    KvCache c;
    const __nv_bfloat16* q;
    int64_t q_stride;
    __nv_bfloat16* out;
    float* lse;
    float scale_log2;        // sm_scale * log2(e)
    int32_t window;          // 0: none
    int32_t G;
    int* status;
};

constexpr int kAttnWarps = 4;
constexpr int kRows = 16;
constexpr int kPShift = 13;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 0x80 in each byte of w that is an E4M3 NaN
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w)
{
    return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// One pass over 16 tokens of V: o += w * v.  vr[i] are the bytes of this lane's token i (k slots
// 2t, 2t + 1, 2t + 8, 2t + 9), NT n-tiles in all.
template <int NT, int VW>
__device__ __forceinline__ void mma_v(float (&o)[NT][4], const uint32_t (&vr)[4][VW], uint32_t a0,
                                      uint32_t a1, uint32_t a2, uint32_t a3)
{
#pragma unroll
    for (int w = 0; w < VW; ++w) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint32_t sel = half ? 0x7362u : 0x5140u;
            uint32_t b0[2], b1[2];
            e4m3x4_to_f16(__byte_perm(vr[0][w], vr[1][w], sel), b0[0], b0[1]);
            e4m3x4_to_f16(__byte_perm(vr[2][w], vr[3][w], sel), b1[0], b1[1]);
            mma_f16(o[4 * w + 2 * half], a0, a1, a2, a3, b0[0], b1[0]);
            mma_f16(o[4 * w + 2 * half + 1], a0, a1, a2, a3, b0[1], b1[1]);
        }
    }
}

// DP: head dimension rounded up to 64, 128 or 256.
template <int DP>
struct Dims {
    static constexpr int kQWords = DP / 16 * 32 * 4;           // q fragments, 32-bit words
    static constexpr int kNT = DP / 8;                          // 8-column tiles of the output
    static constexpr int kVW = DP / 32;                         // words of one token's V chunk(s)
    static constexpr size_t kSmem = kQWords * 4 + kAttnWarps * kRows * (DP + 4) * 4;
};

template <int DP>
__global__ void __launch_bounds__(kAttnWarps * 32) fp8kv_attention_kernel(const AttnParams p)
{
    using S = Dims<DP>;
    extern __shared__ uint4 smem[];
    uint32_t* qs = reinterpret_cast<uint32_t*>(smem);           // [DP/16][32 lanes][4]
    float* os = reinterpret_cast<float*>(qs + S::kQWords);      // [warps][16][DP + 4]
    __shared__ float row_fac[kRows];
    __shared__ float stat_m[kAttnWarps][kRows], stat_l[kAttnWarps][kRows];
    __shared__ int stat_e[kAttnWarps];

    const KvCache& c = p.c;
    griddep_wait();
    griddep_launch_dependents();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    int64_t begin;
    const int b = kv_find_sequence(c, blockIdx.x, p.G, 1, begin);
    const KvRows rows = kv_rows(c, b);
    const int row_base = static_cast<int>(blockIdx.x - begin) * kRows;
    const int nrows = min(kRows, rows.n * p.G - row_base);
    if (nrows <= 0 || blockIdx.x < begin) return;            // the latter: cu_new descends
    const int h = blockIdx.y;
    const int32_t len = kv_length(c, b);
    const int32_t start = len - rows.n;                          // position of the first new token

    // ---- q: f16 fragments in shared memory
    for (int i = 0; i < kRows / kAttnWarps; ++i) {
        const int r = warp * (kRows / kAttnWarps) + i;
        const int rr = row_base + r, tok = rr / p.G, head = rr - tok * p.G;
        const bool ok = r < nrows;
        const __nv_bfloat16* src = p.q + (rows.first + tok) * p.q_stride +
                                   static_cast<int64_t>(h * p.G + head) * c.D;
        uint32_t w[DP / 64];
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < DP / 64; ++j) {
            const int d = 2 * (lane + 32 * j);
            w[j] = ok && d < c.D ? *reinterpret_cast<const uint32_t*>(src + d) : 0u;
            amax = max(amax, max(w[j] << 16 & 0x7FFFFFFFu, w[j] & 0x7FFF0000u));
        }
        amax = __reduce_max_sync(0xFFFFFFFFu, amax);
        int e = static_cast<int>(amax >> 23);                    // biased exponent of the largest
        e = e < 15 ? 15 : e;
        const float up = kv_pow2(254 - e + 14 > 254 ? 254 : 254 - e + 14);   // 2^(14 - (e - 127))
        if (lane == 0) row_fac[r] = p.scale_log2 * kv_pow2(e - 14);
#pragma unroll
        for (int j = 0; j < DP / 64; ++j) {
            const int d = 2 * (lane + 32 * j);
            const int chunk = d >> 4, cg = chunk >> 2, ct = chunk & 3;
            const int jj = (d & 15) >> 2, hi = (d >> 1) & 1;
            qs[((cg * 4 + jj) * 32 + (r & 7) * 4 + ct) * 4 + (r >> 3) + 2 * hi] =
                pack_f16(bf16lo_to_f32(w[j]) * up, bf16hi_to_f32(w[j]) * up);
        }
    }
    __syncthreads();

    const float fac0 = row_fac[g], fac1 = row_fac[g + 8];
    const int pos0 = start + (row_base + min(g, nrows - 1)) / p.G;
    const int pos1 = start + (row_base + min(g + 8, nrows - 1)) / p.G;
    const int pos_lo = start + row_base / p.G, pos_hi = start + (row_base + nrows - 1) / p.G;
    const int first_tok = p.window ? max(0, pos_lo - p.window + 1) : 0;
    const int blk_begin = first_tok / kKvBlock, blk_end = (pos_hi + kKvBlock) / kKvBlock;

    float o[S::kNT][4];
#pragma unroll
    for (int i = 0; i < S::kNT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    int e_ref = -1, e_top = 0;

    for (int blk = blk_begin + warp; blk < blk_end; blk += kAttnWarps) {
        const int pi = blk / c.page_blocks, in_page = blk - pi * c.page_blocks;
        const int32_t page = __ldg(c.table + static_cast<int64_t>(b) * c.max_pages + pi);
        const bool page_ok = page >= 0 && page < c.pages;
        if (!page_ok) {
            if (lane == 0) kv_report_bad_batch(p.status);
            continue;
        }
        const int64_t group = (static_cast<int64_t>(page) * c.Hkv + h) * c.page_blocks + in_page;
        const uint8_t* kp = c.k + group * kKvBlock * c.D;
        const uint8_t* vp = c.v + group * kKvBlock * c.D;
        uint4 kr[2][DP / 64];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int cg = 0; cg < DP / 64; ++cg) {
                const int d = (cg * 4 + t) * 16;
                kr[nt][cg] = d < c.D ? __ldg(reinterpret_cast<const uint4*>(
                                           kp + (nt * 8 + g) * c.D + d))
                                     : make_uint4(0, 0, 0, 0);
            }
        uint32_t vr[4][S::kVW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t* row = vp + (2 * t + (i & 1) + (i >> 1) * 8) * c.D;
            if constexpr (DP == 64) {
                const uint2 x = 8 * g < c.D ? __ldg(reinterpret_cast<const uint2*>(row + 8 * g))
                                            : make_uint2(0, 0);
                vr[i][0] = x.x;
                vr[i][1] = x.y;
            } else {
#pragma unroll
                for (int hh = 0; hh < DP / 128; ++hh) {
                    const int d = 128 * hh + 16 * g;
                    const uint4 x = d < c.D ? __ldg(reinterpret_cast<const uint4*>(row + d))
                                            : make_uint4(0, 0, 0, 0);
                    vr[i][4 * hh] = x.x;
                    vr[i][4 * hh + 1] = x.y;
                    vr[i][4 * hh + 2] = x.z;
                    vr[i][4 * hh + 3] = x.w;
                }
            }
        }
        const int ek = min(static_cast<int>(__ldg(c.k_scale + group)), kKvMaxExp);
        const int ev = min(static_cast<int>(__ldg(c.v_scale + group)), kKvMaxExp);

        // ---- scores
        float s[2][4] = {};
#pragma unroll
        for (int cg = 0; cg < DP / 64; ++cg) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 a = reinterpret_cast<const uint4*>(qs)[(cg * 4 + j) * 32 + lane];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const uint32_t w = j == 0   ? kr[nt][cg].x
                                       : j == 1 ? kr[nt][cg].y
                                       : j == 2 ? kr[nt][cg].z
                                                : kr[nt][cg].w;
                    uint32_t b0, b1;
                    e4m3x4_to_f16(w, b0, b1);
                    mma_f16(s[nt], a.x, a.y, a.z, a.w, b0, b1);
                }
            }
        }
        const float kf = kv_pow2(ek);
        const float f0 = fac0 * kf, f1 = fac1 * kf;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            s[nt][0] *= f0;
            s[nt][1] *= f0;
            s[nt][2] *= f1;
            s[nt][3] *= f1;
        }
        const int tok0 = blk * kKvBlock;
        const bool edge = tok0 + kKvBlock - 1 > pos_lo || (p.window && tok0 <= pos_hi - p.window);
        uint32_t seen = 0xFFu;                    // bit 4 * nt + i: s[nt][i] is in the mask
        if (edge) {
            seen = 0;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = tok0 + nt * 8 + 2 * t + (i & 1);
                    const int pos = i < 2 ? pos0 : pos1;
                    const bool in = tok <= pos && (p.window == 0 || tok > pos - p.window);
                    if (in) seen |= 1u << (4 * nt + i);
                    if (!in) s[nt][i] = -INFINITY;
                }
        }

        // ---- running maximum and sum
        float n0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
        float n1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
            n0 = fmaxf(n0, __shfl_xor_sync(0xFFFFFFFFu, n0, x));
            n1 = fmaxf(n1, __shfl_xor_sync(0xFFFFFFFFu, n1, x));
        }
        n0 = fmaxf(n0, m0);
        n1 = fmaxf(n1, m1);
        int e_new = e_ref;
        e_top = max(e_top, ev);
        if (e_ref < 0 || ev > e_ref + 2 || ev < e_ref - 10) e_new = max(ev, e_top - 40);
        if (__any_sync(0xFFFFFFFFu, n0 != m0 || n1 != m1) || e_new != e_ref) {
            const float de = e_ref < 0 ? 0.0f : static_cast<float>(e_ref - e_new);
            const float c0 = m0 == -INFINITY ? 0.0f : ex2(m0 - n0);
            const float c1 = m1 == -INFINITY ? 0.0f : ex2(m1 - n1);
            l0 *= c0;
            l1 *= c1;
            const float x0 = c0 * ex2(de), x1 = c1 * ex2(de);
#pragma unroll
            for (int i = 0; i < S::kNT; ++i) {
                o[i][0] *= x0;
                o[i][1] *= x0;
                o[i][2] *= x1;
                o[i][3] *= x1;
            }
            m0 = n0;
            m1 = n1;
            e_ref = e_new;
        }
        const float z0 = m0 == -INFINITY ? 0.0f : m0, z1 = m1 == -INFINITY ? 0.0f : m1;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            s[nt][0] = ex2(s[nt][0] - z0);
            s[nt][1] = ex2(s[nt][1] - z0);
            s[nt][2] = ex2(s[nt][2] - z1);
            s[nt][3] = ex2(s[nt][3] - z1);
            l0 += s[nt][0] + s[nt][1];
            l1 += s[nt][2] + s[nt][3];
        }
        const int we = 127 + kPShift + ev - e_ref;
        const float wf = we > 0 ? kv_pow2(we) : 0.0f;
        const uint32_t a0 = pack_f16(s[0][0] * wf, s[0][1] * wf);
        const uint32_t a1 = pack_f16(s[0][2] * wf, s[0][3] * wf);
        const uint32_t a2 = pack_f16(s[1][0] * wf, s[1][1] * wf);
        const uint32_t a3 = pack_f16(s[1][2] * wf, s[1][3] * wf);

        // ---- values.  A masked token's weight is 0, but 0 * NaN is not: where the mask cuts the
        // block, bytes of tokens that no row sees are cleared, and NaNs of tokens that only some
        // rows see are counted with 0 / 1 weights and put into just those rows.
        if (edge) {
            uint32_t nan = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = tok0 + 2 * t + (i & 1) + (i >> 1) * 8;
                const bool any = tok <= pos_hi && (p.window == 0 || tok > pos_lo - p.window);
#pragma unroll
                for (int w = 0; w < S::kVW; ++w) {
                    vr[i][w] = any ? vr[i][w] : 0u;
                    nan |= nan_bytes(vr[i][w]);
                }
            }
            if (__any_sync(0xFFFFFFFFu, nan != 0)) {
                const uint32_t one = 0x3C00u;                    // 1.0 in f16
                const auto bits = [&](int i) {
                    return ((seen >> i) & 1u) * one | ((seen >> (i + 1)) & 1u) * (one << 16);
                };
                const uint32_t i0 = bits(0), i1 = bits(2), i2 = bits(4), i3 = bits(6);
                uint32_t mark[4][S::kVW];                        // 2.0 in E4M3 where V is NaN
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int w = 0; w < S::kVW; ++w) {
                        const uint32_t n = nan_bytes(vr[i][w]);
                        mark[i][w] = n >> 1;
                        vr[i][w] &= ~((n >> 7) * 0xFFu);
                    }
                float count[S::kNT][4] = {};
                mma_v<S::kNT, S::kVW>(count, mark, i0, i1, i2, i3);
#pragma unroll
                for (int i = 0; i < S::kNT; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (count[i][k] > 0.0f) o[i][k] = NAN;
            }
        }
        mma_v<S::kNT, S::kVW>(o, vr, a0, a1, a2, a3);
    }

    // ---- join the warps: common maximum, then the weighted sum of their outputs
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
        l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, x);
        l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, x);
    }
    if (t == 0) {
        stat_m[warp][g] = m0;
        stat_m[warp][g + 8] = m1;
        stat_l[warp][g] = l0;
        stat_l[warp][g + 8] = l1;
    }
    if (lane == 0) stat_e[warp] = e_ref < 0 ? 0 : e_ref;
    {
        float* ow = os + warp * kRows * (DP + 4);
#pragma unroll
        for (int i = 0; i < S::kNT; ++i) {
            // column of B fragment n: DP 64: 8 n + i ; else 128 (i / 16) + 16 n + i % 16
            const int d0 = DP == 64 ? 16 * t + i : (i >> 4) * 128 + 32 * t + (i & 15);
            const int d1 = d0 + (DP == 64 ? 8 : 16);
            ow[g * (DP + 4) + d0] = o[i][0];
            ow[g * (DP + 4) + d1] = o[i][1];
            ow[(g + 8) * (DP + 4) + d0] = o[i][2];
            ow[(g + 8) * (DP + 4) + d1] = o[i][3];
        }
    }
    __syncthreads();
    for (int r = warp; r < nrows; r += kAttnWarps) {
        float m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) m = fmaxf(m, stat_m[w][r]);
        const float z = m == -INFINITY ? 0.0f : m;
        float f[kAttnWarps];
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
            f[w] = ex2(stat_m[w][r] - z);
            l += stat_l[w][r] * f[w];
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int rr = row_base + r, tok = rr / p.G, head = h * p.G + rr - tok * p.G;
        const int64_t at = static_cast<int64_t>(rows.first + tok) * c.Hq + head;
        for (int d = 2 * lane; d < c.D; d += 64) {
            float x = 0.0f, y = 0.0f;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float* ow = os + (w * kRows + r) * (DP + 4) + d;
                const float f1 = f[w] * inv * (1.0f / (1 << kPShift)), f2 = kv_pow2(stat_e[w]);
                x += ow[0] * f1 * f2;
                y += ow[1] * f1 * f2;
            }
            *reinterpret_cast<__nv_bfloat162*>(p.out + at * c.D + d) = __floats2bfloat162_rn(x, y);
        }
        if (p.lse && lane == 0)
            p.lse[at] = m == -INFINITY && l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
}

template <int DP>
int launch_attention(const AttnParams& p, unsigned units, cudaStream_t s)
{
    static std::once_flag once[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return BSP_ERR_CUDA;
    }
    cudaError_t e = cudaSuccess;
    std::call_once(once[dev], [&] {
        e = cudaFuncSetAttribute(fp8kv_attention_kernel<DP>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(Dims<DP>::kSmem));
    });
    if (e != cudaSuccess) {
        cudaGetLastError();
        return BSP_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(units, static_cast<unsigned>(p.c.Hkv), 1);
    cfg.blockDim = dim3(kAttnWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = Dims<DP>::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, fp8kv_attention_kernel<DP>, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return BSP_ERR_CUDA;
    }
    return launch_status();
}

}  // namespace
}  // namespace bsp

extern "C" {

int64_t fp8kv_attention_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D)
{
    if (T < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || Hq % Hkv != 0) return BSP_ERR_INVALID_ARG;
    if (D % 16 != 0 || D > 256) return BSP_ERR_UNSUPPORTED_SHAPE;
    return 16;
}

int fp8kv_attention(const void* q_bf16, int64_t q_stride, const uint8_t* k_cache,
                    const uint8_t* v_cache, const uint8_t* k_scale, const uint8_t* v_scale,
                    int64_t pages, int64_t page_size, const int32_t* block_table,
                    int64_t max_pages, const int32_t* cu_new, const int32_t* kv_len, int64_t B,
                    int64_t T, int64_t Hq, int64_t Hkv, int64_t D, float sm_scale, int64_t window,
                    void* out_bf16, float* lse, void* workspace, int64_t workspace_bytes,
                    bsp_stream_t stream)
{
    using namespace bsp;
    AttnParams p = {};
    int st = kv_check_cache(p.c, k_cache, v_cache, k_scale, v_scale, pages, page_size, block_table,
                            max_pages, cu_new, kv_len, B, T, Hq, Hkv, D);
    if (st != BSP_OK) return st;
    if (Hq == 0 || window < 0) return BSP_ERR_INVALID_ARG;
    if (T == 0 || B == 0) return BSP_OK;
    if (!q_bf16 || !out_bf16 || q_stride < Hq * D || pages == 0 || max_pages == 0)
        return BSP_ERR_INVALID_ARG;
    if (q_stride % 8 != 0) return BSP_ERR_UNSUPPORTED_SHAPE;
    const int64_t need = fp8kv_attention_workspace_bytes(T, Hq, Hkv, D);
    if (!workspace || workspace_bytes < need) return BSP_ERR_INVALID_ARG;
    st = kv_check_pointers(p.c);
    if (st != BSP_OK) return st;
    if (!aligned16(q_bf16) || !aligned16(out_bf16) || !aligned16(workspace) ||
        (reinterpret_cast<uintptr_t>(lse) & 3u))
        return BSP_ERR_MISALIGNED;
    int dev = 0, sms = 0;
    st = check_device(&dev, &sms);
    if (st != BSP_OK) return st;
    p.q = static_cast<const __nv_bfloat16*>(q_bf16);
    p.q_stride = q_stride;
    p.out = static_cast<__nv_bfloat16*>(out_bf16);
    p.lse = lse;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    p.window = window > (int64_t{1} << 30) ? 0 : static_cast<int32_t>(window);
    p.G = static_cast<int32_t>(Hq / Hkv);
    p.status = device_status_ptr(dev);
    const unsigned units = static_cast<unsigned>(T * p.G / kRows + B);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (D <= 64) return launch_attention<64>(p, units, s);
    if (D <= 128) return launch_attention<128>(p, units, s);
    return launch_attention<256>(p, units, s);
}

}  // extern "C"
