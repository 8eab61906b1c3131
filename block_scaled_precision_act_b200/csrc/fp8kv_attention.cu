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

#include <algorithm>
#include <atomic>

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
    float* parts;            // [2 * ctas][slot_rows][D + 2]: output, maximum, sum of a part
    int32_t slot_rows;
};

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr int kRows = 16;
constexpr int kTile = kAttnWarps * kKvBlock;     // tokens of one tile: a block for each warp
constexpr int kMaxCtas = 640;                    // 148 SMs x 4, rounded up
constexpr int kMinTiles = 2;                     // tiles a CTA takes at least
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

// log of the sum l of weights exp2(s - m)
__device__ __forceinline__ float lse_of(float m, float l)
{
    return m == -INFINITY && l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
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

// ---- how the work is split.  An item is one row tile of one key head of a sequence; sequence b
// has items(b) = row tiles * Hkv of tiles(b) token tiles each.  All tiles of all items in a row
// are cut into equal runs, one for each CTA, whatever the lengths are: a run may end one item,
// hold whole ones and begin another.  Only the first and the last item of a run can be cut, so a
// CTA leaves at most two parts; fp8kv_join_kernel adds the parts of a cut item in order.
struct SeqWork {
    int32_t first, n, len;       // rows, new tokens, length
    int32_t row_tiles, tile0, tiles;
};

__device__ __forceinline__ SeqWork seq_work(const AttnParams& p, int b)
{
    SeqWork s;
    const KvRows r = kv_rows(p.c, b);
    s.first = r.first;
    s.n = r.n;
    s.len = kv_length(p.c, b);
    s.row_tiles = (s.n * p.G + kRows - 1) / kRows;
    const int32_t lo = p.window ? max(0, s.len - s.n - p.window + 1) : 0;
    s.tile0 = lo / kTile;
    s.tiles = max(1, (s.len + kTile - 1) / kTile - s.tile0);
    return s;
}

__device__ __forceinline__ int64_t seq_tiles(const AttnParams& p, int b)
{
    const SeqWork s = seq_work(p, b);
    return static_cast<int64_t>(s.row_tiles) * p.c.Hkv * s.tiles;
}

// Where tile `at` of the whole row lies.  total is the row's length.
struct Place {
    int b;
    int64_t before;              // tiles of the sequences before b
};

struct SplitShared {
    int64_t warp_sum[kAttnWarps];
    int64_t before;
    int b;
};

__device__ __forceinline__ int64_t chunk_scan(int64_t w, SplitShared& sh, int64_t& chunk)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) sh.warp_sum[warp] = inc;
    __syncthreads();
    chunk = 0;
    int64_t pre = 0;
#pragma unroll
    for (int i = 0; i < kAttnWarps; ++i) {
        if (i < warp) pre += sh.warp_sum[i];
        chunk += sh.warp_sum[i];
    }
    return pre + inc - w;        // tiles before this thread's sequence, in this chunk
}

// Total number of tiles, and (through `pick`, which maps the total to a tile) the sequence that
// holds that tile.  Called by every thread; Place is valid where pick's tile is below the total.
template <typename Pick>
__device__ __forceinline__ int64_t find_tile(const AttnParams& p, SplitShared& sh, Pick pick,
                                             Place& place)
{
    int64_t total = 0, w = 0, excl = 0, chunk = 0;
    for (int base = 0; base < p.c.B; base += kAttnThreads) {
        const int i = base + threadIdx.x;
        w = i < p.c.B ? seq_tiles(p, i) : 0;
        excl = chunk_scan(w, sh, chunk);
        total += chunk;
    }
    const int64_t at = pick(total);
    if (threadIdx.x == 0) {
        sh.b = 0;
        sh.before = 0;
    }
    __syncthreads();
    if (p.c.B <= kAttnThreads) {                 // one chunk: it is still in registers
        if (at >= excl && at < excl + w) {
            sh.b = threadIdx.x;
            sh.before = excl;
        }
    } else {
        int64_t carry = 0;
        for (int base = 0; base < p.c.B; base += kAttnThreads) {
            const int i = base + threadIdx.x;
            w = i < p.c.B ? seq_tiles(p, i) : 0;
            excl = chunk_scan(w, sh, chunk) + carry;
            if (at >= excl && at < excl + w) {
                sh.b = i;
                sh.before = excl;
            }
            carry += chunk;
        }
    }
    __syncthreads();
    place.b = sh.b;
    place.before = sh.before;
    return total;
}

__device__ __forceinline__ int64_t run_length(int64_t total, int ctas)
{
    const int64_t per = (total + ctas - 1) / ctas;
    return per < kMinTiles ? kMinTiles : per;
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
__global__ void __launch_bounds__(kAttnThreads) fp8kv_attention_kernel(const AttnParams p)
{
    using S = Dims<DP>;
    extern __shared__ uint4 smem[];
    uint32_t* qs = reinterpret_cast<uint32_t*>(smem);           // [DP/16][32 lanes][4]
    float* os = reinterpret_cast<float*>(qs + S::kQWords);      // [warps][16][DP + 4]
    __shared__ float row_fac[kRows];
    __shared__ float stat_m[kAttnWarps][kRows], stat_l[kAttnWarps][kRows];
    __shared__ int stat_e[kAttnWarps];

    __shared__ SplitShared split;

    const KvCache& c = p.c;
    griddep_wait();
    griddep_launch_dependents();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    Place place;
    const int ctas = gridDim.x;
    const int64_t total = find_tile(
        p, split, [&](int64_t n) { return blockIdx.x * run_length(n, ctas); }, place);
    const int64_t per = run_length(total, ctas);
    int64_t at = blockIdx.x * per;
    const int64_t end = min(at + per, total);
    int b = place.b;
    int64_t before = place.before;

  while (at < end) {
    SeqWork sw = seq_work(p, b);
    int64_t mine = static_cast<int64_t>(sw.row_tiles) * c.Hkv * sw.tiles;
    while (at >= before + mine && b + 1 < c.B) {
        before += mine;
        sw = seq_work(p, ++b);
        mine = static_cast<int64_t>(sw.row_tiles) * c.Hkv * sw.tiles;
    }
    const int64_t item = (at - before) / sw.tiles;
    const int seg0 = static_cast<int>((at - before) - item * sw.tiles);
    const int seg1 = static_cast<int>(min(static_cast<int64_t>(sw.tiles), seg0 + (end - at)));
    at += seg1 - seg0;
    const bool whole = seg0 == 0 && seg1 == sw.tiles;
    const int h = static_cast<int>(item / sw.row_tiles);
    const int row_base = static_cast<int>(item - static_cast<int64_t>(h) * sw.row_tiles) * kRows;
    const int nrows = min(kRows, sw.n * p.G - row_base);
    const int32_t len = sw.len;
    const int32_t start = len - sw.n;                            // position of the first new token
    __syncthreads();                                             // the shared buffers are free

    // ---- q: f16 fragments in shared memory
    for (int i = 0; i < kRows / kAttnWarps; ++i) {
        const int r = warp * (kRows / kAttnWarps) + i;
        const int rr = row_base + r, tok = rr / p.G, head = rr - tok * p.G;
        const bool ok = r < nrows;
        const __nv_bfloat16* src = p.q + (sw.first + tok) * p.q_stride +
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
    const int blk_begin = max(first_tok / kKvBlock, (sw.tile0 + seg0) * kAttnWarps);
    const int blk_end = min((pos_hi + kKvBlock) / kKvBlock, (sw.tile0 + seg1) * kAttnWarps);

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
        const int64_t row = static_cast<int64_t>(sw.first + tok) * c.Hq + head;
        float* part = p.parts + (static_cast<int64_t>(2 * blockIdx.x + (seg0 == 0)) * p.slot_rows +
                                 r) * (c.D + 2);
        for (int d = 2 * lane; d < c.D; d += 64) {
            float x = 0.0f, y = 0.0f;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float* ow = os + (w * kRows + r) * (DP + 4) + d;
                const float f1 = f[w] * inv * (1.0f / (1 << kPShift)), f2 = kv_pow2(stat_e[w]);
                x += ow[0] * f1 * f2;
                y += ow[1] * f1 * f2;
            }
            if (whole)
                *reinterpret_cast<__nv_bfloat162*>(p.out + row * c.D + d) =
                    __floats2bfloat162_rn(x, y);
            else
                *reinterpret_cast<float2*>(part + d) = make_float2(x, y);
        }
        if (lane == 0) {
            if (!whole) {
                part[c.D] = m;
                part[c.D + 1] = l;
            } else if (p.lse) {
                p.lse[row] = lse_of(m, l);
            }
        }
    }
  }
}

// Adds the parts of the item that CTA blockIdx.x of the attention kernel began and did not end
// (if it did): part i weighs l_i 2^(m_i - m), in the order of the tokens.  One warp takes one row.
__global__ void __launch_bounds__(kAttnThreads)
    fp8kv_join_kernel(const AttnParams p)
{
    __shared__ SplitShared split;
    const KvCache& c = p.c;
    const int ctas = gridDim.x;
    Place place;
    int64_t last = 0;
    const int64_t total = find_tile(
        p, split,
        [&](int64_t n) {
            last = min((blockIdx.x + int64_t{1}) * run_length(n, ctas), n) - 1;
            return last;
        },
        place);
    const int64_t per = run_length(total, ctas);
    const int64_t begin = blockIdx.x * per;
    griddep_wait();
    if (begin >= total) return;
    const SeqWork sw = seq_work(p, place.b);
    const int64_t item = (last - place.before) / sw.tiles;
    const int64_t s0 = place.before + item * sw.tiles, s1 = s0 + sw.tiles;   // the item's tiles
    if (s0 < begin || s1 <= last + 1) return;
    const int parts = static_cast<int>((s1 - 1) / per - blockIdx.x) + 1;
    const int h = static_cast<int>(item / sw.row_tiles);
    const int row_base = static_cast<int>(item - static_cast<int64_t>(h) * sw.row_tiles) * kRows;
    const int r = blockIdx.y * kAttnWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (r >= min(kRows, sw.n * p.G - row_base)) return;
    const int64_t step = static_cast<int64_t>(2) * p.slot_rows * (c.D + 2);
    // part 0 is the second slot of this CTA, part i > 0 the first slot of CTA blockIdx.x + i
    const float* first = p.parts + (static_cast<int64_t>(2 * blockIdx.x + 1) * p.slot_rows + r) *
                                       (c.D + 2);
    const float* rest = p.parts + (static_cast<int64_t>(2 * blockIdx.x) * p.slot_rows + r) *
                                      (c.D + 2);
    float m = -INFINITY;
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, (i ? rest + i * step : first)[c.D]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float z = m == -INFINITY ? 0.0f : m;
    float l = 0.0f, x[8] = {};
    for (int i = 0; i < parts; ++i) {
        const float* part = i ? rest + i * step : first;
        const float w = part[c.D + 1] * ex2(part[c.D] - z);
        l += w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d = 2 * lane + 64 * j;
            if (d >= c.D) break;
            const float2 v = *reinterpret_cast<const float2*>(part + d);
            x[2 * j] = fmaf(w, v.x, x[2 * j]);
            x[2 * j + 1] = fmaf(w, v.y, x[2 * j + 1]);
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int rr = row_base + r, tok = rr / p.G, head = h * p.G + rr - tok * p.G;
    const int64_t row = static_cast<int64_t>(sw.first + tok) * c.Hq + head;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int d = 2 * lane + 64 * j;
        if (d >= c.D) break;
        *reinterpret_cast<__nv_bfloat162*>(p.out + row * c.D + d) =
            __floats2bfloat162_rn(x[2 * j] * inv, x[2 * j + 1] * inv);
    }
    if (p.lse && lane == 0) p.lse[row] = lse_of(m, l);
}

template <int DP>
int launch_attention(const AttnParams& p, int sms, cudaStream_t s)
{
    // kernel attribute and CTAs per SM, once per device; 0 = not asked yet
    static std::atomic<int> occupancy[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return BSP_ERR_CUDA;
    }
    int occ = occupancy[dev].load(std::memory_order_acquire);
    if (occ == 0) {
        if (cudaFuncSetAttribute(fp8kv_attention_kernel<DP>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(Dims<DP>::kSmem)) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, fp8kv_attention_kernel<DP>,
                                                          kAttnThreads,
                                                          Dims<DP>::kSmem) != cudaSuccess ||
            occ < 1) {
            cudaGetLastError();
            return BSP_ERR_CUDA;
        }
        occupancy[dev].store(occ, std::memory_order_release);
    }
    const unsigned ctas = static_cast<unsigned>(std::min(sms * occ, kMaxCtas));
    if (launch_kernel(fp8kv_attention_kernel<DP>, ctas, kAttnThreads, Dims<DP>::kSmem, s, true,
                      p) != cudaSuccess) {
        cudaGetLastError();
        return BSP_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(ctas, kRows / kAttnWarps, 1);
    cfg.blockDim = dim3(kAttnThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fp8kv_join_kernel, p) != cudaSuccess) {
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
    const int64_t rows = std::min<int64_t>(bsp::kRows, T * (Hq / Hkv));
    return 2 * bsp::kMaxCtas * rows * (D + 2) * static_cast<int64_t>(sizeof(float));
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
    p.parts = static_cast<float*>(workspace);
    p.slot_rows = static_cast<int32_t>(std::min<int64_t>(kRows, T * p.G));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (D <= 64) return launch_attention<64>(p, sms, s);
    if (D <= 128) return launch_attention<128>(p, sms, s);
    return launch_attention<256>(p, sms, s);
}

}  // extern "C"
