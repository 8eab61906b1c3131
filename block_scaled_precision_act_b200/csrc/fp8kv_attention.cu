// fp8kv_attention.cu -- attention of the new tokens over the paged block-scaled E4M3 cache.
//
//   out[r] = sum_t p_rt v_t / sum_t p_rt,  p_rt = exp(sm_scale q_r . k_t), over the tokens t that
//   row r sees: t <= pos(r), and t > pos(r) - window when a window is given.
//
// What bounds it is reading the cache, 2 D bytes for each token and key head.  Converting the codes
// for f16 products on the CUDA cores took 500 instructions per 16 tokens and warp, 1.8 times the
// reading; so the codes go from global memory by TMA to shared memory and into tcgen05.mma
// kind::f8f6f4 as they are, as the M = 128 operand of both products, and the small operands are
// made to fit.  A tile is 128 tokens; a block's two scales are one number each and never touch the
// elements (the key scale multiplies the scores, the value scale the weights).
//   S[128 tokens][3 R] = K Q^T.  A row of q, scaled by a power of two so that its largest element is in
//   [128, 256), is the sum of three E4M3 rows of q, 16 q and 256 q's rounding rests: each holds four bits,
//   so a bf16 element (eight bits) is exact down to 2^-17 of the row's largest, and off by 2^-25 of that (2^-18,
//   half of E4M3's smallest step over 256) at most.
//   O[128 d][4 R] = V^T P^T.  The operand is p 2^e_V 2^(8 - ref), at most 2^15, rounded once, to f16 (11
//   bits down to 2^-21 of the row's largest p 2^e_V, an absolute 2^-32 of that below), which is exactly
//   the sum of an E5M2, 1/8, 1/64 and 1/512 of others: an f16 cut to its upper byte is an E5M2, three bits
//   of it, and the rest, times 8, is an f16 again, whose last bit comes within E5M2's range in time (2^-24
//   512 = 2^-15; without the factors what lies below 2^-16 would be cut off).  Each row has its own reference for p 2^e_V, beside the one for p: a block of large
//   values that a row gives no weight takes no bits from it, whatever other rows make of that block.
// One thread holds one token of a tile: its scores of all rows, so a weight's bytes for all rows and
// terms are 32 or 64 bytes side by side (the operand's rows are tokens).  The rows' two references
// move only when they are exceeded by more than 7 (a factor 2^7 of the weights), which one vote of the
// 128 threads finds; only then are maxima exchanged and O is rescaled.  The sums of the weights stay in
// the threads, in fp32, until a run ends.
//
// Warps: 0 walks over the items and loads the tiles (lanes look up pages and issue one box each), 1
// issues both products (that of tile i + 1's scores before that of tile i's values), 2-5 are
// the 128 threads.  S and P have two buffers: the first product of tile i + 1 runs while tile i's
// weights are made.  The token threads' work is a chain of latencies (one warp to a scheduler), so
// three CTAs share an SM (two where tensor or shared memory has no room for more): one's waits, and its
// beginnings and ends of items, hide behind the others' tiles.
// 131071 tokens, 64 heads on 8: 60 us (4.5 TB/s over all, 6.5 inside a run); 64 ragged sequences, 32 on 8:
// 88 us (4.5 TB/s); 517 tokens, 32 on 8: 12.5 us, the latency of five tiles and of the two ends.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "fp8kv_common.cuh"

namespace bsp {

int kv_check_cache(KvCache& c, const void* k_cache, const void* v_cache, const void* k_scale,
                   const void* v_scale, int64_t pages, int64_t page_size, const int32_t* table,
                   int64_t max_pages, const int32_t* cu_new, const int32_t* kv_len, int64_t B,
                   int64_t T, int64_t Hq, int64_t Hkv, int64_t D);
int kv_check_pointers(const KvCache& c);

namespace {

constexpr int kThreads = 192;                    // loads, issuer, 128 token threads
constexpr int kTile = 128;                       // tokens of a tile
constexpr int kMaxRows = 16;
constexpr int kMaxCtas = 480;
constexpr int kQueue = 4;                        // segments that the loads are ahead by
constexpr int kMaxSlots = 12;
constexpr int kAtom = kTile * 128;               // 128 tokens x 128 bytes
constexpr int kPShift = 8;
constexpr float kMaxGrowth = 7.0f;               // 2^(8 + 7) is below the largest f16

struct Cut;

struct AttnParams {
    KvCache c;
    const __nv_bfloat16* q;
    int64_t q_stride;
    __nv_bfloat16* out;
    float* lse;
    float scale_log2;        // sm_scale * log2(e) = scale_log2 2^scale_exp: one below 1 is given in [1, 2),
    int32_t scale_exp;       // and its power of two goes to the keys' scales
    int32_t window;          // 0: none
    int32_t G;
    int32_t rows;            // R: rows of a row tile
    int32_t slot_rows;       // rows of a part in the workspace
    float* parts;            // [2 * ctas][slot_rows][D + 2]: output, maximum, sum of a part
    Cut* cuts;               // [ctas]
    int32_t box;             // tokens of one load: the largest power of two that divides a page
    int32_t slots;           // of the ring
    bool whole;              // every item fits in a run of W::kWhole and has its own CTA
    int32_t stop_loads;      // a CTA's loads end after that many (tests of the waits; else never)
    uint64_t wait_ns;
    int* status;
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log of the sum l of weights exp2(s - m)
__device__ __forceinline__ float lse_of(float m, float l)
{
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// ---- how the work is split.  An item is one row tile of one key head of a sequence; sequence b
// has items(b) = row tiles * Hkv of tiles(b) token tiles each.  An item weighs its tiles and W::kItem
// for its beginning and end.  All items in a row are cut into runs of equal weight, one for each CTA,
// whatever the lengths are: a run may end one item, hold whole ones and begin another.  Only the first
// and the last item of a run can be cut, so a CTA leaves at most two parts; the CTA that begins an
// item and does not end it notes that, and fp8kv_join_kernel adds the item's parts in order.
// Where there is little work, the items are aligned to the runs: then no CTA goes through the end of one
// item and the beginning of another.  If the tables are so short that every item fits in a run of
// W::kWhole, and there are CTAs for all, none is cut and nothing joined (517 tokens x 8 heads: 12.9 us,
// and 13.6 cut in two); else every item has its own runs of W::kMin, if the CTAs suffice for that
// (9910 tokens x 5 heads: 22 us, 29 in runs of W::kWhole).
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
    s.row_tiles = (s.n * p.G + p.rows - 1) / p.rows;
    const int32_t lo = p.window ? max(0, s.len - s.n - p.window + 1) : 0;
    s.tile0 = lo / kTile;
    s.tiles = max(1, (s.len + kTile - 1) / kTile - s.tile0);
    return s;
}

// Weights, in tiles.  A tile of a wide head takes twice as long, its beginning and end do not (11863
// tokens of 192: 29 us, 31 with 3; 131071 of 128 take 60 either way, ragged batches 1 to 5 % more with 2 or 4).
template <int COST>
struct Weights {
    static constexpr int kItem = COST;           // of an item, besides its tiles
    static constexpr int kWhole = COST + 5;      // items of at most that weight are better not cut
    static constexpr int kMin = COST + 2;        // what a CTA takes at least, where they are
};

// Weight of an item of the sequence, and of all of them
template <class W>
__device__ __forceinline__ int32_t item_weight(const AttnParams& p, const SeqWork& s, bool aligned)
{
    const int32_t w = s.tiles + W::kItem;
    if (!aligned) return w;
    return p.whole ? W::kWhole : (w + W::kMin - 1) / W::kMin * W::kMin;
}

template <class W>
__device__ __forceinline__ int64_t seq_weight(const AttnParams& p, const SeqWork& s, bool aligned)
{
    return static_cast<int64_t>(s.row_tiles) * p.c.Hkv * item_weight<W>(p, s, aligned);
}

struct SplitShared {
    int64_t warp_sum[8];
    int64_t before;              // weight of the sequences before b
    int b;
};

__device__ __forceinline__ int64_t chunk_scan(int64_t w, SplitShared& sh, int64_t& chunk)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
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
    for (int i = 0; i < warps; ++i) {
        if (i < warp) pre += sh.warp_sum[i];
        chunk += sh.warp_sum[i];
    }
    return pre + inc - w;        // weight before this thread's sequence, in this chunk
}

// How the row is cut, and the sequence that holds the beginning of CTA blockIdx.x's run (if the row is
// that long).
struct Split {
    int64_t total, per;
    bool aligned;
    int64_t before;              // weight of the sequences before b
    int b;
};

template <class W>
__device__ __forceinline__ bool cut_by(const AttnParams& p, Split& s, int64_t total, bool aligned)
{
    const int ctas = gridDim.x;
    s.total = total;
    s.aligned = aligned;
    s.per = aligned && p.whole ? W::kWhole : W::kMin;
    if (total <= s.per * ctas) return true;
    s.per = (total + ctas - 1) / ctas;
    return !aligned;
}

// Up to 32 sequences: one warp finds it, without a barrier.
template <class W>
__device__ __forceinline__ Split find_run_warp(const AttnParams& p)
{
    const int lane = threadIdx.x & 31;
    const bool in = lane < p.c.B;
    SeqWork sw = {};
    if (in) sw = seq_work(p, lane);
    Split s;
    for (int aligned = 1; aligned >= 0; --aligned) {
        const int64_t w = in ? seq_weight<W>(p, sw, aligned) : 0;
        int64_t inc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += y;
        }
        if (!cut_by<W>(p, s, __shfl_sync(0xFFFFFFFFu, inc, 31), aligned)) continue;
        const int64_t at = blockIdx.x * s.per;
        const uint32_t here = __ballot_sync(0xFFFFFFFFu, at >= inc - w && at < inc);
        s.b = here ? __ffs(here) - 1 : 0;
        s.before = __shfl_sync(0xFFFFFFFFu, inc - w, s.b);
        break;
    }
    return s;
}

// Any number of them: called by every thread.
template <class W>
__device__ __forceinline__ Split find_run(const AttnParams& p, SplitShared& sh)
{
    const int threads = blockDim.x;
    Split s;
    int64_t w = 0, excl = 0, chunk = 0;
    for (int aligned = 1; aligned >= 0; --aligned) {
        int64_t total = 0;
        for (int base = 0; base < p.c.B; base += threads) {
            const int i = base + threadIdx.x;
            w = i < p.c.B ? seq_weight<W>(p, seq_work(p, i), aligned) : 0;
            excl = chunk_scan(w, sh, chunk);
            total += chunk;
        }
        if (cut_by<W>(p, s, total, aligned)) break;
    }
    const int64_t at = blockIdx.x * s.per;
    if (threadIdx.x == 0) {
        sh.b = 0;
        sh.before = 0;
    }
    __syncthreads();
    int64_t carry = 0;
    for (int base = 0; base < p.c.B; base += threads) {
        const int i = base + threadIdx.x;
        if (p.c.B > threads) {                   // otherwise it is still in registers
            w = i < p.c.B ? seq_weight<W>(p, seq_work(p, i), s.aligned) : 0;
            excl = chunk_scan(w, sh, chunk) + carry;
            carry += chunk;
        }
        if (at >= excl && at < excl + w) {
            sh.b = i;
            sh.before = excl;
        }
    }
    __syncthreads();
    s.b = sh.b;
    s.before = sh.before;
    return s;
}

// An item, or a part of one, in a run.
struct Segment {
    SeqWork sw;
    int b, h, row_base, nrows;   // nrows < 0: the run has ended
    int tile_begin, tile_end;    // token tiles of the sequence
    int parts;                   // of the item from this one on, when it begins and does not end here
    bool begins, whole;
};

// A whole warp walks: every lane holds the same state.
template <class W>
struct SegmentWalk {
    int64_t at, end, before;
    int b;

    // A padded batch may hold many sequences without new tokens: passes the ones behind b, 32 at a time
    __device__ __forceinline__ void skip_empty(const AttnParams& p)
    {
        uint32_t found = 0;
        while (!found && b + 1 < p.c.B) {
            const int i = b + 1 + static_cast<int>(threadIdx.x & 31);
            found = __ballot_sync(0xFFFFFFFFu, i < p.c.B && kv_rows(p.c, i).n > 0);
            b = min(b + (found ? __ffs(found) - 1 : 32), p.c.B - 1);
        }
    }

    __device__ __forceinline__ bool next(const AttnParams& p, const Split& split, Segment& s)
    {
        while (at < end) {
            s.sw = seq_work(p, b);
            int64_t mine = seq_weight<W>(p, s.sw, split.aligned);
            while (at >= before + mine && b + 1 < p.c.B) {
                before += mine;
                s.sw = seq_work(p, ++b);
                mine = seq_weight<W>(p, s.sw, split.aligned);
                if (s.sw.n == 0) skip_empty(p);
            }
            const int weight = item_weight<W>(p, s.sw, split.aligned);
            const int64_t off = at - before;
            const int64_t item = off < (int64_t{1} << 31)
                                     ? static_cast<uint32_t>(off) / static_cast<uint32_t>(weight)
                                     : off / weight;
            const int from = static_cast<int>(off - item * weight);
            const int to = static_cast<int>(min(static_cast<int64_t>(weight), from + (end - at)));
            at += to - from;
            // the item's first W::kItem units hold no tile, and none follows its tiles
            const int seg0 = max(0, from - W::kItem);
            const int seg1 = min(s.sw.tiles, max(0, to - W::kItem));
            if (seg0 >= seg1) continue;
            s.b = b;
            s.begins = seg0 == 0;
            s.whole = seg0 == 0 && seg1 == s.sw.tiles;
            // the run that holds the item's last tile, counted from this one, whose last unit is at - 1
            s.parts = static_cast<int>((before + item * weight + W::kItem + s.sw.tiles - 1) / split.per -
                                       (at - 1) / split.per) + 1;
            s.h = static_cast<int>(static_cast<uint32_t>(item) / static_cast<uint32_t>(s.sw.row_tiles));
            s.row_base = static_cast<int>(item - static_cast<int64_t>(s.h) * s.sw.row_tiles) * p.rows;
            s.nrows = min(p.rows, s.sw.n * p.G - s.row_base);
            s.tile_begin = s.sw.tile0 + seg0;
            s.tile_end = s.sw.tile0 + seg1;
            return true;
        }
        return false;
    }
};

// What the join has to know of an item that CTA i began and did not end; parts = 0: there is none.
struct Cut {
    int32_t parts, nrows, row_base, h, first, pad[3];
};

// ---- PTX
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar,
                                            int32_t x, int32_t y, int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, float (&r)[8])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
          "=f"(r[7])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const float (&r)[8])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
        "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Barriers of the 128 token threads.
__device__ __forceinline__ void token_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ bool token_any(bool b)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "barrier.cta.red.or.pred p, 1, 128, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(b))
        : "memory");
    return r != 0;
}

// Descriptor of an operand whose rows (the K dimension) hold `row_bytes` = 32, 64 or 128 bytes
// of the M or N dimension, swizzled over as many bytes; groups of eight rows follow one another.
__device__ __forceinline__ uint64_t sdesc_mn_major(uint32_t saddr, int row_bytes)
{
    const uint64_t layout = row_bytes == 32 ? 6 : row_bytes == 64 ? 4 : 2;
    uint64_t d = (saddr >> 4) & 0x3FFFu;
    d |= static_cast<uint64_t>(1) << 16;                          // one atom wide: not used
    d |= static_cast<uint64_t>(row_bytes * 8 >> 4) << 32;         // next eight rows
    d |= static_cast<uint64_t>(1) << 46;
    d |= layout << 61;
    return d;
}

// E4M3 x E5M2 -> F32, both operands with their M / N dimension contiguous.
__host__ __device__ constexpr uint32_t idesc_pv(uint32_t M, uint32_t N)
{
    return (1u << 4) | (0u << 7) | (1u << 10) | (1u << 15) | (1u << 16) | ((N >> 3) << 17) |
           ((M >> 4) << 24);
}

// 0x80 in each byte of w that is an E4M3 NaN
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w)
{
    return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Order-preserving map of a float that is not NaN to an int
__device__ __forceinline__ int ordered(float f)
{
    const int i = __float_as_int(f);
    return i ^ ((i >> 31) & 0x7FFFFFFF);
}

__device__ __forceinline__ float from_ordered(int i)
{
    return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF));
}

// A wait's long form as a function of its own: see Cfg::wait.
__device__ __noinline__ bool wait_longer(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                         uint64_t limit_ns, int* status, int where)
{
    return mbar_wait(bar, parity, abort_flag, limit_ns, status, where);
}

// R: rows of a row tile; ATOMS: 128-byte pieces of a head.
template <int R, int ATOMS>
struct Cfg {
    using W = Weights<ATOMS == 1 ? 3 : 2>;
    static constexpr int kNS = (3 * R + 15) / 16 * 16;            // columns of S
    static constexpr int kNO = 4 * R;                             // columns of O
    static constexpr int kOCol = 2 * kNS;                         // tensor memory: S at 0, then O
    static constexpr int kCols = kOCol + ATOMS * kNO;
    static constexpr uint32_t kTmemCols = kCols <= 128 ? 128 : 256;
    static constexpr int kCtas = kTmemCols <= 128 && ATOMS == 1 ? 3 : 2;    // of an SM
    static constexpr int kSlot = ATOMS * kAtom;
    static constexpr int kQ = ATOMS * kNS * 128;
    static constexpr int kP = kTile * kNO;                        // one of two buffers
    static constexpr int kRoom = (kCtas == 3 ? 73 : 110) * 1024;
    static constexpr int kSlots = std::min(kMaxSlots, (kRoom - kQ - 2 * kP) / kSlot);
    static constexpr int kSmem = 1024 + kSlots * kSlot + kQ + 2 * kP;
    static_assert((R == 8 || R == 16) && kSlots >= 2 && kCols <= 256, "shared and tensor memory");
    static_assert(kSmem >= kLeastSmemWithTmem, "no room beside a GEMM's CTA");
    // With 16 rows of a narrow head the code is kept short by calls for the long form of a wait (56 rows of
    // each of 17 sequences: 93 -> 80 us; 8 new tokens of 9910: 22.1 -> 20.8); with 8 rows those cost
    // registers (131071 tokens: 60 -> 65 us; 63 where the token threads make none), with wide heads 2 %.
    static __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                uint64_t limit_ns, int* status, int where)
    {
        if constexpr (R == 16 && ATOMS == 1)
            return mbar_try_wait_for(bar, parity, 20000u) ||
                   wait_longer(bar, parity, abort_flag, limit_ns, status, where);
        else
            return mbar_wait(bar, parity, abort_flag, limit_ns, status, where);
    }
};

template <int R>
struct TokenShared {
    float row_fac[R];                            // scores: sm_scale log2(e) 2^(row's power)
    int row_pos[R];
    // References of a row: m of its scores (base 2), m + d of its scores plus the value blocks' exponents,
    // d the whole number above `top`, the largest of these (less m) when they last moved.  The largest
    // weight is 1 and its product with a power of two exact then.  And what the last change of the
    // references was: m's, and the factors of l and O.
    float m[R], d[R], top[R], dm[R], fl[R], fo[R];
    uint32_t unset;                              // rows whose references are not set yet
    int smax[4][R], tmax[4][R];
    float wsum[4][R];
    float inv[R], unit[R];                       // of a segment's end
    void* to[R];                                 // where the row's output or part goes
    uint32_t nan[R][8];                          // NaN elements of V that a row sees, by d
};

// All elements of a token's values are NaN: so are those of every row that sees it.  (A call: rare, and the
// code of a tile stays short.)
template <int R>
__device__ __noinline__ void note_nan_values(TokenShared<R>& sh, int tok, int window)
{
#pragma unroll 1
    for (int r = 0; r < R; ++r) {
        const int pos = sh.row_pos[r];
        if (tok > pos || (window && tok <= pos - window)) continue;
#pragma unroll 1
        for (int k = 0; k < 8; ++k) atomicOr(&sh.nan[r][k], 0xFFFFFFFFu);
    }
}

template <int R, int ATOMS>
__global__ void __launch_bounds__(kThreads, Cfg<R, ATOMS>::kCtas)
    fp8kv_attention_kernel(const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const AttnParams p)
{
    using C = Cfg<R, ATOMS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* qs = ring + C::kSlots * C::kSlot;                    // [ATOMS][kNS][128]
    uint8_t* ps = qs + C::kQ;                                     // [2][128 tokens][kNO]
    __shared__ uint64_t full[kMaxSlots], empty[kMaxSlots];
    __shared__ uint64_t s_full[2], s_free[2], p_full[2], p_done[2], q_full, fin;
    __shared__ uint64_t seg_full[kQueue], seg_free[kQueue];
    __shared__ Segment queue[kQueue];
    __shared__ uint32_t tmem_holder;
    __shared__ int abort_word;
    __shared__ SplitShared split;
    __shared__ TokenShared<R> sh;
    volatile int* abort_flag = &abort_word;

    const KvCache& c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(s_free + i, 4);
            mbar_init(p_full + i, 4);
            mbar_init(p_done + i, 1);
        }
        for (int i = 0; i < kQueue; ++i) {
            mbar_init(seg_full + i, 1);
            mbar_init(seg_free + i, 5);
        }
        mbar_init(&fin, 1);
        mbar_init(&q_full, 4);
        abort_word = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    if (warp == 1) {
        tmem_alloc(&tmem_holder, C::kTmemCols);
        tmem_relinquish();
    }
    griddep_wait();
    Split cut_up;                                // only the loads ask for it
    if (p.c.B > 32)
        cut_up = find_run<typename C::W>(p, split);
    else if (warp == 0)
        cut_up = find_run_warp<typename C::W>(p);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();                 // not before this CTA has its tensor memory
    const uint32_t tbase = tmem_holder;
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        const int boxes = kTile / p.box, page = c.page_blocks * kKvBlock;
        const uint32_t box_bytes = p.box * 128;
        int slot = 0, used = 0;
        uint32_t phase = 1;                      // of an empty slot's barrier, for the first round
        bool ok = true;
        SegmentWalk<typename C::W> walk;
        walk.at = blockIdx.x * cut_up.per;
        walk.end = min(walk.at + cut_up.per, cut_up.total);
        walk.before = cut_up.before;
        walk.b = cut_up.b;
        Segment seg;
        for (int nseg = 0; ok; ++nseg) {
            const bool more = walk.next(p, cut_up, seg);
            const int e = nseg % kQueue;
            bool room = true;
            if (lane == 0) {
                room = C::wait(seg_free + e, (nseg / kQueue & 1) ^ 1u, abort_flag, p.wait_ns,
                                 p.status, 110);
                if (room) {
                    if (!more) seg.nrows = -1;
                    queue[e] = seg;
                    mbar_arrive(seg_full + e);
                }
            }
            ok = __shfl_sync(0xFFFFFFFFu, room, 0);
            if (!ok || !more) break;
            const int len = seg.sw.len;
            if (lane == 0 && c.kv_len[seg.b] != len) kv_report_bad_batch(p.status);
            const int lo = p.window ? max(0, len - seg.sw.n - p.window + 1) : 0;
            const int32_t* row = c.table + static_cast<int64_t>(seg.b) * c.max_pages;
            // lane i takes box i of a tile; -1: nothing to load
            const auto page_of = [&](int tile) {
                const int tok = tile * kTile + lane * p.box;
                return lane < boxes && tile < seg.tile_end && tok < len && tok + p.box > lo
                           ? row[tok / page]
                           : -1;
            };
            int32_t next_page = page_of(seg.tile_begin);
            for (int tile = seg.tile_begin; ok && tile < seg.tile_end; ++tile) {
                const int32_t id = next_page;
                next_page = page_of(tile + 1);
                const int tok = tile * kTile + lane * p.box;
                const bool mine = id >= 0 && id < c.pages;
                if (!mine && id != -1) kv_report_bad_batch(p.status);
                if (id == -1 && lane < boxes && tok < len && tok + p.box > lo)
                    kv_report_bad_batch(p.status);
                const uint32_t bytes =
                    __popc(__ballot_sync(0xFFFFFFFFu, mine)) * box_bytes * ATOMS;
                const int32_t y = tok % page, z = mine ? id * c.Hkv + seg.h : 0;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    bool got = true;
                    if (lane == 0) {
                        got = used < p.stop_loads &&
                              C::wait(empty + slot, phase, abort_flag, p.wait_ns, p.status, 111);
                        if (got) mbar_arrive_expect_tx(full + slot, bytes);
                    }
                    ok = __shfl_sync(0xFFFFFFFFu, got, 0);
                    if (!ok) break;
                    if (mine)
                        for (int a = 0; a < ATOMS; ++a)
                            tma_load_3d(ring + slot * C::kSlot + a * kAtom + lane * box_bytes,
                                        kv ? &tm_v : &tm_k, full + slot, a * 128, y, z);
                    ++used;
                    if (++slot == C::kSlots) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
        }
        // the last loads must land before shared memory is freed
        __syncwarp();
        if (lane == 0)
            for (int i = max(0, used - C::kSlots); i < used; ++i)
                drain_wait(full + i % C::kSlots, i / C::kSlots & 1, p.wait_ns, p.status);
    } else if (warp == 1) {
        // ------------------------------------------------------------ S = K Q^T, O += V^T P^T
        if (lane == 0) {
            const uint32_t idesc_s = idesc_e4m3(kTile, C::kNS), idesc_o = idesc_pv(kTile, C::kNO);
            const int ksteps = (c.D + 31) / 32;
            int kslot = 0, vslot = 1, i = 0;
            uint32_t kphase = 0, vphase = 0;
            const auto forward = [&](int& slot, uint32_t& phase) {
                slot += 2;
                if (slot >= C::kSlots) {
                    slot -= C::kSlots;
                    phase ^= 1;
                }
            };
            // O += V^T P^T of tile j of the run
            const auto values = [&](int j, bool fresh) {
                if (!C::wait(full + vslot, vphase, abort_flag, p.wait_ns, p.status, 115) ||
                    !C::wait(p_full + (j & 1), j >> 1 & 1, abort_flag, p.wait_ns, p.status, 116))
                    return false;
                tc_fence_after();
                const uint32_t a = smem_u32(ring + vslot * C::kSlot);
                const uint64_t b = sdesc_mn_major(smem_u32(ps + (j & 1) * C::kP), C::kNO);
#pragma unroll
                for (int at = 0; at < ATOMS; ++at) {
                    const uint64_t ad = sdesc_mn_major(a + at * kAtom, 128);
#pragma unroll
                    for (int k = 0; k < 4; ++k)          // 32 tokens each
                        mma_f8f6f4(tbase + C::kOCol + at * C::kNO, ad + k * (32 * 128 / 16),
                                   b + k * (32 * C::kNO / 16), idesc_o, !fresh || k > 0);
                }
                tc_commit(empty + vslot);
                tc_commit(p_done + (j & 1));
                forward(vslot, vphase);
                return true;
            };
            bool ok = true;
            for (int nseg = 0; ok; ++nseg) {
                const int e = nseg % kQueue;
                ok = C::wait(seg_full + e, nseg / kQueue & 1, abort_flag, p.wait_ns, p.status, 122);
                if (!ok || queue[e].nrows < 0) break;
                const int begin = queue[e].tile_begin, end = queue[e].tile_end;
                mbar_arrive(seg_free + e);
                ok = C::wait(&q_full, nseg & 1, abort_flag, p.wait_ns, p.status, 112);
                for (int tile = begin; ok && tile < end; ++tile, ++i) {
                    ok = C::wait(s_free + (i & 1), (i >> 1 & 1) ^ 1u, abort_flag, p.wait_ns,
                                   p.status, 113) &&
                         C::wait(full + kslot, kphase, abort_flag, p.wait_ns, p.status, 114);
                    if (!ok) break;
                    tc_fence_after();
                    uint64_t a = sdesc_kmajor_sw128(smem_u32(ring + kslot * C::kSlot));
                    uint64_t b = sdesc_kmajor_sw128(smem_u32(qs));
#pragma unroll 1
                    for (int k = 0; k < ksteps; ++k) {
                        mma_f8f6f4(tbase + (i & 1) * C::kNS, a, b, idesc_s, k);
                        // 32 bytes a step, four steps to a 128-byte atom; units of 16 bytes
                        a += (k & 3) == 3 ? kAtom / 16 - 6 : 2;
                        b += (k & 3) == 3 ? C::kNS * 8 - 6 : 2;
                    }
                    tc_commit(empty + kslot);
                    // also says that tile i - 2's second product is done, so P's buffer is free
                    tc_commit(s_full + (i & 1));
                    forward(kslot, kphase);
                    if (tile > begin) ok = values(i - 1, tile == begin + 1);
                }
                ok = ok && values(i - 1, end == begin + 1);
            }
        }
    } else {
        // ------------------------------------------------------------ the token threads
        const int q = warp & 3, t = q * 32 + lane;               // TMEM lane, and token of a tile
        const uint32_t tlane = tbase + (static_cast<uint32_t>(q * 32) << 16);
        int i = 0, slot = 1;
        uint32_t phase = 0;                                       // of this tile's V slot
        bool ok = true;
        // a thread's 16-token block one tile on: pages and blocks to add
        const int step_pages = kTile / kKvBlock / c.page_blocks;
        const int step_blocks = kTile / kKvBlock - step_pages * c.page_blocks;
        Cut cut = {};
        for (int nseg = 0;; ++nseg) {
            const int e = nseg % kQueue;
            ok = C::wait(seg_full + e, nseg / kQueue & 1, abort_flag, p.wait_ns, p.status, 123) && ok;
            if (token_any(!ok)) break;
            const Segment seg = queue[e];
            __syncwarp();
            if (lane == 0) mbar_arrive(seg_free + e);
            if (seg.nrows < 0) break;
            if (seg.begins && !seg.whole) {
                cut.parts = seg.parts;
                cut.nrows = seg.nrows;
                cut.row_base = seg.row_base;
                cut.h = seg.h;
                cut.first = seg.sw.first;
            }
            const int len = seg.sw.len, nrows = seg.nrows;
            const int start = len - seg.sw.n;                     // position of the first new token
            const int pos_lo = start + seg.row_base / p.G;
            const int pos_hi = start + (seg.row_base + nrows - 1) / p.G;
            const int lo = p.window ? max(0, pos_lo - p.window + 1) : 0;
            const int32_t* table = c.table + static_cast<int64_t>(seg.b) * c.max_pages;

            // scales: the page of tile i + 2 and the scales of tile i + 1 are on their way during tile i
            struct Scales {                                       // as loaded: combining them would wait
                uint8_t k, v;
                bool in;
            };
            int at_page, at_block;                                // of the tile whose page is asked for
            {
                const uint32_t blk = (seg.tile_begin * kTile + t) / kKvBlock;
                at_page = blk / static_cast<uint32_t>(c.page_blocks);
                at_block = blk - at_page * c.page_blocks;
            }
            const auto page_of = [&](int tile) {
                const int tok = tile * kTile + t;
                return tile < seg.tile_end && tok < len && tok >= lo ? table[at_page] : -1;
            };
            const auto forward = [&] {
                at_page += step_pages;
                at_block += step_blocks;
                if (at_block >= c.page_blocks) {
                    at_block -= c.page_blocks;
                    ++at_page;
                }
            };
            const auto scales_of = [&](int32_t id, int block) {
                Scales x = {127, 0, id >= 0 && id < c.pages};
                if (x.in) {
                    const int64_t at =
                        (static_cast<int64_t>(id) * c.Hkv + seg.h) * c.page_blocks + block;
                    x.k = c.k_scale[at];
                    x.v = c.v_scale[at];
                }
                return x;
            };
            const int32_t page0 = page_of(seg.tile_begin);
            const int block0 = at_block;
            forward();
            int32_t page1 = page_of(seg.tile_begin + 1);
            int block1 = at_block;
            Scales scale0;

            // ---- q: three E4M3 rows each
            constexpr int kSide = 2;                              // rows of a warp whose loads are in flight
#pragma unroll 1
            for (int r0 = q; r0 < R; r0 += 4 * kSide) {
                uint32_t w[kSide][2 * ATOMS];
#pragma unroll
                for (int u = 0; u < kSide; ++u) {
                    const int r = r0 + 4 * u, rr = seg.row_base + r, tok = rr / p.G;
                    const __nv_bfloat16* src = p.q + (seg.sw.first + tok) * p.q_stride +
                                               static_cast<int64_t>(seg.h * p.G + rr - tok * p.G) * c.D;
#pragma unroll
                    for (int j = 0; j < 2 * ATOMS; ++j) {
                        const int d = 2 * (lane + 32 * j);
                        w[u][j] = r < nrows && d < c.D ? *reinterpret_cast<const uint32_t*>(src + d) : 0u;
                    }
                    if (lane == 0)
                        sh.row_pos[r] = start + (seg.row_base + min(r, nrows - 1)) / p.G;
                }
                if (r0 == q) scale0 = scales_of(page0, block0);  // its page has come meanwhile
#pragma unroll
                for (int u = 0; u < kSide; ++u) {
                    const int r = r0 + 4 * u;
                    uint32_t amax = 0;
#pragma unroll
                    for (int j = 0; j < 2 * ATOMS; ++j)
                        amax = max(amax, max(w[u][j] << 16 & 0x7FFFFFFFu, w[u][j] & 0x7FFF0000u));
                    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
                    const int ex = max(static_cast<int>(amax >> 23), 8);  // biased exponent of the largest
                    const float up = kv_pow2(min(254, 261 - ex));         // 2^(7 - (ex - 127))
                    if (lane == 0)
                        sh.row_fac[r] = amax < 0x7F800000u ? p.scale_log2 * kv_pow2(ex - 7) : NAN;
#pragma unroll
                    for (int j = 0; j < 2 * ATOMS; ++j) {
                        const int d = 2 * (lane + 32 * j), byte = d & 127;
                        float x0 = bf16lo_to_f32(w[u][j]) * up, x1 = bf16hi_to_f32(w[u][j]) * up;
#pragma unroll
                        for (int k = 0; k < 3; ++k) {
                            const uint32_t code = cvt_e4m3x2(x0, x1);
                            const int n = k * R + r;
                            *reinterpret_cast<uint16_t*>(qs + (d >> 7) * C::kNS * 128 + n * 128 +
                                                         (((byte >> 4) ^ (n & 7)) << 4) + (byte & 15)) =
                                static_cast<uint16_t>(code);
                            uint32_t h, unused;
                            e4m3x4_to_f16(code, h, unused);
                            float y0, y1;
                            f16x2_to_f32(h, y0, y1);
                            x0 = (x0 - y0) * 16.0f;
                            x1 = (x1 - y1) * 16.0f;
                        }
                    }
                }
            }
            for (int k = t; k < R * 8; k += 128) sh.nan[k >> 3][k & 7] = 0;
            if (t < R) sh.m[t] = sh.d[t] = sh.top[t] = 0.0f;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full);
            token_sync();

            float l[R] = {};
            uint32_t unset = 0xFFFFFFFFu >> (32 - R);             // sh.unset
            bool any_nan = false;

            for (int tile = seg.tile_begin; tile < seg.tile_end; ++tile, ++i) {
                const Scales scale = scale0;
                scale0 = scales_of(page1, block1);
                forward();
                page1 = page_of(tile + 2);
                block1 = at_block;
                const int tok = tile * kTile + t;
                const bool seen = scale.in && tok <= pos_hi;      // by some row, and the page is good
                // byte 255 is a NaN: one of a key makes its scores NaN, one of values is noted below
                const bool nan_v = seen && scale.v == 255;
                const float ev = seen && !nan_v ? static_cast<float>(scale.v) : 0.0f;
                const float kf = !seen ? 1.0f : scale.k < 255 ? kv_pow2_low(scale.k + p.scale_exp) : NAN;
                const bool edge = tile * kTile + kTile - 1 > pos_lo ||
                                  (p.window && tile * kTile <= pos_hi - p.window);

                ok = C::wait(s_full + (i & 1), i >> 1 & 1, abort_flag, p.wait_ns, p.status, 117) &&
                     ok;
                tc_fence_after();
                __syncwarp();
                float s[R];                                       // scores less the row's reference
#pragma unroll
                for (int r0 = 0; r0 < R; r0 += 8) {
                    float x[3][8];
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        tmem_ld_x8(tlane + (i & 1) * C::kNS + k * R + r0, x[k]);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        s[r0 + j] = fmaf(fmaf(fmaf(x[2][j], 0.0625f, x[1][j]), 0.0625f, x[0][j]),
                                         sh.row_fac[r0 + j] * kf, -sh.m[r0 + j]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free + (i & 1));
                if (!seen) {
#pragma unroll
                    for (int r = 0; r < R; ++r) s[r] = -INFINITY;
                } else if (edge) {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const int pos = sh.row_pos[r];
                        if (tok > pos || (p.window && tok <= pos - p.window)) s[r] = -INFINITY;
                    }
                }
                float most = s[0], most_v = s[0] - sh.d[0];       // NaN is no reason to move a reference
#pragma unroll
                for (int r = 1; r < R; ++r) {
                    most = fmaxf(most, s[r]);
                    most_v = fmaxf(most_v, s[r] - sh.d[r]);
                }
                const bool exceed = fmaxf(most, most_v + ev) > (unset ? -INFINITY : kMaxGrowth);

                if (token_any(exceed || !ok)) {
                    if (token_any(!ok)) {                         // a wait ran out
                        ok = false;
                        break;
                    }
                    // ---- new references; l and O follow
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float x = s[r] == s[r] ? s[r] : -INFINITY;
                        const int v = __reduce_max_sync(0xFFFFFFFFu, ordered(x));
                        const int u = __reduce_max_sync(0xFFFFFFFFu, ordered(x + ev));
                        if (lane == 0) {
                            sh.smax[q][r] = v;
                            sh.tmax[q][r] = u;
                        }
                    }
                    token_sync();
                    if (q == 0) {
                        bool still = false;
                        if (lane < R) {
                            // once to the first maximum, then only up
                            const bool first = unset >> lane & 1u;
                            float v = from_ordered(max(max(sh.smax[0][lane], sh.smax[1][lane]),
                                                       max(sh.smax[2][lane], sh.smax[3][lane])));
                            float u = from_ordered(max(max(sh.tmax[0][lane], sh.tmax[1][lane]),
                                                       max(sh.tmax[2][lane], sh.tmax[3][lane])));
                            still = first && v == -INFINITY;      // nothing seen: all stays 0
                            if (still) v = u = 0.0f;
                            if (!first) v = fmaxf(v, 0.0f), u = fmaxf(u, sh.top[lane]);
                            const float d = ceilf(u - v), old = sh.d[lane];
                            sh.dm[lane] = v;
                            sh.m[lane] += v;
                            sh.top[lane] = u - v;
                            sh.d[lane] = d;
                            sh.fl[lane] = first ? 0.0f : ex2(-v);
                            sh.fo[lane] = first ? 0.0f : ex2(old - d - v);
                        }
                        const uint32_t left = __ballot_sync(0xFFFFFFFFu, still);
                        if (lane == 0) sh.unset = left;
                    }
                    token_sync();
                    unset = sh.unset;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        s[r] -= sh.dm[r];
                        l[r] *= sh.fl[r];
                    }
                    if (tile > seg.tile_begin) {
                        ok = C::wait(p_done + ((i - 1) & 1), (i - 1) >> 1 & 1, abort_flag,
                                       p.wait_ns, p.status, 118) &&
                             ok;
                        tc_fence_after();
#pragma unroll 1
                        for (int k = 0; k < ATOMS * 4; ++k)
#pragma unroll
                            for (int r0 = 0; r0 < R; r0 += 8) {
                                float o[8];
                                __syncwarp();
                                tmem_ld_x8(tlane + C::kOCol + k * R + r0, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int j = 0; j < 8; ++j) o[j] *= sh.fo[r0 + j];
                                tmem_st_x8(tlane + C::kOCol + k * R + r0, o);
                            }
                        tmem_st_wait();
                    }
                }

                // ---- weights, their sums, and their four E5M2 terms
                uint8_t* pt = ps + (i & 1) * C::kP + t * C::kNO;
                uint32_t h[R / 2];
#pragma unroll
                for (int r = 0; r < R; r += 2) {
                    const float p0 = ex2(s[r]), p1 = ex2(s[r + 1]);
                    l[r] += p0;
                    l[r + 1] += p1;
                    h[r / 2] = pack_f16(ex2(s[r] + (ev + kPShift - sh.d[r])),
                                        ex2(s[r + 1] + (ev + kPShift - sh.d[r + 1])));
                }
                uint32_t bytes[4][R / 4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
#pragma unroll
                    for (int j = 0; j < R / 4; ++j)
                        bytes[k][j] = __byte_perm(h[2 * j], h[2 * j + 1], 0x7531);
#pragma unroll
                    for (int j = 0; j < R / 2; ++j)               // the rest, times 8
                        h[j] = mul_f16x2(sub_f16x2(h[j], h[j] & 0xFF00FF00u), 0x48004800u);
                }
                // 16-byte chunks of the token's row, swizzled over its 32 or 64 bytes
                if constexpr (R == 8) {
                    const int x = (t >> 2) & 1;
                    *reinterpret_cast<uint4*>(pt + 16 * x) =
                        make_uint4(bytes[0][0], bytes[0][1], bytes[1][0], bytes[1][1]);
                    *reinterpret_cast<uint4*>(pt + 16 * (x ^ 1)) =
                        make_uint4(bytes[2][0], bytes[2][1], bytes[3][0], bytes[3][1]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<uint4*>(pt + 16 * (k ^ ((t >> 1) & 3))) =
                            make_uint4(bytes[k][0], bytes[k][1], bytes[k][2], bytes[k][3]);
                }

                // ---- A masked token's weight is 0, but 0 * NaN is not: the values of a token that no
                // row sees are cleared, and NaNs of one that only some rows see are taken out and
                // noted for just those rows.
                if (nan_v) {
                    note_nan_values(sh, tok, p.window);
                    any_nan = true;
                }
                if (!seen || edge) {
                    // This wait is for one fill of the slot among many, by parity: the fill before it must
                    // be known to be over, or the wait is taken for done while that one is under way.  With
                    // three slots or more it was a fill that the scores of an earlier tile needed; with two
                    // it is the values of the tile before, whose product has to be over anyway before the
                    // slot is filled again.
                    if (C::kSlots == 2 && tile > seg.tile_begin)
                        ok = C::wait(p_done + ((i - 1) & 1), (i - 1) >> 1 & 1, abort_flag, p.wait_ns,
                                     p.status, 119) &&
                             ok;
                    ok = C::wait(full + slot, phase, abort_flag, p.wait_ns, p.status, 120) && ok;
                    uint8_t* v = ring + slot * C::kSlot + t * 128;
#pragma unroll 1
                    for (int a = 0; a < ATOMS; ++a)
#pragma unroll 1
                        for (int k = 0; k < 8; ++k) {
                            uint4* at = reinterpret_cast<uint4*>(v + a * kAtom + 16 * (k ^ (t & 7)));
                            if (!seen) {
                                *at = make_uint4(0, 0, 0, 0);
                                continue;
                            }
                            uint4 x = *at;
                            const uint32_t n[4] = {nan_bytes(x.x), nan_bytes(x.y), nan_bytes(x.z),
                                                   nan_bytes(x.w)};
                            if ((n[0] | n[1] | n[2] | n[3]) == 0) continue;
                            uint32_t bits = 0;                    // of the 16 elements
#pragma unroll
                            for (int j = 0; j < 16; ++j) bits |= (n[j >> 2] >> (8 * (j & 3) + 7) & 1u) << j;
                            for (int r = 0; r < R; ++r) {
                                const int pos = sh.row_pos[r];
                                if (tok <= pos && (p.window == 0 || tok > pos - p.window))
                                    atomicOr(&sh.nan[r][a * 4 + (k >> 1)], bits << (16 * (k & 1)));
                            }
                            x.x &= ~((n[0] >> 7) * 0xFFu);
                            x.y &= ~((n[1] >> 7) * 0xFFu);
                            x.z &= ~((n[2] >> 7) * 0xFFu);
                            x.w &= ~((n[3] >> 7) * 0xFFu);
                            *at = x;
                            any_nan = true;
                        }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + (i & 1));
                slot += 2;
                if (slot >= C::kSlots) {
                    slot -= C::kSlots;
                    phase ^= 1;
                }
            }
            // `ok` is each thread's own here (a wait may have run out between two threads' looks), and
            // what follows is for all of them
            if (token_any(!ok)) break;

            // ---- end of the segment: sums over the tokens, then this thread's d of every row.  This code
            // runs once for many tiles: kept short, it does not wait for its own instructions.
            {
                // R sums over 32 lanes: lanes exchange halves of the rows, so that R / 2 + R / 4 + ..
                // shuffles leave each lane one row
                int row = 0;
#pragma unroll
                for (int n = R / 2, x = 16; x > 0; x >>= 1) {
                    if (n > 0) {
                        const bool up = lane & x;
#pragma unroll
                        for (int r = 0; r < n; ++r) {
                            const float give = up ? l[r] : l[r + n];
                            l[r] = (up ? l[r + n] : l[r]) + __shfl_xor_sync(0xFFFFFFFFu, give, x);
                        }
                        row += up ? n : 0;
                        n /= 2;
                    } else {
                        l[0] += __shfl_xor_sync(0xFFFFFFFFu, l[0], x);
                    }
                }
                sh.wsum[q][row] = l[0];                           // lanes of one row write the same
            }
            ok = C::wait(p_done + ((i - 1) & 1), (i - 1) >> 1 & 1, abort_flag, p.wait_ns, p.status,
                           121) &&
                 ok;
            const bool nans = token_any(any_nan);                 // also: the sums are written
            tc_fence_after();
            if (t < nrows) {
                const float sum = sh.wsum[0][t] + sh.wsum[1][t] + sh.wsum[2][t] + sh.wsum[3][t];
                const int rr = seg.row_base + t, tok = rr / p.G;
                const int64_t row = static_cast<int64_t>(seg.sw.first + tok) * c.Hq + seg.h * p.G + rr -
                                    tok * p.G;
                // the second factor may be subnormal: it comes last
                sh.inv[t] = sum == 0.0f ? 0.0f : 1.0f / sum;
                sh.unit[t] = ex2(sh.d[t] - (127 + kPShift));
                float* part = p.parts + (static_cast<int64_t>(2 * blockIdx.x + seg.begins) *
                                             p.slot_rows +
                                         t) * (c.D + 2);
                sh.to[t] = seg.whole ? static_cast<void*>(p.out + row * c.D) : part;
                if (!seg.whole) {
                    part[c.D] = sum == 0.0f ? -INFINITY : sh.m[t];
                    part[c.D + 1] = sum;
                } else if (p.lse) {
                    p.lse[row] = lse_of(sh.m[t], sum);
                }
            }
            token_sync();
#pragma unroll 1
            for (int a = 0; a < ATOMS; ++a) {
                const int d = a * 128 + t;
#pragma unroll 1
                for (int r0 = 0; r0 < nrows; r0 += 8) {
                    float o[4][8];
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tmem_ld_x8(tlane + C::kOCol + a * C::kNO + k * R + r0, o[k]);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int r = r0 + j;
                        if (r >= nrows || d >= c.D) break;
                        const float sum = fmaf(fmaf(fmaf(o[3][j], 0.125f, o[2][j]), 0.125f, o[1][j]),
                                               0.125f, o[0][j]);
                        float x = sum * sh.inv[r] * sh.unit[r];
                        if (nans && (sh.nan[r][d >> 5] >> (d & 31) & 1u)) x = NAN;
                        if (seg.whole)
                            static_cast<__nv_bfloat16*>(sh.to[r])[d] = __float2bfloat16_rn(x);
                        else
                            static_cast<float*>(sh.to[r])[d] = x;
                    }
                }
            }
            tc_fence_before();
            token_sync();                        // O, the sums and q's rows are free
        }
        if (t == 0) p.cuts[blockIdx.x] = cut;
    }

    // ---------------------------------------------------------------- teardown
    __syncwarp();
    if (warp == 1 && lane == 0) {
        tc_commit(&fin);
        drain_wait(&fin, 0, p.wait_ns, p.status);
    }
    __syncwarp();                                // what follows is for whole warps
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tbase, C::kTmemCols);
}

// Adds the parts of the items that some of the attention kernel's CTAs (`group` of them for each block)
// began and did not end: part i weighs l_i 2^(m_i - m).  `share` warps of the four
// take a row: one where there are many items of few parts, four where a few items have many.
constexpr int kJoinThreads = 128, kJoinWarps = kJoinThreads / 32;

template <int ATOMS>
__global__ void __launch_bounds__(kJoinThreads)
    fp8kv_join_kernel(const AttnParams p, int ctas, int group, int share)
{
    __shared__ float warp_m[kJoinWarps], warp_l[kJoinWarps], warp_x[kJoinWarps][ATOMS * 128];
    constexpr int kSide = 4, kV = 2 * ATOMS;     // parts whose loads are in flight, pairs of a lane
    const KvCache& c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.y * (kJoinWarps / share) + warp / share;
    griddep_wait();
    const int64_t step = static_cast<int64_t>(2) * p.slot_rows * (c.D + 2);
    // the block's CTAs are gridDim.x apart: neighbours' cuts go to different blocks
    const int look = blockIdx.x + lane * gridDim.x;
    uint32_t todo = __ballot_sync(0xFFFFFFFFu, lane < group && look < ctas && p.cuts[look].parts > 0);
    for (; todo; todo &= todo - 1) {
        const int cta = blockIdx.x + (__ffs(todo) - 1) * gridDim.x;
        const Cut cut = p.cuts[cta];
        const bool in = r < cut.nrows;
        const int parts = in ? cut.parts : 0;
        // part 0 is the second slot of this CTA, part i > 0 the first slot of CTA cta + i
        const float* rest = p.parts + (static_cast<int64_t>(2 * cta) * p.slot_rows + r) * (c.D + 2);
        const float* first = rest + step / 2;
        // a warp takes every share-th part: a running maximum, as in the attention itself
        float m = -INFINITY, l = 0.0f, x[2 * kV] = {};
        for (int i0 = warp % share; i0 < parts; i0 += share * kSide) {
            float pm[kSide], pl[kSide];
            float2 v[kSide][kV];
#pragma unroll
            for (int k = 0; k < kSide; ++k) {
                const int i = i0 + share * k;
                const float* part = i ? rest + i * step : first;
                pm[k] = i < parts ? part[c.D] : -INFINITY;
                pl[k] = i < parts ? part[c.D + 1] : 0.0f;
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    const int d = 2 * lane + 64 * j;
                    v[k][j] = make_float2(0.0f, 0.0f);
                    if (i < parts && d < c.D) v[k][j] = *reinterpret_cast<const float2*>(part + d);
                }
            }
#pragma unroll
            for (int k = 0; k < kSide; ++k) {
                const float top = fmaxf(m, pm[k]), z = top == -INFINITY ? 0.0f : top;
                const float old = ex2(m - z), w = pl[k] * ex2(pm[k] - z);
                m = top;
                l = fmaf(l, old, w);
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    x[2 * j] = fmaf(x[2 * j], old, w * v[k][j].x);
                    x[2 * j + 1] = fmaf(x[2 * j + 1], old, w * v[k][j].y);
                }
            }
        }
        __syncthreads();                         // the last item is read
        if (lane == 0) {
            warp_m[warp] = m;
            warp_l[warp] = l;
        }
#pragma unroll
        for (int j = 0; j < kV; ++j)
            *reinterpret_cast<float2*>(&warp_x[warp][2 * lane + 64 * j]) =
                make_float2(x[2 * j], x[2 * j + 1]);
        __syncthreads();
        if (!in) continue;
        const int w0 = warp / share * share;     // the row's first warp
        float top = -INFINITY, sum = 0.0f;
        for (int w = w0; w < w0 + share; ++w) top = fmaxf(top, warp_m[w]);
        const float z = top == -INFINITY ? 0.0f : top;
        for (int w = w0; w < w0 + share; ++w) sum = fmaf(warp_l[w], ex2(warp_m[w] - z), sum);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const int rr = cut.row_base + r, tok = rr / p.G, head = cut.h * p.G + rr - tok * p.G;
        const int64_t row = static_cast<int64_t>(cut.first + tok) * c.Hq + head;
        for (int d = (warp - w0) * 32 + lane; d < c.D; d += share * 32) {
            float y = 0.0f;
            for (int w = w0; w < w0 + share; ++w) y = fmaf(ex2(warp_m[w] - z), warp_x[w][d], y);
            p.out[row * c.D + d] = __float2bfloat16_rn(y * inv);
        }
        if (p.lse && warp == w0 && lane == 0) p.lse[row] = lse_of(top, sum);
    }
}

template <int R, int ATOMS>
int launch_attention(AttnParams p, const CUtensorMap& k, const CUtensorMap& v, int dev,
                     int sms, cudaStream_t s)
{
    using C = Cfg<R, ATOMS>;
    static std::atomic<bool> ready[kMaxDevices];
    if (!ready[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(fp8kv_attention_kernel<R, ATOMS>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::kSmem) != cudaSuccess) {
            cudaGetLastError();
            return BSP_ERR_CUDA;
        }
        ready[dev].store(true, std::memory_order_release);
    }
    const unsigned ctas = static_cast<unsigned>(std::min(sms * C::kCtas, kMaxCtas));
    // Items: at most the row tiles of the batch for each key head.  Where they are far fewer than the CTAs,
    // the cuts are that far apart, and a block of the join looks at several CTAs and gives a row four
    // warps; elsewhere it looks at one and gives a row one warp.
    const int64_t items = (static_cast<int64_t>(p.c.T) * p.G / R + p.c.B) * p.c.Hkv;
    const int64_t longest = (p.c.max_pages * p.c.page_blocks * kKvBlock + kTile - 1) / kTile;
    p.whole = longest + C::W::kItem <= C::W::kWhole && items <= ctas;
    const int group = static_cast<int>(std::clamp<int64_t>(ctas / (2 * items), 1, 16));
    const int share = group > 1 ? kJoinWarps : 1;
    const int rows = std::min(p.rows, p.slot_rows), per_block = kJoinWarps / share;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((ctas + group - 1) / group, (rows + per_block - 1) / per_block, 1);
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (launch_kernel(fp8kv_attention_kernel<R, ATOMS>, ctas, kThreads, C::kSmem, s, true, k, v,
                      p) != cudaSuccess) {
        cudaGetLastError();
        return BSP_ERR_CUDA;
    }
    if (!p.whole &&
        cudaLaunchKernelEx(&cfg, fp8kv_join_kernel<ATOMS>, p, static_cast<int>(ctas), group,
                           share) != cudaSuccess) {
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
    const int64_t rows = std::min<int64_t>(bsp::kMaxRows, T * (Hq / Hkv));
    return bsp::kMaxCtas * (static_cast<int64_t>(sizeof(bsp::Cut)) +
                            2 * rows * (D + 2) * static_cast<int64_t>(sizeof(float)));
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
    if (q_stride % 8 != 0 || pages * Hkv >= (int64_t{1} << 31)) return BSP_ERR_UNSUPPORTED_SHAPE;
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
    const double scale = sm_scale * 1.4426950408889634;
    if (std::isfinite(scale) && scale != 0.0 && std::fabs(scale) < 1.0) p.scale_exp = std::ilogb(scale);
    p.scale_log2 = static_cast<float>(std::ldexp(scale, -p.scale_exp));
    p.window = window > (int64_t{1} << 30) ? 0 : static_cast<int32_t>(window);
    p.G = static_cast<int32_t>(Hq / Hkv);
    p.cuts = static_cast<Cut*>(workspace);
    p.parts = reinterpret_cast<float*>(p.cuts + kMaxCtas);
    p.slot_rows = static_cast<int32_t>(std::min<int64_t>(kMaxRows, T * p.G));
    p.box = 16;
    while (p.box < kTile && page_size % (2 * p.box) == 0) p.box *= 2;
    p.stop_loads = load_stall();
    p.wait_ns = wait_limit_ns();
    p.status = device_status_ptr(dev);
    CUtensorMap tk, tv;
    st = make_page_map(&tk, k_cache, D, page_size, pages * Hkv, p.box);
    if (st != BSP_OK) return st;
    st = make_page_map(&tv, v_cache, D, page_size, pages * Hkv, p.box);
    if (st != BSP_OK) return st;
    // Rows of a row tile: 8 when the average sequence has no more, else 16.  (56 rows of each of 17
    // sequences: 80 us with 16, 99 with 8, which reads the cache from L2 more often, and 115 with 32, which
    // leaves an SM one CTA and nothing to hide its latencies behind.)
    const int64_t rows = p.G * ((T + B - 1) / B);
    p.rows = rows <= 8 ? 8 : 16;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (D <= 128)
        return p.rows == 8 ? launch_attention<8, 1>(p, tk, tv, dev, sms, s)
                           : launch_attention<16, 1>(p, tk, tv, dev, sms, s);
    return p.rows == 8 ? launch_attention<8, 2>(p, tk, tv, dev, sms, s)
                       : launch_attention<16, 2>(p, tk, tv, dev, sms, s);
}

}  // extern "C"
