// fp8kv_append.cu -- rotary positions on the new tokens' q and k, then k and v into the paged
// block-scaled E4M3 cache, in one launch.
//
//   theta(p, j) = p * inv_freq[j], (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin) * rope_scale
//   block of 16 tokens and head: e = max(e_old, ceil(log2(amax / 448))), code = E4M3(x * 2^-e)
//
// The work is memory traffic: q is read and written once in bf16, k and v are read once and
// leave a quarter or half as many bytes.  One CTA takes one unit, the part of a sequence's
// 16-token block that is new, and some of the heads; one warp takes one head of it, holds the
// block in registers (amax and encode need no second read) and owns the block's scale, so no
// atomics are needed.  The angles are the same for every head: the CTA makes them once, in
// shared memory.  They are multiplied and reduced to half a turn in 64 bits (a position near
// 2^20 times an fp32 frequency leaves few correct digits of the angle in 32), then sincospif.
// 12300 tokens of 32 + 8 + 8 heads of 128: 59 us (4.3 TB/s): a warp's loads, the CTA's angles, the rotation
// and the stores come one after the other, and two or three CTAs on an SM hide that in part; one token 4.8
// us, 192 sequences of one token 7.9 us, bound by the chain of launch, batch, angles, store.
#include <cuda_bf16.h>

#include <algorithm>

#include "fp8kv_common.cuh"

namespace bsp {
namespace {

struct AppendParams {
    KvCache c;
    const __nv_bfloat16* q;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    __nv_bfloat16* q_out;
    int64_t q_stride, k_stride, v_stride;
    const float* inv_freq;
    int32_t rot;
    int32_t per;                     // units: see find_unit
    int32_t extra;
    int32_t interleaved;
    // floor(2^16 / n) + 1 for the n slots of a token that are rotated and the n that are not: times i,
    // and shifted, it is floor(i / n), since i * n <= 256 * 16 < 2^16
    int32_t by_rot, by_rest;
    float rope_scale;
    int* status;
};

constexpr int kAppendThreads = 256;

// A lane's 16 elements of one token as loaded.
struct Raw {
    uint4 a, b;
};

__device__ __forceinline__ void unpack(const Raw& w, float (&x)[16])
{
    const uint32_t u[8] = {w.a.x, w.a.y, w.a.z, w.a.w, w.b.x, w.b.y, w.b.z, w.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = bf16lo_to_f32(u[i]);
        x[2 * i + 1] = bf16hi_to_f32(u[i]);
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&b);
}

// One lane's 16 elements of one token: two groups of 8 at element offsets o1, o2, and the slot's place
// among the token's rotated ones (-1: not rotated).  The rotated slots of all tokens come first, so
// that a warp's slots are all of one kind, or nearly.
// All of it is in one register; 0 stands for a slot that is not there or not new.
struct Slot {
    uint32_t bits;
    __device__ bool there() const { return bits != 0; }
    __device__ int token() const { return bits & 15u; }
    __device__ int c() const { return bits >> 4 & 15u; }
    __device__ int o1() const { return bits >> 5 & 0xF8u; }
    __device__ int o2() const { return bits >> 10 & 0xF8u; }
    __device__ bool rotated() const { return bits & 1u << 18; }
};

__device__ __forceinline__ Slot slot_of(const AppendParams& p, int s, int per_token)
{
    const int rs = p.rot >> 4, turned = kKvBlock * rs;
    const bool rotated = s < turned;
    const int of = rotated ? rs : per_token - rs, i = rotated ? s : s - turned;
    const int token = i * (rotated ? p.by_rot : p.by_rest) >> 16;                 // i / of
    const int c = i - token * of + (rotated ? 0 : rs);
    // of 8 elements each
    const int o1 = rotated && !p.interleaved ? c : 2 * c;
    const int o2 = rotated && !p.interleaved ? c + (p.rot >> 4) : 2 * c + 1;
    return {static_cast<uint32_t>(token | c << 4 | o1 << 8 | o2 << 13 | (rotated ? 1 << 18 : 0) |
                                  1 << 19)};
}

// cos and sin of pairs 2 i and 2 i + 1 (of 8) of slot c of a token, as (cos, cos, sin, sin):
// [4][16 tokens][rot / 16], so that the lanes of a warp, whose slots are neighbours, read neighbouring
// words.
__device__ __forceinline__ int angle_at(const AppendParams& p, int token, int c, int i)
{
    return (i * kKvBlock + token) * (p.rot >> 4) + c;
}

// Two fp32 at a time.  Products and sums are kept apart (no contraction), so the result does not
// depend on which of the two products a compiler fuses.
struct Pair {
    float a, b;
};

__device__ __forceinline__ Pair mul2(Pair x, Pair y)
{
    Pair d;
    asm("{\n\t.reg .b64 x, y, d;\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 d, x, y;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.a), "=f"(d.b)
        : "f"(x.a), "f"(x.b), "f"(y.a), "f"(y.b));
    return d;
}

__device__ __forceinline__ Pair add2(Pair x, Pair y)
{
    Pair d;
    asm("{\n\t.reg .b64 x, y, d;\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 d, x, y;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.a), "=f"(d.b)
        : "f"(x.a), "f"(x.b), "f"(y.a), "f"(y.b));
    return d;
}

__device__ __forceinline__ void turn(float4 t, float& x1a, float& x1b, float& x2a, float& x2b)
{
    const Pair x1 = {x1a, x1b}, x2 = {x2a, x2b}, c = {t.x, t.y}, s = {t.z, t.w}, n = {-t.z, -t.w};
    const Pair r1 = add2(mul2(x1, c), mul2(x2, n)), r2 = add2(mul2(x2, c), mul2(x1, s));
    x1a = r1.a;
    x1b = r1.b;
    x2a = r2.a;
    x2b = r2.b;
}

// The largest magnitude, of two elements at a time; a NaN keeps no say in it.
__device__ __forceinline__ float largest(const Raw& w)
{
    const uint32_t u[8] = {w.a.x, w.a.y, w.a.z, w.a.w, w.b.x, w.b.y, w.b.z, w.b.w};
    __nv_bfloat162 m = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u[i])));
    return fmaxf(__low2float(m), __high2float(m));
}

__device__ __forceinline__ void rotate(const AppendParams& p, const Slot& s, const float4* cs,
                                       float (&x)[16])
{
    const float4* t = cs + angle_at(p, s.token(), s.c(), 0);
    const int step = kKvBlock * (p.rot >> 4);
    if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) turn(t[i * step], x[4 * i], x[4 * i + 2], x[4 * i + 1], x[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) turn(t[i * step], x[2 * i], x[2 * i + 1], x[2 * i + 8], x[2 * i + 9]);
    }
}

// Where a task (one head's q, k or v of the unit) reads.
struct Task {
    const __nv_bfloat16* src;        // token 0 of the block
    int64_t stride;
    int h;
    bool is_q, is_k;
};

__device__ __forceinline__ Task task_of(const AppendParams& p, int task, int64_t row0)
{
    const int nq = p.q ? p.c.Hq : 0;
    Task t;
    t.is_q = task < nq;
    t.is_k = !t.is_q && task < nq + p.c.Hkv;
    t.h = t.is_q ? task : (t.is_k ? task - nq : task - nq - p.c.Hkv);
    t.stride = t.is_q ? p.q_stride : (t.is_k ? p.k_stride : p.v_stride);
    t.src = (t.is_q ? p.q : (t.is_k ? p.k : p.v)) + row0 * t.stride + static_cast<int64_t>(t.h) * p.c.D;
    return t;
}

// Units: sequence b's begin at floor(cu_new[b] * per / 16) + extra * b.  With per = 1, extra = 2 they are
// its blocks, of which it touches at most floor(n / 16) + 2; with per = 16, extra = 0 they are its
// tokens, of which the first of each block does the block's work.  The host takes the fewer.
// The sequence whose units contain unit u is found by all threads at once, one load and one barrier for
// 256 sequences, not a chain of dependent loads.  More sequences are first narrowed down to that many, by
// a 256th at a time (the beginnings ascend with cu_new; whatever it holds, the result is looked at again):
// every CTA does this, so looking at all of 2^20 sequences in each would take minutes.
struct Unit {
    int64_t begin;               // the sequence's first unit
    int32_t b, first, n, len;
};

__device__ __forceinline__ bool find_unit(const AppendParams& p, int64_t u, Unit& unit)
{
    __shared__ Unit found;
    const KvCache& c = p.c;
    if (threadIdx.x == 0) found.b = -1;
    __syncthreads();
    int from = 0, to = c.B;
    while (to - from > kAppendThreads) {
        const int step = (to - from + kAppendThreads - 1) / kAppendThreads;
        const int at = from + static_cast<int>(threadIdx.x) * step;
        const bool before =
            at < to && static_cast<int64_t>(kv_clamp_row(c.cu_new[at], c.T)) * p.per / kKvBlock +
                               static_cast<int64_t>(p.extra) * at <=
                           u;
        from += max(__syncthreads_count(before) - 1, 0) * step;
        to = min(to, from + step);
    }
    const int i = from + static_cast<int>(threadIdx.x);
    if (i < to) {
        const KvRows r = kv_rows(c, i);
        const int32_t len = c.kv_len[i];
        const int64_t at = static_cast<int64_t>(r.first) * p.per / kKvBlock +
                           static_cast<int64_t>(p.extra) * i;
        const int64_t next = static_cast<int64_t>(r.first + r.n) * p.per / kKvBlock +
                             static_cast<int64_t>(p.extra) * (i + 1);
        // one sequence at most, unless cu_new descends: then whichever comes first, all of it
        if (at <= u && u < next && atomicCAS(&found.b, -1, i) == -1) {
            found.begin = at;
            found.first = r.first;
            found.n = r.n;
            found.len = len;
        }
    }
    __syncthreads();
    unit = found;
    return unit.b >= 0;
}

// NS: slots of one lane in a block (ceil(D / 32) rounded up to a power of two).  A warp's loads of its
// first task are on their way while the CTA makes the angles; they stay as loaded (8 registers a
// slot), and are rotated again for the second pass over them, rather than held in fp32.
template <int NS>
__global__ void __launch_bounds__(kAppendThreads, NS <= 4 ? 3 : 2)
    fp8kv_append_kernel(const AppendParams p)
{
    extern __shared__ float4 cs[];                       // see angle_at
    const KvCache& c = p.c;
    griddep_wait();
    griddep_launch_dependents();

    Unit unit;
    const int64_t u = blockIdx.x;
    if (!find_unit(p, u, unit)) return;
    // Units counted by block leave room for a sequence that brings nothing, too.  Neither its length nor
    // its row of the table is looked at: they may be stale, and the row's pages another sequence's by now.
    if (unit.n == 0) return;
    const int b = unit.b;
    const int32_t len = unit.len;
    if (len < unit.n || len > kv_capacity(c)) {
        if (u == unit.begin && blockIdx.y == 0 && threadIdx.x == 0) kv_report_bad_batch(p.status);
        return;
    }
    const int32_t start = len - unit.n;                  // position of the first new token
    const int64_t off = u - unit.begin;
    if (p.per != 1 && off > 0 && (start + off) % kKvBlock != 0) return;    // not a block's first token
    const int64_t block = p.per == 1 ? start / kKvBlock + off : (start + off) / kKvBlock;
    const int64_t pos0 = block * kKvBlock;
    if (pos0 >= len) return;
    const int lo = start > pos0 ? static_cast<int>(start - pos0) : 0;     // new: [lo, hi)
    const int hi = len - pos0 < kKvBlock ? static_cast<int>(len - pos0) : kKvBlock;
    const int64_t row0 = unit.first + (pos0 - start);    // row of the block's token 0

    const int lane = threadIdx.x & 31;
    const int per_token = c.D >> 4;
    const int slots = kKvBlock * per_token;
    const int tasks = (p.q ? c.Hq : 0) + 2 * c.Hkv;
    const int stride = gridDim.y * (kAppendThreads / 32);
    int task = blockIdx.y * (kAppendThreads / 32) + (threadIdx.x >> 5);

    // the lane's slots, the same for every task
    Slot slot[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int s = lane + 32 * i;
        slot[i].bits = 0;
        if (s >= slots) continue;
        const Slot w = slot_of(p, s, per_token);
        if (w.token() >= lo && w.token() < hi) slot[i] = w;
    }
    Raw raw[NS];
    const auto load = [&](const Task& t) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const Slot& w = slot[i];
            if (!w.there()) continue;
            const __nv_bfloat16* row = t.src + w.token() * t.stride;
            raw[i].a = *reinterpret_cast<const uint4*>(row + w.o1());
            raw[i].b = *reinterpret_cast<const uint4*>(row + w.o2());
        }
    };
    if (task < tasks) load(task_of(p, task, row0));
    const int32_t page = c.table[static_cast<int64_t>(b) * c.max_pages + block / c.page_blocks];

    const int half = p.rot >> 1;
    for (int i = threadIdx.x; i < kKvBlock * half; i += kAppendThreads) {
        const int t = i / half, j = i - t * half;
        if (t < lo || t >= hi) continue;
        const double x = static_cast<double>(pos0 + t) * static_cast<double>(p.inv_freq[j]);
        const double turns = x * 0.15915494309189535;                    // 1 / (2 pi)
        float sn, cn;
        sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &sn, &cn);
        // frequency j belongs to pair j % 8 of slot j / 8
        float* at = reinterpret_cast<float*>(cs + angle_at(p, t, j >> 3, (j & 7) >> 1)) + (j & 1);
        at[0] = __fmul_rn(cn, p.rope_scale);
        at[2] = __fmul_rn(sn, p.rope_scale);
    }
    __syncthreads();

    const bool page_ok = page >= 0 && page < c.pages;
    if (!page_ok && blockIdx.y == 0 && threadIdx.x == 0) kv_report_bad_batch(p.status);

    for (bool first = true; task < tasks; task += stride, first = false) {
        const Task t = task_of(p, task, row0);
        if (!t.is_q && !page_ok) continue;
        if (!first) load(t);
        if (t.is_q) {
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const Slot& w = slot[i];
                if (!w.there()) continue;
                Raw y = raw[i];
                if (w.rotated()) {
                    float x[16];
                    unpack(y, x);
                    rotate(p, w, cs, x);
                    y.a = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]),
                                     pack2(x[6], x[7]));
                    y.b = make_uint4(pack2(x[8], x[9]), pack2(x[10], x[11]), pack2(x[12], x[13]),
                                     pack2(x[14], x[15]));
                }
                __nv_bfloat16* out = p.q_out + ((row0 + w.token()) * c.Hq + t.h) * c.D;
                *reinterpret_cast<uint4*>(out + w.o1()) = y.a;
                *reinterpret_cast<uint4*>(out + w.o2()) = y.b;
            }
            continue;
        }
        float top = 0.0f;                                // a NaN keeps no say in the scale
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const Slot& w = slot[i];
            if (!w.there()) continue;
            if (t.is_k && w.rotated()) {
                float x[16];
                unpack(raw[i], x);
                rotate(p, w, cs, x);
#pragma unroll
                for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(x[j]));
            } else {
                top = fmaxf(top, largest(raw[i]));
            }
        }
        const uint32_t amax = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top));
        const int64_t group = static_cast<int64_t>(page) * c.Hkv + t.h;
        const int in_page = static_cast<int>(block % c.page_blocks);
        uint8_t* scale = (t.is_k ? c.k_scale : c.v_scale) + group * c.page_blocks + in_page;
        uint8_t* codes =
            (t.is_k ? c.k : c.v) + (group * c.page_blocks + in_page) * kKvBlock * c.D;
        int e = kv_scale_exp(amax);
        if (lo > 0) {                                    // the block holds earlier tokens
            const int old = *scale;
            if (e > old) {
                const int d = e - old;                   // their codes times 2^-d, rounded once
                const float f = d < 126 ? kv_pow2(127 - d) : 0.0f;
                for (int i = lane; i < lo * c.D / 4; i += 32) {
                    uint32_t* at = reinterpret_cast<uint32_t*>(codes) + i;
                    uint32_t a, d2;
                    e4m3x4_to_f16(*at, a, d2);
                    float y0, y1, y2, y3;
                    f16x2_to_f32(a, y0, y1);
                    f16x2_to_f32(d2, y2, y3);
                    *at = cvt_e4m3x2(y0 * f, y1 * f) | cvt_e4m3x2(y2 * f, y3 * f) << 16;
                }
            }
            e = max(e, old);
        }
        __syncwarp();
        if (lane == 0) *scale = static_cast<uint8_t>(e);
        const float f = kv_pow2_low(254 - e);            // 2^(127 - e), a normal number for every e made here
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const Slot& w = slot[i];
            if (!w.there()) continue;
            float x[16];
            unpack(raw[i], x);
            if (t.is_k && w.rotated()) rotate(p, w, cs, x);
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[j] = cvt_e4m3x2(x[4 * j] * f, x[4 * j + 1] * f) |
                       cvt_e4m3x2(x[4 * j + 2] * f, x[4 * j + 3] * f) << 16;
            uint8_t* out = codes + w.token() * c.D;
            *reinterpret_cast<uint2*>(out + w.o1()) = make_uint2(o[0], o[1]);
            *reinterpret_cast<uint2*>(out + w.o2()) = make_uint2(o[2], o[3]);
        }
    }
}

}  // namespace

int kv_check_cache(KvCache& c, const void* k_cache, const void* v_cache, const void* k_scale,
                   const void* v_scale, int64_t pages, int64_t page_size, const int32_t* table,
                   int64_t max_pages, const int32_t* cu_new, const int32_t* kv_len, int64_t B,
                   int64_t T, int64_t Hq, int64_t Hkv, int64_t D)
{
    if (B < 0 || T < 0 || Hq < 0 || Hkv <= 0 || D <= 0 || pages < 0 || max_pages < 0 ||
        page_size <= 0)
        return BSP_ERR_INVALID_ARG;
    constexpr int64_t kMost = int64_t{1} << 30;
    if (D % 16 != 0 || D > 256 || page_size % kKvBlock != 0 || page_size > 4096 ||
        Hq % Hkv != 0 || Hkv > 4096 || Hq > 4096 || B > (1 << 20) || T > kMost / 64 ||
        pages > kMost || max_pages > kMost / page_size || T * Hq > kMost)
        return BSP_ERR_UNSUPPORTED_SHAPE;
    c.k = static_cast<uint8_t*>(const_cast<void*>(k_cache));
    c.v = static_cast<uint8_t*>(const_cast<void*>(v_cache));
    c.k_scale = static_cast<uint8_t*>(const_cast<void*>(k_scale));
    c.v_scale = static_cast<uint8_t*>(const_cast<void*>(v_scale));
    c.table = table;
    c.cu_new = cu_new;
    c.kv_len = kv_len;
    c.max_pages = max_pages;
    c.pages = static_cast<int32_t>(pages);
    c.page_blocks = static_cast<int32_t>(page_size / kKvBlock);
    c.B = static_cast<int32_t>(B);
    c.T = static_cast<int32_t>(T);
    c.Hq = static_cast<int32_t>(Hq);
    c.Hkv = static_cast<int32_t>(Hkv);
    c.D = static_cast<int32_t>(D);
    return BSP_OK;
}

int kv_check_pointers(const KvCache& c)
{
    if (!c.k || !c.v || !c.k_scale || !c.v_scale || !c.table || !c.cu_new || !c.kv_len)
        return BSP_ERR_INVALID_ARG;
    const auto a4 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; };
    if (!aligned16(c.k) || !aligned16(c.v) || !a4(c.table) || !a4(c.cu_new) || !a4(c.kv_len))
        return BSP_ERR_MISALIGNED;
    return BSP_OK;
}

}  // namespace bsp

extern "C" int fp8kv_append(const void* q_bf16, int64_t q_stride, const void* k_bf16,
                            int64_t k_stride, const void* v_bf16, int64_t v_stride,
                            const float* inv_freq, int64_t rot, int interleaved, float rope_scale,
                            void* q_out_bf16, uint8_t* k_cache, uint8_t* v_cache,
                            uint8_t* k_scale, uint8_t* v_scale, int64_t pages, int64_t page_size,
                            const int32_t* block_table, int64_t max_pages, const int32_t* cu_new,
                            const int32_t* kv_len, int64_t B, int64_t T, int64_t Hq, int64_t Hkv,
                            int64_t D, bsp_stream_t stream)
{
    using namespace bsp;
    AppendParams p = {};
    int st = kv_check_cache(p.c, k_cache, v_cache, k_scale, v_scale, pages, page_size, block_table,
                            max_pages, cu_new, kv_len, B, T, Hq, Hkv, D);
    if (st != BSP_OK) return st;
    if (rot < 0 || (interleaved != 0 && interleaved != 1)) return BSP_ERR_INVALID_ARG;
    if (rot % 16 != 0 || rot > D) return BSP_ERR_UNSUPPORTED_SHAPE;
    if (T == 0 || B == 0) return BSP_OK;
    if (!k_bf16 || !v_bf16 || (rot > 0 && !inv_freq) || (q_bf16 && (!q_out_bf16 || Hq == 0)))
        return BSP_ERR_INVALID_ARG;
    if (k_stride < Hkv * D || v_stride < Hkv * D || (q_bf16 && q_stride < Hq * D))
        return BSP_ERR_INVALID_ARG;
    if (k_stride % 8 != 0 || v_stride % 8 != 0 || (q_bf16 && q_stride % 8 != 0))
        return BSP_ERR_UNSUPPORTED_SHAPE;
    if (pages == 0 || max_pages == 0) return BSP_ERR_INVALID_ARG;
    st = kv_check_pointers(p.c);
    if (st != BSP_OK) return st;
    if (!aligned16(q_bf16) || !aligned16(k_bf16) || !aligned16(v_bf16) || !aligned16(q_out_bf16) ||
        (reinterpret_cast<uintptr_t>(inv_freq) & 3u))
        return BSP_ERR_MISALIGNED;
    int dev = 0, sms = 0;
    st = check_device(&dev, &sms);
    if (st != BSP_OK) return st;
    p.q = static_cast<const __nv_bfloat16*>(q_bf16);
    p.k = static_cast<const __nv_bfloat16*>(k_bf16);
    p.v = static_cast<const __nv_bfloat16*>(v_bf16);
    p.q_out = static_cast<__nv_bfloat16*>(q_out_bf16);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.inv_freq = inv_freq;
    p.rot = static_cast<int32_t>(rot);
    p.interleaved = interleaved;
    p.by_rot = rot ? static_cast<int32_t>(65536 / (rot / 16) + 1) : 0;
    p.by_rest = D > rot ? static_cast<int32_t>(65536 / ((D - rot) / 16) + 1) : 0;
    p.rope_scale = rope_scale;
    p.status = device_status_ptr(dev);

    const bool by_token = T < T / kKvBlock + 2 * B;
    p.per = by_token ? kKvBlock : 1;
    p.extra = by_token ? 0 : 2;
    const int64_t units = by_token ? T : T / kKvBlock + 2 * B;
    const int64_t tasks = (q_bf16 ? Hq : 0) + 2 * Hkv;
    constexpr int kWarps = kAppendThreads / 32;
    // CTAs to a unit.  A warp takes one task where all CTAs are resident then, or where there is more than
    // a wave of units anyway (58, 60 and 65 us with one, two and three tasks for 12300 tokens of 48
    // heads); in between, as many CTAs as still make one wave, but no more than three tasks a warp
    // (12.3, 10.1 and 8.6 us with one, two and three for 192 sequences of one token).
    int64_t groups = (tasks + kWarps - 1) / kWarps;
    const int64_t wave = 3 * static_cast<int64_t>(sms);
    if (units <= wave) groups = std::min(groups, std::max(wave / units, (groups + 2) / 3));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(units), static_cast<unsigned>(groups), 1);
    cfg.blockDim = dim3(kAppendThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(kKvBlock) * (rot / 2) * sizeof(float2);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (D <= 64)
        e = cudaLaunchKernelEx(&cfg, fp8kv_append_kernel<2>, p);
    else if (D <= 128)
        e = cudaLaunchKernelEx(&cfg, fp8kv_append_kernel<4>, p);
    else
        e = cudaLaunchKernelEx(&cfg, fp8kv_append_kernel<8>, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return BSP_ERR_CUDA;
    }
    return launch_status();
}
