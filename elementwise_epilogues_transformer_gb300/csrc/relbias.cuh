// relbias.cuh -- what the forward and the backward of the relative-position-
// bias softmax share: the bucket function and its window in shared memory,
// rows and chunks, scores, keep flags, and the host's argument checks and
// launch plan.  See relbias_fwd.cu for the operation and the layout.
#pragma once

#include <cmath>
#include <type_traits>

#include "mfx_device.cuh"
#include "mfx_host.h"

namespace mfx {
namespace relbias {

constexpr int kTeam = 256;            // threads per row where rows are not long
constexpr int kLongTeam = 512;        // ... where they are
constexpr int kSmallBlock = 128;      // threads of a block whose teams are a warp or less (and the largest of kernels for teams of part of a warp)
constexpr int kMaxBuckets = 256;      // buckets of a table
constexpr int kMaxSide = 128;         // buckets of one direction
constexpr int kMaxDistance = 2048;    // keeps the window and one set of its sums (at most 183 KB) within a block's shared memory
constexpr int kMaxCluster = 8;        // blocks that may share a row
constexpr int kBwdBlocksPerSm = 16;   // most blocks of a backward grid per SM (what its workspace goes by)
constexpr float kLog2eF = 1.4426950408889634f;

// The bucket function of one direction: distances below `first` have a bucket
// each, bucket first + 1 + j begins at border[j], and `reach` is where the
// last one begins.
struct Buckets {
    int num, side, first, reach, hi;  // hi: first position right of the query whose bias no longer changes
    int border[kMaxSide];
};

struct Geom {
    int sq, sk, np;
    int rows;                  // b * sq: rows of one head
    int64_t total, mask_total; // elements of the tensor and of the mask
    int64_t mask_b, mask_np, mask_sq;  // strides of the mask in elements (0 = broadcast)
    int q_start;
    const int32_t* seq_start;  // per batch, or null
    int slices;                // blocks (clusters) per head
    int step, step_i, step_q;  // rows, batches and queries from one row of a team to its next
    int64_t step_r, wrap_r;    // rows of the tensor with that, and more where a batch ends
    int team, teams, cluster;  // threads per row, rows per block, blocks per row
    int blocks;                // register blocks that a row takes
    int causal, table_bf16;
    int exact;                 // a row is exactly the chunks that its threads hold
    int drop;                  // p > 0
    int phase0;                // (phase0 + element index) mod 8 = 0 at a chunk's start
    float scale, scale2;       // the score scale; the same times log2 e
    float keep_scale;          // 1 / (1 - p)
    // backward: a row's gradient is formed times fold, the score scale where
    // that is a normal number (1 else); grad = keep_scale * fold, unfold =
    // 1 / fold, post = scale / fold
    float grad, unfold, post;
    uint32_t thresh_hi;        // keep threshold in the upper half-word
    uint64_t elem_base;
    MaskGen gen;
};

// The window holds the bias (times log2 e) of the positions around the query:
// entry i is the one at k - pos = i - reach, -8 <= i <= reach + hi + 8, the
// ones past either end repeating the far values.  A chunk of 8 begins at any
// entry, so each entry is stored with the three after it as one 16-byte
// vector and a chunk is two of them; entries lie by residue mod 8 first, so
// that the lanes of a warp, whose chunks are 8 entries apart, read
// consecutive vectors.
__device__ __host__ __forceinline__ int window_stride(const Buckets& w) { return ((w.reach + w.hi + 16) >> 3) + 1; }
__device__ __forceinline__ int window_slot(int stride, int i)
{
    const int u = i + 8;
    return (u & 7) * stride + (u >> 3);
}
inline size_t window_bytes(const Buckets& w) { return (size_t)8 * window_stride(w) * sizeof(float4); }

__device__ __forceinline__ int side_bucket(const Buckets& w, int n)
{
    if (n < w.first)
        return n;
    int lo = 0, hi = w.side - w.first - 1;  // borders not above n
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (w.border[mid] <= n)
            lo = mid + 1;
        else
            hi = mid;
    }
    return w.first + lo;
}

// First distance of bucket v of a direction (v = side: past the window).
__device__ __forceinline__ int side_start(const Buckets& w, int v)
{
    return v <= w.first ? v : v >= w.side ? w.reach + 1 : w.border[v - w.first - 1];
}

// The bias of head h at window entry i, times log2 e.
__device__ __forceinline__ float window_bias(const Buckets& w, const Geom& g, const void* table, int h, int i)
{
    if (!table)
        return 0.0f;
    const int last = w.reach + w.hi, rel = (i < 0 ? 0 : i > last ? last : i) - w.reach;
    const int u = rel <= 0 ? side_bucket(w, -rel) : side_bucket(w, rel) + w.side;
    const int64_t at = (int64_t)u * g.np + h;
    return kLog2eF * (g.table_bf16 ? load1(static_cast<const bf16*>(table) + at)
                                   : load1(static_cast<const float*>(table) + at));
}

// Fills the block's window for head h (call with all threads, then meet).
// Each value is looked up once and put in the up to four vectors it is part of.
__device__ __forceinline__ void fill_window(const Buckets& w, const Geom& g, const void* table, int h, float4* win)
{
    const int last = w.reach + w.hi, stride = window_stride(w);
    float* f = reinterpret_cast<float*>(win);
    for (int i = (int)threadIdx.x - 8; i <= last + 11; i += blockDim.x) {
        const float v = window_bias(w, g, table, h, i);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i - k >= -8 && i - k <= last + 8)
                f[4 * window_slot(stride, i - k) + k] = v;
    }
}

// 2^t by the hardware exponential (2 ulp); results below 2^-126 flush to zero.
__device__ __forceinline__ float exp2_of(float t)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
    return r;
}

// (Pairs are for the layout only: the two-lane instructions measured slower
// here, 0.104 against 0.094 ms for a 2x8x2048x2048 forward.)
__device__ __forceinline__ float2 pfma(float2 a, float2 b, float2 c)
{
    return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y));
}
__device__ __forceinline__ float2 padd(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ float2 pmul(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }

// Eight elements as four pairs.
__device__ __forceinline__ void pairs_of(const Raw8<bf16>& r, float2 (&f)[4])
{
    f[0] = widen2(r.v.x), f[1] = widen2(r.v.y), f[2] = widen2(r.v.z), f[3] = widen2(r.v.w);
}
__device__ __forceinline__ void pairs_of(const Raw8<float>& r, float2 (&f)[4])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        f[2 * h] = make_float2(__uint_as_float(r.v[h].x), __uint_as_float(r.v[h].y));
        f[2 * h + 1] = make_float2(__uint_as_float(r.v[h].z), __uint_as_float(r.v[h].w));
    }
}
__device__ __forceinline__ void narrow_pairs(const float2 (&f)[4], Raw8<bf16>& r)
{
    r.v = make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                     pack_bf16x2(f[3].x, f[3].y));
}
__device__ __forceinline__ void narrow_pairs(const float2 (&f)[4], Raw8<float>& r)
{
#pragma unroll
    for (int h = 0; h < 2; ++h)
        r.v[h] = make_uint4(__float_as_uint(f[2 * h].x), __float_as_uint(f[2 * h].y),
                            __float_as_uint(f[2 * h + 1].x), __float_as_uint(f[2 * h + 1].y));
}

// Three-operand maximum and minimum (NaN operands are passed over).
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float min3(float a, float b, float c)
{
    float d;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max_of(float t, const float2 (&f)[4])
{
    return max3(max3(t, f[0].x, f[0].y), max3(f[1].x, f[1].y, f[2].x), max3(f[2].y, f[3].x, f[3].y));
}
__device__ __forceinline__ float min_of(const float2 (&f)[4])
{
    return min3(min3(f[0].x, f[0].y, f[1].x), min3(f[1].y, f[2].x, f[2].y), fminf(f[3].x, f[3].y));
}

// A branch that stays one: a loop that runs once where c, because the compiler
// turns a short if into predicated instructions that every chunk pays for
// (measured: 4 of 28 instructions an element, without a chunk that needs it).
__device__ __forceinline__ int done_once()
{
    int v;
    asm volatile("mov.u32 %0, 0;" : "=r"(v));
    return v;
}
#define MFX_RARELY(c) _Pragma("unroll 1") for (int todo_ = (c) ? 1 : 0; todo_; todo_ = done_once())

// Sets the elements of a chunk outside [0, end) to v.
__device__ __forceinline__ void fill_outside(float2 (&f)[4], int k0, int end, float v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i].x = k0 + 2 * i >= 0 && k0 + 2 * i < end ? f[i].x : v;
        f[i].y = k0 + 2 * i + 1 >= 0 && k0 + 2 * i + 1 < end ? f[i].y : v;
    }
}

// Elements [k0, k0 + 8) of a row, of which [0, end) are wanted.  FAST: the row
// is whole chunks of 16-byte vectors.  Otherwise a chunk is read as vectors
// where they are aligned and either the row has all of it or (`inner`) the
// tensor does: what stands outside the row is the neighbours' then, and the
// caller does not use it.  Chunks at a tensor's ends, and ones that are not
// aligned, are read element by element, zero where there is none.
template <typename T>
__device__ __noinline__ void load_ragged(const T* p, int k0, int end, Raw8<T>* raw)
{
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        f[j] = k0 + j >= 0 && k0 + j < end ? load1(p + j) : 0.0f;
    narrow8(f, *raw);
}

template <typename T, bool FAST>
__device__ __forceinline__ void load_chunk(const T* p, int k0, int end, bool inner, Raw8<T>& raw)
{
    if constexpr (FAST) {
        ld8(p, raw);
    } else {
        raw = Raw8<T>{};
        if (k0 < end) {
            if ((inner || (k0 >= 0 && k0 + 8 <= end)) && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
                ld8(p, raw);
            } else {
                Raw8<T> r;
                load_ragged(p, k0, end, &r);
                raw = r;
            }
        }
    }
}

template <typename T, bool FAST>
__device__ __forceinline__ void store_chunk(T* p, int k0, int end, const float2 (&f)[4])
{
    if (FAST || (k0 >= 0 && k0 + 8 <= end && (reinterpret_cast<uintptr_t>(p) & 15u) == 0)) {
        Raw8<T> raw;
        narrow_pairs(f, raw);
        st8(p, raw);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k0 + j >= 0 && k0 + j < end)
                store1(p + j, j & 1 ? f[j >> 1].y : f[j >> 1].x);
    }
}

// A row, as little of it as says which it is (the backward keeps one ahead),
// and what its chunks share.
template <typename T>
struct Seat {
    int64_t r;      // row index of the tensor
    const T* mask;  // its mask row, where there is a mask
    int pos, end;   // clamped query position; keys that take part: [0, end)
};
template <typename T>
struct Row : Seat<T> {
    int64_t e0;       // element index of chunk 0 in the tensor
    uint64_t block0;  // generator block of chunk 0
    int a, chunks;    // chunk phase; chunks of the row
    bool inner, mask_inner;  // all of its chunks lie in the tensor, in the mask (not set where chunks are whole)
};

// The rows that a team walks, `row` of the b * sq of head h and every step-th
// from it, as batch, query and row of the tensor, advanced without divisions.
struct Walk {
    int64_t r;
    int row, i, q;
    __device__ __forceinline__ Walk(const Geom& g, int h, int first) : row(first), i(first / g.sq), q(first % g.sq)
    {
        r = first + i * g.wrap_r + (int64_t)h * g.sq;
    }
    __device__ __forceinline__ void next(const Geom& g)
    {
        row += g.step;
        i += g.step_i;
        q += g.step_q;
        r += g.step_r;
        if (q >= g.sq) {
            q -= g.sq;
            ++i;
            r += g.wrap_r;
        }
    }
    __device__ __forceinline__ bool live(const Geom& g) const { return row < g.rows; }
};

// A team without a row has one without keys, whose tensor row is 0 (chunks
// past a row's end are read at its start: of a row that exists).
template <typename T>
__device__ __forceinline__ Seat<T> seat_at(const Geom& g, const Buckets& w, const T* mask, int h, const Walk& at)
{
    Seat<T> o{0, mask, 0, 0};
    if (!at.live(g))
        return o;
    o.r = at.r;
    o.pos = g.q_start + at.q;
    if (g.seq_start) {
        const int64_t pos = (int64_t)o.pos + g.seq_start[at.i], lo = -w.reach - 1, hi = g.sk + w.reach;
        o.pos = (int)(pos < lo ? lo : pos > hi ? hi : pos);
    }
    o.end = g.causal ? (o.pos < 0 ? 0 : o.pos + 1 < g.sk ? o.pos + 1 : g.sk) : g.sk;
    if (mask)
        o.mask = mask + (at.i * g.mask_b + h * g.mask_np + at.q * g.mask_sq);
    return o;
}

template <typename T, bool FAST>
__device__ __forceinline__ Row<T> row_of(const Geom& g, const Seat<T>& seat, bool live, const T* mask)
{
    Row<T> o;
    static_cast<Seat<T>&>(o) = seat;
    const int64_t e = seat.r * (int64_t)g.sk;
    o.a = FAST ? 0 : (int)((uint64_t)(g.phase0 + e) & 7u);
    o.e0 = e - o.a;
    o.block0 = (g.elem_base + (uint64_t)e) >> 3;
    o.chunks = live ? (g.sk + o.a + 7) >> 3 : 0;
    if (!FAST) {
        const int64_t m0 = seat.mask - mask - o.a;
        o.inner = o.e0 >= 0 && o.e0 + 8 * o.chunks <= g.total;
        o.mask_inner = m0 >= 0 && m0 + 8 * o.chunks <= g.mask_total;
    }
    return o;
}

// Whether any position of the chunk whose first is `rel` from the query has a
// bias of its own (-reach - 7 < rel < hi).
__device__ __forceinline__ bool near_chunk(const Buckets& w, int rel)
{
    return (unsigned)(rel + w.reach + 6) < (unsigned)(w.reach + w.hi + 6);
}

// ---------------------------------------------------------------------------
// Staging: while a team works on one row, the chunks of its next row are on
// their way into shared memory, each thread's into slots of its own (so that
// waiting for its own copies is all it needs), one 16-byte vector a chunk.
// ---------------------------------------------------------------------------

__device__ __forceinline__ void copy16_async(uint4* dst, const void* src, bool there)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most N of this thread's committed groups are under way.
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Starts the copies of a row's chunks (those that take part; the others read as zero).
template <int C>
__device__ __forceinline__ void stage_row(uint4* stage, const bf16* src, const Seat<bf16>& o, int sk, int tid, int team)
{
    const bf16* row = src + o.r * (int64_t)sk;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int ch = tid + c * team;
        const bool there = ch * 8 < o.end;
        copy16_async(stage + c * blockDim.x, row + (there ? 8 * ch : 0), there);
    }
    copies_commit();
}

__device__ __forceinline__ void unstage(const uint4* stage, int c, Raw8<bf16>& raw) { raw.v = stage[c * blockDim.x]; }
__device__ __forceinline__ void restage(uint4* stage, int c, const Raw8<bf16>& raw) { stage[c * blockDim.x] = raw.v; }

// A mask's chunk, kept in L1: rows share it where the mask is broadcast.
__device__ __forceinline__ void ld8_cached(const bf16* p, Raw8<bf16>& r) { r.v = ld16_ca(p); }
__device__ __forceinline__ void ld8_cached(const float* p, Raw8<float>& r) { r.v[0] = ld16_ca(p), r.v[1] = ld16_ca(p + 4); }
template <typename T, bool FAST>
__device__ __forceinline__ void load_mask(const T* p, int k0, int end, bool inner, Raw8<T>& raw)
{
    if (FAST)
        ld8_cached(p, raw);
    else
        load_chunk<T, FAST>(p, k0, end, inner, raw);
}

// Whether a chunk of the mask is all zero (adds nothing) or all -inf (leaves
// nothing).
__device__ __forceinline__ bool all_zero(const Raw8<bf16>& r) { return (r.v.x | r.v.y | r.v.z | r.v.w) == 0u; }
__device__ __forceinline__ bool all_out(const Raw8<bf16>& r)
{
    constexpr uint32_t k = 0xFF80FF80u;
    return ((r.v.x ^ k) | (r.v.y ^ k) | (r.v.z ^ k) | (r.v.w ^ k)) == 0u;
}
__device__ __forceinline__ bool all_zero(const Raw8<float>& r)
{
    return (r.v[0].x | r.v[0].y | r.v[0].z | r.v[0].w | r.v[1].x | r.v[1].y | r.v[1].z | r.v[1].w) == 0u;
}
__device__ __forceinline__ bool all_out(const Raw8<float>& r)
{
    constexpr uint32_t k = 0xFF800000u;
    return ((r.v[0].x ^ k) | (r.v[0].y ^ k) | (r.v[0].z ^ k) | (r.v[0].w ^ k) | (r.v[1].x ^ k) | (r.v[1].y ^ k) |
            (r.v[1].z ^ k) | (r.v[1].w ^ k)) == 0u;
}

// Scores of the chunk at k0 from its raw x, times log2 e: x * scale + bias
// (+ mask - shift).  A key whose mask is -inf is left out whatever x holds there.
// Call with whole warps: one with a near chunk reads the window in all lanes,
// far ones at its ends, and a mask that is zero in all of them is not added.
// False, with nothing computed, where the mask leaves the warp no key at all.
template <typename T, bool FAST, bool MASK>
__device__ __forceinline__ bool score_chunk(const Raw8<T>& raw, const Row<T>& row, const Geom& g, const Buckets& w,
                                            const float4* win, float far_lo, float far_hi, int k0, bool masked,
                                            float shift, float2 (&s)[4])
{
    Raw8<T> mraw;
    bool add = false;
    if (MASK && masked) {  // the same for every lane, as the votes have to be
        load_mask<T, FAST>(row.mask + (FAST && k0 >= row.end ? 0 : k0), k0, row.end, row.mask_inner, mraw);
        add = __any_sync(0xFFFFFFFFu, !all_zero(mraw) || shift != 0.0f);
        if (add && __all_sync(0xFFFFFFFFu, all_out(mraw)))
            return false;
    }
    pairs_of(raw, s);
    const int rel = k0 - row.pos;
    if (!__any_sync(0xFFFFFFFFu, near_chunk(w, rel))) {
        const float2 b = f2(rel >= w.hi ? far_hi : far_lo);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s[i] = pfma(s[i], f2(g.scale2), b);
    } else {
        const int stride = window_stride(w), i0 = min(max(rel + w.reach, -8), w.reach + w.hi + 1);
        const float4 lo = win[window_slot(stride, i0)], hi = win[window_slot(stride, i0 + 4)];
        s[0] = pfma(s[0], f2(g.scale2), make_float2(lo.x, lo.y));
        s[1] = pfma(s[1], f2(g.scale2), make_float2(lo.z, lo.w));
        s[2] = pfma(s[2], f2(g.scale2), make_float2(hi.x, hi.y));
        s[3] = pfma(s[3], f2(g.scale2), make_float2(hi.z, hi.w));
    }
    if (MASK && add) {
        float2 m[4];
        pairs_of(mraw, m);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[i].x = m[i].x == -INFINITY ? -INFINITY : fmaf(m[i].x - shift, kLog2eF, s[i].x);
            s[i].y = m[i].y == -INFINITY ? -INFINITY : fmaf(m[i].y - shift, kLog2eF, s[i].y);
        }
    }
    return true;
}

// Which of a thread's chunks, in a row that may end inside them, the warp
// has to look at.
template <bool CHECK>
__device__ __forceinline__ bool some_part(int k0, int end)
{
    return !CHECK || __any_sync(0xFFFFFFFFu, k0 < end);
}

__device__ __forceinline__ uint4 one_block(const MaskGen& m, uint64_t j)
{
    uint4 c[1];
    mask_blocks<1>(m, j, 0, c);
    return c[0];
}

// Keep flags of a chunk applied to its values: 16-bit word j of the block
// belongs to element j.
__device__ __forceinline__ void drop_pairs(float2 (&v)[4], const uint4& blk, uint32_t thresh_hi)
{
    const uint32_t w[4] = {blk.x, blk.y, blk.z, blk.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i].x = (w[i] << 16) >= thresh_hi ? v[i].x : 0.0f;
        v[i].y = w[i] >= thresh_hi ? v[i].y : 0.0f;
    }
}
__device__ __forceinline__ void drop_raw(Raw8<bf16>& r, const uint4& blk, uint32_t thresh_hi)
{
    const uint32_t t2 = thresh_hi | (thresh_hi >> 16);
    r.v.x &= keep_bits2(blk.x, t2), r.v.y &= keep_bits2(blk.y, t2);
    r.v.z &= keep_bits2(blk.z, t2), r.v.w &= keep_bits2(blk.w, t2);
}
__device__ __forceinline__ void drop_raw(Raw8<float>& r, const uint4& blk, uint32_t thresh_hi)
{
    float2 f[4];
    pairs_of(r, f);
    drop_pairs(f, blk, thresh_hi);
    narrow_pairs(f, r);
}

// Reductions over the lanes of a team that share a warp: all 32, or (ANY) an
// aligned group of 8, 16 or 32.
template <bool ANY>
__device__ __forceinline__ float lanes_max(float v, int lanes)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (!ANY || o < lanes)
            v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}
template <bool ANY>
__device__ __forceinline__ float lanes_sum(float v, int lanes)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (!ANY || o < lanes)
            v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}
__device__ __forceinline__ float2 peer_pair(const float2* p, int rank)
{
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), d;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(d) : "memory");
    return v;
}

// (maximum, sum relative to it) of two parts of a row, in base-2 units.
__device__ __forceinline__ float2 join(float2 a, float2 b)
{
    const float m = fmaxf(a.x, b.x);
    if (m == -INFINITY)
        return make_float2(m, a.y + b.y);
    return make_float2(m, a.y * exp2_of(a.x - m) + b.y * exp2_of(b.x - m));
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
// Whether n^s * a^j >= b^j * a^s in whole numbers (all below 2^14, s and j at
// most 64): products of up to 128 factors of 14 bits in 32-bit words.
inline bool border_reached(int n, int s, int a, int b, int j)
{
    constexpr int kWords = 64;
    uint32_t l[kWords] = {1}, r[kWords] = {1};
    auto mul = [](uint32_t* v, uint32_t by) {
        uint64_t carry = 0;
        for (int i = 0; i < kWords; ++i) {
            carry += (uint64_t)v[i] * by;
            v[i] = (uint32_t)carry;
            carry >>= 32;
        }
    };
    for (int i = 0; i < s; ++i)
        mul(l, n), mul(r, a);
    for (int i = 0; i < j; ++i)
        mul(l, a), mul(r, b);
    for (int i = kWords - 1; i >= 0; --i)
        if (l[i] != r[i])
            return l[i] > r[i];
    return true;
}

// Bucket j past the first ones begins at the least n with
// steps * log(n / first) / log(far / first) >= j.  The logarithms decide where
// they are clearly between whole numbers, whole-number products where not.
inline bool make_buckets(int64_t num, int64_t far, bool bidirectional, Buckets* w)
{
    if (num == 0) {  // no bias: one window entry that stays zero
        *w = Buckets{};
        w->num = 0, w->side = 1, w->first = 1;
        return true;
    }
    if (num < 2 || num > kMaxBuckets || (bidirectional && num % 2))
        return false;
    const int side = (int)(bidirectional ? num / 2 : num), first = side / 2, steps = side - first;
    if (side < 2 || side > kMaxSide || far <= first || far > kMaxDistance)
        return false;
    struct Last {
        int num, far, two;
        Buckets w;
    };
    static thread_local Last last{0, 0, 0, {}};  // a model's calls share one bucket function
    if (last.num != (int)num || last.far != (int)far || last.two != (int)bidirectional) {
        Buckets& o = last.w;
        o = Buckets{};
        o.num = (int)num, o.side = side, o.first = first;
        for (int j = 1; j < steps; ++j) {
            const double t = first * std::pow((double)far / first, (double)j / steps);
            int n = (int)std::ceil(t);
            if (std::fabs(t - std::round(t)) < 1e-6 * t) {
                n = (int)std::round(t) - 1;
                while (!border_reached(n, steps, first, (int)far, j))
                    ++n;
            }
            o.border[j - 1] = n;
        }
        o.reach = steps > 1 ? o.border[steps - 2] : first;
        o.hi = bidirectional ? o.reach : 0;
        last.num = (int)num, last.far = (int)far, last.two = bidirectional;
    }
    *w = last.w;
    return true;
}

struct Args {
    int dt;
    int64_t b, np, sq, sk;
    float scale;
    int table_dt;
    const void* table;
    int64_t num_buckets, max_distance;
    int bidirectional;
    const void* mask;
    int64_t mask_b, mask_np, mask_sq;
    int causal;
    int64_t q_start;
    const int32_t* seq_start;
    float p;
    uint64_t seed, offset, elem_base;
    int64_t n, mask_bytes, table_bytes;  // set by check()
};

// Sizes, dtypes and probabilities (no pointer of the data is looked at).
inline int check(Args& a, Buckets* w)
{
    a.n = a.mask_bytes = a.table_bytes = 0;
    if (!valid_dtype(a.dt) || (a.table && !valid_dtype(a.table_dt)))
        return MFX_ERR_DTYPE;
    if (!(a.p >= 0.0f && a.p < 1.0f))
        return MFX_ERR_PROB;
    constexpr int64_t kMost = (int64_t)1 << 29;
    if (a.b < 0 || a.np < 0 || a.sq < 0 || a.sk < 0 || a.b > kMost || a.np > kMost || a.sq > kMost || a.sk > kMost ||
        a.q_start > kMost || a.q_start < -kMost)
        return MFX_ERR_SHAPE;
    if (a.b * a.sq > ((int64_t)1 << 30))
        return MFX_ERR_SHAPE;
    int64_t n = 1, bytes = 0;
    if (!mul_ok(a.b, a.np, &n) || !mul_ok(n, a.sq, &n) || !mul_ok(n, a.sk, &n) || !mul_ok(n, 16, &bytes))
        return MFX_ERR_SHAPE;
    if (a.mask && ((a.mask_b != 1 && a.mask_b != a.b) || (a.mask_np != 1 && a.mask_np != a.np) ||
                   (a.mask_sq != 1 && a.mask_sq != a.sq)))
        return MFX_ERR_SHAPE;
    if (!make_buckets(a.table ? a.num_buckets : 0, a.max_distance, a.bidirectional != 0, w) ||
        (a.table && a.num_buckets == 0))
        return MFX_ERR_SHAPE;
    if (a.p > 0.0f && a.elem_base > UINT64_MAX - (uint64_t)n)
        return MFX_ERR_SHAPE;
    a.n = n;
    if (a.mask && n)
        a.mask_bytes = a.mask_b * a.mask_np * a.mask_sq * a.sk * dtype_bytes(a.dt);
    if (a.table && !mul_ok(a.np, a.num_buckets * dtype_bytes(a.table_dt), &a.table_bytes))
        return MFX_ERR_SHAPE;
    return MFX_OK;
}

inline Geom make_geom(const Args& a, const Buckets& w, const void* x)
{
    Geom g = {};
    g.sq = (int)a.sq, g.sk = (int)a.sk, g.np = (int)a.np, g.rows = (int)(a.b * a.sq);
    g.total = a.n, g.mask_total = a.mask_bytes / dtype_bytes(a.dt);
    g.mask_sq = a.mask_sq == 1 ? 0 : a.sk;
    g.mask_np = a.mask_np == 1 ? 0 : a.mask_sq * a.sk;
    g.mask_b = a.mask_b == 1 ? 0 : a.mask_np * a.mask_sq * a.sk;
    // positions past the reach of every key have the same buckets wherever
    // they are (with starts of the sequences' own, up to what those may add)
    const int64_t slack = a.seq_start ? 0 : w.reach + 1, lo = -a.sq - slack, hi = a.sk + slack;
    g.q_start = (int)(a.seq_start ? a.q_start : a.q_start < lo ? lo : a.q_start > hi ? hi : a.q_start);
    g.seq_start = a.seq_start;
    g.drop = a.p > 0.0f, g.causal = a.causal != 0, g.table_bf16 = a.table_dt == MFX_BF16;
    // chunks follow the generator's blocks; without dropout, the buffer's vectors
    g.phase0 = a.p > 0.0f ? (int)(a.elem_base & 7)
                          : (int)((reinterpret_cast<uintptr_t>(x) / (size_t)dtype_bytes(a.dt)) & 7);
    g.scale = a.scale, g.scale2 = (float)((double)a.scale * 1.4426950408889634);
    g.keep_scale = 1.0f / (1.0f - a.p);
    const float size = std::fabs(a.scale), fold = size >= 1e-30f && size <= 1e30f ? a.scale : 1.0f;
    g.grad = g.keep_scale * fold, g.unfold = 1.0f / fold, g.post = fold == a.scale ? 1.0f : a.scale;
    const double t = std::ceil((double)a.p * 65536.0);
    g.thresh_hi = (uint32_t)(t > 65535.0 ? 65535.0 : t) << 16;
    g.elem_base = a.elem_base;
    g.gen = make_mask_gen(a.seed, a.offset);
    return g;
}

// Chunks of the longest row.
inline int64_t chunks_of(const Geom& g, bool fast) { return (g.sk + (fast ? 0 : 7) + 7) / 8; }

// Threads, rows and register blocks of a launch; returns the chunks that a
// thread holds, up to `most`.  A row of at most 32 * `most` chunks has 8, 16 or
// 32 lanes of a warp: the fewer, the more rows share a warp's reduction and
// bookkeeping, so as few as still give every SM 512 threads, but not fewer
// than `least` nor more than `shared` chunks to each.  (bf16 forwards,
// 16x16x512x512: 16 lanes 62 us, 8 lanes 48; 32x12x256x256: 32 lanes 33 us, 16
// lanes 25, 8 lanes 20.)
inline int plan(Geom& g, bool fast, int most, int shared, int least)
{
    const int64_t chunks = chunks_of(g, fast), rows = (int64_t)g.rows * g.np;
    g.cluster = 1, g.teams = 1, g.blocks = 1;
    if (chunks <= 32 * most) {
        int c = 1;
        while (32 * c < chunks)
            c *= 2;
        g.team = chunks <= 8 ? 8 : chunks <= 16 ? 16 : 32;
        while (2 * c <= shared && g.team > least && rows * g.team / 2 >= (int64_t)sm_count() * 512)
            c *= 2, g.team /= 2;
        g.teams = kSmallBlock / g.team;
        g.exact = fast && chunks == (int64_t)g.team * c;
        return c;
    }
    if (most > 4 && chunks > (int64_t)kTeam * most)
        most = 4;  // more threads first
    const int64_t team = ((chunks + most - 1) / most + 31) / 32 * 32, held = (int64_t)kLongTeam * most;
    g.team = (int)(team < kLongTeam ? team : kLongTeam);
    g.blocks = (int)(chunks > held ? (chunks + held - 1) / held : 1);
    g.exact = fast && chunks == (int64_t)g.team * most;
    return most;
}

// Blocks per head, of which `slots` run at a time over all heads: the number
// of waves, up to 8, whose longest block times waves is least, a block's start
// (its window, say) counted as `extra` rows.
inline int slices_for(const Geom& g, int64_t slots, int64_t extra)
{
    const int64_t need = ((int64_t)g.rows + g.teams - 1) / g.teams;  // most that have a row each
    int64_t best = 1, cost = INT64_MAX;
    for (int64_t waves = 1; waves <= 8; ++waves) {
        int64_t n = slots * waves / g.np;
        n = n < 1 ? 1 : n < need ? n : need;
        const int64_t rounds = (n * g.np + slots - 1) / slots;
        const int64_t c = rounds * ((need + n - 1) / n + extra);
        if (c < cost)
            cost = c, best = n;
    }
    return (int)best;
}

// The steps of a team's walk, once slices and teams are known.
inline void set_walk(Geom& g)
{
    g.step = g.slices * g.teams;
    g.step_i = g.step / g.sq, g.step_q = g.step % g.sq;
    g.wrap_r = (int64_t)(g.np - 1) * g.sq;
    g.step_r = g.step + g.step_i * g.wrap_r;
}

// Whether every row is whole chunks of 16-byte vectors.
inline bool whole_chunks(const Args& a, const void* p, const void* q, const void* r)
{
    return a.sk % 8 == 0 && aligned16(p) && aligned16(q) && aligned16(r) && aligned16(a.mask) &&
           (a.p == 0.0f || a.elem_base % 8 == 0);
}

// Calls f(type, dropout, mask, whole chunks) with the values as types.  Rows
// that are not whole chunks have one kernel for any dropout and mask, which
// asks at run time.
template <typename F>
int by_variant(const Args& a, bool fast, F f)
{
    using Y = std::true_type;
    using N = std::false_type;
    const auto one = [&](auto t) {
        if (!fast)
            return f(t, Y{}, Y{}, N{});
        if (a.p > 0.0f)
            return a.mask ? f(t, Y{}, Y{}, Y{}) : f(t, Y{}, N{}, Y{});
        return a.mask ? f(t, N{}, Y{}, Y{}) : f(t, N{}, N{}, Y{});
    };
    return a.dt == MFX_BF16 ? one(bf16{}) : one(float{});
}

}  // namespace relbias
}  // namespace mfx
