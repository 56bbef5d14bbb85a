// rmsnorm.cuh -- what the root-mean-square norm's forward and backward share:
// rows that come to shared memory while others are worked on, their layout
// over a team of threads, and sums over a team.
//
// A team of `lanes` threads (8, 16 or 32 lanes of a warp, or a whole block)
// owns a row, E elements a thread; blocks stay on the GPU and take every
// gridDim-th row.  The rows to come (`depth` of them) are on their way to
// shared memory by asynchronous copies, so that HBM works while a team waits
// for its own sum.  A thread has the same columns of every row: their factors,
// places and bounds are formed once, and per element and row there are some
// ten instructions left (loops over columns with all that inside had 60 to 180
// and were bound by them).
//
// A warp has 32 E columns on end.  With vectors a thread's k-th unit is columns
// 32 V k + V lane on of them (V = 8 where all data is bf16, 4 where some of it
// is fp32, so that a warp's accesses cover whole lines of each), and it copies
// what it reads itself: no barrier; places past the row's end are zeros from
// the start.  Without (a width that is not a multiple of 8, or a buffer off a
// vector) units are single columns, 32 k + lane, and rows are copied as the
// 16-byte vectors that cover them, by all threads for all: a barrier more, or
// two.
#pragma once

#include "mfx_device.cuh"
#include "mfx_host.h"

namespace mfx {
namespace rmsnorm {

#ifndef MFX_NORM_DEPTH
#define MFX_NORM_DEPTH 2  // rows on their way (65536x1024 bf16 backward 122 us; 133 with four)
#endif
constexpr int kMostDepth = MFX_NORM_DEPTH;
constexpr int kPad = 32;  // bytes that a row's covering vectors may be longer by

// --- units ------------------------------------------------------------------
template <typename T, int V>
__device__ __forceinline__ void widen_unit(const uint4& w, float (&f)[V])
{
    if constexpr (sizeof(T) == 4) {
        static_assert(V == 4, "fp32 units");
        f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
    } else {
        f[0] = bf16lo(w.x), f[1] = bf16hi(w.x), f[2] = bf16lo(w.y), f[3] = bf16hi(w.y);
        if constexpr (V == 8)
            f[4] = bf16lo(w.z), f[5] = bf16hi(w.z), f[6] = bf16lo(w.w), f[7] = bf16hi(w.w);
    }
}

// A unit at shared address a.
template <typename T, int V>
__device__ __forceinline__ void lds_unit(uint32_t a, float (&f)[V])
{
    constexpr int bytes = V * (int)sizeof(T);
    if constexpr (bytes == 16) {
        uint4 w;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(a) : "memory");
        widen_unit<T, V>(w, f);
    } else if constexpr (bytes == 8) {
        uint4 w;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "r"(a) : "memory");
        widen_unit<T, V>(w, f);
    } else if constexpr (bytes == 4) {
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[0]) : "r"(a) : "memory");
    } else {
        uint16_t h;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(a) : "memory");
        f[0] = __uint_as_float((uint32_t)h << 16);
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_unit(T* p, const float (&f)[V])
{
    if constexpr (V == 1)
        store1(p, f[0]);
    else if constexpr (sizeof(T) == 4)
        st16(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
    else if constexpr (V == 4)
        st8(p, make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])));
    else
        st16(p, make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])));
}

// The factors weight + offset of the unit at column c (1 without a weight).
// The weight's type is asked at run time: it comes from L1.
template <int V>
__device__ __forceinline__ void factors(const void* weight, bool w_bf16, float offset, int c, float (&w)[V])
{
    if (!weight) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            w[j] = 1.0f;
        return;
    }
    if constexpr (V == 1) {
        w[0] = w_bf16 ? load1(static_cast<const bf16*>(weight) + c) : load1(static_cast<const float*>(weight) + c);
    } else if constexpr (V == 8) {
        if (w_bf16)
            widen_unit<bf16, 8>(ld16_ro(static_cast<const bf16*>(weight) + c), w);
        else
            bias8(static_cast<const float*>(weight), c, w);
    } else {
        uint4 r;
        if (w_bf16) {
            asm("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(static_cast<const bf16*>(weight) + c));
            widen_unit<bf16, 4>(r, w);
        } else {
            widen_unit<float, 4>(ld16_ro(static_cast<const float*>(weight) + c), w);
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
        w[j] += offset;
}

// First column of a thread's k-th unit, and how many of its N units begin
// before the row's end (they do in order).
template <int V, int E>
__device__ __forceinline__ int column_of(int k, int tl)
{
    return (tl >> 5) * (32 * E) + k * (32 * V) + (tl & 31) * V;
}
template <int V, int E>
__device__ __forceinline__ int units_of(int cols, int lanes, int tl)
{
    const int left = cols - column_of<V, E>(0, tl), n = left > 0 ? (left + 32 * V - 1) / (32 * V) : 0;
    return min(lanes < 32 ? min(n, 1) : n, E / V);
}

// A thread's factors, 0 past the row's end.
template <int V, int E>
__device__ __forceinline__ void factors_of(const void* weight, bool w_bf16, float offset, int mine, int tl, float (&w)[E / V][V])
{
#pragma unroll
    for (int k = 0; k < E / V; ++k) {
        if (k < mine) {
            factors<V>(weight, w_bf16, offset, column_of<V, E>(k, tl), w[k]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                w[k][j] = 0.0f;
        }
    }
}

// A row's data that a thread reads: its k-th unit at shared address
// a + k * 32 V size; 0 past the row's end.
template <typename T, int V>
__device__ __forceinline__ void read_unit(uint32_t a, int k, int mine, float (&f)[V])
{
    lds_unit<T, V>(a + (uint32_t)(k * 32 * V * (int)sizeof(T)), f);
    if (V == 1 && k >= mine)  // a neighbour's element, or none (vectors: zeros from the start)
        f[0] = 0.0f;
}

// --- rows on their way --------------------------------------------------------
template <int BYTES>
__device__ __forceinline__ void copy_unit(uint32_t to, const void* from)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global.L2::256B [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until all but the last n of this thread's groups have come.
__device__ __forceinline__ void copies_wait(int n)
{
    switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    }
}

// Starts a team's copy of one row (cols elements at p) to shared address `to`.
// Element c is then at to + where(p) + c * size.  Vectors may hold elements of
// the rows beside it; only those that reach out of all rows ([lo, hi), the
// first row's first and the last row's last) are copied by element.
template <typename T>
__device__ __forceinline__ uint32_t where(const T* p)
{
    return (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
}
template <typename T, int V, int E>
__device__ __forceinline__ void copy_row(uint32_t to, const T* p, int cols, const T* lo, const T* hi, int lanes, int tl,
                                         int mine)
{
    if constexpr (V > 1) {
        to += column_of<V, E>(0, tl) * (uint32_t)sizeof(T), p += column_of<V, E>(0, tl);
#pragma unroll
        for (int k = 0; k < E / V; ++k)
            if (k < mine)
                copy_unit<V * (int)sizeof(T)>(to + (uint32_t)(k * 32 * V * (int)sizeof(T)), p + k * 32 * V);
    } else {
        constexpr int E = 16 / (int)sizeof(T);
        const int phase = (int)(where(p) / sizeof(T)), vectors = (cols + phase + E - 1) / E;
        for (int v = tl; v < vectors; v += lanes) {
            const T* from = p + (v * E - phase);
            if (from >= lo && from + E <= hi) {
                copy_unit<16>(to + 16u * v, from);
            } else {
#pragma unroll
                for (int j = 0; j < E; ++j)
                    if (from + j >= lo && from + j < hi) {
                        const uint32_t a = to + 16u * v + (uint32_t)j * (uint32_t)sizeof(T);
                        if constexpr (sizeof(T) == 2)
                            asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(from[j].bits) : "memory");
                        else
                            asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(from[j]) : "memory");
                    }
            }
        }
    }
}

// Zeros for a thread's units past the row's end, in one row of a stream.
template <typename T, int V, int E>
__device__ __forceinline__ void clear_rest(uint32_t to, int tl, int mine)
{
    if constexpr (V > 1) {
#pragma unroll
        for (int k = 0; k < E / V; ++k)
            if (k >= mine)
                for (int j = 0; j < V * (int)sizeof(T); j += 4)
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + (uint32_t)(column_of<V, E>(k, tl) * (int)sizeof(T) + j)),
                                 "r"(0) : "memory");
    }
}

// What others' threads have copied is there for all of a team.
__device__ __forceinline__ void team_barrier(int lanes)
{
    if (lanes > 32)
        __syncthreads();
    else
        __syncwarp();
}

// The largest absolute value of two; NaN counts as nothing.
__device__ __forceinline__ float amax(float a, float b) { return fmaxf(a, fabsf(b)); }

// (sum, maximum) over a team, the same bits in every thread of it.  Teams of
// several warps are a whole block; `slot` alternates between calls, so that
// one barrier each is enough.
template <bool MAX>
__device__ __forceinline__ float2 over_team(float2 v, int lanes, float2 (*part)[32], int slot)
{
    const auto step = [&](int o) {
        v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
        if (MAX)
            v.y = fmaxf(v.y, __shfl_xor_sync(0xFFFFFFFFu, v.y, o));
    };
    if (lanes >= 32)
        step(16);
    if (lanes >= 16)
        step(8);
    step(4), step(2), step(1);
    if (lanes > 32) {
        const int lane = threadIdx.x & 31, warps = lanes >> 5;
        if (lane == 0)
            part[slot][threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < warps ? part[slot][lane] : make_float2(0.0f, 0.0f);
        step(16), step(8), step(4), step(2), step(1);
    }
    return v;
}

// --- host ---------------------------------------------------------------------
// Elements of a thread; threads of a row and of a block, rows that a team has
// on their way, the columns that one of them has room for, and its shared
// bytes.  depth 0: the row does not
// fit, or is longer than 512 threads of 32 elements.
struct Layout {
    int E, lanes, threads, depth;
    int64_t room;
    size_t row, smem;
};

// Rows of up to 512 columns in a warp, others in a block: 8 elements a thread
// up to `most8` columns (and for few rows, up to 1024 threads: the shortest
// way), 16 up to `most16`, 32 up to 16384.  The more a thread has, the less a
// row's sum and bookkeeping weigh, as long as its registers leave enough
// threads for what is on its way.  row_bytes(room): bytes of a row of all
// streams; resident(E): threads of a multiprocessor that the kernel's registers leave.
template <typename B, typename F>
Layout layout(int64_t rows, int64_t cols, int V, int64_t most8, int64_t most16, B row_bytes, F resident)
{
    const auto lanes_of = [&](int64_t e) { return (int)(((cols + e - 1) / e + 31) / 32 * 32); };
    Layout l = {8, 32, 256, 0, 0, 0, 0};
    if (cols <= 16 * V && V > 1) {
        l.lanes = cols <= 8 * V ? 8 : 16;  // one unit each: a group of columns is consecutive lanes' also here
    } else if (cols <= 512) {
        l.E = cols <= 256 ? 8 : 16;
    } else {
        const bool few = rows <= sm_count();
        l.E = cols <= (few ? 8192 : most8) ? 8 : cols <= most16 ? 16 : 32;
        l.lanes = l.threads = lanes_of(l.E);
        if (l.E == 32 && l.lanes > 512)
            return l;
    }
    l.room = (int64_t)(l.lanes < 32 ? 32 : l.lanes) * l.E;
    l.row = (row_bytes(l.room) + 15) / 16 * 16;
    const int64_t teams = l.threads / l.lanes;
    const int most = resident(l.E) / l.threads;
    for (int blocks = most > 0 ? most : 1; blocks >= 1 && l.depth < 2; --blocks) {
        // a block's static arrays and what the system keeps of each: 2 KB
        const size_t each = (kMaxBlockSmem + 1024) / blocks - 2048;
        const size_t d = each / teams / l.row;
        l.depth = d > kMostDepth ? kMostDepth : (int)d;
    }
    const int64_t share = (rows + teams - 1) / teams;
    if (l.depth > 1 && share <= sm_count())
        l.depth = 1;  // no team has a second row
    l.smem = (size_t)teams * l.depth * l.row;
    return l;
}

// What the checks of both directions share.
inline bool sizes_ok(int64_t rows, int64_t cols)
{
    int64_t n;
    return rows >= 0 && cols >= 0 && cols <= (1 << 30) && mul_ok(rows, cols, &n) && n <= INT64_MAX / 8;
}

}  // namespace rmsnorm
}  // namespace mfx
