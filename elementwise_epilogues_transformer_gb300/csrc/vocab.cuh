// vocab.cuh -- what the operators on rows of logits share: a row's elements
// as runs of 8, the running softmax statistics, and joining them over a block
// and the blocks of a cluster.
//
// With p = softmax(scale * z), the exponents are t = (z - max) * scale * log2 e
// <= 0, formed by one subtraction (exact next to the maximum) and one product.
// They are held at -200 from below, where 2^t is zero: columns at -inf then
// add nothing, also to sums of e * t, and NaN stays NaN.
#pragma once

#include "mfx_device.cuh"
#include "mfx_host.h"

namespace mfx {
namespace vocab {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_approx(float t)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    return e;
}

// max(t, -200), NaN where t is.
__device__ __forceinline__ float at_least_zero_power(float t)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(t), "f"(-200.0f));
    return r;
}

// n elements from p on as runs of 8 columns that begin at multiples of 16 bytes:
// run u holds columns [8u - phase, 8u - phase + 8) of [0, n).
template <typename T> struct Runs {
    const T* p;
    int n, phase, count;
    __device__ __forceinline__ Runs(const T* p_, int n_)
        : p(p_), n(n_), phase((int)((reinterpret_cast<uintptr_t>(p_) & 15u) / sizeof(T))), count((n_ + phase + 7) / 8)
    {
    }
    __device__ __forceinline__ int column(int u) const { return 8 * u - phase; }
    __device__ __forceinline__ bool whole(int u) const { return 8 * u >= phase && 8 * u - phase + 8 <= n; }
    // Run u (raw), `fill` where it has no element.
    __device__ __forceinline__ void load(int u, float f[8]) const
    {
        const int c = column(u);
        if (whole(u)) {
            Raw8<T> r;
            ld8(p + c, r);
            widen8(r, f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[j] = c + j >= 0 && c + j < n ? load1(p + c + j) : -INFINITY;
        }
    }
};

// Running statistics of some of a row's elements: their maximum (-inf for
// none), the reference that the exponents are taken from (the maximum, or the
// lowest finite value while there is none), l = sum of e, s = sum of e * t.
struct Stats {
    float m, ref, l, s;
};
__device__ __forceinline__ Stats no_stats() { return {-INFINITY, -3.402823466e38f, 0.0f, 0.0f}; }

// Takes the sums of `v` to the reference `ref`, which is at least its own.
__device__ __forceinline__ void rebase(Stats& v, float ref, float k2)
{
    const float d = at_least_zero_power((v.ref - ref) * k2), f = exp2_approx(d);
    v.s = f * fmaf(v.l, d, v.s);
    v.l *= f;
    v.ref = ref;
}

__device__ __forceinline__ Stats join(Stats a, Stats b, float k2)
{
    const float ref = fmaxf(a.ref, b.ref);
    rebase(a, ref, k2);
    rebase(b, ref, k2);
    return {fmaxf(a.m, b.m), ref, a.l + b.l, a.s + b.s};
}

__device__ __forceinline__ Stats shfl_xor(Stats v, int o)
{
    return {__shfl_xor_sync(0xFFFFFFFFu, v.m, o), __shfl_xor_sync(0xFFFFFFFFu, v.ref, o),
            __shfl_xor_sync(0xFFFFFFFFu, v.l, o), __shfl_xor_sync(0xFFFFFFFFu, v.s, o)};
}

// The block's statistics in every thread, joined in a fixed order.
// `part`: 32 of them in shared memory, free again after the next barrier.
__device__ __forceinline__ Stats join_block(Stats v, float k2, Stats* part)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = join(v, shfl_xor(v, o), k2);
    const int warps = blockDim.x >> 5;
    if (warps > 1) {
        if ((threadIdx.x & 31) == 0)
            part[threadIdx.x >> 5] = v;
        __syncthreads();
        const int lane = threadIdx.x & 31;
        v = lane < warps ? part[lane] : no_stats();
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            v = join(v, shfl_xor(v, o), k2);
    }
    return v;
}

// Adds up e and e * t of eight elements.
__device__ __forceinline__ void add8(Stats& v, const float z[8], float k2)
{
    float l = 0.0f, s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float t = at_least_zero_power((z[j] - v.ref) * k2), e = exp2_approx(t);
        l += e;
        s = fmaf(e, t, s);
    }
    v.l += l;
    v.s += s;
}

__device__ __forceinline__ float max8(const float z[8])
{
    return fmaxf(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])), fmaxf(fmaxf(z[4], z[5]), fmaxf(z[6], z[7])));
}

// Element i of an index array of 32 or 64 bits; a value that is no column of
// [0, n) comes back as -1.
__device__ __forceinline__ int column_of(const void* index, bool wide, int64_t i, int n)
{
    const int64_t c = wide ? static_cast<const int64_t*>(index)[i] : static_cast<const int32_t*>(index)[i];
    return c >= 0 && c < n ? (int)c : -1;
}

// --- clusters -------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// 4 bytes of the same variable in the block `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_word(const void* p, uint32_t rank)
{
    uint32_t v, a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ Stats peer_stats(const Stats* p, uint32_t rank)
{
    return {__uint_as_float(peer_word(&p->m, rank)), __uint_as_float(peer_word(&p->ref, rank)),
            __uint_as_float(peer_word(&p->l, rank)), __uint_as_float(peer_word(&p->s, rank))};
}

// --- host -----------------------------------------------------------------
constexpr int64_t kMostColumns = 1 << 30;

// Blocks of a row and threads of a block.
struct Split {
    int cluster, threads;
};

// A thread has four runs or more of its row, up to `most` threads.
inline int threads_for(int64_t runs, int most)
{
    int t = 32;
    while (t < most && t * 4 <= runs)
        t *= 2;
    return t;
}

// A block works on a row; where rows are too few for all multiprocessors, the
// blocks of a cluster do.
inline Split split(int64_t rows, int64_t n)
{
    const int64_t runs = (n + 7) / 8;
    Split sp = {1, 0};
    while (sp.cluster < 8 && rows * sp.cluster * 2 <= sm_count() && runs >= sp.cluster * 2 * 512)
        sp.cluster *= 2;
    sp.threads = threads_for(runs / sp.cluster, 512);
    return sp;
}

// Launches a kernel over rows (grid.x / cluster at a time).
template <typename A>
cudaError_t launch_rows(void (*kernel)(const A), const A& a, const Split& sp, size_t smem, cudaStream_t s)
{
    const int64_t room = (int64_t)sm_count() * occupancy(reinterpret_cast<const void*>(kernel), sp.threads, smem);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sp.cluster > 1 || a.rows < room ? a.rows * sp.cluster : room));
    cfg.blockDim = dim3((unsigned)sp.threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)sp.cluster, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = sp.cluster > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess)
        cudaGetLastError();  // it is this call's, not the next one's
    return e;
}

inline bool row_sizes_ok(int64_t rows, int64_t vocab, int64_t ld)
{
    int64_t n;
    return rows >= 0 && vocab >= 0 && vocab <= kMostColumns && ld >= vocab && mul_ok(rows, ld, &n) && n <= INT64_MAX / 8;
}

// Bytes from a row array's first to its last element.
inline int64_t span(int64_t rows, int64_t cols, int64_t ld, int64_t size)
{
    return rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * size : 0;
}

// May `out` (rows of ldo) stand on `in` (rows of ldi), both of `cols` elements
// of `size` bytes: not at all, or as the very same rows.
inline bool rows_alias_ok(const void* out, int64_t ldo, const void* in, int64_t ldi, int64_t rows, int64_t cols,
                          int64_t size)
{
    return !overlaps(out, span(rows, cols, ldo, size), in, span(rows, cols, ldi, size)) || (out == in && ldo == ldi);
}

}  // namespace vocab
}  // namespace mfx

namespace mfx {
namespace vocab {

// A block's share of a row: whole runs [first, last), and for its thread 0
// the run at the row's head (run 0, which ends before the first whole one)
// and the one at its tail, where they are not whole.
template <typename T> struct Share {
    Runs<T> r;
    int first, last;
    bool head, tail;
    __device__ __forceinline__ Share(const Runs<T>& r_, int rank, int blocks) : r(r_)
    {
        const int w0 = r.count > 0 && !r.whole(0) ? 1 : 0;
        int w1 = r.count > w0 && !r.whole(r.count - 1) ? r.count - 1 : r.count;
        const int per = (w1 - w0 + blocks - 1) / blocks;
        first = min(w0 + rank * per, w1);
        last = min(first + per, w1);
        head = w0 == 1 && rank == 0;
        tail = w1 < r.count && rank == blocks - 1;
    }
};

// A column and its logit.  Better: a larger logit, or an equal one further
// left.  Threads that saw none have a place of their own behind all columns.
struct Pick {
    float v;
    int i;
};
__device__ __forceinline__ bool better(const Pick& a, const Pick& b) { return a.v > b.v || (a.v == b.v && a.i < b.i); }

// Takes U runs of a thread into its statistics; `best` is its best column.
template <bool BEST, int U>
__device__ __forceinline__ void take(Stats& v, Pick& best, const float (&z)[U][8], const int (&c)[U], float k2)
{
    float m = max8(z[0]);
#pragma unroll
    for (int i = 1; i < U; ++i)
        m = fmaxf(m, max8(z[i]));
    if (m > v.m) {
        if (BEST) {
            best.v = m;
#pragma unroll
            for (int i = U - 1; i >= 0; --i)
#pragma unroll
                for (int j = 7; j >= 0; --j)
                    if (z[i][j] == m)
                        best.i = c[i] + j;
        }
        v.m = m;
        rebase(v, fmaxf(m, v.ref), k2);
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
        add8(v, z[i], k2);
}

// A thread's statistics over its part of a block's share: every blockDim-th
// whole run, U of them in flight.
template <typename T, bool BEST, int U>
__device__ __forceinline__ Stats scan(const Share<T>& sh, float k2, Pick& best)
{
    Stats v = no_stats();
    best = {-INFINITY, (int)kMostColumns + (int)threadIdx.x};
    if (threadIdx.x == 0 && sh.head) {
        float z[1][8];
        const int c[1] = {sh.r.column(0)};
        sh.r.load(0, z[0]);
        take<BEST, 1>(v, best, z, c, k2);
    }
    const int step = blockDim.x;
    for (int u = sh.first + threadIdx.x; u < sh.last; u += U * step) {
        Raw8<T> r[U];
        float z[U][8];
        int c[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            c[i] = sh.r.column(u + i * step);
            if (u + i * step < sh.last)
                ld8(sh.r.p + c[i], r[i]);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (u + i * step < sh.last) {
                widen8(r[i], z[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    z[i][j] = -INFINITY;
            }
        }
        take<BEST, U>(v, best, z, c, k2);
    }
    if (threadIdx.x == 0 && sh.tail) {
        float z[1][8];
        const int c[1] = {sh.r.column(sh.r.count - 1)};
        sh.r.load(sh.r.count - 1, z[0]);
        take<BEST, 1>(v, best, z, c, k2);
    }
    return v;
}

// Statistics over the blocks of a cluster from each block's.
__device__ __forceinline__ Stats join_cluster(Stats v, float k2, Stats* mine, int blocks)
{
    if (threadIdx.x == 0)
        *mine = v;
    cluster_sync();
    const int lane = threadIdx.x & 31;
    v = lane < blocks ? peer_stats(mine, lane) : no_stats();
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
        v = join(v, shfl_xor(v, o), k2);
    const Stats w = {__shfl_sync(0xFFFFFFFFu, v.m, 0), __shfl_sync(0xFFFFFFFFu, v.ref, 0),
                     __shfl_sync(0xFFFFFFFFu, v.l, 0), __shfl_sync(0xFFFFFFFFu, v.s, 0)};
    return w;
}

// Eight elements of a row of n from column c on (some of them may lie outside:
// `fill`), at any alignment.
template <typename T>
__device__ __forceinline__ void load8_at(const T* row, int n, int c, float f[8])
{
    const T* p = row + c;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(row), hi = reinterpret_cast<uintptr_t>(row + n);
    if (c >= 0 && c + 8 <= n && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        Raw8<T> r;
        ld8(p, r);
        widen8(r, f);
    } else if (c >= 0 && c + 8 <= n && in_vectors(p, lo, hi)) {
        Raw8<T> r;
        ld8_any(p, r);
        widen8(r, f);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f[j] = c + j >= 0 && c + j < n ? load1(p + j) : -INFINITY;
    }
}

// Stores run u of an output row.
template <typename T>
__device__ __forceinline__ void store_run(const Runs<T>& o, T* row, int u, const float f[8])
{
    const int c = o.column(u);
    if (o.whole(u)) {
        Raw8<T> r;
        narrow8(f, r);
        st8(row + c, r);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j >= 0 && c + j < o.n)
                store1(row + c + j, f[j]);
    }
}

}  // namespace vocab
}  // namespace mfx
