// vocab.cuh -- what the operators on rows of logits share: a row's elements
// as 16-byte runs kept in shared memory, the running softmax statistics, and
// joining them over a block and the blocks of a cluster.
//
// With p = softmax(scale * z), the exponents are t = (z - max) * scale * log2 e
// <= 0, formed by one subtraction (exact next to the maximum) and one product,
// two elements an instruction.  Where t is a factor it is held at -200 from
// below, where 2^t is zero: columns at -inf then add nothing to sums of e * t,
// and NaN stays NaN.
//
// Two ways through the rows:
//  - Slices (few rows, and calls that read a row twice).  A row is cut into as
//    many slices as leave a block 64 KB or less, one block of a cluster each.
//    A block copies its slice to shared memory (16 bytes an asynchronous copy,
//    every thread its own runs, so that it waits for nobody) and reads it there
//    as often as it has to: HBM sees the row once.  Three blocks share a
//    multiprocessor: while one of them waits or sorts, the others' copies are
//    under way.  (Slices of 32 KB in five blocks of 128 threads: 4096x131072
//    forward and gradient 483 us instead of 425 at that step.)
//  - Rows one after another (many rows that are read once; see Stream): no
//    cluster to wait for, and copies under way over the rows' borders.
//    From two rows a multiprocessor on (see streamed()).
// Four groups of a thread's four runs are in flight; a group's largest element
// is found first, so that its sums are rebased at most once.
#pragma once

#include "mfx_device.cuh"
#include "mfx_host.h"

namespace mfx {
namespace vocab {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
// Tuning knobs (the defaults are the shipped configuration).
#ifndef MFX_VOCAB_THREADS
#define MFX_VOCAB_THREADS 256
#endif
#ifndef MFX_VOCAB_RUNS
#define MFX_VOCAB_RUNS 4096
#endif
#ifndef MFX_VOCAB_BLOCKS
#define MFX_VOCAB_BLOCKS 3
#endif
constexpr int kThreadsMost = MFX_VOCAB_THREADS;  // threads of a block that share a slice
constexpr int kSliceRuns = MFX_VOCAB_RUNS;       // runs of 16 bytes that a block keeps

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

__device__ __forceinline__ float2 exp2_pair(float2 t) { return make_float2(exp2_approx(t.x), exp2_approx(t.y)); }

// The elements of a 16-byte run as fp32 pairs, their maximum (NaN counts for
// nothing), and a run of -inf.
template <typename T> struct Run;
template <> struct Run<bf16> {
    static constexpr int V = 8;
    static __device__ __forceinline__ uint4 none() { return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }
    static __device__ __forceinline__ void widen(const uint4& w, float2 (&f)[4])
    {
        f[0] = widen2(w.x), f[1] = widen2(w.y), f[2] = widen2(w.z), f[3] = widen2(w.w);
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    // Elements below a floor raised to it; NaN stays.
    static __device__ __forceinline__ uint32_t raise2(uint32_t a, uint32_t floor)
    {
        uint32_t r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(floor));
        return r;
    }
    static __device__ __forceinline__ uint4 raise(const uint4& w, uint32_t f)
    {
        return make_uint4(raise2(w.x, f), raise2(w.y, f), raise2(w.z, f), raise2(w.w, f));
    }
    template <int U> static __device__ __forceinline__ float top_of(const uint4 (&w)[U])
    {
        uint32_t m[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            m[i] = max2(max2(w[i].x, w[i].y), max2(w[i].z, w[i].w));
#pragma unroll
        for (int i = 1; i < U; ++i)
            m[0] = max2(m[0], m[i]);
        const float2 f = widen2(m[0]);
        return fmaxf(f.x, f.y);
    }
    static __device__ __forceinline__ uint4 narrow(const float2 (&f)[4])
    {
        return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                          pack_bf16x2(f[3].x, f[3].y));
    }
};
template <> struct Run<float> {
    static constexpr int V = 4;
    static __device__ __forceinline__ uint4 none() { return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u); }
    static __device__ __forceinline__ void widen(const uint4& w, float2 (&f)[2])
    {
        f[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
        f[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
    }
    template <int U> static __device__ __forceinline__ float top_of(const uint4 (&w)[U])
    {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < U; ++i)
            m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(w[i].x), __uint_as_float(w[i].y)),
                               fmaxf(__uint_as_float(w[i].z), __uint_as_float(w[i].w))));
        return m;
    }
    static __device__ __forceinline__ uint4 narrow(const float2 (&f)[2])
    {
        return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
    }
};

// n elements from p on as runs of 16 bytes that begin at multiples of 16
// bytes: run u holds columns [V u - phase, V u - phase + V) of [0, n).
template <typename T> struct Runs {
    static constexpr int V = Run<T>::V;
    const T* p;
    int n, phase, count;
    __device__ __forceinline__ Runs(const T* p_, int n_)
        : p(p_), n(n_), phase((int)((reinterpret_cast<uintptr_t>(p_) & 15u) / sizeof(T))),
          count((int)(((int64_t)n_ + phase + V - 1) / V))
    {
    }
    __device__ __forceinline__ int column(int u) const { return V * u - phase; }
    __device__ __forceinline__ bool whole(int u) const { return V * u >= phase && V * u - phase + V <= n; }
};

// V elements of a row of n from column c on, -inf where there is none, element
// by element.
template <typename T>
__device__ __noinline__ uint4 edge_run(const T* row, int n, int c)
{
    constexpr int V = Run<T>::V;
    uint4 w = Run<T>::none();
    if constexpr (V == 8) {
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            h[j] = c + j >= 0 && c + j < n ? (uint32_t)row[c + j].bits : 0xFF80u;
        w = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    } else {
        const auto at = [&](int i) { return i >= 0 && i < n ? __float_as_uint(row[i]) : 0xFF800000u; };
        w = make_uint4(at(c), at(c + 1), at(c + 2), at(c + 3));
    }
    return w;
}

// The same at any alignment, through the two aligned vectors that hold it
// where those lie in the row.  ALONE: its neighbours are not read.
template <typename T, bool ALONE = false>
__device__ __forceinline__ uint4 load_run(const T* row, int n, int c)
{
    constexpr int V = Run<T>::V;
    const uintptr_t a = reinterpret_cast<uintptr_t>(row + c), v = a & ~(uintptr_t)15;
    const uint32_t off = (uint32_t)(a & 15u);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(row), hi = reinterpret_cast<uintptr_t>(row + n);
    if (c >= 0 && c + V <= n) {
        if (off == 0)
            return ALONE ? ld16_ca(reinterpret_cast<const void*>(a)) : ld16(reinterpret_cast<const void*>(a));
        if (v >= lo && v + 32 <= hi) {
            const uint4 p = ld16_ca(reinterpret_cast<const void*>(v)), q = ld16_ca(reinterpret_cast<const void*>(v + 16));
            const uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
            return extract16(w, off);
        }
    }
    return edge_run(row, n, c);
}

// Stores a run's elements that lie in columns [lo, hi) at run v of an output
// row.
template <typename T>
__device__ __forceinline__ void store_run(const Runs<T>& o, T* row, int v, int lo, int hi, const uint4& w)
{
    constexpr int V = Run<T>::V;
    const int c = o.column(v);
    if (c >= lo && c + V <= hi) {
        st16(row + c, w);
    } else {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c + j >= lo && c + j < hi) {
                if constexpr (V == 8)
                    row[c + j].bits = (uint16_t)(j & 1 ? x[j >> 1] >> 16 : x[j >> 1]);
                else
                    row[c + j] = __uint_as_float(x[j]);
            }
    }
}

// Running statistics of some of a row's elements: the reference that the
// exponents are taken from (their maximum; the lowest finite value while there
// is none above), l = sum of e, s = sum of e * t.
struct Stats {
    float ref, l, s;
};
__device__ __forceinline__ Stats no_stats() { return {-3.402823466e38f, 0.0f, 0.0f}; }

// Takes the sums of `v` to the reference `ref`, which is at least its own.
__device__ __forceinline__ void rebase(Stats& v, float ref, float k2)
{
    const float d = at_least_zero_power((v.ref - ref) * k2), f = exp2_approx(d);
    v.s = f * fmaf(v.l, d, v.s);
    v.l *= f;
    v.ref = ref;
}

// Joins the statistics of 2^LEVELS neighbouring lanes, the same bits in each:
// their references' maximum first, so that each is rebased once.
template <int LEVELS, bool ENTROPY>
__device__ __forceinline__ void join_lanes(Stats& v, float k2)
{
    float ref = v.ref;
#pragma unroll
    for (int o = 1 << (LEVELS - 1); o > 0; o >>= 1)
        ref = fmaxf(ref, __shfl_xor_sync(0xFFFFFFFFu, ref, o));
    rebase(v, ref, k2);
#pragma unroll
    for (int o = 1 << (LEVELS - 1); o > 0; o >>= 1) {
        v.l += __shfl_xor_sync(0xFFFFFFFFu, v.l, o);
        if (ENTROPY)
            v.s += __shfl_xor_sync(0xFFFFFFFFu, v.s, o);
    }
}

// The statistics of the block's first `warps` warps (at most 8) in every
// thread, joined in a fixed order.  `part`: 8 of them in shared memory, free
// again after the next barrier.  A barrier in any case.
template <bool ENTROPY>
__device__ __forceinline__ void join_block(Stats& v, float k2, Stats* part, int warps)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp < warps) {
        join_lanes<5, ENTROPY>(v, k2);
        if (lane == 0)
            part[warp] = v;
    }
    __syncthreads();
    v = (lane & 7) < warps ? part[lane & 7] : no_stats();
    join_lanes<3, ENTROPY>(v, k2);
}

// Element i of an index array of 32 or 64 bits; a value that is no column of
// [0, n) comes back as -1.
__device__ __forceinline__ int column_of(const void* index, bool wide, int64_t i, int n)
{
    const int64_t c = wide ? static_cast<const int64_t*>(index)[i] : static_cast<const int32_t*>(index)[i];
    return c >= 0 && c < n ? (int)c : -1;
}

// --- a block's slice of a row ----------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void copy16(uint32_t to, const void* from)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t a, const uint4& v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

constexpr int kGroups = 4;  // copies are waited for in four steps

// Runs [first, last) of a row in shared memory at `buf` (16-byte aligned, one
// run to spare before and behind).  Those of [whole0, whole1) are whole; one at
// the row's head and one at its tail may not be.  STEP: the threads that share
// it (the block's first ones) where that is known when this is compiled, which
// turns a thread's addresses into constants, else 0.
template <typename T, int STEP> struct Piece {
    Runs<T> r;
    int first, last, whole0, whole1, step_;
    uint32_t buf;

    __device__ __forceinline__ Piece(const Runs<T>& r_, uint32_t buf_, int step) : r(r_), step_(step), buf(buf_) {}
    __device__ __forceinline__ int step() const { return STEP ? STEP : step_; }
    __device__ __forceinline__ void set(int f, int l)
    {
        first = f, last = l;
        whole0 = f < l && !r.whole(f) ? f + 1 : f;
        whole1 = whole0 < l && !r.whole(l - 1) ? l - 1 : l;
    }
    __device__ __forceinline__ uint32_t at(int u) const { return buf + 16u * (uint32_t)(u - first + 1); }
    // runs of a thread that a step copies
    __device__ __forceinline__ int each() const
    {
        const int mine = (last - first + step() - 1) / step();
        return max((mine + kGroups - 1) / kGroups, min(mine, 4));
    }
    // Starts the copies of this thread's runs: every step-th.
    __device__ __forceinline__ void fill() const
    {
        const int n = each(), tid = threadIdx.x;
        const uint32_t tail = (uint32_t)(last - 1 - first - tid);
        if (tid == 0 && whole0 > first)
            sts16(at(first), edge_run(r.p, r.n, r.column(first)));
        if (whole1 < last && tail % (uint32_t)step() == 0 && last - 1 >= first + tid)
            sts16(at(last - 1), edge_run(r.p, r.n, r.column(last - 1)));
        // this thread's runs up to whole1, the first of them left out if it is not whole
        int left = whole1 - first - tid;
        const T* from = r.p + r.column(first + tid);
        uint32_t to = at(first + tid);
        bool skip = tid == 0 && whole0 > first;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            int i = 0;
            for (; i + 4 <= n && left > 3 * step() && !skip; i += 4) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    copy16(to + 16u * (uint32_t)(j * step()), from + j * step() * Run<T>::V);
                left -= 4 * step(), from += 4 * step() * Run<T>::V, to += 64u * (uint32_t)step();
            }
#pragma unroll 1
            for (; i < n; ++i) {
                if (left > 0 && !skip)
                    copy16(to, from);
                skip = false;
                left -= step(), from += step() * Run<T>::V, to += 16u * (uint32_t)step();
            }
            copies_commit();
        }
    }
    // Asks L2 for the same runs of the row that begins `ahead` elements further
    // on (one thread; its vectors there are the ones around these elements).
    __device__ __forceinline__ void prefetch(int64_t ahead) const
    {
        const uintptr_t a = (reinterpret_cast<uintptr_t>(r.p + ahead + r.column(whole0)) + 15u) & ~(uintptr_t)15;
        const uint32_t n = whole1 - whole0 > 1 ? (uint32_t)(whole1 - whole0 - 1) * 16u : 0u;
        prefetch_l2_if(reinterpret_cast<const void*>(a), n, n);
    }
    // Columns [lo, hi) that it holds.
    __device__ __forceinline__ int lo() const { return max(r.column(first), 0); }
    __device__ __forceinline__ int hi() const { return min(r.column(last), r.n); }
    // One of those columns' elements.
    __device__ __forceinline__ float value(int c) const
    {
        const uint32_t a = buf + 16u + (uint32_t)(c - r.column(first)) * (uint32_t)sizeof(T);
        if constexpr (sizeof(T) == 2) {
            uint16_t h;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(a) : "memory");
            return __uint_as_float((uint32_t)h << 16);
        } else {
            float f;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(a) : "memory");
            return f;
        }
    }
    // V elements from column c on, at any alignment (some may lie outside).
    __device__ __forceinline__ uint4 run_at(int c) const
    {
        const uint32_t a = buf + 16u + (uint32_t)((c - r.column(first)) * (int)sizeof(T)), off = a & 15u;
        const uint4 p = lds16(a - off);
        if (off == 0)
            return p;
        const uint4 q = lds16(a - off + 16);
        const uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
        return extract16(w, off);
    }
};

// What a launch's scale says of exponents: scale * log2 e, and up to where a
// row's maximum leaves room for a floor (bf16 pairs of it) that is far enough
// below it to have no power and near enough for a finite exponent.
struct Scaling {
    float k2, tame;
    uint32_t floor;
};
inline Scaling scaling_of(float scale)
{
    Scaling s = {scale * kLog2e, 0.0f, 0u};
    if (s.k2 >= 1e-30f) {
        // 2^122 (about 5e36), or less where the scale is large: a power of two, so exact in bf16
        int e = 122;
        float k = s.k2;
        for (; k > 1.0f && e > -100; k *= 0.5f)
            --e;
        const uint32_t f = 0x8000u | (uint32_t)(e + 127) << 7;
        s.floor = f << 16 | f;
        s.tame = ldexpf(0.5f, e);
    }
    return s;
}

// Adds up e (and e * t) of U runs.  CLAMP: exponents are held at -200.
template <typename T, bool ENTROPY, bool CLAMP, int U>
__device__ __forceinline__ void add_runs(Stats& v, const uint4 (&w)[U], float k2)
{
    constexpr int P = Run<T>::V / 2;
    const float2 ref = f2(-v.ref), k = f2(k2);
    float2 l = f2(0.0f), s = f2(0.0f);
#pragma unroll
    for (int i = 0; i < U; ++i) {
        float2 f[P];
        Run<T>::widen(w[i], f);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            float2 t = mul2(add2(f[j], ref), k);
            if (CLAMP)
                t = make_float2(at_least_zero_power(t.x), at_least_zero_power(t.y));
            const float2 e = exp2_pair(t);
            l = add2(l, e);
            if (ENTROPY)
                s = fma2(e, t, s);
        }
    }
    v.l += l.x + l.y;
    if (ENTROPY)
        v.s += s.x + s.y;
}

// Takes U runs of a thread into its statistics, and (BEST) into its maximum.
template <typename T, bool ENTROPY, bool BEST, int U>
__device__ __forceinline__ void take(Stats& v, float& best, uint4 (&w)[U], const Scaling& k)
{
    const float top = Run<T>::template top_of<U>(w);
    if (BEST)
        best = fmaxf(best, top);
    if (top > v.ref)
        rebase(v, top, k.k2);
    if constexpr (!ENTROPY) {
        add_runs<T, false, false, U>(v, w, k.k2);
    } else if constexpr (sizeof(T) == 4) {
        add_runs<T, true, true, U>(v, w, k.k2);
    } else if (fabsf(v.ref) < k.tame) {  // columns at -inf are raised in pairs, for half the instructions
#pragma unroll
        for (int i = 0; i < U; ++i)
            w[i] = Run<T>::raise(w[i], k.floor);
        add_runs<T, true, false, U>(v, w, k.k2);
    } else {
        add_runs<T, true, true, U>(v, w, k.k2);
    }
}

// This thread's runs of a piece whose copies are under way.
template <typename T, int STEP, bool ENTROPY, bool BEST>
__device__ __forceinline__ void scan(const Piece<T, STEP>& p, const Scaling& k, Stats& v, float& best)
{
    constexpr int U = 4;
    const int n = p.each(), step = p.step();
    int u = p.first + threadIdx.x;
    uint32_t from = p.at(u);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        if (g == 0)
            copies_wait<3>();
        else if (g == 1)
            copies_wait<2>();
        else if (g == 2)
            copies_wait<1>();
        else
            copies_wait<0>();
        int i = 0;
#pragma unroll 1
        for (; i + U <= n && u + (U - 1) * step < p.last; i += U, u += U * step, from += 16u * (uint32_t)(U * step)) {
            uint4 w[U];
#pragma unroll
            for (int j = 0; j < U; ++j)
                w[j] = lds16(from + 16u * (uint32_t)(j * step));
            take<T, ENTROPY, BEST, U>(v, best, w, k);
        }
#pragma unroll 1
        for (; i < n; ++i, u += step, from += 16u * (uint32_t)step)
            if (u < p.last) {
                uint4 w[1];
                w[0] = lds16(from);
                take<T, ENTROPY, BEST, 1>(v, best, w, k);
            }
    }
}

// --- rows one after another -------------------------------------------------
// Many rows that are read once: a block works on one after another, and each
// thread keeps four groups of four runs on their way to shared memory of its
// own, over the rows' borders, so that HBM works while a row's sums are joined.
// A row's whole runs [whole0, whole1) are dealt to the threads in turn; the
// vector at its head goes to the first thread and the one at its tail to the
// last, with the row's last group.
template <typename T> struct RowRuns {
    Runs<T> r;
    int whole0, whole1, groups;
    __device__ __forceinline__ RowRuns(const T* p, int n, int step) : r(p, n)
    {
        whole0 = r.count > 0 && !r.whole(0) ? 1 : 0;
        whole1 = r.count > whole0 && !r.whole(r.count - 1) ? r.count - 1 : max(r.count, whole0);
        groups = max((whole1 - whole0 + 4 * step - 1) / (4 * step), 1);
    }
    __device__ __forceinline__ bool head() const { return whole0 > 0; }
    __device__ __forceinline__ bool tail() const { return whole1 < r.count; }
};

// A vector at a row's border with -inf for what is not the row's.
template <typename T>
__device__ __forceinline__ uint4 only_row(const uint4& w, int c, int n)
{
    uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < Run<T>::V; ++j)
        if (c + j < 0 || c + j >= n) {
            if constexpr (sizeof(T) == 2)
                x[j >> 1] = j & 1 ? (x[j >> 1] & 0xFFFFu) | 0xFF800000u : (x[j >> 1] & 0xFFFF0000u) | 0xFF80u;
            else
                x[j] = 0xFF800000u;
        }
    return make_uint4(x[0], x[1], x[2], x[3]);
}

struct StreamArgs {
    int64_t rows, ld;
    int n, step;
    const void *logits, *tokens;  // tokens (or NULL): rows whose token is no column are passed over
    bool wide;
};

template <typename T, int STEP> struct Stream {
    static constexpr int V = Run<T>::V, kSlots = 4;
    const StreamArgs& a;
    int64_t row;     // whose groups are asked for next
    int left, group, groups, slot;
    const T* from;
    uint32_t buf;    // this thread's place in slot 0; the border vectors' slots lie behind all slots
    bool head, tail; // of that row, this thread's
    bool next_counts;

    __device__ __forceinline__ int step() const { return STEP ? STEP : a.step; }
    __host__ __device__ static size_t smem(int step) { return (size_t)(kSlots * 4 * step + kSlots * 2) * 16; }
    __device__ __forceinline__ uint32_t border(int s, int which) const
    {
        return buf - 16u * threadIdx.x + 16u * (uint32_t)(kSlots * 4 * step() + 2 * s + which);
    }
    __device__ __forceinline__ bool counts(int64_t r) const
    {
        return !a.tokens || (r < a.rows && column_of(a.tokens, a.wide, r, a.n) >= 0);
    }
    // Goes to row `r`, or the next one that counts; `now`: whether it does.
    __device__ __forceinline__ void begin(int64_t r, bool now)
    {
        while (r < a.rows && !now)
            r += gridDim.x, now = counts(r);
        row = r, group = 0;
        if (row >= a.rows)
            return;
        next_counts = counts(row + gridDim.x);  // asked long before it is needed
        const RowRuns<T> q(static_cast<const T*>(a.logits) + row * a.ld, a.n, step());
        groups = q.groups, left = q.whole1 - q.whole0 - (int)threadIdx.x;
        from = q.r.p + q.r.column(q.whole0 + threadIdx.x);
        head = q.head() && threadIdx.x == 0, tail = q.tail() && (int)threadIdx.x == step() - 1;
    }
    __device__ __forceinline__ Stream(const StreamArgs& a_, char* smem) : a(a_), slot(0)
    {
        buf = smem_addr(smem) + 16u * threadIdx.x;
        begin(blockIdx.x, counts(blockIdx.x));
        for (int s = 0; s < kSlots; ++s)
            ask();
    }
    // A vector at a border, or its elements where it reaches out of the logits.
    __device__ __forceinline__ void ask_border(int which, int u) const
    {
        const Runs<T> r(static_cast<const T*>(a.logits) + row * a.ld, a.n);
        const T* v = r.p + r.column(u);
        const T *lo = static_cast<const T*>(a.logits), *hi = lo + (a.rows - 1) * a.ld + a.n;
        if (v >= lo && v + V <= hi)
            copy16(border(slot, which), v);
        else
            sts16(border(slot, which), edge_run(r.p, r.n, r.column(u)));
    }
    // Asks for the next group, into the slot that was read last.
    __device__ __forceinline__ void ask()
    {
        if (row < a.rows) {
            const uint32_t to = buf + 64u * (uint32_t)(slot * step());
            if (left > 3 * step()) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    copy16(to + 16u * (uint32_t)(j * step()), from + j * step() * V);
            } else {
                for (int j = 0; j < 4; ++j)
                    if (left > j * step())
                        copy16(to + 16u * (uint32_t)(j * step()), from + j * step() * V);
            }
            left -= 4 * step(), from += 4 * step() * V;
            if (++group == groups) {
                if (head)
                    ask_border(0, 0);
                if (tail)
                    ask_border(1, Runs<T>(static_cast<const T*>(a.logits) + row * a.ld, a.n).count - 1);
                begin(row + gridDim.x, next_counts);
            }
        }
        copies_commit();
        slot = (slot + 1) & (kSlots - 1);
    }
    // Takes a row (the one that counts next) into `v`; `after(g, last,
    // best)` is called after its g-th group with the maximum of this thread's
    // elements since `best` was last set.
    template <bool ENTROPY, bool BEST, typename F>
    __device__ __forceinline__ void take_row(int64_t which, const Scaling& k, Stats& v, F after)
    {
        const RowRuns<T> q(static_cast<const T*>(a.logits) + which * a.ld, a.n, step());
        int rest = q.whole1 - q.whole0 - (int)threadIdx.x;
        float best = -INFINITY;
#pragma unroll 1
        for (int g = 0; g < q.groups; ++g, rest -= 4 * step()) {
            copies_wait<kSlots - 1>();
            const uint32_t at = buf + 64u * (uint32_t)(slot * step());
            if (rest > 3 * step()) {
                uint4 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = lds16(at + 16u * (uint32_t)(j * step()));
                take<T, ENTROPY, BEST, 4>(v, best, w, k);
            } else {
#pragma unroll 1
                for (int j = 0; j < 4; ++j)
                    if (rest > j * step()) {
                        uint4 w[1] = {lds16(at + 16u * (uint32_t)(j * step()))};
                        take<T, ENTROPY, BEST, 1>(v, best, w, k);
                    }
            }
            if (g == q.groups - 1) {
                if (q.head() && threadIdx.x == 0) {
                    uint4 w[1] = {only_row<T>(lds16(border(slot, 0)), q.r.column(0), a.n)};
                    take<T, ENTROPY, BEST, 1>(v, best, w, k);
                }
                if (q.tail() && (int)threadIdx.x == step() - 1) {
                    uint4 w[1] = {only_row<T>(lds16(border(slot, 1)), q.r.column(q.r.count - 1), a.n)};
                    take<T, ENTROPY, BEST, 1>(v, best, w, k);
                }
            }
            after(g, g == q.groups - 1, best);
            ask();
        }
    }
};

// Rows that are read once, and enough of them, go one after another: from two
// rows a multiprocessor on, which lies between what short and long rows want.
// Measured, us by slices and one after another, inputs not in L2:
//    log probabilities          alone                 with 20 alternatives
//    bf16  288 x  32768       8.2    8.2                12.3   17.1
//    bf16  304 x  32768       8.4    8.3                12.6   16.9
//    bf16  456 x  32768      10.5   10.5                15.6   19.0
//    bf16  608 x  32768      13.6   13.1                21.7   21.9
//    bf16  160 x 131072      16.5   14.4                27.5   27.3
//    bf16  288 x 131072      23.4   15.7                39.9   29.2
//    bf16  304 x 131072      24.1   16.0                41.1   29.4
//    bf16  608 x 131072      41.0   30.7                73.3   47.2
//    fp32  160 x  50021      12.8   10.4                23.5   21.1
//    fp32  304 x  50021      19.2   14.5                34.6   25.4
// The distillation's forward goes like the first pair (304 x 131072 25.2 and
// 16.1).  What tips it is whether the slices of all rows find places at once
// (three a multiprocessor): rows of one slice with alternatives lose up to a
// third from here to 456 rows, rows of four slices as much from one row a
// multiprocessor to here.  A border by slices would suit both.
#ifndef MFX_VOCAB_STREAM
#define MFX_VOCAB_STREAM 2
#endif
inline bool streamed(int64_t rows) { return rows >= MFX_VOCAB_STREAM * (int64_t)sm_count(); }

// A block's runs [u0, u1) of an output row from a row of logits: `f` makes a
// run of results of a run of logits and its first column.  Four runs of a
// thread are in flight.  Rows that lie alike take whole vectors, others the
// vectors around each run.
template <typename T, int STEP, typename F>
__device__ __forceinline__ void map_runs(const T* z, T* o, const Runs<T>& ro, int u0, int u1, int threads, F f)
{
    constexpr int U = 4, V = Run<T>::V;
    const int step = STEP ? STEP : threads;
    const bool alike = (reinterpret_cast<uintptr_t>(z) & 15u) == (reinterpret_cast<uintptr_t>(o) & 15u);
    int u = u0 + threadIdx.x;
    if (alike) {
        // whole runs: all but one at the row's head and one at its tail
        if (u < u1 && !ro.whole(u)) {
            store_run(ro, o, u, 0, ro.n, f(edge_run(z, ro.n, ro.column(u)), ro.column(u)));
            u += step;
        }
        const int whole = u1 > u0 && !ro.whole(u1 - 1) ? u1 - 1 : u1;
        int c = ro.column(u);
        for (; u + (U - 1) * step < whole; u += U * step, c += U * step * V) {
            uint4 w[U];
#pragma unroll
            for (int i = 0; i < U; ++i)
                w[i] = ld16(z + c + i * step * V);
#pragma unroll
            for (int i = 0; i < U; ++i)
                st16(o + c + i * step * V, f(w[i], c + i * step * V));
        }
        for (; u < whole; u += step, c += step * V)
            st16(o + c, f(ld16(z + c), c));
        if (u < u1)
            store_run(ro, o, u, 0, ro.n, f(edge_run(z, ro.n, c), c));
        return;
    }
    for (; u < u1; u += U * step) {
        uint4 w[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            w[i] = u + i * step < u1 ? load_run(z, ro.n, ro.column(u + i * step)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (u + i * step < u1)
                store_run(ro, o, u + i * step, 0, ro.n, f(w[i], ro.column(u + i * step)));
    }
}

// Zeros in a block's runs [u0, u1) of an output row.
template <typename T>
__device__ __forceinline__ void zero_runs(T* o, const Runs<T>& ro, int u0, int u1, int step)
{
    for (int u = u0 + threadIdx.x; u < u1; u += step)
        store_run(ro, o, u, 0, ro.n, make_uint4(0, 0, 0, 0));
}

// --- clusters -------------------------------------------------------------
// The cluster's barrier in two steps.  Only warps that have written what other
// blocks read arrive with a release (`wrote`, the same for a whole warp): for
// it a warp waits until all that it has stored is there.
__device__ __forceinline__ void cluster_arrive(bool wrote)
{
    if (wrote)
        asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    else
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
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
__device__ __forceinline__ float peer_float(const float* p, uint32_t rank) { return __uint_as_float(peer_word(p, rank)); }

// Statistics over the blocks of a cluster (at most 8) from each block's.
template <bool ENTROPY>
__device__ __forceinline__ void join_cluster(Stats& v, float k2, Stats* mine, int blocks)
{
    if (threadIdx.x == 0)
        *mine = v;
    __syncwarp();
    cluster_arrive(threadIdx.x < 32);
    cluster_wait();
    const int peer = threadIdx.x & 7;
    v = no_stats();
    if (peer < blocks) {
        v.ref = peer_float(&mine->ref, peer), v.l = peer_float(&mine->l, peer);
        if (ENTROPY)
            v.s = peer_float(&mine->s, peer);
    }
    join_lanes<3, ENTROPY>(v, k2);
}

// --- host -----------------------------------------------------------------
constexpr int64_t kMostColumns = 1 << 30, kMostClusters = 1 << 26;

// Blocks of a row, threads of a block, and runs that it keeps.
struct Split {
    int cluster, threads, runs;
    size_t smem() const { return (size_t)(runs + 2) * 16; }
};

// A thread has four runs or more of its row, up to `most` threads.
inline int threads_for(int64_t runs, int most)
{
    int t = 32;
    while (t < most && t * 4 <= runs)
        t *= 2;
    return t;
}

// A block works on a row of 64 KB or less, the blocks of a cluster on longer
// ones; where rows are too few for all multiprocessors, on shorter ones too.
// `runs`: what a block keeps in shared memory at a time (rows longer than a
// cluster of 8 holds are taken in pieces).
inline Split split(int64_t rows, int64_t n, int64_t bytes)
{
    const int64_t all = (n * bytes + 15) / 16 + 1;  // with a head and a tail
    Split sp = {1, 0, 0};
    sp.cluster = (int)((all + kSliceRuns) / (kSliceRuns + 1));
    if (sp.cluster > 8)
        sp.cluster = 8;
    while (sp.cluster * 2 <= 8 && rows * sp.cluster * 2 <= sm_count() && all >= sp.cluster * 2 * 2 * kThreadsMost)
        sp.cluster *= 2;
    const int64_t slice = (all + sp.cluster - 1) / sp.cluster;
    sp.threads = threads_for(slice, kThreadsMost);
    sp.runs = (int)(slice <= kSliceRuns + 1 ? slice : kSliceRuns);
    return sp;
}

// A kernel's STEP for a launch.
inline bool known_step(const Split& sp) { return sp.threads == kThreadsMost; }

// Launches a kernel over rows (grid.x / cluster at a time).  a.ahead: rows
// that are worked on at a time, so that a block knows which one comes when it
// is done.
template <typename A>
cudaError_t launch_rows(void (*kernel)(const A), A a, const Split& sp, int threads, size_t smem, cudaStream_t s)
{
    const int64_t room = (int64_t)sm_count() * occupancy(reinterpret_cast<const void*>(kernel), threads, smem);
    a.ahead = room / sp.cluster;
    cudaLaunchConfig_t cfg = {};
    // the blocks of a cluster find places together, which leaves some of them
    // free: clusters come row by row, single blocks stay
    cfg.gridDim = dim3((unsigned)(sp.cluster > 1 ? (a.rows < kMostClusters ? a.rows : kMostClusters) * sp.cluster
                                                 : a.rows < room ? a.rows : room));
    cfg.blockDim = dim3((unsigned)threads);
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

// How the backwards cut rows: threads of a block, runs of a chunk, chunks of a
// row.  A chunk is eight runs a thread or, where those leave multiprocessors
// without one, four.
struct Chunks {
    int threads, per, count;
};
inline Chunks chunks_of(int64_t rows, int64_t n, int64_t bytes)
{
    const int64_t runs = (n * bytes + 15) / 16 + 1;  // with a head and a tail
    Chunks c;
    c.threads = threads_for(runs, kThreadsMost);
    c.per = c.threads * 8;
    if (rows * ((runs + c.per - 1) / c.per) < 8 * sm_count())
        c.per = c.threads * 4;
    c.count = (int)((runs + c.per - 1) / c.per);
    return c;
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
