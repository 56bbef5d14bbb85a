// relbias.cu -- softmax of attention scores with a learned relative position
// bias and dropout, forward and backward.
//
// Per score row (batch i, head h, query q at position pos):
//   s_k = x_k * scale + table[bucket(k - pos), h] + mask_k,   P = softmax(s),
//   y_k = keep_k * P_k / (1 - p),
// and backwards, with P formed again from x and the row's statistics and the
// keep flags from the generator (neither P nor the mask is ever stored),
//   dP_k = keep_k * dy_k / (1 - p),  D = sum_k dP_k P_k,
//   dS_k = P_k (dP_k - D),  dx_k = scale * dS_k,
//   dtable[u, h] = sum of dS over the positions whose bucket is u.
//
// Layout: a team of threads (one or more warps) owns a row and keeps it in
// registers, C chunks of 8 elements a thread; a chunk is exactly one block of
// the generator (chunk boundaries sit where the element index is a multiple
// of 8), so with 16-byte aligned buffers it is also one 16-byte access, at
// any row length.  Rows longer than a team holds are walked in blocks, the
// second walk reading what L2 still has; few long forward rows are split over
// the blocks of a cluster, which exchange (maximum, sum) through distributed
// shared memory.
//
// The bias needs no [np, sq, sk] tensor: along a row it is constant outside
// the `reach` of the bucket function (the distance from which the last bucket
// holds), and inside it comes from a window of 2 * reach + 1 values in shared
// memory, built once per thread block, which works on one head.  The table's
// gradient takes the same form: far positions add into two registers, near
// ones into a shared-memory window with one slot per distance.  Within a row
// every slot belongs to one thread, and rows follow one another behind the
// row reduction's barrier, so the sums need no atomics and their order is
// fixed; each block leaves its per-bucket sums in the workspace and a second
// kernel adds those in block order.
#include <cmath>

#include "mfx_device.cuh"
#include "mfx_host.h"

namespace mfx {
namespace {

constexpr int kMaxTeam = 512;         // threads per row and block
constexpr int kSmallTeams = 4;        // rows per block where one warp holds a row
constexpr int kMaxBuckets = 256;      // buckets of a table
constexpr int kMaxSide = 128;         // buckets of one direction
constexpr int kMaxDistance = 8192;    // keeps the window within 72 KB of shared memory
constexpr int kMaxCluster = 8;        // blocks that may share a row
constexpr int kBwdBlocksPerSm = 16;   // blocks of a backward grid per SM (what its workspace goes by) ...
constexpr int kBwdRows = 16;          // ... with at least so many rows each
constexpr float kLog2eF = 1.4426950408889634f;

// The bucket function of one direction: distances below `first` have a bucket
// each, bucket first + 1 + j begins at border[j], and `reach` is where the
// last one begins.
struct Buckets {
    int num, side, first, reach, hi;  // hi: first position right of the query whose bias no longer changes
    int border[kMaxSide];
};

struct Geom {
    int64_t sq, sk, np, rows;  // rows = b * sq: rows of one head
    int64_t mb, mnp, msq;      // mask sizes (1 = broadcast)
    int64_t q_start;
    const int32_t* seq_start;  // per batch, or null
    int64_t slices;            // blocks (clusters) per head
    int team, teams, cluster;  // threads per row, rows per block, blocks per row
    int blocks;                // register blocks that a row takes
    int causal, table_bf16;
    int phase0;                // (phase0 + element index) mod 8 = 0 at a chunk's start
    float scale, keep_scale;
    uint32_t thresh_hi;        // keep threshold in the upper half-word
    uint64_t seed, offset, elem_base;
};

// Slot of window entry i.  Lanes of a warp read entries 8 apart; one pad per
// eight entries spreads those over the banks.
__device__ __host__ __forceinline__ int window_slot(int i) { return i + (i >> 3); }
inline int window_slots(const Buckets& w) { return window_slot(w.reach + w.hi) + 1; }

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

// Fills the block's window with head h's bias by relative position.
__device__ __forceinline__ void fill_window(const Buckets& w, const Geom& g, const void* table, int64_t h, float* win)
{
    for (int i = threadIdx.x; i <= w.reach + w.hi; i += blockDim.x) {
        float v = 0.0f;
        if (table) {
            const int rel = i - w.reach;
            const int u = rel <= 0 ? side_bucket(w, -rel) : side_bucket(w, rel) + w.side;
            const int64_t at = u * g.np + h;
            v = g.table_bf16 ? load1(static_cast<const bf16*>(table) + at) : load1(static_cast<const float*>(table) + at);
        }
        win[window_slot(i)] = v;
    }
}

// e^(s - m).  bf16: the hardware base-2 exponential of one fused multiply-add
// (m log2 e is rounded once, the same for every term of a row, and cancels in
// the quotient); results below 2^-126 flush to zero.  fp32: expf.
template <typename T>
__device__ __forceinline__ float exp_of(float s, float m, float ml)
{
    if constexpr (DTypeInfo<T>::kBf16) {
        float r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(s, kLog2eF, -ml)));
        return r;
    } else {
        return expf(s - m);
    }
}

// Elements [k0, k0 + 8) of a row, of which [0, end) exist; the others read as
// zero and are not touched.
template <typename T>
__device__ __forceinline__ void load_chunk(const T* p, int k0, int end, Raw8<T>& raw)
{
    if (k0 >= 0 && k0 + 8 <= end && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        ld8(p, raw);
        return;
    }
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        f[j] = k0 + j >= 0 && k0 + j < end ? load1(p + j) : 0.0f;
    narrow8(f, raw);
}

template <typename T>
__device__ __forceinline__ void store_chunk(T* p, int k0, int end, const float (&f)[8])
{
    if (k0 >= 0 && k0 + 8 <= end && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        Raw8<T> raw;
        narrow8(f, raw);
        st8(p, raw);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (k0 + j >= 0 && k0 + j < end)
            store1(p + j, f[j]);
}

// What a row's chunks share.
template <typename T>
struct Row {
    int64_t r;           // row index of the tensor
    int64_t e0;          // element index of the chunk grid's origin relative to the tensor (r * sk - a)
    uint64_t block0;     // generator block of chunk 0
    const T* mask;       // its mask row, or null
    int a, pos, end;     // chunk phase, clamped query position, keys that take part: [0, end)
    int chunks;          // chunks of the row
};

// Batch and query index of the rows a team walks, advanced without divisions.
struct Walk {
    int64_t i, q, step_i, step_q;
    __device__ __forceinline__ Walk(int64_t row, int64_t step, int64_t sq)
        : i(row / sq), q(row % sq), step_i(step / sq), step_q(step % sq)
    {
    }
    __device__ __forceinline__ void next(int64_t sq)
    {
        i += step_i;
        q += step_q;
        if (q >= sq) {
            q -= sq;
            ++i;
        }
    }
};

template <typename T>
__device__ __forceinline__ Row<T> row_at(const Geom& g, const Buckets& w, const T* mask, int64_t h, int64_t i,
                                         int64_t q)
{
    Row<T> o;
    o.r = (i * g.np + h) * g.sq + q;
    const int64_t e = o.r * g.sk;
    o.a = (int)((uint64_t)(g.phase0 + e) & 7u);
    o.e0 = e - o.a;
    o.block0 = (g.elem_base + (uint64_t)e) >> 3;
    const int64_t pos = g.q_start + q + (g.seq_start ? (int64_t)g.seq_start[i] : 0);
    // a position past the reach of every key has the same buckets wherever it is
    const int64_t lo = -(int64_t)w.reach - 1, hi = g.sk + w.reach;
    o.pos = (int)(pos < lo ? lo : pos > hi ? hi : pos);
    o.end = g.causal ? (int)(pos < 0 ? 0 : pos + 1 < g.sk ? pos + 1 : g.sk) : (int)g.sk;
    o.chunks = (int)((g.sk + o.a + 7) >> 3);
    o.mask = mask ? mask + (((g.mb == 1 ? 0 : i) * g.mnp + (g.mnp == 1 ? 0 : h)) * g.msq + (g.msq == 1 ? 0 : q)) * g.sk
                  : nullptr;
    return o;
}

// Scores of chunk k0 from its raw x: x * scale + bias (+ mask - shift), -inf
// where no key takes part.  A key whose mask is -inf is left out whatever x
// holds there.
template <typename T>
__device__ __forceinline__ void score_chunk(const Raw8<T>& raw, const Row<T>& row, const Geom& g, const Buckets& w,
                                            const float* win, float far_lo, float far_hi, int k0, float shift,
                                            float (&s)[8])
{
    widen8(raw, s);
    const int rel = k0 - row.pos;
    float b[8];
    if (rel + 7 <= -w.reach || rel >= w.hi) {
        const float v = rel >= w.hi ? far_hi : far_lo;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            b[j] = v;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = rel + j + w.reach;
            b[j] = win[window_slot(i < 0 ? 0 : i > w.reach + w.hi ? w.reach + w.hi : i)];
        }
    }
    if (row.mask) {
        Raw8<T> mraw;
        load_chunk(row.mask + k0, k0, row.end, mraw);
        float m[8];
        widen8(mraw, m);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s[j] = m[j] == -INFINITY ? -INFINITY : fmaf(s[j], g.scale, b[j]) + (m[j] - shift);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s[j] = fmaf(s[j], g.scale, b[j]);
    }
    if (k0 < 0 || k0 + 8 > row.end) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k0 + j < 0 || k0 + j >= row.end)
                s[j] = -INFINITY;
    }
}

// Keep flags of a chunk's elements, applied to v: kept values times `scale`,
// the others zero.  16-bit word j of the block belongs to element j.
__device__ __forceinline__ void drop_chunk(float (&v)[8], const uint4& blk, uint32_t thresh_hi, float scale)
{
    const uint32_t w[4] = {blk.x, blk.y, blk.z, blk.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = (w[i] << 16) >= thresh_hi ? v[2 * i] * scale : 0.0f;
        v[2 * i + 1] = w[i] >= thresh_hi ? v[2 * i + 1] * scale : 0.0f;
    }
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
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

// (maximum, sum relative to it) of two parts of a row.
__device__ __forceinline__ float2 join(float2 a, float2 b)
{
    const float m = fmaxf(a.x, b.x);
    if (m == -INFINITY)
        return make_float2(m, a.y + b.y);
    return make_float2(m, a.y * expf(a.x - m) + b.y * expf(b.x - m));
}

// ---------------------------------------------------------------------------
// Forward.
// ---------------------------------------------------------------------------
template <typename T, int C, bool DROP>
__global__ void __launch_bounds__(kMaxTeam)
relbias_fwd(const T* x, T* y, float* __restrict__ stats, const T* __restrict__ mask, const void* __restrict__ table,
            const __grid_constant__ Geom g, const __grid_constant__ Buckets w)
{
    extern __shared__ float win[];
    __shared__ float2 part[2][kMaxTeam / 32];
    __shared__ float2 mine[2];
    const int rank = (int)(blockIdx.x % g.cluster);
    const int64_t unit = blockIdx.x / g.cluster;
    const int64_t h = unit / g.slices, slice = unit % g.slices;
    const int tid = threadIdx.x % g.team, tm = threadIdx.x / g.team;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = g.team >> 5;
    fill_window(w, g, table, h, win);
    __syncthreads();
    const float far_lo = win[window_slot(0)], far_hi = win[window_slot(w.reach + w.hi)];

    int64_t row = slice * g.teams + tm;
    const int64_t step = g.slices * g.teams;
    Walk at(row, step, g.sq);
    int slot = 0;
    for (; row < g.rows; row += step, at.next(g.sq), slot ^= 1) {
        const Row<T> o = row_at(g, w, mask, h, at.i, at.q);
        const T* xr = x + o.e0;
        T* yr = y + o.e0;
        float s[C][8];
        float shift = 0.0f, m, l, mw;
        // A row whose scores all lie far from zero (a mask of lowest values,
        // say) is done once more with the mask shifted by its own maximum,
        // which leaves the softmax as it is and the scores their digits.
        for (int pass = 0;; ++pass) {
            m = -INFINITY, l = 0.0f;
            for (int blk = 0; blk < g.blocks; ++blk) {
                const int c0 = (blk * g.cluster + rank) * (C * g.team) + tid;
                Raw8<T> raw[C];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int k0 = (c0 + c * g.team) * 8 - o.a;
                    if (k0 < o.end)
                        load_chunk(xr + (k0 + o.a), k0, o.end, raw[c]);
                }
                float t = -INFINITY;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int k0 = (c0 + c * g.team) * 8 - o.a;
                    if (k0 < o.end) {
                        score_chunk(raw[c], o, g, w, win, far_lo, far_hi, k0, shift, s[c]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            s[c][j] = -INFINITY;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        t = fmaxf(t, s[c][j]);
                }
                t = fmaxf(m, warp_max(t));
                const float ref = t == -INFINITY ? 0.0f : t, refl = ref * kLog2eF;
                l *= expf(m - ref);
#pragma unroll
                for (int c = 0; c < C; ++c) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        s[c][j] = exp_of<T>(s[c][j], ref, refl);
                    l += ((s[c][0] + s[c][1]) + (s[c][2] + s[c][3])) + ((s[c][4] + s[c][5]) + (s[c][6] + s[c][7]));
                }
                m = t;
            }
            mw = m;  // what s is relative to
            l = warp_sum(l);
            if (warps > 1) {
                if (lane == 0)
                    part[slot][warp] = make_float2(m, l);
                __syncthreads();
                float2 v = part[slot][0];
                for (int i = 1; i < warps; ++i)
                    v = join(v, part[slot][i]);
                if (g.cluster > 1) {
                    if (threadIdx.x == 0)
                        mine[slot] = v;
                    cluster_sync();
                    v = peer_pair(&mine[slot], 0);
                    for (int i = 1; i < g.cluster; ++i)
                        v = join(v, peer_pair(&mine[slot], i));
                }
                m = v.x, l = v.y;
            }
            if (!o.mask || pass || !(fabsf(m) > 64.0f) || fabsf(m) == INFINITY)
                break;
            // the mask's maximum over the keys that take part
            float t = -INFINITY;
            for (int64_t k = (int64_t)rank * g.team + tid; k < o.end; k += (int64_t)g.team * g.cluster)
                t = fmaxf(t, load1(o.mask + k));
            t = warp_max(t);
            slot ^= 1;
            if (warps > 1) {
                if (lane == 0)
                    part[slot][warp] = make_float2(t, 0.0f);
                __syncthreads();
                t = part[slot][0].x;
                for (int i = 1; i < warps; ++i)
                    t = fmaxf(t, part[slot][i].x);
                if (g.cluster > 1) {
                    if (threadIdx.x == 0)
                        mine[slot] = make_float2(t, 0.0f);
                    cluster_sync();
                    for (int i = 0; i < g.cluster; ++i)
                        t = fmaxf(t, peer_pair(&mine[slot], i).x);
                }
            }
            slot ^= 1;
            shift = t;
        }
        if (stats && tid == 0 && rank == 0)
            stats[2 * o.r] = shift, stats[2 * o.r + 1] = m == -INFINITY ? m : m + logf(l);
        const float inv = m == -INFINITY && l == 0.0f ? 0.0f : (DROP ? g.keep_scale : 1.0f) / l;
        const float f1 = mw == -INFINITY && l == l ? 0.0f : expf(mw - m) * inv;
        for (int blk = 0; blk < g.blocks; ++blk) {
            const int c0 = (blk * g.cluster + rank) * (C * g.team) + tid;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int ch = c0 + c * g.team, k0 = ch * 8 - o.a;
                if (ch >= o.chunks)
                    continue;
                float f = f1;
                if (g.blocks > 1) {
                    if (k0 < o.end) {
                        Raw8<T> raw;
                        load_chunk(xr + 8 * (int64_t)ch, k0, o.end, raw);
                        score_chunk(raw, o, g, w, win, far_lo, far_hi, k0, shift, s[c]);
                        const float ref = m == -INFINITY ? 0.0f : m, refl = ref * kLog2eF;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            s[c][j] = exp_of<T>(s[c][j], ref, refl);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            s[c][j] = 0.0f;
                    }
                    f = inv;
                }
                float v[8];
                if (DROP && k0 < o.end) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[j] = s[c][j];
                    drop_chunk(v, mask_block(o.block0 + ch, g.seed, g.offset), g.thresh_hi, f);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[j] = s[c][j] * f;
                }
                if (k0 >= o.end) {  // keys that a causal row leaves out
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[j] = 0.0f;
                } else if (k0 + 8 > o.end) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (k0 + j >= o.end)
                            v[j] = 0.0f;
                }
                store_chunk(yr + 8 * (int64_t)ch, k0, (int)g.sk, v);
            }
        }
    }
    if (g.cluster > 1)
        cluster_sync();  // no block leaves while a peer may still read its pair
}

// ---------------------------------------------------------------------------
// Backward.
// ---------------------------------------------------------------------------
template <typename T, int C, bool DROP>
__global__ void __launch_bounds__(kMaxTeam)
relbias_bwd(const T* dy, const T* x, const float* __restrict__ stats, T* dx, const T* __restrict__ mask,
            const void* __restrict__ table, float* __restrict__ ws, const __grid_constant__ Geom g,
            const __grid_constant__ Buckets w)
{
    extern __shared__ float win[];
    __shared__ float part[2][kMaxTeam / 32];
    __shared__ float2 far_part[kMaxTeam / 32];
    const int64_t h = blockIdx.x / g.slices, slice = blockIdx.x % g.slices;
    const int tid = threadIdx.x % g.team, tm = threadIdx.x / g.team;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = g.team >> 5;
    const int last = w.reach + w.hi, slots = window_slot(last) + 1;
    float* acc = win + slots * (1 + tm);
    fill_window(w, g, table, h, win);
    if (ws)
        for (int i = threadIdx.x; i < slots * g.teams; i += blockDim.x)
            win[slots + i] = 0.0f;
    __syncthreads();
    const float far_lo = win[window_slot(0)], far_hi = win[window_slot(last)];
    float sum_lo = 0.0f, sum_hi = 0.0f;

    int64_t row = slice * g.teams + tm;
    const int64_t step = g.slices * g.teams;
    Walk at(row, step, g.sq);
    int slot = 0;
    for (; row < g.rows; row += step, at.next(g.sq), slot ^= 1) {
        const Row<T> o = row_at(g, w, mask, h, at.i, at.q);
        const float shift = stats[2 * o.r], stored = stats[2 * o.r + 1];
        const float lse = stored == -INFINITY ? 0.0f : stored, lsel = lse * kLog2eF;
        float P[C][8], d[C][8], D = 0.0f;
        // P and dP of a block of chunks
        auto load_block = [&](int blk) {
            Raw8<T> rx[C], rd[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int ch = (blk * C + c) * g.team + tid, k0 = ch * 8 - o.a;
                if (k0 < o.end) {
                    load_chunk(x + o.e0 + 8 * (int64_t)ch, k0, o.end, rx[c]);
                    load_chunk(dy + o.e0 + 8 * (int64_t)ch, k0, o.end, rd[c]);
                }
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int ch = (blk * C + c) * g.team + tid, k0 = ch * 8 - o.a;
                if (k0 < o.end) {
                    score_chunk(rx[c], o, g, w, win, far_lo, far_hi, k0, shift, P[c]);
                    widen8(rd[c], d[c]);
                    if (DROP)
                        drop_chunk(d[c], mask_block(o.block0 + ch, g.seed, g.offset), g.thresh_hi, g.keep_scale);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        P[c][j] = exp_of<T>(P[c][j], lse, lsel);
                        // what the upstream gradient holds at keys without weight does not count
                        d[c][j] = P[c][j] > 0.0f ? d[c][j] : 0.0f;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        P[c][j] = d[c][j] = 0.0f;
                }
            }
        };
        for (int blk = 0; blk < g.blocks; ++blk) {
            load_block(blk);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float t[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    t[j] = P[c][j] * d[c][j];
                D += ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
            }
        }
        D = warp_sum(D);
        if (warps > 1) {
            if (lane == 0)
                part[slot][warp] = D;
            __syncthreads();
            D = part[slot][0];
            for (int i = 1; i < warps; ++i)
                D += part[slot][i];
        } else {
            __syncwarp();  // the previous row's window sums before this row's
        }
        for (int blk = 0; blk < g.blocks; ++blk) {
            if (g.blocks > 1)
                load_block(blk);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int ch = (blk * C + c) * g.team + tid, k0 = ch * 8 - o.a;
                if (ch >= o.chunks)
                    continue;
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = P[c][j] * (d[c][j] - D);
                if (ws && k0 < o.end) {
                    const int rel = k0 - o.pos;
                    if (rel + 7 <= -w.reach || rel >= w.hi) {
                        const float t = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
                        sum_lo += rel >= w.hi ? 0.0f : t;
                        sum_hi += rel >= w.hi ? t : 0.0f;
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int i = rel + j + w.reach;
                            acc[window_slot(i < 0 ? 0 : i > last ? last : i)] += v[j];
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] *= g.scale;
                if (k0 + 8 > o.end) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (k0 + j >= o.end)
                            v[j] = 0.0f;
                }
                store_chunk(dx + o.e0 + 8 * (int64_t)ch, k0, (int)g.sk, v);
            }
        }
    }
    if (!ws)
        return;
    // the block's sum of each bucket: its slots of every team's window, in
    // order, and the far sums
    sum_lo = warp_sum(sum_lo);
    sum_hi = warp_sum(sum_hi);
    if (lane == 0)
        far_part[warp] = make_float2(sum_lo, sum_hi);
    __syncthreads();
    const int nw = blockDim.x >> 5;
    for (int u = warp; u < w.num; u += nw) {
        const bool right = u >= w.side;
        const int v = right ? u - w.side : u;
        int n0 = side_start(w, v);
        const int n1 = side_start(w, v + 1);
        if (right && n0 < 1)
            n0 = 1;
        float t = 0.0f;
        for (int n = n0 + lane; n < n1; n += 32) {
            const int i = window_slot(right ? w.reach + n : w.reach - n);
            for (int k = 0; k < g.teams; ++k)
                t += win[slots * (1 + k) + i];
        }
        t = warp_sum(t);
        if (lane == 0) {
            const bool lo = u == w.side - 1, hi = u == (w.hi ? w.num - 1 : 0);
            for (int k = 0; k < nw; ++k)
                t += (lo ? far_part[k].x : 0.0f) + (hi ? far_part[k].y : 0.0f);
            ws[slice * (w.num * g.np) + u * g.np + h] = t;
        }
    }
    pdl_launch_dependents();
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
// Whether n^s * a^j >= b^j * a^s in whole numbers (all below 2^14, s and j at
// most 64): products of up to 128 factors of 14 bits in 32-bit words.
bool border_reached(int n, int s, int a, int b, int j)
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
bool make_buckets(int64_t num, int64_t far, bool bidirectional, Buckets* w)
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
int check(Args& a, Buckets* w)
{
    a.n = a.mask_bytes = a.table_bytes = 0;
    if (!valid_dtype(a.dt) || (a.table && !valid_dtype(a.table_dt)))
        return MFX_ERR_DTYPE;
    if (!(a.p >= 0.0f && a.p < 1.0f))
        return MFX_ERR_PROB;
    if (a.b < 0 || a.np < 0 || a.sq < 0 || a.sk < 0 || a.sk > (1 << 30) || a.q_start > ((int64_t)1 << 40) ||
        a.q_start < -((int64_t)1 << 40))
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

Geom make_geom(const Args& a, const void* x)
{
    Geom g = {};
    g.sq = a.sq, g.sk = a.sk, g.np = a.np, g.rows = a.b * a.sq;
    g.mb = a.mask ? a.mask_b : 1, g.mnp = a.mask ? a.mask_np : 1, g.msq = a.mask ? a.mask_sq : 1;
    g.q_start = a.q_start, g.seq_start = a.seq_start;
    g.causal = a.causal != 0, g.table_bf16 = a.table_dt == MFX_BF16;
    // chunks follow the generator's blocks; without dropout, the buffer's vectors
    g.phase0 = a.p > 0.0f ? (int)(a.elem_base & 7)
                          : (int)((reinterpret_cast<uintptr_t>(x) / (size_t)dtype_bytes(a.dt)) & 7);
    g.scale = a.scale, g.keep_scale = 1.0f / (1.0f - a.p);
    const double t = std::ceil((double)a.p * 65536.0);
    g.thresh_hi = (uint32_t)(t > 65535.0 ? 65535.0 : t) << 16;
    g.seed = a.seed, g.offset = a.offset, g.elem_base = a.elem_base;
    return g;
}

// Threads, rows and register blocks of a launch.  A thread holds up to
// `c_max` chunks: enough that a row's reduction is small beside its work.
// Returns C.
int plan(Geom& g, int c_max)
{
    const bool even = g.phase0 == 0 && g.sk % 8 == 0;
    const int64_t chunks = (g.sk + (even ? 0 : 7) + 7) / 8;  // of the longest row
    g.cluster = 1, g.teams = 1, g.blocks = 1;
    int c = c_max;
    if (chunks <= 32 * c_max) {
        g.team = 32, g.teams = kSmallTeams;
        c = chunks <= 32 ? 1 : chunks <= 64 ? 2 : 4;
        return c < c_max ? c : c_max;
    }
    int64_t team = (chunks + c - 1) / c;
    team = (team + 31) / 32 * 32;
    g.team = (int)(team < kMaxTeam ? team : kMaxTeam);
    g.blocks = (int)((chunks + (int64_t)g.team * c - 1) / ((int64_t)g.team * c));
    return c;
}

// Blocks per head: `blocks_per_sm` of them over the whole grid, so that the
// last wave's idle share is small, with at least `least` rows to a block.
int64_t slices_for(const Geom& g, int64_t blocks_per_sm, int64_t least)
{
    int64_t want = ((int64_t)sm_count() * blocks_per_sm + g.np - 1) / g.np;
    const int64_t most = (g.rows + least - 1) / least;
    want = want < most ? want : most;
    return want < 1 ? 1 : want;
}

template <typename T, int C, bool DROP>
int launch_fwd(Geom g, const Buckets& w, const Args& a, const void* x, void* y, float* stats, cudaStream_t s)
{
    const void* k = reinterpret_cast<const void*>(&relbias_fwd<T, C, DROP>);
    const size_t smem = sizeof(float) * (size_t)window_slots(w);
    const int threads = g.team * g.teams;
    g.slices = slices_for(g, 4 * occupancy(k, threads, smem), g.teams);
    const int64_t blocks = g.slices * g.np * g.cluster;
    if (blocks > INT32_MAX)
        return MFX_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)g.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g.cluster > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, relbias_fwd<T, C, DROP>, static_cast<const T*>(x),
                                             static_cast<T*>(y), stats,
                                             static_cast<const T*>(a.mask), a.table, g, w);
    return e == cudaSuccess ? launch_status() : cuda_failure(e);
}

template <typename T, bool DROP>
int dispatch_fwd(const Args& a, const Buckets& w, const void* x, void* y, float* stats, cudaStream_t s)
{
    Geom g = make_geom(a, x);
    int c = plan(g, 4);
    if (g.team > 32 && a.b * a.np * a.sq < 2 * (int64_t)sm_count()) {
        // few rows: all threads of a block on one row, and long rows over the blocks of a cluster
        const int64_t chunks = (a.sk + 14) / 8;
        c = 1;
        while (c < 4 && chunks > (int64_t)kMaxTeam * c)
            c *= 2;
        while (g.cluster < kMaxCluster && chunks > (int64_t)kMaxTeam * c * g.cluster)
            g.cluster *= 2;
        int64_t team = (chunks + (int64_t)c * g.cluster - 1) / ((int64_t)c * g.cluster);
        team = (team + 31) / 32 * 32;
        g.team = (int)(team < 64 ? 64 : team < kMaxTeam ? team : kMaxTeam);
        const int64_t held = (int64_t)g.team * c * g.cluster;
        g.blocks = (int)((chunks + held - 1) / held);
    }
    return c == 1   ? launch_fwd<T, 1, DROP>(g, w, a, x, y, stats, s)
           : c == 2 ? launch_fwd<T, 2, DROP>(g, w, a, x, y, stats, s)
                    : launch_fwd<T, 4, DROP>(g, w, a, x, y, stats, s);
}

template <typename T, int C, bool DROP>
int launch_bwd(Geom g, const Buckets& w, const Args& a, const void* dy, const void* x, const float* stats, void* dx,
               void* dtable, void* workspace, size_t* workspace_bytes, cudaStream_t s)
{
    const void* k = reinterpret_cast<const void*>(&relbias_bwd<T, C, DROP>);
    const bool query = !workspace && workspace_bytes;
    const size_t win = sizeof(float) * (size_t)window_slots(w);
    if (win * (1 + g.teams) > 64 * 1024)  // a wide window: one row at a time
        g.teams = 1;
    const size_t smem = win * (1 + g.teams);
    const int threads = g.team * g.teams;
    occupancy(k, threads, smem);  // raises the kernel's shared-memory limit where needed
    g.slices = slices_for(g, kBwdBlocksPerSm, kBwdRows);
    if (g.slices * g.np > INT32_MAX)
        return MFX_ERR_SHAPE;
    const int64_t width = w.num * g.np;
    if (dtable || query) {
        bool asked = false;
        const int st = dbias_workspace(g.slices, width, workspace, workspace_bytes, &asked);
        if (st != MFX_OK || asked)
            return st;
    }
    relbias_bwd<T, C, DROP><<<(unsigned)(g.slices * g.np), threads, smem, s>>>(
        static_cast<const T*>(dy), static_cast<const T*>(x), stats,
        static_cast<T*>(dx), static_cast<const T*>(a.mask), a.table, dtable ? static_cast<float*>(workspace) : nullptr, g,
        w);
    const int st = launch_status();
    if (st != MFX_OK || !dtable)
        return st;
    return launch_dbias_finish(a.table_dt, static_cast<const float*>(workspace), g.slices, width, dtable, s);
}

template <typename T, bool DROP>
int dispatch_bwd(const Args& a, const Buckets& w, const void* dy, const void* x, const float* stats, void* dx,
                 void* dtable, void* workspace, size_t* workspace_bytes, cudaStream_t s)
{
    Geom g = make_geom(a, x);
    const int c = plan(g, 2);
    return c == 1 ? launch_bwd<T, 1, DROP>(g, w, a, dy, x, stats, dx, dtable, workspace, workspace_bytes, s)
                  : launch_bwd<T, 2, DROP>(g, w, a, dy, x, stats, dx, dtable, workspace, workspace_bytes, s);
}

}  // namespace
}  // namespace mfx

extern "C" int mfx_relbias_softmax_dropout_fwd(int dt, int64_t b, int64_t np, int64_t sq, int64_t sk, const void* x,
                                               float scale, int table_dt, const void* table, int64_t num_buckets,
                                               int64_t max_distance, int bidirectional, const void* mask,
                                               int64_t mask_b, int64_t mask_np, int64_t mask_sq, int causal,
                                               int64_t q_start, const int32_t* seq_start, float p, uint64_t seed,
                                               uint64_t offset, uint64_t elem_base, void* y, float* stats,
                                               void* stream)
{
    using namespace mfx;
    Args a{dt,     b,      np,      sq,      sk,     scale,   table_dt,  table, num_buckets, max_distance, bidirectional,
           mask,   mask_b, mask_np, mask_sq, causal, q_start, seq_start, p,     seed,        offset,       elem_base,
           0,      0,      0};
    Buckets w;
    const int st = check(a, &w);
    if (st != MFX_OK || a.n == 0)
        return st;
    if (!x || !y)
        return MFX_ERR_NULL;
    const int64_t bytes = a.n * dtype_bytes(dt), sb = b * np * sq * 8;
    if (partial_overlap(x, bytes, y, bytes) || overlaps(mask, a.mask_bytes, y, bytes) ||
        overlaps(table, a.table_bytes, y, bytes) || overlaps(seq_start, 4 * b, y, bytes) ||
        overlaps(stats, sb, y, bytes) || overlaps(stats, sb, x, bytes) || overlaps(stats, sb, mask, a.mask_bytes) ||
        overlaps(stats, sb, table, a.table_bytes) || overlaps(stats, sb, seq_start, 4 * b))
        return MFX_ERR_ALIAS;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dt == MFX_BF16)
        return p > 0.0f ? dispatch_fwd<bf16, true>(a, w, x, y, stats, s)
                        : dispatch_fwd<bf16, false>(a, w, x, y, stats, s);
    return p > 0.0f ? dispatch_fwd<float, true>(a, w, x, y, stats, s)
                    : dispatch_fwd<float, false>(a, w, x, y, stats, s);
}

extern "C" int mfx_relbias_softmax_dropout_bwd(int dt, int64_t b, int64_t np, int64_t sq, int64_t sk, const void* dy,
                                               const void* x, const float* stats, float scale, int table_dt,
                                               const void* table, int64_t num_buckets, int64_t max_distance,
                                               int bidirectional, const void* mask, int64_t mask_b, int64_t mask_np,
                                               int64_t mask_sq, int causal, int64_t q_start,
                                               const int32_t* seq_start, float p, uint64_t seed, uint64_t offset,
                                               uint64_t elem_base, void* dx, void* dtable, void* workspace,
                                               size_t* workspace_bytes, void* stream)
{
    using namespace mfx;
    Args a{dt,     b,      np,      sq,      sk,     scale,   table_dt,  table, num_buckets, max_distance, bidirectional,
           mask,   mask_b, mask_np, mask_sq, causal, q_start, seq_start, p,     seed,        offset,       elem_base,
           0,      0,      0};
    Buckets w;
    int st = check(a, &w);
    if (st != MFX_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool query = workspace_bytes && !workspace;
    if (query && !table) {
        *workspace_bytes = 0;
        return MFX_OK;
    }
    if (a.n == 0) {
        if (query) {
            *workspace_bytes = 0;
            return MFX_OK;
        }
        if (!dtable || a.table_bytes == 0)
            return MFX_OK;
        return cudaMemsetAsync(dtable, 0, (size_t)a.table_bytes, s) == cudaSuccess ? MFX_OK
                                                                                  : cuda_failure(cudaGetLastError());
    }
    if (!query) {
        if (!dy || !x || !stats || !dx || (dtable && (!table || !workspace || !workspace_bytes)))
            return MFX_ERR_NULL;
        const int64_t bytes = a.n * dtype_bytes(dt), sb = b * np * sq * 8, tb = a.table_bytes;
        if (partial_overlap(dy, bytes, dx, bytes) || partial_overlap(x, bytes, dx, bytes) ||
            overlaps(mask, a.mask_bytes, dx, bytes) || overlaps(table, tb, dx, bytes) ||
            overlaps(stats, sb, dx, bytes) || overlaps(seq_start, 4 * b, dx, bytes))
            return MFX_ERR_ALIAS;
        if (dtable) {
            const int64_t wsb = (int64_t)*workspace_bytes;
            const void* const other[] = {dy, x, dx, mask, stats, table, seq_start};
            const int64_t size[] = {bytes, bytes, bytes, a.mask_bytes, sb, tb, 4 * b};
            for (int i = 0; i < 7; ++i)
                if (overlaps(dtable, tb, other[i], size[i]) || overlaps(workspace, wsb, other[i], size[i]))
                    return MFX_ERR_ALIAS;
            if (overlaps(dtable, tb, workspace, wsb))
                return MFX_ERR_ALIAS;
        }
    }
    size_t* need = dtable || query ? workspace_bytes : nullptr;
    if (dt == MFX_BF16)
        return p > 0.0f ? dispatch_bwd<bf16, true>(a, w, dy, x, stats, dx, dtable, workspace, need, s)
                        : dispatch_bwd<bf16, false>(a, w, dy, x, stats, dx, dtable, workspace, need, s);
    return p > 0.0f ? dispatch_bwd<float, true>(a, w, dy, x, stats, dx, dtable, workspace, need, s)
                    : dispatch_bwd<float, false>(a, w, dy, x, stats, dx, dtable, workspace, need, s);
}
