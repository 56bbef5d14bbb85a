// logprobs.cu -- log probabilities of given tokens, with the distribution's
// entropy and the largest alternatives, and the gradients of the first two.
//
// Per row of logits z, with p = softmax(scale * z):
//   logprob = log p[token],   entropy = -sum p log p,
//   dz = scale * (g * (1[token] - p) - ge * p * (log p + entropy)).
// With m the row's maximum, t = (z - m) scale and l = sum exp(t):
//   logprob = t[token] - log l,   entropy = log l + U,   U = -sum exp(t) t / l,
// where U >= 0 and log l >= 0: nothing cancels, however far the row lies from
// zero.  (m, 1 / l, U) are kept for the backward, which is then one pass:
//   dz = scale * (g 1[token] - exp(t) / l * (g + ge * (t + U))).
//
// What bounds them: the backward HBM (8192x32768 bf16 161 us, 6670 GB/s, 0.98
// of the copy rate).  The forward HBM in long rows (1024x131072 bf16 46 us,
// 5860 GB/s), in shorter ones the instructions (8192x32768 99 us, 5440 GB/s:
// nine an element, one of them the power, and a row's sums after every 64 KB);
// rows below some 4 KB the sums alone (16384x1000 bf16 19 us, 5 of bytes).
// Alternatives cost a second kernel for many rows (1024x131072 with 20: 64 us
// in all, with 64: 90; found within the kernel, behind its barriers, they took
// 122 and 361), whose time is the reach of single sectors, and some 4 us
// within the kernel for few (8x131072 with 5: 8.3 us in all).
#include "vocab.cuh"

#include <cmath>

namespace mfx {
namespace vocab {
namespace {

#ifndef MFX_TOP_FEW
#define MFX_TOP_FEW 24
#endif
constexpr int kMostTop = 64;   // alternatives
constexpr int kMostKeys = 128;  // groups of threads that bound the search for them
// Maxima of a thread of logprobs_rows, all used where its runs allow it: what pick_top reads again is 4 runs for each
// that counts, or more in long rows (4096x32768 with 20: 80 us, 102 with 16 runs to a maximum; 1024x131072 with 64: 90 and 97).
constexpr int kMostChunks = 8;
constexpr int kMostListed = kMostChunks * kThreadsMost;
constexpr int kPickThreads = 128;
constexpr int kRound = 64;      // runs of a step that cannot overflow the candidates
constexpr int kKept = 256;      // candidates that a step may find there
constexpr int kCandidates = kRound * 8 + kKept;

struct Args {
    int64_t rows, ld, ahead;
    int n, top, cluster, runs;
    const void *logits, *tokens;
    bool wide, eager;  // eager: rows are read before it is known whether they count
    float scale;
    Scaling k;
    float *logprob, *entropy, *top_logprob, *stats;
    int32_t* top_index;
    // rows one after another
    StreamArgs in;
    int gran, chunks;  // groups of a thread's runs that share a maximum, maxima of a thread
    float* ws;  // of each row: its reference, log l, every thread's largest logits
};

// A column and its logit as one number: larger for larger logits (-0 and 0
// are equal), and among equal ones for the lower column.  0 is nothing.
using Key = unsigned long long;
__device__ __forceinline__ Key key_of(float v, int c)
{
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (Key)(b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u)) << 32 | (0xFFFFFFFFu - (uint32_t)c);
}
__device__ __forceinline__ float value_of(Key k)
{
    const uint32_t b = (uint32_t)(k >> 32);
    return __uint_as_float(b & 0x80000000u ? b ^ 0x80000000u : ~b);
}
__device__ __forceinline__ int column_of(Key k) { return (int)(0xFFFFFFFFu - (uint32_t)k); }

// Shared memory of the search for alternatives.
struct TopSmem {
    Key cand[kCandidates];
    Key keys[kMostKeys];
    Key sel[kMostTop];  // the alternatives in order, 0 behind them
    Key limit;
    int listed, count;
    int list[kThreadsMost];  // threads that may hold some
};

// The `top` largest of cand[0, n) in order to sel, 0 behind them.  Barriers
// around it.  Four threads count for each candidate where they are few.
__device__ __forceinline__ void sort_out(const Key* cand, int n, int top, Key* sel)
{
    const int tid = threadIdx.x, T = blockDim.x;
    for (int j = tid; j < top; j += T)
        if (j >= n)
            sel[j] = 0;
    if (4 * n <= T) {
        const int c = tid >> 2, part = tid & 3;
        const Key k = c < n ? cand[c] : 0;
        int r = 0;
        for (int j = part; j < n; j += 4)
            r += cand[j] > k;
        r += __shfl_xor_sync(0xFFFFFFFFu, r, 1);
        r += __shfl_xor_sync(0xFFFFFFFFu, r, 2);
        if (part == 0 && c < n && r < top)
            sel[r] = k;
        return;
    }
    for (int c = tid; c < n; c += T) {
        const Key k = cand[c];
        int r = 0;
        for (int j = 0; j < n; ++j)
            r += cand[j] > k;
        if (r < top)
            sel[r] = k;
    }
}

// The `top` largest columns above -inf of a block's runs [first, last), every
// blockDim-th of them a thread's, to sm.sel in order.  best: the largest logit
// of this thread's runs; run_at(u): run u.
//
// The top-th largest of 64 groups of threads (128 for more than 24) bounds the
// top-th largest logit from below, and only threads whose largest logit
// reaches it can hold a column that does: of all elements about as many as are
// asked for.  (64 groups for 64 alternatives: five times as many columns, 193
// us instead of 96 at 1024x131072 at that step; 128 for 5: 9.7 us instead of 8.3 at 8x131072.)  Their runs are read again for the columns that reach the bound.
// Should those be more than there is room for (many equal logits, or few
// threads with most of the large ones), the runs are taken in small steps and
// the candidates cut to the best, which raises the bound.
template <typename T, typename F>
__device__ __forceinline__ void find_top(const Runs<T>& r, int first, int last, float best, int top, TopSmem& sm, F run_at)
{
    constexpr int V = Run<T>::V;
    const int tid = threadIdx.x, T_ = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int want = top <= MFX_TOP_FEW ? 64 : kMostKeys, nkeys = T_ < want ? T_ : want, per = T_ / nkeys;
    // equal ones in some order: a thread's place, below all columns
    Key k = (best > -INFINITY ? key_of(best, 0) >> 32 << 32 : 0) | (Key)tid;
    for (int o = 1; o < per; o <<= 1) {
        const Key q = __shfl_xor_sync(0xFFFFFFFFu, k, o);
        k = q > k ? q : k;
    }
    if (tid % per == 0)
        sm.keys[tid / per] = k;
    if (tid == 0)
        sm.listed = 0, sm.count = 0, sm.limit = 0;
    __syncthreads();
    if (top <= nkeys) {
        int rank = 0;
        for (int j = tid % per; j < nkeys; j += per)
            rank += sm.keys[j] > k;
        for (int o = 1; o < per; o <<= 1)
            rank += __shfl_xor_sync(0xFFFFFFFFu, rank, o);
        if (tid % per == 0 && rank == top - 1)
            sm.limit = k >> 32 << 32;
        __syncthreads();
    }
    Key bound = sm.limit;
    float least = bound ? value_of(bound) : -INFINITY;
    if (best > -INFINITY && best >= least)
        sm.list[atomicAdd(&sm.listed, 1)] = tid;
    __syncthreads();
    // A warp goes over a listed thread's runs, a lane each: a group of as many
    // threads as there are warps, 32 runs of each at a time.  A step of `warps`
    // of the group from `w0` on; the group stays until all its runs are through.
    const int each = (last - first + T_ - 1) / T_, listed = sm.listed, all = T_ >> 5;
    for (int warps = all, l0 = 0, w0 = 0, i0 = 0; l0 < listed;) {
        const int before = sm.count;
        __syncthreads();
        const int w = w0 + warp;
        if (warp < warps && w < all && l0 + w < listed && i0 + lane < each) {
            if (const int u = first + sm.list[l0 + w] + (i0 + lane) * T_; u < last) {
                const uint4 x[1] = {run_at(u)};
                const int c = r.column(u);
                if (key_of(Run<T>::template top_of<1>(x), max(c, 0)) >= bound) {
                    float2 f[V / 2];
                    Run<T>::widen(x[0], f);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float z = j & 1 ? f[j >> 1].y : f[j >> 1].x;
                        if (z >= least && z > -INFINITY)
                            if (const Key q = key_of(z, c + j); q >= bound)
                                if (const int at = atomicAdd(&sm.count, 1); at < kCandidates)
                                    sm.cand[at] = q;
                    }
                }
            }
        }
        __syncthreads();
        const int n = sm.count;
        if (n > kCandidates) {  // not all of them had room: again, in steps that cannot overflow
            __syncthreads();
            if (tid == 0)
                sm.count = before;
            warps = kRound / 32;
            __syncthreads();
            continue;
        }
        w0 += warps;
        if (w0 >= all) {
            w0 = 0, i0 += 32;
            if (i0 >= each)
                i0 = 0, l0 += all;
        }
        if (l0 < listed && n > kKept) {
            sort_out(sm.cand, n, top, sm.sel);
            __syncthreads();
            for (int j = tid; j < top; j += T_)
                sm.cand[j] = sm.sel[j];
            bound = sm.sel[top - 1], least = value_of(bound);
            if (tid == 0)
                sm.count = top;
            if (w0 == 0)
                warps = all;
            __syncthreads();
        }
    }
    sort_out(sm.cand, sm.count, top, sm.sel);
    __syncthreads();
}

// The alternatives of a row from its list, by a block.
__device__ __forceinline__ void put_top(const Args& a, int64_t row, const Key* list, float ref, float log_l)
{
    for (int j = threadIdx.x; j < a.top; j += blockDim.x) {
        const Key k = list[j];
        a.top_logprob[row * a.top + j] = k ? (value_of(k) - ref) * a.scale - log_l : -INFINITY;
        a.top_index[row * a.top + j] = k ? column_of(k) : -1;
    }
}

// Few rows: slices of each in the blocks of a cluster, and the alternatives
// found within the kernel.
template <typename T, bool TOP, int STEP>
__global__ void __launch_bounds__(kThreadsMost, MFX_VOCAB_BLOCKS)
logprobs_fwd(const Args a)
{
    extern __shared__ __align__(16) char dynamic[];
    __shared__ Stats part[8], mine;
    TopSmem& sm = *reinterpret_cast<TopSmem*>(dynamic + (size_t)(a.runs + 2) * 16);
    const int rank = a.cluster > 1 ? (int)cluster_rank() : 0, tid = threadIdx.x;
    for (int64_t row = blockIdx.x / a.cluster; row < a.rows; row += gridDim.x / a.cluster) {
        const T* z = static_cast<const T*>(a.logits) + row * a.ld;
        const Runs<T> r(z, a.n);
        const int share = (r.count + a.cluster - 1) / a.cluster;
        const int first = min(rank * share, r.count), last = min(first + share, r.count);
        Piece<T, STEP> p(r, smem_addr(dynamic), blockDim.x);
        p.set(first, min(first + a.runs, last));
        if (a.eager)
            p.fill();
        const int token = vocab::column_of(a.tokens, a.wide, row, a.n);
        if (token < 0) {  // left out; the same for every block of the cluster
            copies_wait<0>();
            if (rank == 0) {
                if (tid == 0) {
                    a.logprob[row] = 0.0f, a.entropy[row] = 0.0f;
                    if (a.stats)
                        a.stats[3 * row] = 0.0f, a.stats[3 * row + 1] = 0.0f, a.stats[3 * row + 2] = 0.0f;
                }
                if (TOP)
                    for (int j = tid; j < a.top; j += blockDim.x)
                        a.top_logprob[row * a.top + j] = -INFINITY, a.top_index[row * a.top + j] = -1;
            }
            continue;
        }
        if (!a.eager)
            p.fill();
        const float zt = load1(z + token);
        Stats v = no_stats();
        float best = -INFINITY;
        if (tid == 0 && row + a.ahead < a.rows)
            p.prefetch(a.ahead * a.ld);
        scan<T, STEP, true, TOP>(p, a.k, v, best);
        while (p.last < last) {  // (threads read only what they copied)
            p.set(p.last, min(p.last + a.runs, last));
            p.fill();
            scan<T, STEP, true, TOP>(p, a.k, v, best);
        }
        if constexpr (TOP) {
            if (p.first == first)
                find_top(r, first, last, best, a.top, sm, [&](int u) { return lds16(p.at(u)); });
            else
                find_top(r, first, last, best, a.top, sm, [&](int u) { return load_run(z, a.n, r.column(u)); });
        }
        join_block<true>(v, a.k.k2, part, blockDim.x >> 5);
        if (a.cluster > 1)
            join_cluster<true>(v, a.k.k2, &mine, a.cluster);
        if (rank == 0 && (TOP || tid < 32)) {
            const bool empty = v.l == 0.0f;
            const float log_l = logf(v.l), inv = empty ? 0.0f : __fdiv_rn(1.0f, v.l), U = empty ? 0.0f : -kLn2 * v.s * inv;
            if (tid == 0) {
                a.logprob[row] = empty ? -INFINITY : (zt - v.ref) * a.scale - log_l;
                a.entropy[row] = empty ? 0.0f : log_l + U;
                if (a.stats)
                    a.stats[3 * row] = empty ? 0.0f : v.ref, a.stats[3 * row + 1] = inv, a.stats[3 * row + 2] = U;
            }
            if (TOP) {
                const Key* list = sm.sel;
                if (a.cluster > 1) {  // the blocks' lists
                    const int n = a.top * a.cluster;
                    for (int j = tid; j < n; j += blockDim.x) {
                        const uint32_t* q = reinterpret_cast<const uint32_t*>(&sm.sel[j % a.top]);
                        sm.cand[j] = (Key)peer_word(q + 1, j / a.top) << 32 | peer_word(q, j / a.top);
                    }
                    for (int j = tid; j < a.top; j += blockDim.x)
                        sm.keys[j] = 0;
                    __syncthreads();
                    for (int c = tid; c < n; c += blockDim.x) {
                        const Key k = sm.cand[c];
                        int s = 0;
                        for (int j = 0; j < n; ++j)
                            s += sm.cand[j] > k;
                        if (s < a.top && k)
                            sm.keys[s] = k;
                    }
                    __syncthreads();
                    list = sm.keys;
                }
                put_top(a, row, list, v.ref, log_l);
            }
        }
        if (a.cluster > 1) {  // nobody leaves, or goes on, while its list is read
            cluster_arrive(false);
            cluster_wait();
        } else {
            __syncthreads();
        }
    }
}

// Many rows.  TOP: every thread leaves the largest logits of its runs, `gran`
// groups at a time, in the workspace for pick_top (a search within the kernel
// has barriers that stand in the way of the next rows).
template <typename T, bool TOP, int STEP>
__global__ void __launch_bounds__(kThreadsMost, MFX_VOCAB_BLOCKS)
logprobs_rows(const Args a)
{
    extern __shared__ __align__(16) char dynamic[];
    __shared__ Stats part[2][8];
    const int tid = threadIdx.x, T_ = blockDim.x;
    Stream<T, STEP> in(a.in, dynamic);
    int slot = 0, token = vocab::column_of(a.tokens, a.wide, blockIdx.x, a.n), next = -1;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, token = next) {
        if (row + gridDim.x < a.rows)
            next = vocab::column_of(a.tokens, a.wide, row + gridDim.x, a.n);
        if (token < 0) {  // left out
            if (tid == 0) {
                a.logprob[row] = 0.0f, a.entropy[row] = 0.0f;
                if (a.stats)
                    a.stats[3 * row] = 0.0f, a.stats[3 * row + 1] = 0.0f, a.stats[3 * row + 2] = 0.0f;
            }
            continue;
        }
        const float zt = load1(static_cast<const T*>(a.logits) + row * a.ld + token);
        Stats v = no_stats();
        float* ws = TOP ? a.ws + row * (2 + a.chunks * T_) : nullptr;
        int chunk = 0, until = a.gran;
        in.template take_row<true, TOP>(row, a.k, v, [&](int g, bool last, float& best) {
            if (TOP && (last || g + 1 == until)) {
                ws[2 + chunk * T_ + tid] = best;
                best = -INFINITY, until += a.gran, ++chunk;
            }
        });
        if (TOP)
            for (; chunk < a.chunks; ++chunk)
                ws[2 + chunk * T_ + tid] = -INFINITY;
        join_block<true>(v, a.k.k2, part[slot], T_ >> 5);
        slot ^= 1;
        if (tid < 32) {
            const bool empty = v.l == 0.0f;
            const float log_l = logf(v.l), inv = empty ? 0.0f : __fdiv_rn(1.0f, v.l), U = empty ? 0.0f : -kLn2 * v.s * inv;
            if (tid == 0) {
                a.logprob[row] = empty ? -INFINITY : (zt - v.ref) * a.scale - log_l;
                a.entropy[row] = empty ? 0.0f : log_l + U;
                if (a.stats)
                    a.stats[3 * row] = empty ? 0.0f : v.ref, a.stats[3 * row + 1] = inv, a.stats[3 * row + 2] = U;
                if (TOP)
                    ws[0] = v.ref, ws[1] = log_l;
            }
        }
    }
}

// Their alternatives, a warp a row: the search of find_top over the maxima in
// the workspace (part p: chunk p / step of thread p % step), without barriers.
struct WarpTop {
    Key cand[kCandidates];  // the keys of groups first
    Key sel[kMostTop];
    Key limit;
    uint16_t list[kMostListed];
};

__device__ __forceinline__ void warp_sort(const Key* cand, int n, int top, Key* sel)
{
    const int lane = threadIdx.x & 31;
    for (int j = lane; j < top; j += 32)
        if (j >= n)
            sel[j] = 0;
    for (int c = lane; c < n; c += 32) {
        const Key k = cand[c];
        int r = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j)
            r += cand[j] > k;
        if (r < top)
            sel[r] = k;
    }
    __syncwarp();
}

template <typename T>
__global__ void __launch_bounds__(kPickThreads)
pick_top(const Args a)
{
    constexpr int U = 4, B = 16, V = Run<T>::V;
    extern __shared__ __align__(16) char dynamic[];
    WarpTop& sm = reinterpret_cast<WarpTop*>(dynamic)[threadIdx.x >> 5];
    const int lane = threadIdx.x & 31, T_ = a.in.step, parts = a.chunks * T_;
    const int each = 4 * a.gran, shift = 31 - __clz(T_);  // runs of a part; T_ is a power of two
    const int log_reach = a.gran == 1 ? 2 : a.gran == 2 ? 3 : 4, reach = 1 << log_reach;  // lanes of a part: 4, 8 or 16
    const int64_t step = (int64_t)gridDim.x * (kPickThreads / 32);
    pdl_wait();
    for (int64_t row = (int64_t)blockIdx.x * (kPickThreads / 32) + (threadIdx.x >> 5); row < a.rows; row += step) {
        if (vocab::column_of(a.tokens, a.wide, row, a.n) < 0) {
            for (int j = lane; j < a.top; j += 32)
                a.top_logprob[row * a.top + j] = -INFINITY, a.top_index[row * a.top + j] = -1;
            continue;
        }
        const T* z = static_cast<const T*>(a.logits) + row * a.ld;
        const float *ws = a.ws + row * (2 + parts), *maxima = ws + 2 + lane;
        const RowRuns<T> q(z, a.n, T_);
        // the bound: 64 or 128 groups' maxima, 2 or 4 of them a lane
        float sub[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        for (int s = 0; s < parts; s += 32 * B) {  // B loads in flight
            float m[B];
#pragma unroll
            for (int i = 0; i < B; ++i)
                m[i] = s + 32 * i < parts ? maxima[s + 32 * i] : -INFINITY;
#pragma unroll
            for (int i = 0; i < B; ++i)
                sub[i & 3] = fmaxf(sub[i & 3], m[i]);
        }
        const int mine = a.top <= MFX_TOP_FEW ? 2 : 4;
        if (mine == 2)
            sub[0] = fmaxf(sub[0], sub[2]), sub[1] = fmaxf(sub[1], sub[3]);
        Key k[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            k[i] = (sub[i] > -INFINITY ? key_of(sub[i], 0) >> 32 << 32 : 0) | (Key)(32 * i + lane);
            if (i < mine)
                sm.cand[32 * i + lane] = k[i];
        }
        __syncwarp();
        int rank[4] = {0, 0, 0, 0};
        if (mine == 2) {
#pragma unroll 8
            for (int j = 0; j < 64; ++j) {
                const Key o = sm.cand[j];
                rank[0] += o > k[0], rank[1] += o > k[1];
            }
        } else {
#pragma unroll 8
            for (int j = 0; j < 128; ++j) {
                const Key o = sm.cand[j];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    rank[i] += o > k[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < mine && rank[i] == a.top - 1)
                sm.limit = k[i] >> 32 << 32;
        __syncwarp();
        Key bound = sm.limit;
        const float least = bound ? value_of(bound) : -INFINITY;
        int listed = 0;
        for (int s = 0; s < parts; s += 32 * B) {
            float m[B];
#pragma unroll
            for (int i = 0; i < B; ++i)
                m[i] = s + 32 * i < parts ? maxima[s + 32 * i] : -INFINITY;
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const bool on = m[i] > -INFINITY && m[i] >= least;
                const uint32_t who = __ballot_sync(0xFFFFFFFFu, on);
                if (on)
                    sm.list[listed + __popc(who & ((1u << lane) - 1u))] = (uint16_t)(s + 32 * i + lane);
                listed += __popc(who);
            }
        }
        __syncwarp();
        int count = 0;
        // Elements of the lanes' runs (at columns c, if `on`) that reach the
        // bound: few runs have any, and a run's V elements go to V lanes.
        const auto collect = [&](const uint4& w, int c, bool on) {
            const uint4 x[1] = {w};
            const float m = Run<T>::template top_of<1>(x);
            uint32_t left = __ballot_sync(0xFFFFFFFFu, on && m > -INFINITY && key_of(m, max(c, 0)) >= bound);
            while (left) {
                uint32_t mine = left;
#pragma unroll
                for (int n = 0; n < 32 / V; ++n) {
                    if (n < lane / V)
                        mine &= mine - 1;
                    left &= left - 1;
                }
                const int from = mine ? __ffs(mine) - 1 : 0, j = lane % V;
                const uint4 y = make_uint4(__shfl_sync(0xFFFFFFFFu, w.x, from), __shfl_sync(0xFFFFFFFFu, w.y, from),
                                           __shfl_sync(0xFFFFFFFFu, w.z, from), __shfl_sync(0xFFFFFFFFu, w.w, from));
                const int at = __shfl_sync(0xFFFFFFFFu, c, from) + j;
                float2 f[V / 2];
                Run<T>::widen(y, f);
                float e = f[0].x;
#pragma unroll
                for (int n = 1; n < V; ++n)
                    if (n == j)
                        e = n & 1 ? f[n >> 1].y : f[n >> 1].x;
                const Key o = key_of(e, at);
                const bool in = mine && e > -INFINITY && o >= bound;
                const uint32_t who = __ballot_sync(0xFFFFFFFFu, in);
                const int to = count + __popc(who & ((1u << lane) - 1u));
                if (in && to < kCandidates)
                    sm.cand[to] = o;
                count += __popc(who);
            }
        };
        // The vectors at the row's borders, then the listed parts' runs: a group of 8, 16 or 32 parts (U times as many as
        // the lanes reach) stays until all its runs are through, and a step takes `rounds` of its U quarters from r0 on.
        if (q.head() || q.tail()) {
            const bool on = lane == 0 ? q.head() : lane == 1 && q.tail();
            const int c = q.r.column(lane == 0 ? 0 : q.r.count - 1);
            collect(on ? load_run(z, a.n, c) : Run<T>::none(), c, on);
        }
        for (int l0 = 0, r0 = 0, i0 = 0, rounds = U; l0 < listed;) {
            const int before = count;
            uint4 w[U];
            int c[U];
            bool on[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int l = l0 + ((r0 + i) << (5 - log_reach)) + (lane >> log_reach), n = i0 + (lane & (reach - 1));
                on[i] = i < rounds && l < listed && n < each;
                const int id = on[i] ? sm.list[l] : 0;
                const int u = q.whole0 + (id & (T_ - 1)) + ((id >> shift) * each + n) * T_;
                on[i] = on[i] && u < q.whole1;
                c[i] = q.r.column(u);
                w[i] = on[i] ? load_run<T, true>(z, a.n, c[i]) : Run<T>::none();
            }
#pragma unroll
            for (int i = 0; i < U; ++i)
                collect(w[i], c[i], on[i]);
            if (count > kCandidates) {  // not all of them had room: again, in steps that cannot overflow
                count = before, rounds = kRound / 32;
                continue;
            }
            r0 += rounds;
            if (r0 >= U) {
                r0 = 0, i0 += reach;
                if (i0 >= each)
                    i0 = 0, l0 += U << (5 - log_reach);
            }
            if (l0 < listed && count > kKept) {
                __syncwarp();
                warp_sort(sm.cand, count, a.top, sm.sel);
                for (int j = lane; j < a.top; j += 32)
                    sm.cand[j] = sm.sel[j];
                bound = sm.sel[a.top - 1], count = a.top;
                if (r0 == 0)
                    rounds = U;
                __syncwarp();
            }
        }
        __syncwarp();
        warp_sort(sm.cand, count, a.top, sm.sel);
        const float ref = ws[0], log_l = ws[1];
        for (int j = lane; j < a.top; j += 32) {
            const Key o = sm.sel[j];
            a.top_logprob[row * a.top + j] = o ? (value_of(o) - ref) * a.scale - log_l : -INFINITY;
            a.top_index[row * a.top + j] = o ? column_of(o) : -1;
        }
        __syncwarp();
    }
}

struct BwdArgs {
    int64_t rows, ld, ldo;
    int n, chunks, per;  // chunks of a row, runs of a chunk
    const void *logits, *tokens;
    bool wide;
    float scale, k2;
    const float *g, *ge, *stats;
    void* out;
};

template <typename T, int STEP>
__global__ void __launch_bounds__(kThreadsMost)
logprobs_bwd(const BwdArgs a)
{
    constexpr int V = Run<T>::V;
    for (int64_t item = blockIdx.x; item < a.rows * a.chunks; item += gridDim.x) {
        const int64_t row = item / a.chunks;
        const T* z = static_cast<const T*>(a.logits) + row * a.ld;
        T* o = static_cast<T*>(a.out) + row * a.ldo;
        const Runs<T> ro(o, a.n);
        const int u0 = min((int)(item % a.chunks) * a.per, ro.count), u1 = min(u0 + a.per, ro.count);
        const int token = vocab::column_of(a.tokens, a.wide, row, a.n);
        const float ref = a.stats[3 * row], inv = a.stats[3 * row + 1], H = a.stats[3 * row + 2];
        const float g = a.g ? a.g[row] : 0.0f, ge = a.ge ? a.ge[row] : 0.0f;
        if (token < 0 || inv == 0.0f) {
            zero_runs(o, ro, u0, u1, blockDim.x);
            continue;
        }
        const float2 A = f2(-a.scale * inv * fmaf(ge, H, g)), B = f2(-a.scale * inv * ge * kLn2), R = f2(-ref), K = f2(a.k2);
        const float sg = a.scale * g;
        map_runs<T, STEP>(z, o, ro, u0, u1, blockDim.x, [&](const uint4& w, int c) {
            float2 f[V / 2];
            Run<T>::widen(w, f);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                float2 t = mul2(add2(f[j], R), K);
                t = make_float2(at_least_zero_power(t.x), at_least_zero_power(t.y));
                f[j] = mul2(exp2_pair(t), fma2(B, t, A));
            }
            if ((uint32_t)(token - c) < (uint32_t)V) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (c + j == token)
                        (j & 1 ? f[j >> 1].y : f[j >> 1].x) += sg;
            }
            return Run<T>::narrow(f);
        });
    }
}

int status_of(cudaError_t e)
{
    if (e != cudaSuccess)
        cudaGetLastError();  // it is this call's, not the next one's
    return e == cudaSuccess ? launch_status() : cuda_failure(e);
}

template <typename T, bool TOP>
int launch_few(Args a, cudaStream_t s)
{
    const Split sp = split(a.rows, a.n, sizeof(T));
    a.cluster = sp.cluster, a.runs = sp.runs;
    a.eager = a.rows * a.cluster <= sm_count();  // time counts, not bytes
    return status_of(launch_rows(known_step(sp) ? logprobs_fwd<T, TOP, kThreadsMost> : logprobs_fwd<T, TOP, 0>, a, sp,
                                 sp.threads, sp.smem() + (TOP ? sizeof(TopSmem) : 0), s));
}

template <typename T, bool TOP>
int launch_many(const Args& a, cudaStream_t s)
{
    const auto kernel = a.in.step == kThreadsMost ? logprobs_rows<T, TOP, kThreadsMost> : logprobs_rows<T, TOP, 0>;
    const size_t smem = Stream<T, 0>::smem(a.in.step);
    const int64_t room = (int64_t)sm_count() * occupancy(reinterpret_cast<const void*>(kernel), a.in.step, smem);
    kernel<<<(unsigned)(a.rows < room ? a.rows : room), a.in.step, smem, s>>>(a);
    const int st = launch_status();
    if (!TOP || st != MFX_OK)
        return st;
    constexpr int warps = kPickThreads / 32;
    const size_t tops = warps * sizeof(WarpTop);
    const int64_t need = (a.rows + warps - 1) / warps;
    const int64_t places = (int64_t)sm_count() * occupancy(reinterpret_cast<const void*>(pick_top<T>), kPickThreads, tops);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(need < places ? need : places));
    cfg.blockDim = dim3(kPickThreads);
    cfg.dynamicSmemBytes = tops;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return status_of(cudaLaunchKernelEx(&cfg, pick_top<T>, a));
}

template <typename T>
int launch_fwd(Args a, void* workspace, size_t* bytes, cudaStream_t s)
{
    const bool many = streamed(a.rows);
    const int64_t runs = (a.n * (int64_t)sizeof(T) + 15) / 16 + 1;  // with a head and a tail
    a.in = {a.rows, a.ld, a.n, threads_for(runs, kThreadsMost), a.logits, a.tokens, a.wide};
    const int64_t groups = (runs + 4 * a.in.step - 1) / (4 * a.in.step);
    a.gran = (int)((groups + kMostChunks - 1) / kMostChunks);
    a.chunks = (int)((groups + a.gran - 1) / a.gran);
    const size_t need = a.top && many ? (size_t)a.rows * (2 + a.chunks * a.in.step) * sizeof(float) : 0;
    if (bytes && !workspace) {
        *bytes = need;
        return MFX_OK;
    }
    if (!many)
        return a.top ? launch_few<T, true>(a, s) : launch_few<T, false>(a, s);
    if (!a.top)
        return launch_many<T, false>(a, s);
    if (!workspace || !bytes)
        return MFX_ERR_NULL;
    if (*bytes < need || !aligned16(workspace))
        return MFX_ERR_WORKSPACE;
    a.ws = static_cast<float*>(workspace);
    return launch_many<T, true>(a, s);
}

template <typename T>
int launch_bwd(BwdArgs a, cudaStream_t s)
{
    const Chunks c = chunks_of(a.rows, a.n, sizeof(T));
    a.per = c.per, a.chunks = c.count;
    const int64_t need = a.rows * a.chunks;
    const auto kernel = c.threads == kThreadsMost ? logprobs_bwd<T, kThreadsMost> : logprobs_bwd<T, 0>;
    const int64_t room = (int64_t)sm_count() * occupancy(reinterpret_cast<const void*>(kernel), c.threads, 0);
    kernel<<<(unsigned)(need < room ? need : room), c.threads, 0, s>>>(a);
    return launch_status();
}

int check(int dt, int64_t rows, int64_t vocab, int64_t ld, int index_bits, float scale)
{
    if (!valid_dtype(dt) || (index_bits != 32 && index_bits != 64))
        return MFX_ERR_DTYPE;
    if (!row_sizes_ok(rows, vocab, ld))
        return MFX_ERR_SHAPE;
    if (!(scale > 0.0f) || !std::isfinite(scale * kLog2e))
        return MFX_ERR_VALUE;
    return MFX_OK;
}

}  // namespace
}  // namespace vocab
}  // namespace mfx

extern "C" {

int mfx_token_logprobs_fwd(int dt, int64_t rows, int64_t vocab, int64_t ld, const void* logits, int index_bits,
                           const void* tokens, float scale, int64_t top, float* logprob, float* entropy,
                           float* top_logprob, int32_t* top_index, float* stats, void* workspace, size_t* workspace_bytes,
                           void* stream)
{
    using namespace mfx;
    namespace V = vocab;
    if (const int st = V::check(dt, rows, vocab, ld, index_bits, scale); st != MFX_OK)
        return st;
    if (top < 0 || top > V::kMostTop)
        return MFX_ERR_VALUE;
    const bool query = workspace_bytes && !workspace;
    if (rows == 0) {
        if (query)
            *workspace_bytes = 0;
        return MFX_OK;
    }
    if (!query && ((!logits && vocab) || !tokens || !logprob || !entropy || (top && (!top_logprob || !top_index))))
        return MFX_ERR_NULL;
    struct Buf { const void* p; int64_t n; };
    const Buf in[2] = {{logits, V::span(rows, vocab, ld, dtype_bytes(dt))}, {tokens, rows * index_bits / 8}};
    const Buf out[6] = {{logprob, rows * 4}, {entropy, rows * 4}, {stats, rows * 12}, {top_logprob, rows * top * 4},
                        {top_index, rows * top * 4}, {workspace, workspace_bytes ? (int64_t)*workspace_bytes : 0}};
    for (int i = 0; i < 6 && !query; ++i) {
        for (const Buf& b : in)
            if (overlaps(out[i].p, out[i].n, b.p, b.n))
                return MFX_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n))
                return MFX_ERR_ALIAS;
    }
    V::Args a = {};
    a.rows = rows, a.ld = ld, a.n = (int)vocab, a.top = (int)top, a.logits = logits, a.tokens = tokens;
    a.wide = index_bits == 64, a.scale = scale, a.k = V::scaling_of(scale);
    a.logprob = logprob, a.entropy = entropy, a.top_logprob = top_logprob, a.top_index = top_index, a.stats = stats;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dt == MFX_BF16 ? V::launch_fwd<bf16>(a, workspace, workspace_bytes, s)
                          : V::launch_fwd<float>(a, workspace, workspace_bytes, s);
}

int mfx_token_logprobs_bwd(int dt, int64_t rows, int64_t vocab, int64_t ld, const float* g_logprob,
                           const float* g_entropy, const void* logits, int index_bits, const void* tokens,
                           const float* stats, float scale, void* dlogits, int64_t ld_out, void* stream)
{
    using namespace mfx;
    namespace V = vocab;
    if (const int st = V::check(dt, rows, vocab, ld, index_bits, scale); st != MFX_OK)
        return st;
    if (!V::row_sizes_ok(rows, vocab, ld_out))
        return MFX_ERR_SHAPE;
    if (rows == 0 || vocab == 0)
        return MFX_OK;
    if (!logits || !tokens || !stats || !dlogits || (!g_logprob && !g_entropy))
        return MFX_ERR_NULL;
    const int64_t z = dtype_bytes(dt), ob = V::span(rows, vocab, ld_out, z);
    if (!V::rows_alias_ok(dlogits, ld_out, logits, ld, rows, vocab, z) || overlaps(dlogits, ob, tokens, rows * index_bits / 8) ||
        overlaps(dlogits, ob, stats, rows * 12) || overlaps(dlogits, ob, g_logprob, rows * 4) ||
        overlaps(dlogits, ob, g_entropy, rows * 4))
        return MFX_ERR_ALIAS;
    V::BwdArgs a = {};
    a.rows = rows, a.ld = ld, a.ldo = ld_out, a.n = (int)vocab, a.logits = logits, a.tokens = tokens;
    a.wide = index_bits == 64, a.scale = scale, a.k2 = scale * V::kLog2e;
    a.g = g_logprob, a.ge = g_entropy, a.stats = stats, a.out = dlogits;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dt == MFX_BF16 ? V::launch_bwd<bf16>(a, s) : V::launch_bwd<float>(a, s);
}

}  // extern "C"
