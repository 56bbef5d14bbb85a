// moe.cu -- tokens sorted by expert and back, with weights applied, and the
// gradients: what stands before and after the expert MLPs whose weighted
// activations glu.cu and sqrelu.cu compute.
//
// A slot is one choice of one token, s = token * topk + j.  The sorted layout
// has the slots of expert 0 first, then those of expert 1, and so on, in slot
// order within an expert, each expert's rows beginning at a multiple of
// `align`; the rows between are padding.
//
//   permute:     out[row_of[s]] = x[s / topk]            (padding rows zero)
//     backward:  dx[t] = sum_j g[row_of[t, j]]
//   unpermute:   out[t] = sum_j w[t, j] * y[row_of[t, j]]
//     backward:  dy[row_of[s]] = w[s] * g[s / topk]      (padding rows zero)
//                dw[s] = sum_c g[s / topk, c] * y[row_of[s], c]
//
// The maps come from a stable counting sort.  The copies work token by token,
// so that x and g are read once however many rows they go to, and sums over a
// token's rows run in choice order in fp32 registers: no atomics on data, the
// same bits on every run.
//
// What bounds them: HBM, each with its bytes moved once.  At 16384 x 4096 bf16,
// 2 of 8 experts: permute 62 us (403 MB, 6490 GB/s), unpermute 67 us
// (6020 GB/s), its backward with weight gradients 107 us (671 MB,
// 6300 GB/s); fp32 136, 117 and 194 us (5940 to 6930 GB/s).  At 8192 x 2048, 8
// of 128, padding to 16: 51, 50 and 93 us; fp32 143, 108 and 211 us (4340 to
// 5730 GB/s: eight choices at once spill 164 bytes a thread in fp32's unpermute
// and 280 in its backward, 88 and 16 in bf16's).  Widths that are not a multiple
// of 8 take their choices one at a time, a token's row read again for each
// (figures below).
// The sort is two launches and 7 us at 32768 slots, 20 us at 524288 for 4 MB of
// maps: at most 128 blocks, each of which reads all blocks' counts, and then up
// to 16 dependent turns to a warp; with few slots one launch and 4.5 us.
// The copies launch a block per few tokens: blocks that went on from token to
// token, looking the next one's rows up meanwhile, spilled the choices and
// took 86 us in place of 70 for that unpermute.
#include <type_traits>

#include "mfx_device.cuh"
#include "mfx_host.h"

namespace mfx {
namespace {

constexpr int kWarps = kThreads / 32;
constexpr int kMaxExperts = 4096;      // per-warp counters of every expert fit in shared memory
constexpr int64_t kChunk = 2048;       // least slots of a sorting block
constexpr int64_t kMaxChunks = 128;    // most sorting blocks (each reads every block's counts)
constexpr int kMostGroup = 8;          // most choices whose rows a thread has in flight at once
constexpr int kPadRows = 32;           // rows whose padding a block clears

// ---------------------------------------------------------------------------
// Sorting.
// ---------------------------------------------------------------------------
struct Sort {
    int64_t slots, rows, chunk, chunks;
    int experts, capacity, align;
};

// Counts of each expert in each block's slots: hist[block][expert].  Integer
// sums, whose order does not matter.
__global__ void __launch_bounds__(kThreads)
moe_count(const int32_t* __restrict__ expert_of, int* __restrict__ hist, const Sort p)
{
    extern __shared__ int count[];
    for (int e = threadIdx.x; e < p.experts; e += kThreads)
        count[e] = 0;
    __syncthreads();
    const int64_t s0 = (int64_t)blockIdx.x * p.chunk, s1 = s0 + p.chunk < p.slots ? s0 + p.chunk : p.slots;
    for (int64_t s = s0 + threadIdx.x; s < s1; s += kThreads) {
        const int e = expert_of[s];
        if (e >= 0 && e < p.experts)
            atomicAdd(&count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kThreads)
        hist[(int64_t)blockIdx.x * p.experts + e] = count[e];
    pdl_launch_dependents();
}

// Exclusive sum over the block's threads; *total gets the sum of all.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* total)
{
    __shared__ int64_t part[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o)
            sum += u;
    }
    if (lane == 31)
        part[warp] = sum;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        before += i < warp ? part[i] : 0;
        all += part[i];
    }
    *total = all;
    return before + sum - v;
}

// Places one block's slots.  Every block forms the experts' totals and first
// rows from all blocks' counts (a single block counts its own slots), then
// ranks its slots: a warp takes a contiguous part of them, 32 at a time, and
// the lanes of one expert rank themselves by lane.
__global__ void __launch_bounds__(kThreads)
moe_place(const int32_t* __restrict__ expert_of, const int* __restrict__ hist, int32_t* __restrict__ row_of,
          int32_t* __restrict__ slot_of, int32_t* __restrict__ offsets, int32_t* __restrict__ counts, const Sort p)
{
    extern __shared__ int sm[];
    const int E = p.experts;
    int* total = sm;             // slots of the expert
    int* next = sm + E;          // rank of the block's first slot of the expert
    int* first = sm + 2 * E;     // the expert's first row
    int* ahead = sm + 3 * E;     // [warp][expert]: counts, then ranks
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < (3 + kWarps) * E; i += kThreads)
        sm[i] = 0;
    __syncthreads();
    // the warps' own slots, counted while the other kernel may still run
    const int64_t s0 = (int64_t)blockIdx.x * p.chunk, s1 = s0 + p.chunk < p.slots ? s0 + p.chunk : p.slots;
    const int64_t per = p.chunk / kWarps, w0 = s0 + warp * per, w1 = w0 + per < s1 ? w0 + per : s1;
    for (int64_t s = w0 + lane; s < w1; s += 32) {
        const int e = expert_of[s];
        if (e >= 0 && e < E)
            atomicAdd(&ahead[warp * E + e], 1);
    }
    pdl_wait();
    if (p.chunks > 1) {
        const int groups = E < kThreads ? kThreads / E : 1;
        for (int i = threadIdx.x; i < E * groups; i += kThreads) {
            const int e = i % E;
            int all = 0, before = 0;
#pragma unroll 8
            for (int64_t c = i / E; c < p.chunks; c += groups) {
                const int v = hist[c * E + e];
                all += v;
                before += c < (int64_t)blockIdx.x ? v : 0;
            }
            atomicAdd(&total[e], all);
            atomicAdd(&next[e], before);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) {
        int sum = 0;
        for (int w = 0; w < kWarps; ++w) {
            const int v = ahead[w * E + e];
            ahead[w * E + e] = next[e] + sum;
            sum += v;
        }
        if (p.chunks == 1)
            total[e] = sum;
        if (p.capacity > 0 && total[e] > p.capacity)
            total[e] = p.capacity;
    }
    __syncthreads();
    // first rows: a thread sums consecutive experts' aligned sizes
    const int each = (E + kThreads - 1) / kThreads, e0 = threadIdx.x * each;
    int64_t mine = 0, rows_used;
    for (int e = e0; e < e0 + each && e < E; ++e)
        mine += ((int64_t)total[e] + p.align - 1) / p.align * p.align;
    int64_t at = block_scan(mine, &rows_used);
    for (int e = e0; e < e0 + each && e < E; ++e) {
        first[e] = (int)at;
        at += ((int64_t)total[e] + p.align - 1) / p.align * p.align;
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e < E; e += kThreads) {
            offsets[e] = first[e];
            counts[e] = total[e];
        }
        if (threadIdx.x == 0)
            offsets[E] = (int32_t)rows_used;
    }
    // padding rows of this block's experts, and its part of the rows past the last expert's
    for (int e = blockIdx.x * kWarps + warp; e < E; e += gridDim.x * kWarps) {
        const int64_t end = e + 1 < E ? first[e + 1] : rows_used;
        for (int64_t r = (int64_t)first[e] + total[e] + lane; r < end; r += 32)
            if (r < p.rows)
                slot_of[r] = -1;
    }
    for (int64_t r = rows_used + (int64_t)blockIdx.x * kThreads + threadIdx.x; r < p.rows;
         r += (int64_t)gridDim.x * kThreads)
        slot_of[r] = -1;
    int* rank = ahead + warp * E;
    for (int64_t base = w0; base < w1; base += 32) {
        const int64_t s = base + lane;
        int e = s < w1 ? expert_of[s] : -1;
        if (e < 0 || e >= E)
            e = -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
        const int before = __popc(same & ((1u << lane) - 1u));
        int mine_rank = 0;
        if (e >= 0)
            mine_rank = rank[e] + before;
        __syncwarp();
        if (e >= 0 && before == 0)
            rank[e] += __popc(same);
        __syncwarp();
        if (s < w1) {
            int64_t r = -1;
            if (e >= 0 && (p.capacity <= 0 || mine_rank < p.capacity))
                r = (int64_t)first[e] + mine_rank;
            if (r >= p.rows)
                r = -1;
            row_of[s] = (int32_t)r;
            if (r >= 0)
                slot_of[r] = (int32_t)s;
        }
    }
}

// ---------------------------------------------------------------------------
// Rows in chunks of 8 elements.  FAST: a width that is a multiple of 8 and
// 16-byte aligned buffers, so every chunk is one (fp32: two) 16-byte access.
// Otherwise the chunk grid follows the destination row's alignment; sources
// are read through the aligned vectors that cover them, and the ragged ends
// element by element (4096 x 4099, 4 of 60 experts: 42, 62 and 116 us for
// permute, unpermute and its backward, of which 25, 25 and 45 are bytes; by
// 4-byte words instead 74, 145, 193).
// ---------------------------------------------------------------------------
template <typename T>
struct Span {
    const T* base;
    uintptr_t lo, hi;  // bytes of the whole buffer
};

template <typename T>
__host__ __device__ __forceinline__ Span<T> span_of(const T* p, int64_t n)
{
    return Span<T>{p, reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + (uintptr_t)n * sizeof(T)};
}

// Elements [k0, k0 + 8) of the row at `row` (a row of `cols`) in fp32; those
// outside [0, cols) are zero.
template <typename T, bool FAST>
__device__ __forceinline__ void load_cols(const Span<T>& b, int64_t row, int64_t k0, int64_t cols, float (&f)[8])
{
    const T* p = b.base + row * cols + k0;
    Raw8<T> raw;
    if (FAST) {
        ld8(p, raw);
        widen8(raw, f);
    } else if (k0 >= 0 && k0 + 8 <= cols && in_vectors(p, b.lo, b.hi)) {
        ld8_any(p, raw);
        widen8(raw, f);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f[j] = k0 + j >= 0 && k0 + j < cols ? load1(p + j) : 0.0f;
    }
}

template <typename T, bool FAST>
__device__ __forceinline__ void store_cols(T* base, int64_t row, int64_t k0, int64_t cols, const float (&f)[8])
{
    T* p = base + row * cols + k0;
    if (FAST || (k0 >= 0 && k0 + 8 <= cols && (reinterpret_cast<uintptr_t>(p) & 15u) == 0)) {
        Raw8<T> raw;
        narrow8(f, raw);
        st8(p, raw);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k0 + j >= 0 && k0 + j < cols)
                store1(p + j, f[j]);
    }
}

// Offset of a row's chunk grid: chunks begin where the destination is 16-byte
// aligned.
template <typename T, bool FAST>
__device__ __forceinline__ int phase_of(const T* base, int64_t row, int64_t cols)
{
    return FAST ? 0 : (int)((reinterpret_cast<uintptr_t>(base + row * cols) / sizeof(T)) & 7u);
}

struct Moe {
    int64_t tokens, cols, rows, slots;
    int topk;
    int team;             // threads on a token's columns (warps of one block)
    int col_blocks;       // teams over a token's columns
    int64_t pad_blocks;   // blocks that clear padding: the first ones, so that theirs is not a tail
    int64_t token_blocks; // blocks that work on tokens
};

// The token and the columns' part of a thread's team; false where there is none.
struct Place {
    int64_t token;
    int index, count;  // the thread among the token's threads
    int part;          // which of the token's teams
};
__device__ __forceinline__ bool place(const Moe& m, Place& p)
{
    const int64_t team = ((int64_t)blockIdx.x - m.pad_blocks) * (kThreads / m.team) + threadIdx.x / m.team;
    p.token = m.col_blocks == 1 ? team : team / m.col_blocks;
    p.part = (int)(team - p.token * m.col_blocks);
    p.index = p.part * m.team + threadIdx.x % m.team;
    p.count = m.col_blocks * m.team;
    return p.token < m.tokens;
}

__device__ __forceinline__ int row_or_none(int r, int64_t rows) { return r >= 0 && r < rows ? r : -1; }

// Zeroes the padding rows among [32 b, 32 b + 32): a warp looks at four rows
// and clears those without a slot.
template <typename T, bool FAST>
__device__ __forceinline__ void clear_padding(T* out, float* out_weight, const int32_t* __restrict__ slot_of,
                                              const Moe& m, int64_t b)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kEach = kPadRows / kWarps;
    const int64_t r0 = b * kPadRows + warp * kEach, r = r0 + lane;
    bool pad = false;
    if (lane < kEach && r < m.rows) {
        const int s = slot_of[r];
        pad = s < 0 || s >= m.slots;
        if (pad && out_weight)
            out_weight[r] = 0.0f;
    }
    const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (unsigned left = __ballot_sync(0xFFFFFFFFu, pad); left; left &= left - 1) {
        const int64_t row = r0 + __ffs(left) - 1;
        for (int64_t k = (int64_t)lane * 8 - phase_of<T, FAST>(out, row, m.cols); k < m.cols; k += 256)
            store_cols<T, FAST>(out, row, k, m.cols, zero);
    }
}

// ---------------------------------------------------------------------------
// Permute: a token's chunk is read once and written to each of its rows.
// Two thirds of its bytes or more are writes.
// ---------------------------------------------------------------------------
template <typename T, bool FAST>
__global__ void __launch_bounds__(kThreads)
moe_permute(const T* __restrict__ x, const int32_t* __restrict__ row_of, const int32_t* __restrict__ slot_of,
            const float* __restrict__ weight, T* __restrict__ out, float* __restrict__ out_weight, const Moe m)
{
    if ((int64_t)blockIdx.x < m.pad_blocks) {
        clear_padding<T, FAST>(out, out_weight, slot_of, m, blockIdx.x);
        return;
    }
    Place p;
    if (!place(m, p))
        return;
    const int32_t* rows = row_of + p.token * m.topk;
    if (weight && p.part == 0)
        for (int j = threadIdx.x % m.team; j < m.topk; j += m.team) {
            const int r = row_or_none(rows[j], m.rows);
            if (r >= 0)
                out_weight[r] = weight[p.token * m.topk + j];
        }
    const T* src = x + p.token * m.cols;
    if constexpr (FAST) {
        const int64_t step = (int64_t)p.count * 8;
        for (int64_t k = (int64_t)p.index * 8; k < m.cols; k += 2 * step) {
            const bool two = k + step < m.cols;
            Raw8<T> raw[2];
            ld8(src + k, raw[0]);
            if (two)
                ld8(src + k + step, raw[1]);
            for (int j = 0; j < m.topk; ++j) {
                const int r = row_or_none(rows[j], m.rows);
                if (r < 0)
                    continue;
                st8(out + r * m.cols + k, raw[0]);
                if (two)
                    st8(out + r * m.cols + k + step, raw[1]);
            }
        }
    } else {
        const Span<T> all = span_of(x, m.tokens * m.cols);
        const int64_t step = (int64_t)p.count * 8;
        for (int j = 0; j < m.topk; ++j) {
            const int r = row_or_none(rows[j], m.rows);
            if (r < 0)
                continue;
            for (int64_t k = (int64_t)p.index * 8 - phase_of<T, FAST>(out, r, m.cols); k < m.cols; k += step) {
                float f[8];
                load_cols<T, FAST>(all, p.token, k, m.cols, f);
                store_cols<T, FAST>(out, r, k, m.cols, f);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Unpermute (and permute's backward, without weights): a token's rows added
// in choice order, G of them in flight at a time.  A choice without a row
// reads row 0 instead, which is not added.  Five blocks an SM for small G: the
// loads of a thread wait for the row numbers, so it is warps that keep HBM busy
// (two choices spill 40 bytes a thread at five and more at six: 102 us in place
// of 70 at 16384 x 4096).
// ---------------------------------------------------------------------------
template <typename T, bool FAST, int G>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : G <= 4 ? 5 : 4)
moe_unpermute(const T* __restrict__ y, const int32_t* __restrict__ row_of, const float* __restrict__ weight,
              const float* __restrict__ row_weight, T* __restrict__ out, float* __restrict__ dweight, const Moe m)
{
    Place p;
    if (!place(m, p))
        return;
    const int32_t* rows = row_of + p.token * m.topk;
    if (dweight && p.part == 0)
        for (int j = threadIdx.x % m.team; j < m.topk; j += m.team) {
            const int r = row_or_none(rows[j], m.rows);
            dweight[p.token * m.topk + j] = r >= 0 ? row_weight[r] : 0.0f;
        }
    const auto choice = [&](int j, int& r, float& w) {
        r = j < m.topk ? row_or_none(rows[j], m.rows) : -1;
        w = weight && r >= 0 ? weight[p.token * m.topk + j] : 1.0f;
    };
    if constexpr (FAST) {
        constexpr int V = G <= 2 ? 2 : 1;  // chunks at once
        const int64_t step = (int64_t)p.count * 8;
        for (int64_t k = (int64_t)p.index * 8; k < m.cols; k += V * step) {
            float acc[V][8] = {};
            for (int j0 = 0; j0 < m.topk; j0 += G) {
                int r[G];
                float w[G];
#pragma unroll
                for (int i = 0; i < G; ++i)
                    choice(j0 + i, r[i], w[i]);
                Raw8<T> raw[G][V];
                if (m.rows > 0) {
#pragma unroll
                    for (int i = 0; i < G; ++i)
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            ld8(y + (r[i] < 0 ? 0 : r[i]) * m.cols + (k + v * step < m.cols ? k + v * step : k), raw[i][v]);
                }
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    if (r[i] < 0)
                        continue;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float f[8];
                        widen8(raw[i][v], f);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            acc[v][c] = fmaf(w[i], f[c], acc[v][c]);
                    }
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v == 0 || k + v * step < m.cols)
                    store_cols<T, FAST>(out, p.token, k + v * step, m.cols, acc[v]);
        }
    } else {
        const Span<T> all = span_of(y, m.rows * m.cols);
        const int64_t step = (int64_t)p.count * 8;
        for (int64_t k = (int64_t)p.index * 8 - phase_of<T, FAST>(out, p.token, m.cols); k < m.cols; k += step) {
            float acc[8] = {};
#pragma unroll 4
            for (int j = 0; j < m.topk; ++j) {
                int r;
                float w, f[8];
                choice(j, r, w);
                if (r < 0)
                    continue;
                load_cols<T, FAST>(all, r, k, m.cols, f);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    acc[c] = fmaf(w, f[c], acc[c]);
            }
            store_cols<T, FAST>(out, p.token, k, m.cols, acc);
        }
    }
}

// ---------------------------------------------------------------------------
// Unpermute's backward: a team reads a token's g and its rows of y once,
// writes w * g to the rows of dy and keeps the dot products, G choices at a
// time.
// ---------------------------------------------------------------------------
// Sums G values a lane over the warp, halving what a lane keeps with each
// exchange: afterwards lane l has the sum of value index_of(l).
template <int G>
__device__ __forceinline__ float warp_sums(float (&v)[G])
{
    const int lane = threadIdx.x & 31;
    int n = G;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < G / 2; ++i)
                if (i < n) {
                    const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
                }
        } else {
            v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
        }
    }
    return v[0];
}
template <int G>
__device__ __forceinline__ int index_of(int lane)
{
    return G == 8 ? lane >> 2 : G == 4 ? lane >> 3 : G == 2 ? lane >> 4 : 0;
}

template <typename T, bool FAST, int G>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && G <= 4 ? 4 : 3)
moe_unpermute_bwd(const T* __restrict__ g, const T* __restrict__ y, const int32_t* __restrict__ row_of,
                  const int32_t* __restrict__ slot_of, const float* __restrict__ weight, T* __restrict__ dy,
                  float* __restrict__ dweight, const Moe m)
{
    if ((int64_t)blockIdx.x < m.pad_blocks) {
        clear_padding<T, FAST>(dy, nullptr, slot_of, m, blockIdx.x);
        return;
    }
    __shared__ float part[kWarps][G];
    Place p;
    const bool live = place(m, p);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = m.team >> 5;
    const T* gs = g + p.token * m.cols;
    for (int j0 = 0; j0 < m.topk; j0 += G) {
        int r[G];
        float w[G], dot[G];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const int64_t s = p.token * m.topk + j0 + i;
            r[i] = live && j0 + i < m.topk ? row_or_none(row_of[s], m.rows) : -1;
            w[i] = weight && r[i] >= 0 ? weight[s] : 1.0f;
            dot[i] = 0.0f;
        }
        if constexpr (FAST) {
            constexpr int V = G <= 2 ? 2 : 1;  // chunks at once
            const int64_t step = (int64_t)p.count * 8;
            for (int64_t k0 = (int64_t)p.index * 8; live && k0 < m.cols; k0 += V * step) {
                Raw8<T> raw[V][G], graw[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int64_t k = k0 + v * step < m.cols ? k0 + v * step : k0;
                    ld8(gs + k, graw[v]);
                    if (dweight && m.rows > 0) {
#pragma unroll
                        for (int i = 0; i < G; ++i)
                            ld8(y + (r[i] < 0 ? 0 : r[i]) * m.cols + k, raw[v][i]);
                    }
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int64_t k = k0 + v * step;
                    if (v > 0 && k >= m.cols)
                        continue;
                    float gf[8];
                    widen8(graw[v], gf);
#pragma unroll
                    for (int i = 0; i < G; ++i) {
                        if (r[i] < 0)
                            continue;
                        float f[8];
                        if (dweight) {
                            widen8(raw[v][i], f);
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                dot[i] = fmaf(gf[c], f[c], dot[i]);
                        }
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            f[c] = gf[c] * w[i];
                        store_cols<T, FAST>(dy, r[i], k, m.cols, f);
                    }
                }
            }
        } else {
            const Span<T> tokens = span_of(g, m.tokens * m.cols), all = span_of(y, m.rows * m.cols);
            const int64_t step = (int64_t)p.count * 8;
#pragma unroll
            for (int i = 0; i < G; ++i) {
                if (r[i] < 0)
                    continue;
                for (int64_t k = (int64_t)p.index * 8 - phase_of<T, FAST>(dy, r[i], m.cols); k < m.cols; k += step) {
                    float gf[8], f[8];
                    load_cols<T, FAST>(tokens, p.token, k, m.cols, gf);
                    if (dweight) {
                        load_cols<T, FAST>(all, r[i], k, m.cols, f);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            dot[i] = fmaf(gf[c], f[c], dot[i]);
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        f[c] = gf[c] * w[i];
                    store_cols<T, FAST>(dy, r[i], k, m.cols, f);
                }
            }
        }
        if (!dweight)
            continue;
        const float sum = warp_sums<G>(dot);
        const int i = index_of<G>(lane);
        const bool first = (lane & (32 / G - 1)) == 0;  // one lane of each value
        if (warps == 1) {
            if (first && live && j0 + i < m.topk)
                dweight[p.token * m.topk + j0 + i] = sum;
            continue;
        }
        if (first)
            part[warp][i] = sum;
        __syncthreads();
        const int t = threadIdx.x % m.team;
        if (live && t < G && j0 + t < m.topk) {
            float v = 0.0f;
            for (int q = 0; q < warps; ++q)
                v += part[warp + q][t];  // t < G <= 32: the team's first warp
            dweight[p.token * m.topk + j0 + t] = v;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
// Sizes shared by the copies.
int check(int dt, int64_t tokens, int64_t topk, int64_t cols, int64_t rows)
{
    if (!valid_dtype(dt))
        return MFX_ERR_DTYPE;
    int64_t slots = 0, n = 0;
    if (tokens < 0 || topk < 0 || cols < 0 || rows < 0 || rows > INT32_MAX || topk > INT32_MAX ||
        !mul_ok(tokens, topk, &slots) || slots > INT32_MAX || !mul_ok(tokens, cols, &n) || !mul_ok(n, 16, &n) ||
        !mul_ok(rows, cols, &n) || !mul_ok(n, 16, &n))
        return MFX_ERR_SHAPE;
    return MFX_OK;
}

// A team of up to a block's threads on each token, two chunks a thread, and
// (`split`) several teams where few tokens would leave SMs idle.
Moe plan(int64_t tokens, int64_t topk, int64_t cols, int64_t rows, bool split, bool clear)
{
    Moe m = {};
    m.tokens = tokens, m.cols = cols, m.rows = rows, m.slots = tokens * topk, m.topk = (int)topk;
    const int64_t chunks = (cols + 7) / 8, fill = (int64_t)sm_count() * 8 * kThreads;
    m.team = kThreads;
    while (m.team > 32 && (int64_t)m.team >= chunks)
        m.team /= 2;
    while (m.team < kThreads && tokens * m.team * 2 <= fill && (int64_t)m.team < chunks)
        m.team *= 2;
    m.col_blocks = 1;
    while (split && (int64_t)m.team * m.col_blocks < chunks && tokens * m.team * m.col_blocks < fill)
        ++m.col_blocks;
    const int64_t teams = kThreads / m.team;
    m.token_blocks = (tokens * m.col_blocks + teams - 1) / teams;
    m.pad_blocks = clear ? (rows + kPadRows - 1) / kPadRows : 0;
    return m;
}

// Calls f(G) with the choices taken at once, as a type: the least power of two
// that has them all, up to kMostGroup.
template <typename F>
int by_group(int64_t topk, F f)
{
    if (topk <= 1)
        return f(std::integral_constant<int, 1>{});
    if (topk <= 2)
        return f(std::integral_constant<int, 2>{});
    if (topk <= 4)
        return f(std::integral_constant<int, 4>{});
    return f(std::integral_constant<int, kMostGroup>{});
}

bool fast_rows(int64_t cols, const void* a, const void* b, const void* c = nullptr)
{
    return cols % 8 == 0 && aligned16(a) && aligned16(b) && aligned16(c);
}

}  // namespace
}  // namespace mfx

extern "C" int64_t mfx_moe_rows(int64_t tokens, int64_t topk, int64_t experts, int64_t align)
{
    using namespace mfx;
    int64_t slots = 0, pad = 0;
    if (tokens < 0 || topk < 0 || experts < 0 || align < 1 || !mul_ok(tokens, topk, &slots) ||
        !mul_ok(slots < experts ? slots : experts, align - 1, &pad) || slots > INT64_MAX - pad)
        return -1;
    return slots + pad;
}

extern "C" int mfx_moe_sort(int64_t tokens, int64_t topk, int64_t experts, int64_t align, int64_t capacity,
                            int64_t rows, const int32_t* expert_of, int32_t* row_of, int32_t* slot_of,
                            int32_t* offsets, int32_t* counts, void* workspace, size_t* workspace_bytes, void* stream)
{
    using namespace mfx;
    int64_t slots = 0;
    if (tokens < 0 || topk < 0 || experts < 1 || experts > kMaxExperts || align < 1 || align > INT32_MAX ||
        capacity < 0 || capacity > INT32_MAX || rows < 0 || rows > INT32_MAX || !mul_ok(tokens, topk, &slots) ||
        slots > INT32_MAX)
        return MFX_ERR_SHAPE;
    // what the layout may need; a capacity bounds every expert
    const int64_t need = mfx_moe_rows(tokens, topk, experts, align);
    int64_t capped = INT64_MAX;
    if (capacity > 0)
        capped = experts * ((capacity + align - 1) / align * align);
    if (need < 0 || rows < (need < capped ? need : capped))
        return MFX_ERR_SHAPE;
    Sort p = {};
    p.slots = slots, p.rows = rows, p.experts = (int)experts, p.capacity = (int)capacity, p.align = (int)align;
    p.chunk = kChunk;
    while ((slots + p.chunk - 1) / p.chunk > kMaxChunks)
        p.chunk *= 2;
    p.chunks = slots > p.chunk ? (slots + p.chunk - 1) / p.chunk : 1;
    const size_t bytes = p.chunks > 1 ? (size_t)(p.chunks * experts) * sizeof(int) : 0;
    if (!workspace_bytes && (workspace || bytes > 0))
        return MFX_ERR_NULL;
    if (!workspace && workspace_bytes) {
        *workspace_bytes = bytes;
        return MFX_OK;
    }
    if (workspace && (*workspace_bytes < bytes || !aligned16(workspace)))
        return MFX_ERR_WORKSPACE;
    if ((slots > 0 && (!expert_of || !row_of)) || (rows > 0 && !slot_of) || !offsets || !counts)
        return MFX_ERR_NULL;
    const void* const out[] = {row_of, slot_of, offsets, counts, workspace};
    const int64_t size[] = {4 * slots, 4 * rows, 4 * (experts + 1), 4 * experts, (int64_t)bytes};
    for (int i = 0; i < 5; ++i) {
        if (overlaps(out[i], size[i], expert_of, 4 * slots))
            return MFX_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i], size[i], out[j], size[j]))
                return MFX_ERR_ALIAS;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int* hist = static_cast<int*>(workspace);
    if (p.chunks > 1) {
        moe_count<<<(unsigned)p.chunks, kThreads, sizeof(int) * experts, s>>>(expert_of, hist, p);
        const int st = launch_status();
        if (st != MFX_OK)
            return st;
    }
    const size_t smem = sizeof(int) * (size_t)(3 + kWarps) * (size_t)experts;
    occupancy((const void*)moe_place, kThreads, smem);  // raises the kernel's shared-memory limit where needed
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.chunks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.chunks > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, moe_place, expert_of, (const int*)hist, row_of, slot_of, offsets,
                                             counts, (const Sort)p);
    return e == cudaSuccess ? launch_status() : cuda_failure(e);
}

namespace mfx {
namespace {
int permute(int dt, int64_t tokens, int64_t topk, int64_t cols, int64_t rows, const void* x, const int32_t* row_of,
            const int32_t* slot_of, const float* weight, void* out, float* out_weight, void* stream)
{
    const Moe m = plan(topk > 0 ? tokens : 0, topk, cols, rows, true, true);
    const int64_t blocks = m.pad_blocks + m.token_blocks;
    if (blocks > INT32_MAX)
        return MFX_ERR_SHAPE;
    const auto go = [&](auto t, auto fast) {
        using T = decltype(t);
        moe_permute<T, decltype(fast)::value><<<(unsigned)blocks, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
            static_cast<const T*>(x), row_of, slot_of, weight, static_cast<T*>(out), out_weight, m);
        return launch_status();
    };
    if (fast_rows(cols, x, out))
        return dt == MFX_BF16 ? go(bf16{}, std::true_type{}) : go(float{}, std::true_type{});
    return dt == MFX_BF16 ? go(bf16{}, std::false_type{}) : go(float{}, std::false_type{});
}
}  // namespace
}  // namespace mfx

extern "C" int mfx_moe_permute_fwd(int dt, int64_t tokens, int64_t topk, int64_t cols, int64_t rows, const void* x,
                                   const int32_t* row_of, const int32_t* slot_of, const float* weight, void* out,
                                   float* out_weight, void* stream)
{
    using namespace mfx;
    const int st = check(dt, tokens, topk, cols, rows);
    if (st != MFX_OK || rows == 0 || (cols == 0 && !weight && !out_weight))
        return st;
    const int64_t slots = tokens * topk, e = dtype_bytes(dt), ob = rows * cols * e, xb = tokens * cols * e;
    // rows without columns still carry their weights
    if ((cols > 0 && !out) || !slot_of || (slots > 0 && ((cols > 0 && !x) || !row_of)) || (weight && !out_weight) ||
        (out_weight && !weight && slots > 0))
        return MFX_ERR_NULL;
    if (overlaps(out, ob, x, xb) || overlaps(out, ob, row_of, 4 * slots) || overlaps(out, ob, slot_of, 4 * rows) ||
        overlaps(out, ob, weight, 4 * slots) || overlaps(out_weight, 4 * rows, out, ob) ||
        overlaps(out_weight, 4 * rows, x, xb) || overlaps(out_weight, 4 * rows, weight, 4 * slots) ||
        overlaps(out_weight, 4 * rows, row_of, 4 * slots) || overlaps(out_weight, 4 * rows, slot_of, 4 * rows))
        return MFX_ERR_ALIAS;
    return permute(dt, tokens, topk, cols, rows, x, row_of, slot_of, weight, out, out_weight, stream);
}

namespace mfx {
namespace {
// out[t] = sum_j w[t, j] * y[row_of[t, j]], and the gather of per-row weights.
int unpermute(int dt, int64_t tokens, int64_t topk, int64_t cols, int64_t rows, const void* y, const int32_t* row_of,
              const float* weight, const float* row_weight, void* out, float* dweight, void* stream)
{
    const int st = check(dt, tokens, topk, cols, rows);
    if (st != MFX_OK || tokens == 0 || (cols == 0 && !row_weight && !dweight))
        return st;
    const int64_t slots = tokens * topk, e = dtype_bytes(dt), ob = tokens * cols * e, yb = rows * cols * e;
    if ((cols > 0 && !out) || (slots > 0 && !row_of) || (slots > 0 && yb > 0 && !y) || (row_weight && !dweight) ||
        (dweight && !row_weight && slots > 0 && rows > 0))
        return MFX_ERR_NULL;
    if (overlaps(out, ob, y, yb) || overlaps(out, ob, row_of, 4 * slots) || overlaps(out, ob, weight, 4 * slots) ||
        overlaps(out, ob, row_weight, 4 * rows) || overlaps(dweight, 4 * slots, out, ob) ||
        overlaps(dweight, 4 * slots, y, yb) || overlaps(dweight, 4 * slots, row_of, 4 * slots) ||
        overlaps(dweight, 4 * slots, row_weight, 4 * rows))
        return MFX_ERR_ALIAS;
    const Moe m = plan(tokens, topk, cols, rows, true, false);
    if (m.token_blocks > INT32_MAX)
        return MFX_ERR_SHAPE;
    const auto go = [&](auto t, auto fast) {
        return by_group(topk, [&](auto group) {
            using T = decltype(t);
            moe_unpermute<T, decltype(fast)::value, decltype(group)::value>
                <<<(unsigned)m.token_blocks, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
                    static_cast<const T*>(y), row_of, weight, row_weight, static_cast<T*>(out), dweight, m);
            return launch_status();
        });
    };
    if (fast_rows(cols, y, out))
        return dt == MFX_BF16 ? go(bf16{}, std::true_type{}) : go(float{}, std::true_type{});
    return dt == MFX_BF16 ? go(bf16{}, std::false_type{}) : go(float{}, std::false_type{});
}
}  // namespace
}  // namespace mfx

extern "C" int mfx_moe_permute_bwd(int dt, int64_t tokens, int64_t topk, int64_t cols, int64_t rows, const void* g,
                                   const int32_t* row_of, const float* g_weight, void* dx, float* dweight,
                                   void* stream)
{
    return mfx::unpermute(dt, tokens, topk, cols, rows, g, row_of, nullptr, g_weight, dx, dweight, stream);
}

extern "C" int mfx_moe_unpermute_fwd(int dt, int64_t tokens, int64_t topk, int64_t cols, int64_t rows, const void* y,
                                     const int32_t* row_of, const float* weight, void* out, void* stream)
{
    return mfx::unpermute(dt, tokens, topk, cols, rows, y, row_of, weight, nullptr, out, nullptr, stream);
}

extern "C" int mfx_moe_unpermute_bwd(int dt, int64_t tokens, int64_t topk, int64_t cols, int64_t rows, const void* g,
                                     const void* y, const int32_t* row_of, const int32_t* slot_of,
                                     const float* weight, void* dy, float* dweight, void* stream)
{
    using namespace mfx;
    const int st = check(dt, tokens, topk, cols, rows);
    if (st != MFX_OK)
        return st;
    const int64_t slots = tokens * topk, e = dtype_bytes(dt), gb = tokens * cols * e, yb = rows * cols * e;
    if ((rows == 0 || cols == 0) && (slots == 0 || !dweight))
        return MFX_OK;
    if (cols == 0)  // sums of no products
        return cudaMemsetAsync(dweight, 0, 4 * (size_t)slots, static_cast<cudaStream_t>(stream)) == cudaSuccess
                   ? MFX_OK
                   : cuda_failure(cudaGetLastError());
    if ((rows > 0 && (!dy || !slot_of)) || (slots > 0 && (!g || !row_of)) || (dweight && rows > 0 && slots > 0 && !y))
        return MFX_ERR_NULL;
    const void* const in[] = {g, y, row_of, slot_of, weight};
    const int64_t size[] = {gb, yb, 4 * slots, 4 * rows, 4 * slots};
    for (int i = 0; i < 5; ++i)
        if (overlaps(dy, yb, in[i], size[i]) || overlaps(dweight, 4 * slots, in[i], size[i]))
            return MFX_ERR_ALIAS;
    if (overlaps(dy, yb, dweight, 4 * slots))
        return MFX_ERR_ALIAS;
    if (!weight && !dweight)  // the rows of g as they are
        return permute(dt, tokens, topk, cols, rows, g, row_of, slot_of, nullptr, dy, nullptr, stream);
    const Moe m = plan(topk > 0 ? tokens : 0, topk, cols, rows, false, true);
    const int64_t blocks = m.pad_blocks + m.token_blocks;
    if (blocks > INT32_MAX)
        return MFX_ERR_SHAPE;
    const auto go = [&](auto t, auto fast) {
        return by_group(topk, [&](auto group) {
            using T = decltype(t);
            moe_unpermute_bwd<T, decltype(fast)::value, decltype(group)::value>
                <<<(unsigned)blocks, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
                    static_cast<const T*>(g), static_cast<const T*>(y), row_of, slot_of, weight, static_cast<T*>(dy),
                    dweight, m);
            return launch_status();
        });
    };
    if (fast_rows(cols, g, dy, dweight ? y : nullptr))
        return dt == MFX_BF16 ? go(bf16{}, std::true_type{}) : go(float{}, std::true_type{});
    return dt == MFX_BF16 ? go(bf16{}, std::false_type{}) : go(float{}, std::false_type{});
}
