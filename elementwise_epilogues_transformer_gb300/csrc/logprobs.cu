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
#include "vocab.cuh"

#include <cmath>

namespace mfx {
namespace vocab {
namespace {

constexpr int kMostTop = 64;    // alternatives
constexpr int kSpare = 1024;    // candidates beside those of one round

struct Args {
    int64_t rows, ld;
    int n, top, cluster;
    const void *logits, *tokens;
    bool wide;
    float scale, k2;
    float *logprob, *entropy, *top_logprob, *stats;
    int32_t* top_index;
};

// Shared memory of the search for alternatives, for T threads.
struct TopSmem {
    Pick* best;   // [T] of every thread
    Pick* four;   // [T / 4] of every four
    int* list;    // [T] threads
    Pick* cand;   // [8 T + kSpare]
    Pick* sel;    // [kMostTop], the block's alternatives in order
    int* count;   // [4]: threads listed, threads that count, candidates
    Pick* limit;  // [2]
    __device__ explicit TopSmem(char* p, int T)
    {
        best = reinterpret_cast<Pick*>(p), four = best + T, cand = four + T / 4, sel = cand + 8 * T + kSpare;
        limit = sel + kMostTop, list = reinterpret_cast<int*>(limit + 2), count = list + T;
    }
    static size_t bytes(int T) { return (size_t)(T + T / 4 + 8 * T + kSpare + kMostTop + 2) * sizeof(Pick) + (T + 4) * 4; }
};

__device__ __forceinline__ Pick shfl_xor(Pick p, int o)
{
    return {__shfl_xor_sync(0xFFFFFFFFu, p.v, o), __shfl_xor_sync(0xFFFFFFFFu, p.i, o)};
}

// How many of list[0, n) are better than p.
__device__ __forceinline__ int rank_in(const Pick* list, int n, const Pick& p)
{
    int r = 0;
    for (int i = 0; i < n; ++i)
        r += better(list[i], p);
    return r;
}

// The `top` best of cand[0, n) in order to sel, (-inf, -1) behind them; a
// barrier before the call and after it.
__device__ __forceinline__ void sort_out(const Pick* cand, int n, int top, Pick* sel)
{
    for (int j = threadIdx.x; j < top; j += blockDim.x)
        if (j >= n)
            sel[j] = {-INFINITY, -1};
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
        const Pick p = cand[c];
        if (const int r = rank_in(cand, n, p); r < top)
            sel[r] = p;
    }
}

// The block's `top` best columns above -inf, to sm.sel in order.
//
// The top-th best of the threads' own best columns bounds the top-th best of
// all from below, and only the `top` threads whose best reaches it can hold a
// column that does.  Their runs alone are read again (from L2, all at once)
// for the few columns that reach the bound.  The order is strict (equal
// logits go by column), so the number of such threads does not depend on the
// data.  A round adds at most 8 candidates a thread; if they pile up (rows
// built so that a few threads hold most large logits), they are cut to the
// `top` best between rounds.
template <typename T>
__device__ __forceinline__ void find_top(const Share<T>& sh, const Pick best, int top, const TopSmem& sm)
{
    const int tid = threadIdx.x, T_ = blockDim.x;
    // a first bound from every four threads' best: fewer to compare
    const Pick none = {-INFINITY, 0x7FFFFFFF};
    Pick four = best;
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        const Pick q = shfl_xor(four, o);
        if (better(q, four))
            four = q;
    }
    if ((tid & 3) == 0)
        sm.four[tid >> 2] = four;
    if (tid < 4)
        sm.count[tid] = 0;
    if (tid < 2)
        sm.limit[tid] = none;
    __syncthreads();
    if (T_ / 4 >= top) {
        if (tid < T_ / 4) {
            const Pick mine = sm.four[tid];
            if (rank_in(sm.four, T_ / 4, mine) == top - 1)
                sm.limit[0] = mine;
        }
        __syncthreads();
        if (!better(sm.limit[0], best))
            sm.best[atomicAdd(&sm.count[0], 1)] = best;
        __syncthreads();
        const int n = sm.count[0];  // at most four for each of `top`
        for (int j = tid; j < n; j += T_) {
            const Pick mine = sm.best[j];
            if (rank_in(sm.best, n, mine) == top - 1)
                sm.limit[1] = mine;
        }
        __syncthreads();
    }
    const Pick limit = sm.limit[1];
    if (best.v > -INFINITY && !better(limit, best))
        sm.list[atomicAdd(&sm.count[1], 1)] = tid;
    __syncthreads();
    const int each = (sh.last - sh.first + T_ - 1) / T_ + 2, items = sm.count[1] * each;
    for (int base = 0; base < items; base += T_) {
        if (base + tid < items) {
            const int t = sm.list[(base + tid) / each], i = (base + tid) % each;
            int u = -1;
            if (i < each - 2)
                u = sh.first + t + i * T_ < sh.last ? sh.first + t + i * T_ : -1;
            else if (t == 0)
                u = i == each - 2 ? (sh.head ? 0 : -1) : (sh.tail ? sh.r.count - 1 : -1);
            if (u >= 0) {
                float z[8];
                sh.r.load(u, z);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const Pick p = {z[j], sh.r.column(u) + j};
                    if (z[j] > -INFINITY && !better(limit, p))
                        sm.cand[atomicAdd(&sm.count[2], 1)] = p;
                }
            }
        }
        __syncthreads();
        if (const int n = sm.count[2]; base + T_ < items && n > kSpare) {
            sort_out(sm.cand, n, top, sm.sel);
            __syncthreads();
            for (int j = tid; j < top; j += T_)
                sm.cand[j] = sm.sel[j];
            if (tid == 0)
                sm.count[2] = top;
            __syncthreads();
        }
    }
    sort_out(sm.cand, sm.count[2], top, sm.sel);
    __syncthreads();
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(512)
logprobs_fwd(const Args a)
{
    extern __shared__ __align__(16) char dynamic[];
    __shared__ Stats part[32], mine;
    const TopSmem sm(dynamic, blockDim.x);
    const int rank = a.cluster > 1 ? (int)cluster_rank() : 0, tid = threadIdx.x;
    for (int64_t row = blockIdx.x / a.cluster; row < a.rows; row += gridDim.x / a.cluster) {
        const int token = column_of(a.tokens, a.wide, row, a.n);
        if (token < 0) {  // left out; the same for every block of the cluster
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
        const T* z = static_cast<const T*>(a.logits) + row * a.ld;
        const float zt = load1(z + token);
        const Share<T> sh(Runs<T>(z, a.n), rank, a.cluster);
        Pick best;
        Stats v = scan<T, TOP, 4>(sh, a.k2, best);
        if (TOP)
            find_top(sh, best, a.top, sm);
        v = join_block(v, a.k2, part);
        if (a.cluster > 1)
            v = join_cluster(v, a.k2, &mine, a.cluster);
        if (rank == 0) {
            const bool empty = v.l == 0.0f;
            const float log_l = logf(v.l), inv = empty ? 0.0f : __fdiv_rn(1.0f, v.l), U = empty ? 0.0f : -kLn2 * v.s * inv;
            if (tid == 0) {
                a.logprob[row] = empty ? -INFINITY : (zt - v.ref) * a.scale - log_l;
                a.entropy[row] = empty ? 0.0f : log_l + U;
                if (a.stats)
                    a.stats[3 * row] = empty ? 0.0f : v.ref, a.stats[3 * row + 1] = inv, a.stats[3 * row + 2] = U;
            }
            if (TOP) {
                if (a.cluster > 1) {
                    for (int j = tid; j < a.top * a.cluster; j += blockDim.x) {
                        const Pick* p = &sm.sel[j % a.top];
                        sm.cand[j] = {__uint_as_float(peer_word(&p->v, j / a.top)), (int)peer_word(&p->i, j / a.top)};
                        if (sm.cand[j].i < 0)
                            sm.cand[j].i = (int)kMostColumns + j;  // nothing: behind all, each in its own place
                    }
                    __syncthreads();
                }
                const Pick* list = sm.sel;
                if (a.cluster > 1) {
                    list = sm.best;  // free by now; at least as long as `top`
                    for (int c = tid; c < a.top * a.cluster; c += blockDim.x) {
                        const Pick p = sm.cand[c];
                        if (const int r = rank_in(sm.cand, a.top * a.cluster, p); r < a.top)
                            sm.best[r] = p;
                    }
                    __syncthreads();
                }
                for (int j = tid; j < a.top; j += blockDim.x) {
                    const Pick p = list[j];
                    const bool none = !(p.v > -INFINITY);
                    a.top_logprob[row * a.top + j] = none ? -INFINITY : (p.v - v.ref) * a.scale - log_l;
                    a.top_index[row * a.top + j] = none ? -1 : p.i;
                }
            }
        }
        if (a.cluster > 1)
            cluster_sync();
        else
            __syncthreads();
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

template <typename T>
__global__ void __launch_bounds__(256)
logprobs_bwd(const BwdArgs a)
{
    for (int64_t item = blockIdx.x; item < a.rows * a.chunks; item += gridDim.x) {
        const int64_t row = item / a.chunks;
        const T* z = static_cast<const T*>(a.logits) + row * a.ld;
        T* o = static_cast<T*>(a.out) + row * a.ldo;
        const Runs<T> ro(o, a.n);
        const int token = column_of(a.tokens, a.wide, row, a.n);
        const float ref = a.stats[3 * row], inv = a.stats[3 * row + 1], U = a.stats[3 * row + 2];
        const float g = a.g ? a.g[row] : 0.0f, ge = a.ge ? a.ge[row] : 0.0f;
        const float A = -a.scale * inv * fmaf(ge, U, g), B = -a.scale * inv * ge * kLn2;
        const bool none = token < 0 || inv == 0.0f;
        const int u0 = (int)(item % a.chunks) * a.per, u1 = min(u0 + a.per, ro.count);
        for (int u = u0 + threadIdx.x; u < u1; u += blockDim.x) {
            const int c = ro.column(u);
            float f[8];
            if (none) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    f[j] = 0.0f;
            } else {
                load8_at(z, a.n, c, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float t = at_least_zero_power((f[j] - ref) * a.k2);
                    f[j] = exp2_approx(t) * fmaf(B, t, A);
                    if (c + j == token)
                        f[j] = fmaf(a.scale, g, f[j]);
                }
            }
            store_run(ro, o, u, f);
        }
    }
}

template <typename T, bool TOP>
int launch_fwd(Args a, cudaStream_t s)
{
    const Split sp = split(a.rows, a.n);
    a.cluster = sp.cluster;
    const cudaError_t e = launch_rows(logprobs_fwd<T, TOP>, a, sp, TOP ? TopSmem::bytes(sp.threads) : 0, s);
    return e == cudaSuccess ? launch_status() : cuda_failure(e);
}

template <typename T>
int launch_bwd(BwdArgs a, cudaStream_t s)
{
    const int64_t runs = (a.n + 14) / 8;  // with a head and a tail
    const int threads = threads_for(runs, 256);
    a.per = threads * 8;
    a.chunks = (int)((runs + a.per - 1) / a.per);
    const int64_t need = a.rows * a.chunks;
    const int64_t room = (int64_t)sm_count() * occupancy(reinterpret_cast<const void*>(logprobs_bwd<T>), threads, 0);
    logprobs_bwd<T><<<(unsigned)(need < room ? need : room), threads, 0, s>>>(a);
    return launch_status();
}

int check(int dt, int64_t rows, int64_t vocab, int64_t ld, int index_bits, float scale)
{
    if (!valid_dtype(dt) || (index_bits != 32 && index_bits != 64))
        return MFX_ERR_DTYPE;
    if (!row_sizes_ok(rows, vocab, ld))
        return MFX_ERR_SHAPE;
    if (!(scale > 0.0f) || std::isinf(scale))
        return MFX_ERR_VALUE;
    return MFX_OK;
}

}  // namespace
}  // namespace vocab
}  // namespace mfx

extern "C" {

int mfx_token_logprobs_fwd(int dt, int64_t rows, int64_t vocab, int64_t ld, const void* logits, int index_bits,
                           const void* tokens, float scale, int64_t top, float* logprob, float* entropy,
                           float* top_logprob, int32_t* top_index, float* stats, void* stream)
{
    using namespace mfx;
    namespace V = vocab;
    if (const int st = V::check(dt, rows, vocab, ld, index_bits, scale); st != MFX_OK)
        return st;
    if (top < 0 || top > V::kMostTop)
        return MFX_ERR_VALUE;
    if (rows == 0)
        return MFX_OK;
    if ((!logits && vocab) || !tokens || !logprob || !entropy || (top && (!top_logprob || !top_index)))
        return MFX_ERR_NULL;
    struct Buf { const void* p; int64_t n; };
    const Buf in[2] = {{logits, V::span(rows, vocab, ld, dtype_bytes(dt))}, {tokens, rows * index_bits / 8}};
    const Buf out[5] = {{logprob, rows * 4}, {entropy, rows * 4}, {stats, rows * 12}, {top_logprob, rows * top * 4}, {top_index, rows * top * 4}};
    for (int i = 0; i < 5; ++i) {
        for (const Buf& b : in)
            if (overlaps(out[i].p, out[i].n, b.p, b.n))
                return MFX_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n))
                return MFX_ERR_ALIAS;
    }
    V::Args a = {};
    a.rows = rows, a.ld = ld, a.n = (int)vocab, a.top = (int)top, a.logits = logits, a.tokens = tokens;
    a.wide = index_bits == 64, a.scale = scale, a.k2 = scale * V::kLog2e;
    a.logprob = logprob, a.entropy = entropy, a.top_logprob = top_logprob, a.top_index = top_index, a.stats = stats;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dt == MFX_BF16)
        return top ? V::launch_fwd<bf16, true>(a, s) : V::launch_fwd<bf16, false>(a, s);
    return top ? V::launch_fwd<float, true>(a, s) : V::launch_fwd<float, false>(a, s);
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
