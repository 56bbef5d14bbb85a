// distill.cu -- distillation from a teacher's top logits: the loss, its
// gradient, and both in one call.
//
// Per row, with p = softmax(scale * z) over the student's logits and the
// teacher's K logits t_j at columns c_j (negative: no entry),
//   q_j = exp(scale * t_j) / sum_i exp(scale * t_i)   or   exp(scale * t_j - lse),
//   loss = sum_j q_j (log q_j - log p[c_j]),
//   dz = g * scale * (Q p - sum of q_j at its columns),   Q = sum_j q_j,
// the second form of q where the teacher's own log of the sum over its whole
// vocabulary is given (Q < 1: the columns beyond the list count for nothing).
// The student's softmax is one pass over its row; the gradient is a second one
// that writes exp(t) * (Q / l) everywhere and then, after a barrier, puts right
// the at most K columns of the list, each by the first entry that names it.
// In the call that does both, a block (or the blocks of a cluster) makes the
// second pass as soon as it has the first, when L2 still has the row: HBM sees
// one read and one write.
#include "vocab.cuh"

#include <cmath>

namespace mfx {
namespace vocab {
namespace {

constexpr int kMostEntries = 1024;

struct Args {
    int64_t rows, ld, ldo;
    int n, K, cluster, chunks, per;
    const void *logits, *index, *teacher;
    bool wide, t_bf16;
    float scale, k2;
    const float *lse, *g;
    float *loss, *stats;
    const float* stats_in;
    void* out;
};

// A row's list in shared memory: columns (-1: no entry), q, and the student's
// logits there.
struct List {
    int* col;
    float *q, *z;
    __device__ List(char* p, int K) : col(reinterpret_cast<int*>(p)), q(reinterpret_cast<float*>(p) + K), z(q + K) {}
};

__device__ __forceinline__ float teacher_at(const Args& a, int64_t i)
{
    return a.t_bf16 ? load1(static_cast<const bf16*>(a.teacher) + i) : load1(static_cast<const float*>(a.teacher) + i);
}

// A sum (or maximum) over the block, the same bits in every thread.
template <bool MAX>
__device__ __forceinline__ float over_block(float v, float* part)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = MAX ? fmaxf(v, w) : v + w;
    }
    if (blockDim.x > 32) {
        __syncthreads();  // what the last call left is read
        if ((threadIdx.x & 31) == 0)
            part[threadIdx.x >> 5] = v;
        __syncthreads();
        const int lane = threadIdx.x & 31;
        v = lane < (int)(blockDim.x >> 5) ? part[lane] : (MAX ? -INFINITY : 0.0f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
            v = MAX ? fmaxf(v, w) : v + w;
        }
    }
    return v;
}

// What q is formed from: q_j = exp((t_j - ref) * scale) * coef = exp((t_j - ref) * scale + log_coef).
struct Teacher {
    float ref, coef, log_coef, Q;
    bool any;
};

__device__ __forceinline__ float q_of(const Args& a, float t, const Teacher& w)
{
    return exp2_approx(at_least_zero_power((t - w.ref) * a.k2)) * w.coef;
}

// Reads the row's list (columns, the student's logits there if Z, q) and forms
// the teacher's statistics.
template <typename T, bool Z>
__device__ __forceinline__ Teacher read_list(const Args& a, int64_t row, const T* z, const List& l, float* part)
{
    float top = -INFINITY;
    bool any = false;
    for (int j = threadIdx.x; j < a.K; j += blockDim.x) {
        const int c = column_of(a.index, a.wide, row * a.K + j, a.n);
        const float t = c >= 0 ? teacher_at(a, row * a.K + j) : -INFINITY;
        l.col[j] = c, l.q[j] = t;
        any |= c >= 0;
        if (Z)
            l.z[j] = c >= 0 ? load1(z + c) : -INFINITY;
        top = fmaxf(top, t);
    }
    top = over_block<true>(top, part);
    Teacher w = {top == -INFINITY ? 0.0f : top, 0.0f, 0.0f, 0.0f, false};
    w.any = __syncthreads_or(any);
    float sum = 0.0f;
    for (int j = threadIdx.x; j < a.K; j += blockDim.x) {
        const float e = exp2_approx(at_least_zero_power((l.q[j] - w.ref) * a.k2));
        l.q[j] = e;
        sum += e;
    }
    sum = over_block<false>(sum, part);
    if (a.lse) {
        w.log_coef = fmaf(w.ref, a.scale, -a.lse[row]);
        w.coef = expf(w.log_coef);
    } else {
        w.log_coef = sum == 0.0f ? 0.0f : -logf(sum);
        w.coef = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
    }
    w.Q = sum * w.coef;
    for (int j = threadIdx.x; j < a.K; j += blockDim.x)
        l.q[j] *= w.coef;
    return w;
}

// The loss from the list and the row's statistics (thread 0 writes it).
__device__ __forceinline__ void put_loss(const Args& a, int64_t row, const List& l, const Teacher& w, const Stats& v,
                                         float* part)
{
    const float log_l = logf(v.l);
    float sum = 0.0f;
    for (int j = threadIdx.x; j < a.K; j += blockDim.x) {
        const float q = l.q[j];
        if (l.col[j] >= 0 && q != 0.0f) {
            // log q from t itself, and not as a logarithm of q
            const float logq = fmaf(teacher_at(a, row * a.K + j) - w.ref, a.scale, w.log_coef);
            const float logp = v.l == 0.0f ? -INFINITY : fmaf(l.z[j] - v.ref, a.scale, -log_l);
            sum = fmaf(q, logq - logp, sum);
        }
    }
    sum = over_block<false>(sum, part);
    if (threadIdx.x == 0)
        a.loss[row] = sum;
}

// The gradient of runs [u0, u1) of an output row; `ratio` is Q / l (0: zeros).
template <typename T>
__device__ __forceinline__ void put_grads(const Args& a, const T* z, T* o, int u0, int u1, const List& l, float ref,
                                          float ratio, float g)
{
    const Runs<T> ro(o, a.n);
    const float A = g * a.scale * ratio;
    for (int u = u0 + threadIdx.x; u < u1; u += blockDim.x) {
        const int c = ro.column(u);
        float f[8];
        if (ratio == 0.0f) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[j] = 0.0f;
        } else {
            load8_at(z, a.n, c, f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[j] = A * exp2_approx(at_least_zero_power((f[j] - ref) * a.k2));
        }
        store_run(ro, o, u, f);
    }
    if (ratio == 0.0f)
        return;
    __syncthreads();
    const int c0 = ro.column(u0), c1 = ro.column(u1);
    for (int j = threadIdx.x; j < a.K; j += blockDim.x) {
        const int c = l.col[j];
        if (c < 0 || c < c0 || c >= c1)
            continue;
        float q = 0.0f;
        bool mine = true;
        for (int i = 0; i < a.K; ++i)
            if (l.col[i] == c) {
                mine &= i >= j;
                q += l.q[i];
            }
        if (mine) {
            const float e = exp2_approx(at_least_zero_power((l.z[j] - ref) * a.k2));
            store1(o + c, g * a.scale * fmaf(e, ratio, -q));
        }
    }
}

template <typename T, bool GRAD>
__global__ void __launch_bounds__(512)
distill_fwd(const Args a)
{
    extern __shared__ __align__(16) char dynamic[];
    __shared__ Stats part[32], mine;
    __shared__ float fpart[32];
    const List l(dynamic, a.K);
    const int rank = a.cluster > 1 ? (int)cluster_rank() : 0, tid = threadIdx.x;
    for (int64_t row = blockIdx.x / a.cluster; row < a.rows; row += gridDim.x / a.cluster) {
        const T* z = static_cast<const T*>(a.logits) + row * a.ld;
        T* o = GRAD ? static_cast<T*>(a.out) + row * a.ldo : nullptr;
        const Teacher w = read_list<T, true>(a, row, z, l, fpart);
        Stats v = no_stats();
        if (w.any) {  // the same for every block of the cluster
            Pick best;
            v = scan<T, false, 4>(Share<T>(Runs<T>(z, a.n), rank, a.cluster), a.k2, best);
            v = join_block(v, a.k2, part);
        }
        if (a.cluster > 1)
            v = join_cluster(v, a.k2, &mine, a.cluster);
        else
            __syncthreads();
        const float ratio = v.l == 0.0f ? 0.0f : __fdiv_rn(w.Q, v.l);
        if (rank == 0) {
            put_loss(a, row, l, w, v, fpart);
            if (!GRAD && a.stats && tid == 0)
                a.stats[4 * row] = v.ref, a.stats[4 * row + 1] = ratio, a.stats[4 * row + 2] = w.ref, a.stats[4 * row + 3] = w.coef;
        }
        if (GRAD) {
            const Runs<T> ro(o, a.n);
            const int per = (ro.count + a.cluster - 1) / a.cluster, u0 = min(rank * per, ro.count);
            put_grads<T>(a, z, o, u0, min(u0 + per, ro.count), l, v.ref, ratio, a.g[row]);
        }
        if (a.cluster > 1)
            cluster_sync();
        else
            __syncthreads();
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
distill_bwd(const Args a)
{
    extern __shared__ __align__(16) char dynamic[];
    const List l(dynamic, a.K);
    for (int64_t item = blockIdx.x; item < a.rows * a.chunks; item += gridDim.x) {
        const int64_t row = item / a.chunks;
        const T* z = static_cast<const T*>(a.logits) + row * a.ld;
        T* o = static_cast<T*>(a.out) + row * a.ldo;
        const float ref = a.stats_in[4 * row], ratio = a.stats_in[4 * row + 1];
        const Teacher w = {a.stats_in[4 * row + 2], a.stats_in[4 * row + 3], 0.0f, 0.0f, true};
        const Runs<T> ro(o, a.n);
        const int u0 = (int)(item % a.chunks) * a.per, u1 = min(u0 + a.per, ro.count);
        const int c0 = ro.column(u0), c1 = ro.column(u1);
        for (int j = threadIdx.x; j < a.K; j += blockDim.x) {
            const int c = column_of(a.index, a.wide, row * a.K + j, a.n);
            const bool here = c >= 0 && c >= c0 && c < c1;
            l.col[j] = here ? c : -1;
            l.q[j] = here ? q_of(a, teacher_at(a, row * a.K + j), w) : 0.0f;
            l.z[j] = here ? load1(z + c) : 0.0f;
        }
        __syncthreads();
        put_grads<T>(a, z, o, u0, u1, l, ref, ratio, a.g[row]);
        __syncthreads();
    }
}

template <typename T, bool GRAD>
int launch_fwd(Args a, cudaStream_t s)
{
    const Split sp = split(a.rows, a.n);
    a.cluster = sp.cluster;
    const cudaError_t e = launch_rows(distill_fwd<T, GRAD>, a, sp, (size_t)a.K * 12, s);
    return e == cudaSuccess ? launch_status() : cuda_failure(e);
}

template <typename T>
int launch_bwd(Args a, cudaStream_t s)
{
    const int64_t runs = (a.n + 14) / 8;
    const int threads = threads_for(runs, 256);
    a.per = threads * 8;
    a.chunks = (int)((runs + a.per - 1) / a.per);
    const size_t smem = (size_t)a.K * 12;
    const int64_t need = a.rows * a.chunks;
    const int64_t room = (int64_t)sm_count() * occupancy(reinterpret_cast<const void*>(distill_bwd<T>), threads, smem);
    distill_bwd<T><<<(unsigned)(need < room ? need : room), threads, smem, s>>>(a);
    return launch_status();
}

// Arguments that the three calls share.
int check(int dt, int t_dt, int64_t rows, int64_t vocab, int64_t ld, int64_t k, int index_bits, float scale)
{
    if (!valid_dtype(dt) || !valid_dtype(t_dt) || (index_bits != 32 && index_bits != 64))
        return MFX_ERR_DTYPE;
    if (!row_sizes_ok(rows, vocab, ld) || k < 0 || k > kMostEntries)
        return MFX_ERR_SHAPE;
    if (!(scale > 0.0f) || std::isinf(scale))
        return MFX_ERR_VALUE;
    return MFX_OK;
}

int run(int dt, int t_dt, int64_t rows, int64_t vocab, int64_t ld, int64_t k, const void* logits, int index_bits,
        const void* index, const void* teacher, const float* lse, float scale, const float* g, float* loss, float* stats,
        const float* stats_in, void* out, int64_t ldo, void* stream)
{
    if (out && !row_sizes_ok(rows, vocab, ldo))
        return MFX_ERR_SHAPE;
    if (rows == 0 || (!loss && vocab == 0))
        return MFX_OK;
    if ((vocab && !logits) || (k && (!index || !teacher)))
        return MFX_ERR_NULL;
    const int64_t z = dtype_bytes(dt), ob = span(rows, vocab, ldo, z);
    struct Buf { const void* p; int64_t n; };
    const Buf in[7] = {{logits, span(rows, vocab, ld, z)}, {index, rows * k * index_bits / 8},
                       {teacher, rows * k * dtype_bytes(t_dt)}, {lse, rows * 4}, {g, rows * 4}, {stats_in, rows * 16}, {nullptr, 0}};
    const Buf outs[3] = {{loss, rows * 4}, {stats, rows * 16}, {out, ob}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 7; ++j)
            if (!(i == 2 && j == 0) && overlaps(outs[i].p, outs[i].n, in[j].p, in[j].n))
                return MFX_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return MFX_ERR_ALIAS;
    }
    if (out && !rows_alias_ok(out, ldo, logits, ld, rows, vocab, z))
        return MFX_ERR_ALIAS;
    Args a = {};
    a.rows = rows, a.ld = ld, a.ldo = ldo, a.n = (int)vocab, a.K = (int)k, a.logits = logits, a.index = index;
    a.teacher = teacher, a.wide = index_bits == 64, a.t_bf16 = t_dt == MFX_BF16, a.scale = scale;
    a.k2 = scale * kLog2e, a.lse = lse, a.g = g, a.loss = loss, a.stats = stats, a.stats_in = stats_in, a.out = out;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!loss)
        return dt == MFX_BF16 ? launch_bwd<bf16>(a, s) : launch_bwd<float>(a, s);
    if (out)
        return dt == MFX_BF16 ? launch_fwd<bf16, true>(a, s) : launch_fwd<float, true>(a, s);
    return dt == MFX_BF16 ? launch_fwd<bf16, false>(a, s) : launch_fwd<float, false>(a, s);
}

}  // namespace
}  // namespace vocab
}  // namespace mfx

extern "C" {

int mfx_topk_distill_fwd(int dt, int t_dt, int64_t rows, int64_t vocab, int64_t ld, int64_t k, const void* logits,
                         int index_bits, const void* index, const void* teacher, const float* teacher_lse, float scale,
                         float* loss, float* stats, void* stream)
{
    using namespace mfx;
    if (const int st = vocab::check(dt, t_dt, rows, vocab, ld, k, index_bits, scale); st != MFX_OK)
        return st;
    if (rows && !loss)
        return MFX_ERR_NULL;
    return vocab::run(dt, t_dt, rows, vocab, ld, k, logits, index_bits, index, teacher, teacher_lse, scale, nullptr,
                      loss, stats, nullptr, nullptr, 0, stream);
}

int mfx_topk_distill_bwd(int dt, int t_dt, int64_t rows, int64_t vocab, int64_t ld, int64_t k, const float* g,
                         const void* logits, int index_bits, const void* index, const void* teacher, const float* stats,
                         float scale, void* dlogits, int64_t ld_out, void* stream)
{
    using namespace mfx;
    if (const int st = vocab::check(dt, t_dt, rows, vocab, ld, k, index_bits, scale); st != MFX_OK)
        return st;
    if (rows && vocab && (!g || !stats || !dlogits))
        return MFX_ERR_NULL;
    return vocab::run(dt, t_dt, rows, vocab, ld, k, logits, index_bits, index, teacher, nullptr, scale, g, nullptr,
                      nullptr, stats, dlogits, ld_out, stream);
}

int mfx_topk_distill_fwd_bwd(int dt, int t_dt, int64_t rows, int64_t vocab, int64_t ld, int64_t k, const void* logits,
                             int index_bits, const void* index, const void* teacher, const float* teacher_lse,
                             const float* weight, float scale, float* loss, void* dlogits, int64_t ld_out, void* stream)
{
    using namespace mfx;
    if (const int st = vocab::check(dt, t_dt, rows, vocab, ld, k, index_bits, scale); st != MFX_OK)
        return st;
    if (rows && (!loss || !weight || (vocab && !dlogits)))
        return MFX_ERR_NULL;
    return vocab::run(dt, t_dt, rows, vocab, ld, k, logits, index_bits, index, teacher, teacher_lse, scale, weight, loss,
                      nullptr, nullptr, dlogits, ld_out, stream);
}

}  // extern "C"
