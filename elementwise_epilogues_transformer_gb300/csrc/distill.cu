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
// In the call that does both, the blocks of a cluster keep the row in shared
// memory between the passes: HBM sees one read and one write.  The list is the
// work of a warp of its own, while the others' copies are under way (by the
// warps that read the row: 519 us instead of 425 at that step).
//
// What bounds them: HBM.  4096x131072 bf16 with 64 columns: both 363 us (5920
// GB/s, 0.87 of the copy rate), where the forward (171) and the backward (333)
// take 504; what is lost to the copy rate is the cluster's barriers and the
// power formed twice (16 instructions an element).  1001x32003 with 16: both
// 27 us, forward 13, backward 25 (19 of bytes).
#include "vocab.cuh"

#include <cmath>

namespace mfx {
namespace vocab {
namespace {

constexpr int kMostEntries = 1024;

struct Args {
    int64_t rows, ld, ldo, ahead;
    int n, K, cluster, runs, chunks, per;
    const void *logits, *index, *teacher;
    bool wide, t_bf16;
    float scale, k2;
    Scaling k;
    const float *lse, *g;
    float *loss, *stats;
    const float* stats_in;
    void* out;
    StreamArgs in;
};

// A row's list in shared memory: columns (-1: no entry), q, and the teacher's
// logits, then log q, then the student's logits.
struct List {
    int* col;
    float *q, *z;
    __device__ List(char* p, int K) : col(reinterpret_cast<int*>(p)), q(reinterpret_cast<float*>(p) + K), z(q + K) {}
};

__device__ __forceinline__ float teacher_at(const Args& a, int64_t i)
{
    return a.t_bf16 ? load1(static_cast<const bf16*>(a.teacher) + i) : load1(static_cast<const float*>(a.teacher) + i);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// What q is formed from: q_j = exp((t_j - ref) * scale) * coef = exp((t_j - ref) * scale + log_coef),
// their sum Q, and how many of the row's entries the list holds.
struct Teacher {
    float ref, coef, log_coef, Q;
    int n;
};

__device__ __forceinline__ float power_of(const Args& a, float t, float ref)
{
    return exp2_approx(at_least_zero_power((t - ref) * a.k2));
}

// One warp reads the row's entries and leaves those of columns [lo, hi) at the
// list's front, in order.  Q is over all entries; `given` has ref and coef
// from the forward (no Q then).
template <bool GIVEN>
__device__ __forceinline__ Teacher read_list(const Args& a, int64_t row, const List& l, int lo, int hi, Teacher w)
{
    const int lane = threadIdx.x & 31;
    float top = -INFINITY, sum = 0.0f;
    for (int j = lane; j < a.K; j += 32) {
        const int c = column_of(a.index, a.wide, row * a.K + j, a.n);
        const float at = teacher_at(a, row * a.K + j), t = c >= 0 ? at : -INFINITY;  // both loads at once
        l.col[j] = c, l.z[j] = t;
        top = fmaxf(top, t);
    }
    if (!GIVEN) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        w.ref = top == -INFINITY ? 0.0f : top;
        for (int j = lane; j < a.K; j += 32)
            sum += power_of(a, l.z[j], w.ref);
        sum = warp_sum(sum);
        if (sum == 0.0f) {  // no entries: q is 0 whatever lse says, whose power may be infinite (a NaN makes the sum one)
            w.log_coef = w.coef = 0.0f;
        } else if (a.lse) {
            w.log_coef = fmaf(w.ref, a.scale, -a.lse[row]);
            w.coef = expf(w.log_coef);
        } else {
            w.log_coef = -logf(sum);
            w.coef = __fdiv_rn(1.0f, sum);
        }
        w.Q = sum * w.coef;
    }
    w.n = 0;
    for (int j0 = 0; j0 < a.K; j0 += 32) {  // places at or before the ones just read
        const int j = j0 + lane, c = j < a.K ? l.col[j] : -1;
        const float t = j < a.K ? l.z[j] : -INFINITY;
        const bool here = c >= lo && c < hi;
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, here);
        __syncwarp();  // all lanes have read
        if (here) {
            const int to = w.n + __popc(who & ((1u << lane) - 1u));
            l.col[to] = c;
            l.q[to] = power_of(a, t, w.ref) * w.coef;
            l.z[to] = fmaf(t - w.ref, a.scale, w.log_coef);  // log q from t, not from q
        }
        w.n += __popc(who);
        __syncwarp();
    }
    return w;
}

// One warp: the loss of the list's entries, whose logits (z_of) stay in it.
template <typename F>
__device__ __forceinline__ float loss_of(const Args& a, const List& l, int n, const Stats& v, F z_of)
{
    const float log_l = logf(v.l);
    float sum = 0.0f;
    for (int j = threadIdx.x & 31; j < n; j += 32) {
        const float z = z_of(l.col[j]), q = l.q[j], logq = l.z[j];
        l.z[j] = z;
        if (q != 0.0f)
            sum = fmaf(q, logq - (v.l == 0.0f ? -INFINITY : fmaf(z - v.ref, a.scale, -log_l)), sum);
    }
    return warp_sum(sum);
}

// What a row's gradient has of p: Q over the student's sum, 0 where nothing
// comes of the row (no entries, whatever its logits are, or no column left).
__device__ __forceinline__ float ratio_of(float Q, const Stats& v)
{
    return Q == 0.0f || v.l == 0.0f ? 0.0f : __fdiv_rn(Q, v.l);
}

// The gradient exp(t) * A of a run.
template <typename T>
__device__ __forceinline__ uint4 grad_run(const uint4& w, float ref, float k2, float A)
{
    constexpr int P = Run<T>::V / 2;
    float2 f[P];
    Run<T>::widen(w, f);
#pragma unroll
    for (int j = 0; j < P; ++j)
        f[j] = mul2(exp2_pair(mul2(add2(f[j], f2(-ref)), f2(k2))), f2(A));
    return Run<T>::narrow(f);
}

// The gradient of columns [lo, hi) of an output row from the piece that holds
// them: runs aligned like the piece's (whole ones of it four at a time), or not.
template <typename T, int STEP>
__device__ __forceinline__ void put_piece(const Piece<T, STEP>& p, T* o, const Runs<T>& ro, int lo, int hi, float ref, float k2,
                                          float A, bool zero)
{
    constexpr int U = 4, V = Run<T>::V;
    const int step = p.step(), tid = threadIdx.x;
    const uint4 none = make_uint4(0, 0, 0, 0);
    // whole runs of the output that lie in [lo, hi): [v0, v1)
    const int v0 = (lo + ro.phase + V - 1) / V, v1 = max((hi + ro.phase) / V, v0);
    if (tid < 2) {  // what is before and behind them
        const int u = tid ? v1 : v0 - 1, c = ro.column(u);
        if (c + V > lo && c < hi && (tid == 0 || v1 != v0 - 1))
            store_run(ro, o, u, lo, hi, zero ? none : grad_run<T>(p.run_at(c), ref, k2, A));
    }
    T* to = o + ro.column(v0 + tid);
    int u = v0 + tid;
    if (zero) {
        for (; u < v1; u += step, to += step * V)
            st16(to, none);
    } else if (ro.phase == p.r.phase) {
        uint32_t from = p.at(u);
        for (; u + (U - 1) * step < v1; u += U * step, to += U * step * V, from += 16u * (uint32_t)(U * step)) {
            uint4 w[U];
#pragma unroll
            for (int i = 0; i < U; ++i)
                w[i] = lds16(from + 16u * (uint32_t)(i * step));
#pragma unroll
            for (int i = 0; i < U; ++i)
                st16(to + i * step * V, grad_run<T>(w[i], ref, k2, A));
        }
        for (; u < v1; u += step, to += step * V, from += 16u * (uint32_t)step)
            st16(to, grad_run<T>(lds16(from), ref, k2, A));
    } else {
        for (; u < v1; u += step, to += step * V)
            st16(to, grad_run<T>(p.run_at(ro.column(u)), ref, k2, A));
    }
}

// Puts the list's columns right: g * scale * (Q p - their q), each by the first
// entry that names it.
template <typename T>
__device__ __forceinline__ void put_listed(const Args& a, T* o, const List& l, int n, float ref, float ratio, float g)
{
    for (int j = threadIdx.x; j < n; j += blockDim.x) {
        const int c = l.col[j];
        float q = 0.0f;
        bool mine = true;
        for (int i = 0; i < n; ++i)
            if (l.col[i] == c) {
                mine &= i >= j;
                q += l.q[i];
            }
        if (mine)
            store1(o + c, g * a.scale * fmaf(power_of(a, l.z[j], ref), ratio, -q));
    }
}

template <typename T, bool GRAD, int STEP>
__global__ void __launch_bounds__(kThreadsMost + 32, MFX_VOCAB_BLOCKS)
distill_fwd(const Args a)
{
    extern __shared__ __align__(16) char dynamic[];
    __shared__ Stats part[8], mine;
    __shared__ float my_loss, Q;
    __shared__ int listed;
    const List l(dynamic + (size_t)(a.runs + 2) * 16, a.K);
    // one warp more than share the slice: it sees to the list
    const int rank = a.cluster > 1 ? (int)cluster_rank() : 0, tid = threadIdx.x, threads = blockDim.x - 32;
    for (int64_t row = blockIdx.x / a.cluster; row < a.rows; row += gridDim.x / a.cluster) {
        const T* z = static_cast<const T*>(a.logits) + row * a.ld;
        const Runs<T> r(z, a.n);
        const int share = (r.count + a.cluster - 1) / a.cluster;
        const int first = min(rank * share, r.count), last = min(first + share, r.count);
        const int lo = max(r.column(first), 0), hi = min(r.column(last), a.n);
        Piece<T, STEP> p(r, smem_addr(dynamic), threads);
        p.set(first, min(first + a.runs, last));
        Teacher w = {};
        Stats v = no_stats();
        if (tid >= threads) {
            w = read_list<false>(a, row, l, lo, hi, w);
            if (tid == threads)
                Q = w.Q, listed = w.n;
            while (p.last < last)
                p.set(p.last, min(p.last + a.runs, last));
        } else {
            float none;
            p.fill();
            if (tid == 0 && row + a.ahead < a.rows)
                p.prefetch(a.ahead * a.ld);
            scan<T, STEP, false, false>(p, a.k, v, none);
            while (p.last < last) {  // (threads read only what they copied)
                p.set(p.last, min(p.last + a.runs, last));
                p.fill();
                scan<T, STEP, false, false>(p, a.k, v, none);
            }
        }
        join_block<false>(v, a.k2, part, threads >> 5);  // and the slice and Q are there for all threads
        if (a.cluster > 1)
            join_cluster<false>(v, a.k2, &mine, a.cluster);
        const float ratio = ratio_of(Q, v);
        if (tid >= threads) {
            const float loss = p.first == first ? loss_of(a, l, w.n, v, [&](int c) { return p.value(c); })
                                                : loss_of(a, l, w.n, v, [&](int c) { return load1(z + c); });
            if (tid == threads) {
                my_loss = loss;
                if (rank == 0 && a.stats)
                    a.stats[4 * row] = v.ref, a.stats[4 * row + 1] = ratio, a.stats[4 * row + 2] = w.ref, a.stats[4 * row + 3] = w.coef;
            }
        }
        __syncwarp();
        if (a.cluster > 1)
            cluster_arrive(tid >= threads);  // my_loss is there; before the gradient's stores, for which it would wait
        if (GRAD) {
            T* o = static_cast<T*>(a.out) + row * a.ldo;
            const Runs<T> ro(o, a.n);
            const float g = a.g[row], A = g * a.scale * ratio;
            if (p.first != first)
                __syncthreads();  // listed logits of other pieces are read before they may be written
            for (;;) {            // the last piece is the one at hand
                if (tid < threads)
                    put_piece(p, o, ro, p.lo(), p.hi(), v.ref, a.k2, A, ratio == 0.0f);
                __syncthreads();
                if (p.first == first)
                    break;
                p.set(max(p.first - a.runs, first), p.first);
                if (tid < threads) {
                    p.fill();
                    copies_wait<0>();
                }
                __syncthreads();
            }
            if (ratio != 0.0f)
                put_listed<T>(a, o, l, listed, v.ref, ratio, g);
        }
        if (a.cluster > 1)
            cluster_wait();
        else
            __syncthreads();
        if (rank == 0 && tid == 0) {
            float s = my_loss;
            for (int i = 1; i < a.cluster; ++i)
                s += peer_float(&my_loss, i);
            a.loss[row] = s;
        }
        __syncwarp();
        if (a.cluster > 1) {  // nobody leaves, or goes on, while its loss is read
            cluster_arrive(false);
            cluster_wait();
        }
    }
}

// The loss of many rows, one after another.
template <typename T, int STEP>
__global__ void __launch_bounds__(kThreadsMost + 32, MFX_VOCAB_BLOCKS)
distill_rows(const Args a)
{
    extern __shared__ __align__(16) char dynamic[];
    __shared__ Stats part[2][8];
    const int threads = blockDim.x - 32, tid = threadIdx.x;
    if (tid >= threads) {  // the warp that sees to the lists
        const List l(dynamic + Stream<T, STEP>::smem(threads), a.K);
        int slot = 0;
        for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, slot ^= 1) {
            const T* z = static_cast<const T*>(a.logits) + row * a.ld;
            const Teacher w = read_list<false>(a, row, l, 0, a.n, {});
            Stats v = no_stats();
            join_block<false>(v, a.k2, part[slot], threads >> 5);
            const float loss = loss_of(a, l, w.n, v, [&](int c) { return load1(z + c); });
            if (tid == threads) {
                a.loss[row] = loss;
                if (a.stats) {
                    const float ratio = ratio_of(w.Q, v);
                    a.stats[4 * row] = v.ref, a.stats[4 * row + 1] = ratio, a.stats[4 * row + 2] = w.ref, a.stats[4 * row + 3] = w.coef;
                }
            }
            __syncwarp();
        }
        return;
    }
    Stream<T, STEP> in(a.in, dynamic);
    int slot = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, slot ^= 1) {
        Stats v = no_stats();
        in.template take_row<false, false>(row, a.k, v, [](int, bool, float&) {});
        join_block<false>(v, a.k2, part[slot], threads >> 5);
    }
}

template <typename T, int STEP>
__global__ void __launch_bounds__(kThreadsMost + 32)
distill_bwd(const Args a)
{
    extern __shared__ __align__(16) char dynamic[];
    __shared__ int listed;
    const List l(dynamic, a.K);
    // one warp more than write the row: it sees to the list
    const int threads = blockDim.x - 32, tid = threadIdx.x;
    for (int64_t item = blockIdx.x; item < a.rows * a.chunks; item += gridDim.x) {
        const int64_t row = item / a.chunks;
        const T* z = static_cast<const T*>(a.logits) + row * a.ld;
        T* o = static_cast<T*>(a.out) + row * a.ldo;
        const float ref = a.stats_in[4 * row], ratio = a.stats_in[4 * row + 1];
        const Runs<T> ro(o, a.n);
        const int u0 = min((int)(item % a.chunks) * a.per, ro.count), u1 = min(u0 + a.per, ro.count);
        if (ratio == 0.0f) {  // the same for all threads
            if (tid < threads)
                zero_runs(o, ro, u0, u1, threads);
            continue;
        }
        const int lo = max(ro.column(u0), 0), hi = min(ro.column(u1), a.n);
        const float g = a.g[row], A = g * a.scale * ratio;
        if (tid >= threads) {
            const Teacher w = read_list<true>(a, row, l, lo, hi, {a.stats_in[4 * row + 2], a.stats_in[4 * row + 3], 0.0f, 0.0f, 0});
            for (int j = tid & 31; j < w.n; j += 32)
                l.z[j] = load1(z + l.col[j]);
            if (tid == threads)
                listed = w.n;
        }
        if (a.out == a.logits)
            __syncthreads();  // listed logits are read before they are written
        if (tid < threads)
            map_runs<T, STEP>(z, o, ro, u0, u1, threads, [&](const uint4& w, int) { return grad_run<T>(w, ref, a.k2, A); });
        __syncthreads();
        put_listed<T>(a, o, l, listed, ref, ratio, g);
        __syncthreads();
    }
}

template <typename T, bool GRAD>
int launch_fwd(Args a, cudaStream_t s)
{
    if (!GRAD && streamed(a.rows)) {
        const int64_t runs = (a.n * (int64_t)sizeof(T) + 15) / 16 + 1;  // with a head and a tail
        a.in = {a.rows, a.ld, a.n, threads_for(runs, kThreadsMost), a.logits, nullptr, false};
        const int threads = a.in.step + 32;
        const auto kernel = a.in.step == kThreadsMost ? distill_rows<T, kThreadsMost> : distill_rows<T, 0>;
        const size_t smem = Stream<T, 0>::smem(a.in.step) + (size_t)a.K * 12;
        const int64_t room = (int64_t)sm_count() * occupancy(reinterpret_cast<const void*>(kernel), threads, smem);
        kernel<<<(unsigned)(a.rows < room ? a.rows : room), threads, smem, s>>>(a);
        return launch_status();
    }
    const Split sp = split(a.rows, a.n, sizeof(T));
    a.cluster = sp.cluster, a.runs = sp.runs;
    const cudaError_t e = launch_rows(known_step(sp) ? distill_fwd<T, GRAD, kThreadsMost> : distill_fwd<T, GRAD, 0>, a, sp,
                                      sp.threads + 32, sp.smem() + (size_t)a.K * 12, s);
    return e == cudaSuccess ? launch_status() : cuda_failure(e);
}

template <typename T>
int launch_bwd(Args a, cudaStream_t s)
{
    const Chunks c = chunks_of(a.rows, a.n, sizeof(T));
    a.per = c.per, a.chunks = c.count;
    const size_t smem = (size_t)a.K * 12;
    const int64_t need = a.rows * a.chunks;
    const int threads = c.threads + 32;
    const auto kernel = c.threads == kThreadsMost ? distill_bwd<T, kThreadsMost> : distill_bwd<T, 0>;
    const int64_t room = (int64_t)sm_count() * occupancy(reinterpret_cast<const void*>(kernel), threads, smem);
    kernel<<<(unsigned)(need < room ? need : room), threads, smem, s>>>(a);
    return launch_status();
}

// Arguments that the three calls share.
int check(int dt, int t_dt, int64_t rows, int64_t vocab, int64_t ld, int64_t k, int index_bits, float scale)
{
    if (!valid_dtype(dt) || !valid_dtype(t_dt) || (index_bits != 32 && index_bits != 64))
        return MFX_ERR_DTYPE;
    if (!row_sizes_ok(rows, vocab, ld) || k < 0 || k > kMostEntries)
        return MFX_ERR_SHAPE;
    if (!(scale > 0.0f) || !std::isfinite(scale * kLog2e))
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
    // rows without columns hold nothing to read, whatever their distance says
    a.rows = rows, a.ld = vocab ? ld : 0, a.ldo = ldo, a.n = (int)vocab, a.K = (int)k, a.logits = logits, a.index = index;
    a.teacher = teacher, a.wide = index_bits == 64, a.t_bf16 = t_dt == MFX_BF16, a.scale = scale;
    a.k2 = scale * kLog2e, a.k = scaling_of(scale), a.lse = lse, a.g = g, a.loss = loss, a.stats = stats, a.stats_in = stats_in, a.out = out;
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
