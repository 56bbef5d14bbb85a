// relbias_fwd.cu -- softmax of attention scores with a learned relative position
// bias and dropout.  The operation and its gradient (relbias_bwd.cu):
//
// Per score row (batch i, head h, query q at position pos):
//   s_k = x_k * scale + table[bucket(k - pos), h] + mask_k,   P = softmax(s),
//   y_k = keep_k * P_k / (1 - p),
// and backwards, with P formed again from x and the row's statistics and the
// keep flags from the generator (neither P nor the keep flags are ever stored),
//   dP_k = keep_k * dy_k / (1 - p),  D = sum_k dP_k P_k,
//   dS_k = P_k (dP_k - D),  dx_k = scale * dS_k,
//   dtable[u, h] = sum of dS over the positions whose bucket is u.
//
// Layout: a team of threads (8, 16 or 32 lanes of a warp, or several warps)
// owns a row and keeps it in registers, C chunks of 8 elements a thread, so x
// is read once and y written once.  A chunk is exactly one block of the
// generator (chunk boundaries sit where the element index is a multiple of
// 8), so with 16-byte aligned buffers and whole chunks it is also one 16-byte
// access.  Rows longer than a team holds are walked in blocks, the second walk
// reading what L2 still has; few long rows are split over the blocks of a
// cluster, which exchange (maximum, sum) through distributed shared memory.
// C is as large as registers allow: a row's reduction, barrier and bookkeeping
// are then shared by most elements (bf16 8, general rows and fp32 4).
//
// The bias needs no [np, sq, sk] tensor: along a row it is constant outside
// the `reach` of the bucket function (the distance from which the last bucket
// holds), and inside it comes from a window in shared memory, built once per
// thread block, which works on one head.  Chunks outside take one of two
// registers; which is asked a warp at a time.
//
// What bounds it: HBM without dropout; with it latency, at the 14 warps an SM
// that the registers leave.  2x8x2048x2048 bf16 with dropout spends 21 warp
// instructions per 32 elements, at 58 % of the issue slots and 47 % of the ALU
// pipe, with loads the second reason to wait; about 7 of the 21 are the
// generator's 10 rounds and the 8 keep words, which run after the reduction,
// when the row's loads are long done.  DRAM reads are x once.
// At 2x32x4096x4096 bf16 (4.29 GB): 691 us (6220 GB/s) without dropout, 968 us
// (4440 GB/s) with; with dropout too, 16x16x512x512 70 us, 4x12x1024x1024 causal
// with padding masks 65 us (chunks that a row leaves out still take their
// exponentials), 2x8x2048x4096 fp32 188 us; decode rows 32x32x8192 9.5 us and
// 1x16x131072 10.8 us of GPU time.  Rows that are not whole chunks are far from
// their bytes (2x8x1027x2051 bf16 with padding masks and dropout 94 us, 20 us of
// bytes): a mask row that is not aligned like its row of x is read element by
// element, as is all data where elem_base % 8 != 0 with dropout.  Masked variants
// spill (bf16 40 to 188 bytes a thread, fp32 up to 496).
#include "relbias.cuh"

namespace mfx {
namespace relbias {
namespace {

// Sums and maxima over a team that may span warps (part) and the blocks of a
// cluster (mine); `slot` alternates between calls so that one barrier each is
// enough.
struct Team {
    float2 (*part)[kLongTeam / 32];
    float2* mine;
    int lanes, warps, cluster;
};

// Joins the pairs of the first n lanes (n a power of two here, the others
// neutral), the same bits in every lane.
__device__ __forceinline__ float2 join_lanes(float2 v, int n)
{
    for (int o = n >> 1; o > 0; o >>= 1)
        v = join(v, make_float2(__shfl_xor_sync(0xFFFFFFFFu, v.x, o), __shfl_xor_sync(0xFFFFFFFFu, v.y, o)));
    return v;
}

// (maximum, sum relative to it) over the team from each warp's.  Few warps'
// pairs are joined one after another by every thread, more by a warp's lanes,
// as are those of a cluster's blocks (one trip through distributed shared
// memory instead of eight).
template <bool LONG>
__device__ __forceinline__ float2 join_team(const Team& tm, float2 v, int slot)
{
    if (tm.warps <= 1)
        return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0)
        tm.part[slot][threadIdx.x >> 5] = v;
    __syncthreads();
    if (!LONG || tm.warps <= 4) {
        v = tm.part[slot][0];
        for (int i = 1; i < tm.warps; ++i)
            v = join(v, tm.part[slot][i]);
    } else {
        v = lane < tm.warps ? tm.part[slot][lane] : make_float2(-INFINITY, 0.0f);
        v = join_lanes(v, kLongTeam / 32);
        v = make_float2(__shfl_sync(0xFFFFFFFFu, v.x, 0), __shfl_sync(0xFFFFFFFFu, v.y, 0));
    }
    if (LONG && tm.cluster > 1) {
        if (threadIdx.x == 0)
            tm.mine[slot] = v;
        cluster_sync();
        v = lane < tm.cluster ? peer_pair(&tm.mine[slot], lane) : make_float2(-INFINITY, 0.0f);
        v = join_lanes(v, tm.cluster);
        v = make_float2(__shfl_sync(0xFFFFFFFFu, v.x, 0), __shfl_sync(0xFFFFFFFFu, v.y, 0));
    }
    return v;
}

// What the backward needs of a row: the mask's shift, the maximum that its
// exponents are taken from (base-2 units) and one over the sum of their
// powers.  (Kept apart, and not as one logarithm, they form P as exactly as
// the forward does: one where a row has a single key.)
__device__ __forceinline__ void put_stats(float* stats, int64_t row, float shift, float top, float inv)
{
    stats[3 * row] = shift, stats[3 * row + 1] = top, stats[3 * row + 2] = inv;
}

// One row whose largest score lies far from zero (a mask of lowest values, say,
// or large scores under any mask), or that has no key left: the mask is shifted
// by its own maximum, which leaves the softmax as it is and the scores their
// digits.  Element by element, three or four passes; out of line, so that it
// costs other rows nothing.
template <typename T, bool DROP, bool LONG>
__device__ __noinline__ void shifted_row(const T* x, T* y, float* stats, const Row<T> o, const Geom& g,
                                         const Buckets& w, const float4* win, const Team& tm, int rank, int tid,
                                         int slot)
{
    const int step = g.team * tm.cluster, first = rank * g.team + tid, last = w.reach + w.hi;
    const int64_t e = o.e0 + o.a;
    float shift = -INFINITY;
    for (int k = first; k < o.end; k += step)
        shift = fmaxf(shift, load1(o.mask + k));
    shift = join_team<LONG>(tm, make_float2(lanes_max<true>(shift, tm.lanes), 0.0f), slot ^ 1).x;
    if (shift == -INFINITY)
        shift = 0.0f;
    const auto score = [&](int k) {
        const float m = load1(o.mask + k);
        const int i = k - o.pos + w.reach;
        const float b = win[window_slot(window_stride(w), i < 0 ? 0 : i > last ? last : i)].x;
        return m == -INFINITY ? -INFINITY : fmaf(m - shift, kLog2eF, fmaf(load1(x + e + k), g.scale2, b));
    };
    float m = -INFINITY, l = 0.0f;
    for (int k = first; k < o.end; k += step)
        m = fmaxf(m, score(k));
    m = join_team<LONG>(tm, make_float2(lanes_max<true>(m, tm.lanes), 0.0f), slot).x;
    const float ref = m == -INFINITY ? 0.0f : m;
    for (int k = first; k < o.end; k += step)
        l += exp2_of(score(k) - ref);
    l = join_team<LONG>(tm, make_float2(ref, lanes_sum<true>(l, tm.lanes)), slot ^ 1).y;
    const float inv = m == -INFINITY && l == 0.0f ? 0.0f : 1.0f / l;
    if (stats && first == 0 && o.chunks)
        put_stats(stats, o.r, shift, ref, inv);
    for (int k = first; o.chunks && k < g.sk; k += step) {
        float v = k < o.end ? exp2_of(score(k) - ref) * inv : 0.0f;
        if (DROP && g.drop && k < o.end)
            v = word16(one_block(g.gen, o.block0 + ((k + o.a) >> 3)), (k + o.a) & 7) >= g.thresh_hi >> 16 ? v * g.keep_scale
                                                                                                       : 0.0f;
        store1(y + e + k, v);
    }
    // the next row's reduction may use either slot
    if (tm.warps > 1)
        __syncthreads();
    if (LONG && tm.cluster > 1)
        cluster_sync();
}

template <typename T, int C, bool DROP, bool MASK, bool FAST, int MT>
__global__ void __launch_bounds__(MT, MT > kTeam ? 1 : (C < 8 ? 3 : 2) * (kTeam / MT))
relbias_fwd(const T* x, T* y, float* __restrict__ stats, const T* __restrict__ mask, const void* __restrict__ table,
            const __grid_constant__ Geom g, const __grid_constant__ Buckets w)
{
    extern __shared__ __align__(16) unsigned char smem[];
    float4* win = reinterpret_cast<float4*>(smem);
    __shared__ float2 part[2][kLongTeam / 32];
    __shared__ float2 mine[2];
    constexpr bool LONG = MT > kTeam, ANY = MT == kSmallBlock;
    const int blocks = LONG ? g.blocks : 1, cluster = LONG ? g.cluster : 1;
    const int rank = LONG ? (int)(blockIdx.x % cluster) : 0;
    const int64_t unit = LONG ? blockIdx.x / cluster : blockIdx.x;
    const int h = (int)(unit / g.slices), slice = (int)(unit % g.slices);
    const int tid = threadIdx.x % g.team, tm = threadIdx.x / g.team;
    const Team team{part, mine, g.team < 32 ? g.team : 32, g.team >> 5, cluster};
    fill_window(w, g, table, h, win);
    __syncthreads();
    const float far_lo = win[window_slot(window_stride(w), 0)].x;
    const float far_hi = win[window_slot(window_stride(w), w.reach + w.hi)].x;

    Walk at(g, h, slice * g.teams + tm);
    int slot = 0;
    Seat<T> seat = seat_at<T>(g, w, MASK ? mask : nullptr, h, at);
    for (int first = slice * g.teams; first < g.rows; first += g.step, slot ^= 1) {
        const bool live = at.live(g);
        const Row<T> o = row_of<T, FAST>(g, seat, live, mask);
        const T* xr = x + o.e0;
        T* yr = y + o.e0;
        // CHECK: some chunk of the row is not there, or not all of it takes part
        const auto run = [&](auto check) {
            constexpr bool CHECK = decltype(check)::value, PART = CHECK || MASK;
            float2 s[C][4];
            unsigned has_keys = ~0u;  // chunks of which the warp has a key that takes part
            float m = -INFINITY, l = 0.0f;
            for (int blk = 0; blk < blocks; ++blk) {
                const int c0 = (blk * cluster + rank) * (C * g.team) + tid;
                Raw8<T> raw[C];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int ch = c0 + c * g.team, k0 = ch * 8 - o.a;
                    load_chunk<T, FAST>(xr + 8 * (CHECK && FAST && k0 >= o.end ? 0 : ch), k0, o.end, o.inner, raw[c]);
                }
                float t = -INFINITY;
                if (PART)
                    has_keys = 0;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int k0 = (c0 + c * g.team) * 8 - o.a;
                    const bool has = some_part<CHECK>(k0, o.end) &&
                                     score_chunk<T, FAST, MASK>(raw[c], o, g, w, win, far_lo, far_hi, k0, mask != nullptr, 0.0f, s[c]);
                    if (has) {
                        if (PART)
                            has_keys |= 1u << c;
                        if (CHECK)
                            MFX_RARELY((!FAST && k0 < 0) || k0 + 8 > o.end)
                                fill_outside(s[c], k0, o.end, -INFINITY);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s[c][i] = f2(-INFINITY);
                    }
                    t = max_of(t, s[c]);
                }
                t = fmaxf(m, lanes_max<ANY>(t, team.lanes));
                const float ref = t == -INFINITY ? 0.0f : t;
                float2 sum = f2(0.0f);
#pragma unroll
                for (int c = 0; c < C; ++c) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[c][i] = make_float2(exp2_of(s[c][i].x - ref), exp2_of(s[c][i].y - ref));
                    sum = padd(sum, padd(padd(s[c][0], s[c][1]), padd(s[c][2], s[c][3])));
                }
                l = (blk ? l * exp2_of(m - ref) : 0.0f) + (sum.x + sum.y);
                m = t;
            }
            const float mw = m;  // what s is relative to
            l = lanes_sum<ANY>(l, team.lanes);
            at.next(g);  // the team's next row, while the parts of this one meet
            seat = seat_at<T>(g, w, MASK ? mask : nullptr, h, at);
            const float2 v = join_team<LONG>(team, make_float2(m, l), slot);
            m = v.x, l = v.y;
            if (MASK && mask) {
                // a largest score far from zero, whether the mask or x took it there, beyond
                // the type's range in either direction, or no key at all (teams that
                // share a warp go together)
                bool again = fabsf(m) > 96.0f;
                if (ANY)
                    again = __any_sync(0xFFFFFFFFu, again);
                if (again) {
                    shifted_row<T, DROP, LONG>(x, y, stats, o, g, w, win, team, rank, tid, slot);
                    return;
                }
            }
            float inv = m == -INFINITY && l == 0.0f ? 0.0f : 1.0f / l;
            if (stats && tid == 0 && rank == 0 && live)
                put_stats(stats, o.r, 0.0f, m == -INFINITY ? 0.0f : m, inv);
            if (DROP)
                inv *= g.keep_scale;
            const float f1 = mw == -INFINITY && l == l ? 0.0f : exp2_of(mw - m) * inv;
            for (int blk = 0; blk < blocks; ++blk) {
                const int c0 = (blk * cluster + rank) * (C * g.team) + tid;
                constexpr int PAIR = C > 1 && sizeof(T) == 2 ? 2 : 1;  // generator blocks drawn together (fp32: no gain)
                uint4 kb[PAIR];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int ch = c0 + c * g.team, k0 = ch * 8 - o.a;
                    if (DROP && !CHECK && c % PAIR == 0)
                        mask_blocks<PAIR>(g.gen, o.block0 + ch, g.team, kb);
                    float2 p[4];
                    bool has = !PART || (has_keys >> c & 1u);
                    if (LONG && blocks > 1) {
                        has = some_part<true>(k0, o.end);
                        if (has) {
                            Raw8<T> raw;
                            load_chunk<T, FAST>(xr + 8 * (FAST && k0 >= o.end ? 0 : ch), k0, o.end, o.inner, raw);
                            has = score_chunk<T, FAST, MASK>(raw, o, g, w, win, far_lo, far_hi, k0, mask != nullptr, 0.0f, s[c]);
                        }
                    }
                    if (has) {
                        float f = f1;
                        if (LONG && blocks > 1) {
                            const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                s[c][i] = make_float2(exp2_of(s[c][i].x - ref), exp2_of(s[c][i].y - ref));
                            f = inv;
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            p[i] = pmul(s[c][i], f2(f));
                        if (DROP && g.drop)
                            drop_pairs(p, CHECK ? one_block(g.gen, o.block0 + ch) : kb[c % PAIR], g.thresh_hi);
                        if (CHECK)
                            MFX_RARELY((!FAST && k0 < 0) || k0 + 8 > o.end)
                                fill_outside(p, k0, o.end, 0.0f);
                    } else {  // keys that a causal row leaves out
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            p[i] = f2(0.0f);
                    }
                    if (CHECK && ch >= o.chunks)
                        continue;
                    store_chunk<T, FAST>(yr + 8 * ch, k0, g.sk, p);
                }
            }
        };
        if constexpr (FAST) {
            bool full = g.exact && o.end == g.sk;
            if (ANY)
                full = __all_sync(0xFFFFFFFFu, full);
            if (full)
                run(std::false_type{});
            else
                run(std::true_type{});
        } else {
            run(std::true_type{});
        }
    }
    if (LONG && cluster > 1)
        cluster_sync();  // no block leaves while a peer may still read its pair
}

template <typename T, int C, bool DROP, bool MASK, bool FAST, int MT>
int launch_fwd(Geom g, const Buckets& w, const Args& a, const void* x, void* y, float* stats, cudaStream_t s)
{
    const auto kern = relbias_fwd<T, C, DROP, MASK, FAST, MT>;
    const int threads = g.team * g.teams;
    const size_t smem = window_bytes(w);
    const int64_t slots = (int64_t)sm_count() * occupancy((const void*)kern, threads, smem) / g.cluster;
    g.slices = slices_for(g, slots > 0 ? slots : 1, 1);
    set_walk(g);
    const int64_t blocks = (int64_t)g.slices * g.np * g.cluster;
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<const T*>(x), static_cast<T*>(y), stats,
                                             static_cast<const T*>(a.mask), a.table, (const Geom)g, (const Buckets)w);
    return e == cudaSuccess ? launch_status() : cuda_failure(e);
}

template <typename T, bool DROP, bool MASK, bool FAST>
int dispatch_fwd(const Args& a, const Buckets& w, const void* x, void* y, float* stats, cudaStream_t s)
{
    Geom g = make_geom(a, w, x);
    constexpr int kMost = FAST && sizeof(T) == 2 ? 8 : 4;
    // (fp32 rows of which all takes part: two chunks to a thread; four took 95 us
    // in place of 85 at 16x16x512x512.  Masked and causal ones take four)
    int c = plan(g, FAST, kMost, sizeof(T) == 4 && FAST && !MASK && !a.causal ? 2 : kMost, 8);
    const int64_t rows = a.b * a.np * a.sq, sms = sm_count(), chunks = chunks_of(g, FAST);
    if (chunks > 32 && rows < 4 * sms) {
        // few rows: as many threads on each as give every SM work, and rows
        // too long for that over the blocks of a cluster
        c = FAST ? 1 : 4;
        while (g.cluster < kMaxCluster && rows * g.cluster < sms && chunks > 32 * c * g.cluster)
            g.cluster *= 2;
        while (c < 4 && chunks > (int64_t)kLongTeam * c * g.cluster)
            c *= 4;
        while (g.cluster < kMaxCluster && chunks > (int64_t)kLongTeam * c * g.cluster)
            g.cluster *= 2;
        const int64_t per = (int64_t)c * g.cluster, team = ((chunks + per - 1) / per + 31) / 32 * 32;
        g.team = (int)(team < 64 ? 64 : team < kLongTeam ? team : kLongTeam);
        g.teams = 1;
        const int64_t held = g.team * per;
        g.blocks = (int)((chunks + held - 1) / held);
        g.exact = FAST && chunks == held;
    }
    const bool big = g.team * g.teams > kTeam || g.cluster > 1 || g.blocks > 1;
    // kernels of small blocks take teams that are part of a warp; for others
    // they are slower (2x32x4096x4096 without dropout 717 us in place of 689)
    if (c == 2)
        return launch_fwd<T, 2, DROP, MASK, FAST, kSmallBlock>(g, w, a, x, y, stats, s);
    if (g.team * g.teams <= kSmallBlock && g.cluster == 1) {
        if (c == 1)
            return launch_fwd<T, 1, DROP, MASK, FAST, kSmallBlock>(g, w, a, x, y, stats, s);
        if (g.team < 32) {
            if constexpr (FAST && sizeof(T) == 2)
                if (c == 8)
                    return launch_fwd<T, 8, DROP, MASK, FAST, kSmallBlock>(g, w, a, x, y, stats, s);
            return launch_fwd<T, 4, DROP, MASK, FAST, kSmallBlock>(g, w, a, x, y, stats, s);
        }
    }
    if constexpr (FAST) {
        if (c == 1)
            return big ? launch_fwd<T, 1, DROP, MASK, FAST, kLongTeam>(g, w, a, x, y, stats, s)
                       : launch_fwd<T, 1, DROP, MASK, FAST, kTeam>(g, w, a, x, y, stats, s);
        if constexpr (sizeof(T) == 2)
            if (c == 8)
                return launch_fwd<T, 8, DROP, MASK, FAST, kTeam>(g, w, a, x, y, stats, s);
    }
    return big ? launch_fwd<T, 4, DROP, MASK, FAST, kLongTeam>(g, w, a, x, y, stats, s)
               : launch_fwd<T, 4, DROP, MASK, FAST, kTeam>(g, w, a, x, y, stats, s);
}

}  // namespace
}  // namespace relbias
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
    using namespace mfx::relbias;
    Args a{dt,     b,      np,      sq,      sk,     scale,   table_dt,  table, num_buckets, max_distance, bidirectional,
           mask,   mask_b, mask_np, mask_sq, causal, q_start, seq_start, p,     seed,        offset,       elem_base,
           0,      0,      0};
    Buckets w;
    const int st = check(a, &w);
    if (st != MFX_OK || a.n == 0)
        return st;
    if (!x || !y)
        return MFX_ERR_NULL;
    const int64_t bytes = a.n * dtype_bytes(dt), sb = b * np * sq * 12;
    if (partial_overlap(x, bytes, y, bytes) || overlaps(mask, a.mask_bytes, y, bytes) ||
        overlaps(table, a.table_bytes, y, bytes) || overlaps(seq_start, 4 * b, y, bytes) ||
        overlaps(stats, sb, y, bytes) || overlaps(stats, sb, x, bytes) || overlaps(stats, sb, mask, a.mask_bytes) ||
        overlaps(stats, sb, table, a.table_bytes) || overlaps(stats, sb, seq_start, 4 * b))
        return MFX_ERR_ALIAS;
    return by_variant(a, whole_chunks(a, x, y, nullptr), [&](auto t, auto drop, auto masked, auto fast) {
        return dispatch_fwd<decltype(t), decltype(drop)::value, decltype(masked)::value, decltype(fast)::value>(
            a, w, x, y, stats, static_cast<cudaStream_t>(stream));
    });
}
