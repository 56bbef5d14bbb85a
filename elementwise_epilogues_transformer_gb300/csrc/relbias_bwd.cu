// relbias_bwd.cu -- backward of the relative-position-bias softmax with
// dropout (relbias_fwd.cu has the operation).
//
// P and the keep flags are formed again from x, the row statistics and the
// generator.  With Q = 2^(score - maximum), so that P = Q / sum Q, and z =
// keep * dy,
//   D = sum Q z / sum Q,   dx = Q (z - D) * scale / ((1 - p) sum Q),
// one factor a row; the table's sums are divided by scale at a block's end.
// (A scale that is not a normal number stays out of them and is multiplied in.)
//
// The table's gradient takes the form of the bias: far positions add into two
// registers a thread, near ones into a window in shared memory.  A row's
// chunks all begin at the same residue (mod 8) of the window, so the window
// is kept once per residue and a chunk adds to two aligned 16-byte vectors of
// its row's.  Within a row every vector belongs to one thread, rows of a warp
// or block follow one another, and teams that share a warp take turns: no
// atomics, a fixed order.  Each block leaves its per-bucket sums in the
// workspace, and a second kernel adds those in block order.
//
// What bounds it: HBM without dropout; with it nothing alone, 36 warp
// instructions per 32 elements at 65 % of the issue slots, no pipe above 50 %,
// 14 warps an SM (2x8x2048x2048 bf16), x and dy read once from DRAM.  Beside the
// forward's work it has dy's conversion, the products and differences, the sums
// of the table's gradient, and dy's two trips through shared memory.
// A thread holds 4 chunks, not the forward's 8, since Q and z live together;
// the next row arrives in shared memory meanwhile.  At 2x32x4096x4096 bf16
// (6.44 GB): 1010 us (6380 GB/s) without dropout, 1356 us (4750 GB/s) with;
// 4x12x1024x1024 causal with padding masks and dropout 90 us; fp32 rows of 1001
// keys, 3x7x333 of them, with full masks 38 us; 2x8x1027x2051 bf16 with padding
// masks and dropout 116 us (30 us of bytes; the forward says why).
// Rows of several register blocks form the first half twice and spill (352 to
// 552 bytes a thread): 1x8x256x32768 bf16 with dropout 222 us (60 us of bytes).
#include "relbias.cuh"

namespace mfx {
namespace relbias {
namespace {

constexpr int kWalkTeam = 2 * kLongTeam;  // kernels whose rows take several register blocks (kLongTeam threads too)
constexpr size_t kMostDynamic = kMaxBlockSmem - 512;  // the kernel's own arrays take less than 512 bytes

// Window sums: vector pair u of residue r holds the sums of entries
// 8 u + r - 8 .. + 7; first the low halves of all pairs, then the high ones.
__device__ __host__ __forceinline__ int sum_vectors(const Buckets& w) { return 8 * window_stride(w); }
inline size_t sum_bytes(const Buckets& w) { return (size_t)2 * sum_vectors(w) * sizeof(float4); }

__device__ __forceinline__ void add4(float4* p, float2 a, float2 b)
{
    float4 v = *p;
    v.x += a.x, v.y += a.y, v.z += b.x, v.w += b.y;
    *p = v;
}

// Whether a row comes through shared memory, copied while the row before is
// worked on, rather than straight into registers (bf16 only: fp32 measured
// slower so, 0.38 against 0.31 ms at 2x8x2048x4096).  The gradient's chunks
// then also wait there for the second half of the work, which saves registers.
template <typename T, bool FAST, int MT>
constexpr bool staged()
{
    return FAST && MT < kWalkTeam && sizeof(T) == 2;
}

// Whether a team may be part of a warp: in the kernels of small blocks, and in
// those of masked fp32 rows, which this form of the sums suits better for any
// team (16x12x1024x1024 447 us in place of 497; elsewhere up to 7 % slower).
template <typename T, bool MASK, bool FAST, int MT>
constexpr bool any_team()
{
    return MT == kSmallBlock || (MT == kTeam && sizeof(T) == 4 && MASK && FAST);
}

template <typename T, int C, bool DROP, bool MASK, bool FAST, int MT>
__global__ void __launch_bounds__(MT < kWalkTeam ? MT : kLongTeam, MT > kTeam ? 1 : MT == kSmallBlock ? 4 : 2)
relbias_bwd(const T* dy, const T* x, const float* __restrict__ stats, T* dx, const T* __restrict__ mask,
            const void* __restrict__ table, float* __restrict__ ws, const __grid_constant__ Geom g,
            const __grid_constant__ Buckets w)
{
    extern __shared__ __align__(16) unsigned char smem[];
    float4* win = reinterpret_cast<float4*>(smem);
    __shared__ float part[2][kLongTeam / 32];
    __shared__ float2 far_part[kLongTeam / 32];
    constexpr bool LONG = MT == kWalkTeam, ANY = any_team<T, MASK, FAST, MT>(), STAGED = staged<T, FAST, MT>();
    const int blocks = LONG ? g.blocks : 1;
    const int h = (int)(blockIdx.x / g.slices), slice = (int)(blockIdx.x % g.slices);
    const int tid = threadIdx.x % g.team, tm = threadIdx.x / g.team;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lanes = g.team < 32 ? g.team : 32, warps = g.team >> 5;
    const int last = w.reach + w.hi, stride = window_stride(w), vectors = sum_vectors(w);
    const int sets = g.team > 32 ? 1 : (int)(blockDim.x >> 5);  // one set of sums a block, or one a warp
    float4* acc = win + 8 * stride + (g.team > 32 ? 0 : warp) * 2 * vectors;
    // staged rows, after the window and the sums: x, and dy twice (this row's and the next one's)
    uint4* stage = reinterpret_cast<uint4*>(win + 8 * stride + (ws ? 2 * vectors * sets : 0)) + threadIdx.x;
    uint4* stage_dy = stage + C * blockDim.x;
    fill_window(w, g, table, h, win);
    if (ws)
        for (int i = threadIdx.x; i < 2 * vectors * sets; i += blockDim.x)
            win[8 * stride + i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    __syncthreads();
    const float far_lo = win[window_slot(stride, 0)].x, far_hi = win[window_slot(stride, last)].x;
    float sum_lo = 0.0f, sum_hi = 0.0f;

    Walk at(g, h, slice * g.teams + tm);
    int slot = 0;
    Seat<T> seat = seat_at<T>(g, w, MASK ? mask : nullptr, h, at);
    if constexpr (STAGED) {
        stage_row<C>(stage, x, seat, g.sk, tid, g.team);
        stage_row<C>(stage_dy, dy, seat, g.sk, tid, g.team);
    }
    for (int first = slice * g.teams; first < g.rows; first += g.step, slot ^= 1) {
        const bool live = at.live(g);
        const Row<T> o = row_of<T, FAST>(g, seat, live, mask);
        uint4* sz = stage_dy + slot * C * blockDim.x;
        float shift = 0.0f, top = 0.0f, inv = 0.0f;
        if (live)
            shift = stats[3 * o.r], top = stats[3 * o.r + 1], inv = stats[3 * o.r + 2];
        const auto run = [&](auto check) {
            constexpr bool CHECK = decltype(check)::value, PART = CHECK || MASK;
            float2 Q[C][4], D2 = f2(0.0f);
            unsigned has_keys = ~0u;  // chunks of which the warp has a key that takes part
            Raw8<T> z[STAGED ? 1 : C];
            // P and z of the row's (or block's) chunks, and their part of D
            const auto first_half = [&](int blk) {
                Raw8<T> rx[C];
                if constexpr (STAGED) {
                    if constexpr (DROP && !CHECK) {
                        // the keep flags of all chunks together, while the copies arrive
                        uint4 kb[C];
                        mask_blocks<C>(g.gen, o.block0 + tid, g.team, kb);
                        copies_wait<0>();
                        Raw8<T> r[C];
#pragma unroll
                        for (int c = 0; c < C; ++c)
                            unstage(sz, c, r[c]);
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            drop_raw(r[c], kb[c], g.thresh_hi);
                            restage(sz, c, r[c]);
                        }
                    } else {
                        copies_wait<0>();
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const int ch = (blk * C + c) * g.team + tid, k0 = ch * 8 - o.a;
                        const int k = 8 * (CHECK && FAST && k0 >= o.end ? 0 : ch);
                        load_chunk<T, FAST>(x + o.e0 + k, k0, o.end, o.inner, rx[c]);
                        load_chunk<T, FAST>(dy + o.e0 + k, k0, o.end, o.inner, z[c]);
                    }
                }
                if (PART)
                    has_keys = 0;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int ch = (blk * C + c) * g.team + tid, k0 = ch * 8 - o.a;
                    if (!some_part<CHECK>(k0, o.end))
                        continue;
                    Raw8<T>& zc = z[STAGED ? 0 : c];
                    if constexpr (STAGED) {
                        unstage(stage, c, rx[c]);
                        unstage(sz, c, zc);
                    }
                    if (!score_chunk<T, FAST, MASK>(rx[c], o, g, w, win, far_lo, far_hi, k0, mask != nullptr, shift, Q[c]))
                        continue;
                    if (PART)
                        has_keys |= 1u << c;
                    if (CHECK)
                        MFX_RARELY((!FAST && k0 < 0) || k0 + 8 > o.end)
                            fill_outside(Q[c], k0, o.end, -INFINITY);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        Q[c][i] = make_float2(exp2_of(Q[c][i].x - top), exp2_of(Q[c][i].y - top));
                    if (DROP && (!STAGED || CHECK) && g.drop)
                        drop_raw(zc, one_block(g.gen, o.block0 + ch), g.thresh_hi);
                    float2 f[4];
                    pairs_of(zc, f);
                    // what the upstream gradient holds at keys left out does not count
                    if (CHECK || MASK) {
                        MFX_RARELY(min_of(Q[c]) == 0.0f) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                f[i] = make_float2(Q[c][i].x == 0.0f ? 0.0f : f[i].x, Q[c][i].y == 0.0f ? 0.0f : f[i].y);
                            narrow_pairs(f, zc);
                        }
                    }
                    if constexpr (STAGED)
                        if (CHECK || MASK)
                            restage(sz, c, zc);
                    float2 t = pmul(Q[c][0], f[0]);
#pragma unroll
                    for (int i = 1; i < 4; ++i)
                        t = pfma(Q[c][i], f[i], t);
                    D2 = padd(D2, t);
                }
            };
            for (int blk = 0; blk < blocks; ++blk)
                first_half(blk);
            float D = lanes_sum<ANY>(D2.x + D2.y, lanes);
            // every chunk of this row has been read: on to the team's next row
            at.next(g);
            seat = seat_at<T>(g, w, MASK ? mask : nullptr, h, at);
            if constexpr (STAGED) {
                stage_row<C>(stage, x, seat, g.sk, tid, g.team);
                stage_row<C>(stage_dy + (slot ^ 1) * C * blockDim.x, dy, seat, g.sk, tid, g.team);
            }
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
            D *= inv;
            const float factor = g.grad * inv;
            for (int blk = 0; blk < blocks; ++blk) {
                if (LONG && blocks > 1)
                    first_half(blk);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int ch = (blk * C + c) * g.team + tid, k0 = ch * 8 - o.a;
                    float2 v[4];
                    if (!PART || (has_keys >> c & 1u)) {
                        if constexpr (STAGED)
                            unstage(sz, c, z[0]);
                        pairs_of(z[STAGED ? 0 : c], v);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[i] = pmul(pmul(Q[c][i], padd(v[i], f2(-D))), f2(factor));
                        if (CHECK)
                            MFX_RARELY((!FAST && k0 < 0) || k0 + 8 > o.end)
                                fill_outside(v, k0, o.end, 0.0f);
                        if (ws) {
                            const int rel = k0 - o.pos;
                            const bool near = near_chunk(w, rel) && (!CHECK || k0 < o.end);
                            const float2 t = padd(padd(v[0], v[1]), padd(v[2], v[3]));
                            const float far = near ? 0.0f : t.x + t.y;
                            sum_lo += rel >= w.hi ? 0.0f : far;
                            sum_hi += rel >= w.hi ? far : 0.0f;
                            if (__any_sync(0xFFFFFFFFu, near)) {
                                float4* p = acc + window_slot(stride, rel + w.reach);
                                if (!ANY) {
                                    if (near) {
                                        add4(p, v[0], v[1]);
                                        add4(p + vectors, v[2], v[3]);
                                    }
                                } else {
                                    for (int turn = 0; turn < 32; turn += lanes) {
                                        if (near && turn == (lane & ~(lanes - 1))) {
                                            add4(p, v[0], v[1]);
                                            add4(p + vectors, v[2], v[3]);
                                        }
                                        __syncwarp();
                                    }
                                }
                            }
                        }
                        if (g.post != 1.0f) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                v[i] = pmul(v[i], f2(g.post));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[i] = f2(0.0f);
                    }
                    if (CHECK && ch >= o.chunks)
                        continue;
                    store_chunk<T, FAST>(dx + o.e0 + 8 * ch, k0, g.sk, v);
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
    if (STAGED)
        copies_wait<0>();
    if (!ws)
        return;
    // the block's sum of each bucket: its entries of every residue and set,
    // in order, and the far sums (entries past the window's ends are far too)
    sum_lo = lanes_sum<false>(sum_lo, 32);
    sum_hi = lanes_sum<false>(sum_hi, 32);
    if (lane == 0)
        far_part[warp] = make_float2(sum_lo, sum_hi);
    __syncthreads();
    float4* all = win + 8 * stride;
    for (int i = threadIdx.x; i < 2 * vectors; i += blockDim.x) {
        float4 t = all[i];
        for (int k = 1; k < sets; ++k) {
            const float4 v = all[k * 2 * vectors + i];
            t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
        }
        all[i] = t;
    }
    __syncthreads();
    // one value per entry, in the window's place
    float* entry = reinterpret_cast<float*>(win) + 8;
    const float* sums = reinterpret_cast<const float*>(all);
    for (int i = (int)threadIdx.x - 8; i <= last + 8; i += blockDim.x) {
        float t = 0.0f;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int u = i + 8 - r;  // vector pair u / 8 of residue r, element u mod 8
            if (u >= 0 && (u >> 3) < stride)
                t += sums[4 * ((u & 4 ? vectors : 0) + r * stride + (u >> 3)) + (u & 3)];
        }
        entry[i] = t;
    }
    __syncthreads();
    // eight lanes to a bucket (a warp to each took 3 us longer at any size: 15.2
    // in place of 12.2 us at 8x16x77x77)
    const int nw = blockDim.x >> 5, sub = threadIdx.x & 7;
    for (int u0 = 0; u0 < w.num; u0 += blockDim.x >> 3) {
        const int u = u0 + (threadIdx.x >> 3);
        const bool right = u >= w.side, lo = u == w.side - 1, hi = u == (w.hi ? w.num - 1 : 0);
        const int v = right ? u - w.side : u;
        int n0 = 0, n1 = 0;
        if (u < w.num)
            n0 = side_start(w, v), n1 = side_start(w, v + 1);
        if (right && n0 < 1)
            n0 = 1;
        float t = 0.0f;
        for (int n = n0 + sub; n < n1; n += 8)
            t += entry[right ? w.reach + n : w.reach - n];
        if (lo)
            t += entry[sub - 8];
        if (hi)
            t += entry[last + 1 + sub];
        t = lanes_sum<true>(t, 8);
        if (u < w.num && sub == 0) {
            if (lo || hi)
                for (int k = 0; k < nw; ++k)
                    t += (lo ? far_part[k].x : 0.0f) + (hi ? far_part[k].y : 0.0f);
            ws[((int64_t)slice * w.num + u) * g.np + h] = t * g.unfold;
        }
    }
    pdl_launch_dependents();
}

// Most blocks per head of a backward: what its workspace is sized by, whatever
// kernel the pointers' alignment leads to.
int64_t bwd_slices(const Args& a)
{
    const int64_t most = ((int64_t)sm_count() * kBwdBlocksPerSm + a.np - 1) / a.np;
    return a.b * a.sq < most ? a.b * a.sq : most;
}

// Shared memory of a block: the window, `sets` sets of sums where the table's
// gradient is formed, and C chunks a thread of x and, twice, of dy where rows
// are staged.
template <typename T, int C, bool FAST, int MT>
size_t block_bytes(const Buckets& w, bool sums, int sets, int threads)
{
    return window_bytes(w) + (sums ? sum_bytes(w) * sets : 0) + (staged<T, FAST, MT>() ? (size_t)3 * C * 16 * threads : 0);
}

template <typename T, int C, bool DROP, bool MASK, bool FAST, int MT>
int launch_bwd(Geom g, const Buckets& w, const Args& a, const void* dy, const void* x, const float* stats, void* dx,
               void* dtable, void* workspace, cudaStream_t s)
{
    const auto kern = relbias_bwd<T, C, DROP, MASK, FAST, MT>;
    while (g.team <= 32 && g.team * g.teams > 32 &&
           window_bytes(w) + (dtable ? sum_bytes(w) * (g.team * g.teams / 32) : 0) > 64 * 1024)
        g.teams /= 2;  // wide windows: fewer rows at a time
    const int threads = g.team * g.teams;
    const size_t smem = block_bytes<T, C, FAST, MT>(w, dtable != nullptr, g.team > 32 ? 1 : threads / 32, threads);
    const int64_t slots = (int64_t)sm_count() * occupancy((const void*)kern, threads, smem);
    g.slices = slices_for(g, slots, 4);
    if (g.slices > bwd_slices(a))
        g.slices = (int)bwd_slices(a);
    set_walk(g);
    if ((int64_t)g.slices * g.np > INT32_MAX)
        return MFX_ERR_SHAPE;
    kern<<<(unsigned)(g.slices * g.np), threads, smem, s>>>(
        static_cast<const T*>(dy), static_cast<const T*>(x), stats, static_cast<T*>(dx), static_cast<const T*>(a.mask),
        a.table, dtable ? static_cast<float*>(workspace) : nullptr, g, w);
    const int st = launch_status();
    if (st != MFX_OK || !dtable)
        return st;
    return launch_dbias_finish(a.table_dt, static_cast<const float*>(workspace), g.slices, (int64_t)w.num * g.np,
                               dtable, s);
}

template <typename T, bool DROP, bool MASK, bool FAST>
int dispatch_bwd(const Args& a, const Buckets& w, const void* dy, const void* x, const float* stats, void* dx,
                 void* dtable, void* workspace, cudaStream_t s)
{
    // fp32 holds half the chunks: a chunk's gradient takes twice the registers
    // (with four, 2x8x1027x2051 with dropout took 142 us in place of 122; bf16
    // with two, 2x4x515x4099 with padding masks, 90 us in place of 68)
    constexpr int kMost = sizeof(T) == 2 ? 4 : 2;
    Geom g = make_geom(a, w, x);
    // fewer lanes to a row make its near chunks take more turns, which pays
    // where a causal row leaves chunks out (64x16x128x128: 57 -> 47 us; else 35 -> 36)
    const int c = plan(g, FAST, kMost, kMost, a.causal ? 8 : 16);
    // Wide windows leave staged rows of many chunks no room in a block (two
    // directions and a distance of 2048: bf16 rows of 7176 keys and more with
    // 256 buckets, 9224 with 128, 13320 with 64): those rows go straight into
    // registers, as ones of several register blocks do (1x8x1024x8192 with 256
    // buckets and dropout 245 us, with 32 buckets to a distance of 128 94 us).
    const bool room = g.team <= 32 || block_bytes<T, kMost, FAST, kTeam>(w, dtable != nullptr, 1, g.team) <= kMostDynamic;
    if (g.blocks > 1 || !room)
        return launch_bwd<T, kMost, DROP, MASK, FAST, kWalkTeam>(g, w, a, dy, x, stats, dx, dtable, workspace, s);
    if (g.team < 32 || c == 1) {
        if (c == 1)
            return launch_bwd<T, 1, DROP, MASK, FAST, kSmallBlock>(g, w, a, dy, x, stats, dx, dtable, workspace, s);
        if (c == 2 && kMost > 2)
            return launch_bwd<T, 2, DROP, MASK, FAST, kSmallBlock>(g, w, a, dy, x, stats, dx, dtable, workspace, s);
        return launch_bwd<T, kMost, DROP, MASK, FAST, kSmallBlock>(g, w, a, dy, x, stats, dx, dtable, workspace, s);
    }
    if (c == 2 && kMost > 2)
        return launch_bwd<T, 2, DROP, MASK, FAST, kTeam>(g, w, a, dy, x, stats, dx, dtable, workspace, s);
    return g.team * g.teams > kTeam
               ? launch_bwd<T, kMost, DROP, MASK, FAST, kLongTeam>(g, w, a, dy, x, stats, dx, dtable, workspace, s)
               : launch_bwd<T, kMost, DROP, MASK, FAST, kTeam>(g, w, a, dy, x, stats, dx, dtable, workspace, s);
}

}  // namespace
}  // namespace relbias
}  // namespace mfx

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
    using namespace mfx::relbias;
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
        const int64_t bytes = a.n * dtype_bytes(dt), sb = b * np * sq * 12, tb = a.table_bytes;
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
    if (query || dtable) {
        bool asked = false;
        st = dbias_workspace(bwd_slices(a), (int64_t)w.num * np, workspace, workspace_bytes, &asked);
        if (st != MFX_OK || asked)
            return st;
    }
    return by_variant(a, whole_chunks(a, x, dy, dx), [&](auto t, auto drop, auto masked, auto fast) {
        return dispatch_bwd<decltype(t), decltype(drop)::value, decltype(masked)::value, decltype(fast)::value>(
            a, w, dy, x, stats, dx, dtable, workspace, s);
    });
}
