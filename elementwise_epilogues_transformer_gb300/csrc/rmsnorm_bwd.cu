// rmsnorm_bwd.cu -- gradients of the root-mean-square norm with the
// residual's addition.  From the stored h and rstd, with n = h * rstd and
// u = dy * (weight + offset),
//   dx = rstd * (u - n * mean(u * n)) + dh
//      = rstd * u - h * (rstd^3 * sum(u * h) / cols) + dh,
//   dweight = sum over rows of dy * n,
// dh being the gradient that reaches h from further on.  x and the residual
// have the same gradient; it is written in each one's type.
//
// The weight's gradient is formed on the way: each thread owns the same
// columns of every row that its team works on and adds them up in registers;
// the blocks' partial sums are joined in a fixed order by the kernel that
// joins those of the bias gradients.
//
// What bounds it: HBM where units are wide and a residual is fp32 (16384x4096
// 164 us, 6540 GB/s, 0.96 of the copy rate); latency at the warps that the
// registers of the sums leave in bf16 (8192x8192 112.5 us, 5960 GB/s); single
// columns their instructions (3001x2051 fp32 29.5 us with 4.5 of the sums'
// kernel; 8192x4099 bf16 139 us).  Reading dy and h a second time from shared
// memory costs less than the registers that would hold them.
#include "rmsnorm.cuh"

#include <cmath>

namespace mfx {
namespace rmsnorm {
namespace {

struct Args {
    int64_t rows;
    int cols, lanes, depth;
    uint32_t row_bytes, x_bytes, r_bytes;  // of a row on its way: all of it, dy's part, h's
    const void *dy, *h, *dh, *weight;
    const float* rstd;
    bool w_bf16;
    float offset;
    void *dx, *dres;
    float *ws, *dots;
};

template <typename XT, typename RT, int V, int E>
__global__ void __launch_bounds__(E == 8 ? 1024 : 512, 1)
norm_bwd(const Args a)
{
    constexpr int N = E / V;
    constexpr bool VEC = V > 1;
    __shared__ float2 part[2][32];
    extern __shared__ __align__(16) char dynamic[];
    const int lanes = a.lanes, teams = blockDim.x / lanes, team = threadIdx.x / lanes, tl = threadIdx.x % lanes;
    const int cols = a.cols, c0 = column_of<V, E>(0, tl), mine = units_of<V, E>(cols, lanes, tl);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(dynamic) + team * (uint32_t)a.depth * a.row_bytes;
    const uint32_t end = ring + (uint32_t)a.depth * a.row_bytes;
    const int64_t step = (int64_t)gridDim.x * teams, all = a.rows * cols;
    const XT* const dy = static_cast<const XT*>(a.dy);
    const RT *const hs = static_cast<const RT*>(a.h), *const dh = static_cast<const RT*>(a.dh);
    int64_t row = (int64_t)blockIdx.x * teams + team;
    const auto start = [&](int64_t r, uint32_t to) {
        if (r - team < a.rows) {  // a team past the end takes the last row
            const int64_t at = (r < a.rows ? r : a.rows - 1) * cols;
            copy_row<XT, V, E>(to, dy + at, cols, dy, dy + all, lanes, tl, mine);
            copy_row<RT, V, E>(to + a.x_bytes, hs + at, cols, hs, hs + all, lanes, tl, mine);
            if (dh)
                copy_row<RT, V, E>(to + a.x_bytes + a.r_bytes, dh + at, cols, dh, dh + all, lanes, tl, mine);
        }
        copies_commit();
    };
    int64_t next = row;
    for (uint32_t to = ring; to != end; to += a.row_bytes, next += step) {
        clear_rest<XT, V, E>(to, tl, mine);
        clear_rest<RT, V, E>(to + a.x_bytes, tl, mine);
        if (dh)
            clear_rest<RT, V, E>(to + a.x_bytes + a.r_bytes, tl, mine);
        start(next, to);
    }
    float w[N][V], acc[N][V];
    factors_of<V, E>(a.weight, a.w_bf16, a.offset, mine, tl, w);
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j)
            acc[k][j] = 0.0f;
    int slot = 0;
    uint32_t buf = ring;
    for (; row - team < a.rows; row += step, next += step, slot ^= 1) {
        const bool on = row < a.rows;
        const int64_t r = on ? row : a.rows - 1, at = r * cols;
        const int put = on ? mine : 0;  // units that count
        const float rstd = a.rstd[r];
        copies_wait(a.depth - 1);
        if (!VEC)
            team_barrier(lanes);
        const uint32_t sg = buf + (VEC ? 0u : where(dy + at)) + c0 * (uint32_t)sizeof(XT);
        const uint32_t sh = buf + a.x_bytes + (VEC ? 0u : where(hs + at)) + c0 * (uint32_t)sizeof(RT);
        const uint32_t se = buf + a.x_bytes + a.r_bytes + (VEC || !dh ? 0u : where(dh + at)) + c0 * (uint32_t)sizeof(RT);
        float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float g[V], h[V];
            read_unit<XT, V>(sg, k, mine, g);
            read_unit<RT, V>(sh, k, mine, h);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float gh = g[j] * h[j];
                if (k < put)
                    acc[k][j] = fmaf(gh, rstd, acc[k][j]);
                v.x = fmaf(gh, w[k][j], v.x);
            }
        }
        v = over_team<false>(v, lanes, part, slot);
        const float b = rstd * (__fdiv_rn(v.x * rstd, (float)cols) * rstd);
        XT* dx = a.dx ? static_cast<XT*>(a.dx) + at + c0 : nullptr;
        RT* dres = a.dres ? static_cast<RT*>(a.dres) + at + c0 : nullptr;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float g[V], h[V];
            read_unit<XT, V>(sg, k, mine, g);
            read_unit<RT, V>(sh, k, mine, h);
#pragma unroll
            for (int j = 0; j < V; ++j)
                g[j] = fmaf(rstd, g[j] * w[k][j], -b * h[j]);
            if (dh) {
                read_unit<RT, V>(se, k, mine, h);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    g[j] += h[j];
            }
            if (k < put) {
                if (dx)
                    store_unit<XT, V>(dx + k * 32 * V, g);
                if (dres)
                    store_unit<RT, V>(dres + k * 32 * V, g);
            }
        }
        if (!VEC)
            team_barrier(lanes);
        start(next, buf);
        buf = buf + a.row_bytes == end ? ring : buf + a.row_bytes;
    }
    if (!a.ws)
        return;
    float* ws = a.ws + (int64_t)blockIdx.x * cols;
    if (teams == 1) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (k < mine)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    ws[c0 + k * 32 * V + j] = acc[k][j];
        return;
    }
    // the teams' sums in order (rows are 512 columns at most; nothing is on its way any more)
    float* sums = reinterpret_cast<float*>(dynamic);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k < mine)
#pragma unroll
            for (int j = 0; j < V; ++j)
                sums[team * cols + c0 + k * 32 * V + j] = acc[k][j];
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += blockDim.x) {
        float s = sums[c];
        for (int t = 1; t < teams; ++t)
            s += sums[t * cols + c];
        ws[c] = s;
    }
}

// Rows longer than that: the sums u * h of every row first, then the gradients
// a slab of columns at a time; column by column.
constexpr int kLongThreads = 512, kSlab = 4;  // columns of a thread of a slab

template <typename XT, typename RT>
__global__ void __launch_bounds__(kLongThreads)
row_dots(const Args a)
{
    __shared__ float2 part[2][32];
    int slot = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, slot ^= 1) {
        const XT* g = static_cast<const XT*>(a.dy) + row * a.cols;
        const RT* h = static_cast<const RT*>(a.h) + row * a.cols;
        float2 v = make_float2(0.0f, 0.0f);
#pragma unroll 4
        for (int c = threadIdx.x; c < a.cols; c += kLongThreads) {
            float w[1];
            factors<1>(a.weight, a.w_bf16, a.offset, c, w);
            v.x = fmaf(load1(g + c) * w[0], load1(h + c), v.x);
        }
        v = over_team<false>(v, kLongThreads, part, slot);
        if (threadIdx.x == 0)
            a.dots[row] = v.x;
    }
}

template <typename XT, typename RT>
__global__ void __launch_bounds__(kThreads)
slab_bwd(const Args a)
{
    const int64_t c0 = (int64_t)blockIdx.x * kSlab * kThreads + threadIdx.x;
    float acc[kSlab], w[kSlab][1];
#pragma unroll
    for (int i = 0; i < kSlab; ++i) {
        const int64_t c = c0 + i * kThreads;
        acc[i] = w[i][0] = 0.0f;
        if (c < a.cols)
            factors<1>(a.weight, a.w_bf16, a.offset, (int)c, w[i]);
    }
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float rstd = a.rstd[row], b = rstd * (__fdiv_rn(a.dots[row] * rstd, (float)a.cols) * rstd);
#pragma unroll
        for (int i = 0; i < kSlab; ++i) {
            const int64_t c = c0 + i * kThreads, at = row * a.cols + c;
            if (c >= a.cols)
                continue;
            const float g = load1(static_cast<const XT*>(a.dy) + at), h = load1(static_cast<const RT*>(a.h) + at);
            acc[i] = fmaf(g, h * rstd, acc[i]);
            float d = fmaf(rstd, g * w[i][0], -b * h);
            if (a.dh)
                d += load1(static_cast<const RT*>(a.dh) + at);
            if (a.dx)
                store1(static_cast<XT*>(a.dx) + at, d);
            if (a.dres)
                store1(static_cast<RT*>(a.dres) + at, d);
        }
    }
    if (a.ws)
#pragma unroll
        for (int i = 0; i < kSlab; ++i)
            if (const int64_t c = c0 + i * kThreads; c < a.cols)
                a.ws[(int64_t)blockIdx.y * a.cols + c] = acc[i];
}

struct Plan {
    Layout l;
    uint32_t x_bytes, r_bytes;
    int64_t blocks;    // partial sums of a column
    int64_t ws, dots;  // floats of each in the workspace
};

// The blocks go by sizes and types alone (a row's bytes with dh, whole vectors
// if the width has them): the workspace's size must not go by addresses.
template <typename XT, typename RT>
constexpr int unit_of() { return sizeof(XT) > sizeof(RT) ? 1 : sizeof(RT) == 2 ? 8 : 4; }

template <typename XT, typename RT, int V>
auto kernel_of(int E)
{
    if (E == 16)
        return norm_bwd<XT, RT, V, 16>;
    return E == 8 ? norm_bwd<XT, RT, V, 8> : norm_bwd<XT, RT, V, 32>;
}

template <typename XT, typename RT>
auto kernel_of(int E, bool vec)
{
    return vec ? kernel_of<XT, RT, unit_of<XT, RT>()>(E) : kernel_of<XT, RT, 1>(E);
}

template <typename XT, typename RT>
Plan plan(int64_t rows, int64_t cols, bool vec)
{
    const auto x_bytes = [](int64_t room) { return ((size_t)room * sizeof(XT) + kPad + 15) / 16 * 16; };
    const auto r_bytes = [](int64_t room) { return ((size_t)room * sizeof(RT) + kPad + 15) / 16 * 16; };
    Plan p = {};
    const auto laid = [&](bool v) {
        // One type: 32 elements a thread beyond 1024 columns (bf16 8192x8192 112.5 us, 128 with 16; 32768x2048 120, 126
        // with 8; 65536x1024 122, 129 with 32; fp32 16384x4096 203, 210 with 16).  Two types 8 and 16 (16384x4096 164,
        // 171 with 32), single columns 8 to the end (8192x4099 bf16 138, 180 with 16).
        const bool wide = sizeof(XT) == sizeof(RT) && v;
        // (teams' sums at the end take no more than a row of dy, h and dh: 6 bytes a column or more)
        return layout(rows, cols, v ? unit_of<XT, RT>() : 1, wide ? 1024 : v ? 2048 : 8192, wide ? 1024 : 8192,
                      [&](int64_t room) { return x_bytes(room) + 2 * r_bytes(room); },
                      [&](int e) { return e == 8 ? 1024 : 512; });
    };
    p.l = laid(vec);
    p.x_bytes = (uint32_t)x_bytes(p.l.room), p.r_bytes = (uint32_t)r_bytes(p.l.room);
    if (p.l.depth == 0) {
        const int64_t slabs = (cols + kSlab * kThreads - 1) / (kSlab * kThreads);
        const int64_t lanes = (8 * sm_count() + slabs - 1) / slabs;
        p.blocks = rows < lanes ? rows : lanes;
        p.dots = (rows + 3) / 4 * 4;
    } else {
        const bool v = cols % 8 == 0;
        const Layout l = laid(v);
        const int64_t teams = l.threads / l.lanes, need = (rows + teams - 1) / teams;
        const int64_t room =
            (int64_t)sm_count() * occupancy(reinterpret_cast<const void*>(kernel_of<XT, RT>(l.E, v)), l.threads, l.smem);
        p.blocks = need < room ? need : room;
    }
    p.ws = p.blocks * cols;
    return p;
}

template <typename XT, typename RT>
int launch(Args a, const Plan& p, bool vec, cudaStream_t s)
{
    if (p.l.depth == 0) {
        const int64_t room = (int64_t)sm_count() * 4;
        row_dots<XT, RT><<<(unsigned)(a.rows < room ? a.rows : room), kLongThreads, 0, s>>>(a);
        if (const int st = launch_status(); st != MFX_OK)
            return st;
        const dim3 grid((unsigned)((a.cols + kSlab * kThreads - 1) / (kSlab * kThreads)), (unsigned)p.blocks);
        slab_bwd<XT, RT><<<grid, kThreads, 0, s>>>(a);
        return launch_status();
    }
    a.lanes = p.l.lanes, a.depth = p.l.depth, a.row_bytes = (uint32_t)p.l.row, a.x_bytes = p.x_bytes, a.r_bytes = p.r_bytes;
    const auto kernel = kernel_of<XT, RT>(p.l.E, vec);
    occupancy(reinterpret_cast<const void*>(kernel), p.l.threads, p.l.smem);  // its shared memory is allowed
    kernel<<<(unsigned)p.blocks, p.l.threads, p.l.smem, s>>>(a);
    return launch_status();
}

template <typename XT, typename RT>
int run(int w_dt, Args& a, void* dweight, void* workspace, size_t* bytes, bool vec, cudaStream_t s)
{
    const Plan p = plan<XT, RT>(a.rows, a.cols, vec);
    // partial sums only where dweight is formed, the rows' sums where rows are long
    const size_t need = (size_t)(p.dots + (dweight ? p.ws : 0)) * sizeof(float);
    if (bytes && !workspace) {
        *bytes = need;
        return MFX_OK;
    }
    if (need) {
        if (!workspace || !bytes)
            return MFX_ERR_NULL;
        if (*bytes < need || !aligned16(workspace))
            return MFX_ERR_WORKSPACE;
        a.dots = p.dots ? static_cast<float*>(workspace) : nullptr;
        a.ws = dweight ? static_cast<float*>(workspace) + p.dots : nullptr;
    }
    if (const int st = launch<XT, RT>(a, p, vec, s); st != MFX_OK)
        return st;
    return dweight ? launch_dbias_finish(w_dt, a.ws, p.blocks, a.cols, dweight, s) : MFX_OK;
}

}  // namespace
}  // namespace rmsnorm
}  // namespace mfx

extern "C" int mfx_add_rmsnorm_bwd(int x_dt, int res_dt, int w_dt, int64_t rows, int64_t cols, const void* dy,
                                   const void* h, const float* rstd, const void* weight, float weight_offset,
                                   const void* dh, void* dx, void* dresidual, void* dweight, void* workspace,
                                   size_t* workspace_bytes, void* stream)
{
    using namespace mfx;
    if (!valid_dtype(x_dt) || !valid_dtype(res_dt) || !valid_dtype(w_dt))
        return MFX_ERR_DTYPE;
    if (!rmsnorm::sizes_ok(rows, cols))
        return MFX_ERR_SHAPE;
    if (!std::isfinite(weight_offset))
        return MFX_ERR_VALUE;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0 || cols == 0) {
        if (workspace_bytes && !workspace) {
            *workspace_bytes = 0;
            return MFX_OK;
        }
        return cols && dweight ? launch_dbias_finish(w_dt, nullptr, 0, cols, dweight, s) : MFX_OK;
    }
    const bool query = workspace_bytes && !workspace;
    if (!query && (!dy || !h || !rstd || (!dx && !dresidual) || (dweight && !weight)))
        return MFX_ERR_NULL;
    const int64_t n = rows * cols, xb = n * dtype_bytes(x_dt), rb = n * dtype_bytes(res_dt);
    struct Buf { const void* p; int64_t n; };
    const Buf in[3] = {{dy, xb}, {h, rb}, {dh, rb}}, more[2] = {{rstd, rows * 4}, {weight, cols * dtype_bytes(w_dt)}};
    const Buf out[4] = {{dx, xb}, {dresidual, rb}, {dweight, cols * dtype_bytes(w_dt)},
                        {workspace, workspace_bytes ? (int64_t)*workspace_bytes : 0}};
    for (int i = 0; i < 4 && !query; ++i) {
        for (const Buf& b : in)
            if (i < 2 ? partial_overlap(out[i].p, out[i].n, b.p, b.n) : overlaps(out[i].p, out[i].n, b.p, b.n))
                return MFX_ERR_ALIAS;
        for (const Buf& b : more)
            if (overlaps(out[i].p, out[i].n, b.p, b.n))
                return MFX_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n))
                return MFX_ERR_ALIAS;
    }
    rmsnorm::Args a = {};
    a.rows = rows, a.cols = (int)cols, a.dy = dy, a.h = h, a.dh = dh, a.weight = weight, a.rstd = rstd;
    a.w_bf16 = w_dt == MFX_BF16, a.offset = weight_offset, a.dx = dx, a.dres = dresidual;
    const bool vec = cols % 8 == 0 && aligned16(dy) && aligned16(h) && aligned16(dh) && aligned16(weight) &&
                     aligned16(dx) && aligned16(dresidual);
    if (x_dt == MFX_BF16)
        return res_dt == MFX_BF16 ? rmsnorm::run<bf16, bf16>(w_dt, a, dweight, workspace, workspace_bytes, vec, s)
                                  : rmsnorm::run<bf16, float>(w_dt, a, dweight, workspace, workspace_bytes, vec, s);
    return res_dt == MFX_F32 ? rmsnorm::run<float, float>(w_dt, a, dweight, workspace, workspace_bytes, vec, s)
                             : rmsnorm::run<float, bf16>(w_dt, a, dweight, workspace, workspace_bytes, vec, s);
}
