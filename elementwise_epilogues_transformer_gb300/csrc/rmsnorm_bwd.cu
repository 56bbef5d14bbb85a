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
// columns of every row that its block works on and adds them up in registers;
// the blocks' partial sums are joined in a fixed order by the kernel that
// joins those of the bias gradients.
#include "rmsnorm.cuh"

#include <cmath>

namespace mfx {
namespace rmsnorm {
namespace {

struct Args {
    int64_t rows;
    int cols, lanes;
    const void *dy, *h, *dh, *weight;
    const float* rstd;
    bool w_bf16;
    float offset;
    void *dx, *dres;
    float *ws, *dots;
};

constexpr int kMaxLanes = 512;    // threads of a row
constexpr int kInRegisters = 512 * 8 * 4;

// Gradient of a piece of a row from its dy (g), h and coefficients, into dx and
// dresidual.
template <typename XT, typename RT, int C, bool VEC>
__device__ __forceinline__ void store_grads(const Args& a, int64_t at, int cols, int lanes, int tl, float (&d)[8 * C])
{
    if (a.dh) {
        float e[8 * C];
        load_row<RT, C, VEC>(static_cast<const RT*>(a.dh) + at, cols, lanes, tl, e);
#pragma unroll
        for (int i = 0; i < 8 * C; ++i)
            d[i] += e[i];
    }
    if (a.dx)
        store_row<XT, C, VEC>(static_cast<XT*>(a.dx) + at, cols, lanes, tl, d);
    if (a.dres)
        store_row<RT, C, VEC>(static_cast<RT*>(a.dres) + at, cols, lanes, tl, d);
}

template <typename XT, typename RT, int C, bool VEC>
__global__ void __launch_bounds__(kMaxLanes)
norm_bwd(const Args a)
{
    __shared__ float2 part[2][32];
    extern __shared__ float sums[];  // teams of a warp or less: their partial sums
    const int lanes = a.lanes, teams = blockDim.x / lanes, team = threadIdx.x / lanes, tl = threadIdx.x % lanes;
    float acc[8 * C];
#pragma unroll
    for (int e = 0; e < 8 * C; ++e)
        acc[e] = 0.0f;
    int slot = 0;
    for (int64_t first = (int64_t)blockIdx.x * teams; first < a.rows; first += (int64_t)gridDim.x * teams, slot ^= 1) {
        const bool on = first + team < a.rows;
        const int64_t row = on ? first + team : a.rows - 1, at = row * a.cols;
        float g[8 * C], h[8 * C];
        load_row<XT, C, VEC>(static_cast<const XT*>(a.dy) + at, a.cols, lanes, tl, g);
        load_row<RT, C, VEC>(static_cast<const RT*>(a.h) + at, a.cols, lanes, tl, h);
        const float rstd = a.rstd[row];
        float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < C; ++k) {
            float w[8];
            factors<VEC>(a.weight, a.w_bf16, a.offset, a.cols, lanes, tl, k, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = 8 * k + j;
                if (on)
                    acc[e] = fmaf(g[e], h[e] * rstd, acc[e]);
                g[e] *= w[j];
                v.x = fmaf(g[e], h[e], v.x);
            }
        }
        v = over_team<false>(v, lanes, part, slot);
        const float b = rstd * (__fdiv_rn(v.x * rstd, (float)a.cols) * rstd);
#pragma unroll
        for (int e = 0; e < 8 * C; ++e)
            g[e] = fmaf(rstd, g[e], -b * h[e]);
        if (on)
            store_grads<XT, RT, C, VEC>(a, at, a.cols, lanes, tl, g);
    }
    if (!a.ws)
        return;
    float* ws = a.ws + (int64_t)blockIdx.x * a.cols;
    if (teams > 1) {  // 8 warps or more teams of a row of at most 1024 columns
        store_row<float, C, false>(sums + team * a.cols, VEC ? 0 : a.cols, lanes, tl, acc);
        if (VEC) {
#pragma unroll
            for (int e = 0; e < 8 * C; ++e)
                if (const int c = ((e >> 3) * lanes + tl) * 8 + (e & 7); c < a.cols)
                    sums[team * a.cols + c] = acc[e];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            float s = 0.0f;
            for (int t = 0; t < teams; ++t)
                s += sums[t * a.cols + c];
            ws[c] = s;
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8 * C; ++e)
        if (const int c = VEC ? ((e >> 3) * lanes + tl) * 8 + (e & 7) : e * lanes + tl; c < a.cols)
            ws[c] = acc[e];
}

// Rows that do not fit a block's registers: the sums u * h of every row first,
// then the gradients a slab of columns at a time.
template <typename XT, typename RT, bool VEC>
__global__ void __launch_bounds__(kMaxLanes)
row_dots(const Args a)
{
    __shared__ float2 part[2][32];
    const int lanes = a.lanes, tl = threadIdx.x, piece = 8 * lanes;
    int slot = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, slot ^= 1) {
        float2 v = make_float2(0.0f, 0.0f);
        for (int c0 = 0; c0 < a.cols; c0 += piece) {
            const int cols = a.cols - c0 < piece ? a.cols - c0 : piece;
            float g[8], h[8], w[8];
            load_row<XT, 1, VEC>(static_cast<const XT*>(a.dy) + row * a.cols + c0, cols, lanes, tl, g);
            load_row<RT, 1, VEC>(static_cast<const RT*>(a.h) + row * a.cols + c0, cols, lanes, tl, h);
            const char* wp = static_cast<const char*>(a.weight);
            factors<VEC>(wp ? wp + (int64_t)c0 * (a.w_bf16 ? 2 : 4) : wp, a.w_bf16, a.offset, cols, lanes, tl, 0, w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v.x = fmaf(g[j] * w[j], h[j], v.x);
        }
        v = over_team<false>(v, lanes, part, slot);
        if (tl == 0)
            a.dots[row] = v.x;
    }
}

template <typename XT, typename RT, bool VEC>
__global__ void __launch_bounds__(kThreads)
slab_bwd(const Args a)
{
    const int lanes = kThreads, tl = threadIdx.x, c0 = blockIdx.x * 8 * lanes;
    const int cols = a.cols - c0 < 8 * lanes ? a.cols - c0 : 8 * lanes;
    float acc[8], w[8];
    const char* wp = static_cast<const char*>(a.weight);
    factors<VEC>(wp ? wp + (int64_t)c0 * (a.w_bf16 ? 2 : 4) : wp, a.w_bf16, a.offset, cols, lanes, tl, 0, w);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        acc[j] = 0.0f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const int64_t at = row * a.cols + c0;
        float g[8], h[8];
        load_row<XT, 1, VEC>(static_cast<const XT*>(a.dy) + at, cols, lanes, tl, g);
        load_row<RT, 1, VEC>(static_cast<const RT*>(a.h) + at, cols, lanes, tl, h);
        const float rstd = a.rstd[row], b = rstd * (__fdiv_rn(a.dots[row] * rstd, (float)a.cols) * rstd);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            acc[j] = fmaf(g[j], h[j] * rstd, acc[j]);
            g[j] = fmaf(rstd, g[j] * w[j], -b * h[j]);
        }
        store_grads<XT, RT, 1, VEC>(a, at, cols, lanes, tl, g);
    }
    if (a.ws)
        store_row<float, 1, false>(a.ws + (int64_t)blockIdx.y * a.cols + c0, VEC ? 0 : cols, lanes, tl, acc);
    if (a.ws && VEC) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (tl * 8 + j < cols)
                a.ws[(int64_t)blockIdx.y * a.cols + c0 + tl * 8 + j] = acc[j];
    }
}

Layout layout(int64_t cols, bool vec)
{
    const int64_t units = (cols + 7) / 8;
    Layout l = {4, 32, 256, false};
    if (units <= 32 * 4) {
        l.C = units <= 32 ? 1 : units <= 64 ? 2 : 4;
        while (vec && l.C == 1 && l.lanes > 8 && units <= l.lanes / 2)
            l.lanes /= 2;
        return l;
    }
    l.C = units <= 256 ? 1 : units <= 1024 ? 2 : 4;
    l.longer = cols > kInRegisters;
    l.lanes = l.threads = l.longer ? kMaxLanes : (int)(((units + l.C - 1) / l.C + 31) / 32 * 32);
    return l;
}

size_t team_smem(const Layout& l, int64_t cols) { return l.lanes < l.threads ? (size_t)(l.threads / l.lanes) * cols * 4 : 0; }

struct Plan {
    int64_t blocks;    // partial sums of a column
    int64_t ws, dots;  // floats of each in the workspace
};

template <typename XT, typename RT>
const void* kernel_of(int C, bool vec)
{
    if (vec)
        return C == 1   ? reinterpret_cast<const void*>(norm_bwd<XT, RT, 1, true>)
               : C == 2 ? reinterpret_cast<const void*>(norm_bwd<XT, RT, 2, true>)
                        : reinterpret_cast<const void*>(norm_bwd<XT, RT, 4, true>);
    return C == 1   ? reinterpret_cast<const void*>(norm_bwd<XT, RT, 1, false>)
           : C == 2 ? reinterpret_cast<const void*>(norm_bwd<XT, RT, 2, false>)
                    : reinterpret_cast<const void*>(norm_bwd<XT, RT, 4, false>);
}

// The same blocks whether the buffers are aligned or not: the workspace's
// size goes by sizes and types alone.
template <typename XT, typename RT>
Plan plan(int64_t rows, int64_t cols)
{
    const Layout l = layout(cols, cols % 8 == 0);
    Plan p = {0, 0, 0};
    if (l.longer) {
        const int64_t slabs = (cols + 8 * kThreads - 1) / (8 * kThreads);
        int64_t lanes = (4 * sm_count() + slabs - 1) / slabs;
        lanes = lanes < 65535 ? lanes : 65535;
        p.blocks = rows < lanes ? rows : lanes;
        p.dots = (rows + 3) / 4 * 4;
    } else {
        const int64_t teams = l.threads / l.lanes, need = (rows + teams - 1) / teams;
        const int64_t room =
            (int64_t)sm_count() * occupancy(kernel_of<XT, RT>(l.C, cols % 8 == 0), l.threads, team_smem(l, cols));
        p.blocks = need < room ? need : room;
    }
    p.ws = p.blocks * cols;
    return p;
}

template <typename XT, typename RT, int C, bool VEC>
void launch(const Args& a, const Layout& l, int64_t blocks, cudaStream_t s)
{
    norm_bwd<XT, RT, C, VEC><<<(unsigned)blocks, l.threads, team_smem(l, a.cols), s>>>(a);
}

template <typename XT, typename RT, bool VEC>
int launch_any(Args a, const Plan& p, cudaStream_t s)
{
    const Layout l = layout(a.cols, VEC);
    a.lanes = l.lanes;
    if (l.longer) {
        const int64_t room = (int64_t)sm_count() * 4;
        row_dots<XT, RT, VEC><<<(unsigned)(a.rows < room ? a.rows : room), l.threads, 0, s>>>(a);
        if (const int st = launch_status(); st != MFX_OK)
            return st;
        const dim3 grid((unsigned)((a.cols + 8 * kThreads - 1) / (8 * kThreads)), (unsigned)p.blocks);
        slab_bwd<XT, RT, VEC><<<grid, kThreads, 0, s>>>(a);
        return launch_status();
    }
    switch (l.C) {
    case 1: launch<XT, RT, 1, VEC>(a, l, p.blocks, s); break;
    case 2: launch<XT, RT, 2, VEC>(a, l, p.blocks, s); break;
    default: launch<XT, RT, 4, VEC>(a, l, p.blocks, s); break;
    }
    return launch_status();
}

template <typename XT, typename RT>
int run(int w_dt, Args& a, void* dweight, void* workspace, size_t* bytes, bool vec, cudaStream_t s)
{
    const Plan p = plan<XT, RT>(a.rows, a.cols);
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
    if (const int st = vec ? launch_any<XT, RT, true>(a, p, s) : launch_any<XT, RT, false>(a, p, s); st != MFX_OK)
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
