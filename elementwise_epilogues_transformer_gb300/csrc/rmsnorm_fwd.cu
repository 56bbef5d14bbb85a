// rmsnorm_fwd.cu -- root-mean-square norm with the residual's addition, and
// with an output in 8 bits with scales.
//
//   h = x + residual,   rstd = 1 / sqrt(mean(h^2) + eps),
//   y = h * rstd * (weight + offset),
// and in 8 bits, per group of a row's columns,
//   s = max |y| / largest,   q = y / s.
// h stays in fp32 registers between the sum of its squares and y, so x and
// the residual are read once, h and y (or q) written once; h is rounded only
// where it is stored for the next layer.
#include "rmsnorm.cuh"

#include <cmath>

namespace mfx {
namespace rmsnorm {
namespace {

struct Args {
    int64_t rows;
    int cols, lanes;
    const void *x, *residual, *weight;
    bool w_bf16;
    float eps, offset;
    void *y, *h;
    float* rstd;
    // output in 8 bits
    bool e5m2, e8m0;
    int group, groups;  // columns of a group (0: the row), groups of a row
    void* scale;
};

// Two values to two bytes, rounded to nearest even and saturated at the
// type's largest value; NaN stays NaN.
__device__ __forceinline__ uint32_t pack_fp8x2(float lo, float hi, bool e5m2)
{
    uint16_t d;
    if (e5m2)
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// A group's scale from its largest absolute value, and the factor that takes
// values to the 8-bit type's range.  The scale of a group of zeros is 1; it
// is at least 2^-126 so that its reciprocal is finite, and finite, so that
// infinities saturate.  Powers of two are rounded up: nothing saturates.
struct Scale {
    float s, inv;
};
__device__ __forceinline__ Scale scale_of(float top, bool e5m2, bool e8m0)
{
    float s = __fdiv_rn(top, e5m2 ? 57344.0f : 448.0f);
    s = fminf(fmaxf(s, 1.17549435e-38f), 1e38f);
    if (e8m0) {
        const uint32_t b = __float_as_uint(s);
        s = __uint_as_float((b + 0x7FFFFFu) & 0x7F800000u);
    }
    if (top == 0.0f)
        s = 1.0f;
    return {s, __fdiv_rn(1.0f, s)};
}

__device__ __forceinline__ void put_scale(const Args& a, int64_t i, float s)
{
    if (a.e8m0)
        static_cast<uint8_t*>(a.scale)[i] = (uint8_t)(__float_as_uint(s) >> 23);
    else
        static_cast<float*>(a.scale)[i] = s;
}

// y of a piece of a row (its first column is c0) as 8 bits.  ROW: `row` holds
// the whole row's scale.
template <int C, bool VEC>
__device__ __forceinline__ void store_fp8(const Args& a, int64_t row, int c0, int cols, int tl, const float (&y)[8 * C],
                                          Scale row_scale, int* tops, bool on)
{
    uint8_t* q = static_cast<uint8_t*>(a.y) + row * a.cols + c0;
    const int lanes = a.lanes;
    if constexpr (VEC) {
        const int n = a.group / 8 < lanes ? a.group / 8 : lanes;  // lanes of a group
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const int c = (k * lanes + tl) * 8;
            Scale s = row_scale;
            if (a.group) {
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    top = amax(top, y[8 * k + j]);
                for (int o = n >> 1; o > 0; o >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                s = scale_of(top, a.e5m2, a.e8m0);
                if (on && c < cols && (tl & (n - 1)) == 0)
                    put_scale(a, row * a.groups + (c0 + c) / a.group, s.s);
            }
            if (on && c < cols) {
                uint32_t b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    b[j] = pack_fp8x2(y[8 * k + 2 * j] * s.inv, y[8 * k + 2 * j + 1] * s.inv, a.e5m2);
                st8(q + c, make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16));
            }
        }
    } else {
        // a warp's e-th elements are 32 columns, one group of 32 or a part of one of 128
        const int g = a.group, first = tl & ~31, lane = tl & 31;
        if (g > 32) {
            for (int i = tl; i * g < 8 * C * lanes; i += lanes)
                tops[i] = 0;
            lanes > 32 ? __syncthreads() : __syncwarp();
        }
#pragma unroll
        for (int e = 0; e < 8 * C; ++e) {
            const int c = e * lanes + tl;
            Scale s = row_scale;
            if (g) {
                const int top = __reduce_max_sync(0xFFFFFFFFu, __float_as_int(amax(0.0f, y[e])));
                if (g > 32) {
                    if (lane == 0)
                        atomicMax(&tops[(e * lanes + first) / g], top);
                    continue;
                }
                s = scale_of(__int_as_float(top), a.e5m2, a.e8m0);
                if (on && lane == 0 && c < cols)
                    put_scale(a, row * a.groups + (c0 + c) / g, s.s);
            }
            if (on && c < cols)
                q[c] = (uint8_t)pack_fp8x2(y[e] * s.inv, 0.0f, a.e5m2);
        }
        if (g > 32) {
            lanes > 32 ? __syncthreads() : __syncwarp();
#pragma unroll
            for (int e = 0; e < 8 * C; ++e) {
                const int c = e * lanes + tl;
                if (on && c < cols) {
                    const Scale s = scale_of(__int_as_float(tops[c / g]), a.e5m2, a.e8m0);
                    if (c % g == 0)
                        put_scale(a, row * a.groups + (c0 + c) / g, s.s);
                    q[c] = (uint8_t)pack_fp8x2(y[e] * s.inv, 0.0f, a.e5m2);
                }
            }
            lanes > 32 ? __syncthreads() : __syncwarp();
        }
    }
}

// h of a piece of a row, in fp32.
template <typename XT, typename RT, int C, bool VEC>
__device__ __forceinline__ void load_h(const Args& a, int64_t at, int cols, int tl, float (&f)[8 * C])
{
    load_row<XT, C, VEC>(static_cast<const XT*>(a.x) + at, cols, a.lanes, tl, f);
    if (a.residual) {
        float r[8 * C];
        load_row<RT, C, VEC>(static_cast<const RT*>(a.residual) + at, cols, a.lanes, tl, r);
#pragma unroll
        for (int e = 0; e < 8 * C; ++e)
            f[e] += r[e];
    }
}

template <int C>
constexpr int max_threads() { return C == 2 ? 512 : 1024; }

// LONG: rows that do not fit a block's registers are walked twice in pieces
// of 8 C elements a thread, the second time from L2.
template <typename XT, typename RT, int C, bool VEC, bool Q, bool LONG>
__global__ void __launch_bounds__(max_threads<C>())
norm_fwd(const Args a)
{
    __shared__ float2 part[2][32];
    __shared__ int tops_of[Q && !VEC ? 256 : 1];
    const int lanes = a.lanes, teams = blockDim.x / lanes, team = threadIdx.x / lanes, tl = threadIdx.x % lanes;
    int* tops = tops_of + (teams > 1 ? team * (8 * C * 32 / 128) : 0);
    const int piece = LONG ? 8 * C * lanes : a.cols;
    int slot = 0;
    for (int64_t first = (int64_t)blockIdx.x * teams; first < a.rows; first += (int64_t)gridDim.x * teams, slot ^= 1) {
        const bool on = first + team < a.rows;
        const int64_t row = on ? first + team : a.rows - 1, at = row * a.cols;  // a team past the end reads the last
        float f[8 * C];
        float2 v = make_float2(0.0f, 0.0f);
        for (int c0 = 0; c0 < a.cols; c0 += piece) {
            const int cols = a.cols - c0 < piece ? a.cols - c0 : piece;
            load_h<XT, RT, C, VEC>(a, at + c0, cols, tl, f);
#pragma unroll
            for (int e = 0; e < 8 * C; ++e)
                v.x = fmaf(f[e], f[e], v.x);
            if (Q && a.group == 0) {
                const char* w = static_cast<const char*>(a.weight);
                w = w ? w + (int64_t)c0 * (a.w_bf16 ? 2 : 4) : w;
#pragma unroll
                for (int k = 0; k < C; ++k) {
                    float wk[8];
                    factors<VEC>(w, a.w_bf16, a.offset, cols, lanes, tl, k, wk);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v.y = amax(v.y, f[8 * k + j] * wk[j]);
                }
            }
        }
        v = over_team<Q>(v, lanes, part, slot);
        const float rstd = __frsqrt_rn(__fdiv_rn(v.x, (float)a.cols) + a.eps);
        if (a.rstd && on && tl == 0)
            a.rstd[row] = rstd;
        Scale s = {1.0f, 1.0f};
        if (Q && a.group == 0) {
            s = scale_of(v.y * rstd, a.e5m2, a.e8m0);
            if (on && tl == 0)
                put_scale(a, row, s.s);
        }
        for (int c0 = 0; c0 < a.cols; c0 += piece) {
            const int cols = a.cols - c0 < piece ? a.cols - c0 : piece;
            if (LONG)
                load_h<XT, RT, C, VEC>(a, at + c0, cols, tl, f);
            if (a.h && on)
                store_row<RT, C, VEC>(static_cast<RT*>(a.h) + at + c0, cols, lanes, tl, f);
            const char* w = static_cast<const char*>(a.weight);
            w = w ? w + (int64_t)c0 * (a.w_bf16 ? 2 : 4) : w;
#pragma unroll
            for (int k = 0; k < C; ++k) {
                float wk[8];
                factors<VEC>(w, a.w_bf16, a.offset, cols, lanes, tl, k, wk);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    f[8 * k + j] = f[8 * k + j] * rstd * wk[j];
            }
            if constexpr (Q)
                store_fp8<C, VEC>(a, row, c0, cols, tl, f, s, tops, on);
            else if (on)
                store_row<XT, C, VEC>(static_cast<XT*>(a.y) + at + c0, cols, lanes, tl, f);
        }
    }
}

// Rows in a warp's lanes up to 1024 columns, in a block's threads up to 32768.
Layout layout(int64_t rows, int64_t cols, bool vec, int sms)
{
    const int64_t units = (cols + 7) / 8;
    Layout l = {4, 32, 256, false};
    if (units <= 32 * 4) {
        l.C = units <= 32 ? 1 : units <= 64 ? 2 : 4;
        while (vec && l.C == 1 && l.lanes > 8 && units <= l.lanes / 2)
            l.lanes /= 2;
        return l;
    }
    // few rows: one run a thread, the shortest way through the block
    l.C = units <= 256 || (rows <= 2 * sms && units <= 1024) ? 1 : units <= 1024 ? 2 : 4;
    l.longer = units > 1024 * 4;
    const int64_t want = (units + l.C - 1) / l.C;
    l.lanes = l.threads = l.longer ? 1024 : (int)((want + 31) / 32 * 32);
    return l;
}

template <typename XT, typename RT, int C, bool VEC, bool Q, bool LONG>
int launch(const Args& a, const Layout& l, cudaStream_t s)
{
    const void* kernel = reinterpret_cast<const void*>(norm_fwd<XT, RT, C, VEC, Q, LONG>);
    const int64_t teams = l.threads / l.lanes, need = (a.rows + teams - 1) / teams;
    const int64_t room = (int64_t)sm_count() * occupancy(kernel, l.threads, 0);
    norm_fwd<XT, RT, C, VEC, Q, LONG><<<(unsigned)(need < room ? need : room), l.threads, 0, s>>>(a);
    return launch_status();
}

template <typename XT, typename RT, bool VEC, bool Q>
int with_layout(const Args& a, const Layout& l, cudaStream_t s)
{
    if (l.longer)
        return launch<XT, RT, 4, VEC, Q, true>(a, l, s);
    switch (l.C) {
    case 1: return launch<XT, RT, 1, VEC, Q, false>(a, l, s);
    case 2: return launch<XT, RT, 2, VEC, Q, false>(a, l, s);
    default: return launch<XT, RT, 4, VEC, Q, false>(a, l, s);
    }
}

template <typename XT, typename RT, bool Q>
int with_types(const Args& a, bool vec, cudaStream_t s)
{
    const Layout l = layout(a.rows, a.cols, vec, sm_count());
    Args b = a;
    b.lanes = l.lanes;
    return vec ? with_layout<XT, RT, true, Q>(b, l, s) : with_layout<XT, RT, false, Q>(b, l, s);
}

template <bool Q>
int run(int x_dt, int res_dt, int w_dt, int64_t rows, int64_t cols, int64_t y_bytes, int64_t scale_bytes, Args& a,
        void* stream)
{
    if (!a.x || !a.y || (Q && !a.scale) || (a.h && !a.residual))
        return MFX_ERR_NULL;
    const int64_t n = rows * cols, xb = n * dtype_bytes(x_dt), rb = n * dtype_bytes(res_dt);
    const int64_t wb = cols * dtype_bytes(w_dt), sb = rows * 4;
    // every output may be an input's own buffer (element by element), nothing else
    struct Buf { const void* p; int64_t n; };
    const Buf in[2] = {{a.x, xb}, {a.residual, rb}}, out[4] = {{a.y, y_bytes}, {a.h, rb}, {a.rstd, sb}, {a.scale, scale_bytes}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 2; ++j)
            if (i < 2 ? partial_overlap(out[i].p, out[i].n, in[j].p, in[j].n) : overlaps(out[i].p, out[i].n, in[j].p, in[j].n))
                return MFX_ERR_ALIAS;
        if (overlaps(out[i].p, out[i].n, a.weight, wb))
            return MFX_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n))
                return MFX_ERR_ALIAS;
    }
    a.rows = rows, a.cols = (int)cols, a.w_bf16 = w_dt == MFX_BF16;
    const bool vec = cols % 8 == 0 && aligned16(a.x) && aligned16(a.residual) && aligned16(a.weight) &&
                     aligned16(a.h) && (Q ? aligned8(a.y) : aligned16(a.y));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (x_dt == MFX_BF16)
        return !a.residual || res_dt == MFX_BF16 ? with_types<bf16, bf16, Q>(a, vec, s)
                                                 : with_types<bf16, float, Q>(a, vec, s);
    return !a.residual || res_dt == MFX_F32 ? with_types<float, float, Q>(a, vec, s)
                                            : with_types<float, bf16, Q>(a, vec, s);
}

int check(int x_dt, int res_dt, int w_dt, int64_t rows, int64_t cols, float eps, float offset)
{
    if (!valid_dtype(x_dt) || !valid_dtype(res_dt) || !valid_dtype(w_dt))
        return MFX_ERR_DTYPE;
    if (!sizes_ok(rows, cols))
        return MFX_ERR_SHAPE;
    if (!(eps >= 0.0f) || std::isinf(eps) || !std::isfinite(offset))
        return MFX_ERR_VALUE;
    return MFX_OK;
}

}  // namespace
}  // namespace rmsnorm
}  // namespace mfx

extern "C" {

int mfx_add_rmsnorm_fwd(int x_dt, int res_dt, int w_dt, int64_t rows, int64_t cols, const void* x,
                        const void* residual, const void* weight, float eps, float weight_offset, void* y, void* h,
                        float* rstd, void* stream)
{
    using namespace mfx;
    if (const int st = rmsnorm::check(x_dt, res_dt, w_dt, rows, cols, eps, weight_offset); st != MFX_OK)
        return st;
    if (rows == 0 || cols == 0)
        return MFX_OK;
    rmsnorm::Args a = {};
    a.x = x, a.residual = residual, a.weight = weight, a.eps = eps, a.offset = weight_offset;
    a.y = y, a.h = h, a.rstd = rstd;
    return rmsnorm::run<false>(x_dt, res_dt, w_dt, rows, cols, rows * cols * dtype_bytes(x_dt), 0, a, stream);
}

int mfx_add_rmsnorm_quant_fwd(int x_dt, int res_dt, int w_dt, int64_t rows, int64_t cols, const void* x,
                              const void* residual, const void* weight, float eps, float weight_offset, int q_dt,
                              int64_t group, int scale_dt, void* q, void* scale, void* h, float* rstd, void* stream)
{
    using namespace mfx;
    if (const int st = rmsnorm::check(x_dt, res_dt, w_dt, rows, cols, eps, weight_offset); st != MFX_OK)
        return st;
    if ((q_dt != MFX_E4M3 && q_dt != MFX_E5M2) || (scale_dt != MFX_F32 && scale_dt != MFX_E8M0))
        return MFX_ERR_DTYPE;
    if (group != 0 && group != 32 && group != 128)
        return MFX_ERR_VALUE;
    if (rows == 0 || cols == 0)
        return MFX_OK;
    rmsnorm::Args a = {};
    a.x = x, a.residual = residual, a.weight = weight, a.eps = eps, a.offset = weight_offset;
    a.y = q, a.h = h, a.rstd = rstd, a.scale = scale;
    a.e5m2 = q_dt == MFX_E5M2, a.e8m0 = scale_dt == MFX_E8M0;
    a.group = (int)group, a.groups = group ? (int)((cols + group - 1) / group) : 1;
    return rmsnorm::run<true>(x_dt, res_dt, w_dt, rows, cols, rows * cols,
                              rows * a.groups * (scale_dt == MFX_E8M0 ? 1 : 4), a, stream);
}

}  // extern "C"
