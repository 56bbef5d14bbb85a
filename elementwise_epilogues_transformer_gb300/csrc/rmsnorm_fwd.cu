// rmsnorm_fwd.cu -- root-mean-square norm with the residual's addition, and
// with an output in 8 bits with scales.
//
//   h = x + residual,   rstd = 1 / sqrt(mean(h^2) + eps),
//   y = h * rstd * (weight + offset),
// and in 8 bits, per group of a row's columns,
//   s = max |y| / largest,   q = y / s.
// h stays in fp32 registers between the sum of its squares and y, so x and
// the residual are read once, h and y (or q) written once; h is rounded only
// where it is stored for the next layer.  rstd is a common factor of a row:
// the largest |h * weight| is found along with the sum, and h * weight goes to
// q by one factor rstd / s.
//
// What bounds it: HBM, at one read and one write of everything; with 8-bit
// outputs the issue slots come near (a group's maximum and scale, the
// conversions: some 30 instructions an element at 70 % of the slots).
// Measured: 16384x4096 bf16 with an fp32 residual 132 us (6120 GB/s, 0.90 of
// the copy rate), all bf16 89 us; 8192x8192 bf16 89 us, as e4m3 with a scale a
// row 80.5 us (5830 GB/s); 16384x4096 as e4m3 with a power of two per 32
// columns 80 us; 3001x2051 fp32 (single columns) 16.8 us (5850 GB/s);
// 8192x4099 bf16 66 us (4050 GB/s: two bytes an access); one row of 4096 2.6 us.
#include "rmsnorm.cuh"

#include <cmath>

namespace mfx {
namespace rmsnorm {
namespace {

struct Args {
    int64_t rows;
    int cols, lanes, depth;
    uint32_t row_bytes, x_bytes;  // of a row on its way: all of it, x's part
    const void *x, *residual, *weight;
    bool w_bf16;
    float eps, offset;
    void *y, *h;
    float* rstd;
    // output in 8 bits
    bool e5m2, e8m0;
    int group, shift, groups;  // columns of a group (0: the row) and their logarithm, groups of a row
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
// is at least 2^-126 and at most 2^125, so that its reciprocal is a normal
// number and infinities saturate.  Both types' largest values are 1.75 times a
// power of two (448 = 1.75 * 2^8, 57344 = 1.75 * 2^15): rounding up to a power
// of two is a matter of the exponent, and exact.  Other scales are formed by a
// product with the rounded reciprocal (2 roundings instead of 1: the divisions
// cost more than all else in a group).
struct Scale {
    float s, inv;
};
__device__ __forceinline__ Scale scale_of(float top, bool e5m2, bool e8m0)
{
    constexpr float least = 1.17549435e-38f, most = 4.25352959e37f;
    Scale r;
    if (e8m0) {
        const uint32_t up = (__float_as_uint(fminf(top, 1e38f)) + 0x1FFFFFu) & 0x7F800000u, by = (e5m2 ? 15u : 8u) << 23;
        const uint32_t b = min(max(up, by + (1u << 23)) - by, __float_as_uint(most));
        r.s = __uint_as_float(b);
        r.inv = __uint_as_float((254u << 23) - b);
    } else {
        r.s = fminf(fmaxf(top * (e5m2 ? 1.0f / 57344.0f : 1.0f / 448.0f), least), most);
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.inv) : "f"(r.s));
    }
    if (!(top > 0.0f))  // zeros, or nothing but NaN
        r.s = r.inv = 1.0f;
    return r;
}

__device__ __forceinline__ void put_scale(const Args& a, int64_t i, float s)
{
    if (a.e8m0)
        static_cast<uint8_t*>(a.scale)[i] = (uint8_t)(__float_as_uint(s) >> 23);
    else
        static_cast<float*>(a.scale)[i] = s;
}

template <int V>
__device__ __forceinline__ void store_fp8(uint8_t* q, const float (&y)[V], float inv, bool e5m2)
{
    if constexpr (V == 1) {
        *q = (uint8_t)pack_fp8x2(y[0] * inv, 0.0f, e5m2);
    } else {
        uint32_t b[V / 4];
        const auto pack = [&](bool as_e5m2) {
#pragma unroll
            for (int j = 0; j < V / 4; ++j)
                b[j] = pack_fp8x2(y[4 * j] * inv, y[4 * j + 1] * inv, as_e5m2) |
                       pack_fp8x2(y[4 * j + 2] * inv, y[4 * j + 3] * inv, as_e5m2) << 16;
        };
        if (e5m2)
            pack(true);
        else
            pack(false);
        if constexpr (V == 8)
            st8(q, make_uint2(b[0], b[1]));
        else
            asm volatile(MFX_ST_OP ".u32 [%0], %1;" ::"l"(q), "r"(b[0]) : "memory");
    }
}

// rstd as a power of two and what is left of it, in [1, 2).  Where the largest
// of a group is below some 1e-36 (e4m3) or 1e-34 (e5m2) and rstd above 4, rstd
// times a scale's reciprocal passes fp32's range, though y and s do not: the
// power goes to the values first, which is exact, and what is left times a
// reciprocal (2^126 at most) stays within.  Only where a thread's values are
// below kTiny, or in single columns: for every row whose rstd is above 2 the
// products cost more (16384x4096 bf16 with rows of 0.05, per 128 columns: 84.8
// us, 82.6 with the question asked, 81.8 without either).
constexpr float kTiny = 1e-33f;
struct Parts {
    float power, rest;
};
__device__ __forceinline__ Parts parts_of(float rstd, bool tiny)
{
    if (!tiny || !(rstd >= 2.0f))  // NaN stays
        return {1.0f, rstd};
    const uint32_t b = __float_as_uint(rstd);
    return {__uint_as_float(b & 0x7F800000u), __uint_as_float((b & 0x007FFFFFu) | 0x3F800000u)};
}

// One scale for the values of a thread's N units from their largest absolute
// value in the group; `c`: the first unit's column.
__device__ __forceinline__ Scale group_scale(const Args& a, float top, int64_t scales, int c, bool put)
{
    const Scale s = scale_of(top, a.e5m2, a.e8m0);
    if (put)
        put_scale(a, scales + (c >> a.shift), s.s);
    return s;
}

// Q: y as it is (0), in 8 bits with a scale per row (1) or per group of columns (2).
template <typename XT, typename RT, int V, int E, int Q>
__global__ void __launch_bounds__(E == 8 ? 1024 : 512, E == 32 ? 1 : E == 16 ? 2 : 1)
norm_fwd(const Args a)
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
    const XT* const x = static_cast<const XT*>(a.x);
    const RT* const res = static_cast<const RT*>(a.residual);
    int64_t row = (int64_t)blockIdx.x * teams + team;
    const auto start = [&](int64_t r, uint32_t to) {
        if (r - team < a.rows) {  // a team past the end takes the last row
            const int64_t at = (r < a.rows ? r : a.rows - 1) * cols;
            copy_row<XT, V, E>(to, x + at, cols, x, x + all, lanes, tl, mine);
            if (res)
                copy_row<RT, V, E>(to + a.x_bytes, res + at, cols, res, res + all, lanes, tl, mine);
        }
        copies_commit();
    };
    int64_t next = row;
    for (uint32_t to = ring; to != end; to += a.row_bytes, next += step) {
        clear_rest<XT, V, E>(to, tl, mine);
        if (res)
            clear_rest<RT, V, E>(to + a.x_bytes, tl, mine);
        start(next, to);
    }
    float w[N][V];
    factors_of<V, E>(a.weight, a.w_bf16, a.offset, mine, tl, w);
    int slot = 0;
    uint32_t buf = ring;
    for (; row - team < a.rows; row += step, next += step, slot ^= 1) {
        const bool on = row < a.rows;
        const int64_t at = (on ? row : a.rows - 1) * cols;
        const int put = on ? mine : 0;  // units to store
        copies_wait(a.depth - 1);
        if (!VEC)
            team_barrier(lanes);
        const uint32_t sx = buf + (VEC ? 0u : where(x + at)) + c0 * (uint32_t)sizeof(XT);
        const uint32_t sr = buf + a.x_bytes + (VEC || !res ? 0u : where(res + at)) + c0 * (uint32_t)sizeof(RT);
        float f[N][V];
        float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < N; ++k)
            read_unit<XT, V>(sx, k, mine, f[k]);
        if (res) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                float g[V];
                read_unit<RT, V>(sr, k, mine, g);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    f[k][j] += g[j];
            }
        }
        if (a.h) {
            RT* h = static_cast<RT*>(a.h) + at + c0;
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (k < put)
                    store_unit<RT, V>(h + k * 32 * V, f[k]);
        }
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v.x = fmaf(f[k][j], f[k][j], v.x);
                f[k][j] *= w[k][j];
                if (Q == 1)
                    v.y = amax(v.y, f[k][j]);
            }
        v = over_team<Q == 1>(v, lanes, part, slot);
        start(next, buf);  // all have what they read there: it is in the sum
        buf = buf + a.row_bytes == end ? ring : buf + a.row_bytes;
        const float rstd = __frsqrt_rn(__fdiv_rn(v.x, (float)cols) + a.eps);
        if (a.rstd && on && tl == 0)
            a.rstd[row] = rstd;
        if constexpr (Q == 0) {
            XT* y = static_cast<XT*>(a.y) + at + c0;
#pragma unroll
            for (int k = 0; k < N; ++k) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    f[k][j] *= rstd;
                if (k < put)
                    store_unit<XT, V>(y + k * 32 * V, f[k]);
            }
        } else {
            uint8_t* q = static_cast<uint8_t*>(a.y) + at + c0;
            const int64_t scales = (on ? row : 0) * a.groups;
            const int share = min(a.group >> (V == 8 ? 3 : V == 4 ? 2 : 0), min(lanes, 32));  // lanes of a group
            Scale s = {1.0f, 1.0f};
            // groups' maxima by units (vectors), before any power
            float tops[N], lowest = INFINITY;
            if (Q == 2 && V > 1) {
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    tops[k] = 0.0f;
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        tops[k] = amax(tops[k], f[k][j]);
                    lowest = fminf(lowest, tops[k]);
                }
            }
            const Parts r = parts_of(rstd, Q == 1 ? v.y < kTiny : V == 1 || lowest < kTiny);
            if (r.power != 1.0f) {
#pragma unroll
                for (int k = 0; k < N; ++k)
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        f[k][j] *= r.power;
            }
            if (Q == 1) {
                s = scale_of(v.y * rstd, a.e5m2, a.e8m0);
                if (on && tl == 0)
                    put_scale(a, row, s.s);
            }
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int c = c0 + k * 32 * V;
                if (Q == 2 && V > 1) {
                    float top = tops[k];
                    for (int o = share >> 1; o > 0; o >>= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                    s = group_scale(a, top * rstd, scales, c, k < put && (c & (a.group - 1)) == 0);
                } else if (Q == 2 && a.group == 32) {
                    const int top = __reduce_max_sync(0xFFFFFFFFu, __float_as_int(amax(0.0f, f[k][0])));
                    s = group_scale(a, __int_as_float(top) * r.rest, scales, c, k < put && (tl & 31) == 0);
                } else if (Q == 2 && k % 4 == 0) {  // a warp's four steps
                    float mine = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mine = amax(mine, f[(k + i) % N][0]);
                    const int top = __reduce_max_sync(0xFFFFFFFFu, __float_as_int(mine));
                    s = group_scale(a, __int_as_float(top) * r.rest, scales, c, k < put && (tl & 31) == 0);
                }
                // (h * weight) * (rstd / s): one rounding less than y itself has
                const float by = r.rest * s.inv;
                if (k < put)
                    store_fp8<V>(q + k * 32 * V, f[k], by, a.e5m2);
            }
        }
    }
}

// Rows longer than that: read twice, column by column, a warp's four steps of
// 32 columns a round.
template <typename XT, typename RT, bool Q>
__global__ void __launch_bounds__(1024, 1)
norm_fwd_long(const Args a)
{
    __shared__ float2 part[2][32];
    const int lane = threadIdx.x & 31, first = (threadIdx.x >> 5) * 128 + lane;
    int slot = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, slot ^= 1) {
        const int64_t at = row * a.cols;
        const XT* x = static_cast<const XT*>(a.x) + at;
        const RT* r = a.residual ? static_cast<const RT*>(a.residual) + at : nullptr;
        float2 v = make_float2(0.0f, 0.0f);
        float f[4], w[4][1];
        const auto read = [&](int c0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + 32 * i;
                f[i] = w[i][0] = 0.0f;
                if (c < a.cols) {
                    f[i] = load1(x + c) + (r ? load1(r + c) : 0.0f);
                    factors<1>(a.weight, a.w_bf16, a.offset, c, w[i]);
                }
            }
        };
        for (int c0 = first; c0 - lane < a.cols; c0 += 4096) {
            read(c0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v.x = fmaf(f[i], f[i], v.x);
                if (Q)
                    v.y = amax(v.y, f[i] * w[i][0]);
            }
        }
        v = over_team<Q>(v, 1024, part, slot);
        const float rstd = __frsqrt_rn(__fdiv_rn(v.x, (float)a.cols) + a.eps);
        if (a.rstd && threadIdx.x == 0)
            a.rstd[row] = rstd;
        Scale s = {1.0f, 1.0f};
        const Parts p = parts_of(rstd, true);
        if (Q && a.group == 0) {
            s = scale_of(v.y * rstd, a.e5m2, a.e8m0);
            if (threadIdx.x == 0)
                put_scale(a, row, s.s);
        }
        for (int c0 = first; c0 - lane < a.cols; c0 += 4096) {
            read(c0);
            float tops[4];
            if (Q && a.group) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tops[i] = __int_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_int(amax(0.0f, f[i] * w[i][0]))));
                if (a.group == 128)
                    tops[0] = tops[1] = tops[2] = tops[3] = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + 32 * i;
                if (Q && a.group)
                    s = group_scale(a, tops[i] * rstd, row * a.groups, c, lane == 0 && c < a.cols && (c & (a.group - 1)) == 0);
                if (c >= a.cols)
                    continue;
                if (a.h)
                    store1(static_cast<RT*>(a.h) + at + c, f[i]);
                if constexpr (Q) {
                    const float y[1] = {f[i] * w[i][0] * p.power};
                    store_fp8<1>(static_cast<uint8_t*>(a.y) + at + c, y, p.rest * s.inv, a.e5m2);
                } else {
                    store1(static_cast<XT*>(a.y) + at + c, f[i] * w[i][0] * rstd);
                }
            }
        }
    }
}

template <typename K>
int launch(K kernel, const Args& a, const Layout& l, cudaStream_t s)
{
    const int64_t teams = l.threads / l.lanes, need = (a.rows + teams - 1) / teams;
    const int64_t room = (int64_t)sm_count() * occupancy(reinterpret_cast<const void*>(kernel), l.threads, l.smem);
    kernel<<<(unsigned)(need < room ? need : room), l.threads, l.smem, s>>>(a);
    return launch_status();
}

template <typename XT, typename RT, int V, int Q>
int with_units(const Args& a, const Layout& l, cudaStream_t s)
{
    if (l.E == 8)
        return launch(norm_fwd<XT, RT, V, 8, Q>, a, l, s);
    if (l.E == 16)
        return launch(norm_fwd<XT, RT, V, 16, Q>, a, l, s);
    return launch(norm_fwd<XT, RT, V, 32, Q>, a, l, s);
}

// fp32 with a bf16 residual is no mix that training makes: it goes column by
// column.
template <typename XT, typename RT, bool Q>
int with_types(Args a, bool vec, cudaStream_t s)
{
    constexpr int V = sizeof(XT) > sizeof(RT) ? 1 : sizeof(RT) == 2 ? 8 : 4;
    const auto x_bytes = [](int64_t room) { return ((size_t)room * sizeof(XT) + kPad + 15) / 16 * 16; };
    const bool res = a.residual != nullptr;
    // One type and no groups: 32 elements a thread (65536x1024 bf16 91 us, 96 with 8; 16384x4096 89, 91.5 with 16; to
    // e4m3 by rows 8192x8192 80.5, 84).  A group's maximum and scale, and two types, leave registers for fewer (e4m3 by
    // 32 columns 16384x4096 79.5, 86 with 32 and 89 with 8; single columns 3001x2051 fp32 16.7, 18.4 with 32).
    const bool wide = sizeof(XT) == sizeof(RT) && vec && !a.group;
    const Layout l = layout(a.rows, a.cols, vec ? V : 1, wide ? 512 : 2048, wide ? 512 : 8192,
                            [&](int64_t room) { return x_bytes(room) + (res ? (size_t)room * sizeof(RT) + kPad : 0); },
                            [](int e) { return e == 32 ? 512 : 1024; });
    a.x_bytes = (uint32_t)x_bytes(l.room);
    if (l.depth == 0) {
        a.lanes = 1024;
        return launch(norm_fwd_long<XT, RT, Q>, a, Layout{0, 1024, 1024, 0, 0, 0, 0}, s);
    }
    a.lanes = l.lanes, a.depth = l.depth, a.row_bytes = (uint32_t)l.row;
    if (Q && a.group)
        return vec ? with_units<XT, RT, V, Q ? 2 : 0>(a, l, s) : with_units<XT, RT, 1, Q ? 2 : 0>(a, l, s);
    return vec ? with_units<XT, RT, V, Q>(a, l, s) : with_units<XT, RT, 1, Q>(a, l, s);
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
    a.group = (int)group, a.shift = group == 32 ? 5 : 7, a.groups = group ? (int)((cols + group - 1) / group) : 1;
    return rmsnorm::run<true>(x_dt, res_dt, w_dt, rows, cols, rows * cols,
                              rows * a.groups * (scale_dt == MFX_E8M0 ? 1 : 4), a, stream);
}

}  // extern "C"
