// rmsnorm.cuh -- what the root-mean-square norm's forward and backward share:
// the layout of a row over a team of threads, and sums over a team.
#pragma once

#include "mfx_device.cuh"
#include "mfx_host.h"

namespace mfx {
namespace rmsnorm {

// A team of `lanes` threads (8, 16 or 32 lanes of a warp, or a whole block)
// owns a row and keeps it in registers, 8 C elements a thread.  With vectors,
// a thread's k-th run of 8 columns begins at 8 (k lanes + lane); without
// (a width that is not a multiple of 8, or a buffer off a vector) its e-th
// element is column e lanes + lane, so that a warp's accesses still cover
// whole lines.
template <typename T, int C, bool VEC>
__device__ __forceinline__ void load_row(const T* p, int cols, int lanes, int tl, float (&f)[8 * C])
{
    if constexpr (VEC) {
        Raw8<T> r[C];
#pragma unroll
        for (int k = 0; k < C; ++k)
            if (const int c = (k * lanes + tl) * 8; c < cols)
                ld8(p + c, r[k]);
#pragma unroll
        for (int k = 0; k < C; ++k) {
            if ((k * lanes + tl) * 8 < cols) {
                widen8(r[k], f + 8 * k);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    f[8 * k + j] = 0.0f;
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8 * C; ++e) {
            const int c = e * lanes + tl;
            f[e] = c < cols ? load1(p + c) : 0.0f;
        }
    }
}

template <typename T, int C, bool VEC>
__device__ __forceinline__ void store_row(T* p, int cols, int lanes, int tl, const float (&f)[8 * C])
{
    if constexpr (VEC) {
#pragma unroll
        for (int k = 0; k < C; ++k)
            if (const int c = (k * lanes + tl) * 8; c < cols) {
                Raw8<T> r;
                narrow8(f + 8 * k, r);
                st8(p + c, r);
            }
    } else {
#pragma unroll
        for (int e = 0; e < 8 * C; ++e)
            if (const int c = e * lanes + tl; c < cols)
                store1(p + c, f[e]);
    }
}

// The factors weight + offset of a thread's k-th eight columns (1 without a
// weight; 0 past the row's end).  The weight's type is asked at run time: its
// rows come from L1.
template <bool VEC>
__device__ __forceinline__ void factors(const void* weight, bool w_bf16, float offset, int cols, int lanes, int tl,
                                        int k, float w[8])
{
    if constexpr (VEC) {
        const int c = (k * lanes + tl) * 8;
        if (c >= cols || !weight) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j] = c < cols ? 1.0f : 0.0f;
            return;
        }
        if (w_bf16)
            bias8(static_cast<const bf16*>(weight), c, w);
        else
            bias8(static_cast<const float*>(weight), c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] += offset;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = (8 * k + j) * lanes + tl;
            w[j] = c >= cols  ? 0.0f
                   : !weight  ? 1.0f
                   : w_bf16   ? load1(static_cast<const bf16*>(weight) + c) + offset
                              : load1(static_cast<const float*>(weight) + c) + offset;
        }
    }
}

// The largest absolute value of two; NaN counts as nothing.
__device__ __forceinline__ float amax(float a, float b) { return fmaxf(a, fabsf(b)); }

// (sum, maximum) over a team, the same bits in every thread of it.  Teams of
// several warps are a whole block; `slot` alternates between calls, so that
// one barrier each is enough.
template <bool MAX>
__device__ __forceinline__ float2 over_team(float2 v, int lanes, float2 (*part)[32], int slot)
{
    const int n = lanes < 32 ? lanes : 32;
    for (int o = n >> 1; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
        if (MAX)
            v.y = fmaxf(v.y, __shfl_xor_sync(0xFFFFFFFFu, v.y, o));
    }
    if (lanes > 32) {
        const int lane = threadIdx.x & 31, warps = lanes >> 5;
        if (lane == 0)
            part[slot][threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < warps ? part[slot][lane] : make_float2(0.0f, 0.0f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
            if (MAX)
                v.y = fmaxf(v.y, __shfl_xor_sync(0xFFFFFFFFu, v.y, o));
        }
    }
    return v;
}

// How a row is laid out: C runs of 8 elements a thread, lanes a row, threads
// a block (the same for teams of several warps).
struct Layout {
    int C, lanes, threads;
    bool longer;  // the row does not fit a block's registers
};

// What the checks of both directions share.
inline bool sizes_ok(int64_t rows, int64_t cols)
{
    int64_t n;
    return rows >= 0 && cols >= 0 && cols <= (1 << 30) && mul_ok(rows, cols, &n) && n <= INT64_MAX / 8;
}

}  // namespace rmsnorm
}  // namespace mfx
