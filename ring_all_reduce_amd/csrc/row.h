// row.h -- device helpers of the kernels that take whole rows: eight elements as
// they are stored, and sums and maxima over the lanes of a row.
#pragma once

#include "act.h"

namespace rar {

// Eight consecutive elements as stored, of which the first cnt exist; the others
// read as `fill`.  A row's end is read one by one, in short code: few lanes have one.
template <class T> struct Eight;

__device__ __forceinline__ int clamp8(int64_t left) { return left >= 8 ? 8 : (left < 0 ? 0 : (int)left); }

template <> struct Eight<float> {
    f32x4 lo, hi;
    // What is computed of these values before and after is not shared: kept
    // results would take more registers than the values.
    __device__ __forceinline__ void forget() { asm volatile("" : "+v"(lo), "+v"(hi)); }
    // Moved down by s places, 1 .. 8; zeros follow.
    __device__ __forceinline__ void shift(int s)
    {
        const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
        if (s & 12) {
            lo = s & 8 ? zero : hi;
            hi = zero;
        }
        if (s & 2) {
            lo = f32x4{lo.z, lo.w, hi.x, hi.y};
            hi = f32x4{hi.z, hi.w, 0.0f, 0.0f};
        }
        if (s & 1) {
            lo = f32x4{lo.y, lo.z, lo.w, hi.x};
            hi = f32x4{hi.y, hi.z, hi.w, 0.0f};
        }
    }
    __device__ __forceinline__ float get(int i) const { return i < 4 ? lo[i & 3] : hi[i & 3]; }
    __device__ __forceinline__ void set(float v)
    {
        lo = f32x4{v, v, v, v};
        hi = lo;
    }
    __device__ __forceinline__ void load(const float *p, int cnt, float fill = 0.0f)
    {
        if (cnt == 8) {
            const f32x4_any *const q = reinterpret_cast<const f32x4_any *>(p);
            lo = q[0];
            hi = q[1];
            return;
        }
        set(fill);
#pragma unroll 1
        for (int i = 0; i < cnt; ++i) {
            const float v = p[i];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                lo[k] = i == k ? v : lo[k];
                hi[k] = i == k + 4 ? v : hi[k];
            }
        }
    }
};

// Where a lane's eight of a row of `cols` is read: whole eights at their place, the
// end of a row by the row's last eight elements, shifted into place by settle() once
// they have arrived, and nothing by any eight of the row.  So every lane reads in
// one load, and none waits for a branch.  (A row of less than eight is read one by one.)
struct Slot {
    int64_t c, from;
    int cnt;      // of the eight, how many exist
    bool tiny;
    __device__ __forceinline__ Slot(int64_t column, int64_t cols)
        : c(column), cnt(clamp8(cols - column)), tiny(cols < 8)
    {
        from = tiny || cnt == 0 ? 0 : (cnt == 8 ? column : cols - 8);
    }
};

template <> struct Eight<bf16> {
    u32x4 w;
    __device__ __forceinline__ void forget() { asm volatile("" : "+v"(w)); }
    __device__ __forceinline__ void shift(int s)
    {
        if (s & 8)
            w = u32x4{0, 0, 0, 0};
        if (s & 4)
            w = u32x4{w.z, w.w, 0, 0};
        if (s & 2)
            w = u32x4{w.y, w.z, w.w, 0};
        if (s & 1)
            w = u32x4{w.x >> 16 | w.y << 16, w.y >> 16 | w.z << 16, w.z >> 16 | w.w << 16, w.w >> 16};
    }
    __device__ __forceinline__ float get(int i) const
    {
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    __device__ __forceinline__ void set(float v)  // v: a bf16 value
    {
        const uint32_t u = __float_as_uint(v) >> 16;
        w = u32x4{u, u, u, u} * 0x10001u;
    }
    __device__ __forceinline__ void load(const bf16 *p, int cnt, float fill = 0.0f)
    {
        if (cnt == 8) {
            w = *reinterpret_cast<const u32x4_any *>(p);
            return;
        }
        set(fill);
#pragma unroll 1
        for (int i = 0; i < cnt; ++i) {
            const uint32_t v = p[i].u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                w[k] = i == 2 * k ? (w[k] & 0xffff0000u) | v : w[k];
                w[k] = i == 2 * k + 1 ? (w[k] & 0xffffu) | v << 16 : w[k];
            }
        }
    }
};

template <class T>
__device__ __forceinline__ void fetch(Eight<T> &v, const void *row, const Slot &at)
{
    if (at.tiny)
        v.load((const T *)row, at.cnt);
    else
        v.load((const T *)row + at.from, 8);
}

// To be called before the values are used; what does not exist is zero.
template <class T>
__device__ __forceinline__ void settle(Eight<T> &v, const Slot &at)
{
    v.forget();  // arrived, and not before: others may write the row from here on
    if (at.cnt < 8 && !at.tiny)
        v.shift(8 - at.cnt);
}

// A vector of a row's columns, or a constant in its place.
template <class T>
__device__ __forceinline__ void fetch_or(Eight<T> &v, const void *p, const Slot &at, float other)
{
    if (p)
        fetch(v, p, at);
    else
        v.set(other);
}

template <class T>
__device__ __forceinline__ void settle_or(Eight<T> &v, const void *p, const Slot &at)
{
    if (p)
        settle(v, at);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float v, float other)
{
    return __uint_as_float(__builtin_amdgcn_update_dpp((int)__float_as_uint(other), (int)__float_as_uint(v), CTRL,
                                                       ROWS, 0xf, false));
}

// Over the 64 lanes of a wave, in a fixed order: rows of 16 by shifts, then the
// rows' ends one after another; the last lane's result goes to all.
__device__ __forceinline__ float wave_sum(float v)
{
    v += dpp<0x111, 0xf>(v, 0.0f);
    v += dpp<0x112, 0xf>(v, 0.0f);
    v += dpp<0x114, 0xf>(v, 0.0f);
    v += dpp<0x118, 0xf>(v, 0.0f);
    v += dpp<0x142, 0xa>(v, 0.0f);
    v += dpp<0x143, 0xc>(v, 0.0f);
    return __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

__device__ __forceinline__ float wave_max(float v)
{
    constexpr float kLow = -__builtin_inff();
    v = __builtin_fmaxf(v, dpp<0x111, 0xf>(v, kLow));
    v = __builtin_fmaxf(v, dpp<0x112, 0xf>(v, kLow));
    v = __builtin_fmaxf(v, dpp<0x114, 0xf>(v, kLow));
    v = __builtin_fmaxf(v, dpp<0x118, 0xf>(v, kLow));
    v = __builtin_fmaxf(v, dpp<0x142, 0xa>(v, kLow));
    v = __builtin_fmaxf(v, dpp<0x143, 0xc>(v, kLow));
    return __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// N sums (or maxima) over the LANES lanes of a row.  Rows of more than a wave
// meet in LDS: one half of `lds` is written while the last reader of the other
// may still be reading, and every lane of the workgroup takes part.
template <int LANES, int N>
struct RowJoin {
    static constexpr int kThreads = LANES > 256 ? LANES : 256;
    static constexpr int kWaves = kThreads / 64;
    float *lds;      // [2][kWaves][N]
    int half = 0;

    static constexpr int kFloats = LANES > 64 ? 2 * kWaves * N : 1;

    template <int M, bool MAX>
    __device__ __forceinline__ void join(float (&v)[M])
    {
        static_assert(M <= N, "room for N values a wave");
#pragma unroll
        for (int i = 0; i < M; ++i)
            v[i] = MAX ? wave_max(v[i]) : wave_sum(v[i]);
        if (LANES == 64)
            return;
        float *const at = lds + half * (kWaves * N);
        half ^= 1;
        const int wave = threadIdx.x >> 6, first = wave / (LANES / 64) * (LANES / 64);
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < M; ++i)
                at[wave * N + i] = v[i];
        __syncthreads();
        constexpr int kEach = LANES / 64;
        if (kEach * M > 32) {
            // a wave's value a lane, joined by shifts: read by every lane they would take more registers than the rows
            const float none = MAX ? -__builtin_inff() : 0.0f;
#pragma unroll
            for (int i = 0; i < M; ++i) {
                float t = at[(threadIdx.x & (kEach - 1)) * N + i], o;
                o = dpp<0x111, 0xf>(t, none);
                t = MAX ? __builtin_fmaxf(t, o) : t + o;
                o = dpp<0x112, 0xf>(t, none);
                t = MAX ? __builtin_fmaxf(t, o) : t + o;
                o = dpp<0x114, 0xf>(t, none);
                t = MAX ? __builtin_fmaxf(t, o) : t + o;
                if (kEach == 16) {
                    o = dpp<0x118, 0xf>(t, none);
                    t = MAX ? __builtin_fmaxf(t, o) : t + o;
                }
                v[i] = __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(t), kEach - 1));
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < M; ++i) {
            float t = at[first * N + i];
#pragma unroll
            for (int w = 1; w < kEach; ++w) {
                const float o = at[(first + w) * N + i];
                t = MAX ? __builtin_fmaxf(t, o) : t + o;
            }
            v[i] = t;
        }
    }
    template <int M> __device__ __forceinline__ void sum(float (&v)[M]) { join<M, false>(v); }
    template <int M> __device__ __forceinline__ void max(float (&v)[M]) { join<M, true>(v); }
};

}  // namespace rar
