// row.h -- device helpers of the kernels that take whole rows: eight elements as
// they are stored, and sums and maxima over the lanes of a row.
#pragma once

#include "act.h"

namespace rar {

// Eight consecutive elements as stored, of which the first cnt exist; the others
// read as `fill`.
template <class T> struct Eight;

template <> struct Eight<float> {
    f32x4 lo, hi;
    // What is computed of these values before and after is not shared: kept
    // results would take more registers than the values.
    __device__ __forceinline__ void forget() { asm volatile("" : "+v"(lo), "+v"(hi)); }
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
        for (int i = 0; i < cnt; ++i) {  // a row's end: few lanes, so short code
            const float v = p[i];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                lo[k] = i == k ? v : lo[k];
                hi[k] = i == k + 4 ? v : hi[k];
            }
        }
    }
};

template <> struct Eight<bf16> {
    u32x4 w;
    __device__ __forceinline__ void forget() { asm volatile("" : "+v"(w)); }
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

// A vector of a row's columns, or a constant in its place.
template <class T>
__device__ __forceinline__ void load_or(Eight<T> &v, const void *p, int64_t c, int cnt, float other)
{
    if (p)
        v.load((const T *)p + c, cnt);
    else
        v.set(other);
}

__device__ __forceinline__ int clamp8(int64_t left) { return left >= 8 ? 8 : (left < 0 ? 0 : (int)left); }

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
#pragma unroll
        for (int i = 0; i < M; ++i) {
            float t = at[first * N + i];
#pragma unroll
            for (int w = 1; w < LANES / 64; ++w) {
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
