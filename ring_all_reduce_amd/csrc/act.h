// act.h -- device helpers shared by the operators' kernels: element access,
// the activations and their derivatives.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rar.h"

namespace rar {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Storage types: float, and bf16 as its bit pattern.
struct bf16 {
    uint16_t u;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16 v) { return __uint_as_float((uint32_t)v.u << 16); }

// One rounding, to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ bf16 from_f32<bf16>(float v) { return bf16{(uint16_t)pack_bf16(v, 0.0f)}; }

__device__ __forceinline__ f32x4 load4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }
__device__ __forceinline__ f32x4 load4(const bf16 *p)
{
    const u32x2 w = *reinterpret_cast<const u32x2 *>(p);
    return f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                 __uint_as_float(w.y & 0xffff0000u)};
}
__device__ __forceinline__ void store4(float *p, f32x4 v) { *reinterpret_cast<f32x4 *>(p) = v; }
__device__ __forceinline__ void store4(bf16 *p, f32x4 v)
{
    *reinterpret_cast<u32x2 *>(p) = u32x2{pack_bf16(v.x, v.y), pack_bf16(v.z, v.w)};
}

// Data that a call reads once: kept from displacing other lines.
template <class V>
__device__ __forceinline__ V load_once(const V *p)
{
    return __builtin_nontemporal_load(p);
}

template <class V>
__device__ __forceinline__ void store_once(V *p, V v)
{
    __builtin_nontemporal_store(v, p);
}

// Eight consecutive elements, of which the first cnt exist.  Whole groups move in
// 16-byte accesses at whatever address the element type allows (global memory
// takes them unaligned).
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <bool ONCE = false>
__device__ __forceinline__ void load8(const float *p, int cnt, float (&v)[8])
{
    if (cnt == 8) {
        const f32x4_any *const w = reinterpret_cast<const f32x4_any *>(p);
        const f32x4 a = ONCE ? __builtin_nontemporal_load(w) : w[0];
        const f32x4 b = ONCE ? __builtin_nontemporal_load(w + 1) : w[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = i < cnt ? to_f32(p[i]) : 0.0f;
}

template <bool ONCE = false>
__device__ __forceinline__ void store8(float *p, int cnt, const float (&v)[8])
{
    if (cnt == 8) {
        f32x4_any *const w = reinterpret_cast<f32x4_any *>(p);
        const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
        if (ONCE) {
            __builtin_nontemporal_store(a, w);
            __builtin_nontemporal_store(b, w + 1);
        } else {
            w[0] = a;
            w[1] = b;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < cnt)
            p[i] = v[i];
}

template <bool ONCE = false>
__device__ __forceinline__ void load8(const bf16 *p, int cnt, float (&v)[8])
{
    if (cnt == 8) {
        const u32x4_any *const q = reinterpret_cast<const u32x4_any *>(p);
        const u32x4 w = ONCE ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = i < cnt ? to_f32(p[i]) : 0.0f;
}

template <bool ONCE = false>
__device__ __forceinline__ void store8(bf16 *p, int cnt, const float (&v)[8])
{
    if (cnt == 8) {
        const u32x4 w = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
        u32x4_any *const q = reinterpret_cast<u32x4_any *>(p);
        if (ONCE)
            __builtin_nontemporal_store(w, q);
        else
            *q = w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < cnt)
            p[i] = from_f32<bf16>(v[i]);
}

// Upper tail of the normal distribution: with a = |z|,
//   1 - Phi(a) = exp(-a^2 / 2) * q(a / sqrt 2) / 2,  q(x) = exp(x^2) erfc(x).
// q is smooth and falls like 1/x, so q/2 is a polynomial in t = 1 / (1 + c x)
// without a constant term.  The coefficients are least-maximum fits made for
// this file.  Relative error of q for 0 <= x <= 10, as the constants below are
// rounded (beyond that exp(-x^2) < 2^-144): degree 8 for binary32, 1.02e-7;
// degree 6 for bf16, 5.2e-6, a seven-hundredth of its half step.  The
// exponential's argument is rounded twice, which adds z^2 * 2^-24 to the
// relative error of the tail: 4e-6 at |z| = 8, where 1 + erf(z / sqrt 2) has no
// digit left in binary32.  About 17 instructions, two of them transcendental,
// against about 60 for erfcf: the epilogue of a matrix product evaluates it with
// the matrix cores idle.
template <class T>
__device__ __forceinline__ void normal_tail(float z, float &q, float &e)
{
    constexpr bool kWide = sizeof(T) == 4;
    constexpr float kC = (kWide ? 0.33f : 0.44f) * 0.70710678118654752f;
    e = __builtin_amdgcn_exp2f(z * (z * -0.72134752044448170f));
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_fabsf(z), kC, 1.0f));
    if (kWide) {
        q = 0.5f * -0.1353447437286377f;
        q = __builtin_fmaf(q, t, 0.5f * 0.4602333605289459f);
        q = __builtin_fmaf(q, t, 0.5f * -0.3511435091495514f);
        q = __builtin_fmaf(q, t, 0.5f * 0.4084944725036621f);
        q = __builtin_fmaf(q, t, 0.5f * 0.04722348973155022f);
        q = __builtin_fmaf(q, t, 0.5f * 0.20122304558753967f);
        q = __builtin_fmaf(q, t, 0.5f * 0.18295608460903168f);
        q = __builtin_fmaf(q, t, 0.5f * 0.1863577961921692f);
    } else {
        q = 0.5f * -0.14610587060451508f;
        q = __builtin_fmaf(q, t, 0.5f * 0.3506527841091156f);
        q = __builtin_fmaf(q, t, 0.5f * 0.04073116183280945f);
        q = __builtin_fmaf(q, t, 0.5f * 0.2635860741138458f);
        q = __builtin_fmaf(q, t, 0.5f * 0.2425696849822998f);
        q = __builtin_fmaf(q, t, 0.5f * 0.24856099486351013f);
    }
    q *= t;  // 1 - Phi(|z|) = e q
}

// |z|, bounded where the density is zero anyway, so that infinity times zero
// does not arise.  (The minimum with a NaN is the bound; z reaches the result
// as a NaN through e.)
__device__ __forceinline__ float bounded(float z) { return __builtin_fminf(__builtin_fabsf(z), 40.0f); }

// z Phi(z) = max(z, 0) - |z| (1 - Phi(|z|)); the limits at +-infinity, NaN at NaN.
template <class T>
__device__ __forceinline__ float gelu(float z)
{
    float q, e;
    normal_tail<T>(z, q, e);
    return __builtin_fmaf(-bounded(z), e * q, __builtin_fmaxf(z, 0.0f));
}

// Phi(z) + z phi(z): with h = (1 - Phi(|z|)) - |z| phi(z), h for z < 0 and
// 1 - h else.
template <class T>
__device__ __forceinline__ float gelu_grad(float z)
{
    float q, e;
    normal_tail<T>(z, q, e);
    const float h = e * __builtin_fmaf(-0.39894228040143268f, bounded(z), q);
    return z < 0.0f ? h : 1.0f - h;
}

template <class T>
__device__ __forceinline__ float act_value(int act, float z)
{
    if (act == RAR_ACT_RELU)
        return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    if (act == RAR_ACT_GELU)
        return gelu<T>(z);
    return z;
}

// act'(z); relu'(0) = 0, NaN at NaN.
template <class T>
__device__ __forceinline__ float act_grad(int act, float z)
{
    if (act == RAR_ACT_RELU)
        return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    if (act == RAR_ACT_GELU)
        return gelu_grad<T>(z);
    return 1.0f;
}

// ---- 8-bit checkpoints (see ckpt.hip) ---------------------------------------

// Largest magnitude pattern among finite values: as integers, magnitudes order
// like the values.
__device__ __forceinline__ uint32_t ckpt_top(uint32_t top, float v)
{
    const uint32_t m = __float_as_uint(v) & 0x7fffffffu;
    return m > top && m < 0x7f800000u ? m : top;
}

// Biased exponent of the scale of a group whose largest magnitude is `top`:
// 448 = 1.75 * 2^8.
__device__ __forceinline__ int ckpt_exponent(uint32_t top)
{
    const int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < 1 ? 1 : e;
}

// Four codes; the multiplication by a power of two is exact, or its result so
// small that its code is zero either way.
__device__ __forceinline__ uint32_t ckpt_codes4(f32x4 v, int e)
{
    const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(v.x * inv, v.y * inv, 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(v.z * inv, v.w * inv, r, true);
    uint32_t w = (uint32_t)r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if ((__float_as_uint(v[i]) & 0x7f800000u) == 0x7f800000u)
            w |= 0x7fu << (8 * i);
    return w;
}

// The four values of codes w with scale byte e.
__device__ __forceinline__ f32x4 ckpt_values4(uint32_t w, uint32_t e)
{
    const float s = __uint_as_float(e << 23);
    const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, false);
    const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, true);
    return f32x4{lo.x, lo.y, hi.x, hi.y};
}

}  // namespace rar
