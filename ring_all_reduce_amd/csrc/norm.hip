// norm.hip -- CDNA4 (gfx950) kernels of the norms before and after a block, with
// its gate and the residual stream.
//
//   n = post(o),  h = a x + s (gate . n),  u = pre(h)
//   g = dh + pre'(du; h),  dx = a g,  do = post'(s gate . g; o)
//
// With v^ = (v - mean) r, r = 1 / sqrt(var + eps) (mean zero for rms) and y = w v^ +
// b, the gradient of v is r (q - mean(q) - v^ mean(q v^)), q = w dy; without
// mean(q) for rms.  The backward kernel makes mean and r again from the rows o
// and h that it reads in any case, so nothing but them is kept.
//
// A row passes once through the registers of its lanes, eight columns a lane; a
// workgroup keeps the vectors and takes rows in turn, the next row's loads under
// this row's sums.  The variance is taken of the centred row, so that a mean far from
// zero costs no more than the mean's own rounding.  65536 x 2048, norms on both
// sides: forward 220 us in bf16 and 415 in binary32 (1.07 and 2.15 GB, 4.9 and 5.2
// TB/s), bound by HBM at the rate of torch's copy of 2 GB, 4.9; backward 330 and 650
// (1.61 and 3.22 GB, 4.9 TB/s) and 12 for the column sums.  Two reads a write can go
// at 5.9 TB/s (dropout does): the backward kernel's vector units are 76% busy, and
// what they do not hide of the rest is some 20%.  8 x 2048 in binary32: 4 us, a launch.
#include <algorithm>

#include "ops_internal.h"
#include "row.h"

#pragma clang fp contract(off)

namespace rar {
namespace {

constexpr int kSums = 4;  // column sums: g o^, g, du h^, du

template <class T, int LANES>
__global__ void __launch_bounds__(LANES > 256 ? LANES : 256) rar_norm_rows(const NormParams p)
{
    typedef RowJoin<LANES, 1> Join;
    constexpr int kRows = Join::kThreads / LANES;
    __shared__ float lds[Join::kFloats];
    Join join{lds};
    const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    const float inv = 1.0f / (float)p.cols;
    const Slot at((int64_t)lane * 8, p.cols);
    const int64_t c = at.c;
    const int cols = at.cnt;
    // (the vectors that a call does not use are null)
    Eight<T> gate, w1, b1, w2, b2, xr, orow;
    auto ahead = [&](int64_t row) __attribute__((always_inline)) {
        row = row < p.rows ? row : p.rows - 1;
        fetch(xr, (const T *)p.x + row * p.ldx, at);
        if (p.o)
            fetch(orow, (const T *)p.o + row * p.ldo, at);
    };
    // v becomes the normalised row; elements behind the row stay zero
    auto normalise = [&](float (&v)[8], int kind) __attribute__((always_inline)) {
        if (kind == RAR_NORM_LAYER) {
            float t[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                t[0] += v[i];
            join.sum(t);
            const float mean = t[0] * inv;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = i < cols ? v[i] - mean : 0.0f;
        }
        float t[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t[0] = __builtin_fmaf(v[i], v[i], t[0]);
        join.sum(t);
        const float r = 1.0f / __builtin_sqrtf(t[0] * inv + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] *= r;
    };

    const int64_t stride = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + sub;
    ahead(row);
    fetch_or(gate, p.gate, at, 1.0f);
    fetch_or(w1, p.post_w, at, 1.0f);
    fetch_or(b1, p.post_b, at, 0.0f);
    fetch_or(w2, p.pre_w, at, 1.0f);
    fetch_or(b2, p.pre_b, at, 0.0f);
    settle_or(gate, p.gate, at);
    settle_or(w1, p.post_w, at);
    settle_or(b1, p.post_b, at);
    settle_or(w2, p.pre_w, at);
    settle_or(b2, p.pre_b, at);
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < p.rows; first += stride, row += stride) {
        settle(xr, at);
        if (p.o)
            settle(orow, at);
        float h[8], n[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[i] = p.a * xr.get(i);
            n[i] = p.o ? orow.get(i) : 0.0f;
        }
        // h over x: the lane at a row's end has read what a lane of another wave may write from here on
        if (LANES > 64 && p.h == p.x)
            __syncthreads();
        ahead(row + stride);
        if (p.o) {
            if (p.post)
                normalise(n, p.post);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = __builtin_fmaf(n[i], w1.get(i), b1.get(i));
                h[i] = i < cols ? __builtin_fmaf(p.s, gate.get(i) * y, h[i]) : 0.0f;
            }
        }
        const bool live = row < p.rows;
        if (p.h && live)
            store8((T *)p.h + row * p.ldh + c, cols, h);
        if (!p.u)
            continue;
        if (p.pre) {
            normalise(h, p.pre);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[i] = __builtin_fmaf(h[i], w2.get(i), b2.get(i));
        }
        if (live)
            store8((T *)p.u + row * p.ldu + c, cols, h);
    }
}

template <class T, int LANES>
__global__ void __launch_bounds__(LANES > 256 ? LANES : 256, LANES >= 512 ? 4 : 1)
    rar_norm_grad_rows(const NormGradParams p)
{
    typedef RowJoin<LANES, 4> Join;
    constexpr int kRows = Join::kThreads / LANES;
    __shared__ float lds[Join::kFloats];
    Join join{lds};
    const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    const float inv = 1.0f / (float)p.cols;
    const Slot at((int64_t)lane * 8, p.cols);
    const int64_t c = at.c;
    const int cols = at.cnt;
    Eight<T> gate, w1, w2;
    // Long rows keep their column sums in LDS (a lane's own, so nothing waits): without them 128 registers hold the
    // rest and the next row, and a compute unit holds 1024 lanes.  16384 x 8192 in bf16 360 us (1.6 GB), 1200 with the
    // sums in registers; 16384 x 4096 176 and 214.  (In binary32 14 registers are spilled at 512 lanes, 2 at 1024.)
    constexpr bool kInLds = LANES >= 512;
    __shared__ f32x4 kept[kInLds ? kSums * 2 : 1][kInLds ? LANES : 1];
    float sums[kSums][8] = {};
    auto put_sums = [&](int q) __attribute__((always_inline)) {
        if (kInLds)
#pragma unroll
            for (int j = 0; j < kSums; ++j)
                kept[j * 2 + q][lane] =
                    f32x4{sums[j][q * 4], sums[j][q * 4 + 1], sums[j][q * 4 + 2], sums[j][q * 4 + 3]};
    };
    auto get_sums = [&](int q) __attribute__((always_inline)) {
        if (kInLds)
#pragma unroll
            for (int j = 0; j < kSums; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sums[j][q * 4 + i] = kept[j * 2 + q][lane][i];
    };
    put_sums(0);
    put_sums(1);
    Eight<T> rdh, rdu, ro, rh;
    rdh.set(0.0f);
    rdu.set(0.0f);
    ro.set(0.0f);
    rh.set(0.0f);
    const bool use_h = p.pre && p.du;
    // (a row in two parts: its gradients are needed later than what its statistics are made of)
    auto ahead = [&](int64_t row) __attribute__((always_inline)) {
        row = row < p.rows ? row : p.rows - 1;
        if (p.o)
            fetch(ro, (const T *)p.o + row * p.ldo, at);
        if (use_h)
            fetch(rh, (const T *)p.h + row * p.ldh, at);
    };
    auto ahead_gradients = [&](int64_t row) __attribute__((always_inline)) {
        row = row < p.rows ? row : p.rows - 1;
        if (p.du)
            fetch(rdu, (const T *)p.du + row * p.lddu, at);
        if (p.dh)
            fetch(rdh, (const T *)p.dh + row * p.lddh, at);
    };
    const int64_t stride = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + sub;
    ahead(row);
    ahead_gradients(row);
    fetch_or(gate, p.gate, at, 1.0f);
    fetch_or(w1, p.post_w, at, 1.0f);
    fetch_or(w2, p.pre_w, at, 1.0f);
    settle_or(gate, p.gate, at);
    settle_or(w1, p.post_w, at);
    settle_or(w2, p.pre_w, at);
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < p.rows; first += stride, row += stride) {
        const bool live = row < p.rows;
        settle(ro, at);
        settle(rh, at);
        if (!live) {
            ro.set(0.0f);
            rh.set(0.0f);
        }
        float o[8], h[8], g[8], du[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            o[i] = ro.get(i);
            h[i] = rh.get(i);
        }
        ahead(row + stride);
        if (p.post == RAR_NORM_LAYER || p.pre == RAR_NORM_LAYER) {
            float t[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                t[0] += o[i];
                t[1] += h[i];
            }
            join.sum(t);
            const float mo = p.post == RAR_NORM_LAYER ? t[0] * inv : 0.0f;
            const float mh = p.pre == RAR_NORM_LAYER ? t[1] * inv : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i] = i < cols ? o[i] - mo : 0.0f;
                h[i] = i < cols ? h[i] - mh : 0.0f;
            }
        }
        // (arrived before the meeting below, behind which dx may be written over dh)
        settle(rdu, at);
        settle(rdh, at);
        if (!live) {
            rdu.set(0.0f);
            rdh.set(0.0f);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            du[i] = rdu.get(i);
            g[i] = rdh.get(i);
        }
        ahead_gradients(row + stride);
        float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = du[i] * w2.get(i);
            t[0] = __builtin_fmaf(o[i], o[i], t[0]);
            t[1] = __builtin_fmaf(h[i], h[i], t[1]);
            t[2] += q;
            t[3] = __builtin_fmaf(q, h[i], t[3]);
        }
        join.sum(t);
        const float rpost = p.post ? 1.0f / __builtin_sqrtf(t[0] * inv + p.eps) : 1.0f;
        const float rpre = p.pre ? 1.0f / __builtin_sqrtf(t[1] * inv + p.eps) : 1.0f;
        const float m1 = p.pre == RAR_NORM_LAYER ? t[2] * inv : 0.0f;
        const float m2 = p.pre ? t[3] * rpre * inv : 0.0f;
        float e[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i % 4 == 0)
                get_sums(i / 4);
            const float hh = h[i] * rpre, oh = o[i] * rpost;
            sums[2][i] = __builtin_fmaf(du[i], hh, sums[2][i]);
            sums[3][i] += du[i];
            const float back = __builtin_fmaf(-hh, m2, __builtin_fmaf(du[i], w2.get(i), -m1));
            // (behind the row both terms would be -m1)
            const float gv = i < cols ? __builtin_fmaf(rpre, back, g[i]) : 0.0f;
            sums[0][i] = __builtin_fmaf(gv, oh, sums[0][i]);
            sums[1][i] += gv;
            const float q = p.s * gate.get(i) * gv * w1.get(i);
            e[0] += q;
            e[1] = __builtin_fmaf(q, oh, e[1]);
            g[i] = gv;
            o[i] = oh;
            if (i % 4 == 3)
                put_sums(i / 4);
        }
        if (p.dx && live) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = p.a * g[i];
            store8((T *)p.dx + row * p.lddx + c, cols, v);
        }
        if (!p.d_o)
            continue;
        if (p.post)
            join.sum(e);
        const float n1 = p.post == RAR_NORM_LAYER ? e[0] * inv : 0.0f, n2 = p.post ? e[1] * inv : 0.0f;
        if (live) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q = p.s * gate.get(i) * g[i] * w1.get(i);
                v[i] = rpost * __builtin_fmaf(-o[i], n2, q - n1);
            }
            store8((T *)p.d_o + row * p.lddo + c, cols, v);
        }
    }
    get_sums(0);
    get_sums(1);
    // the rows that stood beside each other are one chunk: the first of them adds up
    if (kRows > 1) {
        __shared__ f32x4 beside[kRows > 1 ? kRows - 1 : 1][kSums * 2][LANES];
        if (sub > 0)
#pragma unroll
            for (int j = 0; j < kSums * 2; ++j)
                beside[sub - 1][j][lane] = *reinterpret_cast<const f32x4 *>(&sums[j / 2][j % 2 * 4]);
        __syncthreads();
        if (sub > 0)
            return;
#pragma unroll
        for (int n = 0; n < kRows - 1; ++n)
#pragma unroll
            for (int j = 0; j < kSums * 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sums[j / 2][j % 2 * 4 + i] += beside[n][j][lane][i];
    }
    float *const out = p.part + (int64_t)blockIdx.x * kSums * p.pitch;
#pragma unroll
    for (int j = 0; j < kSums; ++j)
        if (cols > 0 && (j < 2 ? p.sum_post : p.sum_pre))
            store8(out + j * p.pitch + c, 8, sums[j]);
}

// ---------------------------------------------------------------------------
// Rows that do not fit the registers
// ---------------------------------------------------------------------------
//
// The same arithmetic, reading the row again (from the caches) for each sum.  A
// row's column sums are added to the chunk's in memory, by the lane that owns
// the columns.

constexpr int kWideLanes = 1024;

struct Affine {
    float mean, r;
};

template <class T>
__device__ __forceinline__ Affine wide_stats(RowJoin<kWideLanes, 4> &join, int kind, float eps, int64_t cols,
                                             const T *row)
{
    if (kind == RAR_NORM_NONE)
        return Affine{0.0f, 1.0f};
    const float inv = 1.0f / (float)cols;
    float v[8], mean = 0.0f;
    if (kind == RAR_NORM_LAYER) {
        float t[1] = {0.0f};
        for (int64_t c = threadIdx.x * 8; c < cols; c += kWideLanes * 8) {
            load8(row + c, clamp8(cols - c), v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                t[0] += v[i];
        }
        join.sum(t);
        mean = t[0] * inv;
    }
    float t[1] = {0.0f};
    for (int64_t c = threadIdx.x * 8; c < cols; c += kWideLanes * 8) {
        const int cnt = clamp8(cols - c);
        load8(row + c, cnt, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = i < cnt ? v[i] - mean : 0.0f;
            t[0] = __builtin_fmaf(d, d, t[0]);
        }
    }
    join.sum(t);
    return Affine{mean, 1.0f / __builtin_sqrtf(t[0] * inv + eps)};
}

template <class T>
__device__ __forceinline__ void wide_or(const void *p, int64_t c, int cnt, float other, float (&v)[8])
{
    if (p) {
        load8((const T *)p + c, cnt, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = other;
}

template <class T>
__global__ void __launch_bounds__(kWideLanes) rar_norm_wide(const NormParams p)
{
    typedef RowJoin<kWideLanes, 4> Join;
    __shared__ float lds[Join::kFloats];
    Join join{lds};
    const float inv = 1.0f / (float)p.cols;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T *const x = (const T *)p.x + row * p.ldx, *const o = (const T *)p.o + row * p.ldo;
        Affine so{0.0f, 1.0f};
        if (p.o)
            so = wide_stats<T>(join, p.post, p.eps, p.cols, o);
        auto stream = [&](int64_t c, int cnt, float (&h)[8]) __attribute__((always_inline)) {
            float v[8], w[8], b[8], g[8];
            load8(x + c, cnt, h);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[i] *= p.a;
            if (!p.o)
                return;
            load8(o + c, cnt, v);
            wide_or<T>(p.post ? p.post_w : nullptr, c, cnt, 1.0f, w);
            wide_or<T>(p.post ? p.post_b : nullptr, c, cnt, 0.0f, b);
            wide_or<T>(p.gate, c, cnt, 1.0f, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = __builtin_fmaf((v[i] - so.mean) * so.r, w[i], b[i]);
                h[i] = i < cnt ? __builtin_fmaf(p.s, g[i] * y, h[i]) : 0.0f;
            }
        };
        Affine sh{0.0f, 1.0f};
        if (p.u && p.pre) {
            float h[8];
            if (p.pre == RAR_NORM_LAYER) {
                float t[1] = {0.0f};
                for (int64_t c = threadIdx.x * 8; c < p.cols; c += kWideLanes * 8) {
                    stream(c, clamp8(p.cols - c), h);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        t[0] += h[i];
                }
                join.sum(t);
                sh.mean = t[0] * inv;
            }
            float t[1] = {0.0f};
            for (int64_t c = threadIdx.x * 8; c < p.cols; c += kWideLanes * 8) {
                const int cnt = clamp8(p.cols - c);
                stream(c, cnt, h);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float d = i < cnt ? h[i] - sh.mean : 0.0f;
                    t[0] = __builtin_fmaf(d, d, t[0]);
                }
            }
            join.sum(t);
            sh.r = 1.0f / __builtin_sqrtf(t[0] * inv + p.eps);
        }
        for (int64_t c = threadIdx.x * 8; c < p.cols; c += kWideLanes * 8) {
            const int cnt = clamp8(p.cols - c);
            float h[8], w[8], b[8];
            stream(c, cnt, h);
            if (p.h)
                store8((T *)p.h + row * p.ldh + c, cnt, h);
            if (!p.u)
                continue;
            wide_or<T>(p.pre ? p.pre_w : nullptr, c, cnt, 1.0f, w);
            wide_or<T>(p.pre ? p.pre_b : nullptr, c, cnt, 0.0f, b);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[i] = p.pre ? __builtin_fmaf((h[i] - sh.mean) * sh.r, w[i], b[i]) : h[i];
            store8((T *)p.u + row * p.ldu + c, cnt, h);
        }
    }
}

template <class T>
__global__ void __launch_bounds__(kWideLanes) rar_norm_grad_wide(const NormGradParams p)
{
    typedef RowJoin<kWideLanes, 4> Join;
    __shared__ float lds[Join::kFloats];
    Join join{lds};
    const float inv = 1.0f / (float)p.cols;
    float *const part = p.part + (int64_t)blockIdx.x * kSums * p.pitch;
    bool begun = false;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T *const o = (const T *)p.o + row * p.ldo, *const h = (const T *)p.h + row * p.ldh;
        const T *const dh = (const T *)p.dh + row * p.lddh, *const du = (const T *)p.du + row * p.lddu;
        const bool pre = p.pre && p.du;
        Affine so{0.0f, 1.0f}, sh{0.0f, 1.0f};
        if (p.o)
            so = wide_stats<T>(join, p.post, p.eps, p.cols, o);
        if (pre)
            sh = wide_stats<T>(join, p.pre, p.eps, p.cols, h);
        float m1 = 0.0f, m2 = 0.0f;
        auto du_h = [&](int64_t c, int cnt, float (&d)[8], float (&hh)[8],
                        float (&w)[8]) __attribute__((always_inline)) {
            wide_or<T>(p.du ? (const void *)du : nullptr, c, cnt, 0.0f, d);
            wide_or<T>(pre ? p.pre_w : nullptr, c, cnt, 1.0f, w);
            wide_or<T>(pre ? (const void *)h : nullptr, c, cnt, 0.0f, hh);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                hh[i] = pre && i < cnt ? (hh[i] - sh.mean) * sh.r : 0.0f;
        };
        if (pre) {
            float t[2] = {0.0f, 0.0f}, d[8], hh[8], w[8];
            for (int64_t c = threadIdx.x * 8; c < p.cols; c += kWideLanes * 8) {
                du_h(c, clamp8(p.cols - c), d, hh, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    t[0] += d[i] * w[i];
                    t[1] = __builtin_fmaf(d[i] * w[i], hh[i], t[1]);
                }
            }
            join.sum(t);
            m1 = p.pre == RAR_NORM_LAYER ? t[0] * inv : 0.0f;
            m2 = t[1] * inv;
        }
        // g, o^ and q of eight columns
        auto grads = [&](int64_t c, int cnt, float (&d)[8], float (&hh)[8], float (&g)[8], float (&oh)[8],
                         float (&q)[8]) __attribute__((always_inline)) {
            float w[8], gate[8], w1[8];
            du_h(c, cnt, d, hh, w);
            wide_or<T>(p.dh ? (const void *)dh : nullptr, c, cnt, 0.0f, g);
            wide_or<T>(p.o ? (const void *)o : nullptr, c, cnt, 0.0f, oh);
            wide_or<T>(p.o ? p.gate : nullptr, c, cnt, 1.0f, gate);
            wide_or<T>(p.post ? p.post_w : nullptr, c, cnt, 1.0f, w1);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float back = __builtin_fmaf(-hh[i], m2, __builtin_fmaf(d[i], w[i], -m1));
                g[i] = i < cnt ? __builtin_fmaf(sh.r, back, g[i]) : 0.0f;
                oh[i] = i < cnt ? (oh[i] - so.mean) * so.r : 0.0f;
                q[i] = p.s * gate[i] * g[i] * w1[i];
            }
        };
        float d[8], hh[8], g[8], oh[8], q[8], n1 = 0.0f, n2 = 0.0f;
        if (p.d_o && p.post) {
            float t[2] = {0.0f, 0.0f};
            for (int64_t c = threadIdx.x * 8; c < p.cols; c += kWideLanes * 8) {
                grads(c, clamp8(p.cols - c), d, hh, g, oh, q);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    t[0] += q[i];
                    t[1] = __builtin_fmaf(q[i], oh[i], t[1]);
                }
            }
            join.sum(t);
            n1 = p.post == RAR_NORM_LAYER ? t[0] * inv : 0.0f;
            n2 = t[1] * inv;
        }
        for (int64_t c = threadIdx.x * 8; c < p.cols; c += kWideLanes * 8) {
            const int cnt = clamp8(p.cols - c);
            grads(c, cnt, d, hh, g, oh, q);
#pragma unroll
            for (int j = 0; j < kSums; ++j) {
                if (!(j < 2 ? p.sum_post : p.sum_pre))
                    continue;
                float v[8] = {};
                float *const to = part + j * p.pitch + c;
                if (begun)
                    load8(to, 8, v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] += j == 0 ? g[i] * oh[i] : (j == 1 ? g[i] : (j == 2 ? d[i] * hh[i] : d[i]));
                store8(to, 8, v);
            }
            float v[8];
            if (p.dx) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = p.a * g[i];
                store8((T *)p.dx + row * p.lddx + c, cnt, v);
            }
            if (p.d_o) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = so.r * __builtin_fmaf(-oh[i], n2, q[i] - n1);
                store8((T *)p.d_o + row * p.lddo + c, cnt, v);
            }
        }
        begun = true;
    }
}

// ---------------------------------------------------------------------------
// Column sums
// ---------------------------------------------------------------------------
//
// A workgroup joins 16 columns of every chunk, of both sums of one norm: four lanes of four columns, 256
// of them beside each other, joined by lane exchanges and through LDS in a
// fixed order.  768 chunks of 2048 columns: 12 us (25 MB).
template <class T>
__global__ void __launch_bounds__(1024) rar_norm_sums(const NormGradParams p)
{
    __shared__ float joined[2][16][16];
    const int quad = threadIdx.x & 3, slice = threadIdx.x >> 2, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 16 + quad * 4;
    const int pair = p.sum_post ? (int)blockIdx.y * 2 : 2;  // the sums of this workgroup
    f32x4 t[2] = {};
    if (c < p.pitch)
#pragma unroll 4
        for (int64_t k = slice; k < p.chunks; k += 256)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                t[j] += load4(p.part + (k * kSums + pair + j) * p.pitch + c);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int d = 4; d < 64; d *= 2)
                t[j][i] += __shfl_xor(t[j][i], d);
            if ((threadIdx.x & 63) < 4)
                joined[j][wave][quad * 4 + i] = t[j][i];
        }
    __syncthreads();
    const int64_t col = (int64_t)blockIdx.x * 16 + threadIdx.x;
    if (threadIdx.x >= 16 || col >= p.cols)
        return;
    float v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        v[j] = 0.0f;
#pragma unroll
        for (int w = 0; w < 16; ++w)
            v[j] += joined[j][w][threadIdx.x];
    }
    auto vec = [&](const void *q, float other) { return q ? to_f32(((const T *)q)[col]) : other; };
    auto put = [&](void *q, float r) {
        if (q)
            ((T *)q)[col] = from_f32<T>(p.accumulate ? to_f32(((const T *)q)[col]) + r : r);
    };
    if (pair == 2) {
        put(p.dpre_w, v[0]);
        put(p.dpre_b, v[1]);
        return;
    }
    const float sg = p.s * vec(p.gate, 1.0f);
    put(p.dpost_w, sg * v[0]);
    put(p.dpost_b, sg * v[1]);
    put(p.dgate, p.s * (p.post ? __builtin_fmaf(vec(p.post_w, 1.0f), v[0], vec(p.post_b, 0.0f) * v[1]) : v[0]));
}

// Lanes of a row at eight columns a lane: a wave at least, a workgroup of 1024 at
// most, or 0 for a row of more.
int row_lanes(int64_t cols)
{
    int lanes = 64;
    while (lanes <= 1024 && (int64_t)lanes * 8 < cols)
        lanes *= 2;
    return lanes <= 1024 ? lanes : 0;
}

int rows_of(int lanes) { return lanes && lanes < 256 ? 256 / lanes : 1; }
unsigned threads_of(int lanes) { return lanes ? std::max(lanes, 256) : kWideLanes; }

int64_t row_groups(int64_t rows, int64_t cols)
{
    const int per = rows_of(row_lanes(cols));
    return (rows + per - 1) / per;
}

// Workgroups of the backward kernel at once.
int64_t most_chunks(int64_t cols)
{
    const int lanes = row_lanes(cols);
    if (!lanes)
        return cols <= 65536 ? 256 : (int64_t(1) << 24) / cols;
    return lanes > 256 ? 256 * 1024 / lanes : 768;
}

template <class P>
struct RowKernels {
    void (*f32)(P), (*bf)(P);
};

}  // namespace

int64_t norm_chunks(int64_t rows, int64_t cols)
{
    // A chunk a workgroup, as many as the registers (or, of rows longer than 2048, the column sums in LDS) let in at
    // once: 65536 x 2048 bf16, kernel and sums, 768 chunks 350 us, 512 369, 1024 (a second turn for some) 398.  The
    // rows are spread evenly over the turns, and few rows take two of them: 1027 x 1001 binary32, 257 chunks of two
    // turns 12.6 us and their sums 4.8, 514 of one 13.2 and 6.5.
    const int64_t most = most_chunks(cols), groups = row_groups(rows, cols);
    const int64_t turns = groups > 256 && groups < most ? 2 : (groups + most - 1) / most;
    return (groups + turns - 1) / turns;
}

int64_t norm_chunks_up_to(int64_t rows, int64_t cols)
{
    // (the number falls where two turns begin)
    const int64_t most = most_chunks(cols), groups = row_groups(rows, cols);
    return groups >= most ? most : std::min(groups, std::max<int64_t>(256, (groups + 1) / 2));
}

hipError_t launch_norm(rar_dtype dt, const NormParams &p, hipStream_t st)
{
    const int lanes = row_lanes(p.cols), per = rows_of(lanes);
    const unsigned threads = threads_of(lanes);
    const int64_t blocks = std::min<int64_t>((p.rows + per - 1) / per, 256 * (2048 / threads));
    RowKernels<NormParams> k{rar_norm_wide<float>, rar_norm_wide<bf16>};
    switch (lanes) {
    case 64: k = {rar_norm_rows<float, 64>, rar_norm_rows<bf16, 64>}; break;
    case 128: k = {rar_norm_rows<float, 128>, rar_norm_rows<bf16, 128>}; break;
    case 256: k = {rar_norm_rows<float, 256>, rar_norm_rows<bf16, 256>}; break;
    case 512: k = {rar_norm_rows<float, 512>, rar_norm_rows<bf16, 512>}; break;
    case 1024: k = {rar_norm_rows<float, 1024>, rar_norm_rows<bf16, 1024>}; break;
    }
    return launch(dt == RAR_BF16 ? k.bf : k.f32, (unsigned)blocks, threads, st, p);
}

hipError_t launch_norm_grad(rar_dtype dt, const NormGradParams &p, hipStream_t st)
{
    const int lanes = row_lanes(p.cols);
    RowKernels<NormGradParams> k{rar_norm_grad_wide<float>, rar_norm_grad_wide<bf16>};
    switch (lanes) {
    case 64: k = {rar_norm_grad_rows<float, 64>, rar_norm_grad_rows<bf16, 64>}; break;
    case 128: k = {rar_norm_grad_rows<float, 128>, rar_norm_grad_rows<bf16, 128>}; break;
    case 256: k = {rar_norm_grad_rows<float, 256>, rar_norm_grad_rows<bf16, 256>}; break;
    case 512: k = {rar_norm_grad_rows<float, 512>, rar_norm_grad_rows<bf16, 512>}; break;
    case 1024: k = {rar_norm_grad_rows<float, 1024>, rar_norm_grad_rows<bf16, 1024>}; break;
    }
    return launch(dt == RAR_BF16 ? k.bf : k.f32, (unsigned)p.chunks, threads_of(lanes), st, p);
}

hipError_t launch_norm_sums(rar_dtype dt, const NormGradParams &p, hipStream_t st)
{
    const dim3 grid((unsigned)((p.pitch + 15) / 16), p.sum_post && p.sum_pre ? 2 : 1);
    return launch(dt == RAR_BF16 ? rar_norm_sums<bf16> : rar_norm_sums<float>, grid, 1024, st, p);
}

}  // namespace rar
