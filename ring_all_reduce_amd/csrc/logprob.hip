// logprob.hip -- CDNA4 (gfx950) kernels of log probabilities of given tokens, with
// entropy, top alternatives and the gradient in the logits.
//
// With m = max z, d = scale (m - z) >= 0, S = sum e^-d:
//   log p = -d - log S,  entropy = log S + (sum d e^-d) / S   (no term cancels)
//   dz = scale (dlogp [j = target] - p (dlogp + dentropy (log p + entropy)))
//
// Bound by HBM: a row passes once through the registers of its lanes, in its own
// type; the exponentials are taken twice rather than kept.  Nothing but the
// results is written, so a loss with its gradient reads the logits once and
// writes dz.
//
// Alternatives: an element's key orders by value, then by the lower index, and
// no two are alike.  The row is cut into 64 groups; the K-th largest of the
// groups' best keys is at most the K-th largest key, since K keys reach it.  The
// few keys that do (some thirty of 32000 for K = 20) are collected in LDS and
// ranked by counting.  Where they are too many (rows of equal or sorted values),
// K rounds each take the largest key under the last.
#include "ops_internal.h"
#include "row.h"

#pragma clang fp contract(off)

namespace rar {
namespace {

constexpr int kMost = RAR_LOGPROB_MAX_TOP;
constexpr int kGroups = 64;
constexpr int kCandidates = 256;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kInf = __builtin_inff();

// Larger for a larger value, then for a lower index; zero for a masked element or
// a NaN.  The two zeros are one value.
__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);
    if (!(v > -kInf))
        return 0;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int d)
{
    const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)v, d), hi = (uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), d);
    return (uint64_t)hi << 32 | lo;
}

template <int LANES>
struct TopLds {
    static constexpr int kRows = LANES >= 256 ? 1 : 256 / LANES;
    uint64_t best[kRows][kGroups];
    uint64_t floor[kRows];
    uint32_t found[kRows];
    uint64_t keys[kRows][kCandidates];
};

// A row of LANES lanes; R eights a lane in registers, or R = 0: read again from
// memory for each pass.
template <class T, int LANES, int R, bool GRAD>
__global__ void __launch_bounds__(LANES > 256 ? LANES : 256) rar_logprob_rows(const LogprobParams p)
{
    typedef RowJoin<LANES, 2> Join;
    constexpr int kRows = Join::kThreads / LANES;
    constexpr int kHeld = R ? R : 1;
    __shared__ float lds[Join::kFloats];
    __shared__ TopLds<LANES> top;
    Join join{lds};
    const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;

    for (int64_t first = (int64_t)blockIdx.x * kRows; first < p.rows; first += (int64_t)gridDim.x * kRows) {
        const int64_t row = first + sub;
        const bool live = row < p.rows;
        const T *const z = (const T *)p.z + row * p.ldz;
        Eight<T> held[kHeld];
        if (R) {
#pragma unroll
            for (int k = 0; k < kHeld; ++k) {
                const int64_t c = ((int64_t)k * LANES + lane) * 8;
                held[k].load(z + c, live ? clamp8(p.cols - c) : 0, -kInf);
            }
        }
        // f(column, how many of the eight exist, values; the others -infinity)
        auto each = [&](auto &&f) __attribute__((always_inline)) {
            if (R) {
#pragma unroll
                for (int k = 0; k < kHeld; ++k) {
                    const int64_t c = ((int64_t)k * LANES + lane) * 8;
                    held[k].forget();
                    f(c, live ? clamp8(p.cols - c) : 0, held[k]);
                }
            } else {
                for (int64_t c = (int64_t)lane * 8; c < p.cols; c += LANES * 8) {
                    Eight<T> v;
                    v.load(z + c, clamp8(p.cols - c), -kInf);
                    f(c, clamp8(p.cols - c), v);
                }
            }
        };
        // (before dz, which may be z, is written)
        int64_t target = -1;
        float zt = 0.0f;
        if (p.targets && live) {
            target = p.targets[row];
            if (target < 0 || target >= p.cols)
                target = -1;
            else
                zt = to_f32(z[target]);
        }

        float t[2] = {-kInf, 0.0f};
        each([&](int64_t, int, const Eight<T> &v) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                t[0] = __builtin_fmaxf(t[0], v.get(i));
        });
        float m[1] = {t[0]};
        join.max(m);
        const float base = m[0] == -kInf ? 0.0f : m[0];
        t[0] = 0.0f;
        each([&](int64_t, int, const Eight<T> &v) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = (base - v.get(i)) * p.scale;
                const float e = __builtin_amdgcn_exp2f(d * -kLog2e);
                t[0] += e;
                t[1] = __builtin_fmaf(e, __builtin_fminf(d, 1e30f), t[1]);  // a masked element adds 0 * 1e30
            }
        });
        join.sum(t);
        const bool none = t[0] == 0.0f;  // (NaN: false)
        const float ls = none ? 0.0f : logf(t[0]);
        const float inv = none ? 0.0f : 1.0f / t[0];
        const float ent = none ? 0.0f : __builtin_fmaf(t[1], inv, ls);
        if (lane == 0 && live) {
            if (p.entropy)
                p.entropy[row] = ent;
            if (p.logp)
                p.logp[row] = target < 0 ? 0.0f : (none ? -kInf : -((base - zt) * p.scale) - ls);
        }

        if (GRAD) {
            const float dl = p.dlogp && target >= 0 && !none ? p.dlogp[row] : 0.0f;
            const float de = p.dentropy && live ? p.dentropy[row] : 0.0f;
            const float add = de == 0.0f ? 0.0f : ent - ls;
            T *const dz = (T *)p.dz + row * p.lddz;
            each([&](int64_t c, int cnt, const Eight<T> &v) __attribute__((always_inline)) {
                float g[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float d = (base - v.get(i)) * p.scale;
                    const float e = __builtin_amdgcn_exp2f(d * -kLog2e) * inv;
                    const float w = __builtin_fmaf(de, add - __builtin_fminf(d, 1e30f), dl);
                    g[i] = -(e * w) * p.scale;
                }
                if (target >= c && target < c + 8)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (target == c + i)
                            g[i] = __builtin_fmaf(p.scale, dl, g[i]);
                if (live)
                    store8<true>(dz + c, cnt, g);
            });
            continue;
        }
        if (!p.top)
            continue;

        // ---- alternatives ----
        const bool bad = t[0] != t[0];
        uint64_t mine = 0;
        each([&](int64_t c, int, const Eight<T> &v) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t k = key_of(v.get(i));
                const uint64_t key = (uint64_t)k << 32 | (uint32_t)~(uint32_t)(c + i);
                if (k && key > mine)
                    mine = key;
            }
        });
        uint64_t group = mine;
#pragma unroll
        for (int d = 1; d < LANES / kGroups; d *= 2) {
            const uint64_t o = shfl_xor64(group, d);
            group = o > group ? o : group;
        }
        if (lane % (LANES / kGroups) == 0)
            top.best[sub][lane / (LANES / kGroups)] = group;
        if (lane == 0)
            top.found[sub] = 0;
        __syncthreads();
        if (lane < 64) {
            const uint64_t own = top.best[sub][lane];
            int above = 0;
            for (int i = 0; i < kGroups; ++i)
                above += top.best[sub][i] > own;
            // the group's best at rank K - 1; equal ones are empty groups, of which each writes zero
            if (lane == 0)
                top.floor[sub] = 0;
            if (above == p.top - 1 && own)
                top.floor[sub] = own;
        }
        __syncthreads();
        const uint64_t low = top.floor[sub] ? top.floor[sub] : 1;
        if (mine >= low && !bad)
            each([&](int64_t c, int, const Eight<T> &v) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t k = key_of(v.get(i));
                    const uint64_t key = (uint64_t)k << 32 | (uint32_t)~(uint32_t)(c + i);
                    if (k && key >= low) {
                        const uint32_t at = atomicAdd(&top.found[sub], 1u);
                        if (at < kCandidates)
                            top.keys[sub][at] = key;
                    }
                }
            });
        __syncthreads();
        const uint32_t found = top.found[sub];
        int64_t *const ids = p.top_ids + row * p.top;
        float *const lps = p.top_logp + row * p.top;
        auto put = [&](int at, uint64_t key) __attribute__((always_inline)) {
            ids[at] = (int64_t)(uint32_t)~(uint32_t)key;
            lps[at] = -((base - value_of((uint32_t)(key >> 32))) * p.scale) - ls;
        };
        if (found <= kCandidates) {
            if (live)
                for (uint32_t i = lane; i < (found > (uint32_t)kMost ? found : (uint32_t)kMost); i += LANES) {
                    if (i < found) {
                        const uint64_t own = top.keys[sub][i];
                        int above = 0;
                        for (uint32_t k = 0; k < found; ++k)
                            above += top.keys[sub][k] > own;
                        if (above < p.top)
                            put(above, own);
                    } else if (i < (uint32_t)p.top) {
                        ids[i] = -1;
                        lps[i] = bad ? __builtin_nanf("") : -kInf;
                    }
                }
        }
        if (LANES == 64) {
            // a wave to a row: no other wave waits for its rounds
            if (found > kCandidates) {
                uint64_t last = ~(uint64_t)0;
                for (int k = 0; k < p.top; ++k) {
                    uint64_t b = 0;
                    each([&](int64_t c, int, const Eight<T> &v) __attribute__((always_inline)) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t w = key_of(v.get(i));
                            const uint64_t key = (uint64_t)w << 32 | (uint32_t)~(uint32_t)(c + i);
                            if (w && key < last && key > b)
                                b = key;
                        }
                    });
#pragma unroll
                    for (int d = 1; d < 64; d *= 2) {
                        const uint64_t o = shfl_xor64(b, d);
                        b = o > b ? o : b;
                    }
                    last = b;
                    if (lane == 0)
                        put(k, b);
                }
            }
        } else if (found > kCandidates) {  // one row: the whole workgroup agrees
            uint64_t last = ~(uint64_t)0;
            for (int k = 0; k < p.top; ++k) {
                uint64_t b = 0;
                each([&](int64_t c, int, const Eight<T> &v) __attribute__((always_inline)) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t w = key_of(v.get(i));
                        const uint64_t key = (uint64_t)w << 32 | (uint32_t)~(uint32_t)(c + i);
                        if (w && key < last && key > b)
                            b = key;
                    }
                });
#pragma unroll
                for (int d = 1; d < 64; d *= 2) {
                    const uint64_t o = shfl_xor64(b, d);
                    b = o > b ? o : b;
                }
                __syncthreads();
                if ((threadIdx.x & 63) == 0)
                    top.keys[0][threadIdx.x >> 6] = b;
                __syncthreads();
                b = 0;
                for (int w = 0; w < LANES / 64; ++w) {
                    const uint64_t o = top.keys[0][w];
                    b = o > b ? o : b;
                }
                last = b;
                if (lane == 0)
                    put(k, b);
            }
        }
        __syncthreads();  // the next row writes these lists again
    }
}

struct Kernels {
    void (*f32)(LogprobParams), (*bf)(LogprobParams);
};

template <int LANES, int R>
Kernels kernels_of(bool grad)
{
    if (grad)
        return {rar_logprob_rows<float, LANES, R, true>, rar_logprob_rows<bf16, LANES, R, true>};
    return {rar_logprob_rows<float, LANES, R, false>, rar_logprob_rows<bf16, LANES, R, false>};
}

}  // namespace

hipError_t launch_logprob(rar_dtype dt, const LogprobParams &p, hipStream_t st)
{
    const bool grad = p.dz != nullptr;
    Kernels k;
    int lanes = 1024;
    if (p.cols <= 64 * 8 * 4) {
        k = kernels_of<64, 4>(grad);
        lanes = 64;
    } else if (p.cols <= 256 * 8 * 4) {
        k = kernels_of<256, 4>(grad);
        lanes = 256;
    } else if (p.cols <= 1024 * 8 * 4) {
        k = kernels_of<1024, 4>(grad);
    } else if (p.cols <= 1024 * 8 * 8) {
        k = kernels_of<1024, 8>(grad);
    } else {
        k = kernels_of<1024, 0>(grad);
    }
    const int threads = lanes > 256 ? lanes : 256, per = threads / lanes;
    const int64_t blocks = (p.rows + per - 1) / per, most = 256 * (2048 / threads);
    return launch(dt == RAR_BF16 ? k.bf : k.f32, (unsigned)(blocks < most ? blocks : most), threads, st, p);
}

}  // namespace rar
