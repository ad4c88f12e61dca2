// logprob.hip -- CDNA4 (gfx950) kernels of log probabilities of given tokens, with
// entropy, top alternatives and the gradient in the logits.
//
// With m = max z, t = (z - m) scale log2 e <= 0, S = sum 2^t:
//   log p = scale (z - m) - log S,  entropy = log S - ln 2 (sum t 2^t) / S   (no term cancels)
//   dz = scale (dlogp [j = target] - p (dlogp + dentropy (log p + entropy))),  p = 2^(t - log2 S)
//
// A row passes once through the registers of its lanes, in its own type, and the
// exponentials are taken twice rather than kept.  Nothing but the results is
// written, so a loss with its gradient reads the logits once and writes dz.
//
// Alternatives: the row is cut into 64 groups of neighbouring lanes.  The K-th
// largest of the groups' maxima is at most the K-th largest element, since K
// elements reach it.  The few that do (some thirty of 32000 for K = 20) are
// collected in LDS under a key that orders by value, then by the lower index, and
// ranked by counting.  Where they are too many (rows of equal or sorted values),
// K rounds each take the largest key under the last.
//
// 8192 x 32000 in bf16: with entropy 121 us (524 MB, 4.3 TB/s), with eight alternatives
// besides 147 (vector units busy for 73%), with the gradient 219 (1.05 GB, 4.8 TB/s); in
// binary32 213 with alternatives and 443 with the gradient, at HBM's rate.  With
// alternatives in bf16 a narrower row waits more for the chain of its joins, under
// which nothing is loaded: 4096 x 20000 54 us (3.0 TB/s), 4096 x 10000 36 (2.3).  Eight
// rows in binary32 with alternatives: 8 us, a launch and a row's own chain of joins.
#include "ops_internal.h"
#include "row.h"

#pragma clang fp contract(off)

namespace rar {
namespace {

constexpr int kMost = RAR_LOGPROB_MAX_TOP;
constexpr int kGroups = 64;
constexpr int kCandidates = 256;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kInf = __builtin_inff();
constexpr float kNothing = -1000.0f;  // 2^this is zero

// Larger for a larger value, then for a lower index, and never zero; the two zeros
// are one value.
__device__ __forceinline__ uint64_t key_at(float v, int64_t index)
{
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (uint64_t)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (uint32_t)~(uint32_t)index;
}

__device__ __forceinline__ float value_of(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int d)
{
    const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)v, d);
    const uint32_t hi = (uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), d);
    return (uint64_t)hi << 32 | lo;
}

// What stands behind is not begun before what stands before: left to itself the
// compiler takes every eight of a row at once, and runs out of registers.
__device__ __forceinline__ void one_after_another()
{
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_sched_barrier(0);
#endif
}

// v, of which nothing is known: what is computed from it is not kept from row to row
// (columns, counts and masks of every eight would take more registers than the row).
__device__ __forceinline__ int forgotten(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}

template <int LANES>
struct TopLds {
    static constexpr int kRows = LANES >= 256 ? 1 : 256 / LANES;
    float best[kRows][kGroups];
    uint32_t found[kRows];
    uint64_t keys[kRows][kCandidates];
};

// A row of LANES lanes; R eights a lane in registers, or R = 0: read again from
// memory for each pass.
// Held to 64 registers where the row takes at most half of them, so that two
// workgroups of 1024 share a compute unit: one waits while the other computes.
// (Two to eight registers a lane are spilled for it, in binary32 with alternatives
// and in bf16 of eight eights: 8192 x 32000 in bf16 with eight alternatives writes
// 16 MB for results of 0.9 and reads 586 for 524.)
template <class T, int LANES, int R, bool GRAD>
__global__ void __launch_bounds__(LANES > 256 ? LANES : 256, R * sizeof(T) <= 16 ? 8 : 4)
    rar_logprob_rows(const LogprobParams p)
{
    typedef RowJoin<LANES, 2> Join;
    constexpr int kRows = Join::kThreads / LANES;
    constexpr int kHeld = R ? R : 1;
    // (with six or eight eights it takes registers that are short there: 6% of 8192 x 32000)
    constexpr bool kSkip = R == 4 || R == 16;
    __shared__ float lds[Join::kFloats];
    __shared__ TopLds<LANES> top;
    Join join{lds};
    const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    const int first_lane = __builtin_amdgcn_readfirstlane(lane & ~63);

    for (int64_t first = (int64_t)blockIdx.x * kRows; first < p.rows; first += (int64_t)gridDim.x * kRows) {
        const int64_t row = first + sub;
        const bool live = row < p.rows;
        const T *const z = (const T *)p.z + row * p.ldz;
        Eight<T> held[kHeld];
        if (R) {
            const int mine = forgotten(lane);
#pragma unroll
            for (int k = 0; k < kHeld; ++k) {
                const int64_t c = ((int64_t)k * LANES + mine) * 8;
                held[k].load(z + c, live ? clamp8(p.cols - c) : 0, -kInf);
            }
        }
        // f(which eight, column, how many of it exist, values; the others -infinity); where rows may fill half the
        // lanes, a wave passes over what it has nothing of
        auto each = [&](auto &&f) __attribute__((always_inline)) {
            if (R) {
                const int mine = forgotten(lane);
#pragma unroll
                for (int k = 0; k < kHeld; ++k) {
                    if (kSkip && k >= R / 2 && (k * LANES + first_lane) * 8 >= (int)p.cols)
                        continue;
                    const int64_t c = ((int64_t)k * LANES + mine) * 8;
                    held[k].forget();
                    f(k, c, live ? clamp8(p.cols - c) : 0, held[k]);
                    one_after_another();
                }
            } else {
                for (int64_t c = (int64_t)lane * 8; c < p.cols; c += LANES * 8) {
                    Eight<T> v;
                    v.load(z + c, clamp8(p.cols - c), -kInf);
                    f(0, c, clamp8(p.cols - c), v);
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

        // the largest of each eight: the row's maximum, and where alternatives can be
        float best[kHeld], m[1] = {-kInf};
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
            best[k] = -kInf;
        each([&](int k, int64_t, int, const Eight<T> &v) __attribute__((always_inline)) {
            float b = v.get(0);
#pragma unroll
            for (int i = 1; i < 8; ++i)
                b = __builtin_fmaxf(b, v.get(i));
            if (R)
                best[k] = b;
            m[0] = __builtin_fmaxf(m[0], b);
        });
        const float mine = m[0];
        join.max(m);
        const float base = m[0] == -kInf ? 0.0f : m[0], unit = p.scale * kLog2e;
        float t[2] = {0.0f, 0.0f};
        each([&](int, int64_t, int, const Eight<T> &v) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = (v.get(i) - base) * unit;
                const float e = __builtin_amdgcn_exp2f(x);
                t[0] += e;
                t[1] = __builtin_fmaf(e, __builtin_fmaxf(x, kNothing), t[1]);  // a masked element adds 0 * kNothing
            }
        });
        join.sum(t);
        const bool none = t[0] == 0.0f;  // (NaN: false)
        const float ls = none ? 0.0f : logf(t[0]);
        const float ent = none ? 0.0f : __builtin_fmaf(t[1] / t[0], -kLn2, ls);
        if (lane == 0 && live) {
            if (p.entropy)
                p.entropy[row] = ent;
            if (p.logp)
                p.logp[row] = target < 0 ? 0.0f : (none ? -kInf : (zt - base) * p.scale - ls);
        }

        if (GRAD) {
            const float dl = p.dlogp && target >= 0 && !none ? p.dlogp[row] : 0.0f;
            const float de = p.dentropy && live ? p.dentropy[row] : 0.0f;
            const float l2 = ls * kLog2e;
            // dz = p (flat + slope t)
            const float flat = -p.scale * (de == 0.0f ? dl : __builtin_fmaf(de, ent, dl));
            const float slope = -p.scale * (de * kLn2);
            T *const dz = (T *)p.dz + row * p.lddz;
            auto write = [&](int64_t c, int cnt, float (&g)[8]) __attribute__((always_inline)) {
                if (target >= c && target < c + 8)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (target == c + i)
                            g[i] = __builtin_fmaf(p.scale, dl, g[i]);
                if (live)
                    store8<true>(dz + c, cnt, g);
            };
            if (p.dentropy)
                each([&](int, int64_t c, int cnt, const Eight<T> &v) __attribute__((always_inline)) {
                    float g[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float x = __builtin_fmaf(v.get(i) - base, unit, -l2);
                        g[i] = __builtin_amdgcn_exp2f(x) * __builtin_fmaf(slope, __builtin_fmaxf(x, kNothing), flat);
                    }
                    write(c, cnt, g);
                });
            else
                each([&](int, int64_t c, int cnt, const Eight<T> &v) __attribute__((always_inline)) {
                    float g[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        g[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(v.get(i) - base, unit, -l2)) * flat;
                    write(c, cnt, g);
                });
            continue;
        }
        if (!p.top)
            continue;

        // ---- alternatives ----
        const bool bad = t[0] != t[0];
        constexpr int kEach = LANES / kGroups;          // lanes of a group
        constexpr int kSome = kGroups * kGroups / LANES;  // groups that a lane compares its own with
        float group = mine;
#pragma unroll
        for (int d = 1; d < kEach; d *= 2)
            group = __builtin_fmaxf(group, __shfl_xor(group, d));
        if (lane % kEach == 0)
            top.best[sub][lane / kEach] = group;
        if (lane == 0)
            top.found[sub] = 0;
        __syncthreads();
        {
            // the lanes of a group count the groups that are as large; those that K or more are not
            // smaller than (and the K-th itself) have the K-th largest value or one above it
            int reach = 0;
#pragma unroll
            for (int i = 0; i < kSome; ++i)
                reach += top.best[sub][lane % kEach * kSome + i] >= group;
#pragma unroll
            for (int d = 1; d < kEach; d *= 2)
                reach += __shfl_xor(reach, d);
            __syncthreads();
            if (lane % kEach == 0)
                top.best[sub][lane / kEach] = reach >= p.top ? group : -kInf;
        }
        __syncthreads();
        const float low = wave_max(top.best[sub][threadIdx.x & 63]);
        if (!bad) {
            each([&](int k, int64_t c, int, const Eight<T> &v) __attribute__((always_inline)) {
                if (R && !__any(best[k] >= low))
                    return;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = v.get(i);
                    if (x >= low && x > -kInf) {
                        const uint32_t n = atomicAdd(&top.found[sub], 1u);
                        if (n < kCandidates)
                            top.keys[sub][n] = key_at(x, c + i);
                    }
                }
            });
        }
        __syncthreads();
        const uint32_t found = top.found[sub];
        int64_t *const ids = p.top_ids + row * p.top;
        float *const lps = p.top_logp + row * p.top;
        auto put = [&](int at, uint64_t key) __attribute__((always_inline)) {
            ids[at] = (int64_t)(uint32_t)~(uint32_t)key;
            lps[at] = (value_of((uint32_t)(key >> 32)) - base) * p.scale - ls;
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
                    each([&](int, int64_t c, int, const Eight<T> &v) __attribute__((always_inline)) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float x = v.get(i);
                            const uint64_t key = key_at(x, c + i);
                            if (x > -kInf && key < last && key > b)
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
                each([&](int, int64_t c, int, const Eight<T> &v) __attribute__((always_inline)) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float x = v.get(i);
                        const uint64_t key = key_at(x, c + i);
                        if (x > -kInf && key < last && key > b)
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

template <class T, int LANES, int R>
auto kernel_of(bool grad)
{
    return grad ? rar_logprob_rows<T, LANES, R, true> : rar_logprob_rows<T, LANES, R, false>;
}

template <int LANES, int R>
Kernels kernels_of(bool grad)
{
    return {kernel_of<float, LANES, R>(grad), kernel_of<bf16, LANES, R>(grad)};
}

}  // namespace

hipError_t launch_logprob(rar_dtype dt, const LogprobParams &p, hipStream_t st)
{
    // Lanes of a row and eights a lane.  More rows than two to a compute unit go to half the lanes as long as 64
    // registers hold the row: four workgroups a unit wait for each other less than two.  8192 x 32000 bf16 with 8
    // alternatives takes 172 us at 1024 lanes and 138 at 512, its gradient 223 and 211; eight rows take 8 at 1024.
    // Six eights besides four and eight: 4096 x 20000 bf16 takes 54 us and 80 with the gradient, 69 and 98 with eight.
    // bf16 rows up to 131072 fit 128 registers: 2048 x 128256 takes 166 and 257 us, read again from memory 220 and 306.
    const bool grad = p.dz != nullptr, many = p.rows > 512;
    Kernels k{};
    int lanes = 1024;
    if (p.cols <= 64 * 8 * 4) {
        k = kernels_of<64, 4>(grad);
        lanes = 64;
    } else if (p.cols <= 256 * 8 * 4) {
        k = kernels_of<256, 4>(grad);
        lanes = 256;
    } else if (many && p.cols <= 512 * 8 * 4) {
        k = kernels_of<512, 4>(grad);
        lanes = 512;
    } else if (many && dt == RAR_BF16 && p.cols <= 512 * 8 * 6) {
        k.bf = kernel_of<bf16, 512, 6>(grad);
        lanes = 512;
    } else if (many && dt == RAR_BF16 && p.cols <= 512 * 8 * 8) {
        k.bf = kernel_of<bf16, 512, 8>(grad);
        lanes = 512;
    } else if (p.cols <= 1024 * 8 * 4) {
        k = kernels_of<1024, 4>(grad);
    } else if (p.cols <= 1024 * 8 * 6) {
        k = kernels_of<1024, 6>(grad);
    } else if (p.cols <= 1024 * 8 * 8) {
        k = kernels_of<1024, 8>(grad);
    } else if (dt == RAR_BF16 && p.cols <= 1024 * 8 * 16) {
        k.bf = kernel_of<bf16, 1024, 16>(grad);
    } else {
        k = kernels_of<1024, 0>(grad);
    }
    const int threads = lanes > 256 ? lanes : 256, per = threads / lanes;
    const int64_t blocks = (p.rows + per - 1) / per, most = 256 * (2048 / threads);
    return launch(dt == RAR_BF16 ? k.bf : k.f32, (unsigned)(blocks < most ? blocks : most), threads, st, p);
}

}  // namespace rar
