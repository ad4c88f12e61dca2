// ckpt.hip -- CDNA4 (gfx950) kernels of activation checkpoints in 8 bits.
//
// A row is cut into groups of 32 values that share a power of two:
//   e    = the smallest exponent (from -126) with max|x| <= 448 * 2^e
//   code = x / 2^e rounded to the nearest e4m3 value, ties to even
// so nothing saturates, and x^ = code * 2^e has at most four significant bits:
// it is exact in bf16, and a matrix product reads it without another rounding.
// The group's maximum is taken over its finite values; a NaN or an infinity
// becomes e4m3's NaN and touches no other value of its group.
//
// Both directions are streaming passes bound by HBM bandwidth: four lanes share
// a group, a lane moves eight values (16 bytes of bf16), and the group's
// maximum takes two lane exchanges.  8192 x 8192 in bf16: store 36 us (5.7
// TB/s); load with gelu 47 us, bound by the activation's arithmetic (its waves
// wait 25% of their cycles, the store's 60%); 8192 x 2048 without an activation 11
// us (4.6 TB/s).
#include "act.h"
#include "ops_internal.h"

#pragma clang fp contract(off)

namespace rar {
namespace {

constexpr int kLane = 8;                         // values of a lane
constexpr int kLanes = kCkptGroup / kLane;       // lanes of a group
constexpr int kPerBlock = 256 / kLanes;          // groups of a workgroup pass
constexpr int kPasses = 4;

// Group `at` of the workgroup's run: its row and its place in the row.  The
// 64-bit division is the same for the whole workgroup.
struct Place {
    int64_t row;
    uint32_t group;
};

__device__ __forceinline__ Place place(uint32_t groups, uint32_t at)
{
    const int64_t first = (int64_t)blockIdx.x * (kPerBlock * kPasses);
    const int64_t row0 = first / groups;
    const uint32_t g = (uint32_t)(first - row0 * groups) + at;
    const uint32_t r = g / groups;
    return Place{row0 + r, g - r * groups};
}

template <class T>
__global__ void __launch_bounds__(256) rar_ckpt_store_rows(const CkptParams p)
{
    const uint32_t groups = (uint32_t)((p.cols + kCkptGroup - 1) / kCkptGroup);
    const int q = threadIdx.x % kLanes;
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
        const Place at = place(groups, u * kPerBlock + threadIdx.x / kLanes);
        if (at.row >= p.rows)
            return;
        const int64_t c = (int64_t)at.group * kCkptGroup + q * kLane;
        const int cnt = p.cols - c >= kLane ? kLane : (p.cols - c < 0 ? 0 : (int)(p.cols - c));
        float v[8];
        load8<true>((const T *)p.x + at.row * p.ldx + c, cnt, v);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            top = ckpt_top(top, v[i]);
#pragma unroll
        for (int d = 1; d < kLanes; d *= 2)
            top = max(top, (uint32_t)__shfl_xor(top, d));
        const int e = ckpt_exponent(top);
        const uint32_t w[2] = {ckpt_codes4(f32x4{v[0], v[1], v[2], v[3]}, e),
                               ckpt_codes4(f32x4{v[4], v[5], v[6], v[7]}, e)};
        *reinterpret_cast<u32x2 *>(p.codes + (at.row * groups + at.group) * kCkptGroup + q * kLane) = u32x2{w[0], w[1]};
        if (q == 0)
            p.scales[at.row * groups + at.group] = (uint8_t)e;
    }
}

template <class T>
__global__ void __launch_bounds__(256) rar_ckpt_load_rows(const CkptParams p)
{
    const uint32_t groups = (uint32_t)((p.cols + kCkptGroup - 1) / kCkptGroup);
    const int64_t width = p.pitch_zero > p.cols ? p.pitch_zero : p.cols;
    const int q = threadIdx.x % kLanes;
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
        const Place at = place(groups, u * kPerBlock + threadIdx.x / kLanes);
        if (at.row >= p.rows)
            return;
        const int64_t c = (int64_t)at.group * kCkptGroup + q * kLane;
        const int64_t g = at.row * groups + at.group;
        const u32x2 w = *reinterpret_cast<const u32x2 *>(p.codes + g * kCkptGroup + q * kLane);
        const uint32_t e = p.scales[g];
        float v[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 x = ckpt_values4(w[h], e);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[4 * h + i] = x[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = act_value<T>(p.act, v[i]);
        if (c + kLane > p.cols)  // codes behind the matrix may hold anything
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = c + i < p.cols ? v[i] : 0.0f;
        const int cnt = width - c >= kLane ? kLane : (width - c < 0 ? 0 : (int)(width - c));
        store8((T *)p.y + at.row * p.ldy + c, cnt, v);
    }
}

unsigned blocks_of(const CkptParams &p)
{
    const int64_t groups = p.rows * ((p.cols + kCkptGroup - 1) / kCkptGroup);
    return (unsigned)((groups + kPerBlock * kPasses - 1) / (kPerBlock * kPasses));
}

}  // namespace

hipError_t launch_ckpt_store(rar_dtype dt, const CkptParams &p, hipStream_t st)
{
    return launch(dt == RAR_BF16 ? rar_ckpt_store_rows<bf16> : rar_ckpt_store_rows<float>, blocks_of(p), 256, st, p);
}

hipError_t launch_ckpt_load(rar_dtype dt, const CkptParams &p, hipStream_t st)
{
    return launch(dt == RAR_BF16 ? rar_ckpt_load_rows<bf16> : rar_ckpt_load_rows<float>, blocks_of(p), 256, st, p);
}

}  // namespace rar
