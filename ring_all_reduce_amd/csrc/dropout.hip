// dropout.hip -- CDNA4 (gfx950) kernel of dropout with a counter-based generator.
//
//   y = r + keep . x 65536 / kept
//
// A lane takes a group of eight elements of a row and makes their eight 16-bit
// draws with one call of Philox4x32-10 (J. Salmon et al., "Parallel random
// numbers: as easy as 1, 2, 3", 2011) on the group's number, so the mask needs
// no memory and is made again by the backward pass.  Sixteen bits a draw: the
// twenty 32 x 32 products of a call are most of the kernel's arithmetic, and
// halves of its words serve twice as many elements.  1 - p is off by at most
// 2^-17, and the scale is that of the draws that are kept, so the mean is not.
// Bound by HBM: 65536 x 2048 in bf16 with a residual 140 us (5.8 TB/s),
// vector units busy half of that.
#include "ops_internal.h"
#include "row.h"

#pragma clang fp contract(off)

namespace rar {
namespace {

constexpr int kPasses = 4;

__device__ __forceinline__ u32x4 philox(u32x4 c, uint32_t k0, uint32_t k1)
{
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)0xD2511F53u * c.x, b = (uint64_t)0xCD9E8D57u * c.z;
        c = u32x4{(uint32_t)(b >> 32) ^ c.y ^ k0, (uint32_t)b, (uint32_t)(a >> 32) ^ c.w ^ k1, (uint32_t)a};
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return c;
}

template <class T>
__global__ void __launch_bounds__(256) rar_dropout_rows(const DropoutParams p)
{
    const uint32_t groups = (uint32_t)((p.cols + 7) / 8);
    const uint64_t step = p.step ? (uint64_t)*p.step : 0;
    // the workgroup's run of groups: one 64-bit division for all of it
    const int64_t first = (int64_t)blockIdx.x * (256 * kPasses);
    const int64_t row0 = first / groups;
    const uint32_t in0 = (uint32_t)(first - row0 * groups);
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
        const uint32_t g = in0 + u * 256 + threadIdx.x;
        const uint32_t down = g / groups;
        const int64_t row = row0 + down, c = (int64_t)(g - down * groups) * 8;
        if (row >= p.rows)
            return;
        const int cnt = clamp8(p.cols - c);
        const uint64_t number = (uint64_t)first + u * 256 + threadIdx.x;
        float v[8], r[8];
        load8<true>((const T *)p.x + row * p.ldx + c, cnt, v);
        if (p.r)
            load8<true>((const T *)p.r + row * p.ldr + c, cnt, r);
        const u32x4 counter = {(uint32_t)number, (uint32_t)(number >> 32), (uint32_t)step, (uint32_t)(step >> 32)};
        const u32x4 w = philox(counter, p.seed_lo, p.seed_hi);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t draw = i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu;
            const float x = draw >= p.threshold ? v[i] : 0.0f;
            v[i] = p.r ? __builtin_fmaf(x, p.scale, r[i]) : x * p.scale;
        }
        store8<true>((T *)p.y + row * p.ldy + c, cnt, v);
    }
}

}  // namespace

hipError_t launch_dropout(rar_dtype dt, const DropoutParams &p, hipStream_t st)
{
    const int64_t groups = p.rows * ((p.cols + 7) / 8), per = 256 * kPasses;
    return launch(dt == RAR_BF16 ? rar_dropout_rows<bf16> : rar_dropout_rows<float>,
                  (unsigned)((groups + per - 1) / per), 256, st, p);
}

}  // namespace rar
