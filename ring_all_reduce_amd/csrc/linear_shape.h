// linear_shape.h -- tile and split of the linear layer's matrix products: host
// arithmetic on sizes only, with no HIP in it.  Not part of the public ABI.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "rar.h"

namespace rar {

constexpr int64_t kMaxLanes = (int64_t(1) << 32) - 1;  // of a grid, along x
constexpr int64_t kMaxOutputs = int64_t(1) << 37;      // elements of a layer's matrix

inline int esize(rar_dtype d) { return d == RAR_BF16 ? 2 : 4; }
inline int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
inline int64_t div_up(int64_t v, int64_t by) { return (v + by - 1) / by; }

// Workgroups of a launch: those of a 256-tile have 512 lanes, all others 256.
// kMaxOutputs in the larger tile take fewer, whatever the sides: at most
// 2^21 + 2^16 + 2^12 + 1 of 256 x 256 and 2^23 + 2^17 + 2^13 + 1 of 128 x 128.
inline int64_t most_blocks(rar_dtype dt, int tile) { return kMaxLanes / (dt == RAR_BF16 && tile == 256 ? 512 : 256); }

struct Shape {
    int tile;
    int64_t tiles_m, tiles_n, splits, steps;
    int64_t pitch;
    int64_t part_bytes;
};

// Microseconds of a product at a shape, from a sweep of tiles and splits on
// MI355X over 13 layers from 333 x 501 x 259 to 8192 x 2048 x 8192: the most
// loaded compute unit runs `rounds` workgroups, whose steps take `step` each
// when several share the unit and at least `alone` by themselves; a split
// reduction also writes its partial sums, reads them and launches the join.
// Both ends, bf16: 2048 x 4096 -> 4096 forward takes 62 us in 128-tiles and 94
// in 256-tiles (256 of them would leave half the chip idle), its weight
// gradient 66 and 54; binary32: 2048^3 takes 139 us in 128-tiles and 132 in
// 64-tiles, 8192 x 2048 -> 2048 500 and 510.  128 x 2048 -> 2048 in bf16 takes
// 15 us split in four and 23 unsplit; 2048 x 512 -> 512 10 unsplit, 15 in two.
// The epilogue is in the constant part only: where the reduction is short the
// estimate is low (10 us for 7178 x 177 -> 2023 in bf16, which takes 45).
inline double cost(rar_dtype dt, const Shape &s)
{
    double step, alone, fixed;
    if (dt == RAR_BF16) {
        step = s.tile == 256 ? 1.45 : 0.445;
        alone = s.tile == 256 ? 1.45 : 0.66;
        fixed = s.tile == 256 ? 8 : 5;
    } else {
        step = s.tile == 128 ? 1.9 : 0.495;
        alone = s.tile == 128 ? 2.12 : 0.72;
        fixed = s.tile == 128 ? 5 : 3;
    }
    const double rounds = std::ceil((double)(s.tiles_m * s.tiles_n * s.splits) / 256);
    const double t = std::max(rounds * step, alone) * (double)s.steps + fixed;
    return s.splits > 1 ? t + 4 + 0.35e-6 * (double)s.part_bytes : t;
}

inline Shape shape_of(rar_dtype dt, int64_t M, int64_t N, int64_t K)
{
    const int64_t total = std::max<int64_t>(1, div_up(K * esize(dt), 128));
    const int large = dt == RAR_BF16 ? 256 : 128;
    Shape best{};
    double least = 0;
    for (int tile = large; tile >= large / 2; tile /= 2) {
        Shape s{};
        s.tile = tile;
        s.tiles_m = div_up(M, tile);
        s.tiles_n = div_up(N, tile);
        s.pitch = up(N, RAR_CKPT_GROUP);
        const int64_t tiles = s.tiles_m * s.tiles_n;
        if (tiles > most_blocks(dt, tile))
            continue;
        for (int64_t want = 1; want <= 32 && (want == 1 || (total / want >= 2 && tiles * want <= 2048)); ++want) {
            s.steps = div_up(total, want);
            s.splits = div_up(total, s.steps);
            s.part_bytes = s.splits > 1 ? s.splits * M * s.pitch * 4 : 0;
            const double t = cost(dt, s);
            if (best.tile == 0 || t < least) {
                best = s;
                least = t;
            }
        }
    }
    return best;
}

}  // namespace rar
