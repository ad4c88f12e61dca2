// attn_shape.h -- how a call of cross attention is cut into workgroups: host
// arithmetic on sizes only, with no HIP in it.  Not part of the public ABI.
#pragma once

#include <algorithm>
#include <cstdint>

#include "sizes.h"

namespace rar {

constexpr int kAttnRows = 128;       // query rows of a workgroup, or keys of one of dk and dv
constexpr int kAttnFewRows = 32;     // rows of a key head that share one tile: the waves share out the keys
constexpr int kAttnTokenRows = 4;    // rows of a key head that the vector units take
constexpr int kAttnFewStage = 128;   // keys that such a call's split is a multiple of
constexpr int kAttnPad = 64;         // whole stages of queries

// Keys of a stage of the forward kernel for `rows` rows a key head.
inline int attn_stage(rar_dtype dt, int64_t rows)
{
    return rows <= kAttnFewRows ? kAttnFewStage : (dt == RAR_BF16 ? 64 : 32);
}

// Rows of a stage of the backward kernels.
inline int attn_backward_stage(rar_dtype dt) { return dt == RAR_BF16 ? 64 : 32; }

// Waves of a workgroup that share out the keys, by the bytes of a row in LDS: what fills LDS.
constexpr int attn_few_waves(int row_bytes) { return 512 / row_bytes; }

// A call's sizes and how its work is cut.
struct AttnShape {
    int64_t B, Tq, Tk, H, Hkv, share, dh, rows;
    rar_dtype dt;
    int64_t cols;      // a head's columns in whole 16-byte groups
    int width;         // of a row of partial results: whole 32 columns
    bool few;          // the keys are shared out among a workgroup's waves
    int64_t tiles;     // of query rows, a key head
    int64_t splits, stages;
    int64_t q_tiles, q_splits;    // of dq: rows, and parts of the keys
    int64_t key_tiles, k_splits;  // of dk and dv: keys, and parts of the queries
    int64_t padded;

    AttnShape(int64_t heads, int64_t key_heads, int64_t columns, rar_dtype dtype, int64_t B_, int64_t Tq_, int64_t Tk_)
        : B(B_), Tq(Tq_), Tk(Tk_), H(heads), Hkv(key_heads), share(heads / key_heads), dh(columns),
          rows(Tq_ * share), dt(dtype)
    {
        cols = up(dh, 16 / esize(dt));
        width = (int)up(dh, 32);
        few = rows <= kAttnFewRows;
        tiles = div_up(rows, few ? kAttnFewRows : kAttnRows);
        // two workgroups a compute unit, or one where a workgroup fills it or the caches' ports (few rows); each
        // with at least two stages of keys.  16 x 16 heads of 128, a token on 2048 keys in bf16: 44 us unsplit,
        // 45 in two parts and 41 in four, and the join 4 more.
        const int64_t all = std::max<int64_t>(1, div_up(Tk, attn_stage(dt, rows)));
        const int64_t work = std::max<int64_t>(1, B * Hkv * tiles);
        // Binary32 is bound by the matrix cores, which a second workgroup on some units would keep the call waiting
        // for: at most one a unit.  3 x 6 heads of 60 on 3, 333 queries on 517 keys: 22 us and a join of 6.6 to 19 and
        // 5.2; 4 x 8 heads of 128, 512 on 512: 55 and 12 to 49 and 11.
        if (!few && dt == RAR_F32)
            splits = parts(work, all);
        else
            splits = std::min<int64_t>(div_up(few ? 256 : 512, work), std::max<int64_t>(1, all / 2));
        splits = std::min<int64_t>(splits, 64);
        stages = div_up(all, splits);
        splits = div_up(all, stages);
        padded = up(Tq, kAttnPad);
        // The backward kernels fill a compute unit with one workgroup.  With fewer of them than units the long axis
        // of each is cut, into parts of at least two stages, and joined.
        q_tiles = div_up(rows, kAttnRows);
        key_tiles = div_up(Tk, kAttnRows);
        q_splits = parts(B * Hkv * q_tiles, div_up(Tk, attn_backward_stage(dt)));
        k_splits = parts(B * Hkv * key_tiles, div_up(Tq, attn_backward_stage(dt)) * share);
    }

    static int64_t parts(int64_t work, int64_t most)
    {
        return std::max<int64_t>(1, std::min<int64_t>(256 / std::max<int64_t>(1, work), most / 2));
    }

    // Rows of partial results that a call of at most these sizes may write, each at least what this one writes, and
    // none smaller for larger sizes: a workspace serves every smaller call.  (Fewer sequences are cut into more parts,
    // so a call's own rows fall where its parts become fewer.)  A call is cut where its whole stages allow two parts,
    // and then into fewer than twice as many workgroups as are aimed at: at most `groups`, of at most `tile` rows.
    static int64_t room(int64_t groups, int64_t tile, int64_t head_rows, int64_t heads, int64_t parts)
    {
        parts = std::min<int64_t>(parts, 256);
        return parts < 2 ? 0 : std::min(groups * std::min(tile, head_rows), heads * head_rows * parts);
    }
    int64_t part_room() const
    {
        const int64_t few_rows = std::min<int64_t>(rows, kAttnFewRows);
        const int64_t most = room(2 * 256, kAttnFewRows, few_rows, B * Hkv,
                                  std::min<int64_t>(64, div_up(Tk, kAttnFewStage) / 2));
        return few ? most
                   : std::max(most, room(dt == RAR_F32 ? 256 : 2 * 512, kAttnRows, rows, B * Hkv,
                                         std::min<int64_t>(64, div_up(Tk, attn_stage(dt, rows)) / 2)));
    }
    int64_t q_room() const
    {
        return room(256, kAttnRows, rows, B * Hkv, div_up(Tk, attn_backward_stage(dt)) / 2);
    }
    int64_t k_room() const
    {
        return room(256, kAttnRows, Tk, B * Hkv, div_up(Tq, attn_backward_stage(dt)) * share / 2);
    }

    // forward: few enough rows for the vector units, which read at any address
    bool token() const { return rows <= kAttnTokenRows; }
    int64_t blocks() const { return B * Hkv * splits * tiles; }
    int64_t part_rows() const { return B * H * Tq; }
    // every launch has at most 2^32 lanes
    bool fits() const
    {
        return blocks() <= kMaxLanes / 512 && B * Hkv * key_tiles * k_splits <= kMaxLanes / 256 &&
               B * Hkv * q_tiles * q_splits <= kMaxLanes / 256 &&
               div_up(B * H * padded, 32) <= kMaxLanes / 256;
    }
};

}  // namespace rar
