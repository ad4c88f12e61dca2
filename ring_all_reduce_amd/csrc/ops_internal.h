// ops_internal.h -- declarations shared by the host code (ops_host.cpp) and the
// kernels (linear.hip, embed.hip, ckpt.hip) of the gradient-producing operators
// of librar.so.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rar.h"

namespace rar {

constexpr int kCkptGroup = RAR_CKPT_GROUP;

// A kernel launch and its own status.  (After <<<>>> the status is HIP's last
// error, which an earlier call of the caller's may have left there: this call
// would take it for its own and end before its next launch.)
template <class T>
struct Same {
    typedef T type;
};

template <class... P>
hipError_t launch(void (*kernel)(P...), dim3 grid, unsigned lanes, hipStream_t st, typename Same<P>::type... a)
{
    void *args[] = {(void *)&a...};
    return hipLaunchKernel((const void *)kernel, grid, dim3(lanes), args, 0, st);
}

// One matrix product D[m][n] = sum_k A(m,k) B(n,k).  An operand is stored either
// with its reduction index contiguous (element (r,k) at r*ld + k) or with the
// reduction index slow (at k*ld + r):
//   forward  A = x [T][K] contiguous,  B = W [K][N] slow
//   grad x   A = dz [T][N] contiguous, B = W [K][N] contiguous
//   grad W   A = x [T][K] slow,        B = dz [T][N] slow
enum GemmMode {
    kModeStore = 0,    // out = D (+ out when accumulate)
    kModeForward = 1,  // z = D + bias; pre = z; out = act(z) + residual
    kModePartial = 2   // part[split] = D in binary32 (joined by launch_finish)
};

struct GemmParams {
    const void *a;
    const void *b;
    int64_t lda, ldb;        // elements
    int64_t M, N, K;         // K: the reduction
    void *out;
    int64_t ldo;
    void *pre;               // forward: z, or checkpoint codes with pre_scales, or nullptr
    int64_t ldp;
    uint8_t *pre_scales;
    const void *bias;        // or nullptr
    const void *res;         // or nullptr
    int64_t ldr;
    float *part;             // [splits][M][pitch]
    int64_t pitch;
    int mode;
    int act;
    int accumulate;
    int splits;
    int64_t steps_per_split; // K steps of one split
    int64_t tiles_m, tiles_n;
};

// Copy of a [rows][cols] matrix with leading dimension ld into one with pitch
// `pitch` whose columns [cols, pitch) are zero.
struct PackParams {
    const void *src;
    void *dst;
    int64_t ld, pitch, rows, cols;
};

// dz = dy * act'(z) and column sums of dz, for a [rows][cols] block.
struct DzParams {
    const void *dy;
    int64_t ldy;
    const void *pre;         // z in the plan's type, or checkpoint codes; nullptr when act is none
    int64_t ldp;
    const uint8_t *pre_scales;
    void *dz;                // nullptr: only the sums
    int64_t pitch;           // dz's row length; columns [cols, pitch) are set to zero
    float *part;             // [chunks][cols] partial column sums, or nullptr
    int64_t rows, cols;
    int64_t rows_per_chunk;
    int act;
};

struct SumParams {
    const float *part;
    int64_t chunks, cols;
    void *out;
    int accumulate;
};

struct CkptParams {
    const void *x;           // store: source; load: unused
    int64_t ldx;
    uint8_t *codes;
    uint8_t *scales;
    void *y;                 // load: destination
    int64_t ldy;
    int64_t pitch_zero;      // load: columns [cols, pitch_zero) of y are set to zero
    int64_t rows, cols;
    int act;
};

struct EmbedParams {
    const void *table;       // lookup
    const int64_t *ids;
    void *out;
    int64_t T, V, D, ldo;
    float scale;
};

struct EmbedGradParams {
    const int64_t *ids;
    const void *dy;
    int64_t ldy;
    void *grad;
    int64_t T, V, D;
    float scale;
    int accumulate;
    void *ws;
};

inline unsigned blocks_of(const GemmParams &p) { return (unsigned)(p.tiles_m * p.tiles_n * p.splits); }

hipError_t launch_forward(rar_dtype dt, const GemmParams &p, int tile, hipStream_t st);
// grad x in the first x_blocks workgroups, grad W in the w_blocks behind them.
struct GemmPair {
    GemmParams x, w;
    unsigned x_blocks;
};
hipError_t launch_backward(rar_dtype dt, const GemmPair &p, unsigned w_blocks, int tile, hipStream_t st);
// A forward product of at most kGemvRows rows; vec: rows of W are whole 16-byte groups.
constexpr int kGemvRows = 4;
hipError_t launch_gemv(rar_dtype dt, const GemmParams &p, bool vec, hipStream_t st);
hipError_t launch_pack(rar_dtype dt, const PackParams &a, const PackParams &b, hipStream_t st);
hipError_t launch_dz(rar_dtype dt, const DzParams &p, hipStream_t st);
// Joins of split products (a_blocks, b_blocks workgroups, 0: none) and column sums (sum.cols 0: none).
struct FinishParams {
    GemmParams a, b;
    unsigned a_blocks, b_blocks;
    SumParams sum;
};
inline unsigned join_blocks(const GemmParams &p)
{
    return p.splits > 1 ? (unsigned)((p.M * (p.pitch / 8) + 255) / 256) : 0;
}
hipError_t launch_finish(rar_dtype dt, const FinishParams &p, hipStream_t st);
hipError_t launch_ckpt_store(rar_dtype dt, const CkptParams &p, hipStream_t st);
hipError_t launch_ckpt_load(rar_dtype dt, const CkptParams &p, hipStream_t st);
hipError_t launch_embed_lookup(rar_dtype dt, const EmbedParams &p, hipStream_t st);
hipError_t launch_embed_grad(rar_dtype dt, const EmbedGradParams &p, hipStream_t st);
// Bytes of workspace rar_embed_grad needs.
int64_t embed_grad_workspace(int64_t T, int64_t V, int64_t D);
// Whether each of its launches has at most `lanes` lanes.
bool embed_grad_fits(int64_t T, int64_t D, int64_t grad_bytes, int64_t lanes);

}  // namespace rar
