// attn.hip -- CDNA4 (gfx950) kernels of cross attention, forward and backward.
//
//   S = scale q k^T over the keys that count, P = softmax(S), o = P v
//   lse = log sum e^S,  delta = sum do . o
//   dv = P^T do,  dP = do v^T,  dS = P (dP - delta),  dq = scale dS k,  dk = scale dS^T q
//
// All products are 32 x 32 tiles of the matrix cores whose reduction runs over 16
// (lane l holds row l % 32 and elements 8 (l / 32) .. +7; the result's lane holds
// column l % 32 and rows 8 (i / 4) + 4 (l / 32) + i % 4, i < 16).  The order of
// a reduction is free as long as both operands keep it.  So scores are taken
// transposed, one query (or, for dk and dv, one key) a lane: softmax runs along a
// lane's registers, and the weights are, as they stand, an operand of the next
// product, whose other operand is read from LDS in the same order of rows by
// transposing reads.  Neither scores nor weights pass through LDS or memory.
//
// bf16: the matrix instructions take both operands in bf16, so weights and score
// gradients are rounded to it once; scores, maxima, sums, lse, delta and
// accumulators stay in binary32.  Each of these roundings adds, independently over
// the terms, what the rounding of the result adds: o and the gradients are off by
// sqrt 2 times a rounding (0.0024 of their norm against 64 bits, where results in
// 64 bits rounded to bf16 are off by 0.0017).  Weights in two bf16 parts would end
// that at four products more beside the nine of a training step.
//
// Query heads that share a key head are rows of one tile: row r is query r /
// share of head r % share.
//
// Measured at 8 x 16 heads of 128 in bf16, 1152 to 2048 queries on 576 to 1024 keys
// (products of 42 GFLOP each): forward 115 to 127 us (two products, 680 TFLOP/s), delta
// 24 (4.4 TB/s), dq 156 to 173 (three, 770), dk and dv 211 to 238 (four, 750).  A large
// product of torch's reaches 1380 on that card.  Binary32, 4 x 8 heads of 128, 512 on 512:
// forward 49 us and a join of 11, dq 65, dk and dv 87 and a sum of 14.
#include <algorithm>

#include "ops_internal.h"
#include "row.h"

#pragma clang fp contract(off)

#define RAR_LDS __attribute__((address_space(3)))

namespace rar {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr uint32_t kOutOfRange = 0x80000000u;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kInf = __builtin_inff();
// How far a row's scores may pass the maximum that its weights are taken from
// before the accumulator is scaled again: weights stay under e^8.
constexpr float kSlack = 8.0f;

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------

template <class T> struct Frag;

template <> struct Frag<bf16> {
    bf16x8 v;
    __device__ __forceinline__ void zero() { v = bf16x8{}; }
    __device__ __forceinline__ void load(const bf16 *p) { v = *reinterpret_cast<const bf16x8 *>(p); }
    // eight consecutive results of a tile, rounded for the next product
    __device__ __forceinline__ void set(const f32x16 &s, int at)
    {
        const u32x4 w = {pack_bf16(s[at], s[at + 1]), pack_bf16(s[at + 2], s[at + 3]), pack_bf16(s[at + 4], s[at + 5]),
                         pack_bf16(s[at + 6], s[at + 7])};
        v = __builtin_bit_cast(bf16x8, w);
    }
};

template <> struct Frag<float> {
    f32x4 lo, hi;
    __device__ __forceinline__ void zero() { lo = hi = f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }
    __device__ __forceinline__ void load(const float *p)
    {
        lo = *reinterpret_cast<const f32x4 *>(p);
        hi = *reinterpret_cast<const f32x4 *>(p + 4);
    }
    __device__ __forceinline__ void set(const f32x16 &s, int at)
    {
        lo = f32x4{s[at], s[at + 1], s[at + 2], s[at + 3]};
        hi = f32x4{s[at + 4], s[at + 5], s[at + 6], s[at + 7]};
    }
};

__device__ __forceinline__ void mma(f32x16 &c, const Frag<bf16> &a, const Frag<bf16> &b)
{
#if defined(__HIP_DEVICE_COMPILE__)
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, c, 0, 0, 0);
#endif
}

__device__ __forceinline__ void mma(f32x16 &c, const Frag<float> &a, const Frag<float> &b)
{
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.lo[j], b.lo[j], c, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.hi[j], b.hi[j], c, 0, 0, 0);
#endif
}

__device__ __forceinline__ f32x16 zeros()
{
    f32x16 v;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = 0.0f;
    return v;
}

// Row of a result's register i, without the lane's 4 (l / 32).
__device__ __forceinline__ constexpr int row_of(int i) { return 8 * (i / 4) + i % 4; }

// ---------------------------------------------------------------------------
// Tiles in LDS
// ---------------------------------------------------------------------------
//
// A tile holds rows of PITCH elements.  The 16-byte chunk c of row r lies at slot
// c ^ spread(r), so that both reads below touch every bank once in 256 bytes: one
// chunk of 16 rows (an operand whose rows are the tile's), and, of bf16, four
// chunks of four rows (an operand whose reduction runs over the tile's rows, by
// the transposing read) or, of binary32, 128 bytes of two rows that lie four apart.
template <class T, int PITCH>
struct Tile {
    static constexpr int ES = sizeof(T);
    static constexpr int kBytes = PITCH * ES;   // of a row
    static constexpr int kChunks = kBytes / 16;

    static __device__ __forceinline__ int spread(int r)
    {
        if (ES == 4)
            return ((r >> 2) & 1) << 3 | (r & 3) << 1 | ((r >> 3) & 1);
        if (kBytes == 256)
            return (r & 3) << 2 | ((r >> 2) & 3);
        return ((r >> 1) & 1) << 2 | ((r >> 2) & 3);  // two rows in 256 bytes
    }

    // Rows r0 + l % 32 (r0 a multiple of 32), elements 16 s + 8 (l / 32) ..
    static __device__ __forceinline__ Frag<T> rows(const RAR_LDS char *__restrict__ lds, int r0, int s)
    {
        const int lane = threadIdx.x & 63, r = lane & 31, half = lane >> 5;
        const RAR_LDS char *const at = lds + (r0 + r) * kBytes;
        Frag<T> f;
        if constexpr (ES == 2) {
            f.v = *(const RAR_LDS bf16x8 *)(at + (((2 * s + half) ^ spread(r)) << 4));
        } else {
            f.lo = *(const RAR_LDS f32x4 *)(at + (((4 * s + 2 * half) ^ spread(r)) << 4));
            f.hi = *(const RAR_LDS f32x4 *)(at + (((4 * s + 2 * half + 1) ^ spread(r)) << 4));
        }
        return f;
    }

    // Column 32 d + l % 32 of the rows that registers 8 j .. 8 j + 7 of a result
    // stand for, in a tile of 32 rows that starts at r0.
    static __device__ __forceinline__ Frag<T> cols(const RAR_LDS char *__restrict__ lds, int r0, int j, int d)
    {
        const int lane = threadIdx.x & 63, half = lane >> 5;
        Frag<T> f;
        if constexpr (ES == 2) {
            i16x4 w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 16 * j + 8 * e + 4 * half + ((lane & 15) >> 2);
                const int c = 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
                const RAR_LDS char *const at =
                    lds + (r0 + r) * kBytes + ((c ^ spread(r)) << 4) + ((lane & 1) << 3);
                w[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((RAR_LDS i16x4 *)at);
            }
            f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(w[0], w[1], 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int r = 16 * j + 8 * (e / 4) + 4 * half + e % 4;
                const int c = 8 * d + ((lane & 31) >> 2);
                const float v =
                    *(const RAR_LDS float *)(lds + (r0 + r) * kBytes + ((c ^ spread(r)) << 4) + ((lane & 3) << 2));
                if (e < 4)
                    f.lo[e & 3] = v;
                else
                    f.hi[e & 3] = v;
            }
        }
        return f;
    }
};

// Memory -> LDS, 16 bytes a lane, without passing through registers.  The
// destination is linear in the lane, so the spread is applied to the address
// that each lane reads.  The descriptor ends with the last row that counts: rows
// behind it, and chunks behind the head's columns, read as zero.
// With WAVES = 1 a wave loads a tile of its own.
template <class T, int PITCH, int ROWS, int WAVES>
struct Loader {
    typedef Tile<T, PITCH> Lds;
    static constexpr int kLoads = ROWS * Lds::kBytes / (WAVES * 1024);
    static_assert(kLoads * WAVES * 1024 == ROWS * Lds::kBytes, "whole loads");
    uint32_t voff[kLoads], in_row;
    const char *base;
    int64_t pitch, width;  // bytes of a row in memory, and of a head
    int64_t left;          // rows from base that count

    __device__ __forceinline__ void init(const AttnOperand &m, int64_t row, int64_t head, int64_t rows)
    {
        const int wave = WAVES > 1 ? threadIdx.x >> 6 : 0, lane = threadIdx.x & 63;
        base = (const char *)m.p + (row * m.ld + head * m.hs) * Lds::ES;
        pitch = m.ld * Lds::ES;
        width = m.cols * Lds::ES;
        left = rows;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int at = (j * WAVES + wave) * 1024 + lane * 16;
            const int r = at / Lds::kBytes, c = ((at % Lds::kBytes) / 16) ^ Lds::spread(r);
            voff[j] = c * 16 < width ? (uint32_t)(r * pitch) + c * 16 : kOutOfRange;
            if (j == 0)
                in_row = c * 16 < width ? c * 16 : kOutOfRange;
        }
    }

    // LAST: the last row that counts stands in place of those behind it (left > 0).
    template <bool LAST = false>
    __device__ __forceinline__ void load(RAR_LDS char *__restrict__ lds)
    {
        static_assert(!LAST || WAVES * 1024 / Lds::kBytes % 16 == 0, "a lane's chunk is the same in all of its rows");
#if defined(__HIP_DEVICE_COMPILE__)
        const int wave = WAVES > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
        int64_t n = left > 0 ? (left - 1) * pitch + width : 0;
        if (n > 0x7fffffff)
            n = 0x7fffffff;
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, (int)n, 0x00020000);
        const uint32_t last = (uint32_t)(n - width) + in_row;
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (RAR_LDS void *)(lds + (j * WAVES + wave) * 1024), 16,
                                                     LAST ? std::min(voff[j], last) : voff[j], 0, 0, 0);
#endif
    }

    __device__ __forceinline__ void advance(int rows = ROWS)
    {
        base += rows * pitch;
        left -= rows;
    }
};

// A half of LDS, as a constant: addresses in it are then parts of the instructions.
template <int N>
struct Half {
    __device__ constexpr int operator()() const { return N; }
};

// Nothing moves across: what stands before is issued before what stands behind.
__device__ __forceinline__ void schedule_fence()
{
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_sched_barrier(0);
#endif
}

// Own loads into LDS and own LDS reads are done; then everyone's.  (By the builtin:
// of a wait in assembly the compiler knows nothing, and it would wait again, in the
// loop, for the loads before it.)
__device__ __forceinline__ void meet()
{
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#endif
}

// Workgroups go to the eight XCDs in turn.  The work of one sequence and key head
// goes to one XCD, whose L2 then holds the keys (or queries) that it shares, and
// neighbouring heads to different ones: sequences of different lengths weigh on
// all XCDs alike.  (Runs of whole sequences left the XCD of the longest one
// working alone.)  From one eight to the next the heads move on by an XCD: a head's
// keys lie a row of all heads apart, and the same heads on an XCD would use few of
// its L2's channels.  What is left behind the last eight heads is spread out.
struct Place {
    int64_t b, hk, in;  // in: which of the head's workgroups
};

__device__ __forceinline__ Place place_of(int64_t heads, int64_t Hkv, int64_t each)
{
    const int64_t id = blockIdx.x, whole = heads / 8 * 8;
    int64_t head, in;
    if (id < whole * each) {
        const int64_t j = id / 8;
        head = j / each * 8 + (id + j / each) % 8;
        in = j % each;
    } else {
        const int64_t j = id - whole * each;
        head = whole + j / each;
        in = j % each;
    }
    return Place{head / Hkv, head % Hkv, in};
}

__device__ __forceinline__ int64_t length_of(const int64_t *lens, int64_t b, int64_t most)
{
    if (!lens)
        return most;
    const int64_t n = lens[b];
    return n < 0 ? 0 : (n > most ? most : n);
}

// Four consecutive columns of a row, of which those before `cols` exist.
template <class T>
__device__ __forceinline__ void put4(T *row, int c, int cols, f32x4 v)
{
    if (c + 4 <= cols) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<f32x4_any *>(row + c) = v;
        } else {
            typedef u32x2 u32x2_any __attribute__((aligned(2)));
            *reinterpret_cast<u32x2_any *>(row + c) = u32x2{pack_bf16(v.x, v.y), pack_bf16(v.z, v.w)};
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (c + i < cols)
            row[c + i] = from_f32<T>(v[i]);
}

// e^(scale s - shift).  bf16 takes scale and shift times log2 e and rounds the
// exponent once; binary32 subtracts first, so that the weights near one, which
// carry the result, keep their digits.
template <class T>
constexpr float kUnit = sizeof(T) == 2 ? kLog2e : 1.0f;

template <class T>
__device__ __forceinline__ float weight(float s, float scale, float shift)
{
    const float x = __builtin_fmaf(s, scale, -shift);
    return __builtin_amdgcn_exp2f(sizeof(T) == 2 ? x : x * kLog2e);
}

template <class T, int W>
struct Shape {
    static constexpr int PITCH = W <= 2 ? 64 : 128;
    static constexpr int STEPS = 2 * W;  // reductions of 16 over a head's columns
    typedef Tile<T, PITCH> Lds;
};

// The fragments of one row of a matrix: row `row`, elements 16 s + 8 half ..
template <class T, int N>
__device__ __forceinline__ void load_row(Frag<T> (&f)[N], const AttnOperand &m, int64_t row, int64_t head, bool live)
{
    const int half = (threadIdx.x & 63) >> 5;
    const T *const p = (const T *)m.p + row * m.ld + head * m.hs;
#pragma unroll
    for (int s = 0; s < N; ++s) {
        const int c = 16 * s + 8 * half;
        if (live && c + 8 <= m.cols) {
            f[s].load(p + c);
        } else if (live && c < m.cols) {  // binary32: the columns are whole fours
            f[s].zero();
            if constexpr (sizeof(T) == 4)
                f[s].lo = *reinterpret_cast<const f32x4 *>(p + c);
        } else {
            f[s].zero();
        }
    }
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
//
// A wave holds 32 query rows, a row a lane and its other half; running maximum,
// sum and accumulator stay there.
template <class T, int W>
struct Rows {
    f32x16 acc[W];
    float m, l;

    __device__ __forceinline__ void init()
    {
#pragma unroll
        for (int d = 0; d < W; ++d)
            acc[d] = zeros();
        m = -kInf;
        l = 0.0f;
    }

    // Scores of TILES * 32 keys, of which `rest` count, become weights.  The
    // accumulator is scaled only where some row's scores have passed its maximum
    // by kSlack: with 32 rows to a wave, some row's maximum grows in almost every
    // step.
    template <int TILES>
    __device__ __forceinline__ void weigh(f32x16 (&s)[TILES], int rest, float scale)
    {
        const int half = (threadIdx.x & 63) >> 5;
        if (rest < TILES * 32)
#pragma unroll
            for (int e = 0; e < TILES; ++e)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (e * 32 + row_of(i) + 4 * half >= rest)
                        s[e][i] = -kInf;
        float top = s[0][0];
#pragma unroll
        for (int e = 0; e < TILES; ++e)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                top = __builtin_fmaxf(top, s[e][i]);
        top = __builtin_fmaxf(top, __shfl_xor(top, 32)) * scale;
        if (__any(top > m + kSlack || (m == -kInf && top > m))) {
            top = __builtin_fmaxf(top, m);
            const float down = __builtin_amdgcn_exp2f((m - (top == -kInf ? 0.0f : top)) * kLog2e);
            l *= down;
#pragma unroll
            for (int d = 0; d < W; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[d][i] *= down;
            m = top;
        }
    }

    // Of one tile, with the sum; to be called after weigh().
    __device__ __forceinline__ void exponentials(f32x16 &s, float scale)
    {
        const float base = m == -kInf ? 0.0f : m * kUnit<T>;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[i] = weight<T>(s[i], scale * kUnit<T>, base);
            l += s[i];
        }
    }

    // Both halves' sums.
    __device__ __forceinline__ void close() { l += __shfl_xor(l, 32); }
};

// Which row a lane holds, and where its results go.
struct RowPlace {
    int64_t row, t, h;
    bool live;
};

__device__ __forceinline__ RowPlace row_place(const AttnParams &p, int64_t hk, int64_t row, int64_t qlen)
{
    const int64_t t = row / p.share;
    return RowPlace{row, t, hk * p.share + row % p.share, row < p.Tq * p.share && t < qlen};
}

// Many rows: the four waves of a workgroup take different rows and share the
// staged keys, two stages in turn.  In bf16 the exponentials (a quarter of the other
// instructions' rate) cost what the products do, so two waves a SIMD run one beside
// the other: of the units' busy cycles the matrix cores take 36%, the vector units
// 41%.  Binary32 is bound by its matrix instruction, at a sixteenth of bf16's rate.
template <class T, int W>
struct Forward {
    typedef Shape<T, W> S;
    typedef typename S::Lds Lds;
    static constexpr int kTiles = sizeof(T) == 2 ? 2 : 1;   // of 32 keys, a stage
    static constexpr int kStage = kTiles * 32;
    static constexpr int kHalf = kStage * Lds::kBytes;      // bytes of a stage's keys
};

template <class T, int W>
__global__ void __launch_bounds__(256, sizeof(T) == 4 && W > 2 ? 1 : 2) rar_attn_rows(const AttnParams p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    typedef Forward<T, W> F;
    typedef typename F::Lds Lds;
    constexpr int STEPS = F::S::STEPS;
    __shared__ __attribute__((aligned(1024))) char memory[4 * F::kHalf];
    RAR_LDS char *const lds = (RAR_LDS char *)memory;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, half = lane >> 5;

    const Place at = place_of(p.B * p.Hkv, p.Hkv, p.tiles * p.splits);
    const int64_t tile = at.in % p.tiles, hk = at.hk, b = at.b;
    const int split = (int)(at.in / p.tiles);
    const int64_t klen = length_of(p.klen, b, p.Tk), qlen = length_of(p.qlen, b, p.Tq);
    const int64_t rows = p.Tq * p.share, first = tile * kAttnRows;
    const RowPlace r = row_place(p, hk, first + wave * 32 + (lane & 31), qlen);
    Frag<T> q[STEPS];
    load_row<T>(q, p.q, b * p.Tq + r.t, r.h, r.live);

    // this workgroup's keys: whole stages
    const int64_t k0 = (int64_t)split * p.stages * F::kStage;
    int64_t kend = k0 + (int64_t)p.stages * F::kStage;
    kend = kend < klen ? kend : klen;
    const int stages = first / p.share < qlen && k0 < kend ? (int)((kend - k0 + F::kStage - 1) / F::kStage) : 0;

    Loader<T, F::S::PITCH, F::kStage, 4> lk, lv;
    lk.init(p.k, b * p.Tk + k0, hk, kend - k0);
    lv.init(p.v, b * p.Tk + k0, hk, kend - k0);
    Rows<T, W> own;
    own.init();

    if (stages) {
        lk.load(lds);
        lv.load(lds + F::kHalf);
    }
    meet();
    // One stage, in the half of LDS that BUF names.
    auto stage = [&](auto BUF, int n) __attribute__((always_inline)) {
        RAR_LDS char *const here = lds + BUF() * 2 * F::kHalf;
        RAR_LDS char *const next = lds + (2 - BUF() * 2) * F::kHalf;
        if (n + 1 < stages) {
            lk.advance();
            lv.advance();
            lk.load(next);
            lv.load(next + F::kHalf);
        }
        // a tile's fragments are on their way before its first product, the next tile's follow in their place
        Frag<T> k[STEPS], v[2][W];
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
            k[i] = Lds::rows(here, 0, i);
        schedule_fence();
        f32x16 s[F::kTiles];
#pragma unroll
        for (int e = 0; e < F::kTiles; ++e) {
            s[e] = zeros();
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                mma(s[e], k[i], q[i]);
                if (e + 1 < F::kTiles)
                    k[i] = Lds::rows(here, e * 32 + 32, i);
            }
        }
        auto values = [&](int e) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int d = 0; d < W; ++d)
                    v[j][d] = Lds::cols(here + F::kHalf, e * 32, j, d);
        };
        values(0);
        schedule_fence();
        own.weigh(s, (int)(kend - k0 - (int64_t)n * F::kStage), p.scale);
#pragma unroll
        for (int e = 0; e < F::kTiles; ++e) {
            own.exponentials(s[e], p.scale);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                Frag<T> w;
                w.set(s[e], 8 * j);
#pragma unroll
                for (int d = 0; d < W; ++d)
                    mma(own.acc[d], v[j][d], w);
            }
            if (e + 1 < F::kTiles)
                values(e + 1);
        }
        meet();
    };
    for (int n = 0; n < stages; n += 2) {
        stage(Half<0>{}, n);
        if (n + 1 < stages)
            stage(Half<1>{}, n + 1);
    }
    own.close();

    if (r.row >= rows)
        return;
    const float inv = p.splits > 1 ? 1.0f : (own.l == 0.0f || !r.live ? 0.0f : 1.0f / own.l);
    const int64_t place = split * p.part_rows + (b * p.Hkv + hk) * rows + r.row;
#pragma unroll
    for (int d = 0; d < W; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x4 v;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                v[x] = r.live ? own.acc[d][4 * i + x] * inv : 0.0f;
            const int c = d * 32 + 8 * i + 4 * half;
            if (p.splits > 1)
                store4(p.part + place * (W * 32) + c, v);
            else
                put4((T *)p.o + (b * p.Tq + r.t) * p.ldo + r.h * p.dh, c, p.dh, v);
        }
    if (half)
        return;
    if (p.splits > 1) {
        p.stats[place * 2] = own.m;
        p.stats[place * 2 + 1] = own.l;
    } else if (p.lse) {
        p.lse[(b * p.Tq + r.t) * p.H + r.h] = r.live && own.l != 0.0f ? own.m + logf(own.l) : -kInf;
    }
#endif
}

// Few rows: every wave of a workgroup takes the same rows and keys of its own, 32
// at a time, through a ring of LDS tiles that it fills itself, so that no wave
// waits for another.  Bound by reading the keys: what counts is how much is in
// flight, all of LDS but the tiles in use.  The waves are joined through LDS at
// the end.  16 x 16 heads of 128, eight queries on 1024 to 2048 keys in bf16: 48 us
// (201 MB, 4.1 TB/s); in binary32, where LDS holds the ring of one wave only, 310
// (403 MB, 1.3 TB/s).
template <class T, int W>
struct Few {
    typedef Shape<T, W> S;
    typedef typename S::Lds Lds;
    static constexpr int kHalf = 32 * Lds::kBytes;               // bytes of a tile's keys
    static constexpr int kWaves = attn_few_waves(Lds::kBytes);
    static constexpr int kRing = kWaves > 1 ? 5 : 3;
    typedef Loader<T, S::PITCH, 32, 1> Load;
    static constexpr int kBehind = (kRing - 2) * 2 * Load::kLoads;  // loads that may be in flight behind a tile
    static_assert(kBehind < 64, "the counter of loads has six bits");
    static constexpr int kJoinPitch = W * 32 * 4 + 16;           // bytes of a row in the join
    static constexpr int kJoin = kWaves * 32 * (kJoinPitch + 8);
    static constexpr int kTiles = kWaves * kRing * 2 * kHalf;
    static constexpr int kLds = kTiles > kJoin ? kTiles : kJoin;
};

template <class T, int W>
__global__ void __launch_bounds__(64 * attn_few_waves((W <= 2 ? 64 : 128) * sizeof(T))) rar_attn_few(const AttnParams p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    typedef Few<T, W> F;
    typedef typename F::Lds Lds;
    constexpr int STEPS = F::S::STEPS, kStep = F::kWaves * 32;
    __shared__ __attribute__((aligned(1024))) char memory[F::kLds];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, half = lane >> 5;
    RAR_LDS char *const lds = (RAR_LDS char *)memory, *const ring = lds + wave * (F::kRing * 2 * F::kHalf);

    const Place at = place_of(p.B * p.Hkv, p.Hkv, p.splits);
    const int64_t hk = at.hk, b = at.b;
    const int split = (int)at.in;
    const int64_t klen = length_of(p.klen, b, p.Tk), qlen = length_of(p.qlen, b, p.Tq);
    const int64_t rows = p.Tq * p.share;
    const RowPlace own_row = row_place(p, hk, lane & 31, qlen);
    Frag<T> q[STEPS];
    load_row<T>(q, p.q, b * p.Tq + own_row.t, own_row.h, own_row.live);

    const int64_t k0 = (int64_t)split * p.stages * kAttnFewStage + wave * 32;
    int64_t kend = (int64_t)(split + 1) * p.stages * kAttnFewStage;
    kend = kend < klen ? kend : klen;
    const int tiles = qlen > 0 && k0 < kend ? (int)((kend - k0 + kStep - 1) / kStep) : 0;
    typename F::Load lk, lv;
    lk.init(p.k, b * p.Tk + k0, hk, kend - k0);
    lv.init(p.v, b * p.Tk + k0, hk, kend - k0);
    auto load = [&](int slot) __attribute__((always_inline)) {
        lk.load(ring + slot * 2 * F::kHalf);
        lv.load(ring + slot * 2 * F::kHalf + F::kHalf);
        lk.advance(kStep);
        lv.advance(kStep);
    };
    Rows<T, W> own;
    own.init();
    for (int n = 0; n < F::kRing - 1 && n < tiles; ++n)
        load(n);
    int slot = 0, fill = F::kRing - 1;
    for (int n = 0; n < tiles; ++n) {
        // this tile has arrived, and the reads of the tile before it, whose slot is filled next, are done
        asm volatile("" ::: "memory");
        if (n + F::kRing - 2 < tiles)
            __builtin_amdgcn_s_waitcnt((F::kBehind & 15) | (F::kBehind >> 4) << 14 | 7 << 4);
        else
            __builtin_amdgcn_s_waitcnt(0);
        asm volatile("" ::: "memory");
        if (n + F::kRing - 1 < tiles)
            load(fill);
        RAR_LDS char *const here = ring + slot * 2 * F::kHalf;
        Frag<T> k[STEPS], v[2][W];
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
            k[i] = Lds::rows(here, 0, i);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int d = 0; d < W; ++d)
                v[j][d] = Lds::cols(here + F::kHalf, 0, j, d);
        f32x16 s[1] = {zeros()};
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
            mma(s[0], k[i], q[i]);
        own.weigh(s, (int)(kend - k0 - (int64_t)n * kStep), p.scale);
        own.exponentials(s[0], p.scale);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            Frag<T> w;
            w.set(s[0], 8 * j);
#pragma unroll
            for (int d = 0; d < W; ++d)
                mma(own.acc[d], v[j][d], w);
        }
        slot = slot + 1 == F::kRing ? 0 : slot + 1;
        fill = fill + 1 == F::kRing ? 0 : fill + 1;
    }
    own.close();

    meet();  // the rings are free
    RAR_LDS float *const mine = (RAR_LDS float *)(lds + (wave * 32 + (lane & 31)) * F::kJoinPitch);
    RAR_LDS float *const stats = (RAR_LDS float *)(lds + F::kWaves * 32 * F::kJoinPitch);  // [wave][32][m, l]
    if (half == 0) {
        stats[(wave * 32 + lane) * 2] = own.m;
        stats[(wave * 32 + lane) * 2 + 1] = own.l;
    }
#pragma unroll
    for (int d = 0; d < W; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *(RAR_LDS f32x4 *)(mine + d * 32 + 8 * i + 4 * half) = f32x4{
                own.acc[d][4 * i], own.acc[d][4 * i + 1], own.acc[d][4 * i + 2], own.acc[d][4 * i + 3]};
    meet();
    // eight lanes a row, W quads of columns a lane
    for (int i = threadIdx.x >> 3; i < rows; i += F::kWaves * 8) {
        const RowPlace r = row_place(p, hk, i, qlen);
        float top = -kInf, sum = 0.0f, w[F::kWaves];
#pragma unroll
        for (int x = 0; x < F::kWaves; ++x)
            top = __builtin_fmaxf(top, stats[(x * 32 + i) * 2]);
#pragma unroll
        for (int x = 0; x < F::kWaves; ++x) {
            const float m = stats[(x * 32 + i) * 2], l = stats[(x * 32 + i) * 2 + 1];
            // (no key of this wave's counts, or all of their scores are -infinity)
            w[x] = l == 0.0f ? 0.0f : __builtin_amdgcn_exp2f((m - (top == -kInf ? 0.0f : top)) * kLog2e);
            sum = __builtin_fmaf(w[x], l, sum);
        }
        const float inv = p.splits > 1 ? 1.0f : (sum == 0.0f ? 0.0f : 1.0f / sum);
        const int64_t place = split * p.part_rows + (b * p.Hkv + hk) * rows + i;
#pragma unroll
        for (int e = 0; e < W; ++e) {
            const int c = ((threadIdx.x & 7) + e * 8) * 4;
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int x = 0; x < F::kWaves; ++x) {
                const f32x4 a = *(RAR_LDS f32x4 *)((RAR_LDS float *)(lds + (x * 32 + i) * F::kJoinPitch) + c);
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    v[y] = w[x] == 0.0f ? v[y] : __builtin_fmaf(w[x], a[y], v[y]);
            }
#pragma unroll
            for (int y = 0; y < 4; ++y)
                v[y] = r.live ? v[y] * inv : 0.0f;
            if (p.splits > 1)
                store4(p.part + place * (W * 32) + c, v);
            else
                put4((T *)p.o + (b * p.Tq + r.t) * p.ldo + r.h * p.dh, c, p.dh, v);
        }
        if ((threadIdx.x & 7) == 0) {
            if (p.splits > 1) {
                p.stats[place * 2] = top;
                p.stats[place * 2 + 1] = sum;
            } else if (p.lse) {
                p.lse[(b * p.Tq + r.t) * p.H + r.h] = r.live && sum != 0.0f ? top + logf(sum) : -kInf;
            }
        }
    }
#endif
}

// ---------------------------------------------------------------------------
// Forward, a token at a time
// ---------------------------------------------------------------------------
//
// Up to four rows a key head (a decoding step): a tile of the matrix cores would
// be mostly padding, and its long chain of reads and products keeps a wave from
// its next loads.  The vector units do it in two passes over registers: the lanes
// of a wave hold 16 bytes each of several keys, a key's lanes add up its products
// by lane exchanges, and the same lanes then weigh their 16 bytes of its value.
// The eight waves of a workgroup take keys in turn and are joined through LDS.
// Loads go straight to registers at any address, so no cache is copied.  Scores
// and their maximum are in units of log 2.  Bound by HBM: 16 x 16 heads of 128 on
// 1024 to 2048 keys in bf16, 201 MB, 44 us (4.6 TB/s; 5.4 at four times the batch);
// in binary32, 403 MB, 74 us (5.4 TB/s).
template <class T>
struct Piece {
    static constexpr int N = 16 / sizeof(T);
    u32x4 w;
    __device__ __forceinline__ void load(const T *p, int cnt)
    {
        if (cnt >= N) {
            w = *reinterpret_cast<const u32x4_any *>(p);
            return;
        }
        w = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < cnt) {
                if constexpr (sizeof(T) == 4)
                    w[i] = __float_as_uint(p[i]);
                else
                    w[i >> 1] |= (uint32_t)p[i].u << (i & 1 ? 16 : 0);
            }
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[i]);
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
};

// The sum over a group of L neighbouring lanes, in all of them.
template <int L>
__device__ __forceinline__ float group_sum(float v)
{
    v += dpp<0xB1, 0xf>(v, 0.0f);   // the neighbour, the neighbouring pair,
    v += dpp<0x4E, 0xf>(v, 0.0f);
    v += dpp<0x141, 0xf>(v, 0.0f);  // the other four of eight,
    if (L >= 16)
        v += dpp<0x140, 0xf>(v, 0.0f);  // the other eight of sixteen
    if (L >= 32)
        v += __shfl_xor(v, 16);
    return v;
}

constexpr int kTokenWaves = 8;

template <class T, int PITCH, int R>
__global__ void __launch_bounds__(64 * kTokenWaves) rar_attn_token(const AttnParams p)
{
    constexpr int N = Piece<T>::N, L = PITCH / N, G = 64 / L;  // lanes of a key, keys of a wave at a time
    constexpr int U = R > 2 ? 2 : 4;                           // keys a group takes in one step
    constexpr float kSlack2 = kSlack * kLog2e;
    __shared__ float joined[kTokenWaves][R][PITCH + 2];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, group = lane / L, c = lane % L * N;

    const Place at = place_of(p.B * p.Hkv, p.Hkv, p.splits);
    const int64_t hk = at.hk, b = at.b;
    const int split = (int)at.in;
    const int64_t klen = length_of(p.klen, b, p.Tk), qlen = length_of(p.qlen, b, p.Tq);
    const int rows = (int)(p.Tq * p.share), cnt = p.dh - c;
    float q[R][N], acc[R][N], m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const RowPlace place = row_place(p, hk, r, qlen);
        Piece<T> w;
        w.load((const T *)p.q.p + (b * p.Tq + place.t) * p.q.ld + place.h * p.q.hs + c, place.live ? cnt : 0);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            q[r][i] = w.get(i) * (p.scale * kLog2e);
            acc[r][i] = 0.0f;
        }
        m[r] = -kInf;
        l[r] = 0.0f;
    }
    const int64_t k0 = (int64_t)split * p.stages * kAttnFewStage;
    int64_t kend = k0 + (int64_t)p.stages * kAttnFewStage;
    kend = kend < klen ? kend : klen;
    const T *const keys = (const T *)p.k.p + (b * p.Tk + k0) * p.k.ld + hk * p.k.hs + c;
    const T *const values = (const T *)p.v.p + (b * p.Tk + k0) * p.v.ld + hk * p.v.hs + c;
    const int64_t count = qlen > 0 ? kend - k0 : 0;
    for (int64_t first = wave * (G * U); first < count; first += kTokenWaves * G * U) {
        Piece<T> k[U], v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t key = first + u * G + group;
            k[u].load(keys + key * p.k.ld, key < count ? cnt : 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t key = first + u * G + group;
            v[u].load(values + key * p.v.ld, key < count ? cnt : 0);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float s[U], top = m[r];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float t = 0.0f;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    t = __builtin_fmaf(q[r][i], k[u].get(i), t);
                t = group_sum<L>(t);
                s[u] = first + u * G + group < count ? t : -kInf;
                top = __builtin_fmaxf(top, s[u]);
            }
            if (__any(top > m[r] + kSlack2 || (m[r] == -kInf && top > m[r]))) {
                const float down = __builtin_amdgcn_exp2f(m[r] - (top == -kInf ? 0.0f : top));
                l[r] *= down;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    acc[r][i] *= down;
                m[r] = top;
            }
            const float base = m[r] == -kInf ? 0.0f : m[r];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float w = __builtin_amdgcn_exp2f(s[u] - base);
                l[r] += w;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    acc[r][i] = __builtin_fmaf(w, v[u].get(i), acc[r][i]);
            }
        }
    }
    // the groups of a wave, then the waves
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float top = m[r];
#pragma unroll
        for (int d = L; d < 64; d *= 2)
            top = __builtin_fmaxf(top, __shfl_xor(top, d));
        const float w = l[r] == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m[r] - (top == -kInf ? 0.0f : top));
        l[r] *= w;
#pragma unroll
        for (int i = 0; i < N; ++i)
            acc[r][i] = w == 0.0f ? 0.0f : acc[r][i] * w;
#pragma unroll
        for (int d = L; d < 64; d *= 2) {
            l[r] += __shfl_xor(l[r], d);
#pragma unroll
            for (int i = 0; i < N; ++i)
                acc[r][i] += __shfl_xor(acc[r][i], d);
        }
        if (lane < L) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                joined[wave][r][c + i] = acc[r][i];
            if (lane == 0) {
                joined[wave][r][PITCH] = top;
                joined[wave][r][PITCH + 1] = l[r];
            }
        }
    }
    __syncthreads();
    const int r = threadIdx.x / PITCH, col = threadIdx.x % PITCH;
    if (r >= rows)
        return;
    float top = -kInf, sum = 0.0f, o = 0.0f;
#pragma unroll
    for (int w = 0; w < kTokenWaves; ++w)
        top = __builtin_fmaxf(top, joined[w][r][PITCH]);
#pragma unroll
    for (int w = 0; w < kTokenWaves; ++w) {
        const float lw = joined[w][r][PITCH + 1];
        if (lw == 0.0f)
            continue;  // no key of this wave's counts
        const float x = __builtin_amdgcn_exp2f(joined[w][r][PITCH] - (top == -kInf ? 0.0f : top));
        sum = __builtin_fmaf(x, lw, sum);
        o = __builtin_fmaf(x, joined[w][r][col], o);
    }
    const RowPlace place = row_place(p, hk, r, qlen);
    if (p.splits > 1) {
        const int64_t part = split * p.part_rows + (b * p.Hkv + hk) * rows + r;
        if (col < p.pitch)
            p.part[part * p.pitch + col] = o;
        if (col == 0) {
            p.stats[part * 2] = top * kLn2;
            p.stats[part * 2 + 1] = sum;
        }
        return;
    }
    if (col < p.dh)
        ((T *)p.o)[(b * p.Tq + place.t) * p.ldo + place.h * p.dh + col] =
            from_f32<T>(place.live && sum != 0.0f ? o / sum : 0.0f);
    if (col == 0 && p.lse)
        p.lse[(b * p.Tq + place.t) * p.H + place.h] = place.live && sum != 0.0f ? top * kLn2 + logf(sum) : -kInf;
}

// Joins the parts of a row whose keys were split: a wave a row, two columns a lane;
// lane s weighs part s.
template <class T>
__global__ void __launch_bounds__(256) rar_attn_join(const AttnParams p)
{
    const int64_t rows = p.Tq * p.share;
    const int64_t place = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (place >= p.part_rows)
        return;
    const int64_t hk = place / rows % p.Hkv, b = place / rows / p.Hkv;
    const RowPlace r = row_place(p, hk, place % rows, length_of(p.qlen, b, p.Tq));
    const int lane = threadIdx.x & 63, c = lane * 2;
    // four parts' values at a time, the first of them on their way before the weights are known
    constexpr int kParts = 4;
    f32x2 a[kParts] = {};
    auto load = [&](int first) __attribute__((always_inline)) {
        if (c < p.pitch)
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                const int s = first + i < p.splits ? first + i : p.splits - 1;  // (lanes behind the last weigh zero)
                a[i] = *reinterpret_cast<const f32x2 *>(p.part + (s * p.part_rows + place) * p.pitch + c);
            }
    };
    load(0);
    float m = -kInf, l = 0.0f;
    if (lane < p.splits) {
        m = p.stats[(lane * p.part_rows + place) * 2];
        l = p.stats[(lane * p.part_rows + place) * 2 + 1];
    }
    const float top = wave_max(m);
    const float w = l == 0.0f ? 0.0f : __builtin_amdgcn_exp2f((m - (top == -kInf ? 0.0f : top)) * kLog2e);
    const float sum = wave_sum(w * l);
    f32x2 v = {0.0f, 0.0f};
    for (int first = 0; first < p.splits; first += kParts) {
        if (first)
            load(first);
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const float ws = __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(w), first + i));
            v.x = ws == 0.0f ? v.x : __builtin_fmaf(ws, a[i].x, v.x);  // (no key of such a part counts)
            v.y = ws == 0.0f ? v.y : __builtin_fmaf(ws, a[i].y, v.y);
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    T *const o = (T *)p.o + (b * p.Tq + r.t) * p.ldo + r.h * p.dh;
    if (c < p.dh)
        o[c] = from_f32<T>(r.live ? v.x * inv : 0.0f);
    if (c + 1 < p.dh)
        o[c + 1] = from_f32<T>(r.live ? v.y * inv : 0.0f);
    if (lane == 0 && p.lse)
        p.lse[(b * p.Tq + r.t) * p.H + r.h] = r.live && sum != 0.0f ? top + logf(sum) : -kInf;
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------

// -lse and -delta of every row of a head, query after query, in whole stages: what is
// added to scores and to dP.  bf16 has -lse / scale, which the scores' accumulator
// starts from, so that the products end with (scores - lse) / scale; in binary32 a
// sum that starts so far from zero would lose a digit.  Rows that do not count have
// -infinity, so that their weights are zero.  Eight lanes a row.
template <class T>
__global__ void __launch_bounds__(256) rar_attn_delta(const AttnParams p)
{
    const int64_t at = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);
    if (at >= p.B * p.H * p.padded)
        return;
    const int64_t t = at % p.padded, h = at / p.padded % p.H, b = at / p.padded / p.H;
    const int lane = threadIdx.x & 7;
    float lse = kInf, sum = 0.0f;
    if (t < length_of(p.qlen, b, p.Tq)) {
        const int64_t row = b * p.Tq + t;
        lse = p.lse[row * p.H + h];
        if (lse == -kInf) {
            lse = kInf;  // no key was left for it
        } else {
            const T *const o = (const T *)p.o + row * p.ldo + h * p.dh;
            const T *const g = (const T *)p.d_o + row * p.lddo + h * p.dh;
            for (int c = lane * 8; c < p.dh; c += 64) {
                float x[8], y[8];
                const int cnt = clamp8(p.dh - c);
                load8(o + c, cnt, x);
                load8(g + c, cnt, y);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sum = __builtin_fmaf(x[i], y[i], sum);
            }
        }
    }
#pragma unroll
    for (int d = 1; d < 8; d *= 2)
        sum += __shfl_xor(sum, d);
    if (lane == 0) {
        p.row_lse[at] = sizeof(T) == 2 ? -lse / p.scale : -lse;
        p.row_delta[at] = -sum;
    }
}

// dq: a wave holds 32 query rows as in the forward kernel.
template <class T, int W>
struct BackwardQ {
    typedef Shape<T, W> S;
    typedef typename S::Lds Lds;
    static constexpr int kTiles = sizeof(T) == 2 ? 2 : 1;  // of 32 rows, a stage
    static constexpr int kStage = kTiles * 32;
    static constexpr int kHalf = kStage * Lds::kBytes;
};

// bf16: two waves a SIMD, one under the other's chain of reads, products and exponentials; to fit, heads of over 96
// columns spill seven registers.  8 x 16 heads of 128, 2048 queries on 1024 keys: 207 us (three products, 1000
// TFLOP/s); one wave a SIMD takes 36% longer, and 19% with its schedule written out as that of dk and dv is.
// Binary32: a product of a tile takes the matrix cores long enough that the reads of the next are hidden one
// fragment ahead, which the compiler does.
template <class T, int W>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) rar_attn_dq(const AttnParams p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    typedef BackwardQ<T, W> F;
    typedef typename F::Lds Lds;
    constexpr int STEPS = F::S::STEPS;
    __shared__ __attribute__((aligned(1024))) char memory[4 * F::kHalf];
    RAR_LDS char *const lds = (RAR_LDS char *)memory;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, half = lane >> 5;

    const Place at = place_of(p.B * p.Hkv, p.Hkv, p.tiles * p.splits);
    const int64_t tile = at.in % p.tiles, split = at.in / p.tiles, hk = at.hk, b = at.b;
    const int64_t klen = length_of(p.klen, b, p.Tk), qlen = length_of(p.qlen, b, p.Tq);
    const int64_t rows = p.Tq * p.share;
    const int64_t first = tile * kAttnRows, row = first + wave * 32 + (lane & 31);
    const int64_t t = row / p.share, h = hk * p.share + row % p.share;
    const bool live = row < rows && t < qlen;
    Frag<T> q[STEPS], g[STEPS];
    load_row<T>(q, p.q, b * p.Tq + t, h, live);
    load_row<T>(g, p.g, b * p.Tq + t, h, live);
    const int64_t place = (b * p.H + h) * p.padded + t;
    const float scale = p.scale * kUnit<T>;
    const float lse = live ? -p.row_lse[place] * (sizeof(T) == 2 ? scale : 1.0f) : kInf;
    const float delta = live ? p.row_delta[place] : 0.0f;
    const bool some = lse != kInf;  // a key is left (weights are zero without, but a product with an infinity is not)

    // this workgroup's stages of keys
    const int64_t all = first / p.share < qlen ? (klen + F::kStage - 1) / F::kStage : 0;
    const int64_t begin = all * split / p.splits, k0 = begin * F::kStage;
    const int stages = (int)(all * (split + 1) / p.splits - begin);
    Loader<T, F::S::PITCH, F::kStage, 4> lk, lv;
    lk.init(p.k, b * p.Tk + k0, hk, klen - k0);
    lv.init(p.v, b * p.Tk + k0, hk, klen - k0);
    f32x16 acc[W];
#pragma unroll
    for (int d = 0; d < W; ++d)
        acc[d] = zeros();
    if (stages) {
        lk.load(lds);
        lv.load(lds + F::kHalf);
    }
    meet();
    auto stage = [&](auto BUF, int n) __attribute__((always_inline)) {
        RAR_LDS char *const here = lds + BUF() * 2 * F::kHalf;
        RAR_LDS char *const next = lds + (2 - BUF() * 2) * F::kHalf;
        if (n + 1 < stages) {
            lk.advance();
            lv.advance();
            lk.load(next);
            lv.load(next + F::kHalf);
        }
        const int rest = (int)(klen - k0 - (int64_t)n * F::kStage);
#pragma unroll
        for (int e = 0; e < F::kTiles; ++e) {
            f32x16 s = zeros(), dp = zeros();
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                mma(s, Lds::rows(here, e * 32, i), q[i]);
                mma(dp, Lds::rows(here + F::kHalf, e * 32, i), g[i]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[i] = weight<T>(s[i], scale, lse) * (dp[i] + delta);
            if (rest < F::kStage)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (e * 32 + row_of(i) + 4 * half >= rest)
                        s[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                Frag<T> w;
                w.set(s, 8 * j);
#pragma unroll
                for (int d = 0; d < W; ++d)
                    mma(acc[d], Lds::cols(here, e * 32, j, d), w);
            }
        }
        meet();
    };
    for (int n = 0; n < stages; n += 2) {
        stage(Half<0>{}, n);
        if (n + 1 < stages)
            stage(Half<1>{}, n + 1);
    }
    if (row >= rows)
        return;
    T *const out = (T *)p.dq + (b * p.Tq + t) * p.lddq + h * p.dh;
    float *const part = p.part + (split * p.part_rows + (b * p.Hkv + hk) * rows + row) * (W * 32);
#pragma unroll
    for (int d = 0; d < W; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = d * 32 + 8 * i + 4 * half;
            f32x4 v;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                v[x] = some ? acc[d][4 * i + x] * p.scale : 0.0f;
            if (p.splits > 1)
                store4(part + c, v);
            else
                put4(out, c, p.dh, v);
        }
#endif
}

// Rows r0 .. r0 + 31 of a result become the values at `from`.
__device__ __forceinline__ void start(f32x16 &v, const RAR_LDS float *__restrict__ from, int r0)
{
    const int half = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x4 a = *(const RAR_LDS f32x4 *)(from + r0 + 8 * i + 4 * half);
#pragma unroll
        for (int x = 0; x < 4; ++x)
            v[4 * i + x] = a[x];
    }
}

// dk and dv: a wave holds 32 keys, and the queries of every head that shares
// them pass by in stages.
template <class T, int W>
struct BackwardK {
    typedef Shape<T, W> S;
    typedef typename S::Lds Lds;
    static constexpr int kTiles = sizeof(T) == 2 ? 2 : 1;  // of 32 rows, a stage
    static constexpr int kStage = kTiles * 32;
    static constexpr int kHalf = kStage * Lds::kBytes;
    static constexpr int kBuffer = 2 * kHalf + 1024;    // q, do, lse and delta
};

// (Binary32.  Heads of over 96 columns take all 512 registers and spill 18.)
template <int W>
__global__ void __launch_bounds__(256, 1) rar_attn_dkv_f32(const AttnParams p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    typedef float T;
    typedef BackwardK<T, W> F;
    typedef typename F::Lds Lds;
    constexpr int STEPS = F::S::STEPS;
    __shared__ __attribute__((aligned(1024))) char memory[2 * F::kBuffer];
    RAR_LDS char *const lds = (RAR_LDS char *)memory;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, half = lane >> 5;

    const Place at = place_of(p.B * p.Hkv, p.Hkv, p.tiles * p.splits);
    const int64_t tile = at.in % p.tiles, split = at.in / p.tiles, hk = at.hk, b = at.b;
    const int64_t klen = length_of(p.klen, b, p.Tk), qlen = length_of(p.qlen, b, p.Tq);
    const int64_t key = tile * kAttnRows + wave * 32 + (lane & 31);
    const bool live = key < klen;
    Frag<T> k[STEPS], v[STEPS];
    load_row<T>(k, p.k, b * p.Tk + key, hk, live);
    load_row<T>(v, p.v, b * p.Tk + key, hk, live);
    f32x16 dk[W], dv[W];
#pragma unroll
    for (int d = 0; d < W; ++d) {
        dk[d] = zeros();
        dv[d] = zeros();
    }
    // this workgroup's stages of queries: one head after the other
    const int64_t per_head = (qlen + F::kStage - 1) / F::kStage;
    const int64_t all = tile * kAttnRows < klen ? per_head * p.share : 0;
    const int64_t begin = all * split / p.splits;
    const int stages = (int)(all * (split + 1) / p.splits - begin);
    Loader<T, F::S::PITCH, F::kStage, 4> lq, lg;
    int64_t head = hk * p.share + (all ? begin / per_head : 0);
    int64_t ahead = all ? begin % per_head : 0;  // stage within the head that is loaded next
    bool entered = false;
    auto load = [&](RAR_LDS char *to) __attribute__((always_inline)) {
        if (!entered) {
            lq.init(p.q, b * p.Tq + ahead * F::kStage, head, qlen - ahead * F::kStage);
            lg.init(p.g, b * p.Tq + ahead * F::kStage, head, qlen - ahead * F::kStage);
            entered = true;
        }
        lq.load(to);
        lg.load(to + F::kHalf);
        if (wave < 2) {
            // lse by the first wave, delta by the second: four bytes a lane, whole stages
            const int64_t row = (b * p.H + head) * p.padded + ahead * F::kStage;
            const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
                (void *)((wave ? p.row_delta : p.row_lse) + row), 0, F::kStage * 4, 0x00020000);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (RAR_LDS void *)(to + 2 * F::kHalf + wave * 256), 4, lane * 4,
                                                     0, 0, 0);
        }
        lq.advance();
        lg.advance();
        if (++ahead == per_head) {
            ahead = 0;
            ++head;
            entered = false;
        }
    };
    if (stages)
        load(lds);
    meet();
    auto stage = [&](auto BUF, int n) __attribute__((always_inline)) {
        RAR_LDS char *const here = lds + BUF() * F::kBuffer;
        if (n + 1 < stages)
            load(lds + (1 - BUF()) * F::kBuffer);
        const RAR_LDS float *const starts = (const RAR_LDS float *)(here + 2 * F::kHalf);
        f32x16 s = zeros(), dp, lse;
        start(dp, starts + 64, 0);
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            mma(s, Lds::rows(here, 0, i), k[i]);
            mma(dp, Lds::rows(here + F::kHalf, 0, i), v[i]);
        }
        start(lse, starts, 0);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            // The minimum with a NaN is the other: zeros in place of rows behind qlen make one with a key that holds an
            // infinity, and lse takes it out.  (Where a row that counts has a NaN, its lse is one.)
            s[i] = weight<T>(__builtin_fminf(s[i], 0x1.fffffep127f), p.scale, -lse[i]);
            dp[i] *= s[i];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            Frag<T> w, ds;
            w.set(s, 8 * j);
            ds.set(dp, 8 * j);
#pragma unroll
            for (int d = 0; d < W; ++d) {
                mma(dv[d], Lds::cols(here + F::kHalf, 0, j, d), w);
                mma(dk[d], Lds::cols(here, 0, j, d), ds);
            }
        }
        meet();
    };
    for (int n = 0; n < stages; n += 2) {
        stage(Half<0>{}, n);
        if (n + 1 < stages)
            stage(Half<1>{}, n + 1);
    }
    if (key >= p.Tk)
        return;
#pragma unroll
    for (int d = 0; d < W; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = d * 32 + 8 * i + 4 * half;
            f32x4 a, e;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                a[x] = live ? dk[d][4 * i + x] * p.scale : 0.0f;
                e[x] = live ? dv[d][4 * i + x] : 0.0f;
            }
            if (p.splits > 1) {
                float *const part = p.part + (split * p.part_rows + (b * p.Hkv + hk) * p.Tk + key) * (2 * W * 32);
                store4(part + c, a);
                store4(part + W * 32 + c, e);
                continue;
            }
            if (p.dk)
                put4((T *)p.dk + (b * p.Tk + key) * p.lddk + hk * p.dh, c, p.dh, a);
            if (p.dv)
                put4((T *)p.dv + (b * p.Tk + key) * p.lddv + hk * p.dh, c, p.dh, e);
        }
#endif
}

// The kernel for bf16 has its schedule in the text: products as statements that
// keep their order, accumulators and what a wave holds of its own in accumulation
// registers, scores in ordinary ones.  (Left to itself the compiler moves scores
// between the register files, three moves a product, and lets products, arithmetic
// and LDS reads wait for each other.)  One wave a SIMD, and what would wait runs
// under the products:
//   A(n)  scores of tile n + 1, between them the weights of tile n and the reads of
//         its transposed fragments
//   B(n)  products into the gradients of tile n, under them the reads of the rows of
//         tile n + 2
// (Heads of up to 64 columns leave room for a second wave.)
// Stages of two tiles of 32 rows pass through a ring of three in LDS, so that a
// stage's loads have the time of one stage to arrive.
__device__ __forceinline__ void product_v(f32x16 &c, const bf16x8 &a, const bf16x8 &b)
{
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "a"(b));
}

__device__ __forceinline__ void product_a(f32x16 &c, const bf16x8 &a, const bf16x8 &b)
{
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}

// A wave's keys and values are its own, scores start from LDS.
// 218 us at the size above, where the compiler's schedule takes 254; of the units'
// busy cycles the matrix cores take 44%, the vector units 28%.  Without the
// exponentials, or without the transposed reads, it takes 6 to 8% less, without the
// loads 8%, without the products of B 15%: what is left is one wave's own chain of
// instructions.  A ring of four took the same.
template <int W>
__global__ void __launch_bounds__(256, 1) rar_attn_dkv_bf16(const AttnParams p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    typedef BackwardK<bf16, W> F;
    typedef typename F::Lds Lds;
    constexpr int STEPS = F::S::STEPS, kProducts = 2 * STEPS;
    __shared__ __attribute__((aligned(1024))) char memory[3 * F::kBuffer];
    RAR_LDS char *const lds = (RAR_LDS char *)memory;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, half = lane >> 5;

    const Place at = place_of(p.B * p.Hkv, p.Hkv, p.tiles * p.splits);
    const int64_t tile = at.in % p.tiles, split = at.in / p.tiles, hk = at.hk, b = at.b;
    const int64_t klen = length_of(p.klen, b, p.Tk), qlen = length_of(p.qlen, b, p.Tq);
    const int64_t key = tile * kAttnRows + wave * 32 + (lane & 31);
    const bool live = key < klen;
    bf16x8 k[STEPS], v[STEPS];
    {
        Frag<bf16> f[STEPS];
        load_row<bf16>(f, p.k, b * p.Tk + key, hk, live);
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
            k[i] = f[i].v;
        load_row<bf16>(f, p.v, b * p.Tk + key, hk, live);
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
            v[i] = f[i].v;
    }
    f32x16 dk[W], dv[W];
#pragma unroll
    for (int d = 0; d < W; ++d) {
        dk[d] = zeros();
        dv[d] = zeros();
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
        asm volatile("" : "+a"(k[i]), "+a"(v[i]));
#pragma unroll
    for (int d = 0; d < W; ++d)
        asm volatile("" : "+a"(dk[d]), "+a"(dv[d]));
    const float scale2 = p.scale * kLog2e;

    // this workgroup's stages of queries: one head after the other
    const int64_t per_head = (qlen + F::kStage - 1) / F::kStage;
    const int64_t all = tile * kAttnRows < klen ? per_head * p.share : 0;
    const int64_t begin = all * split / p.splits;
    const int stages = (int)(all * (split + 1) / p.splits - begin);
    Loader<bf16, F::S::PITCH, F::kStage, 4> lq, lg;
    int64_t head = hk * p.share + (all ? begin / per_head : 0);
    int64_t ahead = all ? begin % per_head : 0;  // stage within the head that is loaded next
    bool entered = false;
    auto load = [&](RAR_LDS char *to) __attribute__((always_inline)) {
        if (!entered) {
            lq.init(p.q, b * p.Tq + ahead * F::kStage, head, qlen - ahead * F::kStage);
            lg.init(p.g, b * p.Tq + ahead * F::kStage, head, qlen - ahead * F::kStage);
            entered = true;
        }
        // (zeros in place of rows behind qlen, whose weights are zero, would make a NaN with a key that holds an
        // infinity: the last row makes one only where it does so itself)
        lq.template load<true>(to);
        lg.template load<true>(to + F::kHalf);
        if (wave < 2) {
            const int64_t row = (b * p.H + head) * p.padded + ahead * F::kStage;
            const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
                (void *)((wave ? p.row_delta : p.row_lse) + row), 0, F::kStage * 4, 0x00020000);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (RAR_LDS void *)(to + 2 * F::kHalf + wave * 256), 4, lane * 4,
                                                     0, 0, 0);
        }
        lq.advance();
        lg.advance();
        if (++ahead == per_head) {
            ahead = 0;
            ++head;
            entered = false;
        }
    };
    bf16x8 q[STEPS], g[STEPS], qt[2][W], gt[2][W];
    f32x16 s[2], dp[2];
    bf16x8 w[2], ds[2];
    // one of a tile's fragments: of a row, or transposed, in the order of their use
    auto read_row = [&](const RAR_LDS char *from, int e, int m) __attribute__((always_inline)) {
        if (m & 1)
            g[m / 2] = Lds::rows(from + F::kHalf, e * 32, m / 2).v;
        else
            q[m / 2] = Lds::rows(from, e * 32, m / 2).v;
    };
    auto read_col = [&](const RAR_LDS char *from, int e, int m) __attribute__((always_inline)) {
        const int j = m / (2 * W), d = m / 2 % W;
        if (m & 1)
            qt[j][d] = Lds::cols(from, e * 32, j, d).v;
        else
            gt[j][d] = Lds::cols(from + F::kHalf, e * 32, j, d).v;
    };
    auto begin_scores = [&](auto E, const RAR_LDS char *from) __attribute__((always_inline)) {
        const RAR_LDS float *const starts = (const RAR_LDS float *)(from + 2 * F::kHalf);
        start(s[E()], starts, E() * 32);
        start(dp[E()], starts + 64, E() * 32);
    };
    auto score = [&](auto E, int m) __attribute__((always_inline)) {
        if (m & 1)
            product_v(dp[E()], g[m / 2], v[m / 2]);
        else
            product_v(s[E()], q[m / 2], k[m / 2]);
    };
    // A: scores of tile N with the weights of the other tile, and the reads of its fragments, between them
    auto phase_a = [&](auto N, const RAR_LDS char *from) __attribute__((always_inline)) {
        constexpr int O = 1 - N();
        // the other tile's products were issued before phase B; its last ones write until here at the latest
        asm volatile("s_nop 15" : "+v"(s[O]), "+v"(dp[O]));
        float x[16], y[16];
        uint32_t pw[8], pd[8];
        auto finish = [&](int i) __attribute__((always_inline)) {
            y[i] = dp[O][i] * x[i];
            if (i & 1) {
                pw[i / 2] = pack_bf16(x[i - 1], x[i]);
                pd[i / 2] = pack_bf16(y[i - 1], y[i]);
                asm volatile("" : "+v"(pw[i / 2]), "+v"(pd[i / 2]));
            }
        };
#pragma unroll
        for (int m = 0; m < kProducts; ++m) {
            score(N, m);
            read_col(from, O, m);
#pragma unroll
            for (int i = m * 16 / kProducts; i < (m + 1) * 16 / kProducts; ++i) {
                x[i] = __builtin_amdgcn_exp2f(s[O][i] * scale2);
                asm volatile("" : "+v"(x[i]));
            }
            // (an exponential's result is used one product later)
            if (m > 0)
#pragma unroll
                for (int i = (m - 1) * 16 / kProducts; i < m * 16 / kProducts; ++i)
                    finish(i);
        }
#pragma unroll
        for (int i = (kProducts - 1) * 16 / kProducts; i < 16; ++i)
            finish(i);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            w[j] = __builtin_bit_cast(bf16x8, u32x4{pw[4 * j], pw[4 * j + 1], pw[4 * j + 2], pw[4 * j + 3]});
            ds[j] = __builtin_bit_cast(bf16x8, u32x4{pd[4 * j], pd[4 * j + 1], pd[4 * j + 2], pd[4 * j + 3]});
        }
        // packed by the vector units, read by the matrix ones
        asm volatile("s_nop 3" : "+v"(w[0]), "+v"(w[1]), "+v"(ds[0]), "+v"(ds[1]));
    };
    auto phase_b = [&](const RAR_LDS char *from, int e) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < kProducts; ++m) {
            const int j = m / (2 * W), d = m / 2 % W;
            if (m & 1)
                product_a(dk[d], qt[j][d], ds[j]);
            else
                product_a(dv[d], gt[j][d], w[j]);
            read_row(from, e, m);
        }
    };

    if (stages)
        load(lds);
    meet();
    if (stages > 1)
        load(lds + F::kBuffer);
    if (stages) {
#pragma unroll
        for (int m = 0; m < kProducts; ++m)
            read_row(lds, 0, m);
        begin_scores(Half<0>{}, lds);
#pragma unroll
        for (int m = 0; m < kProducts; ++m)
            score(Half<0>{}, m);
        begin_scores(Half<1>{}, lds);
#pragma unroll
        for (int m = 0; m < kProducts; ++m)
            read_row(lds, 1, m);
    }
    int slot = 0;
    for (int n = 0; n < stages; ++n) {
        RAR_LDS char *const here = lds + slot * F::kBuffer;
        slot = slot == 2 ? 0 : slot + 1;
        RAR_LDS char *const next = lds + slot * F::kBuffer;
        phase_a(Half<1>{}, here);
        // the next stage has arrived, and the one before this is no longer read
        meet();
        if (n + 2 < stages)
            load(lds + (slot == 2 ? 0 : slot + 1) * F::kBuffer);
        begin_scores(Half<0>{}, next);  // (behind the last stage: of what lies there, for nothing)
        phase_b(next, 0);
        phase_a(Half<0>{}, here);
        begin_scores(Half<1>{}, next);
        phase_b(next, 1);
    }
    // wait for the last products, and tie every use of the accumulators to what follows the wait
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
    for (int d = 0; d < W; ++d)
        asm volatile("" : "+a"(dk[d]), "+a"(dv[d]));
    if (key >= p.Tk)
        return;
#pragma unroll
    for (int d = 0; d < W; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = d * 32 + 8 * i + 4 * half;
            f32x4 a, e;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                a[x] = live ? dk[d][4 * i + x] * p.scale : 0.0f;
                e[x] = live ? dv[d][4 * i + x] : 0.0f;
            }
            if (p.splits > 1) {
                float *const part = p.part + (split * p.part_rows + (b * p.Hkv + hk) * p.Tk + key) * (2 * W * 32);
                store4(part + c, a);
                store4(part + W * 32 + c, e);
                continue;
            }
            if (p.dk)
                put4((bf16 *)p.dk + (b * p.Tk + key) * p.lddk + hk * p.dh, c, p.dh, a);
            if (p.dv)
                put4((bf16 *)p.dv + (b * p.Tk + key) * p.lddv + hk * p.dh, c, p.dh, e);
        }
#endif
}

// Joins the parts of split gradients, in order: first dq's rows, then those of dk and
// dv; four columns a lane.
template <class T>
__global__ void __launch_bounds__(256) rar_attn_sum(const AttnSum p)
{
    const int quads = p.pitch / 4;
    int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const bool keys = i >= p.q_rows * quads;
    if (keys)
        i -= p.q_rows * quads;
    const int width = keys ? 2 * quads : quads;
    const int64_t place = i / width, rows = keys ? p.k_rows : p.q_rows;
    if (place >= rows)
        return;
    const int at = (int)(i - place * width), splits = keys ? p.k_splits : p.q_splits;
    const float *from = (keys ? p.k_part : p.q_part) + place * (width * 4) + at * 4;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int s = 0; s < splits; ++s)
        v += load4(from + s * rows * (width * 4));
    const int64_t per = keys ? p.Tk : p.Tq * p.share, r = place % per;
    const int64_t hk = place / per % p.Hkv, b = place / per / p.Hkv;
    if (!keys) {
        const int64_t t = r / p.share, h = hk * p.share + r % p.share;
        put4((T *)p.dq + (b * p.Tq + t) * p.lddq + h * p.dh, at * 4, p.dh, v);
    } else if (at < quads) {
        if (p.dk)
            put4((T *)p.dk + (b * p.Tk + r) * p.lddk + hk * p.dh, at * 4, p.dh, v);
    } else if (p.dv) {
        put4((T *)p.dv + (b * p.Tk + r) * p.lddv + hk * p.dh, (at - quads) * 4, p.dh, v);
    }
}

// Copies of operands whose heads are not whole 16-byte groups at 16-byte aligned
// addresses: every head's columns to `cols`, zero behind dh.  A lane takes group
// after group, so that a launch takes operands of any size.
constexpr int64_t kPackBlocks = 16384;

template <class T>
__global__ void __launch_bounds__(256) rar_attn_pack(const AttnPack p, const int64_t chunks)
{
    constexpr int kPer = 16 / sizeof(T);
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < chunks; n += (int64_t)gridDim.x * 256) {
        int64_t i = n;
        int e = 0;
        while (i >= p.item[e].chunks)
            i -= p.item[e++].chunks;
        const AttnPack::Item &m = p.item[e];
        const int per_head = p.cols / kPer;
        const int64_t row = i / (m.heads * per_head);
        const int64_t in = i - row * (m.heads * per_head);
        const int64_t head = in / per_head, c = (in - head * per_head) * kPer;
        const T *const from = (const T *)m.src + row * m.ld + head * p.dh + c;
        float v[8];
        load8(from, clamp8(p.dh - c < kPer ? p.dh - c : kPer), v);
        T *const to = (T *)m.dst + (row * m.heads + head) * p.cols + c;
        if constexpr (sizeof(T) == 4)
            store4(to, f32x4{v[0], v[1], v[2], v[3]});
        else
            store8(to, 8, v);
    }
}

template <class P>
struct Kernels {
    void (*f32)(P), (*bf)(P);
};

template <class T>
void (*rows_kernel(int w, bool few))(AttnParams)
{
    switch (w) {
    case 1: return few ? rar_attn_few<T, 1> : rar_attn_rows<T, 1>;
    case 2: return few ? rar_attn_few<T, 2> : rar_attn_rows<T, 2>;
    case 3: return few ? rar_attn_few<T, 3> : rar_attn_rows<T, 3>;
    default: return few ? rar_attn_few<T, 4> : rar_attn_rows<T, 4>;
    }
}

template <class T>
void (*token_kernel(int w, int rows))(AttnParams)
{
    if (w <= 2)
        return rows == 1 ? rar_attn_token<T, 64, 1> : rows == 2 ? rar_attn_token<T, 64, 2> : rar_attn_token<T, 64, 4>;
    return rows == 1 ? rar_attn_token<T, 128, 1> : rows == 2 ? rar_attn_token<T, 128, 2> : rar_attn_token<T, 128, 4>;
}

void (*dq_kernel(rar_dtype dt, int w))(AttnParams)
{
    const bool wide = dt == RAR_F32;
    switch (w) {
    case 1: return wide ? rar_attn_dq<float, 1> : rar_attn_dq<bf16, 1>;
    case 2: return wide ? rar_attn_dq<float, 2> : rar_attn_dq<bf16, 2>;
    case 3: return wide ? rar_attn_dq<float, 3> : rar_attn_dq<bf16, 3>;
    default: return wide ? rar_attn_dq<float, 4> : rar_attn_dq<bf16, 4>;
    }
}

void (*dkv_kernel(rar_dtype dt, int w))(AttnParams)
{
    const bool wide = dt == RAR_F32;
    switch (w) {
    case 1: return wide ? rar_attn_dkv_f32<1> : rar_attn_dkv_bf16<1>;
    case 2: return wide ? rar_attn_dkv_f32<2> : rar_attn_dkv_bf16<2>;
    case 3: return wide ? rar_attn_dkv_f32<3> : rar_attn_dkv_bf16<3>;
    default: return wide ? rar_attn_dkv_f32<4> : rar_attn_dkv_bf16<4>;
    }
}

}  // namespace

hipError_t launch_attn_rows(rar_dtype dt, const AttnParams &p, bool few, hipStream_t st)
{
    const int w = (p.dh + 31) / 32;
    if (p.Tq * p.share <= kAttnTokenRows) {
        const int rows = (int)(p.Tq * p.share);
        return launch(dt == RAR_BF16 ? token_kernel<bf16>(w, rows) : token_kernel<float>(w, rows), (unsigned)p.blocks,
                      64 * kTokenWaves, st, p);
    }
    const int waves = few ? attn_few_waves((w <= 2 ? 64 : 128) * (dt == RAR_BF16 ? 2 : 4)) : 4;
    return launch(dt == RAR_BF16 ? rows_kernel<bf16>(w, few) : rows_kernel<float>(w, few), (unsigned)p.blocks,
                  64 * waves, st, p);
}

hipError_t launch_attn_join(rar_dtype dt, const AttnParams &p, hipStream_t st)
{
    return launch(dt == RAR_BF16 ? rar_attn_join<bf16> : rar_attn_join<float>, (unsigned)((p.part_rows + 3) / 4), 256,
                  st, p);
}

hipError_t launch_attn_delta(rar_dtype dt, const AttnParams &p, hipStream_t st)
{
    return launch(dt == RAR_BF16 ? rar_attn_delta<bf16> : rar_attn_delta<float>,
                  (unsigned)((p.B * p.H * p.padded + 31) / 32), 256, st, p);
}

hipError_t launch_attn_dq(rar_dtype dt, const AttnParams &p, hipStream_t st)
{
    const int w = (p.dh + 31) / 32;
    return launch(dq_kernel(dt, w), (unsigned)p.blocks, 256, st, p);
}

hipError_t launch_attn_dkv(rar_dtype dt, const AttnParams &p, hipStream_t st)
{
    const int w = (p.dh + 31) / 32;
    return launch(dkv_kernel(dt, w), (unsigned)p.blocks, 256, st, p);
}

hipError_t launch_attn_sum(rar_dtype dt, const AttnSum &p, hipStream_t st)
{
    const int64_t lanes = (p.q_rows + 2 * p.k_rows) * (p.pitch / 4);
    return launch(dt == RAR_BF16 ? rar_attn_sum<bf16> : rar_attn_sum<float>, (unsigned)((lanes + 255) / 256), 256, st,
                  p);
}

hipError_t launch_attn_pack(rar_dtype dt, const AttnPack &p, hipStream_t st)
{
    int64_t chunks = 0;
    for (int i = 0; i < p.count; ++i)
        chunks += p.item[i].chunks;
    return launch(dt == RAR_BF16 ? rar_attn_pack<bf16> : rar_attn_pack<float>,
                  (unsigned)std::min((chunks + 255) / 256, kPackBlocks), 256, st, p, chunks);
}

}  // namespace rar
