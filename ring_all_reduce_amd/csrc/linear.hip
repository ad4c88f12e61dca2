// linear.hip -- CDNA4 (gfx950) kernels of the linear layer: the matrix products
// of its forward and backward pass on the matrix cores, with the layer's
// epilogues, and the streaming passes around them.
//
//   forward   z = x W + b, y = act(z) + r       A = x  (k contiguous), B = W  (k slow)
//   grad x    dx = dz W^T                       A = dz (k contiguous), B = W  (k contiguous)
//   grad W    dW = x^T dz                       A = x  (k slow),       B = dz (k slow)
//
// Every product is D[m][n] = sum_k A(m,k) B(n,k).  The matrix instruction's first
// operand takes B and the second A, so a lane ends with four consecutive n of
// one row m and stores them together.
#include "act.h"
#include "ops_internal.h"

#pragma clang fp contract(off)

#define RAR_LDS __attribute__((address_space(3)))

namespace rar {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr uint32_t kOutOfRange = 0x80000000u;
constexpr int kRow = 128;  // bytes of reduction of a contiguous operand's row in one step

// ---------------------------------------------------------------------------
// Staging: memory -> LDS, 16 bytes a lane, without passing through registers
// ---------------------------------------------------------------------------
//
// One step stages kRow / ES reduction indices of R rows of an operand.
//   contiguous: LDS row r holds its 128 bytes of k; the 16-byte chunk c lies at
//               slot c ^ (r & 7), so 16 lanes that read one chunk of 16 rows
//               touch every bank once.  (Rows of 64 bytes, for more and smaller
//               steps in flight, cost twice the requests a byte and were 6%
//               slower.)
//   slow:       LDS row k holds R elements; bf16 units of 16 elements are
//               permuted by f(k), binary32 by one bit of k, so that the four
//               k rows of a transposing read (or the two of a binary32 read)
//               lie in different banks.
// The destination of such a load is linear in the lane, so the permutation is
// applied to the address that each lane reads.
//
// The buffer descriptor's range ends with the operand's last element: rows
// behind it read as zero, whatever lies there.  Where a contiguous operand's
// reduction ends inside a step, the chunks behind the end are sent out of
// range too, since what follows them is the next row.  The descriptor moves
// along the reduction in 64 bits; offsets inside a tile stay under 2^31.
template <int ES>
__device__ __forceinline__ int slow_perm(int k)
{
    return ES == 2 ? ((k & 3) | (((k >> 3) & 3) << 2)) : ((k >> 2) & 1);
}

template <int ES, int R, int WAVES, bool CONTIG>
struct Stage {
    static constexpr int kLoads = R * kRow / (WAVES * 1024);
    static constexpr int kStep = kRow / ES;  // reduction indices of one step
    uint32_t voff[kLoads];
    const char *base;
    int64_t left;     // bytes from base to the end of the operand
    int64_t advance;  // bytes per step

    // Row lengths in whole 16-byte groups: the range is checked by the dword,
    // and the host packs rows that end inside one with zeros.
    static __device__ __forceinline__ int64_t whole(int64_t n) { return (n + 16 / ES - 1) / (16 / ES) * (16 / ES); }

    // Contiguous: row and source chunk of this lane's j-th load.
    static __device__ __forceinline__ int row_of(int j)
    {
        return (j * WAVES + (threadIdx.x >> 6)) * 8 + ((threadIdx.x & 63) >> 3);
    }
    static __device__ __forceinline__ int chunk_of(int j) { return (threadIdx.x & 7) ^ (row_of(j) & 7); }

    // rows [r0, ...) of `rows`, reduction indices [k0, ...) of `kred`
    __device__ __forceinline__ void init(const void *p, int64_t ld, int64_t r0, int64_t rows, int64_t k0, int64_t kred)
    {
        if (CONTIG) {
            base = (const char *)p + (r0 * ld + k0) * ES;
            left = ((rows - 1 - r0) * ld + whole(kred - k0)) * ES;
            advance = kRow;
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                voff[j] = (uint32_t)(row_of(j) * ld * ES) + (chunk_of(j) << 4);
        } else {
            constexpr int kCols = R * ES;
            base = (const char *)p + (k0 * ld + r0) * ES;
            left = ((kred - 1 - k0) * ld + whole(rows - r0)) * ES;
            advance = kStep * ld * ES;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int at = (j * WAVES + (threadIdx.x >> 6)) * 1024 + (threadIdx.x & 63) * 16;
                const int k = at / kCols, slot = (at % kCols) / 16;
                int src;
                if (ES == 2)
                    src = (((slot >> 1) ^ (slow_perm<2>(k) & (R / 16 - 1))) << 1) | (slot & 1);
                else
                    src = slot ^ (slow_perm<4>(k) << 3);
                voff[j] = (uint32_t)(k * ld * ES) + src * 16;
            }
        }
    }

    // Chunks of a contiguous operand behind the last `kleft` reduction indices.
    __device__ __forceinline__ void cut(int64_t kleft)
    {
        if (!CONTIG)
            return;
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if (chunk_of(j) * (16 / ES) >= kleft)
                voff[j] = kOutOfRange;
    }

    // The descriptor of the next step (empty: it reads zeros); load() issues its j-th load.
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t next(bool empty)
    {
        const int64_t n = left < 0 || empty ? 0 : (left > 0x7fffffff ? 0x7fffffff : left);
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, (int)n, 0x00020000);
        base += advance;
        left -= advance;
        return r;
    }

    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, RAR_LDS char *__restrict__ lds, int j) const
    {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (RAR_LDS void *)(lds + (j * WAVES + wave) * 1024), 16, voff[j], 0,
                                                 0, 0);
    }

    __device__ __forceinline__ void load_all(RAR_LDS char *__restrict__ lds, bool empty)
    {
        const __amdgpu_buffer_rsrc_t r = next(empty);
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            load(r, lds, j);
    }
};

// ---------------------------------------------------------------------------
// Fragments
// ---------------------------------------------------------------------------

// bf16, v_mfma_f32_16x16x32: lane l holds row l % 16 and the eight reduction
// indices (l / 16) * 8 .. +7 of a half step of 32.  A slow operand is read with the
// transposing LDS read: each 16 lanes read four k rows of 16 columns and
// receive their own column's four values.
template <int R, bool CONTIG, int NF>
struct Frag16 {
    uint32_t off[CONTIG ? 1 : NF];

    __device__ __forceinline__ void init(int w0)
    {
        const int lane = threadIdx.x & 63;
        if (CONTIG) {
            off[0] = (w0 + (lane & 15)) * kRow + (((lane >> 4) ^ (lane & 7)) << 4);
        } else {
            const int k = (lane >> 4) * 8 + ((lane & 15) >> 2);
            const int f = slow_perm<2>(k) & (R / 16 - 1);
#pragma unroll
            for (int i = 0; i < (CONTIG ? 1 : NF); ++i)
                off[i] = k * (R * 2) + (((w0 / 16 + i) ^ f) << 5) + (lane & 3) * 8;
        }
    }

    __device__ __forceinline__ bf16x8 read(const RAR_LDS char *__restrict__ lds, int half, int i) const
    {
        if (CONTIG)
            return *(const RAR_LDS bf16x8 *)(lds + (off[0] ^ (half << 6)) + i * 16 * kRow);
        const RAR_LDS char *p = lds + off[CONTIG ? 0 : i] + half * 32 * (R * 2);
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((RAR_LDS i16x4 *)p);
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((RAR_LDS i16x4 *)(p + 4 * (R * 2)));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// binary32, v_mfma_f32_32x32x2: lane l holds row l % 32; in a group of eight
// reduction indices the lower half-wave holds the first four, one per
// instruction.
template <int R, bool CONTIG>
struct Frag32 {
    uint32_t off;

    __device__ __forceinline__ void init(int w0)
    {
        const int lane = threadIdx.x & 63;
        const int row = w0 + (lane & 31), half = lane >> 5;
        if (CONTIG)
            off = row * kRow + ((half ^ (row & 7)) << 4);
        else
            off = half * 4 * (R * 4) + ((row * 4) ^ (half << 7));
    }

    __device__ __forceinline__ f32x4 read(const RAR_LDS char *__restrict__ lds, int c, int i) const
    {
        if (CONTIG)
            return *(const RAR_LDS f32x4 *)(lds + (off ^ (c << 5)) + i * 32 * kRow);
        // 32 columns are 128 bytes: an odd block of them flips the permuted bit
        const RAR_LDS char *p = lds + (off ^ (i << 7)) + c * 8 * (R * 4);
        return f32x4{*(const RAR_LDS float *)p, *(const RAR_LDS float *)(p + R * 4),
                     *(const RAR_LDS float *)(p + 2 * R * 4), *(const RAR_LDS float *)(p + 3 * R * 4)};
    }
};

// ---------------------------------------------------------------------------
// Epilogue: eight consecutive n of row m
// ---------------------------------------------------------------------------

// A group of 32 consecutive n lies in four neighbouring lanes.  Every lane of
// the wave calls this; rows and columns outside the matrix take part in the
// group's exchange only.
template <class T>
__device__ __forceinline__ void epilogue(const GemmParams &p, int64_t m, int64_t n, float (&v)[8])
{
    const int cnt = m >= p.M || n >= p.N ? 0 : (p.N - n < 8 ? (int)(p.N - n) : 8);
    T *const out = (T *)p.out + m * p.ldo + n;
    float t[8];
    if (p.mode == kModeForward) {
        if (p.bias) {
            load8((const T *)p.bias + n, cnt, t);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] += t[i];
        }
        if (p.pre_scales) {
            // the checkpoint of z, as rar_ckpt_store makes it of z in the layer's type
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                t[i] = i < cnt ? to_f32(from_f32<T>(v[i])) : 0.0f;
                top = ckpt_top(top, t[i]);
            }
            top = max(top, (uint32_t)__shfl_xor(top, 1));
            top = max(top, (uint32_t)__shfl_xor(top, 2));
            const int e = ckpt_exponent(top);
            const int64_t groups = (p.N + kCkptGroup - 1) / kCkptGroup;
            const int64_t g = n / kCkptGroup;
            if (m < p.M && g < groups) {
                *reinterpret_cast<u32x2 *>((uint8_t *)p.pre + m * groups * kCkptGroup + n) =
                    u32x2{ckpt_codes4(f32x4{t[0], t[1], t[2], t[3]}, e), ckpt_codes4(f32x4{t[4], t[5], t[6], t[7]}, e)};
                if (n % kCkptGroup == 0)
                    p.pre_scales[m * groups + g] = (uint8_t)e;
            }
        } else if (p.pre) {
            store8((T *)p.pre + m * p.ldp + n, cnt, v);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = act_value<T>(p.act, v[i]);
        if (p.res) {
            load8((const T *)p.res + m * p.ldr + n, cnt, t);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] += t[i];
        }
    } else if (p.accumulate) {
        load8(out, cnt, t);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] += t[i];
    }
    store8(out, cnt, v);
}

// A wave's ROWS rows of W columns pass through LDS, so that a lane finishes
// eight consecutive columns of one row and a row's lanes access whole lines.
// The 16-byte chunk c of row r lies at slot c ^ r (of the low bits of r): a
// column of rows spreads over the banks.
template <int W>
__device__ __forceinline__ RAR_LDS f32x4 *tile_slot(RAR_LDS char *tile, int r, int c)
{
    return (RAR_LDS f32x4 *)(tile + r * (W * 4) + ((c ^ (r & (W >= 64 ? 15 : W / 4 - 1))) << 4));
}

template <int W>
__device__ __forceinline__ void tile_row(RAR_LDS char *tile, int r, int q, float (&v)[8])
{
    const f32x4 lo = *tile_slot<W>(tile, r, 2 * q), hi = *tile_slot<W>(tile, r, 2 * q + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = lo[i];
        v[4 + i] = hi[i];
    }
}

// The usual tile: wholly inside the matrix, z kept in the layer's type or not at
// all.  The same results as epilogue(), with the addresses and the bias out of
// the loop.  Rows are written past the caches.  Forward and backward of two bf16
// layers, 2048 -> 8192 with gelu and back, with such stores and with ordinary
// ones: 8192 rows 1342 and 1364 us, 512 rows 165 and 172, 128 rows 105 and 107;
// the first layer's forward call and then the second's, which reads it: 453 and
// 473, 62 and 63, 42.6 and 42.4.  Rows that start off the 128-byte lines lose by
// it: 7178 x 177 -> 2023 takes 45 and 37 in bf16, 115 and 76 in binary32.
template <class T, int W, int ROWS, int ACT>
__device__ __forceinline__ void finish_inside(const GemmParams &p, RAR_LDS char *tile, int64_t m0, int64_t n0)
{
    constexpr int kLanes = W / 8, kRows = 64 / kLanes;
    const int lane = threadIdx.x & 63, q = lane % kLanes;
    const int64_t m = m0 + lane / kLanes, n = n0 + q * 8;
    float bias[8] = {};
    if (p.bias)
        load8((const T *)p.bias + n, 8, bias);
    T *out = (T *)p.out + m * p.ldo + n;
    T *pre = (T *)p.pre + m * p.ldp + n;
    const T *res = (const T *)p.res + m * p.ldr + n;
    const int64_t so = kRows * p.ldo, sp = kRows * p.ldp, sr = kRows * p.ldr;
#pragma unroll 2
    for (int r = lane / kLanes; r < ROWS; r += kRows) {
        float v[8], t[8];
        if (p.res)
            load8(res, 8, t);
        tile_row<W>(tile, r, q, v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] += bias[i];
        if (p.pre)
            store8<true>(pre, 8, v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = act_value<T>(ACT, v[i]);
        if (p.res)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] += t[i];
        store8<true>(out, 8, v);
        out += so;
        pre += sp;
        res += sr;
    }
}

template <class T, int W, int ROWS>
__device__ __forceinline__ void finish_rows(const GemmParams &p, int split, RAR_LDS char *tile, int64_t m0, int64_t n0)
{
    constexpr int kLanes = W / 8, kRows = 64 / kLanes;
    const int lane = threadIdx.x & 63, q = lane % kLanes;
    const int64_t n = n0 + q * 8;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (m0 + ROWS <= p.M && n0 + W <= p.N && !p.pre_scales &&
        (p.mode == kModeForward || (p.mode == kModeStore && !p.accumulate))) {
        // a plain store has no bias, residual, z or activation
        if (p.act == RAR_ACT_GELU)
            finish_inside<T, W, ROWS, RAR_ACT_GELU>(p, tile, m0, n0);
        else if (p.act == RAR_ACT_RELU)
            finish_inside<T, W, ROWS, RAR_ACT_RELU>(p, tile, m0, n0);
        else
            finish_inside<T, W, ROWS, RAR_ACT_NONE>(p, tile, m0, n0);
    } else {
#pragma unroll 1
        for (int r = lane / kLanes; r < ROWS; r += kRows) {
            float v[8];
            tile_row<W>(tile, r, q, v);
            const int64_t m = m0 + r;
            if (p.mode == kModePartial) {
                if (m < p.M && n < p.pitch) {  // pitch is whole groups; columns behind N hold anything
                    float *o = p.part + ((int64_t)split * p.M + m) * p.pitch + n;
                    store4(o, f32x4{v[0], v[1], v[2], v[3]});
                    store4(o + 4, f32x4{v[4], v[5], v[6], v[7]});
                }
                continue;
            }
            epilogue<T>(p, m, n, v);
        }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

// Workgroups go to the eight XCDs in turn; each XCD gets one run of tiles, in
// bands of four tile rows, so that its L2 holds the operands they share.
__device__ __forceinline__ void tile_of(const GemmParams &p, int64_t id, int64_t &tm, int64_t &tn, int &split)
{
    const int64_t tiles = p.tiles_m * p.tiles_n, total = tiles * p.splits;
    const int64_t per = total / 8;
    if (id < per * 8)
        id = (id % 8) * per + id / 8;
    split = (int)(id / tiles);
    id -= split * tiles;
    constexpr int kBand = 4;  // tile rows: 8 and 2 measured 1-2% slower at 8192 x 2048 x 8192
    const int64_t band = kBand * p.tiles_n;
    const int64_t first = id / band * kBand;
    const int64_t rows = p.tiles_m - first < kBand ? p.tiles_m - first : kBand;
    const int64_t in = id % band;
    tm = first + in % rows;
    tn = in / rows;
}

// Own loads into LDS but the last N have arrived; then everyone's.
template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Own loads into LDS and LDS reads are done; then everyone's.
__device__ __forceinline__ void drain()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// acc += b a, with the accumulator kept in an accumulation register: left to
// itself the compiler moves the 256 of a large tile back and forth between the
// two register files, about two moves a product.  The statements keep their
// order among each other and among the LDS accesses between them, so the
// kernel's text is its schedule.
__device__ __forceinline__ void product(f32x4 &acc, bf16x8 b, bf16x8 a)
{
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}

// ---------------------------------------------------------------------------
// bf16 product
// ---------------------------------------------------------------------------
//
// WM x WN waves hold a BM x BN tile in accumulators.  A step of 64 reduction
// indices is staged in one half of LDS while the other is used; its two halves
// of 32 pass through registers:
//   half 0   products of half 0, reading the fragments of half 1
//   half 1   wait for the next step's loads, meet the other waves; products of
//            half 1, reading the next step's half 0, and issuing the loads of
//            the step after it into the LDS half that everyone has now read
// Fragments of A are replaced in place once their row of products is issued;
// those of B need two sets.  Bound: the matrix cores, 68% busy in the backward
// products and 51% in the forward one with its epilogue, at 256 x 256 and the
// 1.9 to 2.0 GHz that the clock falls to under them.  Eight waves rather than four: two
// waves a SIMD cover each other's meeting and address work, and the epilogue's
// arithmetic.  A ring of five smaller buffers with loads further ahead measured
// the same; 32 x 32 x 16 instructions 3 to 5% slower, their reads of 32 rows
// meeting in the same banks.  Measured at 8192 rows, 2048 -> 8192, under a
// profiler (median of 30 passes, and the least): both backward products in one
// launch 412 us (389; 1.33 PFLOP/s), the forward product with gelu and z kept 284
// (253; 0.97 PFLOP/s).  The forward call timed without it takes 250 (1.10
// PFLOP/s), about 50 of it the epilogue.  128 x 128 tiles for products with few
// tiles: 2048 x 4096 -> 4096 62 us (1.1 PFLOP/s).
template <int BM, int BN, int WM, int WN, bool ACONTIG, bool BCONTIG>
__device__ __forceinline__ void gemm_bf16(const GemmParams &p, int64_t block, RAR_LDS char *const lds)
{
    constexpr int kWaves = WM * WN, kEarly = 1;
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // 16-row fragments of a wave
    constexpr int kBuf = (BM + BN) * kRow;

    int64_t tm, tn;
    int split;
    tile_of(p, block, tm, tn, split);
    const int64_t m0 = tm * BM, n0 = tn * BN;
    const int64_t k0 = split * p.steps_per_split * 64;
    const int64_t kend = k0 + p.steps_per_split * 64 < p.K ? k0 + p.steps_per_split * 64 : p.K;
    const int steps = k0 < kend ? (int)((kend - k0 + 63) / 64) : 0;
    const int wave = threadIdx.x >> 6, wm = (wave % WM) * (BM / WM), wn = (wave / WM) * (BN / WN);

    Stage<2, BM, kWaves, ACONTIG> sa;
    Stage<2, BN, kWaves, BCONTIG> sb;
    sa.init(p.a, p.lda, m0, p.M, k0, kend);
    sb.init(p.b, p.ldb, n0, p.N, k0, kend);
    constexpr int kLoads = sa.kLoads + sb.kLoads;
    Frag16<BM, ACONTIG, FM> fa;
    Frag16<BN, BCONTIG, FN> fb;
    fa.init(wm);
    fb.init(wn);

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            asm volatile("" : "+a"(acc[i][j]));

    // The last step's reduction may end inside it.
    auto cut = [&](int s) __attribute__((always_inline)) {
        if (s == steps - 1) {
            sa.cut(kend - k0 - (int64_t)s * 64);
            sb.cut(kend - k0 - (int64_t)s * 64);
        }
    };
    // (the same before the first: the zeros have been written)
    asm volatile("s_nop 7" ::: "memory");
    bf16x8 a[FM], b0[FN], b1[FN];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        cut(s);
        sa.load_all(lds + s * kBuf, s >= steps);
        sb.load_all(lds + s * kBuf + BM * kRow, s >= steps);
    }
    wait_loads<kLoads>();
#pragma unroll
    for (int j = 0; j < FN; ++j)
        b0[j] = fb.read(lds + BM * kRow, 0, j);
#pragma unroll
    for (int i = 0; i < FM; ++i)
        a[i] = fa.read(lds, 0, i);

    for (int s = 0; s < steps; ++s) {
        RAR_LDS char *const here = lds + (s & 1) * kBuf;
        RAR_LDS char *const next = lds + (kBuf - (s & 1) * kBuf);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
                product(acc[i][j], b0[j], a[i]);
            a[i] = fa.read(here, 1, i);
#pragma unroll
            for (int e = i * FN / FM; e < (i + 1) * FN / FM; ++e)
                b1[e] = fb.read(here + BM * kRow, 1, e);
        }
        cut(s + 2);
        const __amdgpu_buffer_rsrc_t ra = sa.next(s + 2 >= steps), rb = sb.next(s + 2 >= steps);
        // a few rows first: the meeting then finds the last reads done
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            if (i == kEarly)
                drain();
#pragma unroll
            for (int j = 0; j < FN; ++j)
                product(acc[i][j], b1[j], a[i]);
            if (i < kEarly)
                continue;
            constexpr int kReads = FM + FN, kRows = FM - kEarly;
#pragma unroll
            for (int e = (i - kEarly) * kReads / kRows; e < (i - kEarly + 1) * kReads / kRows; ++e) {
                // B's fragments, then A's as far as their products are issued
                if (e < FN)
                    b0[e] = fb.read(next + BM * kRow, 0, e);
                else
                    a[e - FN] = fa.read(next, 0, e - FN);
            }
#pragma unroll
            for (int e = (i - kEarly) * kLoads / kRows; e < (i - kEarly + 1) * kLoads / kRows; ++e)
                if (e < sa.kLoads)
                    sa.load(ra, here, e);
                else
                    sb.load(rb, here + BM * kRow, e - sa.kLoads);
        }
    }

    // The compiler does not know the statements' latency: wait for the last
    // products, and tie every use of the accumulators to what follows the wait.
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            asm volatile("" : "+a"(acc[i][j]));
    // every wave has read its last fragments: LDS is free for the results
    drain();
    const int lane = threadIdx.x & 63;
    constexpr int kPass = 64;  // rows of a pass: as many as fit
    static_assert(kWaves * kPass * FN * 16 * 4 <= 2 * kBuf, "results pass through the operands' LDS");
    RAR_LDS char *const tile = lds + wave * (kPass * FN * 16 * 4);
#pragma unroll
    for (int i = 0; i < FM; i += kPass / 16) {
#pragma unroll
        for (int h = 0; h < kPass / 16; ++h)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                *tile_slot<FN * 16>(tile, h * 16 + (lane & 15), j * 4 + (lane >> 4)) = acc[i + h][j];
        finish_rows<bf16, FN * 16, kPass>(p, split, tile, m0 + wm + i * 16, n0 + wn);
    }
}

// ---------------------------------------------------------------------------
// binary32 product
// ---------------------------------------------------------------------------
//
// The binary32 matrix instruction does a sixteenth of the bf16 one's work per
// cycle, so its operands come from LDS with time to spare; what is left is to
// keep the instruction fed across steps.  Four waves as 2 x 2 hold a B x B
// tile; a step of 32 reduction indices is staged in one half of LDS while the
// other is used, in four groups of eight whose fragments are read one group
// ahead.  In the last group of a step the waves meet: the next step has then
// arrived, and this one's half is free for the step after it.  Bound: the
// binary32 matrix instruction, 137-141 TFLOP/s in 128 x 128 tiles at 8192 x
// 2048 -> 2048 (500 us); 64 x 64 tiles spread smaller layers over the chip,
// 2048 x 2048 -> 2048 132 us.
template <int B, bool ACONTIG, bool BCONTIG>
__device__ __forceinline__ void gemm_f32(const GemmParams &p, int64_t block, RAR_LDS char *const lds)
{
    constexpr int kStep = 32, F = B / 64;
    constexpr int kBuf = 2 * B * kRow;

    int64_t tm, tn;
    int split;
    tile_of(p, block, tm, tn, split);
    const int64_t m0 = tm * B, n0 = tn * B;
    const int64_t k0 = split * p.steps_per_split * kStep;
    const int64_t kend = k0 + p.steps_per_split * kStep < p.K ? k0 + p.steps_per_split * kStep : p.K;
    const int steps = k0 < kend ? (int)((kend - k0 + kStep - 1) / kStep) : 0;
    const int wave = threadIdx.x >> 6, wm = (wave & 1) * (B / 2), wn = (wave >> 1) * (B / 2);

    Stage<4, B, 4, ACONTIG> sa;
    Stage<4, B, 4, BCONTIG> sb;
    sa.init(p.a, p.lda, m0, p.M, k0, kend);
    sb.init(p.b, p.ldb, n0, p.N, k0, kend);
    Frag32<B, ACONTIG> fa;
    Frag32<B, BCONTIG> fb;
    fa.init(wm);
    fb.init(wn);

    f32x16 acc[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[i][j][e] = 0.0f;

    auto stage = [&](int s) __attribute__((always_inline)) {
        if (s == steps - 1) {
            sa.cut(kend - k0 - (int64_t)s * kStep);
            sb.cut(kend - k0 - (int64_t)s * kStep);
        }
        RAR_LDS char *to = lds + (s & 1) * kBuf;
        sa.load_all(to, s >= steps);
        sb.load_all(to + B * kRow, s >= steps);
    };
    f32x4 a[2][F], b[2][F];
    auto read = [&](int s, int c, int set) __attribute__((always_inline)) {
        const RAR_LDS char *from = lds + (s & 1) * kBuf;
#pragma unroll
        for (int i = 0; i < F; ++i) {
            a[set][i] = fa.read(from, c, i);
            b[set][i] = fb.read(from + B * kRow, c, i);
        }
    };

    stage(0);
    stage(1);
    wait_loads<sa.kLoads + sb.kLoads>();
    read(0, 0, 0);
    for (int s = 0; s < steps; ++s) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (c < 3)
                read(s, c + 1, (c + 1) & 1);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (c == 3 && e == 1) {
                    drain();
                    read(s + 1, 0, 0);  // behind the last step: zeros
                    stage(s + 2);
                }
#pragma unroll
                for (int i = 0; i < F; ++i)
#pragma unroll
                    for (int j = 0; j < F; ++j)
                        acc[i][j] =
                            __builtin_amdgcn_mfma_f32_32x32x2f32(b[c & 1][j][e], a[c & 1][i][e], acc[i][j], 0, 0, 0);
            }
        }
    }

    drain();
    const int lane = threadIdx.x & 63;
    constexpr int W = B / 2;
    RAR_LDS char *const tile = lds + wave * (W * W * 4);
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *tile_slot<W>(tile, i * 32 + (lane & 31), j * 8 + q * 2 + (lane >> 5)) =
                    f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    finish_rows<float, W, W>(p, split, tile, m0 + wm, n0 + wn);
}

// ---------------------------------------------------------------------------
// The layer's launches
// ---------------------------------------------------------------------------

// (The host pass needs the kernels' names only.)
template <int B, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN, 2) rar_forward_bf16(const GemmParams p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ __attribute__((aligned(1024))) char lds[2 * 2 * B * kRow];
    gemm_bf16<B, B, WM, WN, true, false>(p, blockIdx.x, (RAR_LDS char *)lds);
#endif
}

// Both products of a backward pass in one launch: they need only dz, and of a
// small layer each leaves most of the chip idle.
template <int B, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN, 2) rar_backward_bf16(const GemmPair p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ __attribute__((aligned(1024))) char lds[2 * 2 * B * kRow];
    if (blockIdx.x < p.x_blocks)
        gemm_bf16<B, B, WM, WN, true, true>(p.x, blockIdx.x, (RAR_LDS char *)lds);
    else
        gemm_bf16<B, B, WM, WN, false, false>(p.w, blockIdx.x - p.x_blocks, (RAR_LDS char *)lds);
#endif
}

template <int B>
__global__ void __launch_bounds__(256, B == 128 ? 2 : 4) rar_forward_f32(const GemmParams p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ __attribute__((aligned(1024))) char lds[2 * 2 * B * kRow];
    gemm_f32<B, true, false>(p, blockIdx.x, (RAR_LDS char *)lds);
#endif
}

template <int B>
__global__ void __launch_bounds__(256, B == 128 ? 2 : 4) rar_backward_f32(const GemmPair p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ __attribute__((aligned(1024))) char lds[2 * 2 * B * kRow];
    if (blockIdx.x < p.x_blocks)
        gemm_f32<B, true, true>(p.x, blockIdx.x, (RAR_LDS char *)lds);
    else
        gemm_f32<B, false, false>(p.w, blockIdx.x - p.x_blocks, (RAR_LDS char *)lds);
#endif
}

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------
//
// For up to R rows of x the layer is bound by reading W once, and what counts
// is how much of W is in flight.  A workgroup takes 64 columns and all of K:
// the lanes of a wave read whole 128-byte lines of several rows of W, a lane
// kGemvK consecutive k of its columns and the same k of x in one vector each.
// Partial sums are joined by lane exchanges and through LDS, in an order fixed
// by the sizes; nothing passes through memory.
// 2048 -> 8192 in bf16, one row: 11 us, 3.1 TB/s, with 128 workgroups on the 256
// units and the waves waiting 54% of their cycles; 8.5 where W is left in the
// Infinity Cache, as for the figures that follow.  This kernel and the tiled
// product with its join, for 1, 2 and 4 rows: 2048 -> 8192 bf16 8.5, 10 and 14
// against 15 us, binary32 14.6, 15.2 and 16.7 against 27; 2048 -> 2048 bf16 7.5,
// 8.8 and 12.5 against 12 to 13.5; 512 -> 512 bf16 5.5, 6.8 and 9.4 against 14.
// Eight rows in one pass took 13 to 45, more than the tiles.  Deep narrow layers
// would do better in tiles: 8192 -> 2048 bf16 20.5, 23 and 28 against 20 to 23.
constexpr int kGemvCols = 64, kGemvK = 8;  // 32 columns a workgroup measured the same

template <class T, int E>
__device__ __forceinline__ float element(const u32x4 (&v)[E], int i)
{
    if (sizeof(T) == 4)
        return __uint_as_float(v[i / 4][i % 4]);
    return __uint_as_float(i % 2 ? v[i / 8][i / 2 % 4] & 0xffff0000u : v[i / 8][i / 2 % 4] << 16);
}

template <class T, int R, bool VEC>
__global__ void __launch_bounds__(1024) rar_gemv(const GemmParams p)
{
    constexpr int kPer = 16 / sizeof(T);               // columns of a lane
    constexpr int kLanes = kGemvCols / kPer;           // lanes of a row of W
    constexpr int kGroups = 64 / kLanes;               // rows of W a wave reads at once
    constexpr int kWaves = 16;
    __shared__ float sums[kWaves][R][kGemvCols];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int q = lane % kLanes, g = lane / kLanes;
    const int64_t n0 = (int64_t)blockIdx.x * kGemvCols;
    const T *const w = (const T *)p.b + n0;
    const T *x[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
        x[r] = (const T *)p.a + (r < p.M ? r : 0) * p.lda;
    float acc[R][kPer] = {};
    // columns of this lane: neighbours, or kLanes apart where W is read by the element
    const auto column = [&](int i) __attribute__((always_inline)) { return VEC ? q * kPer + i : q + i * kLanes; };
    const bool live = n0 + column(0) < p.N;            // vectors are inside or outside as a whole
    int64_t k = (wave * kGroups + g) * kGemvK;
    constexpr int kStride = kWaves * kGroups * kGemvK;
    if constexpr (VEC) {
        constexpr int kUnroll = R > 2 ? 1 : 2;
#pragma unroll kUnroll
        for (; k + kGemvK <= p.K; k += kStride) {
            u32x4 wv[kGemvK][1], xv[R][kGemvK / kPer];
            const T *const at = w + k * p.ldb + q * kPer;
#pragma unroll
            for (int j = 0; j < kGemvK; ++j)
                wv[j][0] = live ? *reinterpret_cast<const u32x4_any *>(at + j * p.ldb) : u32x4{0, 0, 0, 0};
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int j = 0; j < kGemvK / kPer; ++j)
                    xv[r][j] = *reinterpret_cast<const u32x4_any *>(x[r] + k + j * kPer);
#pragma unroll
            for (int j = 0; j < kGemvK; ++j)
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const float e = element<T>(wv[j], i);
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        acc[r][i] = __builtin_fmaf(element<T>(xv[r], j), e, acc[r][i]);
                }
        }
    }
    // by the element: the end of K, and everything where rows are not whole vectors
#pragma unroll 1
    for (; k < p.K; k += kStride)
#pragma unroll 4
        for (int64_t kk = k; kk < (k + kGemvK < p.K ? k + kGemvK : p.K); ++kk)
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float e = n0 + column(i) < p.N ? to_f32(w[kk * p.ldb + column(i)]) : 0.0f;
#pragma unroll
                for (int r = 0; r < R; ++r)
                    acc[r][i] = __builtin_fmaf(to_f32(x[r][kk]), e, acc[r][i]);
            }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
#pragma unroll
            for (int d = kLanes; d < 64; d *= 2)
                acc[r][i] += __shfl_xor(acc[r][i], d);
            if (g == 0)
                sums[wave][r][column(i)] = acc[r][i];
        }
    __syncthreads();
    if (threadIdx.x >= 64)
        return;
    // a few lanes finish a row, four of them a group of a checkpoint
    constexpr int kEnd = kGemvCols / 8;
    const int r = lane / kEnd;
    float v[8] = {};
    if (r < R)
#pragma unroll
        for (int s = 0; s < kWaves; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] += sums[s][r][lane % kEnd * 8 + i];
    epilogue<T>(p, r < R ? r : p.M, n0 + lane % kEnd * 8, v);
}

// Partial products of a split reduction, joined in the order of the splits:
// the result does not depend on which workgroup finished first.
template <class T>
__device__ __forceinline__ void join(const GemmParams &p, int64_t block)
{
    const int64_t per_row = p.pitch / 8;  // pitch is whole groups, so a group's four lanes are neighbours
    const int64_t g = block * 256 + threadIdx.x;
    const int64_t m = g / per_row, n = (g - m * per_row) * 8;
    float v[8] = {};
    if (m < p.M && n < p.N) {
        const float *at = p.part + m * p.pitch + n;
        for (int s = 0; s < p.splits; ++s, at += p.M * p.pitch) {
            const f32x4 lo = load4(at), hi = load4(at + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] += lo[i];
                v[4 + i] += hi[i];
            }
        }
    }
    epilogue<T>(p, m, n, v);
}

// ---------------------------------------------------------------------------
// Streaming passes
// ---------------------------------------------------------------------------

// A copy with whole 16-byte rows for operands whose rows are not: the products'
// loads into LDS take 16 aligned bytes.  A streaming pass, 3.4 us for a layer
// of 333 x 501 -> 259; the products it feeds take 11.5.
// Two matrices in one launch, the second's rows behind the first's; a
// workgroup takes every gridDim.x-th row.
template <class T>
__global__ void __launch_bounds__(256) rar_pack_rows(const PackParams first, const PackParams second)
{
    for (int64_t at = blockIdx.x; at < first.rows + second.rows; at += gridDim.x) {
        const bool is_second = at >= first.rows;
        const PackParams &p = is_second ? second : first;
        const int64_t row = at - (is_second ? first.rows : 0);
        const T *src = (const T *)p.src + row * p.ld;
        T *dst = (T *)p.dst + row * p.pitch;
        for (int64_t c = (int64_t)blockIdx.y * 2048 + threadIdx.x * 8; c < p.pitch; c += (int64_t)gridDim.y * 2048) {
            float v[8];
            load8(src + c, p.cols - c < 8 ? (p.cols - c < 0 ? 0 : (int)(p.cols - c)) : 8, v);
            store8(dst + c, p.pitch - c < 8 ? (int)(p.pitch - c) : 8, v);
        }
    }
}

// dz = dy * act'(z) and the column sums of dz in one pass over dy and z.  A
// workgroup takes 512 columns (a lane eight, a wave four rows at a time, so
// that eight 16-byte loads are in flight) of rows_per_chunk rows; its sums go
// to part[chunk], joined in chunk order by rar_column_sum.  Sums are of the
// binary32 dz; the dz that the matrix products read is rounded to the layer's
// type.
// 8192 x 8192 in bf16, gelu: 82 us, 406 MB at 5 TB/s; z in 8 bits 79 us, 341 MB at
// 4.3 TB/s.
enum DzSource { kDzNone = 0, kDzPre = 1, kDzCkpt = 2 };
constexpr int kDzRows = 4;

template <class T, int ACT, int SOURCE>
__global__ void __launch_bounds__(256) rar_dz(const DzParams p)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 512 + lane * 8;
    const int64_t r0 = (int64_t)blockIdx.y * p.rows_per_chunk;
    const int64_t r1 = r0 + p.rows_per_chunk < p.rows ? r0 + p.rows_per_chunk : p.rows;
    const int cnt = p.cols - c < 8 ? (p.cols - c < 0 ? 0 : (int)(p.cols - c)) : 8;
    const int put = p.pitch - c < 8 ? (p.pitch - c < 0 ? 0 : (int)(p.pitch - c)) : 8;
    const int64_t groups = (p.cols + kCkptGroup - 1) / kCkptGroup;
    float sum[8] = {};
    for (int64_t r = r0 + wave; r < r1; r += 4 * kDzRows) {
        float d[kDzRows][8], z[kDzRows][8];
        u32x2 w[kDzRows];
        uint32_t e[kDzRows];
#pragma unroll
        for (int u = 0; u < kDzRows; ++u) {
            const int64_t row = r + 4 * u;
            const int n = row < r1 ? cnt : 0;
            load8<true>((const T *)p.dy + row * p.ldy + c, n, d[u]);
            if (SOURCE == kDzPre)
                load8<true>((const T *)p.pre + row * p.ldp + c, n, z[u]);
            w[u] = u32x2{0, 0};
            e[u] = 0;
            if (SOURCE == kDzCkpt && n > 0) {
                w[u] = load_once((const u32x2 *)((const uint8_t *)p.pre + row * groups * kCkptGroup + c));
                e[u] = p.pre_scales[row * groups + c / kCkptGroup];
            }
        }
#pragma unroll
        for (int u = 0; u < kDzRows; ++u) {
            const int64_t row = r + 4 * u;
            if (row >= r1)
                continue;
            if (SOURCE == kDzCkpt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const f32x4 x = ckpt_values4(w[u][h], e[u]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        z[u][4 * h + i] = x[i];
                }
            if (SOURCE != kDzNone)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[u][i] *= act_grad<T>(ACT, z[u][i]);
            if (SOURCE == kDzCkpt && cnt < 8)  // codes behind the matrix may hold anything
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[u][i] = i < cnt ? d[u][i] : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum[i] += d[u][i];
            if (p.dz)
                store8((T *)p.dz + row * p.pitch + c, put, d[u]);
        }
    }
    if (!p.part)
        return;
    __shared__ float sums[4][8][64];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        sums[wave][i][lane] = sum[i];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int j = threadIdx.x + k * 256;  // column of the workgroup
        const int64_t col = (int64_t)blockIdx.x * 512 + j;
        if (col < p.cols)
            p.part[blockIdx.y * p.cols + col] = (sums[0][j % 8][j / 8] + sums[1][j % 8][j / 8]) +
                                                (sums[2][j % 8][j / 8] + sums[3][j % 8][j / 8]);
    }
}

// db: 64 columns a workgroup; each wave sums every fourth chunk.
template <class T>
__device__ __forceinline__ void column_sum(const SumParams &p, int64_t block)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = block * 64 + lane;
    float s = 0.0f;
    if (c < p.cols)
#pragma unroll 16
        for (int64_t k = wave; k < p.chunks; k += 4)
            s += p.part[k * p.cols + c];
    __shared__ float sums[4][64];
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < p.cols) {
        float t = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
        T *out = (T *)p.out + c;
        if (p.accumulate)
            t += to_f32(*out);
        *out = from_f32<T>(t);
    }
}

// What is left after the products, in one launch: the joins of split
// reductions and db.
template <class T>
__global__ void __launch_bounds__(256) rar_finish(const FinishParams p)
{
    int64_t block = blockIdx.x;
    if (block < p.a_blocks) {
        join<T>(p.a, block);
        return;
    }
    block -= p.a_blocks;
    if (block < p.b_blocks) {
        join<T>(p.b, block);
        return;
    }
    column_sum<T>(p.sum, block - p.b_blocks);
}

}  // namespace

hipError_t launch_forward(rar_dtype dt, const GemmParams &p, int tile, hipStream_t st)
{
    const unsigned grid = blocks_of(p);
    if (dt == RAR_BF16)
        return tile == 256 ? launch(rar_forward_bf16<256, 2, 4>, grid, 512, st, p)
                           : launch(rar_forward_bf16<128, 2, 2>, grid, 256, st, p);
    return launch(tile == 128 ? rar_forward_f32<128> : rar_forward_f32<64>, grid, 256, st, p);
}

hipError_t launch_backward(rar_dtype dt, const GemmPair &p, unsigned w_blocks, int tile, hipStream_t st)
{
    const unsigned grid = p.x_blocks + w_blocks;
    if (dt == RAR_BF16)
        return tile == 256 ? launch(rar_backward_bf16<256, 2, 4>, grid, 512, st, p)
                           : launch(rar_backward_bf16<128, 2, 2>, grid, 256, st, p);
    return launch(tile == 128 ? rar_backward_f32<128> : rar_backward_f32<64>, grid, 256, st, p);
}

namespace {

template <class T, bool VEC>
hipError_t run_gemv(const GemmParams &p, unsigned grid, hipStream_t st)
{
    return launch(p.M == 1   ? rar_gemv<T, 1, VEC>
                  : p.M == 2 ? rar_gemv<T, 2, VEC>
                             : rar_gemv<T, kGemvRows, VEC>,
                  grid, 1024, st, p);
}

}  // namespace

hipError_t launch_gemv(rar_dtype dt, const GemmParams &p, bool vec, hipStream_t st)
{
    const unsigned grid = (unsigned)((p.N + kGemvCols - 1) / kGemvCols);
    if (dt == RAR_BF16)
        return vec ? run_gemv<bf16, true>(p, grid, st) : run_gemv<bf16, false>(p, grid, st);
    return vec ? run_gemv<float, true>(p, grid, st) : run_gemv<float, false>(p, grid, st);
}

hipError_t launch_pack(rar_dtype dt, const PackParams &a, const PackParams &b, hipStream_t st)
{
    const int64_t pitch = a.pitch > b.pitch ? a.pitch : b.pitch;
    const int64_t rows = a.rows + b.rows;
    const dim3 grid((unsigned)(rows < (1 << 20) ? rows : 1 << 20),  // a grid holds 2^32 lanes along x
                    (unsigned)((pitch + 2047) / 2048 < 64 ? (pitch + 2047) / 2048 : 64));
    return launch(dt == RAR_BF16 ? rar_pack_rows<bf16> : rar_pack_rows<float>, grid, 256, st, a, b);
}

namespace {

template <class T>
hipError_t run_dz(const DzParams &p, dim3 grid, hipStream_t st)
{
    void (*kernel)(DzParams) = rar_dz<T, RAR_ACT_NONE, kDzNone>;
    if (p.act == RAR_ACT_RELU)
        kernel = p.pre_scales ? rar_dz<T, RAR_ACT_RELU, kDzCkpt> : rar_dz<T, RAR_ACT_RELU, kDzPre>;
    else if (p.act == RAR_ACT_GELU)
        kernel = p.pre_scales ? rar_dz<T, RAR_ACT_GELU, kDzCkpt> : rar_dz<T, RAR_ACT_GELU, kDzPre>;
    return launch(kernel, grid, 256, st, p);
}

}  // namespace

hipError_t launch_dz(rar_dtype dt, const DzParams &p, hipStream_t st)
{
    const int64_t width = p.dz && p.pitch > p.cols ? p.pitch : p.cols;
    const dim3 grid((unsigned)((width + 511) / 512), (unsigned)((p.rows + p.rows_per_chunk - 1) / p.rows_per_chunk));
    return dt == RAR_BF16 ? run_dz<bf16>(p, grid, st) : run_dz<float>(p, grid, st);
}

hipError_t launch_finish(rar_dtype dt, const FinishParams &p, hipStream_t st)
{
    const unsigned grid = p.a_blocks + p.b_blocks + (unsigned)((p.sum.cols + 63) / 64);
    return launch(dt == RAR_BF16 ? rar_finish<bf16> : rar_finish<float>, grid, 256, st, p);
}

}  // namespace rar
