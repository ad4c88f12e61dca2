// embed.hip -- CDNA4 (gfx950) kernels of the embedding: lookup with scaling, and
// its gradient by sorted tokens.
//
// Lookup: out[t] = scale * table[ids[t]], a gather bound by HBM bandwidth: 65536
// rows of 2048 bf16, 59 us for 131 MB of distinct rows and 268 MB of out (6.8
// TB/s).  out is written past the caches, which pays for large calls and costs
// the reader of small ones up to 3%.  Lookup alone and with the 2048 -> 2048
// product that reads out, in brackets with ordinary stores: 65536 rows 59 and
// 523 us (82 and 542), 4096 rows 5.6 and 51 (6.7 and 49), 512 rows 4.0 and 29.4
// (4.3 and 28.7).
//
// Gradient: grad[v] = scale * sum of dy[t] over the t with ids[t] == v, dense
// (every row of the vocabulary is written) or accumulated into the rows that
// occur.  The token positions are sorted by id, stably, so each row's terms
// stand together in token order; no floating-point atomic is used and the
// result does not depend on timing.  Then one wave sums every 32 (or 8) sorted
// positions of 512 columns, whatever ids they hold: dy is read once, evenly,
// however often a token occurs.  A run of one id inside a chunk is finished
// there; the parts of a run that crosses chunks go to memory and are added in
// order, of long runs first 32 at a time.  The order of the terms depends on
// the ids alone.
//
// Bound: dy read once, grad written once; the sort moves 16 bytes a token, and
// its launches also clear the gradient.  65536 tokens of 2048 bf16 columns into
// 32000 rows: 121 us, of them the sort with the clearing 39 (16 workgroups of
// 4096 keys, two passes), the chunks 68 (268 MB of dy read, 72 MB of finished and
// partial rows written, 5.0 TB/s together), the joins 16.
#include "act.h"
#include "ops_internal.h"

#pragma clang fp contract(off)

namespace rar {
namespace {

// ---------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------

// 16-byte vectors of a row, or single elements where rows are not whole
// vectors.  The workgroup's first row is found by one uniform division.
template <class T, bool VEC>
__global__ void __launch_bounds__(256) rar_embed_rows(const EmbedParams p)
{
    constexpr int kPer = VEC ? 16 / sizeof(T) : 1;
    constexpr int kPasses = 4;
    const uint32_t nv = (uint32_t)(p.D / kPer);
    const int64_t first = (int64_t)blockIdx.x * (256 * kPasses);
    const int64_t row0 = first / nv;
    const uint32_t rem = (uint32_t)(first - row0 * nv);
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
        const uint32_t g = rem + u * 256 + threadIdx.x;
        const uint32_t dr = g / nv;
        const int64_t row = row0 + dr;
        if (row >= p.T)
            return;
        const int64_t c = (int64_t)(g - dr * nv) * kPer;
        const int64_t id = p.ids[row];
        const bool ok = id >= 0 && id < p.V;
        const T *src = (const T *)p.table + (ok ? id : 0) * p.D + c;
        T *dst = (T *)p.out + row * p.ldo + c;
        if constexpr (!VEC) {
            *dst = from_f32<T>(ok ? to_f32(*src) * p.scale : 0.0f);
        } else if constexpr (sizeof(T) == 4) {
            const f32x4 v = *reinterpret_cast<const f32x4_any *>(src);
            __builtin_nontemporal_store(ok ? v * p.scale : f32x4{0.0f, 0.0f, 0.0f, 0.0f},
                                        reinterpret_cast<f32x4_any *>(dst));
        } else {
            const u32x4 w = *reinterpret_cast<const u32x4_any *>(src);
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
                o[i] = ok ? pack_bf16(lo * p.scale, hi * p.scale) : 0u;
            }
            __builtin_nontemporal_store(o, reinterpret_cast<u32x4_any *>(dst));
        }
    }
}

// ---------------------------------------------------------------------------
// Stable sort of token positions by id, eight bits a pass
// ---------------------------------------------------------------------------

constexpr int kSortThreads = 1024;                      // sixteen waves
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kRounds = 4;                              // keys of a lane
constexpr int kSortKeys = kRounds * kSortThreads;       // keys of a workgroup
// Batches that one workgroup sorts.  The whole call with one workgroup and with
// one for every 4096 keys: 2000 tokens of 509 binary32 columns 20 and 29 us, 4096
// 27 and 36, 8192 38 and 42; 8192 of 2048 bf16 columns 51 and 60.  Up to 1024 they
// take the same; more than 8192 in one were not measured.
constexpr int kSmallKeys = 2 * kSortKeys;
constexpr int kGroup = 32;                              // chunks of a long run that are added beforehand

__device__ __forceinline__ uint32_t key_of(int64_t id, int64_t V)
{
    return id >= 0 && id < V ? (uint32_t)id : (uint32_t)V;  // ids outside the vocabulary sort last
}

struct SortShared {
    uint32_t count[kSortWaves][256];
    uint32_t base[256];
    uint32_t scan[4];
};

// Ranks of this wave's keys among the wave's equal digits (in order), counting
// them in count[wave].  Lanes with `live` false take no part.
template <int N>
__device__ __forceinline__ void wave_ranks(SortShared &s, const uint32_t (&digit)[N], const bool (&live)[N],
                                           uint32_t (&rank)[N], int rounds, int bits)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < kSortWaves * 256; i += kSortThreads)
        (&s.count[0][0])[i] = 0;
    __syncthreads();
    volatile uint32_t *count = s.count[wave];
#pragma unroll
    for (int r = 0; r < N; ++r) {
        if (r >= rounds)
            break;
        uint64_t peers = __ballot(live[r]);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((digit[r] >> b) & 1);
            peers &= (digit[r] >> b) & 1 ? set : ~set;
        }
        const uint32_t before = live[r] ? count[digit[r]] : 0;
        const uint32_t mine = __popcll(peers & ((1ull << lane) - 1));
        __builtin_amdgcn_wave_barrier();
        if (live[r] && mine == 0)
            count[digit[r]] = before + __popcll(peers);
        __builtin_amdgcn_wave_barrier();
        rank[r] = before + mine;
    }
    __syncthreads();
}

// count[w][d] becomes the number of digit d in earlier waves; returns (threads
// below 256) the workgroup's total of digit d = threadIdx.x.
__device__ __forceinline__ uint32_t scan_waves(SortShared &s)
{
    uint32_t run = 0;
    if (threadIdx.x < 256) {
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t c = s.count[w][threadIdx.x];
            s.count[w][threadIdx.x] = run;
            run += c;
        }
    }
    return run;
}

// base[d] = add + the sum of v over the digits below d (threads below 256).
__device__ __forceinline__ void scan_digits(SortShared &s, uint32_t v, uint32_t add)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t inc = v;
    if (threadIdx.x < 256) {
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint32_t o = __shfl_up(inc, d);
            inc += lane >= d ? o : 0;
        }
        if (lane == 63)
            s.scan[wave] = inc;
    }
    __syncthreads();
    if (threadIdx.x < 256) {
        for (int w = 0; w < wave; ++w)
            inc += s.scan[w];
        s.base[threadIdx.x] = inc - v + add;
    }
    __syncthreads();
}

// The gradient's rows are cleared by workgroups beside the sort's, which leaves
// the memory idle: share `part` of `parts` of the bytes, kClearBytes a
// workgroup.
constexpr int64_t kClearBytes = 64 * 1024;

struct Clear {
    char *at;
    int64_t bytes;
};

__device__ __forceinline__ void clear(const Clear &c, int64_t block)
{
    const int64_t lo = block * kClearBytes, hi = lo + kClearBytes < c.bytes ? lo + kClearBytes : c.bytes;
    // whole 16-byte groups, and what lies before and behind them by two bytes
    const int64_t a = lo + (16 - (int64_t)((uintptr_t)(c.at + lo) & 15)) % 16;
    const int64_t b = hi - (int64_t)((uintptr_t)(c.at + hi) & 15);
    if (a > b) {
        for (int64_t i = lo + threadIdx.x * 2; i < hi; i += kSortThreads * 2)
            *reinterpret_cast<uint16_t *>(c.at + i) = 0;
        return;
    }
    if (lo + threadIdx.x * 2 < a)
        *reinterpret_cast<uint16_t *>(c.at + lo + threadIdx.x * 2) = 0;
    if (b + threadIdx.x * 2 < hi)
        *reinterpret_cast<uint16_t *>(c.at + b + threadIdx.x * 2) = 0;
    for (int64_t i = a + threadIdx.x * 16; i < b; i += kSortThreads * 16)
        store_once(reinterpret_cast<u32x4 *>(c.at + i), u32x4{0, 0, 0, 0});
}

// A whole batch of at most N * kSortThreads tokens in one workgroup, a wave
// `rounds` times 64 of them in a row.
template <int N>
__global__ void __launch_bounds__(kSortThreads) rar_sort_small(const int64_t *ids, int T, int64_t V, int passes,
                                                               int bits, uint32_t *keys, uint32_t *pos, Clear c)
{
    if (blockIdx.x > 0) {
        clear(c, blockIdx.x - 1);
        return;
    }
    __shared__ SortShared s;
    __shared__ uint32_t k_lds[N * kSortThreads], p_lds[N * kSortThreads];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t key[N], at[N], digit[N], rank[N];
    bool live[N];
    const int rounds = (T + kSortThreads - 1) / kSortThreads;
#pragma unroll
    for (int r = 0; r < N; ++r) {
        const int i = wave * (64 * rounds) + r * 64 + lane;
        live[r] = r < rounds && i < T;
        key[r] = live[r] ? key_of(ids[i], V) : 0;
        at[r] = i;
    }
    for (int pass = 0; pass < passes; ++pass) {
#pragma unroll
        for (int r = 0; r < N; ++r)
            digit[r] = (key[r] >> (bits * pass)) & ((1u << bits) - 1);
        wave_ranks(s, digit, live, rank, rounds, bits);
        const uint32_t total = scan_waves(s);
        scan_digits(s, total, 0);
#pragma unroll
        for (int r = 0; r < N; ++r)
            if (live[r]) {
                const uint32_t to = s.base[digit[r]] + s.count[wave][digit[r]] + rank[r];
                k_lds[to] = key[r];
                p_lds[to] = at[r];
            }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < N; ++r) {
            const int i = wave * (64 * rounds) + r * 64 + lane;
            if (live[r]) {
                key[r] = k_lds[i];
                at[r] = p_lds[i];
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < N; ++r) {
        const int i = wave * (64 * rounds) + r * 64 + lane;
        if (live[r]) {
            keys[i] = key[r];
            pos[i] = at[r];
        }
    }
}

// Larger batches: digit counts of each kSortKeys tokens, then their placement,
// for which every workgroup adds up all workgroups' counts.  That is a read of
// 16 KB a workgroup at 65536 tokens and of 4 MB at 2^24: a placement takes 11 us at
// 2^16 tokens, 31 at 2^20 and 2.2 ms at 2^24, where it is most of the call.
__global__ void __launch_bounds__(kSortThreads) rar_sort_count(const int64_t *ids, const uint32_t *keys, int64_t T,
                                                               int64_t V, int shift, int bits, uint32_t *hist,
                                                               unsigned blocks, Clear c)
{
    if (blockIdx.x >= blocks) {
        clear(c, blockIdx.x - blocks);
        return;
    }
    __shared__ uint32_t count[256];
    if (threadIdx.x < 256)
        count[threadIdx.x] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * kSortKeys;
    for (int i = threadIdx.x; i < kSortKeys; i += kSortThreads)
        if (first + i < T) {
            const uint32_t key = ids ? key_of(ids[first + i], V) : keys[first + i];
            atomicAdd(&count[(key >> shift) & ((1u << bits) - 1)], 1u);
        }
    __syncthreads();
    if (threadIdx.x < 256)
        hist[(int64_t)blockIdx.x * 256 + threadIdx.x] = count[threadIdx.x];
}

__global__ void __launch_bounds__(kSortThreads) rar_sort_place(const int64_t *ids, const uint32_t *keys,
                                                               const uint32_t *pos, int64_t T, int64_t V, int shift,
                                                               int bits,
                                                               const uint32_t *hist, uint32_t *keys_out,
                                                               uint32_t *pos_out, unsigned blocks, Clear c)
{
    if (blockIdx.x >= blocks) {
        clear(c, blockIdx.x - blocks);
        return;
    }
    __shared__ SortShared s;
    __shared__ uint32_t part[2][4][256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t first = (int64_t)blockIdx.x * kSortKeys;
    uint32_t key[kRounds], at[kRounds], digit[kRounds], rank[kRounds];
    bool live[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int64_t i = first + wave * (64 * kRounds) + r * 64 + lane;
        live[r] = i < T;
        key[r] = live[r] ? (ids ? key_of(ids[i], V) : keys[i]) : 0;
        at[r] = live[r] ? (ids ? (uint32_t)i : pos[i]) : 0;
        digit[r] = (key[r] >> shift) & ((1u << bits) - 1);
    }
    // digit totals of all workgroups and of those before this one
    const int d = threadIdx.x & 255, quarter = threadIdx.x >> 8;
    uint32_t all = 0, before = 0;
    for (int b = quarter; b < (int)blocks; b += 4) {
        const uint32_t c = hist[(int64_t)b * 256 + d];
        all += c;
        before += b < (int)blockIdx.x ? c : 0;
    }
    part[0][quarter][d] = all;
    part[1][quarter][d] = before;
    wave_ranks(s, digit, live, rank, kRounds, bits);  // synchronises
    scan_waves(s);
    uint32_t total = 0, mine = 0;
    if (threadIdx.x < 256) {
        total = part[0][0][d] + part[0][1][d] + part[0][2][d] + part[0][3][d];
        mine = part[1][0][d] + part[1][1][d] + part[1][2][d] + part[1][3][d];
    }
    scan_digits(s, total, mine);
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
        if (live[r]) {
            const uint32_t to = s.base[digit[r]] + s.count[wave][digit[r]] + rank[r];
            keys_out[to] = key[r];
            pos_out[to] = at[r];
        }
}

// ---------------------------------------------------------------------------
// Sums
// ---------------------------------------------------------------------------

// A wave sums a strip of kCols columns.  Column of lane l's i-th value: l * 8 +
// i where rows are whole eights, else i * 64 + l, so that either
// way a wave reads consecutive memory.
constexpr int kCols = 512;

struct GradWs {
    uint32_t *keys, *pos;  // sorted
    // [chunk][pitch]: the part of a run that crosses into the chunk from the
    // left, and of one that starts in it and goes on to the right; [group]: the
    // sum of kGroup aligned chunks' `from_left` that hold one id
    float *from_left, *to_right, *long_run;
    int64_t pitch;         // whole strips, in the lanes' order
    int chunk;             // sorted positions that a wave sums
};

// Eight values of a row as they were loaded: widened only when they are added,
// which halves the registers of bf16 rows in flight.
template <class T, bool VEC>
struct Raw {
    T v[8];
    __device__ __forceinline__ float at(int i) const { return to_f32(v[i]); }
};

template <class T>
struct Raw<T, true> {
    u32x4 v[sizeof(T) / 2];
    __device__ __forceinline__ float at(int i) const
    {
        if (sizeof(T) == 4)
            return __uint_as_float(v[i / 4][i % 4]);
        return __uint_as_float(i % 2 ? v[0][i / 2] & 0xffff0000u : v[0][i / 2] << 16);
    }
};

template <class T, bool VEC>
struct Columns {
    int64_t c0;  // first column of the strip
    int64_t D;

    __device__ __forceinline__ int64_t col(int i) const
    {
        const int lane = threadIdx.x & 63;
        return c0 + (VEC ? lane * 8 + i : i * 64 + lane);
    }

    __device__ __forceinline__ void load(const T *row, Raw<T, VEC> &v) const
    {
        if constexpr (VEC) {
            // D is whole eights; lanes behind it read the row's first values
            const u32x4_any *p = reinterpret_cast<const u32x4_any *>(row + (col(0) < D ? col(0) : 0));
#pragma unroll
            for (int h = 0; h < (int)sizeof(T) / 2; ++h)
                v.v[h] = __builtin_nontemporal_load(p + h);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v.v[i] = row[col(i) < D ? col(i) : 0];
        }
    }

    // Partial rows are kept in the lanes' order: eight consecutive floats a lane.
    __device__ __forceinline__ int64_t place() const { return c0 + (threadIdx.x & 63) * 8; }

    __device__ __forceinline__ void add_partials(const float *part, int64_t pitch, int64_t at, int64_t n,
                                                 float (&acc)[8]) const
    {
        const float *row = part + at * pitch + place();
#pragma unroll 8
        for (int64_t i = 0; i < n; ++i, row += pitch) {
            const f32x4 a = load4(row), b = load4(row + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[e] += a[e];
                acc[4 + e] += b[e];
            }
        }
    }

    __device__ __forceinline__ void put_partial(float *row, const float (&acc)[8]) const
    {
        store4(row + place(), f32x4{acc[0], acc[1], acc[2], acc[3]});
        store4(row + place() + 4, f32x4{acc[4], acc[5], acc[6], acc[7]});
    }

    // The finished sum of row `key` of the gradient.
    __device__ __forceinline__ void put_row(const EmbedGradParams &p, uint32_t key, float (&acc)[8]) const
    {
        T *out = (T *)p.grad + (int64_t)key * D;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[i] *= p.scale;
        if (p.accumulate) {
            Raw<T, VEC> old;
            load(out, old);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[i] += old.at(i);
        }
        if constexpr (VEC) {
            store8<true>(out + col(0), col(0) < D ? 8 : 0, acc);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col(i) < D)
                    out[col(i)] = from_f32<T>(acc[i]);
        }
    }
};

__device__ __forceinline__ int64_t wave_job(int64_t block)
{
    return block * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// One wave: a chunk of sorted positions of one strip, two batches of rows in
// flight.
template <class T, bool VEC>
__global__ void __launch_bounds__(256) rar_embed_chunks(const EmbedGradParams p, const GradWs w, int strips)
{
    const int lane = threadIdx.x & 63;
    const int64_t job = wave_job(blockIdx.x);
    const int64_t chunk = job / strips;
    const int64_t at = chunk * w.chunk;
    if (at >= p.T)
        return;
    // lane l: position at - 1 + l, for one position on either side of the chunk
    const int64_t i = at - 1 + lane;
    const bool have = i >= 0 && i < p.T && lane <= w.chunk + 1;
    const uint32_t none = 0xffffffffu;
    const uint32_t key = have ? w.keys[i] : none;
    const uint32_t pos = have ? w.pos[i] : 0;
    // ids outside the vocabulary stand at the end
    const int n = __popcll(__ballot(lane >= 1 && lane <= w.chunk && key < (uint32_t)p.V));
    if (n == 0)
        return;
    const Columns<T, VEC> cols{(job - chunk * strips) * kCols, p.D};
    const T *dy = (const T *)p.dy;
    float acc[8] = {};
    bool left = __builtin_amdgcn_readlane(key, 0) == __builtin_amdgcn_readlane(key, 1);
    constexpr int B = sizeof(Raw<T, VEC>) <= 16 ? 8 : 4;  // rows of a batch
    const auto fetch = [&](Raw<T, VEC>(&v)[B], int r) __attribute__((always_inline)) {
        // the last row again in place of rows behind it: no branch between the loads
#pragma unroll
        for (int u = 0; u < B; ++u)
            cols.load(dy + (int64_t)(uint32_t)__builtin_amdgcn_readlane(pos, 1 + (r + u < n ? r + u : n - 1)) * p.ldy,
                      v[u]);
    };
    const auto add = [&](const Raw<T, VEC>(&v)[B], int r) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < B; ++u) {
            if (r + u >= n)
                break;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                acc[e] += v[u].at(e);
            const uint32_t k = __builtin_amdgcn_readlane(key, 1 + r + u);
            const uint32_t next = __builtin_amdgcn_readlane(key, 2 + r + u);
            const bool right = r + u == n - 1 && k == next;
            if (k == next && !right)
                continue;
            if (left)
                cols.put_partial(w.from_left + chunk * w.pitch, acc);
            else if (right)
                cols.put_partial(w.to_right + chunk * w.pitch, acc);
            else
                cols.put_row(p, k, acc);
            left = false;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                acc[e] = 0.0f;
        }
    };
    // A batch is loaded before the one before it is added: loads that follow
    // that one's stores would wait for them.
    Raw<T, VEC> v0[B], v1[B];
    fetch(v0, 0);
    for (int r = 0; r < n; r += 2 * B) {
        fetch(v1, r + B);
        add(v0, r);
        if (r + B >= n)
            break;
        fetch(v0, r + 2 * B);
        add(v1, r + B);
    }
}

// The sum of kGroup aligned chunks that hold one id which came in from the left.
__global__ void __launch_bounds__(256) rar_embed_long(const EmbedGradParams p, const GradWs w, int strips)
{
    const int64_t len = (int64_t)kGroup * w.chunk;
    const int64_t job = wave_job(blockIdx.x);
    const int64_t group = job / strips;
    const int64_t at = group * len;
    if (at + len > p.T || at == 0)
        return;
    const uint32_t k = w.keys[at];
    if (k >= (uint32_t)p.V || k != w.keys[at - 1] || k != w.keys[at + len - 1])
        return;
    const Columns<float, true> cols{(job - group * strips) * kCols, p.D};
    float acc[8] = {};
    cols.add_partials(w.from_left, w.pitch, group * kGroup, kGroup, acc);
    cols.put_partial(w.long_run + group * w.pitch, acc);
}

// Runs that cross chunks: the wave of the chunk in which a run starts adds its
// parts in order.
template <class T, bool VEC>
__global__ void __launch_bounds__(256) rar_embed_join(const EmbedGradParams p, const GradWs w, int strips)
{
    const int lane = threadIdx.x & 63;
    const int64_t job = wave_job(blockIdx.x);
    const int64_t chunk = job / strips;
    const int64_t next = (chunk + 1) * w.chunk;
    if (next >= p.T)
        return;
    const uint32_t k = w.keys[next];
    if (k >= (uint32_t)p.V || w.keys[next - 1] != k)
        return;
    // a run that also fills this chunk from the left starts in an earlier one
    if (chunk > 0 && w.keys[chunk * w.chunk - 1] == k)
        return;
    // the last chunk whose first position still holds the id
    int64_t last = chunk;
    for (;;) {
        const int64_t c = last + 1 + lane;
        const uint64_t same = __ballot(c * w.chunk < p.T && w.keys[c * w.chunk < p.T ? c * w.chunk : 0] == k);
        const int run = __builtin_ctzll(~same | (1ull << 63)) + (same == ~0ull ? 1 : 0);
        last += run;
        if (run < 64)
            break;
    }
    const Columns<T, VEC> cols{(job - chunk * strips) * kCols, p.D};
    float acc[8] = {};
    cols.add_partials(w.to_right, w.pitch, chunk, 1, acc);
    int64_t c = chunk + 1;
    while (c <= last) {
        // whole aligned groups: the run fills all but its last chunk
        if (c % kGroup == 0 && last - c >= kGroup) {
            const int64_t n = (last - c) / kGroup;
            cols.add_partials(w.long_run, w.pitch, c / kGroup, n, acc);
            c += n * kGroup;
        } else {
            int64_t n = kGroup - c % kGroup;
            n = n < last - c + 1 ? n : last - c + 1;
            cols.add_partials(w.from_left, w.pitch, c, n, acc);
            c += n;
        }
    }
    cols.put_row(p, k, acc);
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Byte offsets of the workspace's parts.
struct Layout {
    int64_t keys[2], pos[2], hist, from_left, to_right, long_run, total, pitch;
    int chunk;
};

Layout layout(int64_t T, int64_t D)
{
    Layout l{};
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += up(bytes, 256);
        return here;
    };
    l.pitch = up(D, kCols);
    const bool small = T <= kSmallKeys;
    for (int i = 0; i < 2; ++i) {
        l.keys[i] = i && small ? l.keys[0] : take(4 * T);
        l.pos[i] = i && small ? l.pos[0] : take(4 * T);
    }
    l.hist = take(small ? 0 : (T + kSortKeys - 1) / kSortKeys * 1024);
    // A wave sums 32 sorted positions, or 8 where 32 would leave most of the chip
    // without a wave.  The whole call in chunks of 8 and of 32, by positions times
    // strips: 4097 (509 binary32 columns) 29 and 36 us, 8192 (bf16) 36 and 37 to
    // 37 and 42, 16384 (either type) 45 and 45 to 54 and 53, 32768 55 and 48 (bf16)
    // to 94 and 80 (binary32), 65536 68 and 60 to 118 and 107, 262144 139 and 124.
    // The two cross near 16384; between there and the border chunks of 8 cost up to
    // 16%.
    l.chunk = T <= 32 || T * (l.pitch / kCols) >= 65536 ? 32 : 8;  // up to 32 need no join
    const int64_t chunks = T > l.chunk ? (T + l.chunk - 1) / l.chunk : 0;
    l.from_left = take(chunks * l.pitch * 4);
    l.to_right = take(chunks * l.pitch * 4);
    l.long_run = take(T / (kGroup * l.chunk) * l.pitch * 4);
    l.total = at;
    return l;
}

template <class T, bool VEC>
hipError_t sums(const EmbedGradParams &p, const GradWs &w, hipStream_t st)
{
    const int64_t strips = (p.D + kCols - 1) / kCols;
    const int64_t chunks = (p.T + w.chunk - 1) / w.chunk, longs = p.T / (kGroup * w.chunk);
    const auto grid = [strips](int64_t n) { return (unsigned)((n * strips + 3) / 4); };
    hipError_t e = hipSuccess;
    if (chunks > 0)
        e = launch(rar_embed_chunks<T, VEC>, grid(chunks), 256, st, p, w, (int)strips);
    if (e == hipSuccess && longs > 1)  // the first group has nothing on its left
        e = launch(rar_embed_long, grid(longs), 256, st, p, w, (int)strips);
    if (e == hipSuccess && chunks > 1)
        e = launch(rar_embed_join<T, VEC>, grid(chunks - 1), 256, st, p, w, (int)strips);
    return e;
}

}  // namespace

int64_t embed_grad_workspace(int64_t T, int64_t V, int64_t D) { return layout(T, D).total; }

bool embed_grad_fits(int64_t T, int64_t D, int64_t grad_bytes, int64_t lanes)
{
    const int64_t chunks = T / layout(T, D).chunk + 1, strips = (D + kCols - 1) / kCols;
    return (chunks * strips / 4 + 1) * 256 <= lanes &&
           (grad_bytes / kClearBytes + T / kSortKeys + 3) * kSortThreads <= lanes;
}

hipError_t launch_embed_lookup(rar_dtype dt, const EmbedParams &p, hipStream_t st)
{
    const int es = dt == RAR_BF16 ? 2 : 4;
    const bool vec = p.D * es % 16 == 0;  // rows of whole 16-byte groups, at any address
    const int64_t width = vec ? p.D * es / 16 : p.D;
    const int64_t most = (int64_t(1) << 33) / width;  // rows of a launch: a grid holds 2^32 lanes, each four items
    for (int64_t t = 0; t < p.T; t += most) {
        EmbedParams q = p;
        q.ids = p.ids + t;
        q.out = (char *)p.out + t * p.ldo * es;
        q.T = p.T - t < most ? p.T - t : most;
        const unsigned grid = (unsigned)((q.T * width + 1023) / 1024);
        void (*const kernel)(EmbedParams) = dt == RAR_BF16
                                                ? (vec ? rar_embed_rows<bf16, true> : rar_embed_rows<bf16, false>)
                                                : (vec ? rar_embed_rows<float, true> : rar_embed_rows<float, false>);
        const hipError_t e = launch(kernel, grid, 256, st, q);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_embed_grad(rar_dtype dt, const EmbedGradParams &p, hipStream_t st)
{
    const Layout l = layout(p.T, p.D);
    char *const ws = (char *)p.ws;
    uint32_t *keys[2], *pos[2];
    for (int i = 0; i < 2; ++i) {
        keys[i] = (uint32_t *)(ws + l.keys[i]);
        pos[i] = (uint32_t *)(ws + l.pos[i]);
    }
    int width = 0;  // bits of the keys 0..V
    while (width < 32 && (p.V >> width) != 0)
        ++width;
    const int passes = (width + 7) / 8, bits = (width + passes - 1) / passes;
    // the gradient in as many shares as the sort has launches
    const int64_t bytes = p.accumulate ? 0 : p.V * p.D * (dt == RAR_BF16 ? 2 : 4);
    int share = 0;
    const int shares = p.T <= kSmallKeys ? 1 : 2 * passes;
    auto next_clear = [&]() {
        const int64_t lo = bytes / 256 * share / shares * 256;
        const int64_t hi = share + 1 == shares ? bytes : bytes / 256 * (share + 1) / shares * 256;
        ++share;
        return Clear{(char *)p.grad + lo, hi - lo};
    };
    auto clear_blocks = [](const Clear &c) { return (unsigned)((c.bytes + kClearBytes - 1) / kClearBytes); };
    int last = 0;
    hipError_t e = hipSuccess;
    if (p.T <= kSmallKeys) {
        const Clear c = next_clear();
        e = launch(p.T <= kSortKeys ? rar_sort_small<kRounds> : rar_sort_small<2 * kRounds>, 1 + clear_blocks(c),
                   kSortThreads, st, p.ids, (int)p.T, p.V, passes, bits, keys[0], pos[0], c);
    } else {
        const unsigned blocks = (unsigned)((p.T + kSortKeys - 1) / kSortKeys);
        uint32_t *const hist = (uint32_t *)(ws + l.hist);
        for (int pass = 0; pass < passes && e == hipSuccess; ++pass) {
            const int64_t *ids = pass == 0 ? p.ids : nullptr;
            const int from = (pass + 1) & 1, to = pass & 1;
            const Clear c0 = next_clear();
            e = launch(rar_sort_count, blocks + clear_blocks(c0), kSortThreads, st, ids, keys[from], p.T, p.V,
                       bits * pass, bits, hist, blocks, c0);
            const Clear c1 = next_clear();
            if (e == hipSuccess)
                e = launch(rar_sort_place, blocks + clear_blocks(c1), kSortThreads, st, ids, keys[from], pos[from], p.T,
                           p.V, bits * pass, bits, hist, keys[to], pos[to], blocks, c1);
            last = to;
        }
    }
    const GradWs w{keys[last], pos[last], (float *)(ws + l.from_left), (float *)(ws + l.to_right),
                   (float *)(ws + l.long_run), l.pitch, l.chunk};
    if (e != hipSuccess)
        return e;
    const bool vec = p.D % 8 == 0;
    if (dt == RAR_BF16)
        return vec ? sums<bf16, true>(p, w, st) : sums<bf16, false>(p, w, st);
    return vec ? sums<float, true>(p, w, st) : sums<float, false>(p, w, st);
}

}  // namespace rar
