// embed.hip -- CDNA4 (gfx950) kernels of the embedding: lookup with scaling, and
// its gradient by sorted tokens.
//
// Lookup: out[t] = scale * table[ids[t]], a gather bound by HBM bandwidth.
//
// Gradient: grad[v] = scale * sum of dy[t] over the t with ids[t] == v, dense
// (every row of the vocabulary is written) or accumulated into the rows that
// occur.  The token positions are sorted by id, stably, so each row's terms
// stand together in token order; no floating-point atomic is used and the
// result does not depend on timing.  A row is then summed by one wave per 512
// columns.  A frequent token's run can be most of the batch, so runs are
// summed in two levels beforehand: every aligned 32 sorted positions that hold
// one id give a partial row, and every aligned 32 of those again; the wave adds
// the ragged ends and the partial rows, at most about 64 + 64 + T / 1024 terms.
// The order of the terms depends on the ids alone.
//
// Bound: dy read once, grad written once; the sort moves 16 bytes a token.
#include "act.h"
#include "ops_internal.h"

#pragma clang fp contract(off)

namespace rar {
namespace {

// ---------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------

// 16-byte vectors of a row, or single elements where rows are not 16-byte
// aligned.  The workgroup's first row is found by one uniform division.
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
            const f32x4 v = load4(src);
            store4(dst, ok ? v * p.scale : f32x4{0.0f, 0.0f, 0.0f, 0.0f});
        } else {
            const u32x4 w = *reinterpret_cast<const u32x4 *>(src);
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
                o[i] = ok ? pack_bf16(lo * p.scale, hi * p.scale) : 0u;
            }
            *reinterpret_cast<u32x4 *>(dst) = o;
        }
    }
}

// ---------------------------------------------------------------------------
// Stable sort of token positions by id, eight bits a pass
// ---------------------------------------------------------------------------

constexpr int kSortThreads = 1024;                      // sixteen waves
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortKeys = 4096;                         // keys of a workgroup: four rounds of 64 a wave
constexpr int kRounds = kSortKeys / kSortThreads;
constexpr int kChunk = 32;                              // sorted positions of a first-level partial row

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
__device__ __forceinline__ void wave_ranks(SortShared &s, const uint32_t (&digit)[kRounds], const bool (&live)[kRounds],
                                           uint32_t (&rank)[kRounds])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < kSortWaves * 256; i += kSortThreads)
        (&s.count[0][0])[i] = 0;
    __syncthreads();
    volatile uint32_t *count = s.count[wave];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        uint64_t peers = __ballot(live[r]);
#pragma unroll
        for (int b = 0; b < 8; ++b) {
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

// A whole batch of at most kSortKeys tokens in one workgroup.
__global__ void __launch_bounds__(kSortThreads) rar_sort_small(const int64_t *ids, int T, int64_t V, int passes,
                                                               uint32_t *keys, uint32_t *pos)
{
    __shared__ SortShared s;
    __shared__ uint32_t k_lds[kSortKeys], p_lds[kSortKeys];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t key[kRounds], at[kRounds], digit[kRounds], rank[kRounds];
    bool live[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int i = wave * (64 * kRounds) + r * 64 + lane;
        live[r] = i < T;
        key[r] = live[r] ? key_of(ids[i], V) : 0;
        at[r] = i;
    }
    for (int pass = 0; pass < passes; ++pass) {
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            digit[r] = (key[r] >> (8 * pass)) & 255;
        wave_ranks(s, digit, live, rank);
        const uint32_t total = scan_waves(s);
        scan_digits(s, total, 0);
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if (live[r]) {
                const uint32_t to = s.base[digit[r]] + s.count[wave][digit[r]] + rank[r];
                k_lds[to] = key[r];
                p_lds[to] = at[r];
            }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int i = wave * (64 * kRounds) + r * 64 + lane;
            if (live[r]) {
                key[r] = k_lds[i];
                at[r] = p_lds[i];
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int i = wave * (64 * kRounds) + r * 64 + lane;
        if (live[r]) {
            keys[i] = key[r];
            pos[i] = at[r];
        }
    }
}

// Larger batches: digit counts of each kSortKeys tokens, then their placement.
__global__ void __launch_bounds__(kSortThreads) rar_sort_count(const int64_t *ids, const uint32_t *keys, int64_t T,
                                                               int64_t V, int shift, uint32_t *hist)
{
    __shared__ uint32_t count[256];
    if (threadIdx.x < 256)
        count[threadIdx.x] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * kSortKeys;
    for (int i = threadIdx.x; i < kSortKeys; i += kSortThreads)
        if (first + i < T) {
            const uint32_t key = ids ? key_of(ids[first + i], V) : keys[first + i];
            atomicAdd(&count[(key >> shift) & 255], 1u);
        }
    __syncthreads();
    if (threadIdx.x < 256)
        hist[(int64_t)blockIdx.x * 256 + threadIdx.x] = count[threadIdx.x];
}

__global__ void __launch_bounds__(kSortThreads) rar_sort_place(const int64_t *ids, const uint32_t *keys,
                                                               const uint32_t *pos, int64_t T, int64_t V, int shift,
                                                               const uint32_t *hist, uint32_t *keys_out,
                                                               uint32_t *pos_out)
{
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
        digit[r] = (key[r] >> shift) & 255;
    }
    // digit totals of all workgroups and of those before this one
    const int d = threadIdx.x & 255, quarter = threadIdx.x >> 8;
    uint32_t all = 0, before = 0;
    for (int b = quarter; b < (int)gridDim.x; b += 4) {
        const uint32_t c = hist[(int64_t)b * 256 + d];
        all += c;
        before += b < (int)blockIdx.x ? c : 0;
    }
    part[0][quarter][d] = all;
    part[1][quarter][d] = before;
    wave_ranks(s, digit, live, rank);  // synchronises
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

constexpr int kCols = 512;  // columns of a wave: eight a lane

template <class T>
__device__ __forceinline__ void row8(const T *row, int64_t c, int cnt, bool vec, float (&v)[8])
{
    if (vec && cnt == 8) {
        const f32x4 a = load4(row + c), b = load4(row + c + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = i < cnt ? to_f32(row[c + i]) : 0.0f;
}

// acc += rows of dy at the `n` <= 64 sorted positions from `at`, in order; the
// positions are loaded together, four rows are in flight at a time.
template <class T>
__device__ __forceinline__ void add_rows(const EmbedGradParams &p, const uint32_t *pos, int64_t at, int n, int64_t c,
                                         int cnt, bool vec, float (&acc)[8])
{
    const int lane = threadIdx.x & 63;
    const uint32_t mine = lane < n ? pos[at + lane] : 0;
    const T *dy = (const T *)p.dy;
    int i = 0;
    for (; i + 4 <= n; i += 4) {
        float v[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            row8(dy + (int64_t)(uint32_t)__builtin_amdgcn_readlane(mine, i + u) * p.ldy, c, cnt, vec, v[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                acc[e] += v[u][e];
    }
    for (; i < n; ++i) {
        float v[8];
        row8(dy + (int64_t)(uint32_t)__builtin_amdgcn_readlane(mine, i) * p.ldy, c, cnt, vec, v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            acc[e] += v[e];
    }
}

__device__ __forceinline__ void add_partials(const float *part, int64_t pitch, int64_t at, int64_t n, int64_t c, int cnt,
                                             float (&acc)[8])
{
    if (cnt <= 0)
        return;
    const float *row = part + at * pitch + c;  // pitch is whole eights, so every lane's eight exist
#pragma unroll 4
    for (int64_t i = 0; i < n; ++i, row += pitch) {
        const f32x4 a = load4(row), b = load4(row + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            acc[e] += a[e];
            acc[4 + e] += b[e];
        }
    }
}

struct GradWs {
    uint32_t *keys, *pos;    // sorted
    uint32_t *start;         // [V + 1] first sorted position of each id
    float *part1, *part2;    // [T / 32][pitch], [T / 1024][pitch]
    int64_t pitch;
};

// First workgroups: start[v] by binary search.  The others: one first-level
// partial row each wave, where 32 aligned positions hold one id.
template <class T>
__global__ void __launch_bounds__(256) rar_embed_part1(const EmbedGradParams p, const GradWs w, int64_t start_blocks,
                                                       int strips)
{
    if ((int64_t)blockIdx.x < start_blocks) {
        const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
        if (v > p.V)
            return;
        int64_t lo = 0, hi = p.T;  // first position with key >= v
        while (lo < hi) {
            const int64_t mid = (lo + hi) / 2;
            if (w.keys[mid] < (uint32_t)v)
                lo = mid + 1;
            else
                hi = mid;
        }
        w.start[v] = (uint32_t)lo;
        return;
    }
    const int64_t job = ((int64_t)blockIdx.x - start_blocks) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t chunk = job / strips;
    const int64_t at = chunk * kChunk;
    if (at + kChunk > p.T)
        return;
    const uint32_t k = w.keys[at];
    if (k >= (uint32_t)p.V || k != w.keys[at + kChunk - 1])
        return;
    const int64_t c = (job - chunk * strips) * kCols + (threadIdx.x & 63) * 8;
    const int cnt = p.D - c >= 8 ? 8 : (p.D - c < 0 ? 0 : (int)(p.D - c));
    const bool vec = (uintptr_t)p.dy % 16 == 0 && (p.ldy * sizeof(T)) % 16 == 0;
    float acc[8] = {};
    add_rows<T>(p, w.pos, at, kChunk, c, cnt, vec, acc);
    if (cnt > 0) {
        float *o = w.part1 + chunk * w.pitch + c;
        store4(o, f32x4{acc[0], acc[1], acc[2], acc[3]});
        store4(o + 4, f32x4{acc[4], acc[5], acc[6], acc[7]});
    }
}

// Second-level partial rows: 32 aligned first-level rows of one id.
__global__ void __launch_bounds__(256) rar_embed_part2(const EmbedGradParams p, const GradWs w, int strips)
{
    const int64_t job = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t big = job / strips;
    const int64_t at = big * (kChunk * kChunk);
    if (at + kChunk * kChunk > p.T)
        return;
    const uint32_t k = w.keys[at];
    if (k >= (uint32_t)p.V || k != w.keys[at + kChunk * kChunk - 1])
        return;
    const int64_t c = (job - big * strips) * kCols + (threadIdx.x & 63) * 8;
    const int cnt = p.D - c >= 8 ? 8 : (p.D - c < 0 ? 0 : (int)(p.D - c));
    float acc[8] = {};
    add_partials(w.part1, w.pitch, big * kChunk, kChunk, c, cnt, acc);
    if (cnt > 0) {
        float *o = w.part2 + big * w.pitch + c;
        store4(o, f32x4{acc[0], acc[1], acc[2], acc[3]});
        store4(o + 4, f32x4{acc[4], acc[5], acc[6], acc[7]});
    }
}

// One wave per vocabulary row and 512 columns.
template <class T>
__global__ void __launch_bounds__(256) rar_embed_sum(const EmbedGradParams p, const GradWs w, int strips)
{
    const int64_t job = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t v = job / strips;
    if (v >= p.V)
        return;
    int64_t at = w.start[v];
    const int64_t end = w.start[v + 1];
    if (at == end && p.accumulate)
        return;
    const int64_t c = (job - v * strips) * kCols + (threadIdx.x & 63) * 8;
    const int cnt = p.D - c >= 8 ? 8 : (p.D - c < 0 ? 0 : (int)(p.D - c));
    const bool vec = (uintptr_t)p.dy % 16 == 0 && (p.ldy * sizeof(T)) % 16 == 0;
    constexpr int64_t kBig = kChunk * kChunk;
    float acc[8] = {};
    while (at < end) {
        const int64_t left = end - at;
        if (at % kBig == 0 && left >= kBig) {
            const int64_t n = left / kBig;
            add_partials(w.part2, w.pitch, at / kBig, n, c, cnt, acc);
            at += n * kBig;
        } else if (at % kChunk == 0 && left >= kChunk) {
            int64_t n = left / kChunk;
            const int64_t to_big = kChunk - at / kChunk % kChunk;  // rows up to the next second-level one
            n = n < to_big ? n : to_big;
            add_partials(w.part1, w.pitch, at / kChunk, n, c, cnt, acc);
            at += n * kChunk;
        } else {
            const int64_t to_chunk = kChunk - at % kChunk;
            const int n = (int)(left < to_chunk ? left : to_chunk);
            add_rows<T>(p, w.pos, at, n, c, cnt, vec, acc);
            at += n;
        }
    }
    if (cnt <= 0)
        return;
    T *out = (T *)p.grad + v * p.D + c;
    const bool vout = cnt == 8 && ((uintptr_t)out % 16 == 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        acc[i] *= p.scale;
        if (p.accumulate && i < cnt)
            acc[i] += to_f32(out[i]);
    }
    if (vout) {
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<u32x4 *>(out) = u32x4{pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]),
                                                    pack_bf16(acc[4], acc[5]), pack_bf16(acc[6], acc[7])};
        } else {
            store4(out, f32x4{acc[0], acc[1], acc[2], acc[3]});
            store4(out + 4, f32x4{acc[4], acc[5], acc[6], acc[7]});
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < cnt)
            out[i] = from_f32<T>(acc[i]);
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Byte offsets of the workspace's parts.
struct Layout {
    int64_t keys[2], pos[2], hist, start, part1, part2, total, pitch;
};

Layout layout(int64_t T, int64_t V, int64_t D)
{
    Layout l{};
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += up(bytes, 256);
        return here;
    };
    l.pitch = up(D, 8);
    const bool small = T <= kSortKeys;
    for (int i = 0; i < 2; ++i) {
        l.keys[i] = i && small ? l.keys[0] : take(4 * T);
        l.pos[i] = i && small ? l.pos[0] : take(4 * T);
    }
    l.hist = take(small ? 0 : (T + kSortKeys - 1) / kSortKeys * 1024);
    l.start = take(4 * (V + 1));
    l.part1 = take(T / kChunk * l.pitch * 4);
    l.part2 = take(T / (kChunk * kChunk) * l.pitch * 4);
    l.total = at;
    return l;
}

template <class T>
void sums(const EmbedGradParams &p, const GradWs &w, hipStream_t st)
{
    const int strips = (int)((p.D + kCols - 1) / kCols);
    const int64_t start_blocks = (p.V + 1 + 255) / 256;
    const int64_t jobs1 = p.T / kChunk * strips, jobs2 = p.T / (kChunk * kChunk) * strips;
    rar_embed_part1<T><<<(unsigned)(start_blocks + (jobs1 + 3) / 4), 256, 0, st>>>(p, w, start_blocks, strips);
    if (jobs2)
        rar_embed_part2<<<(unsigned)((jobs2 + 3) / 4), 256, 0, st>>>(p, w, strips);
    rar_embed_sum<T><<<(unsigned)((p.V * strips + 3) / 4), 256, 0, st>>>(p, w, strips);
}

}  // namespace

int64_t embed_grad_workspace(int64_t T, int64_t V, int64_t D) { return layout(T, V, D).total; }

hipError_t launch_embed_lookup(rar_dtype dt, const EmbedParams &p, hipStream_t st)
{
    const int es = dt == RAR_BF16 ? 2 : 4;
    const bool vec = (uintptr_t)p.table % 16 == 0 && (uintptr_t)p.out % 16 == 0 && (p.D * es) % 16 == 0 &&
                     (p.ldo * es) % 16 == 0;
    const int64_t items = p.T * (vec ? p.D * es / 16 : p.D);
    const unsigned grid = (unsigned)((items + 1023) / 1024);
    if (dt == RAR_BF16)
        vec ? rar_embed_rows<bf16, true><<<grid, 256, 0, st>>>(p) : rar_embed_rows<bf16, false><<<grid, 256, 0, st>>>(p);
    else
        vec ? rar_embed_rows<float, true><<<grid, 256, 0, st>>>(p)
            : rar_embed_rows<float, false><<<grid, 256, 0, st>>>(p);
    return hipGetLastError();
}

hipError_t launch_embed_grad(rar_dtype dt, const EmbedGradParams &p, hipStream_t st)
{
    const Layout l = layout(p.T, p.V, p.D);
    char *const ws = (char *)p.ws;
    uint32_t *keys[2], *pos[2];
    for (int i = 0; i < 2; ++i) {
        keys[i] = (uint32_t *)(ws + l.keys[i]);
        pos[i] = (uint32_t *)(ws + l.pos[i]);
    }
    int bits = 0;  // of the keys 0..V
    while (bits < 32 && (p.V >> bits) != 0)
        ++bits;
    const int passes = (bits + 7) / 8;
    int last = 0;
    if (p.T <= kSortKeys) {
        rar_sort_small<<<1, kSortThreads, 0, st>>>(p.ids, (int)p.T, p.V, passes, keys[0], pos[0]);
    } else {
        const unsigned blocks = (unsigned)((p.T + kSortKeys - 1) / kSortKeys);
        uint32_t *const hist = (uint32_t *)(ws + l.hist);
        for (int pass = 0; pass < passes; ++pass) {
            const int64_t *ids = pass == 0 ? p.ids : nullptr;
            const int from = (pass + 1) & 1, to = pass & 1;
            rar_sort_count<<<blocks, kSortThreads, 0, st>>>(ids, keys[from], p.T, p.V, 8 * pass, hist);
            rar_sort_place<<<blocks, kSortThreads, 0, st>>>(ids, keys[from], pos[from], p.T, p.V, 8 * pass, hist,
                                                            keys[to], pos[to]);
            last = to;
        }
    }
    const GradWs w{keys[last], pos[last], (uint32_t *)(ws + l.start), (float *)(ws + l.part1), (float *)(ws + l.part2),
                   l.pitch};
    if (dt == RAR_BF16)
        sums<bf16>(p, w, st);
    else
        sums<float>(p, w, st);
    return hipGetLastError();
}

}  // namespace rar
