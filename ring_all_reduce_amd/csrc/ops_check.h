// ops_check.h -- argument checks and workspace layout shared by the host side of
// the operators (ops_host.cpp, block_host.cpp).  Not part of the public ABI.
#pragma once

#include <cstdint>
#include <initializer_list>

#include "linear_shape.h"
#include "ops_internal.h"

namespace rar {

constexpr int64_t kMaxWidth = int64_t(1) << 20;   // K, N, D, V of a row
constexpr int64_t kMaxLd = int64_t(1) << 22;      // offsets inside a 256-row tile stay under 2^31 bytes
constexpr int64_t kMaxRows = int64_t(1) << 24;    // T
constexpr int64_t kMaxVocab = int64_t(1) << 30;

inline bool valid_dtype(int d) { return d == RAR_F32 || d == RAR_BF16; }
inline bool valid_act(int a) { return a == RAR_ACT_NONE || a == RAR_ACT_RELU || a == RAR_ACT_GELU; }
inline bool valid_rows(int64_t T) { return T >= 0 && T <= kMaxRows; }
inline bool valid_width(int64_t n) { return n >= 1 && n <= kMaxWidth; }
inline bool valid_ld(int64_t ld, int64_t cols) { return ld >= cols && ld <= kMaxLd; }

inline rar_status launched(hipError_t e)
{
    if (e == hipSuccess)
        return RAR_OK;
    (void)hipGetLastError();  // the caller's next HIP call must not report it again
    return RAR_EHIP;
}

// A matrix argument: rows x cols elements of es bytes, ld elements apart.
struct Mat {
    const void *p;
    int64_t rows, cols, ld;
    int es;
    uintptr_t lo() const { return (uintptr_t)p; }
    uintptr_t hi() const { return lo() + (uintptr_t)(((rows - 1) * ld + cols) * es); }
    bool empty() const { return !p || rows <= 0 || cols <= 0; }
};

inline Mat vec(const void *p, int64_t n, int es) { return Mat{p, 1, n, n, es}; }

// Whether two matrices share memory.  Views of one leading dimension may lie
// side by side: then only their columns count.
inline bool overlap(const Mat &a, const Mat &b)
{
    if (a.empty() || b.empty() || a.lo() >= b.hi() || b.lo() >= a.hi())
        return false;
    const int64_t pa = a.ld * a.es, pb = b.ld * b.es;
    if (pa == pb) {
        const int64_t d = (int64_t)((b.lo() >= a.lo() ? b.lo() - a.lo() : a.lo() - b.lo()) % (uint64_t)pa);
        const int64_t first = (b.lo() >= a.lo() ? a.cols * a.es : b.cols * b.es);
        const int64_t second = (b.lo() >= a.lo() ? b.cols * b.es : a.cols * a.es);
        return !(d >= first && pa - d >= second);
    }
    return true;
}

// Outputs must be apart from each other and from the inputs.
inline bool apart(std::initializer_list<Mat> outs, std::initializer_list<Mat> ins)
{
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (auto q = o + 1; q != outs.end(); ++q)
            if (overlap(*o, *q))
                return false;
        for (const Mat &i : ins)
            if (overlap(*o, i))
                return false;
    }
    return true;
}

// The same matrix given twice: an output that an input may be.
inline bool same(const Mat &a, const Mat &b)
{
    return a.p == b.p && a.ld == b.ld && a.rows == b.rows && a.cols == b.cols;
}

inline bool aligned(const void *p, int to) { return ((uintptr_t)p & (uintptr_t)(to - 1)) == 0; }

// Rows that the products may read 16 bytes at a time.
inline bool direct(const Mat &m)
{
    return aligned(m.p, 16) && (m.ld * m.es) % 16 == 0 && (m.cols * m.es) % 16 == 0;
}

// Bytes of the workspace's parts, each a multiple of 256.
struct Carve {
    char *at;
    int64_t used = 0;
    void *take(int64_t bytes)
    {
        void *p = at ? at + used : nullptr;
        used += up(bytes, 256);
        return p;
    }
};

}  // namespace rar
