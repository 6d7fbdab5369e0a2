// Which of a call's tensors share memory (host code, no CUDA).  A written
// tensor may lie between the rows of a strided one, as the parts of one packed
// buffer do, so byte ranges alone do not decide.
#pragma once

#include <cstddef>
#include <cstdint>

namespace la {

// A strided tensor as nested runs: `run` bytes at p + sum_k i_k stride[k], 0 <= i_k < count[k],
// strides descending.
struct Region {
    const char* p = nullptr;
    int axes = 0;
    long long stride[3] = {0, 0, 0}, count[3] = {0, 0, 0};
    long long run = 0;       // 0: an empty tensor, or none

    // bytes from the first to past the last one, without the outermost `from` axes
    long long extent(int from = 0) const
    {
        long long e = run;
        for (int k = from; k < axes; ++k) e += (count[k] - 1) * stride[k];
        return e;
    }
};

// Rows of `cols` elements of e bytes, element strides per axis (outer axes of any order; an axis of one
// entry, or of stride 0, which visits the same bytes again, is left out).
inline Region region(const void* p, size_t e, long long cols, const long long (&counts)[3], const long long (&strides)[3])
{
    Region r;
    r.p = static_cast<const char*>(p);
    r.run = p ? cols * (long long)e : 0;
    for (int k = 0; k < 3; ++k) {
        if (counts[k] <= 0 || cols <= 0) r.run = 0;
        if (counts[k] <= 1 || strides[k] == 0) continue;
        int at = r.axes++;
        for (; at > 0 && r.stride[at - 1] < strides[k] * (long long)e; --at) {
            r.stride[at] = r.stride[at - 1];
            r.count[at] = r.count[at - 1];
        }
        r.stride[at] = strides[k] * (long long)e;
        r.count[at] = counts[k];
    }
    // an axis that continues the run, or the axis inside it, is one with it
    while (r.axes > 0 && r.stride[r.axes - 1] == r.run) r.run *= r.count[--r.axes];
    for (int k = r.axes - 2; k >= 0; --k) {
        if (r.stride[k] != r.stride[k + 1] * r.count[k + 1]) continue;
        r.stride[k] = r.stride[k + 1];
        r.count[k] *= r.count[k + 1];
        for (int j = k + 1; j + 1 < r.axes; ++j) {
            r.stride[j] = r.stride[j + 1];
            r.count[j] = r.count[j + 1];
        }
        --r.axes;
    }
    return r;
}

inline Region dense(const void* p, size_t bytes) { return region(p, 1, (long long)bytes, {1, 1, 1}, {0, 0, 0}); }

// Some byte belongs to a (without its outermost i axes) at 0 and to b (without its outermost j) at `diff`.
// Exact, but for shapes that take more than `budget` steps, which count as sharing memory.
inline bool meet(const Region& a, int i, const Region& b, int j, long long diff, int* budget)
{
    if (diff >= a.extent(i) || diff + b.extent(j) <= 0) return false;
    if (i == a.axes && j == b.axes) return true;
    if (--*budget < 0) return true;
    const long long sa = i < a.axes ? a.stride[i] : 0, sb = j < b.axes ? b.stride[j] : 0, s = sa > sb ? sa : sb;
    // entries k of b's axis, or of a's counted down, or of both (their difference): diff moves by k s
    const int ni = i + (sa == s), nj = j + (sb == s);
    const long long lo = sa == s ? 1 - a.count[i] : 0, hi = sb == s ? b.count[j] - 1 : 0;
    // those that bring the rest of b into reach of the rest of a: -extent(b) < diff + k s < extent(a)
    const long long first = -b.extent(nj) - diff, end = a.extent(ni) - diff;
    auto floor_div = [](long long x, long long y) { return x >= 0 ? x / y : -((-x + y - 1) / y); };
    long long k = floor_div(first, s) + 1;
    if (k < lo) k = lo;
    for (; k <= hi && k * s < end; ++k)
        if (meet(a, ni, b, nj, diff + k * s, budget)) return true;
    return false;
}

inline bool shared(const Region& a, const Region& b)
{
    if (a.run == 0 || b.run == 0) return false;
    int budget = 1 << 14;
    return meet(a, 0, b, 0, b.p - a.p, &budget);
}

// Two entries of the outer axes share a byte (an axis of stride 0 is not seen here: region() leaves it out).
inline bool overlaps_itself(const Region& a)
{
    int budget = 1 << 14;
    for (int k = 0; k < a.axes; ++k)       // axis k is the outermost one in which the two entries differ
        for (long long n = 1; n < a.count[k] && n * a.stride[k] < a.extent(k + 1); ++n)
            if (meet(a, k + 1, a, k + 1, n * a.stride[k], &budget)) return true;
    return false;
}

}  // namespace la
