// Whether the rows of a strided tensor share elements: plain host code.
#pragma once
#include <stdint.h>
#include <algorithm>

namespace qg {

struct Dim {
    int64_t count, stride;    // entries, elements from one to the next
};

// Rows of `width` elements, one for each combination of the dimensions'
// entries: true where no two share an element.  Counts and strides are at most
// 2^31.  Ordinary layouts are nested: each dimension steps over all that the
// ones of smaller strides span.  Otherwise two rows that overlap differ by some
// entries of the two shorter dimensions, which are tried, and by at most one of
// two numbers of entries of the longest; beyond 2^20 tries (where no such layout
// has a use) the answer is false.
template <int N>
bool rows_disjoint(Dim (&dims)[N], int64_t width)
{
    static_assert(N == 2 || N == 3, "two or three dimensions");
    for (Dim& d : dims)
        if (d.count <= 1) d = {1, 0};
    std::sort(dims, dims + N, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
    __int128 span = width;
    bool nested = true;
    for (const Dim& d : dims) {
        if (d.count > 1 && d.stride < span) nested = false;
        span += __int128(d.count - 1) * d.stride;
    }
    if (nested) return true;

    std::sort(dims, dims + N, [](const Dim& a, const Dim& b) { return a.count < b.count; });
    const Dim a = N == 3 ? dims[0] : Dim{1, 0}, b = dims[N - 2], c = dims[N - 1];
    if (c.stride < width) return false;
    if (__int128(2 * a.count - 1) * b.count > (1 << 20)) return false;
    for (int64_t j = 0; j < b.count; ++j)
        for (int64_t i = 1 - a.count; i < a.count; ++i) {
            // (a difference and its negative are the same pair)
            if (i == 0 && j == 0) continue;
            const int64_t off = i * a.stride + j * b.stride, near = off / c.stride;
            for (int64_t k = near - 1; k <= near + 1; ++k) {
                const int64_t d = off - k * c.stride;
                if (k < c.count && -k < c.count && d < width && -d < width) return false;
            }
        }
    return true;
}

}  // namespace qg
