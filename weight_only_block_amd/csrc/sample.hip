// A token per row of logits by temperature, top-k, top-p and min-p, from
// given uniform numbers.
//
// The tokens that survive the cuts are always the first ones of the order
// (larger logit, then lower index), so all cuts together are one 64-bit key
// of that order (argmax_key): a token is kept when its key is not below it.
// Sums over the order's head (top-p) are integers in fixed point, and sums
// over indices (the draw) are fp64 in a fixed order, so nothing depends on
// the order in which atomics arrive.
//
// A row is split into chunks, one work-group each, in three launches:
//   1. the largest key of each chunk;
//   2. where some cut is asked for, a histogram of the row over bins of
//      (largest - logit): counts, and for top-p weights;
//   3. from the histogram, the bins that the cuts fall into: tokens above are
//      kept for sure and summed, tokens in those bins become candidates; the
//      row's last work-group ranks the candidates against each other, which
//      gives the key, adds the kept ones to the sums of their groups (256
//      tokens, more in very long rows), finds the group that the uniform number
//      falls into and the token in it.
// No row has all its logits weighed twice: the histogram weighs rows with
// top-p, the draw all tokens of rows without a cut and the kept ones of others.
// 64 rows of 151936, 39 MB, in mixed settings: 9 us for the largest logits, 18
// for the histogram, bound by its fp64 weights, and 33 for the draw, bound by
// fp64 weights one after another in rows without a cut (17 us of its scan, 7 with
// top-k) and by the dependent steps at the end of rows with one (6 to 11 us).
// All without a cut take 36 us, with top-k 44, top-p 61, both 56.  Few rows are
// bound by latency (one: 4 + 6 + 14 us, most of the last a chain of reads and
// sums by the row's last work-group).
// Rows of up to 8192 logits, and rows of any length where there are more than
// 128, are a work-group's each, with all steps in one launch.  A row whose cut
// falls into bins of more than 4096 tokens (many nearly equal logits) gets its
// key by a radix selection over the row, by one work-group (151936 logits within
// 0.1 of each other and top-p: 256 us for one row, 313 for 64).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "argmax_key.h"
#include "decode_ops.h"

namespace qg {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 2048;
constexpr int kCandidates = 4096;
constexpr int kMaxChunks = 64;
constexpr int kAhead = 2;                  // rounds of loads in the last launch
constexpr int kGroups = kThreads;          // of a row: a thread sums one up
constexpr int64_t kSmallRow = 8192;        // one work-group at once
// Work-groups of the last launch that the chip holds at once (112 registers a
// thread leave room for one a compute unit; 64 of them spill and cost more).
constexpr int64_t kResident = 256;

// How a row is divided: at most 1024 groups of 256 q tokens, whose kept weight
// is remembered so that only one of them is read again for the draw, and
// chunks of whole groups, a work-group each.
struct Division {
    int64_t chunk, group;     // tokens of a chunk, of a group
    int chunks, groups;       // chunks of a row, groups of a chunk
};

__host__ __device__ inline int64_t group_size(int64_t N)
{
    return 256 * ((N + 256 * kGroups - 1) / (256 * kGroups));
}

__host__ __device__ inline Division division(int64_t m, int64_t N)
{
    Division d;
    // about as many chunks as the chip holds work-groups, of at least 4096 logits
    int64_t chunks = (N + 4095) / 4096;
    const int64_t fit = m < kResident ? kResident / m : 1;
    if (chunks > fit) chunks = fit;
    if (chunks > kMaxChunks) chunks = kMaxChunks;
    if (N <= kSmallRow) chunks = 1;
    d.group = group_size(N);
    const int64_t groups = (N + d.group - 1) / d.group;
    d.groups = int((groups + chunks - 1) / chunks);
    d.chunk = d.group * d.groups;
    d.chunks = int((groups + d.groups - 1) / d.groups);
    return d;
}

// Row r's part of the workspace.
struct RowSpace {
    unsigned long long weight[kBins];
    unsigned int count[kBins];
    unsigned long long key[kMaxChunks];
    unsigned long long sum[kGroups];       // fp64 bits
    unsigned long long candidate[kCandidates];
    unsigned int candidates, arrived, pad[14];
};

// Weights in fixed point: N weights of at most 1 fit 62 bits.
__device__ __forceinline__ int weight_bits(int64_t N)
{
    const int b = 62 - (64 - __clzll((long long)N));
    return b > 50 ? 50 : b;
}

__device__ __forceinline__ uint32_t order_of(float v) { return uint32_t(argmax_key(v, 0) >> 32); }

__device__ __forceinline__ float value_of(uint32_t order)
{
    return __uint_as_float((order & 0x80000000u) ? order & 0x7fffffffu : ~order);
}

// A row's settings; weights are 2^y with y = (x - top) log2(e) / temperature.
struct Row {
    float top, low;
    double rate;          // log2(e) / temperature
    int64_t N, k;
    double top_p, floor;
    double unit;          // fixed-point steps of a weight of 1
    const double* powers; // LDS: 2^(i / 256)
    bool greedy;
    int32_t top_idx;

    // Tokens below `low` have a weight far under the smallest fp64 one (or are
    // -infinity): never drawn, and left out of the ranks behind every token
    // that can be.
    __device__ __forceinline__ bool live(float v) const { return v >= low; }

    // (equal infinities differ by NaN, which counts as 0)
    __device__ __forceinline__ double exponent(float v) const
    {
        return fmax(fmin((double(v) - double(top)) * rate, 0.0), -1100.0);
    }

    // 2^y for -1100 <= y <= 0 as 2^(n / 256) 2^f: the first factor from a table
    // of 256 and the exponent, the second by its Taylor series in f ln 2, below
    // 0.0014, whose fifth term is below 2^-54 (without a table the series takes
    // 13 terms: 29 us in place of 25 for 64 rows of 151936 without a cut).
    // Adding 1.5 * 2^52 leaves n in the sum's low bits.
    __device__ __forceinline__ double weight(double y) const
    {
        constexpr double kLn2 = 0.69314718055994530942;
        const double t = __builtin_fma(y, 256.0, 0x1.8p52);
        const int i = int(uint32_t(__double_as_longlong(t)));
        const double f = __builtin_fma(t - 0x1.8p52, -1.0 / 256.0, y);
        double p = __builtin_fma(f, kLn2 * kLn2 * kLn2 * kLn2 / 24.0, kLn2 * kLn2 * kLn2 / 6.0);
        p = __builtin_fma(p, f, kLn2 * kLn2 / 2.0);
        p = __builtin_fma(p, f, kLn2);
        p = __builtin_fma(p, f, 1.0);
        return ldexp(p * powers[i & 255], i >> 8);
    }
    // Rounded to an integer by adding 2^52: what is below the point leaves the mantissa.
    __device__ __forceinline__ unsigned long long fixed(double w) const
    {
        return (unsigned long long)__double_as_longlong(__builtin_fma(w, unit, 0x1p52)) & 0xfffffffffffffull;
    }
    // Weight of a kept token in the draw.
    __device__ __forceinline__ double drawn(float v) const
    {
        const double w = weight(exponent(v));
        return w >= floor ? w : 0.0;
    }
    __device__ __forceinline__ bool cut() const { return k < N || top_p < 1.0; }
};

// 2^(i / 256) for i < 256: the Taylor series of exp(i ln 2 / 256), whose 18th
// term is below 2^-58.
__device__ __forceinline__ void fill_powers(double* powers)
{
    if (threadIdx.x >= 256) return;
    const double z = double(threadIdx.x) * (0.69314718055994530942 / 256.0);
    double p = 1.0;
#pragma unroll
    for (int k = 17; k >= 1; --k) p = __builtin_fma(p, z * (1.0 / k), 1.0);
    powers[threadIdx.x] = p;
}

__device__ __forceinline__ Row row_of(const SampleParams& p, int64_t row, uint64_t best, const double* powers)
{
    Row r;
    r.powers = powers;
    r.top_idx = key_index(best);
    r.top = value_of(uint32_t(best >> 32));
    const float t = p.temperature ? p.temperature[row] : 1.0f;
    // greedy, or nothing to weigh: a NaN wins, and a row of -infinity gives its first
    r.greedy = !(t > 0.0f) || r.top != r.top || r.top == -INFINITY;
    // (never 0: under an infinite temperature -infinity still weighs nothing, and
    // finite logits differ by too little to tell)
    r.rate = fmax(1.44269504088896340736 / double(t), 1e-300);
    r.low = r.top == INFINITY ? INFINITY : float(fmax(double(r.top) - 1100.0 / r.rate, double(-__FLT_MAX__)));
    r.N = p.N;
    r.k = p.top_k && p.top_k[row] > 0 ? min(int64_t(p.top_k[row]), p.N) : p.N;
    const float tp = p.top_p ? p.top_p[row] : 1.0f, mp = p.min_p ? p.min_p[row] : 0.0f;
    r.top_p = tp < 1.0f ? double(tp) : 1.0;          // NaN: none
    r.floor = mp != mp ? 0.0 : fmin(double(mp), 1.0);
    r.unit = ldexp(1.0, weight_bits(p.N));
    return r;
}

// Bins of d = top - x, finest near the top in proportion (d < 1: 32 an octave
// down to 2^-12), then 32 a unit to 33, then 32 an octave.
__device__ __forceinline__ float below_top(float top, float v) { return fmaxf(top - v, 0.0f); }

__device__ __forceinline__ int bin_of(float d)
{
    const uint32_t bits = __float_as_uint(d);
    const int near = int((max(bits, 0x39800000u) - 0x39800000u) >> 18), mid = 384 + int((d - 1.0f) * 32.0f);
    const int far = min(1408 + int((bits - 0x42040000u) >> 18), kBins - 1);
    return d < 1.0f ? near : d < 33.0f ? mid : far;
}

// The smallest d of a bin; no d is below that of bin 0, every d (infinity too)
// is below the NaN of bin kBins.
__device__ __forceinline__ float edge_of(int bin)
{
    if (bin <= 0) return 0.0f;
    if (bin <= 384) return __uint_as_float(0x39800000u + (uint32_t(bin) << 18));
    if (bin <= 1408) return 1.0f + float(bin - 384) * (1.0f / 32.0f);
    return bin < kBins ? __uint_as_float(0x42040000u + (uint32_t(bin - 1408) << 18)) : __uint_as_float(0x7fc00000u);
}

template <class T>
struct ScanSpace {
    T wave[kWaves];
};

// Inclusive sums over the block in thread order, a fixed tree; the total in *total.
template <class T>
__device__ __forceinline__ T scan(ScanSpace<T>& s, T v, T* total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const T o = __shfl_up(v, off, 64);
        if (lane >= off) v += o;
    }
    __syncthreads();
    if (lane == 63) s.wave[wave] = v;
    __syncthreads();
    T before = T(0), all = T(0);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w == wave) before = all;
        all += s.wave[w];
    }
    *total = all;
    return before + v;
}

// The largest value of an ascending thread's: that of the wave's last thread that has one.
__device__ __forceinline__ void wave_max(int* at, int v)
{
    const uint64_t some = __ballot(v > 0);
    if (some && int(threadIdx.x & 63) == 63 - __clzll((long long)some)) atomicMax(at, v);
}

struct Shared {
    double powers[256];
    unsigned long long weight[kBins];      // the histogram; then, by halves, groups' sums and what is added to them
    unsigned int count[kBins];
    ScanSpace<double> d;
    ScanSpace<unsigned long long> u;
    ScanSpace<unsigned int> n;
    unsigned long long best[kWaves];
    unsigned long long above_weight, sum_k, cut, pick;
    unsigned int above_count, in_bin;
    int bin, bin2, flag;
};

__device__ __forceinline__ uint64_t block_max(Shared& s, uint64_t best)
{
#pragma unroll
    for (int off = 32; off; off >>= 1) best = max_key(best, __shfl_xor((unsigned long long)best, off, 64));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s.best[threadIdx.x >> 6] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) best = max_key(best, s.best[w]);
    return best;
}

// Inclusive sums of two values at once, as scan.
__device__ __forceinline__ void scan_both(Shared& s, unsigned int* c, unsigned long long* w, unsigned int* call,
                                          unsigned long long* wall)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const unsigned int co = __shfl_up(*c, off, 64);
        const unsigned long long wo = __shfl_up(*w, off, 64);
        if (lane >= off) *c += co, *w += wo;
    }
    if (lane == 63) s.n.wave[wave] = *c, s.u.wave[wave] = *w;
    __syncthreads();
    *call = 0, *wall = 0;
    unsigned int cb = 0;
    unsigned long long wb = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        if (i == wave) cb = *call, wb = *wall;
        *call += s.n.wave[i];
        *wall += s.u.wave[i];
    }
    *c += cb;
    *w += wb;
}

// ------------------------------------------------ one work-group for a row

// The last kept key of a cut, by count (the k-th token) or by weight (the last
// one whose preceding weight is below `limit`): three passes over the order's
// 11, 11 and 10 bits.
__device__ void select(Shared& s, const Row& r, const float* x, bool by_count, uint64_t k, double limit, uint32_t* cut,
                       uint64_t* above_count, uint64_t* above_weight, uint64_t* ties)
{
    uint32_t prefix = 0, known = 0;
    uint64_t ac = 0, aw = 0;
    for (int level = 0; level < 3; ++level) {
        const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, width = level == 2 ? 10 : 11;
        __syncthreads();
        for (int i = threadIdx.x; i < kBins; i += kThreads) s.weight[i] = 0, s.count[i] = 0;
        if (threadIdx.x == 0) s.bin = -1;
        __syncthreads();
        for (int64_t i = threadIdx.x; i < r.N; i += kThreads) {
            const float v = x[i];
            const uint32_t o = order_of(v);
            if ((o & known) != prefix) continue;
            const int bin = int((o >> shift) & ((1u << width) - 1));
            atomicAdd(&s.count[bin], 1u);
            atomicAdd(&s.weight[bin], r.fixed(r.weight(r.exponent(v))));
        }
        __syncthreads();
        // thread t holds bins kBins - 1 - 2 t and the one below: descending
        const int hi = kBins - 1 - 2 * threadIdx.x, lo = hi - 1;
        const unsigned int c0 = s.count[hi], c1 = s.count[lo];
        const unsigned long long w0 = s.weight[hi], w1 = s.weight[lo];
        unsigned int call;
        unsigned long long wall;
        const uint64_t cb = ac + scan(s.n, c0 + c1, &call) - (c0 + c1);
        const uint64_t wb = aw + scan(s.u, w0 + w1, &wall) - (w0 + w1);
        // the last bin (lowest) with something in it that begins inside the cut
        const auto inside = [&](uint64_t c, uint64_t w) { return by_count ? c < k : c == 0 || double(w) < limit; };
        int mine = -1;
        if (c0 && inside(cb, wb)) mine = 2 * threadIdx.x;
        if (c1 && inside(cb + c0, wb + w0)) mine = 2 * threadIdx.x + 1;
        if (mine >= 0) atomicMax(&s.bin, mine);
        __syncthreads();
        const int at = s.bin;
        if (at >> 1 == int(threadIdx.x)) {
            s.above_count = unsigned(at & 1 ? cb + c0 : cb);
            s.above_weight = at & 1 ? wb + w0 : wb;
            s.in_bin = at & 1 ? c1 : c0;
        }
        __syncthreads();
        prefix |= uint32_t(kBins - 1 - at) << shift;
        known |= ((1u << width) - 1) << shift;
        ac = s.above_count, aw = s.above_weight, *ties = s.in_bin;
    }
    *cut = prefix;
    *above_count = ac;
    *above_weight = aw;
}

// The row's cut as a key.
__device__ uint64_t cut_by_selection(Shared& s, const Row& r, const float* x)
{
    uint32_t cut = 0;
    uint64_t kept = uint64_t(r.N), ties = uint64_t(r.N);
    uint64_t sum = 0;
    if (r.k < r.N) {
        uint64_t ac, aw;
        select(s, r, x, true, uint64_t(r.k), 0.0, &cut, &ac, &aw, &ties);
        kept = uint64_t(r.k) - ac;
        sum = aw + kept * r.fixed(r.weight(r.exponent(value_of(cut))));
    }
    if (r.top_p < 1.0) {
        if (r.k >= r.N) {
            unsigned long long mine = 0, all;
            for (int64_t i = threadIdx.x; i < r.N; i += kThreads) mine += r.fixed(r.weight(r.exponent(x[i])));
            scan(s.u, mine, &all);
            sum = all;
        }
        uint32_t pcut;
        uint64_t ac, aw, pties;
        const double limit = r.top_p * double(sum);
        select(s, r, x, false, 0, limit, &pcut, &ac, &aw, &pties);
        const uint64_t w = r.fixed(r.weight(r.exponent(value_of(pcut))));
        // ties j = 0, 1, ... are kept while the weight before them is below the limit
        uint64_t lo = 1, hi = pties;
        while (lo < hi) {
            const uint64_t mid = (lo + hi + 1) / 2;
            if (double(aw + w * (mid - 1)) < limit) lo = mid;
            else hi = mid - 1;
        }
        if (pcut > cut || (pcut == cut && lo < kept)) cut = pcut, kept = lo, ties = pties;
    }
    if (kept >= ties) return uint64_t(cut) << 32;
    // index of the last tie kept
    uint64_t seen = 0;
    for (int64_t base = 0; base < r.N; base += kThreads) {
        const int64_t i = base + threadIdx.x;
        const unsigned int is = i < r.N && order_of(x[i]) == cut;
        unsigned int all;
        const uint64_t upto = seen + scan(s.n, is, &all);
        if (is && upto == kept) s.cut = uint64_t(cut) << 32 | uint64_t(~uint32_t(i));
        seen += all;
        if (seen >= kept) break;
    }
    __syncthreads();
    return s.cut;
}

// The token of [from, to) where the running sum of kept weights passes
// `target`, else the last kept one, r.N without any; by one wave, 256 tokens
// at a time, four neighbours a lane.
__device__ int64_t walk_wave(const Row& r, const float* x, int64_t from, int64_t to, uint64_t cut, double run, double target)
{
    const int lane = threadIdx.x & 63;
    int64_t last = r.N;
#pragma unroll 1
    for (int64_t base = from; base < to; base += 256) {
        const int64_t i = base + 4 * lane;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = i + e < to ? x[i + e] : -INFINITY;
        double w[4], strip = 0.0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = i + e < to && argmax_key(v[e], uint32_t(i + e)) >= cut ? r.drawn(v[e]) : 0.0;
            strip += w[e];
        }
        double upto = strip;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const double o = __shfl_up(upto, off, 64);
            if (lane >= off) upto += o;
        }
        const uint64_t some = __ballot(strip > 0.0), past = __ballot(strip > 0.0 && run + upto > target);
        // the last of a lane's kept tokens, or the first whose sum passes
        double sum = run + (upto - strip);
        int at = 0;
        bool found = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (found || !(w[e] > 0.0)) continue;
            at = e;
            sum += w[e];
            found = sum > target;
        }
        const int src = past ? __ffsll((unsigned long long)past) - 1 : some ? 63 - __clzll((long long)some) : 0;
        if (some) last = base + 4 * src + __shfl(at, src, 64);
        if (past) break;
        run += __shfl(upto, 63, 64);
    }
    return last;
}

// The token in which the running sum of kept weights passes u times their
// sum, r.N without any: thread t holds the kept weight of group t, one wave
// walks the group that the token is in.
__device__ int64_t draw_token(Shared& s, const Row& r, const float* x, uint64_t cut, double mine, int64_t size, double u)
{
    if (threadIdx.x == 0) s.bin = kThreads, s.bin2 = 0;
    double all;
    const double upto = scan(s.d, mine, &all);
    const double target = u * all;
    const uint64_t past = __ballot(mine > 0.0 && upto > target);
    if (past && int(threadIdx.x & 63) == __ffsll((unsigned long long)past) - 1) atomicMin(&s.bin, int(threadIdx.x));
    wave_max(&s.bin2, mine > 0.0 ? int(threadIdx.x) + 1 : 0);
    __syncthreads();
    // (rounding may leave the target past the end: then the last group with a kept token)
    const int g = s.bin < kThreads ? s.bin : s.bin2 - 1;
    if (g < 0 || !(u < 1.0)) return r.N;
    if (int(threadIdx.x) == g) s.d.wave[0] = upto - mine;
    __syncthreads();
    int64_t pick = r.N;
    if (threadIdx.x < 64) pick = walk_wave(r, x, g * size, min(r.N, (g + 1) * size), cut, s.d.wave[0], target);
    return pick;                               // (the first wave's)
}

// A wave's sum, in every lane.
__device__ __forceinline__ double wave_sum(double w)
{
#pragma unroll
    for (int off = 32; off; off >>= 1) w += __shfl_xor(w, off, 64);
    return w;
}

__device__ void draw_by_selection(Shared& s, const SampleParams& p, int64_t row, const Row& r)
{
    const float* x = p.x + row * p.ldx;
    const uint64_t cut = r.cut() ? cut_by_selection(s, r, x) : 0;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double* group_sum = reinterpret_cast<double*>(s.weight);
    const int64_t size = group_size(r.N);
    const int groups = int((r.N + size - 1) / size);
    __syncthreads();
    for (int g = wave; g < kGroups; g += kWaves) {
        double w = 0.0;
        for (int64_t base = g * size; g < groups && base < (g + 1) * size; base += 256) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = base + 64 * e + lane < r.N ? x[base + 64 * e + lane] : -INFINITY;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (base + 64 * e + lane < r.N && argmax_key(v[e], uint32_t(base + 64 * e + lane)) >= cut) w += r.drawn(v[e]);
        }
        w = wave_sum(w);
        if (lane == 0) group_sum[g] = w;
    }
    __syncthreads();
    const int64_t pick = draw_token(s, r, x, cut, group_sum[threadIdx.x], size, p.u[row]);
    if (threadIdx.x == 0) p.idx[row] = pick < r.N ? int32_t(pick) : r.top_idx;
}

// ------------------------------------------------------------ three launches

// Calls f(values, first token) for the tokens [from, to), eight a thread at a
// time, the e-th of them kThreads * e past the first; the next eight are on
// their way meanwhile.  Past the end f sees -infinity.
template <class F>
__device__ __forceinline__ void each_token(const float* x, int64_t from, int64_t to, F f)
{
    constexpr uint32_t kStep = 8 * kThreads;
    const uint32_t n = uint32_t(to - from);        // below 2^31
    x += from;
    float next[8];
    const auto load = [&](uint32_t base) {
        const float* at = x + base;                // the same in every lane
        if (base + kStep <= n) {
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e) next[e] = at[e * kThreads + threadIdx.x];
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e) next[e] = x[min(base + e * kThreads + threadIdx.x, n - 1)];
        }
    };
    load(0);
    for (uint32_t base = 0; base < n; base += kStep) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = next[e];
        if (base + kStep < n) load(base + kStep);
        if (base + kStep > n) {
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e)
                if (base + e * kThreads + threadIdx.x >= n) v[e] = -INFINITY;
        }
        f(v, from + base + threadIdx.x);
    }
}

// The largest key of [from, to).
__device__ __forceinline__ uint64_t top_of(Shared& s, const float* x, int64_t from, int64_t to)
{
    uint64_t best = 0;
    each_token(x, from, to, [&](const float (&v)[8], int64_t i) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (i + e * kThreads < to) best = max_key(best, argmax_key(v[e], uint32_t(i + e * kThreads)));
    });
    return block_max(s, best);
}

// Adds [from, to) to the histogram in LDS: counts for top-k, weights for top-p.
__device__ __forceinline__ void add_to_bins(Shared& s, const Row& r, const float* x, int64_t from, int64_t to)
{
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.weight[i] = 0, s.count[i] = 0;
    __syncthreads();
    const bool weigh = r.top_p < 1.0, rank = r.k < r.N;
    // (four weights side by side, as their operations wait on each other)
    each_token(x, from, to, [&](const float (&v)[8], int64_t i) {
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
            if (i - threadIdx.x + h * kThreads >= to) break;         // the same in every lane
            int bin[4];
            unsigned long long w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) bin[e] = bin_of(below_top(r.top, v[h + e]));
            if (weigh) {
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = r.fixed(r.weight(r.exponent(v[h + e])));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!r.live(v[h + e])) continue;
                if (rank) atomicAdd(&s.count[bin[e]], 1u);
                if (weigh) atomicAdd(&s.weight[bin[e]], w[e]);
            }
        }
    });
    __syncthreads();
}

__global__ __launch_bounds__(kThreads) void sample_top(SampleParams p, Division dv)
{
    fetch_arguments<sizeof(SampleParams) + sizeof(Division)>();
    __shared__ Shared s;
    const int64_t row = blockIdx.y;
    RowSpace& ws = static_cast<RowSpace*>(p.workspace)[row];
    const int64_t from = blockIdx.x * dv.chunk, to = min(p.N, from + dv.chunk);
    // the row's histogram and counters begin at zero for the launches below
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < kBins; i += gridDim.x * kThreads) ws.weight[i] = 0, ws.count[i] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) ws.candidates = 0, ws.arrived = 0;
    const uint64_t best = top_of(s, p.x + row * p.ldx, from, to);
    if (threadIdx.x == 0) ws.key[blockIdx.x] = best;
}

// The row's largest key from its chunks' (at most 64).
__device__ __forceinline__ uint64_t row_best(const RowSpace& ws)
{
    const int lane = threadIdx.x & 63;
    uint64_t best = lane < int(gridDim.x) ? ws.key[lane] : 0;
#pragma unroll
    for (int off = 32; off; off >>= 1) best = max_key(best, __shfl_xor((unsigned long long)best, off, 64));
    return best;
}

__global__ __launch_bounds__(kThreads) void sample_histogram(SampleParams p, Division dv)
{
    fetch_arguments<sizeof(SampleParams) + sizeof(Division)>();
    __shared__ Shared s;
    const int64_t row = blockIdx.y;
    RowSpace& ws = static_cast<RowSpace*>(p.workspace)[row];
    fill_powers(s.powers);
    const Row r = row_of(p, row, row_best(ws), s.powers);
    if (r.greedy || !r.cut()) return;
    const int64_t from = blockIdx.x * dv.chunk, to = min(p.N, from + dv.chunk);
    add_to_bins(s, r, p.x + row * p.ldx, from, to);
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        if (s.count[i]) atomicAdd(&ws.count[i], s.count[i]);
        if (s.weight[i]) atomicAdd(&ws.weight[i], s.weight[i]);
    }
}

__device__ __forceinline__ void put(unsigned long long* p, unsigned long long v)
{
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned long long get(const unsigned long long* p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Bins that the cuts fall into: tokens of bins below `first` are kept,
// candidates are in [first, second] or in `kbin`.
struct Bins {
    int first, second, kbin;
    uint64_t first_count, first_weight;   // before bin `first`
    uint64_t k_count, k_weight;           // before bin `kbin`
    uint64_t total_weight;
    bool by_k;                            // top-k takes tokens away
};

__device__ Bins find_bins(Shared& s, const Row& r, const unsigned int* count, const unsigned long long* weight)
{
    Bins b;
    const int i0 = 2 * threadIdx.x;
    const unsigned int c0 = count[i0], c1 = count[i0 + 1];
    const unsigned long long w0 = weight[i0], w1 = weight[i0 + 1];
    unsigned int call, cb = c0 + c1;
    unsigned long long wall, wb = w0 + w1;
    scan_both(s, &cb, &wb, &call, &wall);
    cb -= c0 + c1, wb -= w0 + w1;
    b.total_weight = wall;
    b.by_k = r.k < r.N && uint64_t(r.k) < call;
    b.kbin = kBins;
    b.k_count = call, b.k_weight = wall;
    uint64_t upper = wall;
    if (b.by_k) {
        for (int e = 0; e < 2; ++e) {
            const uint64_t c = e ? cb + c0 : cb, n = e ? c1 : c0;
            if (c < uint64_t(r.k) && uint64_t(r.k) <= c + n) {
                s.bin = i0 + e;
                s.above_count = unsigned(c);
                s.above_weight = e ? wb + w0 : wb;
                s.sum_k = e ? wb + w0 + w1 : wb + w0;
            }
        }
        __syncthreads();
        b.kbin = s.bin;
        b.k_count = s.above_count;
        b.k_weight = s.above_weight;
        upper = s.sum_k;
    }
    b.first = b.second = b.kbin;
    b.first_count = b.k_count, b.first_weight = b.k_weight;
    if (r.top_p < 1.0) {
        // the sum that top-p refers to lies between these, its last bin then too
        const double lo = r.top_p * double(b.by_k ? b.k_weight : wall), hi = r.top_p * double(upper);
        __syncthreads();
        if (threadIdx.x == 0) s.bin = 0, s.bin2 = 0;
        __syncthreads();
        int at_lo = 0, at_hi = 0;
        for (int e = 0; e < 2; ++e) {
            if (!(e ? w1 : w0)) continue;       // (weights of 0 lie past every limit)
            const double w = double(e ? wb + w0 : wb);
            if (w < lo) at_lo = i0 + e;
            if (w < hi) at_hi = i0 + e;
        }
        wave_max(&s.bin, at_lo);
        wave_max(&s.bin2, at_hi);
        __syncthreads();
        b.first = s.bin, b.second = s.bin2;
        if (b.first >> 1 == int(threadIdx.x)) {
            s.above_count = b.first & 1 ? cb + c0 : cb;
            s.above_weight = b.first & 1 ? wb + w0 : wb;
        }
        __syncthreads();
        b.first_count = s.above_count, b.first_weight = s.above_weight;
    }
    return b;
}

// Sorts the first n keys (at most kCandidates), largest first, zeros after
// them, by a bitonic network over the next power of two.  Up to 1024 keys are
// a register of each thread: comparisons within a wave exchange lanes, the
// others go through LDS.
__device__ void sort_keys(unsigned long long* key, int n)
{
    int size = 64;
    while (size < n) size *= 2;
    for (int i = n + threadIdx.x; i < size; i += kThreads) key[i] = 0;
    __syncthreads();
    if (size <= kThreads) {
        const int i = threadIdx.x;
        const bool mine = i < size;
        unsigned long long a = mine ? key[i] : 0;
        for (int k = 2; k <= size; k *= 2)
            for (int j = k / 2; j >= 1; j /= 2) {
                unsigned long long o;
                if (j >= 64) {
                    if (mine) key[i] = a;
                    __syncthreads();
                    o = mine ? key[i ^ j] : 0;
                    __syncthreads();
                } else {
                    if (!mine) continue;
                    o = __shfl_xor(a, j, 64);
                }
                // the pair's lower place takes the larger key where its run descends
                const bool larger = ((i & k) == 0) == ((i & j) == 0);
                a = (o > a) == larger ? o : a;
            }
        if (mine) key[i] = a;
        __syncthreads();
        return;
    }
    for (int k = 2; k <= size; k *= 2)
        for (int j = k / 2; j >= 1; j /= 2) {
            for (int t = threadIdx.x; t < size / 2; t += kThreads) {
                const int i = 2 * t - (t & (j - 1));
                const unsigned long long a = key[i], b = key[i + j];
                if ((a < b) == ((i & k) == 0)) key[i] = b, key[i + j] = a;
            }
            __syncthreads();
        }
}

// The cut's key from the row's candidates: sorted, their ranks and the weight
// before them in the row's order follow from what the histogram holds before.
template <int kEach>
__device__ uint64_t cut_of_candidates(Shared& s, const Row& r, const Bins& b, unsigned long long* key, int n)
{
    sort_keys(key, n);
    unsigned long long w[kEach], sum = 0, all;
    bool in_k[kEach], in_p[kEach];
    int range = 0;
    const int at = kEach * threadIdx.x;          // this thread's candidates, in order
    if (threadIdx.x == 0) s.bin = 0, s.sum_k = b.by_k ? b.k_weight : b.total_weight, s.cut = ~0ull;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        w[e] = 0;
        in_k[e] = in_p[e] = false;
        if (at + e >= n) continue;
        const float v = value_of(uint32_t(key[at + e] >> 32));
        const int bin = bin_of(below_top(r.top, v));
        w[e] = r.fixed(r.weight(r.exponent(v)));
        in_k[e] = bin == b.kbin;
        in_p[e] = bin >= b.first && bin <= b.second;
        if (in_p[e]) range = at + e + 1;
        sum += w[e];
    }
    wave_max(&s.bin, range);                     // candidates of [first, second], the first ones
    unsigned long long before = scan(s.u, sum, &all) - sum;
    const int in_range = s.bin;
    uint64_t rank[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        rank[e] = in_p[e] ? b.first_count + (at + e) : b.k_count + (at + e) - in_range;
        if (b.by_k && in_k[e] && rank[e] < uint64_t(r.k)) atomicAdd(&s.sum_k, w[e]);
    }
    __syncthreads();
    const double limit = r.top_p * double(s.sum_k);
    int keep = 0;                                // kept candidates come first too
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        if (in_p[e] && rank[e] < uint64_t(r.k) &&
            (r.top_p >= 1.0 || rank[e] == 0 || double(b.first_weight + before) < limit))
            keep = at + e + 1;
        before += w[e];
    }
    if (threadIdx.x == 0) s.bin2 = 0;
    __syncthreads();
    wave_max(&s.bin2, keep);
    __syncthreads();
    return s.bin2 ? key[s.bin2 - 1] : ~0ull;
}

// Where one range of bins holds the cut, by rank or by weight: a second
// histogram, of the range's candidates over 1024 places of the order between
// its ends, then those of the place that holds the cut against each other.
// False where more than 64 lie there.
__device__ bool cut_by_places(Shared& s, const Row& r, const Bins& b, const unsigned long long* key, int n, uint64_t* cut)
{
    const bool by_k = r.top_p >= 1.0;
    if (b.by_k && !by_k) return false;
    constexpr int kPlaces = 1024;
    static_assert(kPlaces == kThreads, "a thread scans a place");
    uint32_t lo = ~0u, hi = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint32_t o = uint32_t(key[i] >> 32);
        lo = min(lo, o), hi = max(hi, o);
    }
    __syncthreads();
    if (threadIdx.x == 0) s.in_bin = ~0u, s.above_count = 0, s.flag = 0, s.bin = 0, s.cut = ~0ull;
    s.weight[threadIdx.x] = 0, s.count[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int off = 32; off; off >>= 1) {
        lo = min(lo, uint32_t(__shfl_xor(int(lo), off, 64)));
        hi = max(hi, uint32_t(__shfl_xor(int(hi), off, 64)));
    }
    if ((threadIdx.x & 63) == 0) atomicMin(&s.in_bin, lo), atomicMax(&s.above_count, hi);
    __syncthreads();
    lo = s.in_bin, hi = s.above_count;
    const float scale = float(kPlaces) / (float(hi - lo) + 1.0f);
    const auto place = [&](unsigned long long k) { return min(kPlaces - 1, int(float(hi - uint32_t(k >> 32)) * scale)); };
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int at = place(key[i]);
        atomicAdd(&s.count[at], 1u);
        atomicAdd(&s.weight[at], r.fixed(r.weight(r.exponent(value_of(uint32_t(key[i] >> 32))))));
    }
    __syncthreads();
    const unsigned int c = s.count[threadIdx.x];
    const unsigned long long w = s.weight[threadIdx.x];
    unsigned int call;
    unsigned long long wall;
    const uint64_t cb = b.first_count + scan(s.n, c, &call) - c;
    const uint64_t wb = b.first_weight + scan(s.u, w, &wall) - w;
    const double limit = r.top_p * double(b.total_weight);
    // the last place that begins inside the cut
    const bool inside = c && (by_k ? cb < uint64_t(r.k) : cb == 0 || double(wb) < limit);
    wave_max(&s.bin, inside ? int(threadIdx.x) + 1 : 0);
    __syncthreads();
    const int at = s.bin - 1;
    if (int(threadIdx.x) == at) s.sum_k = cb, s.above_weight = wb;
    __syncthreads();
    const uint64_t before_count = s.sum_k, before_weight = s.above_weight;
    unsigned long long* chosen = s.weight;      // that place's candidates
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads)
        if (place(key[i]) == at) {
            const int j = atomicAdd(&s.flag, 1);
            if (j < 64) chosen[j] = key[i];
        }
    __syncthreads();
    const int m = s.flag;
    if (m > 64) return false;
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        const unsigned long long mine = lane < m ? chosen[lane] : 0;
        const unsigned long long mw = lane < m ? r.fixed(r.weight(r.exponent(value_of(uint32_t(mine >> 32))))) : 0;
        uint64_t rank = before_count, weight = before_weight;
        for (int j = 0; j < m; ++j) {
            const unsigned long long o = __shfl(mine, j, 64), ow = __shfl(mw, j, 64);
            if (o > mine) ++rank, weight += ow;
        }
        const bool keep = lane < m && (by_k ? rank < uint64_t(r.k) : rank == 0 || double(weight) < limit);
        if (keep) atomicMin(&s.cut, mine);
    }
    __syncthreads();
    *cut = s.cut;
    return true;
}

// The cut's key where there are at most 64 candidates (the usual row): each
// wave compares all of them with its share, the first wave then has their
// ranks and the weights before them.
__device__ uint64_t cut_of_few(Shared& s, const Row& r, const Bins& b, const unsigned long long* key, int n)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    unsigned long long* before = s.weight + kGroups;
    unsigned long long* weight = before + 64;
    unsigned int* rank = s.count;
    const bool is = lane < n;
    const unsigned long long mine = is ? key[lane] : 0;
    const float v = value_of(uint32_t(mine >> 32));
    const unsigned long long w = is ? r.fixed(r.weight(r.exponent(v))) : 0;
    if (wave == 0) before[lane] = 0, weight[lane] = w, rank[lane] = 0;
    if (threadIdx.x == 0) s.cut = ~0ull;
    __syncthreads();
    unsigned int ahead = 0;
    unsigned long long sum = 0;
    for (int j = wave; j < n; j += kWaves)
        if (key[j] > mine) ++ahead, sum += weight[j];
    if (is && ahead) atomicAdd(&rank[lane], ahead), atomicAdd(&before[lane], sum);
    __syncthreads();
    if (wave == 0) {
        const int bin = is ? bin_of(below_top(r.top, v)) : -1;
        const bool in_k = is && bin == b.kbin, in_p = is && bin >= b.first && bin <= b.second;
        const int in_range = __popcll(__ballot(in_p));      // the first ones in order
        const uint64_t place = in_p ? b.first_count + rank[lane] : b.k_count + rank[lane] - in_range;
        unsigned long long sum_k = in_k && place < uint64_t(r.k) ? w : 0;
#pragma unroll
        for (int off = 32; off; off >>= 1) sum_k += __shfl_xor(sum_k, off, 64);
        sum_k = b.by_k ? b.k_weight + sum_k : b.total_weight;
        const double limit = r.top_p * double(sum_k);
        const bool keep = in_p && place < uint64_t(r.k) &&
                          (r.top_p >= 1.0 || place == 0 || double(b.first_weight + before[lane]) < limit);
        const int kept = __popcll(__ballot(keep));
        if (keep && int(rank[lane]) == kept - 1) s.cut = mine;
    }
    __syncthreads();
    return s.cut;
}

// ONE: a work-group has the whole row and does the first two steps as well.
template <bool ONE>
__global__ __launch_bounds__(kThreads) void sample_draw(SampleParams p, Division dv)
{
    fetch_arguments<sizeof(SampleParams) + sizeof(Division)>();
    __shared__ Shared s;
    __shared__ unsigned long long key[kCandidates];
    const int64_t row = blockIdx.y;
    RowSpace& ws = static_cast<RowSpace*>(p.workspace)[ONE ? 0 : row];
    const float* x = p.x + row * p.ldx;
    const int64_t from = blockIdx.x * dv.chunk, to = min(p.N, from + dv.chunk);
    // A wave takes every 16th group of the chunk, 256 tokens a round, four a
    // lane; kAhead rounds are on their way while as many are used.
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // (a chunk is below 2^31 tokens, and steps past its end below 2^32)
    const uint32_t group = uint32_t(dv.group), rounds = group / 256, count = uint32_t(to - from);
    const float* chunk = x + from;
    const auto step = [&](uint32_t& at, uint32_t& in_group) {
        at += 256;
        if (++in_group == rounds) in_group = 0, at += (kWaves - 1) * group;
    };
    const auto load = [&](uint32_t at, float* v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (at + 256 <= count) v[e] = (chunk + at)[64 * e + lane];
            else v[e] = chunk[min(at + 64 * e + lane, count - 1)];
        }
    };
    uint32_t at = uint32_t(__builtin_amdgcn_readfirstlane(wave)) * group, in_group = 0, next = at, next_group = 0;
    float ahead[kAhead][4];
    const auto load_ahead = [&] {
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            load(next, ahead[a]);
            step(next, next_group);
        }
    };
    load_ahead();
    fill_powers(s.powers);
    const Row r = row_of(p, row, ONE ? top_of(s, x, from, to) : row_best(ws), s.powers);
    if (r.greedy) {
        if (blockIdx.x == 0 && threadIdx.x == 0) p.idx[row] = r.top_idx;
        return;
    }
    Bins b;
    b.first = b.second = b.kbin = kBins;
    b.by_k = false;
    const bool cut = r.cut();
    if (cut) {
        if (ONE) add_to_bins(s, r, x, from, to);
        b = ONE ? find_bins(s, r, s.count, s.weight) : find_bins(s, r, ws.count, ws.weight);
    }
    // d = top - x of the tokens kept for sure (below `sure`), and of the candidates
    const float sure = edge_of(b.first), end = edge_of(b.second + 1), k_from = edge_of(b.kbin), k_to = edge_of(b.kbin + 1);
    // No token below `least` counts: past the last candidate's bin, or in rows
    // without a cut below min_p (the slack covers every rounding).
    float least = r.low;
    {
        const float reach = fmaxf(end, b.kbin < kBins ? k_to : 0.0f), slack = fabsf(r.top) * 0x1p-20f;
        if (cut && end == end && (b.kbin >= kBins || k_to == k_to)) least = fmaxf(least, r.top - reach * (1.0f + 0x1p-20f) - slack);
        if (!cut && r.floor > 0.0)
            least = fmaxf(least, float(double(r.top) + (double(__log2f(float(r.floor))) - 1e-3) / r.rate) - slack);
    }
    double* group_sum = reinterpret_cast<double*>(s.weight);
    __syncthreads();
    group_sum[threadIdx.x] = 0.0;
    if (threadIdx.x == 0) s.flag = 0;
    __syncthreads();
    double w = 0.0;
    const auto round = [&](float* v) {
        if (at >= count) return;
        const uint32_t here = at, g = here / group;
        step(at, in_group);
        if (here + 256 > count) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (here + 64 * e + lane >= count) v[e] = -INFINITY;
        }
        if (__any(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])) >= least)) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!(v[e] >= least)) continue;
                const float d = below_top(r.top, v[e]);
                if (!(d >= sure)) {
                    w += r.drawn(v[e]);
                } else if (!(d >= end) || (d >= k_from && !(d >= k_to))) {
                    const int c = atomicAdd(&s.flag, 1);
                    if (c < kCandidates) key[c] = argmax_key(v[e], uint32_t(from) + here + 64 * e + lane);
                }
            }
        }
        if (in_group && at < count) return;
        if (__any(w != 0.0)) w = wave_sum(w);
        if (lane == 0) {
            if (ONE) group_sum[g] = w;
            else put(&ws.sum[blockIdx.x * dv.groups + g], (unsigned long long)__double_as_longlong(w));
        }
        w = 0.0;
    };
    while (at < count) {
        float v[kAhead][4];
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[a][e] = ahead[a][e];
        load_ahead();
#pragma unroll
        for (int a = 0; a < kAhead; ++a) round(v[a]);
    }
    __syncthreads();
    // the work-group's candidates join the row's list
    unsigned int n = unsigned(s.flag);
    if (!ONE) {
        if (n) {
            if (threadIdx.x == 0) s.in_bin = atomicAdd(&ws.candidates, n);
            __syncthreads();
            const unsigned int at = s.in_bin;
            for (int i = threadIdx.x; i < int(min(n, unsigned(kCandidates))); i += kThreads)
                if (at + i < unsigned(kCandidates)) put(&ws.candidate[at + i], key[i]);
        }
        // every store of the work-group is at the device-wide level before it counts itself
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0) s.flag = atomicAdd(&ws.arrived, 1u) == gridDim.x - 1;
        __syncthreads();
        if (!s.flag) return;
        n = __hip_atomic_load(&ws.candidates, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }

    // ---- the row's last work-group
    if (n > kCandidates) {
        draw_by_selection(s, p, row, r);
        return;
    }
    const int groups = int((p.N + dv.group - 1) / dv.group);
    double own = 0.0;
    if (int(threadIdx.x) < groups)
        own = ONE ? group_sum[threadIdx.x] : __longlong_as_double((long long)get(&ws.sum[threadIdx.x]));
    const double u = p.u[row];
    uint64_t last = 0;
    if (n) {
        if (!ONE) {
            for (int i = threadIdx.x; i < int(n); i += kThreads) key[i] = get(&ws.candidate[i]);
            __syncthreads();
        }
        if (n <= 64)
            last = cut_of_few(s, r, b, key, int(n));
        else if (!cut_by_places(s, r, b, key, int(n), &last))
            last = n <= kThreads ? cut_of_candidates<1>(s, r, b, key, int(n))
                                 : cut_of_candidates<kCandidates / kThreads>(s, r, b, key, int(n));
        // Kept candidates join their groups' sums, in fixed point, where the
        // smallest kept weight still counts and the order does not.
        unsigned long long* add = s.weight + kGroups;
        __syncthreads();
        add[threadIdx.x] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < int(n); i += kThreads) {
            if (key[i] < last) continue;
            const double x = r.drawn(value_of(uint32_t(key[i] >> 32)));
            if (x > 0.0) atomicAdd(&add[int64_t(~uint32_t(key[i])) / dv.group], max(1ull, r.fixed(x)));
        }
        __syncthreads();
        own += double(add[threadIdx.x]) / r.unit;
    }
    const int64_t pick = draw_token(s, r, x, last, own, dv.group, u);
    if (threadIdx.x == 0) p.idx[row] = pick < p.N ? int32_t(pick) : r.top_idx;
}

}  // namespace

size_t sample_workspace_need(int64_t m, int64_t N)
{
    if (m == 0 || division(m, N).chunks == 1) return 256;
    return size_t(m) * sizeof(RowSpace);
}

// The largest need of up to m rows of up to N logits: rows of several
// work-groups come in batches of up to kResident / 2.
size_t sample_workspace_bytes(int64_t m, int64_t N)
{
    return sample_workspace_need(m < kResident / 2 ? m : kResident / 2, N);
}

hipError_t launch_sample(const SampleParams& p, hipStream_t s)
{
    const Division d = division(p.m, p.N);
    const dim3 grid{unsigned(d.chunks), unsigned(p.m), 1};
    if (d.chunks == 1) {
        hipLaunchKernelGGL(sample_draw<true>, grid, dim3(kThreads), 0, s, p, d);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(sample_top, grid, dim3(kThreads), 0, s, p, d);
    if (p.top_k || p.top_p) hipLaunchKernelGGL(sample_histogram, grid, dim3(kThreads), 0, s, p, d);
    hipLaunchKernelGGL(sample_draw<false>, grid, dim3(kThreads), 0, s, p, d);
    return hipGetLastError();
}

}  // namespace qg
