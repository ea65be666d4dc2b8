// A token per row of logits by temperature, top-k, top-p and min-p, from
// given uniform numbers.
//
// The tokens that survive the cuts are always the first ones of the order
// (larger logit, then lower index), so each cut is a place in that order: a
// key and, where several logits equal it, the last index kept.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "argmax_key.h"
#include "decode_ops.h"

namespace qg {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 2048;
constexpr int kTile = kThreads * 4;

// Weights in fixed point for the sums over the order's head: integer sums do
// not depend on the order of the atomics.  N weights of at most 1 fit 62 bits.
__device__ __forceinline__ int weight_bits(int64_t N)
{
    int b = 62 - (64 - __clzll(uint64_t(N)));
    return b > 52 ? 52 : b;
}

__device__ __forceinline__ uint32_t order_of(float v) { return uint32_t(argmax_key(v, 0) >> 32); }

__device__ __forceinline__ double weight_of(float x, float top, double t)
{
    if (x == top) return 1.0;
    if (x == -INFINITY) return 0.0;
    return exp((double(x) - double(top)) / t);
}

struct Shared {
    unsigned long long weight[kBins];
    unsigned int count[kBins];
    unsigned long long key[kWaves];
    double wave_sum[kWaves];
    unsigned int wave_cnt[kWaves];
    uint32_t prefix;
    uint64_t above_count, above_weight, in_bin;
    int64_t pick;
};

// The last kept key of a cut: by count (the k-th element) or by weight (the
// last one whose preceding weight is below `limit`).  Three passes over the
// key's 11, 11 and 10 bits.
__device__ void select(Shared& s, const float* x, int64_t N, float top, double t, bool by_count, uint64_t k,
                       double limit, uint32_t* cut, uint64_t* above_count, uint64_t* above_weight, uint64_t* ties)
{
    const int bits = weight_bits(N);
    uint32_t prefix = 0, known = 0;
    uint64_t ac = 0, aw = 0;
    for (int level = 0; level < 3; ++level) {
        const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
        const int width = level == 2 ? 10 : 11;
        for (int i = threadIdx.x; i < kBins; i += kThreads) s.weight[i] = 0, s.count[i] = 0;
        __syncthreads();
        for (int64_t i = threadIdx.x; i < N; i += kThreads) {
            const float v = x[i];
            const uint32_t o = order_of(v);
            if ((o & known) != prefix) continue;
            const int bin = int((o >> shift) & ((1u << width) - 1));
            atomicAdd(&s.count[bin], 1u);
            const double w = weight_of(v, top, t);
            atomicAdd(&s.weight[bin], (unsigned long long)(ldexp(w, bits) + 0.5));
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            uint64_t c = ac, w = aw;
            int found = -1;
            uint64_t fc = 0, fw = 0;
            for (int bin = kBins - 1; bin >= 0; --bin) {
                if (!s.count[bin]) continue;
                if (by_count ? c >= k : (found >= 0 && !(double(w) < limit))) break;
                found = bin, fc = c, fw = w;
                c += s.count[bin];
                w += s.weight[bin];
            }
            s.prefix = prefix | (uint32_t(found) << shift);
            s.above_count = fc;
            s.above_weight = fw;
            s.in_bin = s.count[found];
        }
        __syncthreads();
        prefix = s.prefix;
        known |= ((1u << width) - 1) << shift;
        ac = s.above_count, aw = s.above_weight;
        *ties = s.in_bin;
        __syncthreads();
    }
    *cut = prefix;
    *above_count = ac;
    *above_weight = aw;
}

// Inclusive sums over the block in thread order; total of all in *total.
__device__ double scan(Shared& s, double v, double* total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int off = 1; off < 64; off <<= 1) {
        const double o = __shfl_up(v, off, 64);
        if (lane >= off) v += o;
    }
    if (lane == 63) s.wave_sum[wave] = v;
    __syncthreads();
    double before = 0.0, all = 0.0;
    for (int w = 0; w < kWaves; ++w) {
        if (w == wave) before = all;
        all += s.wave_sum[w];
    }
    __syncthreads();
    *total = all;
    return before + v;
}

__global__ __launch_bounds__(kThreads) void sample_rows(SampleParams p)
{
    __shared__ Shared s;
    const int64_t row = blockIdx.x;
    const float* x = p.x + row * p.ldx;
    const int64_t N = p.N;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint64_t best = 0;
    for (int64_t i = threadIdx.x; i < N; i += kThreads) best = max_key(best, argmax_key(x[i], uint32_t(i)));
    for (int off = 32; off; off >>= 1) best = max_key(best, __shfl_xor((unsigned long long)best, off, 64));
    if (lane == 0) s.key[wave] = best;
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) best = max_key(best, s.key[w]);
    const int32_t top_idx = key_index(best);
    const float top = x[top_idx];
    const float temp = p.temperature ? p.temperature[row] : 1.0f;
    // greedy, or nothing to weigh: a NaN wins, and a row of -inf gives its first
    if (!(temp > 0.0f) || top != top || top == -INFINITY) {
        if (threadIdx.x == 0) p.idx[row] = top_idx;
        return;
    }
    const double t = temp;
    const int bits = weight_bits(N);
    const int64_t k = p.top_k && p.top_k[row] > 0 ? min(int64_t(p.top_k[row]), N) : N;
    const float top_p = p.top_p ? p.top_p[row] : 1.0f;
    const float min_p = p.min_p ? p.min_p[row] : 0.0f;
    uint32_t cut = 0;
    uint64_t kept_ties = N, ties = N;
    double sum = -1.0;
    __syncthreads();
    if (k < N) {
        uint64_t ac, aw;
        select(s, x, N, top, t, true, uint64_t(k), 0.0, &cut, &ac, &aw, &ties);
        kept_ties = uint64_t(k) - ac;
        const uint32_t raw = (cut & 0x80000000u) ? cut & 0x7fffffffu : ~cut;
        const uint64_t w = (unsigned long long)(ldexp(weight_of(__uint_as_float(raw), top, t), bits) + 0.5);
        sum = double(aw + w * kept_ties);
    }
    if (top_p < 1.0f) {
        if (sum < 0.0) {
            // the whole row's weight, in the same fixed point
            if (threadIdx.x == 0) s.above_weight = 0;
            __syncthreads();
            unsigned long long mine = 0;
            for (int64_t i = threadIdx.x; i < N; i += kThreads)
                mine += (unsigned long long)(ldexp(weight_of(x[i], top, t), bits) + 0.5);
            atomicAdd((unsigned long long*)&s.above_weight, mine);
            __syncthreads();
            sum = double(s.above_weight);
            __syncthreads();
        }
        uint32_t pcut;
        uint64_t ac, aw, pties;
        const double limit = double(top_p) * sum;
        select(s, x, N, top, t, false, 0, limit, &pcut, &ac, &aw, &pties);
        const uint32_t raw = (pcut & 0x80000000u) ? pcut & 0x7fffffffu : ~pcut;
        const uint64_t w = (unsigned long long)(ldexp(weight_of(__uint_as_float(raw), top, t), bits) + 0.5);
        // ties j = 0, 1, ... are kept while the weight before them is below the limit
        uint64_t lo = 1, hi = pties;
        while (lo < hi) {
            const uint64_t mid = (lo + hi + 1) / 2;
            if (double(aw + w * (mid - 1)) < limit) lo = mid;
            else hi = mid - 1;
        }
        if (pcut > cut || (pcut == cut && lo < kept_ties)) cut = pcut, kept_ties = lo, ties = pties;
    }
    // Index of the last tie kept.
    int64_t last_tie = N;
    if (kept_ties < ties) {
        uint64_t seen = 0;
        for (int64_t base = 0; base < N && last_tie == N; base += kTile) {
            int mine = 0;
            for (int j = 0; j < 4; ++j) {
                const int64_t i = base + threadIdx.x * 4 + j;
                if (i < N && order_of(x[i]) == cut) ++mine;
            }
            double total;
            const uint64_t upto = seen + uint64_t(scan(s, double(mine), &total));
            if (threadIdx.x == 0) s.pick = N;
            __syncthreads();
            uint64_t at = upto - mine;
            for (int j = 0; j < 4; ++j) {
                const int64_t i = base + threadIdx.x * 4 + j;
                if (i < N && order_of(x[i]) == cut && ++at == kept_ties) s.pick = i;
            }
            __syncthreads();
            last_tie = s.pick;
            seen += uint64_t(total);
            __syncthreads();
        }
    }
    const double floor_w = min_p != min_p ? 0.0 : fmin(double(min_p), 1.0);
    const double u = p.u[row];
    auto kept = [&](int64_t i) -> double {
        if (i >= N) return 0.0;
        const uint32_t o = order_of(x[i]);
        if (o < cut || (o == cut && i > last_tie)) return 0.0;
        const double w = weight_of(x[i], top, t);
        return w >= floor_w ? w : 0.0;
    };
    double all = 0.0;
    for (int64_t base = 0; base < N; base += kTile) {
        double mine = 0.0, total;
        for (int j = 0; j < 4; ++j) mine += kept(base + threadIdx.x * 4 + j);
        scan(s, mine, &total);
        all += total;
    }
    const double target = u * all;
    double run = 0.0;
    for (int64_t base = 0; base < N; base += kTile) {
        double w[4], mine = 0.0, total;
        for (int j = 0; j < 4; ++j) mine += w[j] = kept(base + threadIdx.x * 4 + j);
        const double upto = scan(s, mine, &total);
        if (run + total > target) {
            if (threadIdx.x == 0) s.pick = N;
            __syncthreads();
            double cum = run + (upto - mine);
            int64_t pick = N;
            for (int j = 3; j >= 0; --j) {
                double c = cum;
                for (int q = 0; q <= j; ++q) c += w[q];
                if (w[j] > 0.0 && c > target) pick = base + threadIdx.x * 4 + j;
            }
            if (pick < N) atomicMin((unsigned long long*)&s.pick, (unsigned long long)pick);
            __syncthreads();
            if (s.pick < N) {
                if (threadIdx.x == 0) p.idx[row] = int32_t(s.pick);
                return;
            }
        }
        run += total;
        __syncthreads();
    }
    // u of 1 or more, or a NaN: the most likely token
    if (threadIdx.x == 0) p.idx[row] = top_idx;
}

}  // namespace

size_t sample_workspace_bytes(int64_t m, int64_t N)
{
    (void)m, (void)N;
    return 256;
}

hipError_t launch_sample(const SampleParams& p, hipStream_t s)
{
    hipLaunchKernelGGL(sample_rows, dim3(unsigned(p.m)), dim3(kThreads), 0, s, p);
    return hipGetLastError();
}

}  // namespace qg
