// Rotary positions on queries and keys, with keys and values quantised into
// the paged cache in blocks of 32 dimensions (4-bit codes and an exponent
// byte), in one pass over the QKV projection's output.
//
// A block's scale is 2^e with e the smallest by which its largest magnitude is
// at most 7; a code is the nearest of 0, 0.5, 1, 1.5, 2, 3, 4 and 6 to the
// element over the scale, ties to the even code.  A rotated key that lies next
// to a border between two codes, or a block's largest next to 7 scales, must
// fall to the side of the definition: keys are rotated in fp64 from angles that
// are exact (as in rope.hip), and both decisions are integer comparisons.
// Queries take the same fp32 steps as with the other caches.
//
// What bounds it: of many tokens the memory (6001 tokens of 32 + 8 heads of 128
// in bf16, 129 MB: 28.6 us, 24.2 where they lie in the last-level cache, a copy
// 25.5; vector instructions busy in 56% of the cycles); of a few the call on the
// host (one token 8.3 us of it, 4.4 on the GPU).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decode_ops.h"

namespace qg {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kRun = 4;           // dimensions of a thread; eight threads are a block

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }

template <bool F32>
__device__ __forceinline__ float load(const void* p, int64_t i)
{
    return F32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

template <bool F32>
__device__ __forceinline__ void load_run(const void* p, int64_t i, float* x)
{
    if (F32) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = v[j];
    } else {
        const u32x2 v = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x[2 * j] = __uint_as_float(v[j] << 16);
            x[2 * j + 1] = __uint_as_float(v[j] & 0xffff0000u);
        }
    }
}

// cos and sin of pos turns of `per` each, modulo one turn.
__device__ __forceinline__ void turn(uint64_t pos, uint64_t per, float amplitude, float* cs, float* sn)
{
    sincospif(float(int64_t(pos * per)) * 0x1p-63f, sn, cs);   // 2^63 is half a turn
    *sn *= amplitude;
    *cs *= amplitude;
}
__device__ __forceinline__ void turn(uint64_t pos, uint64_t per, float amplitude, double* cs, double* sn)
{
    sincospi(double(int64_t(pos * per)) * 0x1p-63, sn, cs);
    *sn *= double(amplitude);
    *cs *= double(amplitude);
}

// The dimensions [d, d + 4) of a head that a thread holds, and their partners.
struct Run {
    int d;
    bool turns[kRun];
    bool second[kRun];     // of its pair
    int pair[kRun], other[kRun];
};

template <bool INTER>
__device__ __forceinline__ Run make_run(int d, int rot)
{
    Run r;
    r.d = d;
    const int half = rot / 2;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        const int e = d + i;
        r.turns[i] = e < rot;
        r.second[i] = INTER ? (e & 1) : e >= half;
        r.pair[i] = INTER ? e / 2 : r.second[i] ? e - half : e;
        r.other[i] = INTER ? e ^ 1 : r.second[i] ? e - half : e + half;
    }
    return r;
}

// Elements and the partners that turn with them.  WIDE: the run lies on one
// side of every border, and so does its partners'.
template <bool F32, bool INTER, bool WIDE>
__device__ __forceinline__ void load_pairs(const void* src, int64_t at, const Run& r, bool rotated, float* x, float* z)
{
    if (WIDE) {
        load_run<F32>(src, at + r.d, x);
        if (INTER) {
#pragma unroll
            for (int i = 0; i < kRun; ++i) z[i] = x[i ^ 1];
        } else if (rotated && r.turns[0]) {
            load_run<F32>(src, at + r.other[0], z);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            x[i] = load<F32>(src, at + r.d + i);
            z[i] = rotated && r.turns[i] ? load<F32>(src, at + r.other[i]) : 0.0f;
        }
    }
}

// A token's angles, each worked out by one thread of the work-group: in 32 bits
// for queries by the lower half of it, in 64 for keys by the upper (8191 tokens
// of 32 + 8 heads, written and read back: 49 us, 51 where each thread works out
// its queries' angles; 6613 tokens of 14 + 2 heads of 96 in the second kernel
// below: 23 us, 38 where it does so with its keys' too).
struct Table {
    float cs[kMaxRotPairs], sn[kMaxRotPairs];
    double key_cs[kMaxRotPairs], key_sn[kMaxRotPairs];

    __device__ __forceinline__ void fill(const RopeParams& p, uint64_t pos, bool queries, bool keys)
    {
        static_assert(kThreads == 2 * kMaxRotPairs, "a thread a pair");
        const int i = threadIdx.x % kMaxRotPairs;
        if (i < p.rot_dim / 2) {
            if (threadIdx.x >= kMaxRotPairs) {
                if (keys) turn(pos, p.turns[i], p.amplitude, &key_cs[i], &key_sn[i]);
            } else if (queries) {
                turn(pos, p.turns[i], p.amplitude, &cs[i], &sn[i]);
            }
        }
        __syncthreads();
    }
};

// Those of a run's dimensions.
template <class T>
struct Angles {
    T cs[kRun], sn[kRun];      // sin with the sign that the partner takes

    __device__ __forceinline__ void fill(const T* all_cs, const T* all_sn, const Run& r)
    {
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            cs[i] = T(1), sn[i] = T(0);
            if (r.turns[i]) cs[i] = all_cs[r.pair[i]], sn[i] = r.second[i] ? all_sn[r.pair[i]] : -all_sn[r.pair[i]];
        }
    }
};

// y in fp32, rounded to odd where it is not exact: a later rounding to fewer
// bits, and a comparison with a number of fewer bits, go as those of y.
__device__ __forceinline__ float to_odd(double y)
{
    const float f = float(y);
    const double d = __builtin_fabs(double(f)), a = __builtin_fabs(y);
    const uint32_t bits = __float_as_uint(f);
    const uint32_t step = bits & 1 ? 0 : d < a ? 1 : d > a ? ~0u : 0;
    return __uint_as_float(bits + step);
}

// A block's largest magnitude, as bits, to the exponent of its scale: 1.75 2^k
// is 7 times 2^(k - 2).
__device__ __forceinline__ int exponent_of(uint32_t most)
{
    const int e = int(most >> 23) - 127 - 2 + ((most & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, -125), 125);
}
__device__ __forceinline__ float scale_of(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }
__device__ __forceinline__ bool is_nan(uint32_t most) { return most > 0x7f800000u; }
__device__ __forceinline__ uint32_t magnitude(float y) { return __float_as_uint(y) & 0x7fffffffu; }

// The same value of the threads around: of the other in its pair, of the other
// pair of its four, of the other four of its eight (where each four agree).
__device__ __forceinline__ uint32_t most_of_four(uint32_t x)
{
    x = max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0xb1, 0xf, 0xf, true)));
    return max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0x4e, 0xf, 0xf, true)));
}
__device__ __forceinline__ uint32_t other_four(uint32_t x) { return uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0x141, 0xf, 0xf, true)); }

// A thread's four elements into the cache, with the seven threads around it
// that hold the rest of their block.
__device__ __forceinline__ void store_block(const double* x, int d, uint8_t* codes, uint8_t* exponents)
{
    float y[kRun];
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        y[i] = to_odd(x[i]);
        most = max(most, magnitude(y[i]));
    }
    most = most_of_four(most);
    most = max(most, other_four(most));
    const int e = exponent_of(most);
    uint32_t word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, y[0], y[1], scale_of(e), 0);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, y[2], y[3], scale_of(e), 1);
    *reinterpret_cast<uint16_t*>(codes + d / 2) = uint16_t(is_nan(most) ? 0 : word);
    if (d % kBlock == 0) exponents[d / kBlock] = uint8_t(is_nan(most) ? 255 : e + 127);
}

// Rows on 16 bytes, and pairs (i, i + rot_dim / 2) with rot_dim and the head in
// whole 64s, or pairs of neighbours with rot_dim in whole 8s.  As rope.hip's
// wide kernel: a thread holds one eighth-of-a-dimension place, two runs of four
// elements, of every LANES-th head.  Runs that turn with one another lie in
// blocks of eight threads each, runs of neighbours in one of four threads.
template <bool F32, bool INTER>
__global__ __launch_bounds__(kThreads) void rope_append_mxfp4_wide(RopeParams p, BlockView blocks)
{
    __shared__ __align__(16) Table table;
    const int64_t token = blockIdx.x;
    const int dim = p.cache.head_dim, places = dim / 8;
    const int lanes = kThreads / places;             // heads at a time
    const int j = threadIdx.x % places, first = threadIdx.x / places + blockIdx.y * lanes;
    const int kv_heads = p.cache.kv_heads, heads = p.q_heads + 2 * kv_heads;
    const uint64_t pos = uint64_t(int64_t(p.pos[token]));
    const int64_t slot = p.slots[token], page = slot >> p.cache.page_shift;
    const bool live = slot >= 0 && page < p.cache.pages;
    // (one round of heads a work-group, or all of them)
    const int round = blockIdx.y;
    const bool keys = live && (gridDim.y == 1 || (round >= p.q_heads / lanes && round <= (p.q_heads + kv_heads - 1) / lanes));
    table.fill(p, pos, gridDim.y == 1 || round * lanes < p.q_heads, keys);
    const bool turns = 8 * j < p.rot_dim, split = turns && !INTER;
    const int a = split ? 4 * j : 8 * j, b = split ? a + p.rot_dim / 2 : a + 4;
    const int step = lanes * gridDim.y;
    int head = first < int(blockIdx.y + 1) * lanes ? first : heads;     // (threads past the last place have none)
    if (head < p.q_heads) {
        float cs[4], sn[4];
        if (turns) {
#pragma unroll
            for (int i = 0; i < 4; ++i) cs[i] = table.cs[4 * j + i], sn[i] = table.sn[4 * j + i];
        }
        for (; head < p.q_heads; head += step) {
            const int64_t at = token * p.q_token + head * p.q_head;
            float x[8], y[8];
            load_run<F32>(p.q, at + a, x);
            load_run<F32>(p.q, at + b, x + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = INTER ? 2 * i : i, o = INTER ? 2 * i + 1 : i + 4;
                y[e] = turns ? __builtin_fmaf(x[e], cs[i], -(x[o] * sn[i])) : x[e];
                y[o] = turns ? __builtin_fmaf(x[o], cs[i], x[e] * sn[i]) : x[o];
            }
            uint16_t* out = p.q_out + token * p.o_token + head * p.o_head;
            bf16x4 u, v;
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = (__bf16)y[i], v[i] = (__bf16)y[4 + i];
            *reinterpret_cast<bf16x4*>(out + a) = u;
            *reinterpret_cast<bf16x4*>(out + b) = v;
        }
    }
    if (!live) return;               // (all threads of the work-group)
    const int64_t row = slot & ((int64_t(1) << p.cache.page_shift) - 1);
    const int64_t cell = (page * p.cache.page_stride + row * p.cache.slot_stride) / 2;
    const int64_t block = page * blocks.page_stride + row * blocks.slot_stride;
    for (; head < heads; head += step) {
        const bool is_k = head < p.q_heads + kv_heads;
        const int h = head - p.q_heads - (is_k ? 0 : kv_heads);
        const void* src = is_k ? p.k : p.v;
        const int64_t at = is_k ? token * p.k_token + h * p.k_head : token * p.v_token + h * p.v_head;
        float x[8], y[8];
        load_run<F32>(src, at + a, x);
        load_run<F32>(src, at + b, x + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i];
        if (turns && is_k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = INTER ? 2 * i : i, o = INTER ? 2 * i + 1 : i + 4;
                const double c = table.key_cs[4 * j + i], s = table.key_sn[4 * j + i], u = double(x[e]), v = double(x[o]);
                y[e] = to_odd(__builtin_fma(u, c, -(v * s)));
                y[o] = to_odd(__builtin_fma(v, c, u * s));
            }
        }
        uint32_t most_a = 0, most_b = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) most_a = max(most_a, magnitude(y[i])), most_b = max(most_b, magnitude(y[4 + i]));
        if (!split) most_a = most_b = max(most_a, most_b);
        most_a = most_of_four(most_a);
        most_b = most_of_four(most_b);
        const uint32_t more_a = other_four(most_a), more_b = other_four(most_b);
        if (split) most_a = max(most_a, more_a), most_b = max(most_b, more_b);
        const int ea = exponent_of(most_a), eb = exponent_of(most_b);
        uint32_t word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, y[0], y[1], scale_of(ea), 0);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, y[2], y[3], scale_of(ea), 1);
        if (is_nan(most_a)) word = 0;
        uint32_t more = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, y[4], y[5], scale_of(eb), 0);
        more = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(more, y[6], y[7], scale_of(eb), 1);
        if (is_nan(most_b)) more = 0;
        const uint8_t byte_a = uint8_t(is_nan(most_a) ? 255 : ea + 127), byte_b = uint8_t(is_nan(most_b) ? 255 : eb + 127);
        uint8_t* codes = (is_k ? p.cache.k : p.cache.v) + cell + h * (p.cache.head_stride / 2);
        uint8_t* exponents = (is_k ? blocks.k : blocks.v) + block + h * blocks.head_stride;
        if (split) {
            *reinterpret_cast<uint16_t*>(codes + a / 2) = uint16_t(word);
            *reinterpret_cast<uint16_t*>(codes + b / 2) = uint16_t(more);
            if (j % 8 == 0) exponents[a / kBlock] = byte_a, exponents[b / kBlock] = byte_b;
        } else {
            *reinterpret_cast<uint32_t*>(codes + a / 2) = word | more << 16;
            if (j % 4 == 0) exponents[a / kBlock] = byte_a;
        }
    }
}

// Any rot_dim, alignment and stride.  A thread holds four neighbours; a
// work-group takes rounds of heads of one token: first of queries, then of
// keys, then of values, as many heads a round as the threads hold.
template <bool F32, bool INTER, bool WIDE>
__global__ __launch_bounds__(kThreads) void rope_append_mxfp4(RopeParams p, BlockView blocks)
{
    const int64_t token = blockIdx.x;
    const int dim = p.cache.head_dim, places = dim / kRun, lanes = kThreads / places;
    const int j = threadIdx.x % places, lane = threadIdx.x / places;
    const int q_rounds = (p.q_heads + lanes - 1) / lanes, kv_rounds = (p.cache.kv_heads + lanes - 1) / lanes;
    const uint64_t pos = uint64_t(int64_t(p.pos[token]));
    const int64_t slot = p.slots[token], page = slot >> p.cache.page_shift;
    const bool live = slot >= 0 && page < p.cache.pages;
    const int64_t row = slot & ((int64_t(1) << p.cache.page_shift) - 1);
    const int64_t cell = (page * p.cache.page_stride + row * p.cache.slot_stride) / 2;
    const int64_t block = page * blocks.page_stride + row * blocks.slot_stride;
    const Run run = make_run<INTER>(j * kRun, p.rot_dim);
    __shared__ Table table;

    int round = blockIdx.y;
    const bool all = gridDim.y == 1;               // rounds, or one
    table.fill(p, pos, all || round < q_rounds, live && (all || (round >= q_rounds && round < q_rounds + kv_rounds)));
    if (lane >= lanes) return;                     // whole blocks of threads
    if (round < q_rounds) {
        Angles<float> a;
        a.fill(table.cs, table.sn, run);
        for (; round < q_rounds; round += gridDim.y) {
            const int h = round * lanes + lane;
            if (h >= p.q_heads) continue;
            float x[kRun], z[kRun], y[kRun];
            load_pairs<F32, INTER, WIDE>(p.q, token * p.q_token + h * p.q_head, run, true, x, z);
#pragma unroll
            for (int i = 0; i < kRun; ++i) y[i] = run.turns[i] ? __builtin_fmaf(x[i], a.cs[i], z[i] * a.sn[i]) : x[i];
            uint16_t* out = p.q_out + token * p.o_token + h * p.o_head + run.d;
            bf16x4 v;
#pragma unroll
            for (int i = 0; i < kRun; ++i) v[i] = (__bf16)y[i];
            if (WIDE) {
                *reinterpret_cast<bf16x4*>(out) = v;
            } else {
#pragma unroll
                for (int i = 0; i < kRun; ++i) reinterpret_cast<__bf16*>(out)[i] = v[i];
            }
        }
    }
    if (!live) return;
    round -= q_rounds;
    if (round < kv_rounds) {
        Angles<double> a;
        a.fill(table.key_cs, table.key_sn, run);
        for (; round < kv_rounds; round += gridDim.y) {
            const int h = round * lanes + lane;
            if (h >= p.cache.kv_heads) continue;
            float x[kRun], z[kRun];
            double y[kRun];
            load_pairs<F32, INTER, WIDE>(p.k, token * p.k_token + h * p.k_head, run, true, x, z);
#pragma unroll
            for (int i = 0; i < kRun; ++i)
                y[i] = run.turns[i] ? __builtin_fma(double(x[i]), a.cs[i], double(z[i]) * a.sn[i]) : double(x[i]);
            store_block(y, run.d, p.cache.k + cell + h * (p.cache.head_stride / 2), blocks.k + block + h * blocks.head_stride);
        }
    }
    round -= kv_rounds;
    for (; round < kv_rounds; round += gridDim.y) {
        const int h = round * lanes + lane;
        if (h >= p.cache.kv_heads) continue;
        float x[kRun], z[kRun];
        double y[kRun];
        load_pairs<F32, INTER, WIDE>(p.v, token * p.v_token + h * p.v_head, run, false, x, z);
#pragma unroll
        for (int i = 0; i < kRun; ++i) y[i] = double(x[i]);
        store_block(y, run.d, p.cache.v + cell + h * (p.cache.head_stride / 2), blocks.v + block + h * blocks.head_stride);
    }
}

template <bool F32, bool INTER>
void launch(const RopeParams& p, const BlockView& blocks, hipStream_t s)
{
    const int dim = p.cache.head_dim;
    const bool eights = p.wide && (INTER ? p.rot_dim % 8 == 0 : p.rot_dim % 64 == 0 && dim % 64 == 0);
    const int lanes = kThreads / (dim / (eights ? 8 : kRun)), kv = p.cache.kv_heads;
    const int rounds = eights ? (p.q_heads + 2 * kv + lanes - 1) / lanes : (p.q_heads + lanes - 1) / lanes + 2 * ((kv + lanes - 1) / lanes);
    // few tokens: a work-group a round; many: all rounds of a token share the angles
    const dim3 grid(unsigned(p.tokens), p.tokens * rounds <= 1024 ? rounds : 1);
    if (eights) hipLaunchKernelGGL((rope_append_mxfp4_wide<F32, INTER>), grid, dim3(kThreads), 0, s, p, blocks);
    // a run and its partners begin on a multiple of four dimensions
    else if (p.wide && p.rot_dim % 8 == 0) hipLaunchKernelGGL((rope_append_mxfp4<F32, INTER, true>), grid, dim3(kThreads), 0, s, p, blocks);
    else hipLaunchKernelGGL((rope_append_mxfp4<F32, INTER, false>), grid, dim3(kThreads), 0, s, p, blocks);
}

}  // namespace

hipError_t launch_rope_mxfp4(const RopeParams& p, const BlockView& blocks, hipStream_t s)
{
    if (p.f32) {
        if (p.interleaved) launch<true, true>(p, blocks, s);
        else launch<true, false>(p, blocks, s);
    } else {
        if (p.interleaved) launch<false, true>(p, blocks, s);
        else launch<false, false>(p, blocks, s);
    }
    return hipGetLastError();
}

}  // namespace qg
