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

template <class T>
struct Angles {
    T cs[kRun], sn[kRun];      // sin with the sign that the partner takes

    template <bool INTER>
    __device__ __forceinline__ void fill(const RopeParams& p, uint64_t pos, const Run& r)
    {
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            cs[i] = T(1), sn[i] = T(0);
            if (INTER && i % 2) {      // rot_dim is even: both of a pair turn
                cs[i] = cs[i - 1], sn[i] = -sn[i - 1];
            } else if (r.turns[i]) {
                turn(pos, p.turns[r.pair[i]], p.amplitude, &cs[i], &sn[i]);
                if (!r.second[i]) sn[i] = -sn[i];
            }
        }
    }
};

// A magnitude as an integer that orders as it does: the upper word of the fp64
// number, and whether anything is set below it.
__device__ __forceinline__ uint32_t magnitude(double x)
{
    const uint64_t b = uint64_t(__double_as_longlong(x));
    return uint32_t(b >> 32) << 1 | (uint32_t(b) != 0 ? 1u : 0u);
}

__device__ __forceinline__ uint32_t code_of(double x, int e)
{
    const double y = __builtin_ldexp(x, -e);
    const uint32_t m = magnitude(y);
    const uint32_t size = (m > 0x3fd00000u * 2u ? 1 : 0) + (m >= 0x3fe80000u * 2u ? 1 : 0) + (m > 0x3ff40000u * 2u ? 1 : 0) +
                          (m >= 0x3ffc0000u * 2u ? 1 : 0) + (m > 0x40040000u * 2u ? 1 : 0) + (m >= 0x400c0000u * 2u ? 1 : 0) +
                          (m > 0x40140000u * 2u ? 1 : 0);
    return size | uint32_t(uint64_t(__double_as_longlong(x)) >> 60 & 8);
}

// A thread's four elements into the cache, with the seven threads around it
// that hold the rest of their block.
__device__ __forceinline__ void store_block(const double* y, int d, uint8_t* codes, uint8_t* exponents)
{
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) most = max(most, magnitude(y[i]));
#pragma unroll
    for (int x = 1; x < kBlock / kRun; x <<= 1) most = max(most, uint32_t(__shfl_xor(int(most), x, 64)));
    const bool nan = most > 0x7ff00000u * 2u;
    // 1.75 2^k is 7 times the scale 2^(k - 2)
    const int k = int(most >> 21) - 1023;
    int e = k - 2 + ((most & 0x1fffffu) > 0x180000u ? 1 : 0);
    e = min(max(e, -125), 125);
    uint32_t word = 0;
    if (!nan) {
#pragma unroll
        for (int i = 0; i < kRun; ++i) word |= code_of(y[i], e) << (4 * i);
    }
    *reinterpret_cast<uint16_t*>(codes + d / 2) = uint16_t(word);
    if (d % kBlock == 0) exponents[d / kBlock] = uint8_t(nan ? 255 : e + 127);
}

// A work-group takes rounds of heads of one token: first of queries, then of
// keys, then of values, as many heads a round as the threads hold.
template <bool F32, bool INTER, bool WIDE>
__global__ __launch_bounds__(kThreads) void rope_append_mxfp4(RopeParams p, BlockView blocks)
{
    const int64_t token = blockIdx.x;
    const int dim = p.cache.head_dim, places = dim / kRun, lanes = kThreads / places;
    const int j = threadIdx.x % places, lane = threadIdx.x / places;
    if (lane >= lanes) return;                     // whole blocks of threads
    const int q_rounds = (p.q_heads + lanes - 1) / lanes, kv_rounds = (p.cache.kv_heads + lanes - 1) / lanes;
    const uint64_t pos = uint64_t(int64_t(p.pos[token]));
    const int64_t slot = p.slots[token], page = slot >> p.cache.page_shift;
    const bool live = slot >= 0 && page < p.cache.pages;
    const int64_t row = slot & ((int64_t(1) << p.cache.page_shift) - 1);
    const int64_t cell = (page * p.cache.page_stride + row * p.cache.slot_stride) / 2;
    const int64_t block = page * blocks.page_stride + row * blocks.slot_stride;
    const Run run = make_run<INTER>(j * kRun, p.rot_dim);

    int round = blockIdx.y;
    if (round < q_rounds) {
        Angles<float> a;
        a.template fill<INTER>(p, pos, run);
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
        a.template fill<INTER>(p, pos, run);
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
void launch(const RopeParams& p, const BlockView& blocks, dim3 grid, hipStream_t s)
{
    // a run and its partners begin on a multiple of four dimensions
    if (p.wide && p.rot_dim % 8 == 0) hipLaunchKernelGGL((rope_append_mxfp4<F32, INTER, true>), grid, dim3(kThreads), 0, s, p, blocks);
    else hipLaunchKernelGGL((rope_append_mxfp4<F32, INTER, false>), grid, dim3(kThreads), 0, s, p, blocks);
}

}  // namespace

hipError_t launch_rope_mxfp4(const RopeParams& p, const BlockView& blocks, hipStream_t s)
{
    const int lanes = kThreads / (p.cache.head_dim / kRun);
    const int rounds = (p.q_heads + lanes - 1) / lanes + 2 * ((p.cache.kv_heads + lanes - 1) / lanes);
    // few tokens: a work-group a round; many: all rounds of a token share the angles
    const dim3 grid(unsigned(p.tokens), p.tokens * rounds <= 1024 ? rounds : 1);
    if (p.f32) {
        if (p.interleaved) launch<true, true>(p, blocks, grid, s);
        else launch<true, false>(p, blocks, grid, s);
    } else {
        if (p.interleaved) launch<false, true>(p, blocks, grid, s);
        else launch<false, false>(p, blocks, grid, s);
    }
    return hipGetLastError();
}

}  // namespace qg
