// Rotary positions on queries and keys, and the append of rotated keys and
// of values to the paged cache, in one pass over the QKV projection's output.
//
// Pair i of a head turns by the angle pos * f_i.  A position far into a long
// context times a frequency near 1 loses the angle in fp32 (at 2^20 the
// spacing of fp32 is 1/16 of a radian), so f_i comes as a 64-bit binary
// fraction of a turn: pos * f_i modulo 2^64 is the angle modulo one turn,
// exact but for f_i's own rounding (2^-65 turns per position), in one integer
// product.  Only the remainder, within half a turn, becomes fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decode_ops.h"

namespace qg {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }

__device__ __forceinline__ uint16_t f32_to_bf16(float f)
{
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0x7fc0;
    return uint16_t((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

__device__ __forceinline__ float load(const void* p, bool f32, int64_t i)
{
    return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

__device__ __forceinline__ void store_cache(uint8_t* base, bool e4m3, float scale, int64_t i, float x)
{
    if (!e4m3) {
        reinterpret_cast<uint16_t*>(base)[i] = f32_to_bf16(x);
        return;
    }
    // fminf and fmaxf drop a NaN, which has to reach the cache as one
    const float y = x / scale;
    const float c = y != y ? y : fminf(fmaxf(y, -448.0f), 448.0f);
    base[i] = uint8_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, c, 0, false) & 0xff);
}

struct Place {
    bool live;        // the token has a place in the cache
    int64_t cell;     // its element offset there, of kv head 0
};

__device__ __forceinline__ Place place_of(const CacheView& c, int64_t slot)
{
    const int64_t page = slot >> c.page_shift;
    const bool live = slot >= 0 && page < c.pages;
    return {live, page * c.page_stride + (slot & ((int64_t(1) << c.page_shift) - 1)) * c.slot_stride};
}

__device__ __forceinline__ void turn(uint64_t pos, uint64_t per, float amplitude, float* cs, float* sn)
{
    sincospif(float(int64_t(pos * per)) * 0x1p-63f, sn, cs);   // 2^63 is half a turn
    *sn *= amplitude;
    *cs *= amplitude;
}

// Any rot_dim, alignment and stride: one thread per element.
__global__ __launch_bounds__(256) void rope_append_narrow(RopeParams p)
{
    const int64_t token = blockIdx.x;
    const int heads = p.q_heads + 2 * p.cache.kv_heads;
    const int dim = p.cache.head_dim, half = p.rot_dim / 2;
    const uint64_t pos = uint64_t(int64_t(p.pos[token]));
    const Place place = place_of(p.cache, p.slots[token]);
    for (int i = threadIdx.x; i < heads * dim; i += blockDim.x) {
        const int head = i / dim, d = i % dim;
        const bool is_q = head < p.q_heads, is_k = !is_q && head < p.q_heads + p.cache.kv_heads;
        const int h = is_q ? head : is_k ? head - p.q_heads : head - p.q_heads - p.cache.kv_heads;
        const void* src = is_q ? p.q : is_k ? p.k : p.v;
        const int64_t at = is_q ? token * p.q_token + h * p.q_head : is_k ? token * p.k_token + h * p.k_head
                                                                          : token * p.v_token + h * p.v_head;
        float y = load(src, p.f32, at + d);
        if ((is_q || is_k) && d < p.rot_dim) {
            const int pair = p.interleaved ? d / 2 : d < half ? d : d - half;
            const bool second = p.interleaved ? (d & 1) : d >= half;
            const int other = p.interleaved ? d ^ 1 : second ? d - half : d + half;
            const float z = load(src, p.f32, at + other);
            float sn, cs;
            turn(pos, p.turns[pair], p.amplitude, &cs, &sn);
            y = second ? __builtin_fmaf(y, cs, z * sn) : __builtin_fmaf(y, cs, -(z * sn));
        }
        if (is_q)
            p.q_out[token * p.o_token + h * p.o_head + d] = f32_to_bf16(y);
        else if (place.live)
            store_cache(is_k ? p.cache.k : p.cache.v, p.cache.e4m3,
                        p.cache.e4m3 ? (is_k ? p.cache.k_scale : p.cache.v_scale)[h] : 1.0f,
                        place.cell + h * p.cache.head_stride + d, y);
    }
}

// Four elements at a time.
template <bool F32>
__device__ __forceinline__ void load4(const void* p, int64_t i, float* x)
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

__device__ __forceinline__ void store4_bf16(uint16_t* p, const float* x)
{
    bf16x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = (__bf16)x[j];
    *reinterpret_cast<bf16x4*>(p) = v;
}

__device__ __forceinline__ float clamped(float x, float scale)
{
    const float y = x / scale;
    return y != y ? y : fminf(fmaxf(y, -448.0f), 448.0f);
}

template <bool E4M3>
__device__ __forceinline__ void store4(uint8_t* base, int64_t i, const float* x, float scale)
{
    if (!E4M3) {
        store4_bf16(reinterpret_cast<uint16_t*>(base) + i, x);
    } else {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(clamped(x[0], scale), clamped(x[1], scale), 0, false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(clamped(x[2], scale), clamped(x[3], scale), v, true);
        *reinterpret_cast<int*>(base + i) = v;
    }
}

// Rows on 16 bytes and rot_dim a multiple of 8.  A thread holds one eighth-
// of-a-dimension place, two runs of four elements (the halves' matching ones,
// or eight neighbours where pairs are interleaved or nothing turns), and
// takes that place of every LANES-th head, so that its four angles are worked
// out once for them.  Neighbouring threads hold neighbouring places.
template <bool F32, bool INTER, bool E4M3>
__global__ __launch_bounds__(256) void rope_append_wide(RopeParams p)
{
    const int64_t token = blockIdx.x;
    const int dim = p.cache.head_dim, places = dim / 8;
    const int lanes = 256 / places;                  // heads at a time
    const int j = threadIdx.x % places, first = threadIdx.x / places + blockIdx.y * lanes;
    if (first >= int(blockIdx.y + 1) * lanes) return;
    const int heads = p.q_heads + 2 * p.cache.kv_heads;
    const bool turns = 8 * j < p.rot_dim;
    const int a = turns && !INTER ? 4 * j : 8 * j, b = turns && !INTER ? a + p.rot_dim / 2 : a + 4;
    const uint64_t pos = uint64_t(int64_t(p.pos[token]));
    const Place place = place_of(p.cache, p.slots[token]);
    float cs[4], sn[4];
    if (turns) {
#pragma unroll
        for (int i = 0; i < 4; ++i) turn(pos, p.turns[4 * j + i], p.amplitude, &cs[i], &sn[i]);
    }
    for (int head = first; head < heads; head += lanes * gridDim.y) {
        const bool is_q = head < p.q_heads, is_k = !is_q && head < p.q_heads + p.cache.kv_heads;
        if (!is_q && !place.live) break;
        const int h = is_q ? head : is_k ? head - p.q_heads : head - p.q_heads - p.cache.kv_heads;
        const void* src = is_q ? p.q : is_k ? p.k : p.v;
        const int64_t at = is_q ? token * p.q_token + h * p.q_head : is_k ? token * p.k_token + h * p.k_head
                                                                          : token * p.v_token + h * p.v_head;
        float x[8], y[8];
        load4<F32>(src, at + a, x);
        load4<F32>(src, at + b, x + 4);
        if (turns && (is_q || is_k)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = INTER ? 2 * i : i, o = INTER ? 2 * i + 1 : i + 4;
                y[e] = __builtin_fmaf(x[e], cs[i], -(x[o] * sn[i]));
                y[o] = __builtin_fmaf(x[o], cs[i], x[e] * sn[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[i];
        }
        if (is_q) {
            uint16_t* out = p.q_out + token * p.o_token + h * p.o_head;
            store4_bf16(out + a, y);
            store4_bf16(out + b, y + 4);
        } else {
            uint8_t* base = is_k ? p.cache.k : p.cache.v;
            const float scale = E4M3 ? (is_k ? p.cache.k_scale : p.cache.v_scale)[h] : 1.0f;
            const int64_t cell = place.cell + h * p.cache.head_stride;
            store4<E4M3>(base, cell + a, y, scale);
            store4<E4M3>(base, cell + b, y + 4, scale);
        }
    }
}

template <bool F32, bool INTER>
void launch_wide(const RopeParams& p, dim3 grid, hipStream_t s)
{
    if (p.cache.e4m3) hipLaunchKernelGGL((rope_append_wide<F32, INTER, true>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((rope_append_wide<F32, INTER, false>), grid, dim3(256), 0, s, p);
}

}  // namespace

static hipError_t launch_tokens(const RopeParams& p, hipStream_t s)
{
    if (!p.wide || p.rot_dim % 8 != 0) {
        hipLaunchKernelGGL(rope_append_narrow, dim3(unsigned(p.tokens)), dim3(256), 0, s, p);
        return hipGetLastError();
    }
    // Few tokens: a work-group for every few heads, so that the call is one
    // short chain of loads; many: all heads of a token share the angles.
    const int lanes = 256 / (p.cache.head_dim / 8);
    const int rounds = (p.q_heads + 2 * p.cache.kv_heads + lanes - 1) / lanes;
    const dim3 grid(unsigned(p.tokens), p.tokens * rounds <= 1024 ? rounds : 1);
    if (p.f32) {
        if (p.interleaved) launch_wide<true, true>(p, grid, s);
        else launch_wide<true, false>(p, grid, s);
    } else {
        if (p.interleaved) launch_wide<false, true>(p, grid, s);
        else launch_wide<false, false>(p, grid, s);
    }
    return hipGetLastError();
}

// A grid has fewer than 2^32 threads (more are dropped without an error), and
// a token takes 256: more tokens go in several launches.
hipError_t launch_rope(const RopeParams& p, hipStream_t s)
{
    constexpr int64_t kMost = int64_t(1) << 23;
    if (p.tokens <= kMost) return launch_tokens(p, s);
    const int64_t size = p.f32 ? 4 : 2;
    const auto on = [&](const void* x, int64_t elements) { return static_cast<const uint8_t*>(x) + elements * size; };
    for (int64_t t = 0; t < p.tokens; t += kMost) {
        RopeParams part = p;
        part.q = on(p.q, t * p.q_token);
        part.k = on(p.k, t * p.k_token);
        part.v = on(p.v, t * p.v_token);
        part.q_out += t * p.o_token;
        part.pos += t;
        part.slots += t;
        part.tokens = p.tokens - t < kMost ? p.tokens - t : kMost;
        const hipError_t e = launch_tokens(part, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qg
