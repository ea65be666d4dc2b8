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

// One thread per element; the simple form.
__global__ __launch_bounds__(256) void rope_append_kernel(RopeParams p)
{
    const int64_t token = blockIdx.x;
    const int heads = p.q_heads + 2 * p.cache.kv_heads;
    const int dim = p.cache.head_dim, half = p.rot_dim / 2;
    const uint64_t pos = uint64_t(int64_t(p.pos[token]));
    const int64_t slot = p.slots[token];
    const int64_t page = slot >> p.cache.page_shift;
    const bool live = slot >= 0 && page < p.cache.pages;
    const int64_t cell = page * p.cache.page_stride + (slot & ((int64_t(1) << p.cache.page_shift) - 1)) * p.cache.slot_stride;
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
            const int64_t frac = int64_t(pos * p.turns[pair]);
            float sn, cs;
            sincospif(float(frac) * 0x1p-63f, &sn, &cs);
            sn *= p.amplitude;
            cs *= p.amplitude;
            y = second ? y * cs + z * sn : y * cs - z * sn;
        }
        if (is_q)
            p.q_out[token * p.o_token + h * p.o_head + d] = f32_to_bf16(y);
        else if (live)
            store_cache(is_k ? p.cache.k : p.cache.v, p.cache.e4m3,
                        p.cache.e4m3 ? (is_k ? p.cache.k_scale : p.cache.v_scale)[h] : 1.0f,
                        cell + h * p.cache.head_stride + d, y);
    }
}

}  // namespace

hipError_t launch_rope(const RopeParams& p, hipStream_t s)
{
    hipLaunchKernelGGL(rope_append_kernel, dim3(unsigned(p.tokens)), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace qg
