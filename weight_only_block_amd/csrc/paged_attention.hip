// Attention of a chunk of new tokens over the paged cache.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decode_ops.h"

namespace qg {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }

__device__ __forceinline__ uint16_t f32_to_bf16(float f)
{
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0x7fc0;
    return uint16_t((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

__device__ __forceinline__ float cache_value(const uint8_t* base, bool e4m3, int64_t i)
{
    if (!e4m3) return bf16_to_f32(reinterpret_cast<const uint16_t*>(base)[i]);
    return __builtin_amdgcn_cvt_f32_fp8(int(base[i]), 0);
}

// The simple form: a wave per (token, query head).  Each lane takes one key
// of 64 at a time for the scores, then each lane takes dimensions of the
// output.
__global__ __launch_bounds__(64) void attention_simple(AttnParams p)
{
    __shared__ float qs[kMaxHeadDim];
    __shared__ float ps[64];
    __shared__ int64_t vrow[64];
    const int lane = threadIdx.x, dim = p.cache.head_dim;
    const int b = blockIdx.z;
    const int h = blockIdx.y, kvh = h / p.group;
    const int64_t q0 = max(int64_t(0), min(int64_t(p.q_start[b]), p.tokens));
    const int64_t q1 = max(q0, min(min(int64_t(p.q_start[b + 1]), p.tokens), q0 + p.max_q));
    const int64_t token = q0 + blockIdx.x;
    if (token >= q1) return;
    const int64_t cap = min(p.max_kv, p.table_cols << p.cache.page_shift);
    const int64_t kv = max(int64_t(0), min(int64_t(p.kv_len[b]), cap));
    const int64_t at = kv - (q1 - token);            // this token's own place
    const int64_t lo = p.window > 0 ? max(int64_t(0), at - p.window + 1) : 0;
    const int64_t hi = min(kv, at + 1);
    const float ks = p.cache.e4m3 ? p.cache.k_scale[kvh] : 1.0f;
    const float vs = p.cache.e4m3 ? p.cache.v_scale[kvh] : 1.0f;
    for (int d = lane; d < dim; d += 64) qs[d] = bf16_to_f32(p.q[token * p.q_token + h * p.q_head + d]);
    __syncthreads();
    float m = -INFINITY, l = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const float fac = p.scale * ks * kLog2e;
    const int64_t mask = (int64_t(1) << p.cache.page_shift) - 1;
    for (int64_t base = lo; base < hi; base += 64) {
        const int64_t key = base + lane;
        float s = -INFINITY;
        int64_t row = -1;
        if (key < hi) {
            const int64_t id = p.table[b * p.table_stride + (key >> p.cache.page_shift)];
            s = __builtin_nanf("");
            if (id >= 0 && id < p.cache.pages) {
                row = id * p.cache.page_stride + kvh * p.cache.head_stride + (key & mask) * p.cache.slot_stride;
                float dot = 0.0f;
                for (int d = 0; d < dim; ++d) dot += qs[d] * cache_value(p.cache.k, p.cache.e4m3, row + d);
                s = dot * fac;
            }
        }
        float top = s;
        for (int off = 32; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
        const float mn = fmaxf(m, top);
        const float ref = mn == -INFINITY ? 0.0f : mn;
        const float w = exp2f(s - ref), keep = exp2f(m - ref);
        float sum = w;
        for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off, 64);
        l = l * keep + sum;
        m = mn;
        ps[lane] = w;
        vrow[lane] = row;
        __syncthreads();
        for (int i = 0; i < 4; ++i) acc[i] *= keep;
        const int n = int(min(int64_t(64), hi - base));
        for (int j = 0; j < n; ++j)
            if (vrow[j] >= 0)
                for (int i = 0; i < 4; ++i)
                    if (lane + 64 * i < dim) acc[i] += ps[j] * cache_value(p.cache.v, p.cache.e4m3, vrow[j] + lane + 64 * i);
        __syncthreads();
    }
    const float inv = hi > lo ? vs / l : 0.0f;
    for (int i = 0; i < 4; ++i)
        if (lane + 64 * i < dim)
            p.out[token * p.o_token + h * p.o_head + lane + 64 * i] = f32_to_bf16(hi > lo ? acc[i] * inv : 0.0f);
    if (p.lse && lane == 0) p.lse[token * p.lse_token + h] = hi > lo ? m * kLn2 + logf(l) : -INFINITY;
}

}  // namespace

size_t attention_workspace_bytes(int64_t tokens, int q_heads, int kv_heads, int head_dim, int seqs, int64_t max_q,
                                 int64_t max_kv)
{
    (void)tokens, (void)q_heads, (void)kv_heads, (void)head_dim, (void)seqs, (void)max_q, (void)max_kv;
    return 256;
}

hipError_t launch_attention(const AttnParams& p, hipStream_t s)
{
    hipLaunchKernelGGL(attention_simple, dim3(unsigned(p.max_q), unsigned(p.q_heads), unsigned(p.seqs)), dim3(64), 0, s, p);
    return hipGetLastError();
}

}  // namespace qg
