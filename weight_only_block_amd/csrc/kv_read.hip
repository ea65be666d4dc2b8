// Cached tokens read back, as the numbers they stand for, in bf16 or fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decode_ops.h"

namespace qg {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;
constexpr int kRun = 8;            // dimensions of a thread

enum Kind { kBf16, kE4m3, kMxfp4 };

// Eight elements from element `at` on.
template <int KIND>
__device__ __forceinline__ void load_run(const uint8_t* base, int64_t at, float scale, float* x)
{
    if (KIND == kBf16) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(base + 2 * at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(v[i] << 16);
            x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
        }
    } else if (KIND == kE4m3) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(base + at);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(int(v[i]), false), b = __builtin_amdgcn_cvt_pk_f32_fp8(int(v[i]), true);
            x[4 * i] = a[0] * scale, x[4 * i + 1] = a[1] * scale;
            x[4 * i + 2] = b[0] * scale, x[4 * i + 3] = b[1] * scale;
        }
    } else {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(base + at / 2);
        f32x2 a[4];
        a[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, scale, 0);
        a[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, scale, 1);
        a[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, scale, 2);
        a[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, scale, 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = a[i][0], x[2 * i + 1] = a[i][1];
    }
}

template <bool F32, bool WIDE>
__device__ __forceinline__ void store_run(void* base, int64_t at, const float* x)
{
    if (F32) {
        float* o = static_cast<float*>(base) + at;
        if (WIDE) {
            *reinterpret_cast<f32x4*>(o) = f32x4{x[0], x[1], x[2], x[3]};
            *reinterpret_cast<f32x4*>(o + 4) = f32x4{x[4], x[5], x[6], x[7]};
        } else {
#pragma unroll
            for (int i = 0; i < kRun; ++i) o[i] = x[i];
        }
    } else {
        __bf16* o = static_cast<__bf16*>(base) + at;
        bf16x8 v;
#pragma unroll
        for (int i = 0; i < kRun; ++i) v[i] = (__bf16)x[i];
        if (WIDE) {
            *reinterpret_cast<bf16x8*>(o) = v;
        } else {
#pragma unroll
            for (int i = 0; i < kRun; ++i) o[i] = v[i];
        }
    }
}

// One thread per eight elements of keys and of values, tokens along x.
template <int KIND, bool F32, bool WIDE>
__global__ __launch_bounds__(kThreads) void read_kernel(ReadParams p)
{
    const CacheView& c = p.cache;
    const int places = c.head_dim / kRun;
    const int64_t items = int64_t(places) * c.kv_heads, all = items * p.tokens;
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < all; i += int64_t(gridDim.x) * kThreads) {
        const int64_t token = i / items;
        const int rest = int(i - token * items), h = rest / places, d = (rest - h * places) * kRun;
        const int64_t slot = p.slots[token], page = slot >> c.page_shift;
        if (slot < 0 || page >= c.pages) continue;
        const int64_t row = slot & ((int64_t(1) << c.page_shift) - 1);
        const int64_t at = page * c.page_stride + h * c.head_stride + row * c.slot_stride + d;
        float ks = 1.0f, vs = 1.0f;
        if (KIND == kE4m3) {
            ks = c.k_scale[h], vs = c.v_scale[h];
        } else if (KIND == kMxfp4) {
            const int64_t b = page * p.blocks.page_stride + h * p.blocks.head_stride + row * p.blocks.slot_stride + d / kBlock;
            const int kb = p.k ? p.blocks.k[b] : 0, vb = p.v ? p.blocks.v[b] : 0;
            ks = block_scale(kb), vs = block_scale(vb);
        }
        float x[kRun];
        if (p.k) {
            load_run<KIND>(c.k, at, ks, x);
            store_run<F32, WIDE>(p.k, token * p.k_token + h * p.k_head + d, x);
        }
        if (p.v) {
            load_run<KIND>(c.v, at, vs, x);
            store_run<F32, WIDE>(p.v, token * p.v_token + h * p.v_head + d, x);
        }
    }
}

template <int KIND>
hipError_t launch(const ReadParams& p, hipStream_t s)
{
    const int64_t all = int64_t(p.cache.head_dim / kRun) * p.cache.kv_heads * p.tokens;
    const int64_t groups = (all + kThreads - 1) / kThreads;
    const dim3 grid(unsigned(groups < 8192 ? groups : 8192));
    if (p.f32) {
        if (p.wide) hipLaunchKernelGGL((read_kernel<KIND, true, true>), grid, dim3(kThreads), 0, s, p);
        else hipLaunchKernelGGL((read_kernel<KIND, true, false>), grid, dim3(kThreads), 0, s, p);
    } else {
        if (p.wide) hipLaunchKernelGGL((read_kernel<KIND, false, true>), grid, dim3(kThreads), 0, s, p);
        else hipLaunchKernelGGL((read_kernel<KIND, false, false>), grid, dim3(kThreads), 0, s, p);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_read(const ReadParams& p, hipStream_t s)
{
    return p.cache.mxfp4 ? launch<kMxfp4>(p, s) : p.cache.e4m3 ? launch<kE4m3>(p, s) : launch<kBf16>(p, s);
}

}  // namespace qg
