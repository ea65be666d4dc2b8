// Cached tokens read back, as the numbers they stand for, in bf16 or fp32.
//
// A thread holds 16 bytes of an output row and what they come from.  Of many
// tokens the writes bound it: 90001 tokens of 8 heads of 128 from a 4-bit cache
// to bf16, 98 MB read and 369 MB written, 98 us (74 where they were read just
// before; a copy moves as much in 92, a fill writes the output in 54), from a bf16
// cache 132 us and from an 8-bit one 100 (737 and 553 MB moved); of a few
// the call on the host (513 tokens 6 us, 3.5 of it on the GPU).  Rows are
// written past the caches: what reads them next is another kernel's product.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "decode_ops.h"

namespace qg {

namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
// Elements of a thread: 16 bytes of the output, so that a wave writes whole
// lines at a time.
template <bool F32>
constexpr int kRun = F32 ? 4 : 8;
// Work-groups of a launch: 90001 tokens of 8 heads of 128 take 98 us, 103 with
// at most 4096 that go on to further tokens.
constexpr int64_t kMostGroups = 1 << 23;
// Places (tokens x heads x dim / 8) from which a thread takes two tokens at a
// time: 98 us in place of 101 there, while few tokens (513: 66k places) want
// as many threads as they can have.
constexpr int64_t kFewPlaces = 1 << 19;

enum Kind { kBf16, kE4m3, kMxfp4 };

// RUN elements as they lie in memory, and as numbers.
template <int KIND, int RUN>
using Raw = std::conditional_t<
    KIND == kBf16, std::conditional_t<RUN == 8, u32x4, u32x2>,
    std::conditional_t<KIND == kE4m3, std::conditional_t<RUN == 8, u32x2, uint32_t>, std::conditional_t<RUN == 8, uint32_t, uint16_t>>>;

template <int KIND, int RUN>
__device__ __forceinline__ Raw<KIND, RUN> load_run(const uint8_t* base, int64_t at)
{
    return *reinterpret_cast<const Raw<KIND, RUN>*>(base + (KIND == kBf16 ? 2 * at : KIND == kE4m3 ? at : at / 2));
}

template <int KIND, int RUN>
__device__ __forceinline__ void widen(const Raw<KIND, RUN>& v, float scale, float* x)
{
    uint32_t w[4] = {};
    __builtin_memcpy(w, &v, sizeof(v));
    if constexpr (KIND == kBf16) {
#pragma unroll
        for (int i = 0; i < RUN / 2; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else if constexpr (KIND == kE4m3) {
#pragma unroll
        for (int i = 0; i < RUN / 4; ++i) {
            const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(int(w[i]), false), b = __builtin_amdgcn_cvt_pk_f32_fp8(int(w[i]), true);
            x[4 * i] = a[0] * scale, x[4 * i + 1] = a[1] * scale;
            x[4 * i + 2] = b[0] * scale, x[4 * i + 3] = b[1] * scale;
        }
    } else {
        f32x2 a[4];
        a[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], scale, 0);
        a[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], scale, 1);
        a[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], scale, 2);
        a[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], scale, 3);
#pragma unroll
        for (int i = 0; i < RUN / 2; ++i) x[2 * i] = a[i][0], x[2 * i + 1] = a[i][1];
    }
}

// 16 bytes of the output, which this call does not read again: past the caches
// (20000 tokens of 8 heads of 128, bf16: 18.5 us, 25.8 through them).
template <bool F32, bool WIDE>
__device__ __forceinline__ void store_run(void* base, int64_t at, const float* x)
{
    constexpr int RUN = kRun<F32>;
    using T = std::conditional_t<F32, float, __bf16>;
    typedef T run __attribute__((ext_vector_type(RUN)));
    T* o = static_cast<T*>(base) + at;
    run v;
#pragma unroll
    for (int i = 0; i < RUN; ++i) v[i] = T(x[i]);
    if (WIDE) {
        __builtin_nontemporal_store(v, reinterpret_cast<run*>(o));
    } else {
#pragma unroll
        for (int i = 0; i < RUN; ++i) o[i] = v[i];
    }
}

// A thread holds one place of a token's row (kRun elements of a head) and
// takes it of every `apart`-th token, TOKENS at a time, so that their loads
// are in flight together.
template <int KIND, bool F32, bool WIDE, int TOKENS>
__global__ __launch_bounds__(kThreads) void read_kernel(ReadParams p)
{
    const CacheView& c = p.cache;
    constexpr int RUN = kRun<F32>;
    const int places = c.head_dim / RUN, items = places * c.kv_heads;
    const int apart = items < kThreads ? kThreads / items : 1;          // tokens side by side
    const int item = items < kThreads ? threadIdx.x % items : blockIdx.y * kThreads + threadIdx.x;
    const int beside = items < kThreads ? threadIdx.x / items : 0;
    if (item >= items || beside >= apart) return;
    const int h = item / places, d = (item - h * places) * RUN;
    const int64_t head = h * c.head_stride + d, head_block = KIND == kMxfp4 ? h * p.blocks.head_stride + d / kBlock : 0;
    const int64_t k_head = h * p.k_head + d, v_head = h * p.v_head + d;
    float ks0 = 1.0f, vs0 = 1.0f;
    if (KIND == kE4m3) ks0 = c.k_scale[h], vs0 = c.v_scale[h];
    const int64_t mask = (int64_t(1) << c.page_shift) - 1;
    for (int64_t t0 = int64_t(blockIdx.x) * apart * TOKENS + beside; t0 < p.tokens; t0 += int64_t(gridDim.x) * apart * TOKENS) {
        int64_t at[TOKENS], block[TOKENS];
        bool live[TOKENS];
#pragma unroll
        for (int u = 0; u < TOKENS; ++u) {
            const int64_t token = t0 + u * apart;
            const int64_t slot = token < p.tokens ? p.slots[token] : -1, page = slot >> c.page_shift;
            live[u] = slot >= 0 && page < c.pages;
            // (others read the cache's first row)
            at[u] = head + (live[u] ? page * c.page_stride + (slot & mask) * c.slot_stride : 0);
            block[u] = head_block + (live[u] ? page * p.blocks.page_stride + (slot & mask) * p.blocks.slot_stride : 0);
        }
        const auto one = [&](const uint8_t* base, const uint8_t* exponents, float scale, void* out, int64_t head_at, int64_t token_stride) {
            Raw<KIND, RUN> raw[TOKENS];
            float s[TOKENS];
#pragma unroll
            for (int u = 0; u < TOKENS; ++u) {
                raw[u] = load_run<KIND, RUN>(base, at[u]);
                s[u] = KIND == kMxfp4 ? block_scale(exponents[block[u]]) : scale;
            }
#pragma unroll
            for (int u = 0; u < TOKENS; ++u) {
                float x[RUN];
                widen<KIND, RUN>(raw[u], s[u], x);
                if (live[u]) store_run<F32, WIDE>(out, (t0 + u * apart) * token_stride + head_at, x);
            }
        };
        if (p.k) one(c.k, p.blocks.k, ks0, p.k, k_head, p.k_token);
        if (p.v) one(c.v, p.blocks.v, vs0, p.v, v_head, p.v_token);
    }
}

template <int KIND, int TOKENS>
hipError_t launch(const ReadParams& p, hipStream_t s)
{
    const int items = p.cache.head_dim / (p.f32 ? kRun<true> : kRun<false>) * p.cache.kv_heads;
    const int apart = items < kThreads ? kThreads / items : 1;
    const int64_t groups = (p.tokens + apart * TOKENS - 1) / (apart * TOKENS);
    // (a grid has fewer than 2^32 threads: more are dropped without an error)
    const int64_t parts = items < kThreads ? 1 : (items + kThreads - 1) / kThreads, most = kMostGroups / parts;
    const dim3 grid(unsigned(groups < most ? groups : most), unsigned(parts));
    if (p.f32) {
        if (p.wide) hipLaunchKernelGGL((read_kernel<KIND, true, true, TOKENS>), grid, dim3(kThreads), 0, s, p);
        else hipLaunchKernelGGL((read_kernel<KIND, true, false, TOKENS>), grid, dim3(kThreads), 0, s, p);
    } else {
        if (p.wide) hipLaunchKernelGGL((read_kernel<KIND, false, true, TOKENS>), grid, dim3(kThreads), 0, s, p);
        else hipLaunchKernelGGL((read_kernel<KIND, false, false, TOKENS>), grid, dim3(kThreads), 0, s, p);
    }
    return hipGetLastError();
}

template <int KIND>
hipError_t launch(const ReadParams& p, hipStream_t s)
{
    // few tokens: as many threads as there are places
    const int64_t places = int64_t(p.cache.head_dim / 8) * p.cache.kv_heads * p.tokens;
    return places < kFewPlaces ? launch<KIND, 1>(p, s) : launch<KIND, 2>(p, s);
}

}  // namespace

hipError_t launch_read(const ReadParams& p, hipStream_t s)
{
    return p.cache.mxfp4 ? launch<kMxfp4>(p, s) : p.cache.e4m3 ? launch<kE4m3>(p, s) : launch<kBf16>(p, s);
}

}  // namespace qg
