// What the attention kernels share (paged_attention.hip, paged_attention_few.hip):
// types, arguments, and small device functions.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decode_ops.h"

namespace qg {

// What the kernels of few rows on a 4-bit cache are chosen and sized by:
// `rows`, the most of a sequence and kv head; `even`, 16 keys of a tile lie in
// one page, and offsets within it in 32 bits.
struct FewSize {
    int dim, kv_heads, seqs, rows;
    bool even;
    int64_t max_kv;
};
size_t attention_few_need(const FewSize& z);    // of this shape
size_t attention_few_bytes(const FewSize& z);   // of this shape and every smaller one
hipError_t launch_attention_few(const FewSize& z, const void* block_args, hipStream_t s);

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.0f;             // log2 by which a score may pass the reference
constexpr int kComputeUnits = 256;
// Counts of arrived parts come first in the workspace, in every shape as many
// bytes: calls of other shapes leave them alone.
constexpr size_t kCounterBytes = 4096;
constexpr int32_t kMaxWindow = 1 << 30;    // no shorter than the longest sequence

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;

template <int N>
__device__ __forceinline__ void wait_loads()   // all but the last N
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    bf16x2 v;
    v[0] = (__bf16)a;
    v[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, v);
}

// The largest, and the sum, of a lane's value and that of the wave's other half.
__device__ __forceinline__ float max_halves(float x)
{
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float sum_halves(float x)
{
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// Partial sums cross work-groups on different XCDs: device-scope accesses.
__device__ __forceinline__ void put2(float* p, float a, float b)
{
    const uint64_t v = uint64_t(__float_as_uint(a)) | uint64_t(__float_as_uint(b)) << 32;
    __hip_atomic_store(reinterpret_cast<uint64_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void get2(const float* p, float* a, float* b)
{
    const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *a = __uint_as_float(uint32_t(v));
    *b = __uint_as_float(uint32_t(v >> 32));
}

// A value the compiler knows nothing of.  Lane numbers pass through it where a
// part of the kernel begins: what depends on them is then worked out there,
// not all together ahead of the loop over units, where hundreds of
// instructions, each fetched from a cold cache, stood before the first load.
__device__ __forceinline__ int opaque(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// a / b for a below 2^52, b > 0.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b)
{
    int64_t q = int64_t(double(a) * __builtin_amdgcn_rcp(double(b)));   // off by a little
    while (q * b > a) --q;
    while ((q + 1) * b <= a) ++q;
    return q;
}

// One step of a wave's running sum and largest value: with what lies in the
// lane that CTRL names, in the rows of lanes ROWS (elsewhere with zero).
template <int CTRL, int ROWS>
__device__ __forceinline__ void scan_step(int64_t& sum, int& most)
{
    const uint32_t lo = uint32_t(__builtin_amdgcn_update_dpp(0, int(sum), CTRL, ROWS, 0xf, false));
    const uint32_t hi = uint32_t(__builtin_amdgcn_update_dpp(0, int(sum >> 32), CTRL, ROWS, 0xf, false));
    sum += int64_t(uint64_t(hi) << 32 | lo);
    most = max(most, __builtin_amdgcn_update_dpp(0, most, CTRL, ROWS, 0xf, false));
}

// The sum of the lanes up to each one, and the largest of them (none negative).
__device__ __forceinline__ void scan_lanes(int64_t& sum, int& most)
{
    scan_step<0x111, 0xf>(sum, most);      // lanes 1, 2, 4 and 8 before in their sixteen,
    scan_step<0x112, 0xf>(sum, most);
    scan_step<0x114, 0xf>(sum, most);
    scan_step<0x118, 0xf>(sum, most);
    scan_step<0x142, 0xa>(sum, most);      // the last of the sixteen before, of the half before
    scan_step<0x143, 0xc>(sum, most);
}

// The same value in every lane, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t x)
{
    const uint32_t lo = uint32_t(__builtin_amdgcn_readfirstlane(int(x)));
    const uint32_t hi = uint32_t(__builtin_amdgcn_readfirstlane(int(x >> 32)));
    return int64_t(uint64_t(hi) << 32 | lo);
}

// The kernel's arguments, strides and sizes in 32 bits (few scalar registers).
struct Args {
    const uint8_t* k;
    const uint8_t* v;
    const float* k_scale;
    const float* v_scale;
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* table;
    uint8_t* workspace;
    uint32_t page16, head16, slot16;          // cache strides in 16 bytes
    uint32_t q_token, q_head, o_token, o_head, lse_token, table_stride;
    int32_t pages, kv_heads, page_shift, dim;
    int32_t tokens, max_q, cap, window, seqs; // cap: keys a sequence may have; window 0: none
    int32_t group;
    uint32_t by_group;                        // ceil(2^31 / group)
    float scale;
};

// A 4-bit cache has exponent bytes beside its codes (strides in bytes).
struct BlockArgs : Args {
    const uint8_t* k_block;
    const uint8_t* v_block;
    uint32_t block_page, block_head, block_slot;
};

enum Kind { kBf16, kE4m3, kMxfp4 };

// Rows of a sequence and kv head (tokens x group) up to which a 4-bit cache's
// calls may go in row tiles, see few_rows() of paged_attention.hip.
constexpr int64_t kFewRows = 512;

// x / group, exact while x * group is below 2^31.  In the shared tiles x is a row
// of a unit beside the heads before its first, below 255 + group, and group below
// 2^15; in row tiles a row of the whole sequence, below kFewRows, as is group - 1.
static_assert((255 + (int64_t(1) << 15)) << 15 < int64_t(1) << 31 && kFewRows * kFewRows < int64_t(1) << 31, "by_group is exact");
__device__ __forceinline__ uint32_t by_group(const Args& p, uint32_t x) { return __umulhi(2 * x, p.by_group); }

__device__ __forceinline__ Seq load_seq(const Args& p, int b)
{
    return cut_seq(p.q_start[b], p.q_start[b + 1], p.kv_len[b], p.tokens, p.max_q, p.cap);
}

}  // namespace

}  // namespace qg
