// Internal interface of the operators between a decode step's GEMV calls:
// rotary positions with cache append (rope.hip), attention over the paged
// cache (paged_attention.hip) and token sampling (sample.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qg {

#ifdef __HIP_DEVICE_COMPILE__
// Reads a word of each 64-byte line of the kernel's first BYTES argument bytes
// at once.  A line's first read misses every cache (about 1 us); without this
// each line's miss comes where its first argument is used, one after another.
template <int BYTES>
__device__ __forceinline__ void fetch_arguments()
{
    typedef const __attribute__((address_space(4))) uint32_t* words;
    words a = (words)__builtin_amdgcn_kernarg_segment_ptr();
    uint32_t v[(BYTES + 63) / 64];
#pragma unroll
    for (int i = 0; i < (BYTES + 63) / 64; ++i) v[i] = a[16 * i];
#pragma unroll
    for (int i = 0; i < (BYTES + 63) / 64; ++i) asm volatile("" ::"s"(v[i]));
}
#else
template <int BYTES>
__device__ inline void fetch_arguments()
{
}
#endif

constexpr int kMaxHeadDim = 256;
constexpr int kMaxRotPairs = kMaxHeadDim / 2;

// The paged cache as the kernels see it (strides in elements).
struct CacheView {
    uint8_t* k;
    uint8_t* v;
    const float* k_scale;   // one per kv head; null for bf16
    const float* v_scale;
    int64_t page_stride, head_stride, slot_stride;
    int64_t pages;
    int32_t kv_heads, page_shift, head_dim;
    bool e4m3;
};

struct RopeParams {
    CacheView cache;
    const void* q;
    const void* k;
    const void* v;
    int64_t q_token, q_head, k_token, k_head, v_token, v_head;   // strides, elements
    uint16_t* q_out;
    int64_t o_token, o_head;
    const int32_t* pos;
    const int64_t* slots;
    int64_t tokens;
    int32_t q_heads;
    int32_t rot_dim;
    bool f32, interleaved;
    bool wide;              // every row starts 16-byte aligned and divides into whole vectors
    float amplitude;
    uint64_t turns[kMaxRotPairs];   // turns per position, 64-bit binary fraction
};

hipError_t launch_rope(const RopeParams& p, hipStream_t s);

struct AttnParams {
    CacheView cache;
    const uint16_t* q;
    int64_t q_token, q_head;
    uint16_t* out;
    int64_t o_token, o_head;
    float* lse;             // null: not wanted
    int64_t lse_token;
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* table;
    int64_t table_stride, table_cols;
    int64_t tokens, max_q, max_kv, window;   // window 0: none
    int32_t seqs, q_heads, group;
    float scale;
    void* workspace;
};

// A sequence's new rows [q0, q0 + n) and cached keys.
struct Seq {
    int q0, n, kv;
};

// From its starts and length as the caller's device memory holds them, whatever
// that is, cut to the call's rows, to max_q rows and to cap keys.
__host__ __device__ inline Seq cut_seq(int start, int next, int kv, int tokens, int max_q, int cap)
{
    const auto cut = [](int x, int most) { return x < 0 ? 0 : x < most ? x : most; };
    Seq s;
    s.q0 = cut(start, tokens);
    s.n = cut(cut(next, tokens) - s.q0, max_q);   // (both within [0, tokens]: no wrap)
    s.kv = cut(kv, cap);
    return s;
}

// Of this shape; of this shape and every smaller one.
size_t attention_workspace_need(bool e4m3, int64_t tokens, int q_heads, int kv_heads, int head_dim, int seqs,
                                int64_t max_q, int64_t max_kv);
size_t attention_workspace_bytes(bool e4m3, int64_t tokens, int q_heads, int kv_heads, int head_dim, int seqs,
                                 int64_t max_q, int64_t max_kv);
hipError_t launch_attention(const AttnParams& p, hipStream_t s);

struct SampleParams {
    const float* x;
    int64_t m, N, ldx;
    const float* u;
    const float* temperature;   // null: 1
    const int32_t* top_k;       // null or <= 0: none
    const float* top_p;         // null: 1
    const float* min_p;         // null: 0
    int32_t* idx;
    void* workspace;
};

size_t sample_workspace_need(int64_t m, int64_t N);    // of this shape
size_t sample_workspace_bytes(int64_t m, int64_t N);   // of this shape and every smaller one
hipError_t launch_sample(const SampleParams& p, hipStream_t s);

}  // namespace qg
