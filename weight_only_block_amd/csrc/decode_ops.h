// Internal interface of the operators between a decode step's GEMV calls:
// rotary positions with cache append (rope.hip, rope_mxfp4.hip), cached tokens
// read back (kv_read.hip), attention over the paged cache (paged_attention.hip)
// and token sampling (sample.hip).
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

#ifdef __HIP_DEVICE_COMPILE__
// The scale that the 4-bit conversions take for a block's exponent byte: they
// read its exponent bits alone, all set for NaN and none for 2^-127.
__device__ __forceinline__ float block_scale(uint32_t b) { return __uint_as_float((b > 252 ? 255u : b) << 23); }
#else
__device__ inline float block_scale(uint32_t) { return 0.0f; }
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
    bool e4m3, mxfp4;                          // mxfp4: codes, two elements a byte
};

// A 4-bit cache's exponent bytes (strides in bytes).
struct BlockView {
    uint8_t* k;
    uint8_t* v;
    int64_t page_stride, head_stride, slot_stride;
};

constexpr int kBlock = 32;        // dimensions that share an exponent byte

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

hipError_t launch_rope(const RopeParams& p, const BlockView& blocks, hipStream_t s);
hipError_t launch_rope_mxfp4(const RopeParams& p, const BlockView& blocks, hipStream_t s);   // at most 2^23 tokens

struct ReadParams {
    CacheView cache;
    const int64_t* slots;
    void* k;                // null: not wanted
    void* v;
    int64_t k_token, k_head, v_token, v_head;   // strides, elements
    int64_t tokens;
    bool f32;
    bool wide;              // every row starts on 16 bytes
    BlockView blocks;
};

hipError_t launch_read(const ReadParams& p, hipStream_t s);

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
    BlockView blocks;
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
size_t attention_workspace_need(const CacheView& cache, const BlockView& blocks, int64_t tokens, int q_heads, int seqs,
                                int64_t max_q, int64_t max_kv);
size_t attention_workspace_bytes(const CacheView& cache, const BlockView& blocks, int64_t tokens, int q_heads, int seqs,
                                 int64_t max_q, int64_t max_kv);
hipError_t launch_attention(const AttnParams& p, hipStream_t s);

// Successful launches by kernel, for tests: waves that stream keys of their own;
// tiles that four or eight waves share; row tiles of a 4-bit cache.
enum AttentionRoute { kSplit, kTiles4, kTiles8, kRowTiles, kAttentionRoutes };
constexpr const char* kAttentionRouteNames[kAttentionRoutes] = {"attention_split", "attention_tiles4", "attention_tiles8",
                                                                 "attention_rows"};
uint64_t attention_route_count(int route);
void attention_route_reset();

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
