// Attention of a chunk of new tokens over the paged cache, on the matrix
// cores.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q . k_j - m)
//
// with m a running reference of the row's scores, raised (and the sums scaled
// down) only when a score passes it by 2^8: any reference gives the same
// quotient, and p up to 2^8 loses nothing in fp32 or bf16.
//
// Rows.  The query heads that share a kv head are rows beside the tokens: row
// r of a sequence is token r / group, head r % group, so a key tile is read
// once for all of them.  A unit of work is (kv head, sequence, tile of rows).
//
// Products.  S^T = K Q^T and O^T = V^T P^T, 32x32x16 tiles: a lane then holds
// scores of one row (its column) in both, so the softmax needs one exchange
// between the wave's halves, and the lane's scores are, in order, the B
// operand of the second product when V's keys are taken in that order
// (key 16 t + 8 (j / 4) + 4 h + j % 4 for half h, element j).  V^T comes from
// the row-major tile through the transposing LDS reads.
//
// Two shapes.  `Shared`: the work-group's four waves hold 32 rows each and
// share key tiles of K and V in LDS, so a tile is read once for 128 rows; for
// prompts and chunks, bound by the matrix cores.  `Split`: the waves hold the
// same up to 32 rows and each streams key tiles of its own, joined in LDS at
// the end; for single and drafted tokens, bound by reading the cache.
//
// Division of the work.  All units' key steps are laid out in one line, head
// by head, and cut into equal runs, one per work-group, whatever the lengths
// are: lengths live on the device, so every work-group sums them itself.  A
// unit that falls into several runs leaves fp32 partial sums in the
// workspace; the work-group that finishes last joins them in run order, so
// the result does not depend on timing.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "decode_ops.h"

namespace qg {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.0f;             // log2 by which a score may pass the reference
constexpr int kListPages = 1024;           // page ids of a run's segment, in LDS
constexpr int kListSeqs = 128;             // sequences whose lengths are kept in LDS
constexpr int kComputeUnits = 256;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;

__device__ __forceinline__ uint32_t lds_offset(const void* p)
{
    return uint32_t(uintptr_t((__attribute__((address_space(3))) const char*)p));
}

// 16 bytes per lane from global memory to LDS at lds + 16 * lane, with no
// register between.  The compiler does not count these loads: every use waits
// by hand (wait_loads).
__device__ __forceinline__ void load_lds_uniform(uint32_t lds, uint64_t base, uint32_t offset)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(offset), "s"(base)
                 : "memory");
}
__device__ __forceinline__ void load_lds(uint32_t lds, uint64_t address)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(address) : "memory");
}
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

__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32, 64); }

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

// One kernel shape.  DP: head dimension padded to a matrix-core multiple.
template <int DP_, bool E4M3_, bool SHARED_>
struct Shape {
    static constexpr int DP = DP_;
    static constexpr bool E4M3 = E4M3_, SHARED = SHARED_;
    // Waves.  Split: two, so that two to four work-groups share a compute
    // unit and one streams while another begins or ends a unit.
    static constexpr int W = SHARED ? 4 : DP == 256 && !E4M3 ? 1 : 2;
    static constexpr int THREADS = 64 * W;
    static constexpr int WAVES_PER_SIMD = DP <= 128 ? 2 : 1;
    static constexpr int M = SHARED ? 32 * W : 32;                      // rows of a unit
    static constexpr int KT = SHARED && DP <= 128 ? 64 : 32;            // keys of a wave's tile
    static constexpr int BLOCKS = KT / 32;
    static constexpr int STEP = SHARED ? KT : KT * W;                   // keys of a work-group's step
    static constexpr int ES = E4M3 ? 1 : 2;
    static constexpr int RB = (DP == 96 ? 128 : DP) * ES;               // bytes of a tile row
    static constexpr int CPR = RB / 16;                                 // 16-byte chunks of it
    static constexpr int RPI = 64 / CPR;                                // rows of one load instruction
    static constexpr int TILE = KT * RB;                                // bytes of K or of V
    static constexpr int ROWS = SHARED ? KT / W : KT;                   // rows a wave loads
    static constexpr int LOADS = ROWS / RPI;                            // for K, and as many for V
    static constexpr int RING = 2 * 2 * TILE * (SHARED ? 1 : W);        // two stages of K and V
    static constexpr int OS = DP + 4;                                   // floats of a row in the joining buffer
    static constexpr int JOIN = SHARED ? 0 : W * M * OS * 4;
    static constexpr int BUFFER = RING > JOIN ? RING : JOIN;
    static constexpr int LDS = BUFFER + kListPages * 4 + 2 * W * 32 * 4 + 64 + kListSeqs * 12;
    // work-groups that a compute unit holds (160 KB of LDS, two waves of up to
    // 256 registers a SIMD or one of 512)
    static constexpr int BY_LDS = 160 * 1024 / LDS, BY_WAVES = 4 * WAVES_PER_SIMD / W;
    static constexpr int PER_CU = BY_LDS < BY_WAVES ? BY_LDS : BY_WAVES;
    // Steps that a run has at least: a shorter one costs more in joining its
    // part than it saves.
    static constexpr int LEAST = SHARED ? 8 : 4;
    static constexpr int EXTRA = SHARED ? 4 : 3;
    static constexpr int SLOT = M * DP + 2 * M;                         // floats of a partial result
    static constexpr int STEPS = DP / 16;                               // products along the dimension
    static constexpr int DB = DP / 32;

    // Swizzles: the chunk of a row's 16 bytes is moved so that the rows of one
    // LDS access lie in different banks.
    static __device__ __forceinline__ int k_swizzle(int row) { return CPR == 4 ? (row >> 1) & 3 : row & 7; }
    static __device__ __forceinline__ int v_swizzle(int row)
    {
        if (!E4M3) return (row & 3) << 1;
        return CPR == 4 ? ((row >> 1) & 1) | (((row >> 3) & 1) << 1) : (row & 3) | (((row >> 3) & 1) << 2);
    }
};

struct Seq {
    int q0, n, kv;
};

__device__ __forceinline__ Seq load_seq(const AttnParams& p, int b)
{
    Seq s;
    const int64_t q0 = max(int64_t(0), min(int64_t(p.q_start[b]), p.tokens));
    const int64_t q1 = max(q0, min(min(int64_t(p.q_start[b + 1]), p.tokens), q0 + p.max_q));
    const int64_t cap = min(p.max_kv, p.table_cols << p.cache.page_shift);
    s.q0 = int(q0);
    s.n = int(q1 - q0);
    s.kv = int(max(int64_t(0), min(int64_t(p.kv_len[b]), cap)));
    return s;
}

// From LDS where all sequences fit.
__device__ __forceinline__ Seq get_seq(const AttnParams& p, const Seq* seqs, int b)
{
    return p.seqs <= kListSeqs ? seqs[b] : load_seq(p, b);
}

struct Range {
    int lo, hi, base;   // keys [lo, hi) that some row sees; the first tile starts at base
};

template <class S>
__device__ __forceinline__ Range unit_range(const AttnParams& p, const Seq& s, int tile)
{
    const int rows = s.n * p.group, r0 = tile * S::M, r1 = min(r0 + S::M, rows) - 1;
    const int first = s.kv - s.n + r0 / p.group, last = s.kv - s.n + r1 / p.group;
    Range g;
    g.hi = max(0, last + 1);
    g.lo = p.window > 0 ? int(max(int64_t(0), int64_t(first) - p.window + 1)) : 0;
    if (g.lo > g.hi) g.lo = g.hi;
    g.base = g.lo & ~15;
    return g;
}

template <class S>
__device__ __forceinline__ int unit_steps(const AttnParams& p, const Seq& s, int tile)
{
    const Range g = unit_range<S>(p, s, tile);
    return g.hi > g.lo ? (g.hi - g.base + S::STEP - 1) / S::STEP : 1;   // a unit without keys still writes its rows
}

// A unit's length in the line: its steps and what beginning and ending it
// costs, in steps.
template <class S>
__device__ __forceinline__ int unit_cost(const AttnParams& p, const Seq& s, int tile)
{
    return unit_steps<S>(p, s, tile) + S::EXTRA;
}

template <class S>
__device__ __forceinline__ int seq_tiles(const AttnParams& p, const Seq& s)
{
    return int((int64_t(s.n) * p.group + S::M - 1) / S::M);
}

// What a wave accumulates: its 32 rows are the lanes' columns.
template <class S>
struct State {
    f32x16 o[S::DB];
    bf16x8 q[S::STEPS];
    float m, l;          // reference; this half's share of the sum
    int rlo, rhi;        // keys the lane's row sees
};

// A key tile (K and V, 32 or 64 keys from k0) against the wave's rows.
// `masked`: some row does not see some key.
template <class S>
__device__ __forceinline__ void compute(State<S>& st, const uint8_t* kt, const uint8_t* vt, int k0, float c, bool masked)
{
    const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5, i16 = lane & 15, dh = (lane >> 4) & 1;
    f32x16 s[S::BLOCKS];
#pragma unroll
    for (int b = 0; b < S::BLOCKS; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[b][i] = 0.0f;
    // scores
    const int ksw = S::k_swizzle(col);
#pragma unroll
    for (int b = 0; b < S::BLOCKS; ++b) {
        const uint8_t* row = kt + (b * 32 + col) * S::RB;
        if (!S::E4M3) {
#pragma unroll
            for (int t = 0; t < S::STEPS; ++t) {
                const bf16x8 a = *reinterpret_cast<const bf16x8*>(row + (((2 * t + h) ^ ksw) << 4));
                s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, st.q[t], s[b], 0, 0, 0);
            }
        } else {
            // one 16-byte read is two steps: step 2 t + e takes dimensions 32 t + 16 h + 8 e on
#pragma unroll
            for (int t = 0; t < S::STEPS / 2; ++t) {
                const u32x4 raw = *reinterpret_cast<const u32x4*>(row + (((2 * t + h) ^ ksw) << 4));
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    union { bf16x8 v; bf16x2 p[4]; } a;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        a.p[2 * x] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[2 * e + x], 1.0f, false);
                        a.p[2 * x + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[2 * e + x], 1.0f, true);
                    }
                    s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, st.q[2 * t + e], s[b], 0, 0, 0);
                }
            }
        }
    }
    if (masked) {
        const uint32_t width = uint32_t(st.rhi - st.rlo);
        const int first = k0 + 4 * h - st.rlo;
#pragma unroll
        for (int b = 0; b < S::BLOCKS; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (uint32_t(first + 32 * b + 8 * (i / 4) + i % 4) >= width) s[b][i] = -INFINITY;
    }
    // reference
    float top = s[0][0];
#pragma unroll
    for (int b = 0; b < S::BLOCKS; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
    top = fmaxf(top, other_half(top)) * c;
    const bool raise = top > st.m + kRaise;
    if (__any(raise)) {
        // of this lane's row alone: other rows keep their reference and their bits
        const float mn = raise ? top : st.m;
        const float keep = raise ? __builtin_amdgcn_exp2f(st.m - mn) : 1.0f;
        st.m = mn;
        st.l *= keep;
#pragma unroll
        for (int d = 0; d < S::DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) st.o[d][i] *= keep;
    }
    const float ref = st.m == -INFINITY ? 0.0f : st.m;
    float sum = 0.0f;
#pragma unroll
    for (int b = 0; b < S::BLOCKS; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[b][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][i], c, -ref));
            sum += s[b][i];
        }
    st.l += sum;
    // Output.  Probabilities become bf16 (half a step, 2^-9 of each on
    // average less: errors of many keys cancel) for the matrix cores.
#pragma unroll
    for (int b = 0; b < S::BLOCKS; ++b)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            union { bf16x8 v; uint32_t u[4]; } pb;
#pragma unroll
            for (int x = 0; x < 4; ++x) pb.u[x] = pack_bf16(s[b][8 * t + 2 * x], s[b][8 * t + 2 * x + 1]);
#pragma unroll
            for (int d = 0; d < S::DB; ++d) {
                union { bf16x8 v; s16x4 h[2]; bf16x2 p[4]; } a;
                if (!S::E4M3) {
                    const int row = b * 32 + 16 * t + 4 * h + i16 / 4;
                    const int chunk = (4 * d + 2 * dh + (i16 & 3) / 2) ^ S::v_swizzle(row);
                    const uint8_t* at = vt + row * S::RB + (chunk << 4) + (i16 & 1) * 8;
                    a.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
                    a.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 8 * S::RB));
                } else {
                    const int rr = i16 / 2, row = b * 32 + 16 * t + 8 * (rr / 4) + 4 * h + rr % 4;
                    const int chunk = (2 * d + dh) ^ S::v_swizzle(row);
                    const i32x2 raw = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                        (lds_i32x2*)(vt + row * S::RB + (chunk << 4) + (i16 & 1) * 8));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        a.p[2 * x] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[x], 1.0f, false);
                        a.p[2 * x + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[x], 1.0f, true);
                    }
                }
                st.o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, pb.v, st.o[d], 0, 0, 0);
            }
        }
}

// The loads of one tile, and what the tile needs before use.
template <class S>
struct Loader {
    const AttnParams& p;
    const int32_t* list;      // LDS: page ids from page `first_page` on, -1 outside the sequence or the cache
    int first_page;
    const int32_t* table;     // the sequence's row of the page table
    int pages;                // of the sequence
    uint64_t kbase, vbase;    // of this kv head
    int lo, hi;               // keys that some row of the unit sees
    int all_lo, all_hi;       // and that every row sees
    int64_t* poisoned;        // LDS

    // Rows [0, ROWS) of the wave's part, the first being key k0 + row0 of the tile at LDS kt, vt.
    __device__ __forceinline__ bool issue(uint8_t* kt, uint8_t* vt, int k0, int row0) const
    {
        const int lane = threadIdx.x & 63, lr = lane / S::CPR, lc = lane % S::CPR;
        const int chunks = p.cache.head_dim * S::ES / 16;
        const uint64_t slot_bytes = uint64_t(p.cache.slot_stride) * S::ES, page_bytes = uint64_t(p.cache.page_stride) * S::ES;
        const int mask = (1 << p.cache.page_shift) - 1;
        bool dirty = k0 + row0 < all_lo || k0 + row0 + S::ROWS > all_hi;
        int ids[S::LOADS];
        if (p.cache.page_shift >= 4 && slot_bytes < (1u << 24)) {
            // all rows of one load lie in one page
            const uint32_t row_off = uint32_t(lr) * uint32_t(slot_bytes);
#pragma unroll
            for (int j = 0; j < S::LOADS; ++j) ids[j] = list[((k0 + row0 + j * S::RPI) >> p.cache.page_shift) - first_page];
#pragma unroll
            for (int j = 0; j < S::LOADS; ++j) {
                const int row = row0 + j * S::RPI, key = k0 + row;
                int id = __builtin_amdgcn_readfirstlane(ids[j]);
                if (id < 0) dirty = true, id = 0;
                const uint64_t off = uint64_t(id) * page_bytes + uint64_t(key & mask) * slot_bytes;
                const int ck = lc ^ S::k_swizzle(row + lr), cv = lc ^ S::v_swizzle(row + lr);
                const uint32_t dk = __builtin_amdgcn_readfirstlane(lds_offset(kt + row * S::RB));
                const uint32_t dv = __builtin_amdgcn_readfirstlane(lds_offset(vt + row * S::RB));
                if (ck < chunks) load_lds_uniform(dk, kbase + off, row_off + 16 * ck);
                if (cv < chunks) load_lds_uniform(dv, vbase + off, row_off + 16 * cv);
            }
        } else {
#pragma unroll
            for (int j = 0; j < S::LOADS; ++j) ids[j] = list[((k0 + row0 + j * S::RPI + lr) >> p.cache.page_shift) - first_page];
#pragma unroll
            for (int j = 0; j < S::LOADS; ++j) {
                const int row = row0 + j * S::RPI, key = k0 + row + lr;
                int id = ids[j];
                if (__any(id < 0)) dirty = true;
                if (id < 0) id = 0;
                const uint64_t off = uint64_t(id) * page_bytes + uint64_t(key & mask) * slot_bytes;
                const int ck = lc ^ S::k_swizzle(row + lr), cv = lc ^ S::v_swizzle(row + lr);
                const uint32_t dk = __builtin_amdgcn_readfirstlane(lds_offset(kt + row * S::RB));
                const uint32_t dv = __builtin_amdgcn_readfirstlane(lds_offset(vt + row * S::RB));
                if (ck < chunks) load_lds(dk, kbase + off + 16 * ck);
                if (cv < chunks) load_lds(dv, vbase + off + 16 * cv);
            }
        }
        return dirty;
    }

    // Rows outside [lo, hi) hold another's data: their values become zeros
    // (their scores are masked).  Keys of a page outside the cache become NaN.
    // A value that is not finite at a key that only some rows see would be
    // NaN times 0 in the others: it becomes 0 too, and rows that see it get it
    // back at the end (restore).
    __device__ __forceinline__ void patch(uint8_t* kt, uint8_t* vt, int k0, int row0) const
    {
        const int lane = threadIdx.x & 63, lr = lane / S::CPR, lc = lane % S::CPR;
        const int chunks = p.cache.head_dim * S::ES / 16;   // those past the dimension stay zero
        const uint32_t nan = S::E4M3 ? 0x7f7f7f7fu : 0x7fc07fc0u;
#pragma unroll 1
        for (int j = 0; j < S::LOADS; ++j) {
            const int row = row0 + j * S::RPI + lr, key = k0 + row;
            const bool outside = key < lo || key >= hi;
            const int page = key >> p.cache.page_shift;
            int64_t id = -1;
            if (!outside && page < pages) id = table[page];
            const bool lost = !outside && (id < 0 || id >= p.cache.pages);
            u32x4* v = reinterpret_cast<u32x4*>(vt + row * S::RB + 16 * lc);
            if (outside || lost) {
                *v = u32x4{0, 0, 0, 0};
            } else if (key < all_lo || key >= all_hi) {
                u32x4 x = *v;
                uint32_t dropped = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t drop = 0;
                    if (!S::E4M3) {
                        const uint32_t w = x[e] & 0x7f807f80u;
                        drop = ((w & 0xffff0000u) == 0x7f800000u ? 0xffff0000u : 0u) | ((w & 0xffffu) == 0x7f80u ? 0xffffu : 0u);
                    } else {
                        // a NaN code is 0x7f but for its sign; there is no infinity
                        drop = (((x[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
                        drop *= 255u;
                    }
                    dropped |= drop;
                    x[e] &= ~drop;
                }
                if (dropped) {
                    *v = x;
                    *poisoned = 1;
                }
            }
            if (lost && (lc ^ S::k_swizzle(row)) < chunks) *reinterpret_cast<u32x4*>(kt + row * S::RB + 16 * lc) = u32x4{nan, nan, nan, nan};
        }
        wait_lds();
    }
};

// Gives the lane's row the values that patch() took out, of keys [from, to).
template <class S>
__device__ __forceinline__ void restore(State<S>& st, const AttnParams& p, const Loader<S>& ld, int from, int to)
{
    const int h = (threadIdx.x & 63) >> 5;
    const int mask = (1 << p.cache.page_shift) - 1;
#pragma unroll 1
    for (int key = max(from, ld.lo); key < min(to, ld.hi); ++key) {
        if (key >= ld.all_lo && key < ld.all_hi) continue;
        const int64_t id = ld.table[key >> p.cache.page_shift];
        if (id < 0 || id >= p.cache.pages) continue;
        const uint8_t* row = reinterpret_cast<const uint8_t*>(ld.vbase) +
                             (id * p.cache.page_stride + int64_t(key & mask) * p.cache.slot_stride) * S::ES;
        const bool sees = key >= st.rlo && key < st.rhi;
#pragma unroll
        for (int d = 0; d < S::DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int dim = 32 * d + 8 * (i / 4) + 4 * h + i % 4;
                if (dim >= p.cache.head_dim) continue;
                float v;
                if (!S::E4M3) v = __uint_as_float(uint32_t(reinterpret_cast<const uint16_t*>(row)[dim]) << 16);
                else v = __builtin_amdgcn_cvt_f32_fp8(int(row[dim]), 0);
                if (sees && !(fabsf(v) < INFINITY)) st.o[d][i] += v;
            }
    }
}

template <class S>
__global__ __launch_bounds__(S::THREADS, S::WAVES_PER_SIMD) void attention_kernel(AttnParams p, int64_t counters)
{
    extern __shared__ __align__(1024) uint8_t lds[];
    int32_t* list = reinterpret_cast<int32_t*>(lds + S::BUFFER);
    float* ml = reinterpret_cast<float*>(list + kListPages);      // [2][W][32]
    int64_t* plan = reinterpret_cast<int64_t*>(ml + 2 * S::W * 32);   // 8 values
    Seq* seqs = reinterpret_cast<Seq*>(plan + 8);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, h = lane >> 5, dim = p.cache.head_dim;

    fetch_arguments<sizeof(AttnParams)>();

    // ---- the line of work: this run's part of it
    int64_t mine = 0;
    int mine_units = 0;
    const int per = (p.seqs + S::THREADS - 1) / S::THREADS;
    const int b0 = min(int(threadIdx.x) * per, p.seqs), b1 = min(b0 + per, p.seqs);
    for (int b = b0; b < b1; ++b) {
        const Seq s = load_seq(p, b);
        if (p.seqs <= kListSeqs) seqs[b] = s;
        const int tiles = seq_tiles<S>(p, s);
        mine_units += tiles;
        for (int t = 0; t < tiles; ++t) mine += unit_cost<S>(p, s, t);
    }
    int64_t upto = mine;
    int upto_units = mine_units;
    for (int off = 1; off < 64; off <<= 1) {
        const int64_t a = __shfl_up((long long)upto, off, 64);
        const int u = __shfl_up(upto_units, off, 64);
        if (lane >= off) upto += a, upto_units += u;
    }
    int64_t* sums = reinterpret_cast<int64_t*>(lds);              // [W] steps, [W] units
    if (lane == 63) sums[wave] = upto, sums[S::W + wave] = upto_units;
    __syncthreads();
    int64_t head_steps = 0, before = 0;
    int head_units = 0, before_units = 0;
    for (int w = 0; w < S::W; ++w) {
        if (w == wave) before = head_steps, before_units = head_units;
        head_steps += sums[w];
        head_units += int(sums[S::W + w]);
    }
    upto += before;
    upto_units += before_units;
    const int64_t total = head_steps * p.cache.kv_heads;
    // starts that are not ascending claim more rows than there are
    if (int64_t(head_units) * p.cache.kv_heads > counters) return;
    const int64_t runs = max(int64_t(1), min(int64_t(gridDim.x), total / S::LEAST));
    // consecutive work-groups go to different XCDs: give each XCD one stretch
    // of the line, so that its L2 holds few heads' keys
    const int xcds = gridDim.x % 8 == 0 ? 8 : 1;
    const int64_t run = runs < int64_t(gridDim.x) ? int64_t(blockIdx.x)   // few: over all XCDs
                                                  : int64_t(blockIdx.x % xcds) * (gridDim.x / xcds) + blockIdx.x / xcds;
    if (run >= runs || total == 0) return;
    // the first `longer` runs have base + 1 steps, the others base
    const int64_t base = total / runs, longer = total - base * runs;
    const auto run_start = [&](int64_t w) { return w * base + min(w, longer); };
    const auto run_of = [&](int64_t x) {
        const int64_t split = longer * (base + 1);
        return x < split ? x / (base + 1) : longer + (x - split) / base;
    };
    int64_t at = run_start(run);
    const int64_t end = run_start(run + 1);
    int kvh = int(at / head_steps);
    {
        const int64_t r = at - kvh * head_steps;
        if (r >= upto - mine && r < upto) {
            int64_t left = r - (upto - mine);
            int unit = upto_units - mine_units;
            for (int b = b0; b < b1; ++b) {
                const Seq s = get_seq(p, seqs, b);
                const int tiles = seq_tiles<S>(p, s);
                bool found = false;
                for (int t = 0; t < tiles && !found; ++t) {
                    const int n = unit_cost<S>(p, s, t);
                    if (left < n) {
                        plan[0] = b, plan[1] = t, plan[2] = left, plan[3] = unit;
                        found = true;
                    } else {
                        left -= n;
                        ++unit;
                    }
                }
                if (found) break;
            }
        }
    }
    __syncthreads();
    int b = __builtin_amdgcn_readfirstlane(int(plan[0])), tile = __builtin_amdgcn_readfirstlane(int(plan[1]));
    int off = __builtin_amdgcn_readfirstlane(int(plan[2])), unit = __builtin_amdgcn_readfirstlane(int(plan[3]));

    // dimensions past the head's end stay zero in every tile
    const auto clear = [&] {
        if (dim < S::DP)
            for (int i = threadIdx.x; i < S::BUFFER / 16; i += S::THREADS) reinterpret_cast<u32x4*>(lds)[i] = u32x4{0, 0, 0, 0};
    };
    clear();

    uint32_t* arrived = static_cast<uint32_t*>(p.workspace);
    float* slots = reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) + (size_t(counters) * 4 + 255) / 256 * 256);

    // Goes on to the next unit of the line.
    const auto advance = [&](int cost) {
        at += cost;
        off = 0;
        if (at >= end) return;
        ++tile;
        ++unit;
        Seq q = get_seq(p, seqs, b);
        while (tile >= seq_tiles<S>(p, q)) {
            tile = 0;
            if (++b == p.seqs) b = 0, unit = 0, ++kvh;
            q = get_seq(p, seqs, b);
        }
    };

    while (at < end) {
        const Seq s = get_seq(p, seqs, b);
        const int rows = min(S::M, s.n * p.group - tile * S::M);
        const Range g = unit_range<S>(p, s, tile);
        const int steps = unit_steps<S>(p, s, tile);
        const int take = int(min(int64_t(steps + S::EXTRA - off), end - at));
        const int from = max(0, off - S::EXTRA), count = max(0, off + take - S::EXTRA) - from;
        if (count == 0) {       // only what stands for the unit's beginning
            advance(take);
            continue;
        }
        const float ks = S::E4M3 ? p.cache.k_scale[kvh] : 1.0f;
        float c = p.scale * ks * kLog2e;
        const bool neg = c < 0.0f;
        const bool none = c == 0.0f;
        c = none ? 1.0f : fabsf(c);

        // ---- the wave's rows
        State<S> st;
        const int row = S::SHARED ? wave * 32 + col : col;
        const bool live = row < rows;
        const int r = tile * S::M + row;
        const int token = r / p.group, head = kvh * p.group + r % p.group;
        const int pos = s.kv - s.n + token;
        st.rhi = live ? max(0, pos + 1) : 0;
        st.rlo = live && p.window > 0 ? int(min(int64_t(st.rhi), max(int64_t(0), int64_t(pos) - p.window + 1))) : 0;
        st.m = -INFINITY;
        st.l = 0.0f;
#pragma unroll
        for (int d = 0; d < S::DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) st.o[d][i] = 0.0f;
#pragma unroll
        for (int t = 0; t < S::STEPS; ++t) {
            const int d = S::E4M3 ? 32 * (t / 2) + 16 * h + 8 * (t % 2) : 16 * t + 8 * h;
            u32x4 x = {0, 0, 0, 0};
            if (live && d < dim)
                x = *reinterpret_cast<const u32x4*>(p.q + (s.q0 + token) * p.q_token + head * p.q_head + d);
            // the scale's sign goes into the queries, so that the largest
            // score stays the largest; a scale of zero leaves equal scores
            if (neg) x ^= 0x80008000u;
            if (none) x = u32x4{0, 0, 0, 0};
            st.q[t] = __builtin_bit_cast(bf16x8, x);
        }
        // keys that every row of this wave sees, and that any does
        const int wr0 = S::SHARED ? wave * 32 : 0, wr1 = min(wr0 + 32, rows) - 1;
        const bool busy = wr0 < rows;
        int all_lo = 0, all_hi = 0, any_lo = 0, any_hi = 0;
        if (busy) {
            const int f = s.kv - s.n + (tile * S::M + wr0) / p.group, l = s.kv - s.n + (tile * S::M + wr1) / p.group;
            all_hi = f + 1;
            any_hi = max(0, l + 1);
            if (p.window > 0) {
                all_lo = int(max(int64_t(0), int64_t(l) - p.window + 1));
                any_lo = int(max(int64_t(0), int64_t(f) - p.window + 1));
            }
        }

        Loader<S> ld{p, list, 0, p.table + int64_t(b) * p.table_stride, 0, 0, 0, g.lo, g.hi, 0, 0, plan + 5};
        ld.all_hi = s.kv - s.n + tile * S::M / p.group + 1;
        ld.all_lo = p.window > 0 ? int(max(int64_t(0), int64_t(s.kv - s.n + (tile * S::M + rows - 1) / p.group) - p.window + 1)) : 0;
        if (threadIdx.x == 0) plan[5] = 0;
        ld.pages = int((int64_t(s.kv) + (int64_t(1) << p.cache.page_shift) - 1) >> p.cache.page_shift);
        ld.kbase = reinterpret_cast<uint64_t>(p.cache.k) + uint64_t(kvh) * p.cache.head_stride * S::ES;
        ld.vbase = reinterpret_cast<uint64_t>(p.cache.v) + uint64_t(kvh) * p.cache.head_stride * S::ES;

        auto run_tile = [&](const uint8_t* kt, const uint8_t* vt, int k0) {
            if (!busy || k0 >= any_hi || k0 + S::KT <= any_lo) return;
            compute<S>(st, kt, vt, k0, c, k0 < all_lo || k0 + S::KT > all_hi);
        };

        // ---- segments of the run whose page ids fit the list
        for (int done = 0; done < count && g.hi > g.lo;) {
            const int start = g.base + (from + done) * S::STEP;
            ld.first_page = start >> p.cache.page_shift;
            // steps whose last key's page is in the list
            const int64_t span = (int64_t(ld.first_page + kListPages) << p.cache.page_shift) - start;
            const int n = int(min(int64_t(count - done), span / S::STEP));
            const int want = int(min(int64_t(kListPages), (int64_t(start) + int64_t(n) * S::STEP - 1 >> p.cache.page_shift) - ld.first_page + 1));
            __syncthreads();
            for (int i = threadIdx.x; i < want; i += S::THREADS) {
                int id = -1;
                if (ld.first_page + i < ld.pages) id = ld.table[ld.first_page + i];
                list[i] = id >= p.cache.pages ? -1 : id;
            }
            __syncthreads();
            if (S::SHARED) {
                const int row0 = wave * S::ROWS;
                bool dirty = ld.issue(lds, lds + S::TILE, start, row0);
                for (int i = 0; i < n; ++i) {
                    uint8_t* kt = lds + (i & 1) * 2 * S::TILE;
                    const int k0 = start + i * S::STEP;
                    wait_loads<0>();
                    if (dirty) ld.patch(kt, kt + S::TILE, k0, row0);
                    __syncthreads();
                    if (i + 1 < n) {
                        uint8_t* nt = lds + ((i + 1) & 1) * 2 * S::TILE;
                        dirty = ld.issue(nt, nt + S::TILE, k0 + S::STEP, row0);
                    }
                    run_tile(kt, kt + S::TILE, k0);
                }
            } else {
                uint8_t* ring = lds + wave * 4 * S::TILE;
                const int k1 = start + wave * S::KT;
                bool dirty = ld.issue(ring, ring + S::TILE, k1, 0), next = false;
                for (int i = 0; i < n; ++i) {
                    uint8_t* kt = ring + (i & 1) * 2 * S::TILE;
                    const int k0 = k1 + i * S::STEP;
                    if (i + 1 < n) {
                        uint8_t* nt = ring + ((i + 1) & 1) * 2 * S::TILE;
                        wait_lds();
                        next = ld.issue(nt, nt + S::TILE, k0 + S::STEP, 0);
                        wait_loads<2 * S::LOADS>();
                    } else {
                        wait_loads<0>();
                    }
                    if (dirty) ld.patch(kt, kt + S::TILE, k0, 0);
                    run_tile(kt, kt + S::TILE, k0);
                    dirty = next;
                }
            }
            done += n;
        }
        st.l += other_half(st.l);
        __syncthreads();
        if (plan[5]) restore(st, p, ld, g.base + from * S::STEP, g.base + (from + count) * S::STEP);

        // ---- results: whole units to the output, parts to the workspace
        const bool whole = count == steps;
        const float vs = S::E4M3 ? p.cache.v_scale[kvh] : 1.0f;
        float* slot = slots + (run * 2 + (off > 0 ? 0 : 1)) * S::SLOT;
        auto put_out = [&](int row, int d, float a0, float a1, float a2, float a3, float inv) {
            const int rr = tile * S::M + row;
            uint16_t* o = p.out + (s.q0 + rr / p.group) * p.o_token + (kvh * p.group + rr % p.group) * p.o_head + d;
            *reinterpret_cast<u32x2*>(o) = u32x2{pack_bf16(a0 * inv, a1 * inv), pack_bf16(a2 * inv, a3 * inv)};
        };
        auto put_lse = [&](int row, float m, float l) {
            const int rr = tile * S::M + row;
            p.lse[(s.q0 + rr / p.group) * p.lse_token + kvh * p.group + rr % p.group] =
                m == -INFINITY && l == 0.0f ? -INFINITY : (m + __log2f(l)) * kLn2;
        };
        // rows that see nothing have l = 0 and o = 0
        auto inverse = [&](float l) { return l == 0.0f ? 0.0f : vs / l; };
        if (S::SHARED) {
            if (live) {
                const float inv = inverse(st.l);
#pragma unroll
                for (int d = 0; d < S::DB; ++d)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int at_d = 32 * d + 8 * x + 4 * h;
                        if (at_d >= dim) continue;
                        if (whole) {
                            put_out(row, at_d, st.o[d][4 * x], st.o[d][4 * x + 1], st.o[d][4 * x + 2], st.o[d][4 * x + 3], inv);
                        } else {
                            float* o = slot + row * S::DP + at_d;
                            put2(o, st.o[d][4 * x], st.o[d][4 * x + 1]);
                            put2(o + 2, st.o[d][4 * x + 2], st.o[d][4 * x + 3]);
                        }
                    }
                if (h == 0) {
                    if (!whole) put2(slot + S::M * S::DP + 2 * row, st.m, st.l);
                    else if (p.lse) put_lse(row, st.m, st.l);
                }
            }
        } else {
            // the waves' sums meet in LDS
            __syncthreads();
            if (h == 0) ml[wave * 32 + col] = st.m, ml[(S::W + wave) * 32 + col] = st.l;
            __syncthreads();
            float m = -INFINITY, l = 0.0f;
            for (int w = 0; w < S::W; ++w) m = fmaxf(m, ml[w * 32 + col]);
            const float ref = m == -INFINITY ? 0.0f : m;
            for (int w = 0; w < S::W; ++w) l += ml[(S::W + w) * 32 + col] * __builtin_amdgcn_exp2f(ml[w * 32 + col] - ref);
            const float keep = __builtin_amdgcn_exp2f(st.m - ref);
            float* buf = reinterpret_cast<float*>(lds) + wave * S::M * S::OS;
            if (live) {
#pragma unroll
                for (int d = 0; d < S::DB; ++d)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        float4 v = {st.o[d][4 * x] * keep, st.o[d][4 * x + 1] * keep, st.o[d][4 * x + 2] * keep, st.o[d][4 * x + 3] * keep};
                        *reinterpret_cast<float4*>(buf + col * S::OS + 32 * d + 8 * x + 4 * h) = v;
                    }
            }
            __syncthreads();
            if (wave == 0 && h == 0) ml[col] = m, ml[S::W * 32 + col] = l;
            if (wave == 0 && h == 0 && live) {
                if (!whole) put2(slot + S::M * S::DP + 2 * row, m, l);
                else if (p.lse) put_lse(row, m, l);
            }
            __syncthreads();
            const int quads = dim / 4;
            for (int i = threadIdx.x; i < rows * quads; i += S::THREADS) {
                const int rw = i / quads, d = (i % quads) * 4;
                const float* src = reinterpret_cast<const float*>(lds) + rw * S::OS + d;
                float4 a = *reinterpret_cast<const float4*>(src);
                for (int w = 1; w < S::W; ++w) {
                    const float4 v = *reinterpret_cast<const float4*>(src + w * S::M * S::OS);
                    a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
                }
                if (whole) {
                    put_out(rw, d, a.x, a.y, a.z, a.w, inverse(ml[S::W * 32 + rw]));
                } else {
                    put2(slot + rw * S::DP + d, a.x, a.y);
                    put2(slot + rw * S::DP + d + 2, a.z, a.w);
                }
            }
        }

        // The unit's parts, run by run.  Each part's share, exp2(its reference
        // less the largest), is worked out once a row, then every thread adds
        // up places of its own, eight parts' loads at a time.
        const auto join = [&](int64_t unit_start, int steps, int rows) {
            const int64_t wf = run_of(unit_start + S::EXTRA), wl = run_of(unit_start + S::EXTRA + steps - 1);
            const auto part = [&](int64_t w) { return slots + (w * 2 + (run_start(w) > unit_start ? 0 : 1)) * S::SLOT; };
            const int parts = int(wl - wf + 1), quads = dim / 4;
            for (int i = threadIdx.x; i < rows * quads; i += S::THREADS) {
                const int rw = i / quads, d = (i % quads) * 4;
                float m = -INFINITY, l = 0.0f, a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int x = 0; x < parts; x += 8) {
                    float pm[8], pl[8], v[8][4];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        // past the last part: the last again, with no share
                        const float* src = part(wf + min(x + e, parts - 1));
                        get2(src + S::M * S::DP + 2 * rw, &pm[e], &pl[e]);
                        get2(src + rw * S::DP + d, &v[e][0], &v[e][1]);
                        get2(src + rw * S::DP + d + 2, &v[e][2], &v[e][3]);
                    }
                    float mn = m;
#pragma unroll
                    for (int e = 0; e < 8; ++e) mn = fmaxf(mn, pm[e]);
                    const float ref = mn == -INFINITY ? 0.0f : mn, keep = __builtin_amdgcn_exp2f(m - ref);
                    m = mn;
                    l *= keep;
#pragma unroll
                    for (int j = 0; j < 4; ++j) a[j] *= keep;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (x + e >= parts) break;
                        const float share = __builtin_amdgcn_exp2f(pm[e] - ref);
                        l += pl[e] * share;
#pragma unroll
                        for (int j = 0; j < 4; ++j) a[j] += v[e][j] * share;
                    }
                }
                put_out(rw, d, a[0], a[1], a[2], a[3], inverse(l));
                if (d == 0 && p.lse) put_lse(rw, m, l);
            }
        };

        if (!whole) {
            // The partial stores have reached the device-wide level before
            // this work-group counts its steps; whoever completes the count
            // finds every part there.
            wait_loads<0>();
            __syncthreads();
            const int64_t unit_start = at - off;
            if (threadIdx.x == 0) {
                uint32_t* cnt = arrived + int64_t(kvh) * head_units + unit;
                const uint32_t old = __hip_atomic_fetch_add(cnt, uint32_t(count), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                const bool last = old + uint32_t(count) == uint32_t(steps);
                if (last) __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                plan[4] = last;
            }
            __syncthreads();
            if (plan[4]) {
                join(unit_start, steps, rows);
            }
        }

        __syncthreads();
        // the joining buffer wrote over the tiles' empty dimensions
        if (!S::SHARED) clear();
        advance(take);
    }
}

template <class S>
int64_t workers(int64_t tokens, int group, int kv_heads, int seqs, int64_t max_kv)
{
    const int64_t units = (tokens * group / S::M + seqs) * kv_heads;
    const int64_t steps = (max_kv + 15 + S::STEP - 1) / S::STEP + 1;
    const int64_t most = kComputeUnits * S::PER_CU, need = units * steps / S::LEAST + 1;
    return need < most ? (need + 7) / 8 * 8 : most;
}

template <class S>
int64_t unit_bound(int64_t tokens, int group, int kv_heads, int seqs)
{
    return (tokens * group / S::M + seqs) * kv_heads;
}

template <class S>
size_t bytes(int64_t tokens, int group, int kv_heads, int seqs, int64_t max_kv)
{
    const size_t head = (size_t(unit_bound<S>(tokens, group, kv_heads, seqs)) * 4 + 255) / 256 * 256;
    return head + size_t(workers<S>(tokens, group, kv_heads, seqs, max_kv)) * 2 * S::SLOT * 4;
}

template <class S>
hipError_t run(const AttnParams& p, hipStream_t s)
{
    const int64_t grid = workers<S>(p.tokens, p.group, p.cache.kv_heads, p.seqs, p.max_kv);
    const int64_t counters = unit_bound<S>(p.tokens, p.group, p.cache.kv_heads, p.seqs);
    static const hipError_t attr = [] {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(attention_kernel<S>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, S::LDS);
        if (e != hipSuccess) (void)hipGetLastError();
        return e;
    }();
    if (attr != hipSuccess && S::LDS > 64 * 1024) return attr;
    hipLaunchKernelGGL((attention_kernel<S>), dim3(unsigned(grid)), dim3(S::THREADS), S::LDS, s, p, counters);
    return hipGetLastError();
}

// Calls f with the shape for a cache and a bound on a sequence's rows.
template <class F>
auto with_shape(bool e4m3, int dim, bool shared, F f)
{
    const auto by_dim = [&](auto e, auto sh) {
        constexpr bool E = decltype(e)::value, SH = decltype(sh)::value;
        if (dim <= 64) return f(Shape<64, E, SH>());
        if (dim <= 96) return f(Shape<96, E, SH>());
        if (dim <= 128) return f(Shape<128, E, SH>());
        return f(Shape<256, E, SH>());
    };
    if (e4m3) return shared ? by_dim(std::true_type(), std::true_type()) : by_dim(std::true_type(), std::false_type());
    return shared ? by_dim(std::false_type(), std::true_type()) : by_dim(std::false_type(), std::false_type());
}

// Up to 32 rows a sequence and kv head stream the cache once either way.
bool is_shared(int64_t max_q, int group) { return max_q * group > 32; }

}  // namespace

size_t attention_workspace_bytes(bool e4m3, int64_t tokens, int q_heads, int kv_heads, int head_dim, int seqs,
                                 int64_t max_q, int64_t max_kv)
{
    const int group = q_heads / kv_heads;
    return with_shape(e4m3, head_dim, is_shared(max_q < tokens ? max_q : tokens, group), [&](auto shape) {
        return bytes<decltype(shape)>(tokens, group, kv_heads, seqs, max_kv);
    });
}

hipError_t launch_attention(const AttnParams& p, hipStream_t s)
{
    return with_shape(p.cache.e4m3, p.cache.head_dim, is_shared(p.max_q, p.group),
                      [&](auto shape) { return run<decltype(shape)>(p, s); });
}

}  // namespace qg
