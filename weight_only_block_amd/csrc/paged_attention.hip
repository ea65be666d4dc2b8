// Attention of a chunk of new tokens over the paged cache, on the matrix
// cores.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q . k_j - m)
//
// with m a running reference of the row's scores, raised (and the sums scaled
// down) only when a score passes it by 2^8: any reference gives the same
// quotient, and p up to 2^8 loses nothing in fp32 or bf16 (sums stay in range
// for values up to 2^120 / keys).
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
// Two shapes.  `Shared`: the work-group's four or eight waves hold 32 rows
// each and share key tiles of K and V in LDS, so a tile is read once for 128 or
// 256 rows; for prompts and chunks, bound by the matrix cores and the vector
// instructions of the softmax, which hardly overlap (busy 49% and 46% of the
// cycles of 4099 tokens over 12301 keys, 32 heads of 128: 649 to 690 us by the
// card's clock, 1.0 to 1.06 PFLOP/s where a large library product reaches 1.24;
// 722 us with e4m3 keys, whose fragments each wave converts for itself).  `Split`: the waves hold the
// same up to 32 rows and each streams key tiles of its own, joined in LDS at
// the end; for single and drafted tokens, bound by reading the cache (two
// sequences of 131072 bf16 keys, 1.07 GB: 174 us, 6.2 TB/s where a plain read
// reaches 6.8; 32 ragged ones, 215 MB: 44 us).
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
constexpr int kAhead = 4;                  // LDS reads ahead of their matrix products
constexpr float kRaise = 8.0f;             // log2 by which a score may pass the reference
constexpr int kListPages = 1024;           // page ids of a run's segment, in LDS
constexpr int kListSeqs = 128;             // sequences whose lengths are kept in LDS
constexpr int kComputeUnits = 256;
// Rows a sequence (tokens x group) from which eight waves share tiles in place
// of four: 256 rows to a tile halve its reads, but a unit's beginning and end
// cost more.  4099 tokens over 12301 keys (16396 rows): 735 us with four, 655
// with eight; 2048 over 8192: 262 and 250; 512 over 8192: 91 both; 128 over
// 4096: 39 and 46.
constexpr int64_t kManyRows = 2048;
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

__device__ __forceinline__ uint32_t lds_offset(const void* p)
{
    return uint32_t(uintptr_t((__attribute__((address_space(3))) const char*)p));
}

// 16 bytes per lane from global memory to LDS at lds + 16 * lane, with no
// register between.  The compiler does not count these loads: every use waits
// by hand (wait_loads).
// ONCE: what no other work-group reads, which need not stay in the caches.
template <bool ONCE>
__device__ __forceinline__ void load_lds_uniform(uint32_t lds, uint64_t base, uint32_t offset)
{
    if (ONCE)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(lds), "v"(offset), "s"(base)
                     : "memory");
    else
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

// x / group, exact while x * group is below 2^31: x is a row of a unit beside
// the heads before its first, below 255 + group, and group below 2^15.
__device__ __forceinline__ uint32_t by_group(const Args& p, uint32_t x) { return __umulhi(2 * x, p.by_group); }

// One kernel shape.  DP: head dimension padded to a matrix-core multiple;
// FULL: the head has all of it; SHARING: waves that share tiles, 0 for Split.
template <int DP_, bool E4M3_, int SHARING, bool FULL_>
struct Shape {
    static constexpr int DP = DP_;
    static constexpr bool E4M3 = E4M3_, SHARED = SHARING != 0, FULL = FULL_;
    static constexpr int ES = E4M3 ? 1 : 2;
    static constexpr int RB = (DP == 96 ? 128 : DP) * ES;               // bytes of a tile row
    // Waves.  Split: as many as leave a compute unit two work-groups or more,
    // so that one streams while another begins or ends a unit; with rows of 128
    // bytes that is four, and half as many parts to join as with two (one
    // sequence of 32768 e4m3 keys: 30 us with two, 25 with four).
    static constexpr int W = SHARED ? SHARING : RB <= 128 ? 4 : DP == 256 && !E4M3 ? 1 : 2;
    static constexpr int THREADS = 64 * W;
    static constexpr int WAVES_PER_SIMD = DP <= 128 ? 2 : 1;
    static constexpr int M = SHARED ? 32 * W : 32;                      // rows of a unit
    static constexpr int KT = SHARED && DP <= 128 ? 64 : 32;            // keys of a wave's tile
    static constexpr int BLOCKS = KT / 32;
    static constexpr int STEP = SHARED ? KT : KT * W;                   // keys of a work-group's step
    static constexpr int CPR = RB / 16;                                 // 16-byte chunks of it
    static constexpr int RPI = 64 / CPR;                                // rows of one load instruction
    static constexpr int TILE = KT * RB;                                // bytes of K or of V
    static constexpr int RAW = SHARED ? KT / W : KT, ROWS = RAW < RPI ? RPI : RAW;   // rows a wave loads
    // tiles in LDS: two where two work-groups share a compute unit
    static constexpr int STAGES = SHARED && (W == 8 || WAVES_PER_SIMD == 1) ? 4 : 2;
    static constexpr int LOADS = ROWS / RPI;                            // for K, and as many for V
    static constexpr int RING = STAGES * 2 * TILE * (SHARED ? 1 : W);   // stages of K and V
    static constexpr int OS = DP + 4;                                   // floats of a row in the joining buffer
    static constexpr int JOIN = SHARED ? 0 : W * M * OS * 4;
    static constexpr int BUFFER = RING > JOIN ? RING : JOIN;
    static constexpr int LDS = BUFFER + kListPages * 4 + 2 * W * 32 * 4 + 64 + kListSeqs * 12;
    // work-groups that a compute unit holds (160 KB of LDS, two waves of up to
    // 256 registers a SIMD or one of 512)
    static constexpr int BY_LDS = 160 * 1024 / LDS, BY_WAVES = 4 * WAVES_PER_SIMD / W;
    static constexpr int PER_CU = BY_LDS < BY_WAVES ? BY_LDS : BY_WAVES;
    // Steps that a run has at least: a shorter one costs more in joining its
    // part than it saves.  What beginning and ending a unit costs, in steps.
    static constexpr int LEAST = SHARED ? 4 : 2;
    static constexpr int EXTRA = SHARED ? 5 : 3;
    static constexpr float JOINED = SHARED ? 1.0f : 0.25f;               // what joining a part costs
    static constexpr int SLOT = SHARED ? W * (DP * 32 + 128) : M * DP + 2 * M;   // floats of a partial result
    static constexpr int STEPS = DP / 16;                               // products along the dimension
    static constexpr int DB = DP / 32;

    // Swizzles: the chunk of a row's 16 bytes is moved so that what 32 lanes of
    // an LDS access read lies in different banks: 16 rows of one chunk (K), or
    // of two halves of 32 dimensions four rows of 32 bytes or eight of 16 (V).
    static __device__ __forceinline__ int k_swizzle(int row)
    {
        return CPR == 4 ? (row >> 2) & 3 : CPR == 8 ? (row >> 1) & 7 : row & 15;
    }
    static __device__ __forceinline__ int v_swizzle(int row)
    {
        if (!E4M3) return CPR == 8 ? ((row >> 1) & 1) << 2 : (row & 3) << 2;
        return CPR == 4 ? ((row >> 3) & 1) << 1 : CPR == 8 ? (row & 2) | ((row >> 3) & 1) << 2
                                                          : (row & 3) << 1 | ((row >> 3) & 1) << 3;
    }
};

__device__ __forceinline__ Seq load_seq(const Args& p, int b)
{
    return cut_seq(p.q_start[b], p.q_start[b + 1], p.kv_len[b], p.tokens, p.max_q, p.cap);
}

// From LDS where all sequences fit.
__device__ __forceinline__ Seq get_seq(const Args& p, const Seq* seqs, int b)
{
    return p.seqs <= kListSeqs ? seqs[b] : load_seq(p, b);
}

// A unit: rows [row0, row0 + rows) of a sequence's tokens x group.
struct Unit {
    int rows, token0, lane0;   // token and head of its first row
    int first, last;           // positions of the first and last row's tokens
    int lo, hi, base;          // keys [lo, hi) that some row sees; the first tile starts at base
    int steps;
};

template <class S>
__device__ __forceinline__ Unit make_unit(const Args& p, const Seq& s, int tile)
{
    Unit u;
    const uint32_t row0 = uint32_t(tile) * S::M;
    u.rows = int(min(uint32_t(S::M), uint32_t(s.n) * uint32_t(p.group) - row0));
    u.token0 = int(row0 / uint32_t(p.group));
    u.lane0 = int(row0 - uint32_t(u.token0) * uint32_t(p.group));
    u.first = s.kv - s.n + u.token0;
    u.last = u.first + int(by_group(p, uint32_t(u.lane0 + u.rows - 1)));
    u.hi = max(0, u.last + 1);
    u.lo = p.window > 0 ? max(0, u.first - p.window + 1) : 0;
    if (u.lo > u.hi) u.lo = u.hi;
    u.base = u.lo & ~15;
    // a unit without keys still writes its rows
    u.steps = u.hi > u.lo ? int(uint32_t(u.hi - u.base + S::STEP - 1) / S::STEP) : 1;
    return u;
}

template <class S>
__device__ __forceinline__ int seq_tiles(const Args& p, const Seq& s)
{
    return int((uint32_t(s.n) * uint32_t(p.group) + S::M - 1) / S::M);
}

// What a wave accumulates: its 32 rows are the lanes' columns.
template <class S>
struct State {
    f32x16 o[S::DB];
    bf16x8 q[S::STEPS];
    float m, l;          // reference; this half's share of the sum
    int rlo, rhi;        // keys the lane's row sees
};

template <class S>
struct Scores {
    f32x16 s[S::BLOCKS];
};
template <class S>
struct Probs {
    u32x4 p[2 * S::BLOCKS];   // bf16, as the second product takes them
};

// Scores of a key tile (32 or 64 keys) for the wave's rows.
template <class S>
__device__ __forceinline__ void scores(const State<S>& st, Scores<S>& sc, const uint8_t* kt, int lane)
{
    const int col = lane & 31, h = lane >> 5;
#pragma unroll
    for (int b = 0; b < S::BLOCKS; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) sc.s[b][i] = 0.0f;
    const int ksw = S::k_swizzle(col);
    const uint8_t* row = kt + col * S::RB;
    // Blocks alternate, so that a product does not wait on the one before it.
    // Reads run kAhead products ahead: left to itself the compiler puts each
    // next to its product, which then waits for it.
    constexpr int READS = S::E4M3 ? S::STEPS / 2 * S::BLOCKS : S::STEPS * S::BLOCKS;
    u32x4 f[READS];
    const auto read = [&](int i) {
        const int t = i / S::BLOCKS, b = i % S::BLOCKS;
        f[i] = *reinterpret_cast<const u32x4*>(row + b * 32 * S::RB + (((2 * t + h) ^ ksw) << 4));
    };
#pragma unroll
    for (int i = 0; i < (kAhead < READS ? kAhead : READS); ++i) read(i);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < READS; ++i) {
        const int t = i / S::BLOCKS, b = i % S::BLOCKS;
        if (i + kAhead < READS) read(i + kAhead);
        if (!S::E4M3) {
            sc.s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, f[i]), st.q[t], sc.s[b], 0, 0, 0);
        } else {
            // one 16-byte read is two steps: step 2 t + e takes dimensions 32 t + 16 h + 8 e on
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                union { bf16x8 v; bf16x2 p[4]; } a;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    a.p[2 * x] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[i][2 * e + x], 1.0f, false);
                    a.p[2 * x + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[i][2 * e + x], 1.0f, true);
                }
                sc.s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, st.q[2 * t + e], sc.s[b], 0, 0, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Keys from k0 that the lane's row does not see.
template <class S>
__device__ __forceinline__ void mask(const State<S>& st, Scores<S>& sc, int k0, int lane)
{
    const uint32_t width = uint32_t(st.rhi - st.rlo);
    const int first = k0 + 4 * (lane >> 5) - st.rlo;
#pragma unroll
    for (int b = 0; b < S::BLOCKS; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (uint32_t(first + 32 * b + 8 * (i / 4) + i % 4) >= width) sc.s[b][i] = -INFINITY;
}

// The largest score of the lane's half of the row.
template <class S>
__device__ __forceinline__ float largest(const Scores<S>& sc)
{
    float top = sc.s[0][0];
#pragma unroll
    for (int b = 0; b < S::BLOCKS; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, sc.s[b][i]);
    return top;
}

// Raises the row's reference where a score passes it by too much.
template <class S>
__device__ __forceinline__ void raise(State<S>& st, float top, float c)
{
    top = max_halves(top) * c;
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
}

// Probabilities, which become bf16 for the matrix cores (each off by at most
// half a step, 2^-8 of it; over many keys the errors cancel), and their sum,
// which takes them unrounded.
template <class S>
__device__ __forceinline__ void probs(State<S>& st, const Scores<S>& sc, Probs<S>& pb, float c)
{
    const float ref = st.m == -INFINITY ? 0.0f : st.m;
    float sum = 0.0f;
#pragma unroll
    for (int b = 0; b < S::BLOCKS; ++b)
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc.s[b][2 * x], c, -ref));
            const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc.s[b][2 * x + 1], c, -ref));
            sum += p0;
            sum += p1;
            pb.p[2 * b + x / 4][x % 4] = pack_bf16(p0, p1);
        }
    st.l += sum;
}

// A tile's values as the second product takes them: fragment i is 16 keys
// (i / DB) by 32 dimensions (i % DB).
template <class S>
struct Values {
    static constexpr int COUNT = 2 * S::BLOCKS * S::DB;
    s16x4 f[COUNT][2];
    const uint8_t* vt;
    int row, chunk, half;

    __device__ __forceinline__ Values(const uint8_t* tile, int lane) : vt(tile)
    {
        const int h = lane >> 5, i16 = lane & 15, dh = (lane >> 4) & 1, rr = i16 / 2;
        row = S::E4M3 ? 8 * (rr / 4) + 4 * h + rr % 4 : 4 * h + i16 / 4;
        chunk = (S::E4M3 ? dh : 2 * dh + (i16 & 3) / 2) ^ S::v_swizzle(row);
        half = (i16 & 1) * 8;
    }
    __device__ __forceinline__ void read(int i)
    {
        const int kb = i / S::DB, d = i % S::DB;
        // (16 keys on have the same swizzle)
        const uint8_t* at = vt + (16 * kb + row) * S::RB + ((chunk ^ (S::E4M3 ? 2 * d : 4 * d)) << 4) + half;
        if (!S::E4M3) {
            f[i][0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
            f[i][1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 8 * S::RB));
        } else {
            f[i][0] = __builtin_bit_cast(s16x4, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)at));
        }
    }
    __device__ __forceinline__ void begin()
    {
#pragma unroll
        for (int i = 0; i < (kAhead < COUNT ? kAhead : COUNT); ++i) read(i);
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ bf16x8 value(int i) const
    {
        union { bf16x8 v; s16x4 h[2]; bf16x2 p[4]; } a;
        if (!S::E4M3) {
            a.h[0] = f[i][0];
            a.h[1] = f[i][1];
        } else {
            const i32x2 raw = __builtin_bit_cast(i32x2, f[i][0]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                a.p[2 * x] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[x], 1.0f, false);
                a.p[2 * x + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[x], 1.0f, true);
            }
        }
        return a.v;
    }
};

// Adds the tile's values, weighed by the probabilities; the first reads have
// begun.
template <class S>
__device__ __forceinline__ void output(State<S>& st, const Probs<S>& pb, Values<S>& v)
{
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < Values<S>::COUNT; ++i) {
        if (i + kAhead < Values<S>::COUNT) v.read(i + kAhead);
        st.o[i % S::DB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v.value(i), __builtin_bit_cast(bf16x8, pb.p[i / S::DB]),
                                                                 st.o[i % S::DB], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// A key tile (K and V, 32 or 64 keys from k0) against the wave's rows.
// `masked`: some row does not see some key.
template <class S>
__device__ __forceinline__ void compute(State<S>& st, const uint8_t* kt, const uint8_t* vt, int k0, float c, bool masked,
                                        int lane)
{
    Scores<S> sc;
    Probs<S> pb;
    scores<S>(st, sc, kt, lane);
    Values<S> v(vt, lane);
    v.begin();
    if (masked) mask<S>(st, sc, k0, lane);
    raise<S>(st, largest<S>(sc), c);
    probs<S>(st, sc, pb, c);
    output<S>(st, pb, v);
}

// The loads of one tile, and what the tile needs before use.
template <class S>
struct Loader {
    const Args& p;
    const int32_t* list;      // LDS: page ids from page `first_page` on, -1 outside the sequence or the cache
    int first_page;
    const int32_t* table;     // the sequence's row of the page table
    int pages;                // of the sequence
    uint64_t kbase, vbase;    // of this kv head
    int lo, hi;               // keys that some row of the unit sees
    int all_lo, all_hi;       // and that every row sees
    int64_t* poisoned;        // LDS
    int lane;

    // Rows [row0, row0 + ROWS) of the tile, the wave's part; its K and V at
    // LDS offsets kt and vt, its first key k0.  True: it needs patch().
    __device__ __forceinline__ bool issue(uint32_t kt, uint32_t vt, int k0, int row0) const
    {
        const int lr = lane / S::CPR, lc = lane % S::CPR;
        const int chunks = S::FULL ? S::CPR : p.dim * S::ES / 16;
        const int mask = (1 << p.page_shift) - 1;
        bool dirty = k0 + row0 < all_lo || k0 + row0 + S::ROWS > all_hi;
        kt += row0 * S::RB;
        vt += row0 * S::RB;
        if (p.page_shift >= 4 && p.slot16 < (1u << 20)) {
            // all rows of one load lie in one page; lane j looks up load j's
            const int mine = list[((k0 + row0 + min(lane, S::LOADS - 1) * S::RPI) >> p.page_shift) - first_page];
            if (__any(mine < 0)) dirty = true;
            const uint32_t row_off = uint32_t(lr) * (p.slot16 * 16);
#pragma unroll
            for (int j = 0; j < S::LOADS; ++j) {
                const uint32_t id = uint32_t(max(0, __builtin_amdgcn_readlane(mine, j)));
                const uint32_t slot = uint32_t((k0 + row0 + j * S::RPI) & mask);
                const uint64_t off = (uint64_t(id) * p.page16 + uint64_t(slot) * p.slot16) << 4;
                const int ck = lc ^ S::k_swizzle(row0 + j * S::RPI + lr), cv = lc ^ S::v_swizzle(row0 + j * S::RPI + lr);
                if (S::FULL || ck < chunks) load_lds_uniform<!S::SHARED>(kt + j * 1024, kbase + off, row_off + 16 * ck);
                if (S::FULL || cv < chunks) load_lds_uniform<!S::SHARED>(vt + j * 1024, vbase + off, row_off + 16 * cv);
            }
        } else {
#pragma unroll 1
            for (int j = 0; j < S::LOADS; ++j) {
                const int row = row0 + j * S::RPI + lr, key = k0 + row;
                int id = list[(key >> p.page_shift) - first_page];
                if (__any(id < 0)) dirty = true;
                id = max(0, id);
                const uint64_t off = (uint64_t(uint32_t(id)) * p.page16 + uint64_t(uint32_t(key & mask)) * p.slot16) << 4;
                const int ck = lc ^ S::k_swizzle(row), cv = lc ^ S::v_swizzle(row);
                if (S::FULL || ck < chunks) load_lds(kt + j * 1024, kbase + off + 16 * ck);
                if (S::FULL || cv < chunks) load_lds(vt + j * 1024, vbase + off + 16 * cv);
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
        const int lane = opaque(this->lane), lr = lane / S::CPR, lc = lane % S::CPR;
        const int chunks = S::FULL ? S::CPR : p.dim * S::ES / 16;   // those past the dimension stay zero
        const uint32_t nan = S::E4M3 ? 0x7f7f7f7fu : 0x7fc07fc0u;
#pragma unroll 1
        for (int j = 0; j < S::LOADS; ++j) {
            const int row = row0 + j * S::RPI + lr, key = k0 + row;
            const bool outside = key < lo || key >= hi;
            const int page = key >> p.page_shift;
            int id = -1;
            if (!outside && page < pages) id = table[page];
            const bool lost = !outside && (id < 0 || id >= p.pages);
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

// Gives the lane's row the values that patch() took out, of keys [from, to),
// each times its probability: infinity stays one, but for a probability of
// zero, as in a tile that all rows see.  Split: a key is its own wave's alone;
// tiles begin at `from`.
template <class S>
__device__ __forceinline__ void restore(State<S>& st, const Args& p, const Loader<S>& ld, int from, int to, float c, int wave)
{
    const int mask = (1 << p.page_shift) - 1;
    const float ref = st.m == -INFINITY ? 0.0f : st.m;
#pragma unroll 1
    for (int key = max(from, ld.lo); key < min(to, ld.hi); ++key) {
        if (key >= ld.all_lo && key < ld.all_hi) continue;
        if (!S::SHARED && (key - from) / S::KT % S::W != wave) continue;
        const int id = ld.table[key >> p.page_shift];
        if (id < 0 || id >= p.pages) continue;
        const uint64_t off = (uint64_t(uint32_t(id)) * p.page16 + uint64_t(uint32_t(key & mask)) * p.slot16) << 4;
        const uint8_t* krow = reinterpret_cast<const uint8_t*>(ld.kbase + off);
        const uint8_t* vrow = reinterpret_cast<const uint8_t*>(ld.vbase + off);
        const int h = opaque(threadIdx.x & 63) >> 5;     // (here: offsets of all dimensions take no registers around the loop)
        const auto value = [&](const uint8_t* row, int dim) {
            return S::E4M3 ? __builtin_amdgcn_cvt_f32_fp8(int(row[dim]), 0)
                           : __uint_as_float(uint32_t(reinterpret_cast<const uint16_t*>(row)[dim]) << 16);
        };
        float score = 0.0f;
#pragma unroll
        for (int t = 0; t < S::STEPS; ++t) {
            const int d = S::E4M3 ? 32 * (t / 2) + 16 * h + 8 * (t % 2) : 16 * t + 8 * h;
            if (S::FULL || d < p.dim) {
#pragma unroll
                for (int e = 0; e < 8; ++e) score = __builtin_fmaf(float(st.q[t][e]), value(krow, d + e), score);
            }
            asm volatile("" ::: "memory");       // few loads, and registers for them, at a time
            __builtin_amdgcn_sched_barrier(0);
        }
        const float pr = __builtin_amdgcn_exp2f(__builtin_fmaf(sum_halves(score), c, -ref));
        const bool sees = key >= st.rlo && key < st.rhi;
#pragma unroll
        for (int d = 0; d < S::DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (!S::FULL && 32 * d + 16 * (i / 8) >= p.dim) continue;    // (whole sixteens)
                const float v = value(vrow, 32 * d + 8 * (i / 4) + 4 * h + i % 4);
                if (sees && !(fabsf(v) < INFINITY)) st.o[d][i] += pr * v;
                if (i % 4 == 3) {
                    asm volatile("" ::: "memory");
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
    }
}

template <class S>
__global__ __launch_bounds__(S::THREADS, S::WAVES_PER_SIMD) void attention_kernel(Args p)
{
    extern __shared__ __align__(1024) uint8_t lds[];
    int32_t* list = reinterpret_cast<int32_t*>(lds + S::BUFFER);
    float* ml = reinterpret_cast<float*>(list + kListPages);      // [2][W][32]
    int64_t* plan = reinterpret_cast<int64_t*>(ml + 2 * S::W * 32);   // 8 values
    Seq* seqs = reinterpret_cast<Seq*>(plan + 8);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    fetch_arguments<sizeof(Args)>();

    // ---- the line of work: this run's part of it.  Each thread sums a run of
    // units: those of some sequences, or where sequences have many tiles and
    // fit the list, its share of all units.
    int b0, t0 = 0, mine_units = 0;
    if (S::SHARED && p.seqs <= kListSeqs) {
        for (int b = threadIdx.x; b < p.seqs; b += S::THREADS) seqs[b] = load_seq(p, b);
        __syncthreads();
        int units = 0;
        for (int b = 0; b < p.seqs; ++b) units += seq_tiles<S>(p, seqs[b]);
        const int per = (units + S::THREADS - 1) / S::THREADS, u0 = min(int(threadIdx.x) * per, units);
        mine_units = min(per, units - u0);
        int before = 0;
        for (b0 = 0; b0 < p.seqs; ++b0) {
            const int tiles = seq_tiles<S>(p, seqs[b0]);
            if (u0 < before + tiles) break;
            before += tiles;
        }
        t0 = u0 - before;
    } else {
        const int per = (p.seqs + S::THREADS - 1) / S::THREADS;
        b0 = min(int(threadIdx.x) * per, p.seqs);
        for (int b = b0; b < min(b0 + per, p.seqs); ++b) {
            const Seq s = load_seq(p, b);
            if (p.seqs <= kListSeqs) seqs[b] = s;
            mine_units += seq_tiles<S>(p, s);
        }
    }
    // The units of this thread one after another, until `f` says so.
    const auto walk = [&](auto f) {
        int b = b0, t = t0;
        for (int k = 0; k < mine_units; ++k) {
            Seq s = get_seq(p, seqs, b);
            while (t >= seq_tiles<S>(p, s)) {
                t = 0;
                s = get_seq(p, seqs, ++b);
            }
            if (f(b, t, make_unit<S>(p, s, t).steps + S::EXTRA)) break;
            ++t;
        }
    };
    int64_t mine = 0;
    int longest = 0;
    walk([&](int, int, int cost) {
        mine += cost;
        longest = max(longest, cost);
        return false;
    });
    int64_t upto = mine;
    for (int off = 1; off < 64; off <<= 1) {
        const int64_t a = __shfl_up((long long)upto, off, 64);
        if (lane >= off) upto += a;
        longest = max(longest, __shfl_xor(longest, off, 64));
    }
    int64_t* sums = reinterpret_cast<int64_t*>(lds);              // [W] each: steps, longest unit
    if (lane == 63) sums[wave] = upto, sums[S::W + wave] = longest;
    __syncthreads();
    int64_t head_steps = 0, before = 0;
#pragma unroll
    for (int w = 0; w < S::W; ++w) {
        if (w == wave) before = head_steps;
        head_steps += sums[w];
        longest = max(longest, int(sums[S::W + w]));
    }
    upto += before;
    head_steps = uniform(head_steps);
    const int64_t total = head_steps * p.kv_heads;
    if (total == 0) return;
    // A unit of n steps in runs of x takes about x + JOINED n / x steps: no
    // shorter runs than where that is least, and no more runs than work-groups.
    const float least = fmaxf(float(S::LEAST), __builtin_amdgcn_sqrtf(float(longest) * S::JOINED));
    const int runs = __builtin_amdgcn_readfirstlane(int(fmaxf(1.0f, fminf(float(gridDim.x), float(total) / least))));
    // consecutive work-groups go to different XCDs: give each XCD one stretch
    // of the line, so that its L2 holds few heads' keys; few go over all XCDs
    const int xcds = gridDim.x % 8 == 0 ? 8 : 1;
    const int run = runs < int(gridDim.x) ? int(blockIdx.x) : int(blockIdx.x % xcds) * int(gridDim.x / xcds) + int(blockIdx.x / xcds);
    if (run >= runs) return;
    // the first `longer` runs have base + 1 steps, the others base
    const int64_t base = uniform(divide(total, runs));
    const int longer = int(total - base * runs);
    const auto run_start = [&](int w) { return w * base + min(w, longer); };
    const auto run_of = [&](int64_t x) {
        const int64_t split = longer * (base + 1);
        return int(x < split ? divide(x, base + 1) : longer + divide(x - split, base));
    };
    int64_t at = run_start(run);
    const int64_t end = run_start(run + 1);
    int kvh = int(uniform(divide(at, head_steps)));
    {
        const int64_t r = at - kvh * head_steps;
        if (r >= upto - mine && r < upto) {
            int64_t left = r - (upto - mine);
            walk([&](int b, int t, int cost) {
                if (left < cost) {
                    plan[0] = b, plan[1] = t, plan[2] = left;
                    return true;
                }
                left -= cost;
                return false;
            });
        }
    }
    __syncthreads();
    int b = __builtin_amdgcn_readfirstlane(int(plan[0])), tile = __builtin_amdgcn_readfirstlane(int(plan[1]));
    int off = __builtin_amdgcn_readfirstlane(int(plan[2]));
    Seq s = get_seq(p, seqs, b);

    // dimensions past the head's end stay zero in every tile
    const auto clear = [&] {
        if (!S::FULL)
            for (int i = threadIdx.x; i < S::BUFFER / 16; i += S::THREADS) reinterpret_cast<u32x4*>(lds)[i] = u32x4{0, 0, 0, 0};
    };
    clear();

    // Goes on to the next unit of the line.
    const auto advance = [&](int cost) {
        at += cost;
        off = 0;
        if (at >= end) return;
        ++tile;
        while (tile >= seq_tiles<S>(p, s)) {
            tile = 0;
            if (++b == p.seqs) b = 0, ++kvh;
            s = get_seq(p, seqs, b);
        }
    };

    const uint32_t lds0 = lds_offset(lds);
    while (at < end) {
        s.q0 = __builtin_amdgcn_readfirstlane(s.q0);
        s.n = __builtin_amdgcn_readfirstlane(s.n);
        s.kv = __builtin_amdgcn_readfirstlane(s.kv);
        const Unit u = make_unit<S>(p, s, tile);
        const int take = int(min(int64_t(u.steps + S::EXTRA - off), end - at));
        const int from = max(0, off - S::EXTRA), count = max(0, off + take - S::EXTRA) - from;
        if (count == 0) {       // only what stands for the unit's beginning
            advance(take);
            continue;
        }
        const float ks = S::E4M3 ? p.k_scale[kvh] : 1.0f;

        // ---- the wave's rows
        const int ulane = opaque(lane), col = ulane & 31, h = ulane >> 5;
        State<S> st;
        const int row = S::SHARED ? wave * 32 + col : col;
        // rows past the last repeat it and are never written
        const uint32_t r = uint32_t(u.lane0 + min(row, u.rows - 1)), step = by_group(p, r);
        const uint32_t head = uint32_t(kvh) * uint32_t(p.group) + (r - step * uint32_t(p.group));
        const uint16_t* qrow = p.q + uint64_t(uint32_t(s.q0 + u.token0) + step) * p.q_token + uint64_t(head) * p.q_head;
        const int pos = u.first + int(step);
        st.rhi = max(0, pos + 1);
        st.rlo = p.window > 0 ? min(st.rhi, max(0, pos - p.window + 1)) : 0;
        st.m = -INFINITY;
        st.l = 0.0f;
#pragma unroll
        for (int t = 0; t < S::STEPS; ++t) {
            const int d = S::E4M3 ? 32 * (t / 2) + 16 * h + 8 * (t % 2) : 16 * t + 8 * h;
            u32x4 x = {0, 0, 0, 0};
            if (S::FULL || d < p.dim) x = *reinterpret_cast<const u32x4*>(qrow + d);
            st.q[t] = __builtin_bit_cast(bf16x8, x);
        }
#pragma unroll
        for (int d = 0; d < S::DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) st.o[d][i] = 0.0f;
        // keys that every row of this wave sees, and that any does
        const int wr0 = S::SHARED ? wave * 32 : 0;
        const bool busy = wr0 < u.rows;
        int all_lo = 0, all_hi = 0, any_lo = 0, any_hi = 0;
        if (busy) {
            const int wr1 = min(wr0 + 32, u.rows) - 1;
            const int f = u.first + int(by_group(p, uint32_t(u.lane0 + wr0)));
            const int l = u.first + int(by_group(p, uint32_t(u.lane0 + wr1)));
            all_hi = f + 1;
            any_hi = max(0, l + 1);
            if (p.window > 0) {
                all_lo = max(0, l - p.window + 1);
                any_lo = max(0, f - p.window + 1);
            }
        }

        Loader<S> ld{p, list, 0, p.table + uint64_t(uint32_t(b)) * p.table_stride, 0, 0, 0, u.lo, u.hi, 0, u.first + 1, plan + 5, ulane};
        if (p.window > 0) ld.all_lo = max(0, u.last - p.window + 1);
        ld.pages = int((uint32_t(s.kv) + (1u << p.page_shift) - 1) >> p.page_shift);
        const uint64_t head_bytes = uint64_t(uniform(int64_t(uint64_t(uint32_t(kvh)) * p.head16 << 4)));
        ld.kbase = reinterpret_cast<uint64_t>(p.k) + head_bytes;
        ld.vbase = reinterpret_cast<uint64_t>(p.v) + head_bytes;
        if (threadIdx.x == 0) plan[5] = 0;

        // The scale's sign goes into the queries, so that the largest score
        // stays the largest; a scale of zero becomes one that leaves scores
        // equal.
        float c = p.scale * ks * kLog2e;
        if (c < 0.0f) {
            c = -c;
#pragma unroll
            for (int t = 0; t < S::STEPS; ++t) st.q[t] = __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, st.q[t]) ^ 0x80008000u);
        }
        if (c < 1e-37f) c = 1e-37f;

        const auto run_tile = [&](uint32_t at_lds, int k0) {
            if (!busy || k0 >= any_hi || k0 + S::KT <= any_lo) return;
            const uint8_t* kt = lds + (at_lds - lds0);
            compute<S>(st, kt, kt + S::TILE, k0, c, k0 < all_lo || k0 + S::KT > all_hi, ulane);
        };

        // ---- segments of the run whose page ids fit the list
        for (int done = 0; done < count && u.hi > u.lo;) {
            const int start = __builtin_amdgcn_readfirstlane(u.base + (from + done) * S::STEP);
            ld.first_page = start >> p.page_shift;
            // steps whose last key's page is in the list
            const int64_t span = (int64_t(ld.first_page + kListPages) << p.page_shift) - start;
            const int n = int(min(int64_t(count - done), span / S::STEP));
            const int want = int((uint32_t(start + n * S::STEP - 1) >> p.page_shift) - ld.first_page + 1);
            __syncthreads();
            for (int i = threadIdx.x; i < want; i += S::THREADS) {
                int id = -1;
                if (ld.first_page + i < ld.pages) id = ld.table[ld.first_page + i];
                list[i] = id >= p.pages ? -1 : id;
            }
            __syncthreads();
            if constexpr (S::SHARED) {
                const int row0 = wave * S::ROWS;
                const bool loads = row0 < S::KT;
                uint32_t flags = 0;
                const auto fetch = [&](int i) {
                    const uint32_t to = lds0 + (i % S::STAGES) * 2 * S::TILE;
                    if (loads && ld.issue(to, to + S::TILE, start + i * S::STEP, row0)) flags |= 1u << (i % S::STAGES);
                };
                for (int i = 0; i < min(n, S::STAGES - 1); ++i) fetch(i);
                for (int i = 0; i < n; ++i) {
                    const uint32_t kt = lds0 + (i % S::STAGES) * 2 * S::TILE;
                    const int k0 = start + i * S::STEP;
                    if (i + S::STAGES - 2 < n) wait_loads<(S::STAGES - 2) * 2 * S::LOADS>();
                    else wait_loads<0>();
                    if (flags >> (i % S::STAGES) & 1) {
                        ld.patch(lds + (kt - lds0), lds + (kt - lds0) + S::TILE, k0, row0);
                        flags &= ~(1u << (i % S::STAGES));
                    }
                    wait_lds();
                    __builtin_amdgcn_s_barrier();
                    asm volatile("" ::: "memory");
                    if (i + S::STAGES - 1 < n) fetch(i + S::STAGES - 1);
                    run_tile(kt, k0);
                }
            } else {
                bool dirty = false, next = false;
                const uint32_t ring = lds0 + wave * 4 * S::TILE;
                const int k1 = start + wave * S::KT;
                for (int i = -1; i < n; ++i) {
                    const uint32_t kt = ring + (i & 1) * 2 * S::TILE;
                    const int k0 = k1 + i * S::STEP;
                    if (i + 1 < n) {
                        const uint32_t nt = ring + ((i + 1) & 1) * 2 * S::TILE;
                        wait_lds();
                        next = ld.issue(nt, nt + S::TILE, k0 + S::STEP, 0);
                    }
                    if (i >= 0) {
                        if (i + 1 < n) wait_loads<2 * S::LOADS>();
                        else wait_loads<0>();
                        if (dirty) ld.patch(lds + (kt - lds0), lds + (kt - lds0) + S::TILE, k0, 0);
                        run_tile(kt, k0);
                    }
                    dirty = next;
                }
            }
            done += n;
        }
        st.l = sum_halves(st.l);
        __syncthreads();
        if (plan[5]) restore(st, p, ld, u.base + from * S::STEP, u.base + (from + count) * S::STEP, c, wave);

        // ---- results: whole units to the output, parts to the workspace
        const bool whole = count == u.steps;
        const int tid = opaque(threadIdx.x), lane2 = tid & 63, col2 = lane2 & 31, h2 = lane2 >> 5;
        const float vs = S::E4M3 ? p.v_scale[kvh] : 1.0f;
        float* slots = reinterpret_cast<float*>(p.workspace + kCounterBytes);
        float* slot = slots + uint64_t(run * 2 + (off > 0 ? 0 : 1)) * S::SLOT;
        const auto put_out = [&](int row, int d, float a0, float a1, float a2, float a3, float inv) {
            const uint32_t r = uint32_t(u.lane0 + row), step = by_group(p, r);
            const uint32_t head = uint32_t(kvh) * uint32_t(p.group) + (r - step * uint32_t(p.group));
            uint16_t* o = p.out + uint64_t(uint32_t(s.q0 + u.token0) + step) * p.o_token + uint64_t(head) * p.o_head + d;
            *reinterpret_cast<u32x2*>(o) = u32x2{pack_bf16(a0 * inv, a1 * inv), pack_bf16(a2 * inv, a3 * inv)};
        };
        const auto put_lse = [&](int row, float m, float l) {
            const uint32_t r = uint32_t(u.lane0 + row), step = by_group(p, r);
            const uint32_t head = uint32_t(kvh) * uint32_t(p.group) + (r - step * uint32_t(p.group));
            p.lse[uint64_t(uint32_t(s.q0 + u.token0) + step) * p.lse_token + head] =
                m == -INFINITY && l == 0.0f ? -INFINITY : (m + __log2f(l)) * kLn2;
        };
        // rows that see nothing have l = 0 and o = 0
        const auto inverse = [&](float l) { return l == 0.0f ? 0.0f : vs / l; };
        // A part of a Shared unit is what the waves' lanes hold, register pair
        // by register pair, so that its stores and loads are contiguous.
        const uint32_t lane_at = uint32_t(wave) * (S::DB * 8 + 1) * 128 + 2 * lane2;
        const auto write_rows = [&] {
            const int row = wave * 32 + col2;
            if (row >= u.rows) return;
            const float inv = inverse(st.l);
#pragma unroll
            for (int d = 0; d < S::DB; ++d)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int at_d = 32 * d + 8 * x + 4 * h2;
                    if (!S::FULL && at_d >= p.dim) continue;
                    put_out(row, at_d, st.o[d][4 * x], st.o[d][4 * x + 1], st.o[d][4 * x + 2], st.o[d][4 * x + 3], inv);
                }
            if (p.lse && h2 == 0) put_lse(row, st.m, st.l);
        };
        if (S::SHARED) {
            if (!whole && busy) {
                float* o = slot + lane_at;
#pragma unroll
                for (int d = 0; d < S::DB; ++d)
#pragma unroll
                    for (int i = 0; i < 8; ++i) put2(o + (8 * d + i) * 128, st.o[d][2 * i], st.o[d][2 * i + 1]);
                put2(o + S::DB * 8 * 128, st.m, st.l);
            }
        } else {
            // the waves' sums meet in LDS
            if (h2 == 0) ml[wave * 32 + col2] = st.m, ml[(S::W + wave) * 32 + col2] = st.l;
            __syncthreads();
            float m = -INFINITY, l = 0.0f;
#pragma unroll
            for (int w = 0; w < S::W; ++w) m = fmaxf(m, ml[w * 32 + col2]);
            const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int w = 0; w < S::W; ++w) l += ml[(S::W + w) * 32 + col2] * __builtin_amdgcn_exp2f(ml[w * 32 + col2] - ref);
            const float keep = __builtin_amdgcn_exp2f(st.m - ref);
            float* buf = reinterpret_cast<float*>(lds) + wave * S::M * S::OS + col2 * S::OS + 4 * h2;
            if (col2 < u.rows) {
#pragma unroll
                for (int d = 0; d < S::DB; ++d)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        float4 v = {st.o[d][4 * x] * keep, st.o[d][4 * x + 1] * keep, st.o[d][4 * x + 2] * keep, st.o[d][4 * x + 3] * keep};
                        *reinterpret_cast<float4*>(buf + 32 * d + 8 * x) = v;
                    }
                if (wave == 0 && h2 == 0) {
                    if (!whole) put2(slot + S::M * S::DP + 2 * col2, m, l);
                    else if (p.lse) put_lse(col2, m, l);
                }
            }
            __syncthreads();
            // (references and sums of the rows stay in ml)
            constexpr int QUADS = S::DP / 4;
            for (int i = tid; i < u.rows * QUADS; i += S::THREADS) {
                const int rw = i / QUADS, d = (i % QUADS) * 4;
                if (!S::FULL && d >= p.dim) continue;
                const float* src = reinterpret_cast<const float*>(lds) + rw * S::OS + d;
                float4 a = *reinterpret_cast<const float4*>(src);
#pragma unroll
                for (int w = 1; w < S::W; ++w) {
                    const float4 v = *reinterpret_cast<const float4*>(src + w * S::M * S::OS);
                    a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
                }
                if (whole) {
                    float m = -INFINITY, l = 0.0f;
#pragma unroll
                    for (int w = 0; w < S::W; ++w) m = fmaxf(m, ml[w * 32 + rw]);
                    const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
                    for (int w = 0; w < S::W; ++w) l += ml[(S::W + w) * 32 + rw] * __builtin_amdgcn_exp2f(ml[w * 32 + rw] - ref);
                    put_out(rw, d, a.x, a.y, a.z, a.w, inverse(l));
                } else {
                    put2(slot + rw * S::DP + d, a.x, a.y);
                    put2(slot + rw * S::DP + d + 2, a.z, a.w);
                }
            }
        }

        bool ready = whole;     // the unit's sums are complete
        if (!whole) {
            // The partial stores have reached the device-wide level before
            // this work-group counts its steps; whoever completes the count
            // finds every part there.
            wait_loads<0>();
            __syncthreads();
            // a run begins at most one unit that it does not end: the run in
            // which a unit's first step lies numbers its count
            const int64_t begin = at - off;
            const int wf = run_of(begin + S::EXTRA);
            if (threadIdx.x == 0) {
                uint32_t* cnt = reinterpret_cast<uint32_t*>(p.workspace) + wf;
                const uint32_t old = __hip_atomic_fetch_add(cnt, uint32_t(count), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                const bool last = old + uint32_t(count) == uint32_t(u.steps);
                if (last) __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                plan[4] = last;
            }
            __syncthreads();
            if (plan[4]) {
                // The unit's parts in run order; Split: sixteen parts' loads at a time.
                const int parts = run_of(begin + S::EXTRA + u.steps - 1) - wf + 1;
                // only the first can have begun in its run, all others continue one
                const int slot0 = wf * 2 + (run_start(wf) > begin ? 0 : 1);
                if constexpr (S::SHARED) if (busy) {
                    st.m = -INFINITY;
                    st.l = 0.0f;
#pragma unroll
                    for (int d = 0; d < S::DB; ++d)
#pragma unroll
                        for (int i = 0; i < 16; ++i) st.o[d][i] = 0.0f;
#pragma unroll 1
                    for (int x = 0; x < parts; ++x) {
                        const float* src = slots + uint64_t(x ? 2 * (wf + x) : slot0) * S::SLOT + lane_at;
                        float pm, pl;
                        get2(src + S::DB * 8 * 128, &pm, &pl);
                        const float m = fmaxf(st.m, pm), ref = m == -INFINITY ? 0.0f : m;
                        const float keep = __builtin_amdgcn_exp2f(st.m - ref), share = __builtin_amdgcn_exp2f(pm - ref);
                        st.m = m;
                        st.l = st.l * keep + pl * share;
#pragma unroll
                        for (int d0 = 0; d0 < S::DB; d0 += 4) {
                            float v[4][16];          // four blocks' loads at a time
#pragma unroll
                            for (int d = 0; d < 4 && d0 + d < S::DB; ++d)
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    get2(src + (8 * (d0 + d) + i) * 128, &v[d][2 * i], &v[d][2 * i + 1]);
                            asm volatile("" ::: "memory");
#pragma unroll
                            for (int d = 0; d < 4 && d0 + d < S::DB; ++d)
#pragma unroll
                                for (int i = 0; i < 16; ++i) st.o[d0 + d][i] = st.o[d0 + d][i] * keep + v[d][i] * share;
                        }
                    }
                }
                ready = true;
                constexpr int QUADS = S::DP / 4;
                for (int i = opaque(threadIdx.x); !S::SHARED && i < u.rows * QUADS; i += S::THREADS) {
                    const int rw = i / QUADS, d = (i % QUADS) * 4;
                    if (!S::FULL && d >= p.dim) continue;
                    float m = -INFINITY, l = 0.0f, a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    for (int x = 0; x < parts; x += 16) {
                        float pm[16], pl[16], v[16][4];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            // Narrow heads: past the last part it once more, for at a branch
                            // the loads before are waited for (8 sequences of up to 9000 keys,
                            // 32 heads of 64: 23.6 -> 20.0 us); with 128 dimensions the loads
                            // themselves take longer (16 x 8 tokens: 45 -> 52 us).
                            pm[e] = -INFINITY, pl[e] = v[e][0] = v[e][1] = v[e][2] = v[e][3] = 0.0f;
                            if (S::DP > 64 && x + e >= parts) continue;
                            const int part = min(x + e, parts - 1);
                            const float* src = slots + uint64_t(part ? 2 * (wf + part) : slot0) * S::SLOT;
                            get2(src + S::M * S::DP + 2 * rw, &pm[e], &pl[e]);
                            get2(src + rw * S::DP + d, &v[e][0], &v[e][1]);
                            get2(src + rw * S::DP + d + 2, &v[e][2], &v[e][3]);
                        }
                        asm volatile("" ::: "memory");
#pragma unroll
                        for (int e = 1; e < 16; ++e)
                            if (S::DP <= 64 && x + e >= parts) pm[e] = -INFINITY, pl[e] = v[e][0] = v[e][1] = v[e][2] = v[e][3] = 0.0f;
                        float mn = m;
#pragma unroll
                        for (int e = 0; e < 16; ++e) mn = fmaxf(mn, pm[e]);
                        const float ref = mn == -INFINITY ? 0.0f : mn, keep = __builtin_amdgcn_exp2f(m - ref);
                        m = mn;
                        l *= keep;
#pragma unroll
                        for (int j = 0; j < 4; ++j) a[j] *= keep;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float share = __builtin_amdgcn_exp2f(pm[e] - ref);
                            l += pl[e] * share;
#pragma unroll
                            for (int j = 0; j < 4; ++j) a[j] += v[e][j] * share;
                        }
                    }
                    put_out(rw, d, a[0], a[1], a[2], a[3], inverse(l));
                    if (d == 0 && p.lse) put_lse(rw, m, l);
                }
            }
        }
        if constexpr (S::SHARED)
            if (ready && busy) write_rows();
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
    const int64_t steps = (max_kv + 15 + S::STEP - 1) / S::STEP + 1 + S::EXTRA;
    const int64_t most = kComputeUnits * S::PER_CU, need = units * steps / S::LEAST + 1;
    return need < most ? (need + 7) / 8 * 8 : most;
}

template <class S>
size_t bytes(int64_t tokens, int group, int kv_heads, int seqs, int64_t max_kv)
{
    static_assert(kComputeUnits * S::PER_CU * 4 <= kCounterBytes, "a count a run");
    return kCounterBytes + size_t(workers<S>(tokens, group, kv_heads, seqs, max_kv)) * 2 * S::SLOT * 4;
}

template <class S>
hipError_t run(const AttnParams& a, Args p, hipStream_t s)
{
    const int64_t grid = workers<S>(a.tokens, a.group, a.cache.kv_heads, a.seqs, a.max_kv);
    static const hipError_t attr = [] {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(attention_kernel<S>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, S::LDS);
        if (e != hipSuccess) (void)hipGetLastError();
        return e;
    }();
    if (attr != hipSuccess && S::LDS > 64 * 1024) return attr;
    hipLaunchKernelGGL((attention_kernel<S>), dim3(unsigned(grid)), dim3(S::THREADS), S::LDS, s, p);
    return hipGetLastError();
}

// Waves that share key tiles.  Up to 32 rows a sequence and kv head stream
// the cache once either way: none (32 sequences of up to 9000 bf16 keys, 28
// rows: 82 us, shared 90; a few short ones are faster shared, 36 and 28).
int sharing(int64_t tokens, int64_t max_q, int group, int seqs)
{
    if (max_q * group <= 32) return 0;
    return tokens * group >= kManyRows * seqs ? 8 : 4;
}

// Calls f with the shape for a cache and a call's rows.
template <class F>
auto with_shape(bool e4m3, int dim, int waves, F f)
{
    const auto by_dim = [&](auto e, auto w) {
        constexpr bool E = decltype(e)::value;
        constexpr int W = decltype(w)::value, W256 = W == 8 ? 4 : W;   // (a wave of 256 dimensions takes a whole SIMD's registers)
        if (dim == 64) return f(Shape<64, E, W, true>());
        if (dim == 128) return f(Shape<128, E, W, true>());
        if (dim == 256) return f(Shape<256, E, W256, true>());
        if (dim <= 64) return f(Shape<64, E, W, false>());
        if (dim <= 96) return f(Shape<96, E, W, false>());
        if (dim <= 128) return f(Shape<128, E, W, false>());
        return f(Shape<256, E, W256, false>());
    };
    const auto by_type = [&](auto w) { return e4m3 ? by_dim(std::true_type(), w) : by_dim(std::false_type(), w); };
    if (waves == 0) return by_type(std::integral_constant<int, 0>());
    return waves == 4 ? by_type(std::integral_constant<int, 4>()) : by_type(std::integral_constant<int, 8>());
}

}  // namespace

size_t attention_workspace_need(bool e4m3, int64_t tokens, int q_heads, int kv_heads, int head_dim, int seqs,
                                int64_t max_q, int64_t max_kv)
{
    const int group = q_heads / kv_heads;
    return with_shape(e4m3, head_dim, sharing(tokens, max_q < tokens ? max_q : tokens, group, seqs), [&](auto shape) {
        return bytes<decltype(shape)>(tokens, group, kv_heads, seqs, max_kv);
    });
}

// The largest need of any shape within the bounds: each kernel shape's grows
// with all of them, and smaller calls may take another one than the largest.
size_t attention_workspace_bytes(bool e4m3, int64_t tokens, int q_heads, int kv_heads, int head_dim, int seqs,
                                 int64_t max_q, int64_t max_kv)
{
    const int group = q_heads / kv_heads;
    size_t most = 0;
    for (int waves : {0, 4, 8}) {
        if (waves > sharing(tokens, max_q < tokens ? max_q : tokens, group, 1)) break;
        const size_t n = with_shape(e4m3, head_dim, waves, [&](auto shape) {
            return bytes<decltype(shape)>(tokens, group, kv_heads, seqs, max_kv);
        });
        if (n > most) most = n;
    }
    return most;
}

hipError_t launch_attention(const AttnParams& a, hipStream_t s)
{
    const int unit = a.cache.e4m3 ? 16 : 8;   // elements in 16 bytes
    const int64_t cap = a.table_cols << a.cache.page_shift;
    Args p;
    p.k = a.cache.k;
    p.v = a.cache.v;
    p.k_scale = a.cache.k_scale;
    p.v_scale = a.cache.v_scale;
    p.q = a.q;
    p.out = a.out;
    p.lse = a.lse;
    p.q_start = a.q_start;
    p.kv_len = a.kv_len;
    p.table = a.table;
    p.workspace = static_cast<uint8_t*>(a.workspace);
    p.page16 = uint32_t(a.cache.page_stride / unit);
    p.head16 = uint32_t(a.cache.head_stride / unit);
    p.slot16 = uint32_t(a.cache.slot_stride / unit);
    p.q_token = uint32_t(a.q_token);
    p.q_head = uint32_t(a.q_head);
    p.o_token = uint32_t(a.o_token);
    p.o_head = uint32_t(a.o_head);
    p.lse_token = uint32_t(a.lse_token);
    p.table_stride = uint32_t(a.table_stride);
    p.pages = int32_t(a.cache.pages);
    p.kv_heads = a.cache.kv_heads;
    p.page_shift = a.cache.page_shift;
    p.dim = a.cache.head_dim;
    p.tokens = int32_t(a.tokens);
    p.max_q = int32_t(a.max_q);
    p.cap = int32_t(cap < a.max_kv ? cap : a.max_kv);
    p.window = a.window > kMaxWindow ? kMaxWindow : int32_t(a.window);
    p.seqs = a.seqs;
    p.group = a.group;
    p.by_group = uint32_t(((uint64_t(1) << 31) + a.group - 1) / a.group);
    p.scale = a.scale;
    return with_shape(a.cache.e4m3, a.cache.head_dim, sharing(a.tokens, a.max_q, a.group, a.seqs),
                      [&](auto shape) { return run<decltype(shape)>(a, p, s); });
}

}  // namespace qg
