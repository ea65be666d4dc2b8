// Attention of few rows (single and drafted tokens, short chunks) over a 4-bit
// paged cache, on the matrix cores.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q . k_j - m)
//
// with m a running reference, as in paged_attention.hip, whose line of work,
// parts and workspace these kernels share: a unit is (kv head, sequence, row
// tile) with up to 16 R rows (tokens x query heads of the kv head), all units'
// steps lie in one line, and each work-group takes an equal run of it.  What bounds it:
// the cache's bytes on long contexts (three sequences of up to 131071 keys, 400
// MB: 73 us, of which some 8 pass before the first keys arrive and while parts
// are joined: 6.1 TB/s between, where a plain read reaches 6.8), and on short
// ones a chain of dependent accesses (one sequence of 1023 keys: lengths, page
// ids, keys, the parts' stores, their count and their join, 8.7 us).
//
// Products.  S^T = K Q^T and O^T = V^T P^T, 16x16x32.  Lane l holds of key
// l % 16 the 8 T dimensions from 8 T (l / 16) on, as they lie in memory: a
// register is eight codes, one conversion of two codes at a time applies the
// block's scale, and the result is the A operand of one product, whose
// dimensions the queries take in the same order.  So keys never see LDS.  A
// lane's values have to be of one dimension and eight keys: they are written to
// LDS as bf16 rows and read back through the transposing reads, keys in the
// order that the scores' lanes hold them (4 g .. 4 g + 3 of two tiles of 16).
// Every value is exact in bf16.
//
// A wave works out the plan, looks up its pages (lane j holds the page of its
// tile j) and streams its tiles without the work-group's other waves; they meet
// where a unit ends.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attention_common.h"
#include "decode_ops.h"

namespace qg {

namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
// An address in global memory, which a generic pointer would make a flat
// access of, counted with those of LDS and waited for with them.
typedef __attribute__((address_space(1))) const uint8_t* global_ptr;

constexpr int kAhead = 4;          // LDS reads ahead of their matrix products
// Of a buffer access: past the XCD's own cache; not to stay in the caches.
constexpr int kDeviceScope = 16, kOnce = 2;
constexpr uint32_t kNowhere = 0x1fffffffu;   // floats: past every buffer below

// 32 T dimensions, tiles of 16 R rows; EVEN: 16 keys of a tile lie in one page;
// W waves a work-group; TILED: a sequence may have more than one tile of rows
// (of its own, as it costs 0.3 to 0.7 us: 12 sequences of 24 rows 20.4 and 21.1).
template <int T_, int R_, bool EVEN_, int W_, bool TILED_>
struct Few {
    static constexpr bool TILED = TILED_;
    static constexpr int T = T_, R = R_, DP = 32 * T;
    static constexpr bool EVEN = EVEN_;
    static constexpr int RB = T <= 2 ? 64 * T : T <= 4 ? 256 : 512;     // bytes of a row of V in LDS, a power of two
    static constexpr int W = W_, THREADS = 64 * W;
    static constexpr int M = 16 * R;
    // bf16 numbers that a probability enters the second product as
    static constexpr int NP = TILED && EVEN ? 1 : 2;
    static constexpr int KT = 32, STEP = KT * W;                        // keys of a wave's tiles, of a step
    static constexpr int TILE = KT * RB;
    // exponent bytes that a lane's 8 T dimensions of a key reach into
    static constexpr int NS = T == 7 ? 3 : T == 3 || T >= 5 ? 2 : 1;
    static constexpr int REGISTERS = 8 * T * R + 4 * T * R + 4 * T + 4 * NS + 72;
    // (four waves of 128 registers a SIMD are not better than three of 168)
    static constexpr int WAVES_PER_SIMD = REGISTERS <= 110 ? 4 : REGISTERS <= 160 && W == 4 ? 3 : REGISTERS <= 240 ? 2 : 1;
    static constexpr int OS = DP + 4;                                   // floats of a row in the joining buffer
    static constexpr int RING = W * TILE, JOIN = W * M * OS * 4;
    static constexpr int BUFFER = RING > JOIN ? RING : JOIN;
    static constexpr int LDS = BUFFER + 2 * W * M * 4 + 64;
    static constexpr int BY_LDS = 160 * 1024 / LDS, BY_WAVES = 4 * WAVES_PER_SIMD / W;
    static constexpr int PER_CU = BY_LDS < BY_WAVES ? BY_LDS : BY_WAVES;
    // Steps that a run has at least, what beginning and ending a unit costs in
    // steps, what joining a part costs.
    static constexpr int LEAST = 2, EXTRA = 3;
    static constexpr float JOINED = 0.25f;
    static constexpr int SLOT = M * DP + 2 * M;                         // floats of a partial result
    // Joining: four values at a time, and parts whose loads are in flight together.
    static constexpr int QUADS = DP / 4, PARTS = 8;

    // The chunk of 8 dimensions is moved so that 16 keys of one chunk (what a
    // wave's quarter writes) and 8 keys of two neighbours (what a half reads)
    // lie in different banks of 256 bytes.
    static __device__ __forceinline__ int swizzle(int key)
    {
        if (T == 1) return ((key >> 2) & 1) << 1 | ((key >> 3) & 1);
        if (T == 2) return ((key >> 1) & 3) << 1 | ((key >> 3) & 1);
        return (key & 7) << 1 | ((key >> 3) & 1);
    }
};

// Keys [lo, hi) that some row of a sequence sees, and that every row sees; the
// first tile starts at `base`.
struct Span {
    int lo, hi, all_lo, all_hi, base, steps;
};

template <class S>
__device__ __forceinline__ Span make_span(const Args& p, const Seq& s)
{
    Span x;
    const int first = s.kv - s.n;
    x.hi = s.kv;
    x.lo = p.window > 0 ? min(max(0, first - p.window + 1), x.hi) : 0;
    x.all_lo = p.window > 0 ? max(0, s.kv - p.window) : 0;
    x.all_hi = first + 1;
    x.base = x.lo & ~15;
    // a unit without keys still writes its rows
    x.steps = x.hi > x.lo ? int(uint32_t(x.hi - x.base + S::STEP - 1) / S::STEP) : 1;
    return x;
}

// Tiles of M rows, each a unit of its own.
template <class S>
__device__ __forceinline__ int tiles_of(const Args& p, const Seq& s)
{
    return !S::TILED ? 1 : int(uint32_t(s.n * p.group + S::M - 1) / S::M);
}

template <class S>
__device__ __forceinline__ int unit_cost(const Args& p, const Seq& s)
{
    return s.n > 0 ? make_span<S>(p, s).steps + S::EXTRA : 0;
}

template <class S>
__device__ __forceinline__ int cost_of(const Args& p, const Seq& s)
{
    return tiles_of<S>(p, s) * unit_cost<S>(p, s);
}

// Where a sequence's keys lie for one kv head.
struct Place {
    const BlockArgs& p;
    const int32_t* table;
    int pages;                         // of the sequence
    uint64_t k, v, k_block, v_block;

    // Page id of a key: -1 outside the sequence or the cache.
    __device__ __forceinline__ int page_of(int key) const
    {
        const int page = key >> p.page_shift;
        int id = -1;
        if (page < pages) id = table[page];
        return id >= p.pages ? -1 : id;
    }
};

// Memory from an address that all lanes share, for offsets of 32 bits.
__device__ __forceinline__ auto buffer_at(uint64_t address)
{
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(address), 0, -1, 0x00020000);
}

// Two tiles of 16 keys of K and of V on their way through registers.
template <class S>
struct Tile {
    uint32_t k[2][S::T], v[2][S::T];
    uint32_t ke[2][S::NS], ve[2][S::NS];
    int page[2];                       // of the lane's key

    // N words at a lane's part of a row, which begins on 4 bytes.
    template <int N>
    __device__ __forceinline__ static void load_words(uint32_t* to, global_ptr at)
    {
        constexpr int n = N >= 4 ? 4 : N;
        if constexpr (n == 1) {
            to[0] = *reinterpret_cast<__attribute__((address_space(1))) const uint32_t*>(at);
        } else {
            typedef uint32_t words __attribute__((ext_vector_type(n), aligned(4)));
            const words x = *reinterpret_cast<__attribute__((address_space(1))) const words*>(at);
#pragma unroll
            for (int i = 0; i < n; ++i) to[i] = x[i];
        }
        if constexpr (N > 4) load_words<N - 4>(to + 4, at + 16);
    }
    // The same at an offset from an address that all lanes share.
    template <int N, class B>
    __device__ __forceinline__ static void load_words(uint32_t* to, B base, uint32_t at)
    {
        if constexpr (N >= 4) {
            const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(base, at, 0, kOnce);
#pragma unroll
            for (int i = 0; i < 4; ++i) to[i] = x[i];
        } else if constexpr (N == 3) {
            const auto x = __builtin_amdgcn_raw_buffer_load_b96(base, at, 0, kOnce);
#pragma unroll
            for (int i = 0; i < 3; ++i) to[i] = x[i];
        } else if constexpr (N == 2) {
            const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(base, at, 0, kOnce);
            to[0] = x[0], to[1] = x[1];
        } else {
            to[0] = __builtin_amdgcn_raw_buffer_load_b32(base, at, 0, kOnce);
        }
        if constexpr (N > 4) load_words<N - 4>(to + 4, base, at + 16);
    }

    // Tile a's parts of the lanes' keys, 16 rows of a page from `slot` on.
    __device__ __forceinline__ void fetch_page(const Place& at, int a, int id, uint32_t slot, uint32_t code_at, uint32_t byte_at, int b0)
    {
        page[a] = id;
        const uint64_t n = uint32_t(max(0, id));
        const uint64_t codes = (n * at.p.page16 + uint64_t(slot) * at.p.slot16) << 4;
        const uint64_t bytes = n * at.p.block_page + uint64_t(slot) * at.p.block_slot;
        load_words<S::T>(k[a], buffer_at(at.k + codes), code_at);
        load_words<S::T>(v[a], buffer_at(at.v + codes), code_at);
#pragma unroll
        for (int x = 0; x < S::NS; ++x) {
            // (past the row's last block: not used)
            const uint32_t byte = byte_at + uint32_t(min(b0 + x, S::T - 1));
            ke[a][x] = __builtin_amdgcn_raw_buffer_load_b8(buffer_at(at.k_block + bytes), byte, 0, 0);
            ve[a][x] = __builtin_amdgcn_raw_buffer_load_b8(buffer_at(at.v_block + bytes), byte, 0, 0);
        }
    }

    // The same for a page of the lane's own.
    __device__ __forceinline__ void fetch_row(const Place& at, int a, int id, uint32_t slot, uint32_t part, int b0)
    {
        page[a] = id;
        const uint64_t n = uint32_t(max(0, id));
        const uint64_t codes = ((n * at.p.page16 + uint64_t(slot) * at.p.slot16) << 4) + part;
        const uint64_t bytes = n * at.p.block_page + uint64_t(slot) * at.p.block_slot;
        load_words<S::T>(k[a], global_ptr(at.k + codes));
        load_words<S::T>(v[a], global_ptr(at.v + codes));
#pragma unroll
        for (int x = 0; x < S::NS; ++x) {
            const int b = min(b0 + x, S::T - 1);
            ke[a][x] = global_ptr(at.k_block + bytes)[b];
            ve[a][x] = global_ptr(at.v_block + bytes)[b];
        }
    }

    // Of the lane's dimensions, step t (eight of them) lies in this of its blocks.
    __device__ __forceinline__ static float scale_of(const float* scales, int t, int g)
    {
        if constexpr (S::T == 8) return scales[t / 4];
        if constexpr (S::NS == 1) return scales[0];
        // (loaded before the choice: a choice of addresses would put them in memory)
        const float first = scales[0], second = scales[1], third = scales[S::NS - 1];
        const int b = (S::T * g + t) / 4 - S::T * g / 4;
        return b == 0 ? first : b == 1 ? second : third;
    }

    __device__ __forceinline__ static bf16x8 values(uint32_t codes, float scale)
    {
        union { bf16x8 v; bf16x2 p[4]; } a;
        a.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
        a.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
        a.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
        a.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
        return a.v;
    }
};

// What a wave accumulates for its rows, a lane's columns.
template <class S>
struct State {
    f32x4 o[S::R][2 * S::T];
    bf16x8 q[S::R][S::T];
    float m[S::R], l[S::R];            // reference; this quarter's share of the sum
    int rlo[S::R], rhi[S::R];          // keys the lane's rows see
};

// A value over the four lanes that hold a row's keys.
template <class F>
__device__ __forceinline__ float over_quarters(float x, F f)
{
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = f(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return f(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// Scores of the tiles' keys, and their values into the wave's rows of LDS: what
// needs the loaded registers.  Returns whether values were taken out.
template <class S>
__device__ __forceinline__ bool consume(const State<S>& st, Tile<S>& tile, f32x4 (&sc)[S::R][2], const Span& span, bool masked,
                                        uint8_t* vt, int k0, int lane)
{
    const int col = lane & 15, g = lane >> 4;
    bool poisoned = false;
    if (masked || __any((tile.page[0] | tile.page[1]) < 0)) {
        // Rows outside [lo, hi) hold another's data, which must not be NaN (their
        // scores are masked): an exponent byte of 0 makes it too small to count.
        // Keys of a page outside the cache become NaN.  Values that are NaN at
        // a key that only some rows see are taken out as well; rows that see it
        // get them back at the end (restore).
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int key = k0 + 16 * a + col;
            const bool outside = key < span.lo || key >= span.hi, lost = tile.page[a] < 0;
            const bool some = key < span.all_lo || key >= span.all_hi;
#pragma unroll
            for (int x = 0; x < S::NS; ++x) {
                if (lost) tile.ke[a][x] = 255;
                const bool nan = tile.ve[a][x] > 252 && some && !outside && !lost;
                poisoned |= nan;
                if (outside || lost || nan) tile.ve[a][x] = 0;
            }
        }
        poisoned = __any(poisoned);
    }
    float ks[2][S::NS], vs[2][S::NS];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int x = 0; x < S::NS; ++x) ks[a][x] = block_scale(tile.ke[a][x]), vs[a][x] = block_scale(tile.ve[a][x]);
#pragma unroll
    for (int r = 0; r < S::R; ++r)
#pragma unroll
        for (int a = 0; a < 2; ++a) sc[r][a] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int t = 0; t < S::T; ++t)
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const bf16x8 f = tile.values(tile.k[a][t], tile.scale_of(ks[a], t, g));
#pragma unroll
            for (int r = 0; r < S::R; ++r) sc[r][a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, st.q[r][t], sc[r][a], 0, 0, 0);
        }
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int t = 0; t < S::T; ++t)
            *reinterpret_cast<bf16x8*>(vt + (16 * a + col) * S::RB + (((S::T * g + t) ^ S::swizzle(col)) << 4)) =
                tile.values(tile.v[a][t], tile.scale_of(vs[a], t, g));
    return poisoned;
}

// Probabilities of the scores and the values weighed by them.  The matrix cores
// take bf16, half a step of which is 2^-8 of a probability.  Such errors do not
// cancel beside values that cancel likewise: outputs are off by 0.0018 to 0.0022
// of their norm, by 0.0016 to 0.0017 where the exact one is rounded once.  So
// probabilities of up to 32 rows go in as two numbers, the second what rounding
// the first left (2^-16 is lost), for 1 to 5% of the time of single and drafted
// tokens (40 ragged ones 26.2 and 26.7 us, 3 of up to 131071 keys 70.5 and 73.6,
// 12 x 6 tokens 20.5 and 21.6) and up to 14% over long contexts (8 tokens over
// 80000 keys 42.5 and 48).  Tiles of more rows, bound by the matrix cores and
// vector instructions, would take up to a fifth longer (64 rows, 32 sequences of
// 6000 keys: 84 and 99 us), and have one, as chunks have.  (fp16 would cost
// nothing, but has no bits for probabilities far below a row's largest, all that
// remains where its value is zero.)
template <class S>
__device__ __forceinline__ void accumulate(State<S>& st, f32x4 (&sc)[S::R][2], bool masked, const uint8_t* vt, int k0, float c,
                                           int lane)
{
    const int col = lane & 15, g = lane >> 4;
    bf16x8 pb[S::R][S::NP];
#pragma unroll
    for (int r = 0; r < S::R; ++r) {
        if (masked) {
            const uint32_t width = uint32_t(st.rhi[r] - st.rlo[r]);
            const int first = k0 + 4 * g - st.rlo[r];
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (uint32_t(first + 16 * a + i) >= width) sc[r][a][i] = -INFINITY;
        }
        float top = sc[r][0][0];
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[r][a][i]);
        // the row's largest only where some lane's passes the reference by too much
        if (__any(top * c > st.m[r] + kRaise)) {
            top = over_quarters(top, [](float x, float y) { return fmaxf(x, y); }) * c;
            const bool raise = top > st.m[r] + kRaise;
            // of this lane's row alone: other rows keep their reference and their bits
            const float mn = raise ? top : st.m[r];
            const float keep = raise ? __builtin_amdgcn_exp2f(st.m[r] - mn) : 1.0f;
            st.m[r] = mn;
            st.l[r] *= keep;
#pragma unroll
            for (int n = 0; n < 2 * S::T; ++n) st.o[r][n] *= keep;
        }
        const float ref = st.m[r] == -INFINITY ? 0.0f : st.m[r];
        union { bf16x8 v; uint32_t u[4]; } pr, rest;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[r][a][2 * x], c, -ref));
                const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[r][a][2 * x + 1], c, -ref));
                st.l[r] += p0;
                st.l[r] += p1;
                const uint32_t both = pack_bf16(p0, p1);
                pr.u[2 * a + x] = both;
                if (S::NP > 1) rest.u[2 * a + x] = pack_bf16(p0 - __uint_as_float(both << 16), p1 - __uint_as_float(both & 0xffff0000u));
            }
        pb[r][0] = pr.v;
        if constexpr (S::NP > 1) pb[r][1] = rest.v;
    }

    const int key = 4 * g + col / 4;
    const uint8_t* row = vt + key * S::RB + (col & 1) * 8;
    const int chunk = ((col & 3) / 2) ^ S::swizzle(key);      // (16 keys on have the same)
    union { bf16x8 v; s16x4 h[2]; } f[2 * S::T];
    const auto read = [&](int n) {
        const uint8_t* at = row + ((chunk ^ (2 * n)) << 4);
        f[n].h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
        f[n].h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 16 * S::RB));
    };
#pragma unroll
    for (int n = 0; n < (kAhead < 2 * S::T ? kAhead : 2 * S::T); ++n) read(n);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < 2 * S::T; ++n) {
        if (n + kAhead < 2 * S::T) read(n + kAhead);
#pragma unroll
        for (int e = 0; e < S::NP; ++e)
#pragma unroll
            for (int r = 0; r < S::R; ++r)
                st.o[r][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[n].v, pb[r][e], st.o[r][n], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Gives the lane's rows the blocks of NaN that were taken out of values at the
// wave's keys of [from, to), which no probability takes away.
template <class S>
__device__ __forceinline__ void restore(State<S>& st, const Place& at, const Span& span, int from, int to, int wave)
{
    const int mask = (1 << at.p.page_shift) - 1;
#pragma unroll 1
    for (int key = max(from, span.lo); key < min(to, span.hi); ++key) {
        if (key >= span.all_lo && key < span.all_hi) {
            key = span.all_hi - 1;     // none between
            continue;
        }
        if ((key - from) / S::KT % S::W != wave) continue;
        const int id = at.page_of(key);
        if (id < 0) continue;
        const global_ptr e = global_ptr(at.v_block + uint64_t(uint32_t(id)) * at.p.block_page +
                                        uint64_t(uint32_t(key & mask)) * at.p.block_slot);
#pragma unroll
        for (int b = 0; b < S::T; ++b) {
            if (e[b] <= 252) continue;
#pragma unroll
            for (int r = 0; r < S::R; ++r)
                if (key >= st.rlo[r] && key < st.rhi[r])
#pragma unroll
                    for (int i = 0; i < 8; ++i) st.o[r][2 * b + i / 4][i % 4] = __builtin_nanf("");
        }
    }
}

// Partial results, `at` floats from a base that all lanes share; at kNowhere
// zeros, with no access.
__device__ __forceinline__ auto parts_buffer(float* base)
{
    return __builtin_amdgcn_make_buffer_rsrc(base, 0, 0x7ffffff0, 0x00020000);
}
__device__ __forceinline__ void put4(float* base, uint32_t at, f32x4 v)
{
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), parts_buffer(base), at * 4, 0, kDeviceScope);
}
__device__ __forceinline__ f32x4 get4(float* base, uint32_t at)
{
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(parts_buffer(base), at * 4, 0, kDeviceScope));
}
__device__ __forceinline__ f32x2 get2(float* base, uint32_t at)
{
    return __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(parts_buffer(base), at * 4, 0, kDeviceScope));
}

template <class S>
__global__ __launch_bounds__(S::THREADS, S::WAVES_PER_SIMD) void few_rows_kernel(BlockArgs p)
{
    extern __shared__ __align__(1024) uint8_t lds[];
    float* ml = reinterpret_cast<float*>(lds + S::BUFFER);          // [2][W][M]
    int* last_part = reinterpret_cast<int*>(ml + 2 * S::W * S::M);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    fetch_arguments<sizeof(p)>();

    // ---- the line of work: this run's part of it.  Each lane has a run of
    // sequences, most often one.
    const int per = (p.seqs + 63) / 64, b0 = lane * per;
    Seq own = {0, 0, 0};
    int64_t mine = 0;
    int longest = 0;
    for (int b = b0; b < min(b0 + per, p.seqs); ++b) {
        own = load_seq(p, b);
        mine += cost_of<S>(p, own);
        longest = max(longest, unit_cost<S>(p, own));
    }
    int64_t upto = mine;
    scan_lanes(upto, longest);
    longest = __builtin_amdgcn_readlane(longest, 63);
    const auto of_lane = [](int64_t x, int l) {
        return int64_t(uint64_t(uint32_t(__builtin_amdgcn_readlane(int(x >> 32), l))) << 32 | uint32_t(__builtin_amdgcn_readlane(int(x), l)));
    };
    const int64_t head_steps = of_lane(upto, 63);
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
        const bool in = x < split;
        return int((in ? 0 : longer) + divide(in ? x : x - split, in ? base + 1 : base));
    };
    int64_t at = run_start(run);
    const int64_t end = run_start(run + 1);
    int kvh = int(uniform(divide(at, head_steps)));

    const auto get_seq = [&](int b) {
        if (per > 1) return load_seq(p, __builtin_amdgcn_readfirstlane(b));
        return Seq{__builtin_amdgcn_readlane(own.q0, b), __builtin_amdgcn_readlane(own.n, b), __builtin_amdgcn_readlane(own.kv, b)};
    };
    const int64_t r = at - kvh * head_steps;
    const int owner = __builtin_amdgcn_readfirstlane(int(__builtin_ctzll(__ballot(r < upto))));
    int b = owner * per;
    int64_t left = r - of_lane(upto - mine, owner);
    Seq s = get_seq(b);
    for (int cost; left >= (cost = cost_of<S>(p, s)); s = get_seq(++b)) left -= cost;
    int tile = 0, off = int(left);
    if (S::TILED)
        for (const int unit = unit_cost<S>(p, s); off >= unit; ++tile) off -= unit;

    while (true) {
        s.q0 = __builtin_amdgcn_readfirstlane(s.q0);
        s.n = __builtin_amdgcn_readfirstlane(s.n);
        s.kv = __builtin_amdgcn_readfirstlane(s.kv);
        const Span u = make_span<S>(p, s);
        const int take = int(min(int64_t(u.steps + S::EXTRA - off), end - at));
        const int from = max(0, off - S::EXTRA), count = max(0, off + take - S::EXTRA) - from;
        if (count > 0) {       // (else only what stands for the unit's beginning)
            const int ulane = opaque(lane), col = ulane & 15, g = ulane >> 4;
            const int row0 = S::TILED ? tile * S::M : 0, rows = min(S::M, s.n * p.group - row0);
            Place place{p, p.table + uint64_t(uint32_t(b)) * p.table_stride, 0, 0, 0, 0, 0};
            place.pages = int((uint32_t(s.kv) + (1u << p.page_shift) - 1) >> p.page_shift);
            const uint64_t head_bytes = uint64_t(uint32_t(kvh)) * p.head16 << 4, head_blocks = uint64_t(uint32_t(kvh)) * p.block_head;
            place.k = reinterpret_cast<uint64_t>(p.k) + head_bytes;
            place.v = reinterpret_cast<uint64_t>(p.v) + head_bytes;
            place.k_block = reinterpret_cast<uint64_t>(p.k_block) + head_blocks;
            place.v_block = reinterpret_cast<uint64_t>(p.v_block) + head_blocks;

            // ---- this wave's tiles: two of 16 keys a step.  A tile lies in one
            // page: lane j holds that of tile j of 64, or lanes look up their keys'.
            const int k1 = u.base + from * S::STEP + wave * S::KT;
            int ids = -1;
            const auto look_up = [&](int step) { ids = place.page_of(k1 + (step + (ulane >> 1)) * S::STEP + 16 * (ulane & 1)); };
            const bool keys = u.hi > u.lo;
            if (S::EVEN && keys) look_up(0);

            // ---- the rows
            State<S> st;
#pragma unroll
            for (int x = 0; x < S::R; ++x) {
                // rows past the last repeat it and are never written
                const uint32_t row = uint32_t(row0 + min(16 * x + col, rows - 1)), step = by_group(p, row);
                const uint32_t head = uint32_t(kvh) * uint32_t(p.group) + (row - step * uint32_t(p.group));
                const uint16_t* qrow = p.q + uint64_t(uint32_t(s.q0) + step) * p.q_token + uint64_t(head) * p.q_head + 8 * S::T * g;
                const int pos = s.kv - s.n + int(step);
                st.rhi[x] = max(0, pos + 1);
                st.rlo[x] = p.window > 0 ? min(st.rhi[x], max(0, pos - p.window + 1)) : 0;
                st.m[x] = -INFINITY;
                st.l[x] = 0.0f;
#pragma unroll
                for (int t = 0; t < S::T; ++t)
                    st.q[x][t] = __builtin_bit_cast(
                        bf16x8, *reinterpret_cast<__attribute__((address_space(1))) const u32x4*>(global_ptr(reinterpret_cast<uint64_t>(qrow + 8 * t))));
#pragma unroll
                for (int n = 0; n < 2 * S::T; ++n) st.o[x][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
            // The scale's sign goes into the queries, so that the largest score
            // stays the largest; a scale of zero becomes one that leaves scores
            // equal.
            const float c = fmaxf(fabsf(p.scale * kLog2e), 1e-37f);
            if (p.scale < 0.0f) {
#pragma unroll
                for (int x = 0; x < S::R * S::T; ++x) {
                    bf16x8& q = st.q[x / S::T][x % S::T];
                    q = __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, q) ^ 0x80008000u);
                }
            }

            // ---- the tiles
            uint8_t* vt = lds + wave * S::TILE;
            bool poisoned = false;
            const int n = keys ? count : 0;
            const auto fetch = [&](Tile<S>& tile, int i) {
                const int k0 = k1 + i * S::STEP, mask = (1 << p.page_shift) - 1, b0 = 8 * S::T * g / kBlock;
                const uint32_t part = 4 * S::T * g;
                if (S::EVEN && i > 0 && i % 32 == 0) look_up(i);
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    if (S::EVEN) {
                        tile.fetch_page(place, a, __builtin_amdgcn_readlane(ids, 2 * (i % 32) + a), uint32_t((k0 + 16 * a) & mask),
                                        uint32_t(col) * (p.slot16 * 16) + part, uint32_t(col) * p.block_slot, b0);
                    } else {
                        const int key = k0 + 16 * a + col;
                        tile.fetch_row(place, a, place.page_of(key), uint32_t(key & mask), part, b0);
                    }
                }
            };
            // The loads of the step after next begin once this one's registers are
            // converted, ahead of the softmax and the second product.
            const auto step = [&](Tile<S>& tile, int i) {
                const int k0 = k1 + i * S::STEP;
                const bool live = k0 < u.hi, masked = k0 < u.all_lo || k0 + S::KT > u.all_hi;
                f32x4 sc[S::R][2];
                if (live) poisoned |= consume<S>(st, tile, sc, u, masked, vt, k0, ulane);
                asm volatile("" ::: "memory");
                if (i + 1 < n) fetch(tile, i + 1);
                if (live) accumulate<S>(st, sc, masked, vt, k0, c, ulane);
                asm volatile("" ::: "memory");
            };
            Tile<S> keys_values;
            if (n > 0) fetch(keys_values, 0);
#pragma unroll 1
            for (int i = 0; i < n; ++i) step(keys_values, i);
            if (poisoned) restore<S>(st, place, u, u.base + from * S::STEP, u.base + (from + count) * S::STEP, wave);

            // ---- the waves' sums meet in LDS; whole units go to the output, parts
            // to the workspace
            const bool whole = count == u.steps;
            const int tid = opaque(threadIdx.x);
            float* slots = reinterpret_cast<float*>(p.workspace + kCounterBytes);
            const uint32_t slot = uint32_t(run * 2 + (off > 0 ? 0 : 1)) * S::SLOT;
            const auto put_out = [&](int row, int d, f32x4 a, float m, float l) {
                const uint32_t step = by_group(p, uint32_t(row0 + row));
                const uint32_t head = uint32_t(kvh) * uint32_t(p.group) + (uint32_t(row0 + row) - step * uint32_t(p.group));
                // rows that see nothing have l = 0 and o = 0
                a *= l == 0.0f ? 0.0f : 1.0f / l;
                uint16_t* o = p.out + uint64_t(uint32_t(s.q0) + step) * p.o_token + uint64_t(head) * p.o_head + d;
                *reinterpret_cast<u32x2*>(o) = u32x2{pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3])};
                if (d == 0 && p.lse)
                    p.lse[uint64_t(uint32_t(s.q0) + step) * p.lse_token + head] =
                        m == -INFINITY && l == 0.0f ? -INFINITY : (m + __log2f(l)) * kLn2;
            };
#pragma unroll
            for (int x = 0; x < S::R; ++x) {
                st.l[x] = over_quarters(st.l[x], [](float a, float b) { return a + b; });
                if (g == 0) ml[wave * S::M + 16 * x + col] = st.m[x], ml[(S::W + wave) * S::M + 16 * x + col] = st.l[x];
            }
            __syncthreads();
            // a row's reference and sum over the waves
            const auto over_waves = [&](int row, float* m, float* l) {
                *m = -INFINITY, *l = 0.0f;
#pragma unroll
                for (int w = 0; w < S::W; ++w) *m = fmaxf(*m, ml[w * S::M + row]);
                const float ref = *m == -INFINITY ? 0.0f : *m;
#pragma unroll
                for (int w = 0; w < S::W; ++w) *l += ml[(S::W + w) * S::M + row] * __builtin_amdgcn_exp2f(ml[w * S::M + row] - ref);
                return ref;
            };
#pragma unroll
            for (int x = 0; x < S::R; ++x) {
                const int row = 16 * x + col;
                float m, l;
                const float keep = __builtin_amdgcn_exp2f(st.m[x] - over_waves(row, &m, &l));
                float* buf = reinterpret_cast<float*>(lds) + (wave * S::M + row) * S::OS + 4 * g;
                if (row < rows) {
#pragma unroll
                    for (int n = 0; n < 2 * S::T; ++n) *reinterpret_cast<f32x4*>(buf + 16 * n) = st.o[x][n] * keep;
                    if (wave == 0 && g == 0 && !whole) put2(slots + slot + S::M * S::DP + 2 * row, m, l);
                }
            }
            __syncthreads();
#pragma unroll 1
            for (int i = tid; i < rows * S::QUADS; i += S::THREADS) {
                const int row = i / S::QUADS, d = i % S::QUADS * 4;
                const float* src = reinterpret_cast<const float*>(lds) + row * S::OS + d;
                f32x4 a = *reinterpret_cast<const f32x4*>(src);
#pragma unroll
                for (int w = 1; w < S::W; ++w) a += *reinterpret_cast<const f32x4*>(src + w * S::M * S::OS);
                if (whole) {
                    float m, l;
                    over_waves(row, &m, &l);
                    put_out(row, d, a, m, l);
                } else {
                    put4(slots, slot + row * S::DP + d, a);
                }
            }

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
                    *last_part = last;
                }
                __syncthreads();
                if (*last_part) {
                    // The unit's parts, PARTS parts' loads at a time.  Past the last
                    // part they read nowhere: at a branch the loads before it would
                    // be waited for.  Many parts of few rows: groups of threads
                    // take PARTS of them in turn, and their sums meet in LDS (one
                    // sequence of 131072 keys: 33.4 us, 35.2 without).
                    const int parts = run_of(begin + S::EXTRA + u.steps - 1) - wf + 1;
                    // only the first can have begun in its run, all others continue one
                    const int slot0 = wf * 2 + (run_start(wf) > begin ? 0 : 1);
                    const int items = rows * S::QUADS, log_items = 32 - __builtin_clz(items - 1);
                    int groups = 1;
                    while (S::R == 1 && groups * S::PARTS < parts && (groups * 2 << log_items) <= S::THREADS) groups *= 2;
                    const int me = opaque(threadIdx.x), group = groups > 1 ? me >> log_items : 0;
                    f32x4* sums = reinterpret_cast<f32x4*>(lds);               // [group][item]
                    f32x2* refs = reinterpret_cast<f32x2*>(sums + S::THREADS);
#pragma unroll 1
                    for (int i = groups > 1 ? me - (group << log_items) : me; i < items && group < groups; i += S::THREADS) {
                        const int row = i / S::QUADS, d = i % S::QUADS * 4;
                        float m = -INFINITY, l = 0.0f;
                        f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
                        for (int x = group * S::PARTS; x < parts; x += groups * S::PARTS) {
                            f32x2 pm[S::PARTS];
                            f32x4 v[S::PARTS];
#pragma unroll
                            for (int e = 0; e < S::PARTS; ++e) {
                                const uint32_t from = uint32_t(x + e ? 2 * (wf + x + e) : slot0) * S::SLOT;
                                const bool none = x + e >= parts;
                                pm[e] = get2(slots, none ? kNowhere : from + S::M * S::DP + 2 * row);
                                v[e] = get4(slots, none ? kNowhere : from + row * S::DP + d);
                            }
                            float mn = m;
#pragma unroll
                            for (int e = 0; e < S::PARTS; ++e) {
                                if (x + e >= parts) pm[e][0] = -INFINITY;
                                mn = fmaxf(mn, pm[e][0]);
                            }
                            const float ref = mn == -INFINITY ? 0.0f : mn, keep = __builtin_amdgcn_exp2f(m - ref);
                            m = mn;
                            l *= keep;
                            a *= keep;
#pragma unroll
                            for (int e = 0; e < S::PARTS; ++e) {
                                const float share = __builtin_amdgcn_exp2f(pm[e][0] - ref);
                                l += pm[e][1] * share;
                                a += v[e] * share;
                            }
                        }
                        if (groups == 1) put_out(row, d, a, m, l);
                        else sums[me] = a, refs[me] = f32x2{m, l};
                        if (groups > 1) break;
                    }
                    if (groups > 1) {
                        __syncthreads();
                        if (me < items) {
                            f32x2 r = refs[me];
                            f32x4 a = sums[me];
#pragma unroll 1
                            for (int x = 1; x < groups; ++x) {
                                const f32x2 o = refs[me + (x << log_items)];
                                const float mn = fmaxf(r[0], o[0]), ref = mn == -INFINITY ? 0.0f : mn;
                                const float keep = __builtin_amdgcn_exp2f(r[0] - ref), share = __builtin_amdgcn_exp2f(o[0] - ref);
                                r = f32x2{mn, r[1] * keep + o[1] * share};
                                a = a * keep + sums[me + (x << log_items)] * share;
                            }
                            put_out(me / S::QUADS, me % S::QUADS * 4, a, r[0], r[1]);
                        }
                    }
                }
            }
            __syncthreads();       // LDS is free again
        }
        at += take;
        if (at >= end) break;
        off = 0;
        if (S::TILED) {
            if (++tile < tiles_of<S>(p, s)) continue;
            tile = 0;
        }
        do {
            if (++b == p.seqs) b = 0, ++kvh;
            s = get_seq(b);
        } while (s.n == 0);
    }
}

template <class S>
int64_t workers(const FewSize& z)
{
    const int64_t units = int64_t(z.seqs) * z.kv_heads * ((z.rows + S::M - 1) / S::M);
    const int64_t steps = (z.max_kv + 15 + S::STEP - 1) / S::STEP + 1 + S::EXTRA;
    const int64_t most = kComputeUnits * S::PER_CU, need = units * steps / S::LEAST + 1;
    return need < most ? (need + 7) / 8 * 8 : most;
}

// Pages of fewer than 16 tokens, and rows gigabytes apart, have one kernel.
// Second sixteens of rows make parts twice as large: eight waves a work-group
// leave half as many parts, but half as many runs, which lose where each begins
// and ends several units (5 tokens over 8000 keys, 2 sequences of 8 heads: 17.8
// us against 21.4; 6 over up to 6007, 12 sequences: 21.8 against 23.9; 8 over
// 2000: 15.9 against 17.6; 24 over 8000: 59.8 against 59.3; 32 over up to 4000:
// 30.5 against 28.5; 100 over up to 2000: 44.9 against 37.0; 4 over up to 900:
// 14.3 against 13.2), with several tiles of rows as with one (48 rows, 16
// sequences of 4000 keys and 8 heads: 31.7 against 41.1).
bool wide_groups(const FewSize& z)
{
    return z.rows > 16 && z.even && z.dim <= 128 && int64_t(z.seqs) * z.kv_heads <= 192 && z.max_kv > 1024;
}

template <class F>
auto with_few(const FewSize& z, bool wide, F f)
{
    const auto by_dim = [&](auto r, auto even, auto tiled) {
        constexpr int R = decltype(r)::value;
        constexpr bool E = decltype(even)::value, TILED = decltype(tiled)::value;
        switch (z.dim / kBlock) {
        case 1: return f(Few<1, R, E, 4, TILED>());
        case 2: return f(Few<2, R, E, 4, TILED>());
        case 3: return f(Few<3, R, E, 4, TILED>());
        case 4: return f(Few<4, R, E, 4, TILED>());
        case 5: return f(Few<5, R, E, 4, TILED>());
        case 6: return f(Few<6, R, E, 4, TILED>());
        case 7: return f(Few<7, R, E, 4, TILED>());
        default: return f(Few<8, R, E, 4, TILED>());
        }
    };
    const auto by_rows = [&](auto tiled) {
        constexpr bool TILED = decltype(tiled)::value;
        if (!wide) return by_dim(std::integral_constant<int, 2>(), std::true_type(), tiled);
        switch (z.dim / kBlock) {
        case 1: return f(Few<1, 2, true, 8, TILED>());
        case 2: return f(Few<2, 2, true, 8, TILED>());
        case 3: return f(Few<3, 2, true, 8, TILED>());
        default: return f(Few<4, 2, true, 8, TILED>());
        }
    };
    if (!z.even) return by_dim(std::integral_constant<int, 2>(), std::false_type(), std::true_type());
    if (z.rows <= 16) return by_dim(std::integral_constant<int, 1>(), std::true_type(), std::false_type());
    return z.rows <= 32 ? by_rows(std::false_type()) : by_rows(std::true_type());
}

}  // namespace

static size_t few_bytes(const FewSize& z, bool wide)
{
    return with_few(z, wide, [&](auto shape) {
        using S = decltype(shape);
        static_assert(kComputeUnits * S::PER_CU * 4 <= kCounterBytes, "a count a run");
        static_assert(size_t(kComputeUnits) * S::PER_CU * 2 * S::SLOT < kNowhere - 4, "offsets of parts in 31 bits");
        return kCounterBytes + size_t(workers<S>(z)) * 2 * S::SLOT * 4;
    });
}

size_t attention_few_need(const FewSize& z) { return few_bytes(z, wide_groups(z)); }

// (smaller calls may take the four waves, whose runs are as many or more)
size_t attention_few_bytes(const FewSize& z) { return few_bytes(z, false); }

hipError_t launch_attention_few(const FewSize& z, const void* args, hipStream_t s)
{
    return with_few(z, wide_groups(z), [&](auto shape) {
        using S = decltype(shape);
        static const hipError_t attr = [] {
            const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(few_rows_kernel<S>),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, S::LDS);
            if (e != hipSuccess) (void)hipGetLastError();
            return e;
        }();
        if (attr != hipSuccess && S::LDS > 64 * 1024) return attr;
        hipLaunchKernelGGL((few_rows_kernel<S>), dim3(unsigned(workers<S>(z))), dim3(S::THREADS), S::LDS, s,
                           *static_cast<const BlockArgs*>(args));
        return hipGetLastError();
    });
}

}  // namespace qg
