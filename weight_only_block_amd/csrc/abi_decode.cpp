// C ABI of the operators between a decode step's GEMV calls (rotary positions
// with cache append, cached tokens read back, paged attention, sampling): argument checks on the host
// and one launch sequence on the caller's stream.  Nothing here allocates or
// synchronizes, and nothing is enqueued for a rejected call.
#include <hip/hip_runtime.h>
#include <cmath>
#include <math.h>

#include "../../include/qgemv.h"
#include "decode_ops.h"
#include "rows.h"

namespace {

constexpr int64_t kMaxCount = (int64_t(1) << 31) - 1;
// Elements a stride may span: products with a 31-bit index stay in 63 bits.
constexpr int64_t kMaxCachedTokens = int64_t(1) << 30;   // of one sequence
constexpr int64_t kMaxStride = int64_t(1) << 31;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

// The cache's description; head_dim a multiple of 16 up to 256, pages of a
// power of two tokens, every row starting on 16 bytes.
qg_status check_cache(const qg_kv_cache* c, qg::CacheView* out, qg::BlockView* blocks)
{
    if (!c || !c->k || !c->v) return QG_ERR_INVALID_ARG;
    if (c->dtype != QG_KV_BF16 && c->dtype != QG_KV_E4M3 && c->dtype != QG_KV_MXFP4) return QG_ERR_UNSUPPORTED;
    const bool e4m3 = c->dtype == QG_KV_E4M3, mxfp4 = c->dtype == QG_KV_MXFP4;
    if (mxfp4 && (!c->k_block_scale || !c->v_block_scale)) return QG_ERR_INVALID_ARG;
    if (e4m3 && (!c->k_scale || !c->v_scale)) return QG_ERR_INVALID_ARG;
    if (c->pages < 1 || c->pages > kMaxCount || c->kv_heads < 1 || c->page_size < 1 || c->head_dim < 1)
        return QG_ERR_INVALID_ARG;
    if (c->head_dim % 16 != 0 || c->head_dim > qg::kMaxHeadDim || c->kv_heads > 65535) return QG_ERR_UNSUPPORTED;
    if (mxfp4 && c->head_dim % qg::kBlock != 0) return QG_ERR_UNSUPPORTED;
    if ((c->page_size & (c->page_size - 1)) != 0 || c->page_size > (1 << 20)) return QG_ERR_UNSUPPORTED;
    if (!stride_ok(c->page_stride) || !stride_ok(c->head_stride) || !stride_ok(c->slot_stride))
        return QG_ERR_INVALID_ARG;
    // (dimensions of one entry have no stride that matters)
    if ((c->page_size > 1 && c->slot_stride < c->head_dim) || (c->kv_heads > 1 && c->head_stride < c->head_dim) ||
        (c->pages > 1 && c->page_stride < c->head_dim))
        return QG_ERR_INVALID_ARG;
    const int64_t unit = mxfp4 ? 32 : e4m3 ? 16 : 8;   // elements in 16 bytes
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->page_stride % unit || c->head_stride % unit ||
        c->slot_stride % unit)
        return QG_ERR_ALIGNMENT;
    if (e4m3 && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))) return QG_ERR_ALIGNMENT;
    qg::Dim dims[] = {{c->pages, c->page_stride}, {c->kv_heads, c->head_stride}, {c->page_size, c->slot_stride}};
    if (!qg::rows_disjoint(dims, c->head_dim)) return QG_ERR_INVALID_ARG;
    out->mxfp4 = mxfp4;
    *blocks = {};
    if (mxfp4) {
        const int64_t page = c->pages > 1 ? c->scale_page_stride : 0, head = c->kv_heads > 1 ? c->scale_head_stride : 0;
        const int64_t slot = c->page_size > 1 ? c->scale_slot_stride : 0;
        if (!stride_ok(page) || !stride_ok(head) || !stride_ok(slot)) return QG_ERR_INVALID_ARG;
        qg::Dim rows[] = {{c->pages, page}, {c->kv_heads, head}, {c->page_size, slot}};
        if (!qg::rows_disjoint(rows, c->head_dim / qg::kBlock)) return QG_ERR_INVALID_ARG;
        *blocks = {c->k_block_scale, c->v_block_scale, page, head, slot};
    }
    out->k = static_cast<uint8_t*>(c->k);
    out->v = static_cast<uint8_t*>(c->v);
    out->k_scale = e4m3 ? c->k_scale : nullptr;
    out->v_scale = e4m3 ? c->v_scale : nullptr;
    out->page_stride = c->page_stride;
    out->head_stride = c->head_stride;
    out->slot_stride = c->slot_stride;
    out->pages = c->pages;
    out->kv_heads = c->kv_heads;
    out->page_shift = 0;
    while ((1 << out->page_shift) < c->page_size) ++out->page_shift;
    out->head_dim = c->head_dim;
    out->e4m3 = e4m3;
    return QG_OK;
}

}  // namespace

extern "C" {

qg_status qg_rope_init(qg_rope* rope, int32_t rot_dim, int32_t interleaved, double base, int32_t scaling,
                       double factor, int64_t original_len, double beta_fast, double beta_slow, double amplitude)
{
    if (!rope) return QG_ERR_INVALID_ARG;
    if (rot_dim < 2 || rot_dim % 2 != 0 || !(base > 1.0) || !std::isfinite(base)) return QG_ERR_INVALID_ARG;
    if (rot_dim > 2 * qg::kMaxRotPairs) return QG_ERR_UNSUPPORTED;
    if (scaling < QG_ROPE_PLAIN || scaling > QG_ROPE_YARN) return QG_ERR_UNSUPPORTED;
    if (scaling != QG_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return QG_ERR_INVALID_ARG;
    const long double two_pi = 2.0L * acosl(-1.0L);
    long double low = 0.0L, high = 0.0L;
    if (scaling == QG_ROPE_YARN) {
        if (original_len < 1 || !(beta_fast > 0.0) || !(beta_slow > 0.0) || !std::isfinite(beta_fast) ||
            !std::isfinite(beta_slow))
            return QG_ERR_INVALID_ARG;
        const auto pair_with = [&](double turns) {
            return rot_dim * logl((long double)original_len / (turns * two_pi)) / (2.0L * logl((long double)base));
        };
        low = fmaxl(floorl(pair_with(beta_fast)), 0.0L);
        high = fminl(ceill(pair_with(beta_slow)), (long double)(rot_dim - 1));
    }
    if (amplitude < 0.0 || !std::isfinite(amplitude)) return QG_ERR_INVALID_ARG;
    // 0 asks for the scaling's own amplitude
    rope->amplitude = float(amplitude > 0.0 ? amplitude : scaling == QG_ROPE_YARN ? 0.1 * log(factor) + 1.0 : 1.0);
    rope->rot_dim = rot_dim;
    rope->interleaved = interleaved != 0;
    rope->reserved = 0;
    for (int i = 0; i < qg::kMaxRotPairs; ++i) {
        if (i >= rot_dim / 2) {
            rope->turns[i] = 0;
            continue;
        }
        long double f = powl((long double)base, -2.0L * i / rot_dim);
        if (scaling == QG_ROPE_LINEAR) f /= factor;
        if (scaling == QG_ROPE_YARN) {
            const long double ramp = fminl(fmaxl((i - low) / fmaxl(high - low, 0.001L), 0.0L), 1.0L);
            f = f * (1.0L - ramp) + f / factor * ramp;
        }
        // f is at most 1, so the fraction of a turn is below 0.16
        rope->turns[i] = uint64_t(ldexpl(f / two_pi, 64) + 0.5L);
    }
    return QG_OK;
}

qg_status qg_rope_append(const qg_kv_cache* cache, const qg_rope* rope, const void* q, const void* k, const void* v,
                         int32_t src_dtype, int64_t q_token_stride, int64_t q_head_stride, int64_t k_token_stride,
                         int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride, const int32_t* pos,
                         const int64_t* slots, uint16_t* q_out, int64_t out_token_stride, int64_t out_head_stride,
                         int64_t tokens, int32_t q_heads, void* hip_stream)
{
    if (!rope || !q || !k || !v || !pos || !slots || !q_out) return QG_ERR_INVALID_ARG;
    if (tokens < 0 || tokens > kMaxCount || q_heads < 1) return QG_ERR_INVALID_ARG;
    if (q_heads > 65535 || (src_dtype != QG_SRC_F32 && src_dtype != QG_SRC_BF16)) return QG_ERR_UNSUPPORTED;
    qg::RopeParams p;
    qg::BlockView blocks;
    const qg_status st = check_cache(cache, &p.cache, &blocks);
    if (st != QG_OK) return st;
    // a dimension of one entry has no stride that matters
    if (tokens <= 1) q_token_stride = k_token_stride = v_token_stride = out_token_stride = 0;
    if (q_heads == 1) q_head_stride = out_head_stride = 0;
    if (p.cache.kv_heads == 1) k_head_stride = v_head_stride = 0;
    if (rope->rot_dim < 2 || rope->rot_dim % 2 != 0 || rope->rot_dim > p.cache.head_dim) return QG_ERR_INVALID_ARG;
    const int64_t strides[] = {q_token_stride, q_head_stride, k_token_stride, k_head_stride,
                               v_token_stride, v_head_stride, out_token_stride, out_head_stride};
    for (int64_t s : strides)
        if (!stride_ok(s)) return QG_ERR_INVALID_ARG;
    // one write per output element
    if ((tokens > 1 && out_token_stride < p.cache.head_dim) || (q_heads > 1 && out_head_stride < p.cache.head_dim))
        return QG_ERR_INVALID_ARG;
    const bool f32 = src_dtype == QG_SRC_F32;
    const uintptr_t size = f32 ? 4 : 2;
    if (!aligned(q, size) || !aligned(k, size) || !aligned(v, size) || !aligned(pos, 4) || !aligned(slots, 8) ||
        !aligned(q_out, 2))
        return QG_ERR_ALIGNMENT;
    qg::Dim dims[] = {{tokens, out_token_stride}, {q_heads, out_head_stride}};
    if (!qg::rows_disjoint(dims, p.cache.head_dim)) return QG_ERR_INVALID_ARG;
    if (tokens == 0) return QG_OK;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_token = q_token_stride;
    p.q_head = q_head_stride;
    p.k_token = k_token_stride;
    p.k_head = k_head_stride;
    p.v_token = v_token_stride;
    p.v_head = v_head_stride;
    p.q_out = q_out;
    p.o_token = out_token_stride;
    p.o_head = out_head_stride;
    p.pos = pos;
    p.slots = slots;
    p.tokens = tokens;
    p.q_heads = q_heads;
    p.rot_dim = rope->rot_dim;
    p.f32 = f32;
    p.interleaved = rope->interleaved != 0;
    p.amplitude = rope->amplitude;
    for (int i = 0; i < qg::kMaxRotPairs; ++i) p.turns[i] = rope->turns[i];
    const int64_t unit = 16 / int64_t(size);
    p.wide = aligned(q, 16) && aligned(k, 16) && aligned(v, 16) && aligned(q_out, 16);
    for (int i = 0; i < 8; ++i) p.wide = p.wide && strides[i] % (i < 6 ? unit : 8) == 0;
    (void)hipGetLastError();  // clear a stale error so the check below is ours
    return qg::launch_rope(p, blocks, static_cast<hipStream_t>(hip_stream)) == hipSuccess ? QG_OK : QG_ERR_HIP;
}

qg_status qg_kv_read(const qg_kv_cache* cache, const int64_t* slots, void* k_out, void* v_out, int32_t out_dtype,
                     int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                     int64_t tokens, void* hip_stream)
{
    if (!slots || (!k_out && !v_out)) return QG_ERR_INVALID_ARG;
    if (tokens < 0 || tokens > kMaxCount) return QG_ERR_INVALID_ARG;
    if (out_dtype != QG_SRC_F32 && out_dtype != QG_SRC_BF16) return QG_ERR_UNSUPPORTED;
    qg::ReadParams p;
    const qg_status st = check_cache(cache, &p.cache, &p.blocks);
    if (st != QG_OK) return st;
    const int64_t heads = p.cache.kv_heads, dim = p.cache.head_dim;
    p.f32 = out_dtype == QG_SRC_F32;
    p.wide = true;
    const uintptr_t size = p.f32 ? 4 : 2;
    if (!aligned(slots, 8)) return QG_ERR_ALIGNMENT;
    struct Rows {
        void* at;
        int64_t* token;
        int64_t* head;
    };
    for (const Rows& r : {Rows{k_out, &k_token_stride, &k_head_stride}, Rows{v_out, &v_token_stride, &v_head_stride}}) {
        if (!r.at) continue;
        // a dimension of one entry has no stride that matters
        if (tokens <= 1) *r.token = 0;
        if (heads == 1) *r.head = 0;
        if (!stride_ok(*r.token) || !stride_ok(*r.head)) return QG_ERR_INVALID_ARG;
        if (!aligned(r.at, size)) return QG_ERR_ALIGNMENT;
        qg::Dim dims[] = {{tokens, *r.token}, {heads, *r.head}};
        if (!qg::rows_disjoint(dims, dim)) return QG_ERR_INVALID_ARG;
        const int64_t unit = 16 / int64_t(size);
        p.wide = p.wide && aligned(r.at, 16) && *r.token % unit == 0 && *r.head % unit == 0;
    }
    if (tokens == 0) return QG_OK;
    p.slots = slots;
    p.k = k_out;
    p.v = v_out;
    p.k_token = k_token_stride;
    p.k_head = k_head_stride;
    p.v_token = v_token_stride;
    p.v_head = v_head_stride;
    p.tokens = tokens;
    (void)hipGetLastError();
    return qg::launch_read(p, static_cast<hipStream_t>(hip_stream)) == hipSuccess ? QG_OK : QG_ERR_HIP;
}

static qg_status check_attention_shape(const qg_kv_cache* cache, int64_t tokens, int32_t q_heads, int32_t seqs,
                                       int64_t max_q, int64_t max_kv, qg::CacheView* view,
                                       qg::BlockView* blocks)
{
    const qg_status st = check_cache(cache, view, blocks);
    if (st != QG_OK) return st;
    if (tokens < 0 || tokens > kMaxCount || seqs < 0 || max_q < 0 || max_q > kMaxCount || max_kv < 0 ||
        max_kv > kMaxCount || q_heads < 1 || q_heads % view->kv_heads != 0)
        return QG_ERR_INVALID_ARG;
    if (seqs > 65535 || q_heads > 32767 || max_kv > kMaxCachedTokens || tokens * q_heads > kMaxCount)
        return QG_ERR_UNSUPPORTED;
    return QG_OK;
}

size_t qg_paged_attention_workspace_size(const qg_kv_cache* cache, int64_t tokens, int32_t q_heads, int32_t seqs,
                                         int64_t max_q, int64_t max_kv)
{
    qg::CacheView view;
    qg::BlockView blocks;
    if (check_attention_shape(cache, tokens, q_heads, seqs, max_q, max_kv, &view, &blocks) != QG_OK) return 0;
    return qg::attention_workspace_bytes(view, blocks, tokens, q_heads, seqs, max_q, max_kv);
}

qg_status qg_paged_attention(const qg_kv_cache* cache, const uint16_t* q_bf16, int64_t q_token_stride,
                             int64_t q_head_stride, uint16_t* out_bf16, int64_t out_token_stride,
                             int64_t out_head_stride, float* lse, int64_t lse_token_stride, const int32_t* q_start,
                             const int32_t* kv_len, const int32_t* page_table, int64_t table_stride,
                             int64_t table_cols, int64_t tokens, int32_t q_heads, int32_t seqs, int64_t max_q,
                             int64_t max_kv, float scale, int64_t window, void* workspace, size_t workspace_bytes,
                             void* hip_stream)
{
    if (!q_bf16 || !out_bf16 || !q_start || !kv_len || !page_table || !workspace) return QG_ERR_INVALID_ARG;
    qg::AttnParams p;
    const qg_status st = check_attention_shape(cache, tokens, q_heads, seqs, max_q, max_kv, &p.cache, &p.blocks);
    if (st != QG_OK) return st;
    // a dimension of one entry has no stride that matters
    if (tokens <= 1) q_token_stride = out_token_stride = lse_token_stride = 0;
    if (q_heads == 1) q_head_stride = out_head_stride = 0;
    if (seqs <= 1) table_stride = 0;
    if (table_cols < 0 || table_cols > kMaxCount || !stride_ok(table_stride) || window < 0 || !std::isfinite(scale))
        return QG_ERR_INVALID_ARG;
    if (!stride_ok(q_token_stride) || !stride_ok(q_head_stride) || !stride_ok(out_token_stride) ||
        !stride_ok(out_head_stride) || !stride_ok(lse_token_stride))
        return QG_ERR_INVALID_ARG;
    if ((tokens > 1 && out_token_stride < p.cache.head_dim) || (q_heads > 1 && out_head_stride < p.cache.head_dim) ||
        (lse && tokens > 1 && lse_token_stride < q_heads))
        return QG_ERR_INVALID_ARG;
    if (!aligned(q_bf16, 16) || q_token_stride % 8 != 0 || q_head_stride % 8 != 0 || !aligned(out_bf16, 8) ||
        out_token_stride % 4 != 0 || out_head_stride % 4 != 0 || (lse && !aligned(lse, 4)) || !aligned(q_start, 4) ||
        !aligned(kv_len, 4) || !aligned(page_table, 4) || !aligned(workspace, 16))
        return QG_ERR_ALIGNMENT;
    qg::Dim dims[] = {{tokens, out_token_stride}, {q_heads, out_head_stride}};
    if (!qg::rows_disjoint(dims, p.cache.head_dim)) return QG_ERR_INVALID_ARG;
    if (tokens == 0 || seqs == 0 || max_q == 0) return QG_OK;
    if (workspace_bytes < qg::attention_workspace_need(p.cache, p.blocks, tokens, q_heads, seqs, max_q, max_kv))
        return QG_ERR_INVALID_ARG;
    p.q = q_bf16;
    p.q_token = q_token_stride;
    p.q_head = q_head_stride;
    p.out = out_bf16;
    p.o_token = out_token_stride;
    p.o_head = out_head_stride;
    p.lse = lse;
    p.lse_token = lse_token_stride;
    p.q_start = q_start;
    p.kv_len = kv_len;
    p.table = page_table;
    p.table_stride = table_stride;
    p.table_cols = table_cols;
    p.tokens = tokens;
    p.max_q = max_q < tokens ? max_q : tokens;
    p.max_kv = max_kv;
    p.window = window;
    p.seqs = seqs;
    p.q_heads = q_heads;
    p.group = q_heads / p.cache.kv_heads;
    p.scale = scale;
    p.workspace = workspace;
    (void)hipGetLastError();
    return qg::launch_attention(p, static_cast<hipStream_t>(hip_stream)) == hipSuccess ? QG_OK : QG_ERR_HIP;
}

size_t qg_sample_workspace_size(int64_t m, int64_t N)
{
    if (m < 0 || m > 65535 || N < 1 || N > kMaxCount) return 0;
    return qg::sample_workspace_bytes(m, N);
}

qg_status qg_sample_f32(const float* logits, int64_t m, int64_t N, int64_t ldx, const float* u,
                        const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                        int32_t* idx_out, void* workspace, size_t workspace_bytes, void* hip_stream)
{
    if (!logits || !u || !idx_out || !workspace) return QG_ERR_INVALID_ARG;
    if (m == 0) return QG_OK;
    if (m < 0 || m > 65535 || N < 1 || N > kMaxCount || ldx < N || ldx > kMaxStride) return QG_ERR_INVALID_ARG;
    if (workspace_bytes < qg::sample_workspace_need(m, N)) return QG_ERR_INVALID_ARG;
    if (!aligned(logits, 4) || !aligned(u, 4) || !aligned(idx_out, 4) || !aligned(workspace, 16) ||
        (temperature && !aligned(temperature, 4)) || (top_k && !aligned(top_k, 4)) || (top_p && !aligned(top_p, 4)) ||
        (min_p && !aligned(min_p, 4)))
        return QG_ERR_ALIGNMENT;
    qg::SampleParams p;
    p.x = logits;
    p.m = m;
    p.N = N;
    p.ldx = ldx;
    p.u = u;
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p;
    p.min_p = min_p;
    p.idx = idx_out;
    p.workspace = workspace;
    (void)hipGetLastError();
    return qg::launch_sample(p, static_cast<hipStream_t>(hip_stream)) == hipSuccess ? QG_OK : QG_ERR_HIP;
}

}  // extern "C"
