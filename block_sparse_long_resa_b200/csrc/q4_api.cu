// Host side of the rotary appends and of the 4-bit cache's entry points:
// argument validation and launches (include/resa.h).
#include "api_common.cuh"
#include "q4_common.cuh"

namespace resa {
namespace {

constexpr int kMaxGridBatch = 65535;  // sequences along a grid's y

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The checks of check_cache on a 4-bit cache.
resa_status_t check_cache_q4(const resa_cache_q4_t *c, Shape *s, bool need_desc, Q4Cache *q4) {
    if (!c) return RESA_ERR_NULL;
    if (!c->v || !c->k_sf || !c->v_sf) return RESA_ERR_NULL;
    resa_cache_t as{};
    as.k = c->k;
    as.v = c->v;
    as.desc = c->desc;
    as.page_table = c->page_table;
    as.seq_len = c->seq_len;
    as.batch = c->batch;
    as.max_pages = c->max_pages;
    as.num_pages = c->num_pages;
    as.rows = c->rows;
    as.table_rows = c->table_rows;
    RESA_TRY(check_cache(&as, s, true, need_desc));
    if (!aligned16(c->k_sf) || !aligned16(c->v_sf) || !aligned4(c->k_scale) ||
        !aligned4(c->v_scale))
        return RESA_ERR_UNSUPPORTED;
    q4->k = static_cast<uint8_t *>(c->k);
    q4->v = static_cast<uint8_t *>(c->v);
    q4->k_sf = static_cast<uint8_t *>(c->k_sf);
    q4->v_sf = static_cast<uint8_t *>(c->v_sf);
    q4->k_scale = c->k_scale;
    q4->v_scale = c->v_scale;
    return RESA_OK;
}

// Rotation and fresh tokens into the kernel's arguments.
resa_status_t check_append(const Shape &s, const resa_rope_t *rope, const resa_tokens_t *t,
                           void *q_out, AppendArgs *a) {
    if (!rope || !t) return RESA_ERR_NULL;
    if (!t->k || !t->v || (t->q != nullptr) != (q_out != nullptr)) return RESA_ERR_NULL;
    if (rope->rot_dim < 0 || rope->rot_dim > s.d) return RESA_ERR_RANGE;
    if (rope->rot_dim % 16 != 0) return RESA_ERR_UNSUPPORTED;
    if (rope->rot_dim > 0 && !rope->inv_freq) return RESA_ERR_NULL;
    if (!isfinite(rope->mscale)) return RESA_ERR_RANGE;
    if (t->f < 1) return RESA_ERR_RANGE;
    if (s.batch > kMaxGridBatch) return RESA_ERR_UNSUPPORTED;
    const long long q_row = (long long)s.hq * s.d, kv_row = (long long)s.hkv * s.d;
    a->q_stride = t->q_stride ? t->q_stride : q_row;
    a->k_stride = t->k_stride ? t->k_stride : kv_row;
    a->v_stride = t->v_stride ? t->v_stride : kv_row;
    if ((t->q && a->q_stride < q_row) || a->k_stride < kv_row || a->v_stride < kv_row)
        return RESA_ERR_SHAPE;
    if (a->q_stride % 8 || a->k_stride % 8 || a->v_stride % 8) return RESA_ERR_UNSUPPORTED;
    if (t->q && q_out == t->q && a->q_stride != q_row) return RESA_ERR_SHAPE;
    if (!aligned16(t->q) || !aligned16(q_out) || !aligned16(t->k) || !aligned16(t->v) ||
        !aligned4(rope->inv_freq) || !aligned4(t->n_new) || !aligned4(t->positions))
        return RESA_ERR_UNSUPPORTED;
    a->q = t->q;
    a->kn = t->k;
    a->vn = t->v;
    a->q_out = q_out;
    a->n_new = t->n_new;
    a->positions = t->positions;
    a->inv_freq = rope->inv_freq;
    a->mscale = rope->mscale != 0.f ? (double)rope->mscale : 1.0;
    a->f = t->f;
    a->rot = rope->rot_dim;
    a->interleaved = rope->interleaved != 0;
    return RESA_OK;
}

}  // namespace
}  // namespace resa

using namespace resa;

extern "C" {

resa_status_t resa_append_rope(const resa_config_t *cfg, const resa_cache_t *cache,
                               const resa_rope_t *rope, const resa_tokens_t *tokens, void *q_out,
                               void *ws, size_t ws_bytes, cudaStream_t stream) {
    Shape s{};
    AppendArgs a{};
    RESA_TRY(check_config(cfg, &s));
    RESA_TRY(check_cache(cache, &s, true, true));
    RESA_TRY(check_append(s, rope, tokens, q_out, &a));
    const WsLayout w = layout_of(s, 0);
    RESA_TRY(check_ws(ws, ws_bytes, w));
    a.k = cache->k;
    a.v = cache->v;
    a.desc = cache->desc;
    a.page_table = cache->page_table;
    a.seq_len = cache->seq_len;
    return cuda_status(launch_append_rope(s, a, false, at<uint32_t>(ws, w.err), stream));
}

resa_status_t resa_append_rope_q4(const resa_config_t *cfg, const resa_cache_q4_t *cache,
                                  const resa_rope_t *rope, const resa_tokens_t *tokens,
                                  void *q_out, void *ws, size_t ws_bytes, cudaStream_t stream) {
    Shape s{};
    Q4Cache c{};
    AppendArgs a{};
    RESA_TRY(check_config(cfg, &s));
    RESA_TRY(check_cache_q4(cache, &s, true, &c));
    RESA_TRY(check_append(s, rope, tokens, q_out, &a));
    const WsLayout w = layout_of(s, 0);
    RESA_TRY(check_ws(ws, ws_bytes, w));
    a.k = c.k;
    a.v = c.v;
    a.k_sf = c.k_sf;
    a.v_sf = c.v_sf;
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    a.desc = cache->desc;
    a.page_table = cache->page_table;
    a.seq_len = cache->seq_len;
    return cuda_status(launch_append_rope(s, a, true, at<uint32_t>(ws, w.err), stream));
}

resa_status_t resa_expand_q4(const resa_config_t *cfg, const resa_cache_q4_t *cache, void *k_out,
                             void *v_out, void *ws, size_t ws_bytes, cudaStream_t stream) {
    Shape s{};
    Q4Cache c{};
    RESA_TRY(check_config(cfg, &s));
    RESA_TRY(check_cache_q4(cache, &s, false, &c));
    if (!k_out || !v_out) return RESA_ERR_NULL;
    if (s.batch > kMaxGridBatch) return RESA_ERR_UNSUPPORTED;
    if (!aligned16(k_out) || !aligned16(v_out)) return RESA_ERR_UNSUPPORTED;
    const WsLayout w = layout_of(s, 0);
    RESA_TRY(check_ws(ws, ws_bytes, w));
    return cuda_status(launch_expand_q4(s, c, cache->page_table, cache->seq_len, k_out, v_out,
                                        at<uint32_t>(ws, w.err), stream));
}

resa_status_t resa_sparse_decode_q4(const resa_config_t *cfg, const resa_cache_q4_t *cache,
                                    const void *q, const int32_t *block_idx,
                                    const int32_t *block_cnt, int32_t max_topk, float *out,
                                    float *lse_opt, void *ws, size_t ws_bytes,
                                    cudaStream_t stream) {
    Shape s{};
    Q4Cache c{};
    RESA_TRY(check_config(cfg, &s));
    RESA_TRY(check_cache_q4(cache, &s, false, &c));
    if (!q || !block_idx || !block_cnt || !out) return RESA_ERR_NULL;
    if (max_topk < 0 || (long long)s.batch * s.hkv * ((long long)max_topk + 1) > 0x7fffffffLL)
        return RESA_ERR_RANGE;
    if (!aligned16(q) || !aligned16(out) || !aligned4(block_idx) || !aligned4(block_cnt) ||
        !aligned4(lse_opt))
        return RESA_ERR_UNSUPPORTED;
    const WsLayout w = layout_of(s, 0);
    RESA_TRY(check_ws(ws, ws_bytes, w));
    return cuda_status(launch_decode_q4(s, c, cache->page_table, cache->seq_len, q, 1, nullptr,
                                        block_idx, block_cnt, max_topk, sm_count(),
                                        at<float>(ws, w.dec_o), at<float>(ws, w.dec_lse),
                                        at<uint32_t>(ws, w.err + kDecBarrierOffset), out, lse_opt,
                                        at<uint32_t>(ws, w.err), stream));
}

resa_status_t resa_attention_q4(const resa_config_t *cfg, const resa_cache_q4_t *cache, int32_t f,
                                const int32_t *n_new_opt, const void *q, float *out,
                                float *lse_opt, void *ws, size_t ws_bytes, cudaStream_t stream) {
    Shape s{};
    Q4Cache c{};
    RESA_TRY(check_config(cfg, &s));
    RESA_TRY(check_cache_q4(cache, &s, false, &c));
    if (!q || !out) return RESA_ERR_NULL;
    if (f < 1) return RESA_ERR_RANGE;
    if (f > kMaxRowTiles * kRectRowsPerCta) return RESA_ERR_UNSUPPORTED;
    if (rect_row_groups(f, s.g) > kMaxRowTiles) return RESA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(out) || !aligned4(n_new_opt) || !aligned4(lse_opt))
        return RESA_ERR_UNSUPPORTED;
    WsLayout w = layout_of(s, 0);
    const bool chunk = f * s.g > kMaxGroup;
    const int units = (int)((long long)s.batch * s.hkv * rect_row_groups(f, s.g) < kNumSms
                                ? s.batch * s.hkv * rect_row_groups(f, s.g) : kNumSms);
    if (chunk) w.total = w.rect_o + chunk_q4_bytes(units, s.d);
    RESA_TRY(check_ws(ws, ws_bytes, w));
    if ((long long)s.batch * s.hkv * rect_row_groups(f, s.g) > 0x7fffffffLL / s.max_pages)
        return RESA_ERR_RANGE;  // entries of work are counted in 32 bits
    uint32_t *err = at<uint32_t>(ws, w.err);
    if (!chunk)
        return cuda_status(launch_decode_q4(s, c, cache->page_table, cache->seq_len, q, f, n_new_opt,
                                            nullptr, nullptr, 0, sm_count(), at<float>(ws, w.dec_o),
                                            at<float>(ws, w.dec_lse), at<uint32_t>(ws, w.err + kDecBarrierOffset),
                                            out, lse_opt, err, stream));
    return cuda_status(launch_chunk_q4(s, c, cache->page_table, cache->seq_len, q, f, n_new_opt,
                                       sm_count(), at<float>(ws, w.rect_o),
                                       at<float>(ws, w.rect_o) + chunk_q4_partial_floats(units, s.d),
                                       at<uint32_t>(ws, w.rect_ticket), out, lse_opt, err, stream));
}

}  // extern "C"
