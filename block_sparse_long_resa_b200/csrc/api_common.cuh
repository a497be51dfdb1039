// Host-side argument checks shared by the files that define entry points.
#pragma once

#include <math.h>

#include "resa_common.cuh"

namespace resa {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline resa_status_t check_config(const resa_config_t *cfg, Shape *s) {
    if (!cfg) return RESA_ERR_NULL;
    if (cfg->num_q_heads <= 0 || cfg->num_kv_heads <= 0 || cfg->head_dim <= 0 ||
        cfg->block_size <= 0)
        return RESA_ERR_SHAPE;
    if (cfg->num_q_heads % cfg->num_kv_heads != 0) return RESA_ERR_SHAPE;
    const int g = cfg->num_q_heads / cfg->num_kv_heads;
    if (g > kMaxGroup) return RESA_ERR_UNSUPPORTED;
    const int hkv = cfg->num_kv_heads;
    if (!(hkv == 1 || hkv == 2 || hkv == 4 || hkv == 8)) return RESA_ERR_UNSUPPORTED;
    if (!(cfg->head_dim == 64 || cfg->head_dim == 128)) return RESA_ERR_UNSUPPORTED;
    if (!(cfg->block_size == 16 || cfg->block_size == 32 || cfg->block_size == 64))
        return RESA_ERR_UNSUPPORTED;
    if (!(cfg->sm_scale >= 0.f) || isinf(cfg->sm_scale)) return RESA_ERR_RANGE;
    s->hq = cfg->num_q_heads;
    s->hkv = hkv;
    s->g = g;
    s->d = cfg->head_dim;
    s->bs = cfg->block_size;
    s->sm_scale = cfg->sm_scale > 0.f ? cfg->sm_scale : 1.0f / sqrtf((float)cfg->head_dim);
    return RESA_OK;
}

inline resa_status_t check_cache(const resa_cache_t *c, Shape *s, bool need_v, bool need_desc) {
    if (!c) return RESA_ERR_NULL;
    if (!c->k || !c->page_table || !c->seq_len) return RESA_ERR_NULL;
    if (need_v && !c->v) return RESA_ERR_NULL;
    if (need_desc && !c->desc) return RESA_ERR_NULL;
    if (c->batch <= 0 || c->max_pages <= 0 || c->num_pages <= 0) return RESA_ERR_SHAPE;
    if ((long long)c->max_pages * s->bs > 0x7fffffffLL) return RESA_ERR_RANGE;
    if ((long long)c->num_pages * s->hkv * s->bs > 0x7fffffffLL) return RESA_ERR_RANGE;
    if (!aligned16(c->k) || (c->v && !aligned16(c->v)) || (c->desc && !aligned16(c->desc)) ||
        !aligned16(c->page_table) || !aligned16(c->seq_len))
        return RESA_ERR_UNSUPPORTED;
    if (c->rows != nullptr && (c->table_rows <= 0 || !aligned16(c->rows)))
        return c->table_rows <= 0 ? RESA_ERR_SHAPE : RESA_ERR_UNSUPPORTED;
    s->batch = c->batch;
    s->max_pages = c->max_pages;
    s->num_pages = c->num_pages;
    s->rows = RowMap{c->rows, c->rows ? c->table_rows : c->batch};
    return RESA_OK;
}

inline resa_status_t check_ws(void *ws, size_t ws_bytes, const WsLayout &w) {
    if (!ws) return RESA_ERR_NULL;
    if (!aligned16(ws)) return RESA_ERR_UNSUPPORTED;
    if (ws_bytes < w.total) return RESA_ERR_SHAPE;
    return RESA_OK;
}

template <typename T>
T *at(void *ws, size_t off) {
    return reinterpret_cast<T *>(static_cast<uint8_t *>(ws) + off);
}

inline resa_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? RESA_OK : RESA_ERR_CUDA; }

#define RESA_TRY(expr)                        \
    do {                                      \
        resa_status_t _st = (expr);           \
        if (_st != RESA_OK) return _st;       \
    } while (0)

inline WsLayout layout_of(const Shape &s, int chunk) {
    return ws_layout(s.hq, s.hkv, s.d, s.bs, s.batch, s.max_pages, chunk);
}

inline int sm_count() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int c = cache[dev].load();
    if (c == 0) {
        if (cudaDeviceGetAttribute(&c, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cache[dev].store(c);
    }
    return c;
}

}  // namespace resa
