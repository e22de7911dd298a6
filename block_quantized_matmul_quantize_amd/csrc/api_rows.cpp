// C ABI of the row operators (embedding, expert sort / gather / combine, low-rank adapters):
// argument checks and launches.  The contract of every entry point is in include/qmm.h.
#include "../../include/qmm.h"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "launch.hpp"

namespace {

constexpr int64_t kMaxLen = 1 << 20;      // row lengths
constexpr int64_t kMaxCount = 1 << 30;    // rows, pairs, ids

qmm_status fail(qmm_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
qmm_status fail(qmm_status st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return qmm::report(st, buf);
}

qmm_status done(hipError_t e, const char *what) {
    return e == hipSuccess ? QMM_OK : fail(QMM_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

int elem(int type) { return type == QMM_F32 ? 4 : type == QMM_F16 || type == QMM_BF16 ? 2 : 0; }
int block_values(int type) {
    switch (type) {
        case QMM_Q4_K: case QMM_Q5_K: case QMM_Q6_K: case QMM_Q3_K: case QMM_IQ4_XS: return 256;
        case QMM_Q8_0: case QMM_Q4_0: return 32;
        default: return 0;
    }
}

// null, or at a multiple of `to` bytes
bool at(const void *p, size_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

qmm_status need_elem(int type, const char *name) {
    if (elem(type)) return QMM_OK;
    return fail(QMM_ERR_TYPE, "%s %d is no element type (F32=0, F16=1, BF16=30)", name, type);
}
qmm_status need_len(int64_t v, const char *name) {
    if (v < 1) return fail(QMM_ERR_ARG, "%s must be >= 1 (got %lld)", name, (long long)v);
    if (v > kMaxLen) return fail(QMM_ERR_SHAPE, "%s=%lld exceeds the supported maximum %lld", name, (long long)v,
                                 (long long)kMaxLen);
    return QMM_OK;
}
qmm_status need_count(int64_t v, int64_t least, const char *name) {
    if (v < least) return fail(QMM_ERR_ARG, "%s must be >= %lld (got %lld)", name, (long long)least, (long long)v);
    if (v > kMaxCount) return fail(QMM_ERR_SHAPE, "%s=%lld exceeds the supported maximum %lld", name, (long long)v,
                                   (long long)kMaxCount);
    return QMM_OK;
}
qmm_status need_ws(const void *ws, size_t have, size_t need) {
    if (need == 0) return QMM_OK;
    if (!ws || have < need) return fail(QMM_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", ws ? have : (size_t)0, need);
    if (!at(ws, 256)) return fail(QMM_ERR_ARG, "the workspace must be 256-byte aligned");
    return QMM_OK;
}
#define TRY(call)                          \
    do {                                   \
        if (qmm_status st_ = (call)) return st_; \
    } while (0)

// Shape of the (token, slot) operators.
qmm_status need_pairs(int type, int64_t n_tok, int64_t top_k, int64_t k) {
    TRY(need_elem(type, "type"));
    TRY(need_count(n_tok, 0, "n_tok"));
    TRY(need_count(top_k, 1, "top_k"));
    TRY(need_len(k, "k"));
    if (n_tok > kMaxCount / top_k)
        return fail(QMM_ERR_SHAPE, "n_tok * top_k exceeds the supported maximum %lld", (long long)kMaxCount);
    return QMM_OK;
}

// Both forms of the combine: pos of places, or of ids in [0, n_ids).
qmm_status need_ids(const int32_t *ids, int64_t n_ids, int64_t n_tok) {
    TRY(need_count(n_ids, 1, "n_ids"));
    return ids || n_tok == 0 ? QMM_OK : fail(QMM_ERR_ARG, "null ids");
}
qmm_status combine(int type, const void *h, int64_t n_tok, int64_t top_k, int64_t k, const int32_t *pos,
                   int64_t n_ids, const float *w, const void *base, void *y, void *stream, const char *what) {
    if (n_tok == 0) return QMM_OK;
    if (!h || !y) return fail(QMM_ERR_ARG, "null h or y");
    if (h == y) return fail(QMM_ERR_ARG, "y must not be h");
    if (!at(h, elem(type)) || !at(y, elem(type)) || !at(base, elem(type)) || !at(pos, 4) || !at(w, 4))
        return fail(QMM_ERR_ARG, "h, y, base, w and the places or ids must be aligned to their elements");
    return done(qmm::launch_combine(type, h, n_tok, top_k, k, pos, n_ids, w, base, y, (hipStream_t)stream), what);
}
qmm_status combine_backward(int type, const void *dy, const void *h, int64_t n_tok, int64_t top_k, int64_t k,
                            const int32_t *pos, int64_t n_ids, const float *w, const int32_t *n_valid, void *dh,
                            float *dw, void *stream, const char *what) {
    if (n_tok == 0) return QMM_OK;
    if (!dy || !h || !dh || !dw) return fail(QMM_ERR_ARG, "null dy, h, dh or dw");
    if (dh == dy || dh == h) return fail(QMM_ERR_ARG, "dh must not be dy or h");
    if (!at(dy, elem(type)) || !at(h, elem(type)) || !at(dh, elem(type)) || !at(pos, 4) || !at(w, 4) || !at(dw, 4) ||
        !at(n_valid, 4))
        return fail(QMM_ERR_ARG, "dy, h, dh, dw, w, n_valid and the places or ids must be aligned to their elements");
    return done(qmm::launch_combine_backward(type, dy, h, n_tok, top_k, k, pos, n_ids, w, n_valid, dh, dw,
                                             (hipStream_t)stream), what);
}

qmm_status need_lora(int64_t n, int64_t k, int64_t rows, int64_t rank, int64_t n_adapters) {
    TRY(need_count(n, 0, "n"));
    TRY(need_len(k, "k"));
    TRY(need_len(rows, "rows"));
    if (rank < 1) return fail(QMM_ERR_ARG, "rank must be >= 1 (got %lld)", (long long)rank);
    if (rank > 128) return fail(QMM_ERR_SHAPE, "rank=%lld exceeds the supported maximum 128", (long long)rank);
    if (n_adapters < 1) return fail(QMM_ERR_ARG, "n_adapters must be >= 1 (got %lld)", (long long)n_adapters);
    if (n_adapters > kMaxLen || n_adapters * rank > ((int64_t)1 << 40) / (k > rows ? k : rows))
        return fail(QMM_ERR_SHAPE, "n_adapters=%lld of rank %lld are too large", (long long)n_adapters, (long long)rank);
    return QMM_OK;
}
qmm_status need_lora_types(int x_type, int w_type) {
    TRY(need_elem(x_type, "x_type"));
    TRY(need_elem(w_type, "w_type"));
    if (x_type != QMM_F32 && w_type != x_type)
        return fail(QMM_ERR_TYPE, "w_type %d beside x_type %d: it must be the same, or x fp32", w_type, x_type);
    return QMM_OK;
}
bool sort_ok(int64_t n, int64_t n_keys) { return n >= 0 && n <= kMaxCount && n_keys >= 1 && n_keys <= kMaxCount; }

}  // namespace

extern "C" {

size_t qmm_sort_ids_workspace(int64_t n, int64_t n_keys) {
    return sort_ok(n, n_keys) ? qmm::sort_ids_bytes(n, n_keys, false) : 0;
}

qmm_status qmm_sort_ids(const int32_t *ids, int64_t n, int64_t n_keys, int32_t *order, int32_t *pos, int32_t *bounds,
                        void *ws, size_t ws_bytes, void *stream) {
    TRY(need_count(n, 0, "n"));
    TRY(need_count(n_keys, 1, "n_keys"));
    if (!bounds || (n > 0 && (!ids || !order))) return fail(QMM_ERR_ARG, "null ids, order or bounds");
    if (!at(ids, 4) || !at(order, 4) || !at(pos, 4) || !at(bounds, 4))
        return fail(QMM_ERR_ARG, "ids, order, pos and bounds must be 4-byte aligned");
    TRY(need_ws(ws, ws_bytes, qmm::sort_ids_bytes(n, n_keys, false)));
    return done(qmm::launch_sort_ids(ids, n, n_keys, order, pos, bounds, false, (uint8_t *)ws, (hipStream_t)stream),
                "qmm_sort_ids");
}

qmm_status qmm_gather_sorted(int type, const void *x, int64_t n_tok, int64_t top_k, int64_t k, const int32_t *pos,
                             const int32_t *n_valid, void *y, void *stream) {
    TRY(need_pairs(type, n_tok, top_k, k));
    if (n_tok == 0) return QMM_OK;
    if (!x || !pos || !n_valid || !y) return fail(QMM_ERR_ARG, "null x, pos, n_valid or y");
    if (x == y) return fail(QMM_ERR_ARG, "y must not be x");
    if (!at(x, elem(type)) || !at(y, elem(type)) || !at(pos, 4) || !at(n_valid, 4))
        return fail(QMM_ERR_ARG, "x, y, pos and n_valid must be aligned to their elements");
    return done(qmm::launch_gather_sorted(type, x, n_tok, top_k, k, pos, n_valid, y, (hipStream_t)stream),
                "qmm_gather_sorted");
}

qmm_status qmm_combine(int type, const void *h, int64_t n_tok, int64_t top_k, int64_t k, const int32_t *pos,
                       const float *w, const void *base, void *y, void *stream) {
    TRY(need_pairs(type, n_tok, top_k, k));
    return combine(type, h, n_tok, top_k, k, pos, 0, w, base, y, stream, "qmm_combine");
}

qmm_status qmm_combine_ids(int type, const void *h, int64_t n_tok, int64_t top_k, int64_t k, const int32_t *ids,
                           int64_t n_ids, const float *w, const void *base, void *y, void *stream) {
    TRY(need_pairs(type, n_tok, top_k, k));
    TRY(need_ids(ids, n_ids, n_tok));
    return combine(type, h, n_tok, top_k, k, ids, n_ids, w, base, y, stream, "qmm_combine_ids");
}

qmm_status qmm_combine_backward(int type, const void *dy, const void *h, int64_t n_tok, int64_t top_k, int64_t k,
                                const int32_t *pos, const float *w, const int32_t *n_valid, void *dh, float *dw,
                                void *stream) {
    TRY(need_pairs(type, n_tok, top_k, k));
    if (n_tok > 0 && pos && !n_valid) return fail(QMM_ERR_ARG, "null n_valid");
    return combine_backward(type, dy, h, n_tok, top_k, k, pos, 0, w, n_valid, dh, dw, stream, "qmm_combine_backward");
}

qmm_status qmm_combine_ids_backward(int type, const void *dy, const void *h, int64_t n_tok, int64_t top_k, int64_t k,
                                    const int32_t *ids, int64_t n_ids, const float *w, void *dh, float *dw,
                                    void *stream) {
    TRY(need_pairs(type, n_tok, top_k, k));
    TRY(need_ids(ids, n_ids, n_tok));
    return combine_backward(type, dy, h, n_tok, top_k, k, ids, n_ids, w, nullptr, dh, dw, stream,
                            "qmm_combine_ids_backward");
}

qmm_status qmm_embed(int type, const void *table, int64_t vocab, int64_t k, const int32_t *ids, int64_t n, float scale,
                     int y_type, void *y, void *stream) {
    const int qk = block_values(type);
    if (!qk && !elem(type)) return fail(QMM_ERR_TYPE, "unsupported table type %d", type);
    TRY(need_elem(y_type, "y_type"));
    TRY(need_count(vocab, 1, "vocab"));
    TRY(need_count(n, 0, "n"));
    TRY(need_len(k, "k"));
    if (qk && k % qk) return fail(QMM_ERR_SHAPE, "k=%lld is not a positive multiple of the block size %d", (long long)k, qk);
    if (n == 0) return QMM_OK;
    if (!table || !ids || !y) return fail(QMM_ERR_ARG, "null table, ids or y");
    // rows of blocks hold a multiple of 8 values and y's are written 8 at a time
    if (!at(table, qk ? 2 : elem(type)) || !at(ids, 4) || !at(y, qk ? 16 : elem(y_type)))
        return fail(QMM_ERR_ARG, "table, ids and y must be aligned to their elements (blocks 2 bytes, their y 16)");
    return done(qmm::launch_embed(type, table, vocab, k, ids, n, scale, y_type, y, (hipStream_t)stream), "qmm_embed");
}

size_t qmm_embed_backward_workspace(int64_t n, int64_t k, int64_t vocab) {
    return sort_ok(n, vocab) && k >= 1 && k <= kMaxLen ? qmm::embed_backward_bytes(n, k, vocab) : 0;
}

qmm_status qmm_embed_backward(int dy_type, const void *dy, int64_t n, int64_t k, const int32_t *ids, int64_t vocab,
                              float scale, int g_type, void *grad, void *ws, size_t ws_bytes, void *stream) {
    TRY(need_elem(dy_type, "dy_type"));
    TRY(need_elem(g_type, "g_type"));
    TRY(need_count(n, 0, "n"));
    TRY(need_count(vocab, 1, "vocab"));
    TRY(need_len(k, "k"));
    if (!grad || (n > 0 && (!dy || !ids))) return fail(QMM_ERR_ARG, "null dy, ids or grad");
    if (!at(dy, elem(dy_type)) || !at(ids, 4) || !at(grad, elem(g_type)))
        return fail(QMM_ERR_ARG, "dy, ids and grad must be aligned to their elements");
    TRY(need_ws(ws, ws_bytes, qmm::embed_backward_bytes(n, k, vocab)));
    return done(qmm::launch_embed_backward(dy_type, dy, n, k, ids, vocab, scale, g_type, grad, (uint8_t *)ws,
                                           (hipStream_t)stream), "qmm_embed_backward");
}

size_t qmm_lora_workspace(int64_t n, int64_t k, int64_t rows, int64_t rank, int64_t n_adapters) {
    return need_lora(n, k, rows, rank, n_adapters) ? 0 : qmm::lora_bytes(n, k, rows, rank, n_adapters);
}

qmm_status qmm_lora(int x_type, int w_type, const void *x, int64_t n, int64_t k, const void *a, const void *b,
                    int64_t rows, int64_t rank, int64_t n_adapters, const int32_t *ids, const float *scale,
                    const void *base, void *y, float *h, void *ws, size_t ws_bytes, void *stream) {
    TRY(need_lora_types(x_type, w_type));
    TRY(need_lora(n, k, rows, rank, n_adapters));
    if (n == 0) return QMM_OK;
    if (!x || !a || !b || !ids || !y) return fail(QMM_ERR_ARG, "null x, a, b, ids or y");
    if (y == x) return fail(QMM_ERR_ARG, "y must not be x");
    if (!at(x, elem(x_type)) || !at(base, elem(x_type)) || !at(y, elem(x_type)) || !at(a, elem(w_type)) ||
        !at(b, elem(w_type)) || !at(ids, 4) || !at(scale, 4) || !at(h, 4))
        return fail(QMM_ERR_ARG, "every array must be aligned to its elements");
    TRY(need_ws(ws, ws_bytes, qmm::lora_bytes(n, k, rows, rank, n_adapters)));
    const qmm::LoraCall c{x_type, w_type, x, n, k, a, b, rows, rank, n_adapters, ids, scale};
    return done(qmm::launch_lora(c, base, y, h, (uint8_t *)ws, (hipStream_t)stream), "qmm_lora");
}

size_t qmm_lora_backward_workspace(int64_t n, int64_t k, int64_t rows, int64_t rank, int64_t n_adapters) {
    return need_lora(n, k, rows, rank, n_adapters) ? 0 : qmm::lora_backward_bytes(n, k, rows, rank, n_adapters);
}

qmm_status qmm_lora_backward(int x_type, int w_type, const void *x, const void *dy, const float *h, int64_t n,
                             int64_t k, const void *a, const void *b, int64_t rows, int64_t rank, int64_t n_adapters,
                             const int32_t *ids, const float *scale, const void *dx_base, void *dx, float *da,
                             float *db, void *ws, size_t ws_bytes, void *stream) {
    TRY(need_lora_types(x_type, w_type));
    TRY(need_lora(n, k, rows, rank, n_adapters));
    if (n > 0 && (!dy || !ids || ((dx || da) && !b) || (dx && !a) || (da && !x) || (db && !h)))
        return fail(QMM_ERR_ARG, "null x, dy, h, a, b or ids");
    if (dx && (dx == x || dx == dy)) return fail(QMM_ERR_ARG, "dx must not be x or dy");
    if (!at(x, elem(x_type)) || !at(dy, elem(x_type)) || !at(dx_base, elem(x_type)) || !at(dx, elem(x_type)) ||
        !at(a, elem(w_type)) || !at(b, elem(w_type)) || !at(ids, 4) || !at(scale, 4) || !at(h, 4) || !at(da, 4) ||
        !at(db, 4))
        return fail(QMM_ERR_ARG, "every array must be aligned to its elements");
    if (!(dx && n > 0) && !da && !db) return QMM_OK;
    TRY(need_ws(ws, ws_bytes, qmm::lora_backward_bytes(n, k, rows, rank, n_adapters)));
    const qmm::LoraCall c{x_type, w_type, x, n, k, a, b, rows, rank, n_adapters, ids, scale};
    return done(qmm::launch_lora_backward(c, dy, h, dx_base, dx, da, db, (uint8_t *)ws, (hipStream_t)stream),
                "qmm_lora_backward");
}

}  // extern "C"
