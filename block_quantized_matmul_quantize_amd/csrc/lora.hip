// Low-rank adapters of many requests beside a shared projection: row i with adapter c adds
// scale[c] * B[c] (A[c] x[i]) to the projection's result, and the gradients of that.  The forward pass
// is two launches (lora_narrow.hip: A x, lora_wide.hip: B h onto base); the backward pass the same two
// on dy and the transposed roles of B and A, and, on rows sorted by adapter, the gradients of A and B
// in one (lora_outer.hip).
#include "common.hpp"
#include "launch.hpp"
#include "rowtypes.hpp"

namespace qmm {

namespace {

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct Layout { size_t order, bounds, part, dh, outer, total; };
Layout layout(int64_t n, int64_t k, int64_t rows, int64_t rank, int64_t n_adapters) {
    Layout L{};
    const size_t row = (size_t)lora_padded_rank(rank) * 4;
    size_t off = up256(sort_ids_bytes(n, n_adapters, false));
    L.order = off;
    off += up256((size_t)n * 4);
    L.bounds = off;
    off += up256((size_t)(n_adapters + 1) * 4);
    L.part = off;
    off += n ? up256((size_t)lora_narrow_slices(n, rows) * n * row) : 0;
    L.dh = off;
    off += up256((size_t)n * row);
    L.outer = off;
    off += up256(lora_outer_bytes(n, k, rows, rank, n_adapters));
    L.total = off;
    return L;
}

}  // namespace

size_t lora_bytes(int64_t n, int64_t k, int64_t rows, int64_t rank, int64_t n_adapters) {
    return n == 0 ? 0 : up256((size_t)lora_narrow_slices(n, k) * n * lora_padded_rank(rank) * 4);
}
size_t lora_backward_bytes(int64_t n, int64_t k, int64_t rows, int64_t rank, int64_t n_adapters) {
    return layout(n, k, rows, rank, n_adapters).total;
}

hipError_t launch_lora(const LoraCall &c, const void *base, void *y, float *h_out, uint8_t *ws, hipStream_t s) {
    float *part = (float *)ws;
    hipError_t e = launch_lora_narrow(c.x_type, c.w_type, true, c.x, c.n, c.k, c.a, c.rank, c.n_adapters, c.ids, part, s);
    if (e != hipSuccess) return e;
    return launch_lora_wide(c.x_type, c.w_type, false, part, lora_narrow_slices(c.n, c.k), c.n, c.rows, c.b, c.rank,
                            c.n_adapters, c.ids, c.scale, base, y, h_out, c.rank, false, s);
}

hipError_t launch_lora_backward(const LoraCall &c, const void *dy, const float *h, const void *dx_base, void *dx,
                                float *da, float *db, uint8_t *ws, hipStream_t s) {
    const Layout L = layout(c.n, c.k, c.rows, c.rank, c.n_adapters);
    int32_t *order = (int32_t *)(ws + L.order), *bounds = (int32_t *)(ws + L.bounds);
    float *part = (float *)(ws + L.part), *dh = (float *)(ws + L.dh);
    hipError_t e = hipSuccess;
    if (c.n > 0 && (dx || da)) {
        e = launch_lora_narrow(c.x_type, c.w_type, false, dy, c.n, c.rows, c.b, c.rank, c.n_adapters, c.ids, part, s);
        if (e != hipSuccess) return e;
        e = launch_lora_wide(c.x_type, c.w_type, true, part, lora_narrow_slices(c.n, c.rows), c.n, c.k, c.a, c.rank,
                             c.n_adapters, c.ids, c.scale, dx_base, dx, da ? dh : nullptr, lora_padded_rank(c.rank), true,
                             s);
        if (e != hipSuccess) return e;
    }
    if (!da && !db) return hipSuccess;
    e = launch_sort_ids(c.ids, c.n, c.n_adapters, order, nullptr, bounds, false, ws, s);
    if (e != hipSuccess) return e;
    return launch_lora_outer(c.x_type, c.x, dh, lora_padded_rank(c.rank), c.k, da, dy, h, c.rows, c.scale, db, c.n, c.rank,
                             c.n_adapters, order, bounds, (float *)(ws + L.outer), s);
}

}  // namespace qmm
