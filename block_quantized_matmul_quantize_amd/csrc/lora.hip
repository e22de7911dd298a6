// Low-rank adapters of many requests beside a shared projection: row i with adapter c adds
// scale[c] * B[c] (A[c] x[i]) to the projection's result, and the gradients of that.
//
// Forward: lora_narrow.hip multiplies by A in slices of K, lora_wide.hip adds the slices up and multiplies
// by B onto base.  Where h is kept a launch between them adds up the slices and writes it.  It is left out
// otherwise: every workgroup of the second half reads its rows' slices again, 1 MB for each of 28 blocks of
// columns for 2048 rows into 14336 columns, 29 MB from L2, which takes 2.6 us more there (46.2 against
// 43.7 us) against 4.2 us for the launch.  Backward: the same two on
// dy, with B and A in transposed roles, and the gradients of A and B on rows sorted by adapter in one
// launch (lora_outer.hip), for which the launch in between lays h and dh out.
#include "launch.hpp"
#include "lora_parts.hpp"

namespace qmm {

namespace {

struct Finish {
    LoraFinish c;
    int32_t padded;
};

// A workgroup takes 64 rows and 16 ranks, a thread 4 ranks of a row.
__global__ __launch_bounds__(256) void finish_kernel(Finish f) {
    const LoraFinish &c = f.c;
    __shared__ alignas(16) uint16_t stage[3][kWindow][16 + 4];
    const int slot = threadIdx.x >> 2, r4 = 4 * (threadIdx.x & 3), rank = (int)c.rank;
    const int r = 16 * blockIdx.x + r4;
    for (int64_t i0 = (int64_t)blockIdx.y * kWindow; i0 < c.n; i0 += (int64_t)gridDim.y * kWindow) {
        const int64_t row = i0 + slot < c.n ? i0 + slot : c.n - 1;
        const bool mine = i0 + slot < c.n;
        const int32_t id = c.ids[row];
        const bool some = (uint32_t)id < (uint32_t)c.n_adapters;
        auto lay_out = [&](const float (&x)[4], uint16_t *out) {
            uint32_t p[3][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float mid = rest_of(x[i]);
                p[0][i] = __float_as_uint(x[i]);
                p[1][i] = __float_as_uint(mid);
                p[2][i] = __float_as_uint(mid - __uint_as_float(p[1][i] & 0xffff0000u));
            }
#pragma unroll
            for (int j = 0; j < 3; ++j)
                *(u32x2 *)&stage[j][slot][r4] = u32x2{high_halves(p[j][0], p[j][1]), high_halves(p[j][2], p[j][3])};
            __syncthreads();
            const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
            const int64_t place = i0 + lane < c.n ? c.pos[i0 + lane] : -1;
            if (place >= 0)
#pragma unroll
                for (int j = 0; j < 3; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        out[((place / 32 * 3 + j) * f.padded + 16 * blockIdx.x + 4 * wave + q) * 32 + place % 32] =
                            stage[j][lane][4 * wave + q];
            __syncthreads();
        };
        if (c.kept) {
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = c.kept[row * rank + (r + q < rank ? r + q : rank - 1)];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = r + q < rank ? v[q] : 0.f;
            lay_out(v, c.parts_h);
        }
        if (c.part) {
            f32x4 sum = {0.f, 0.f, 0.f, 0.f};
            const float *p = c.part + row * f.padded + r;
            const int64_t next = c.n * f.padded;
            for (int s0 = 0; s0 < c.parts; s0 += 8) {   // a slice past the last is read as the first, and left out
                f32x4 u[8];
#pragma unroll
                for (int s = 0; s < 8; ++s) u[s] = *(const f32x4 *)(p + (s0 + s < c.parts ? s0 + s : 0) * next);
#pragma unroll
                for (int s = 0; s < 8; ++s) sum += s0 + s < c.parts ? u[s] : f32x4{0.f, 0.f, 0.f, 0.f};
            }
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = some && r + q < rank ? sum[q] : 0.f;
            if (mine && c.sum) *(f32x4 *)(c.sum + row * f.padded + r) = f32x4{v[0], v[1], v[2], v[3]};
            if (mine && c.h)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (r + q < rank) c.h[row * rank + r + q] = v[q];
            if (c.parts_dh) {
                const float scale = some && c.scale ? c.scale[id] : 1.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] *= scale;
                lay_out(v, c.parts_dh);
            }
        }
    }
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct Layout { size_t order, pos, bounds, part, parts_h, parts_dh, outer, total; };
Layout layout(int64_t n, int64_t k, int64_t rows, int64_t rank, int64_t n_adapters) {
    Layout L{};
    const int64_t padded = lora_padded_rank(rank);
    size_t off = up256(sort_ids_bytes(n, n_adapters, false));
    L.order = off;
    off += up256((size_t)n * 4);
    L.pos = off;
    off += up256((size_t)n * 4);
    L.bounds = off;
    off += up256((size_t)(n_adapters + 1) * 4);
    L.part = off;
    off += n ? up256((size_t)(lora_narrow_slices(n, rows) * n * padded) * 4) : 0;
    L.parts_h = off;
    off += up256((size_t)(3 * padded * ((n + 31) / 32 * 32)) * 2);
    L.parts_dh = off;
    off += up256((size_t)(3 * padded * ((n + 31) / 32 * 32)) * 2);
    L.outer = off;
    off += up256(lora_outer_bytes(n, k, rows, rank, n_adapters));
    L.total = off;
    return L;
}

}  // namespace

hipError_t launch_lora_finish(const LoraFinish &c, hipStream_t s) {
    const Finish f{c, lora_padded_rank(c.rank)};
    const int64_t windows = (c.n + kWindow - 1) / kWindow;
    hipLaunchKernelGGL(finish_kernel, dim3((unsigned)(f.padded / 16), (unsigned)(windows < 65535 ? windows : 65535)),
                       dim3(256), 0, s, f);
    return hipGetLastError();
}

size_t lora_bytes(int64_t n, int64_t k, int64_t rows, int64_t rank, int64_t n_adapters) {
    return n == 0 ? 0 : up256((size_t)lora_narrow_slices(n, k) * n * lora_padded_rank(rank) * 4);
}
size_t lora_backward_bytes(int64_t n, int64_t k, int64_t rows, int64_t rank, int64_t n_adapters) {
    return layout(n, k, rows, rank, n_adapters).total;
}

hipError_t launch_lora(const LoraCall &c, const void *base, void *y, float *h_out, uint8_t *ws, hipStream_t s) {
    float *part = (float *)ws;
    hipError_t e = launch_lora_narrow(c.x_type, c.w_type, true, c.x, c.n, c.k, c.a, c.rank, c.n_adapters, c.ids, part,
                                      nullptr, nullptr, nullptr, s);
    if (e != hipSuccess) return e;
    int parts = lora_narrow_slices(c.n, c.k);
    if (h_out) {
        LoraFinish f{};
        f.part = part;
        f.parts = parts;
        f.n = c.n;
        f.rank = c.rank;
        f.n_adapters = c.n_adapters;
        f.ids = c.ids;
        f.sum = part;
        f.h = h_out;
        e = launch_lora_finish(f, s);
        if (e != hipSuccess) return e;
        parts = 1;
    }
    return launch_lora_wide(c.x_type, c.w_type, false, part, parts, c.n, c.rows, c.b, c.rank, c.n_adapters, c.ids, c.scale,
                            base, y, s);
}

hipError_t launch_lora_backward(const LoraCall &c, const void *dy, const float *h, const void *dx_base, void *dx,
                                float *da, float *db, uint8_t *ws, hipStream_t s) {
    const Layout L = layout(c.n, c.k, c.rows, c.rank, c.n_adapters);
    int32_t *order = (int32_t *)(ws + L.order), *pos = (int32_t *)(ws + L.pos), *bounds = (int32_t *)(ws + L.bounds);
    uint16_t *parts_h = (uint16_t *)(ws + L.parts_h), *parts_dh = (uint16_t *)(ws + L.parts_dh);
    float *part = (float *)(ws + L.part);
    hipError_t e = hipSuccess;
    // where the first product runs anyway, one of its workgroups sorts the rows
    const bool beside = (da || db) && c.n > 0 && (dx || da) && lora_narrow_sorts(c.n, c.n_adapters);
    if ((da || db) && !beside) {
        e = launch_sort_ids(c.ids, c.n, c.n_adapters, order, pos, bounds, false, ws, s);
        if (e != hipSuccess) return e;
    }
    if (c.n > 0) {
        if (dx || da) {
            e = launch_lora_narrow(c.x_type, c.w_type, false, dy, c.n, c.rows, c.b, c.rank, c.n_adapters, c.ids, part,
                                   beside ? order : nullptr, pos, bounds, s);
            if (e != hipSuccess) return e;
        }
        int parts = lora_narrow_slices(c.n, c.rows);
        if (da || db) {
            LoraFinish f{};
            f.part = dx || da ? part : nullptr;
            f.parts = parts;
            f.n = c.n;
            f.rank = c.rank;
            f.n_adapters = c.n_adapters;
            f.ids = c.ids;
            f.scale = c.scale;
            f.sum = dx ? part : nullptr;
            f.kept = db ? h : nullptr;
            f.parts_h = parts_h;
            f.parts_dh = da ? parts_dh : nullptr;
            f.pos = pos;
            e = launch_lora_finish(f, s);
            if (e != hipSuccess) return e;
            parts = 1;
        }
        if (dx) {
            e = launch_lora_wide(c.x_type, c.w_type, true, part, parts, c.n, c.k, c.a, c.rank, c.n_adapters, c.ids, c.scale,
                                 dx_base, dx, s);
            if (e != hipSuccess) return e;
        }
    }
    if (!da && !db) return hipSuccess;
    return launch_lora_outer(c.x_type, c.x, parts_dh, c.k, da, dy, parts_h, c.rows, c.scale, db, c.n, c.rank,
                             c.n_adapters, order, bounds, (float *)(ws + L.outer), s);
}

}  // namespace qmm
