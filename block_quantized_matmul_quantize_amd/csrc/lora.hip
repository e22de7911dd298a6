// Low-rank adapters of many requests beside a shared projection: row i with adapter c adds
// scale[c] * B[c] (A[c] x[i]) to the projection's result, and the gradients of that.
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"
#include "rowtypes.hpp"

namespace qmm {

namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

// out[i][r] = c * sum_j v[i][j] * m[id][..]: a wave per (i, r).  By rows: m [id][rank][k]; by columns:
// m [id][k][rank], scaled.
template <class X, class W, bool kByRow>
__global__ __launch_bounds__(256) void narrow_kernel(const X *__restrict__ v, int64_t n, int64_t k,
                                                     const W *__restrict__ m, int64_t rank, int64_t n_adapters,
                                                     const int32_t *__restrict__ ids, const float *__restrict__ scale,
                                                     float *__restrict__ out) {
    const int lane = threadIdx.x & 63;
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < n * rank; t += (int64_t)gridDim.x * 4) {
        const int64_t i = t / rank, r = t - i * rank, id = ids[i];
        float s = 0.f;
        if (id >= 0 && id < n_adapters) {
            for (int64_t j = lane; j < k; j += 64)
                s += (float)v[i * k + j] * (float)m[kByRow ? (id * rank + r) * k + j : (id * k + j) * rank + r];
            s = wave_sum(s);
            if (!kByRow && scale) s *= scale[id];
        }
        if (lane == 0) out[t] = s;
    }
}

// out[i][j] = base[i][j] + c * sum_r h[i][r] * m: a thread per (i, j).
template <class X, class W, bool kByRow>
__global__ __launch_bounds__(256) void wide_kernel(const float *__restrict__ h, int64_t n, int64_t k,
                                                   const W *__restrict__ m, int64_t rank, int64_t n_adapters,
                                                   const int32_t *__restrict__ ids, const float *__restrict__ scale,
                                                   const X *base, X *out) {
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < n * k; t += (int64_t)gridDim.x * 256) {
        const int64_t i = t / k, j = t - i * k, id = ids[i];
        float s = 0.f;
        if (id >= 0 && id < n_adapters) {
            for (int64_t r = 0; r < rank; ++r)
                s += h[i * rank + r] * (float)m[kByRow ? (id * rank + r) * k + j : (id * k + j) * rank + r];
            if (!kByRow && scale) s *= scale[id];
        }
        out[t] = (X)((base ? (float)base[t] : 0.f) + s);
    }
}

// da[c][r][j] (kByRow) or db[c][j][r] = c * sum over the adapter's rows of h[i][r] * v[i][j].
template <class X, bool kByRow>
__global__ __launch_bounds__(256) void outer_kernel(const float *__restrict__ h, const X *__restrict__ v, int64_t k,
                                                    int64_t rank, int64_t n_adapters, const int32_t *__restrict__ order,
                                                    const int32_t *__restrict__ bounds,
                                                    const float *__restrict__ scale, float *__restrict__ out) {
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < n_adapters * rank * k;
         t += (int64_t)gridDim.x * 256) {
        const int64_t c = t / (rank * k), u = t - c * rank * k;
        const int64_t r = kByRow ? u / k : u % rank, j = kByRow ? u % k : u / rank;
        float s = 0.f;
        for (int64_t p = bounds[c]; p < bounds[c + 1]; ++p) {
            const int64_t i = order[p];
            s += h[i * rank + r] * (float)v[i * k + j];
        }
        out[t] = !kByRow && scale ? s * scale[c] : s;
    }
}

unsigned grid_of(int64_t blocks) { return (unsigned)(blocks < 65536 ? (blocks > 0 ? blocks : 1) : 65536); }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Element types of x and of the adapters.
template <class F> hipError_t with_types(int x_type, int w_type, F f) {
    return with_type(x_type, [&](auto x) -> hipError_t {
        return with_type(w_type, [&](auto w) -> hipError_t {
            if constexpr (sizeof(x) == 4 || std::is_same<decltype(x), decltype(w)>::value) return f(x, w);
            else return hipErrorInvalidValue;
        });
    });
}

struct Layout { size_t sort, order, bounds, h, total; };
Layout layout(int64_t n, int64_t rank, int64_t n_adapters) {
    Layout L{};
    size_t off = up256(sort_ids_bytes(n, n_adapters, false));
    L.order = off;
    off += up256((size_t)n * 4);
    L.bounds = off;
    off += up256((size_t)(n_adapters + 1) * 4);
    L.h = off;
    off += up256((size_t)n * rank * 4);
    L.total = off;
    return L;
}

}  // namespace

size_t lora_bytes(int64_t n, int64_t k, int64_t rows, int64_t rank, int64_t n_adapters) {
    return n == 0 ? 0 : layout(n, rank, n_adapters).total;
}
size_t lora_backward_bytes(int64_t n, int64_t k, int64_t rows, int64_t rank, int64_t n_adapters) {
    return layout(n, rank, n_adapters).total;
}

hipError_t launch_lora(const LoraCall &c, const void *base, void *y, float *h_out, uint8_t *ws, hipStream_t s) {
    return with_types(c.x_type, c.w_type, [&](auto x, auto w) -> hipError_t {
        typedef decltype(x) X;
        typedef decltype(w) W;
        float *h = h_out ? h_out : (float *)(ws + layout(c.n, c.rank, c.n_adapters).h);
        hipLaunchKernelGGL((narrow_kernel<X, W, true>), dim3(grid_of((c.n * c.rank + 3) / 4)), dim3(256), 0, s,
                           (const X *)c.x, c.n, c.k, (const W *)c.a, c.rank, c.n_adapters, c.ids, c.scale, h);
        hipLaunchKernelGGL((wide_kernel<X, W, false>), dim3(grid_of((c.n * c.rows + 255) / 256)), dim3(256), 0, s, h,
                           c.n, c.rows, (const W *)c.b, c.rank, c.n_adapters, c.ids, c.scale, (const X *)base, (X *)y);
        return hipGetLastError();
    });
}

hipError_t launch_lora_backward(const LoraCall &c, const void *dy, const float *h, const void *dx_base, void *dx,
                                float *da, float *db, uint8_t *ws, hipStream_t s) {
    const Layout L = layout(c.n, c.rank, c.n_adapters);
    int32_t *order = (int32_t *)(ws + L.order), *bounds = (int32_t *)(ws + L.bounds);
    float *dh = (float *)(ws + L.h);
    if (da || db) {
        hipError_t e = launch_sort_ids(c.ids, c.n, c.n_adapters, order, nullptr, bounds, false, ws, s);
        if (e != hipSuccess) return e;
    }
    return with_types(c.x_type, c.w_type, [&](auto x, auto w) -> hipError_t {
        typedef decltype(x) X;
        typedef decltype(w) W;
        if (c.n > 0 && (dx || da))
            hipLaunchKernelGGL((narrow_kernel<X, W, false>), dim3(grid_of((c.n * c.rank + 3) / 4)), dim3(256), 0, s,
                               (const X *)dy, c.n, c.rows, (const W *)c.b, c.rank, c.n_adapters, c.ids, c.scale, dh);
        if (c.n > 0 && dx)
            hipLaunchKernelGGL((wide_kernel<X, W, true>), dim3(grid_of((c.n * c.k + 255) / 256)), dim3(256), 0, s, dh,
                               c.n, c.k, (const W *)c.a, c.rank, c.n_adapters, c.ids, c.scale, (const X *)dx_base,
                               (X *)dx);
        if (da)
            hipLaunchKernelGGL((outer_kernel<X, true>), dim3(grid_of((c.n_adapters * c.rank * c.k + 255) / 256)),
                               dim3(256), 0, s, dh, (const X *)c.x, c.k, c.rank, c.n_adapters, order, bounds, c.scale,
                               da);
        if (db)
            hipLaunchKernelGGL((outer_kernel<X, false>), dim3(grid_of((c.n_adapters * c.rank * c.rows + 255) / 256)),
                               dim3(256), 0, s, h, (const X *)dy, c.rows, c.rank, c.n_adapters, order, bounds, c.scale,
                               db);
        return hipGetLastError();
    });
}

}  // namespace qmm
