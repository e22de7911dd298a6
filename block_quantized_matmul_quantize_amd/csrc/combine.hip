// Rows to expert order and back: the gather of each token's row to the places of its (token, slot)
// pairs, the weighted sum of a token's expert results, and that sum's gradient.  All of them move
// rows and do at most three operations an element, so HBM bounds them, 16 bytes a lane where rows allow it.
// Gather and combine read every row once (a token's row once for all its slots) and write it once; the
// gradient has a workgroup a pair, so it reads a token's dy once for each slot (from cache after the first).
// No LDS, as nothing is shared between lanes but the sum of a weight's gradient.  2048 tokens x 8 slots of
// 2048 fp32 values: gather 24 us, combine onto a base 25 us (6.7 TB/s with the rows partly in the 256 MB
// cache, 34 us and 5.0 TB/s, a copy's rate, on rows from HBM); the gradient of 4096 x 2 of 4096 bf16
// values 31 us.  A decode step (16 x 8 of 2048) is latency, 4.2 us: a token's rows are loaded one after the other.
#include "common.hpp"
#include "launch.hpp"
#include "rowtypes.hpp"

namespace qmm {

namespace {

// Workgroup (t, column slice): the row of token t goes to its slots' places; places from n_valid on
// that fall to this token (t * top_k .. + top_k) are cleared.
template <class E, int N>
__global__ __launch_bounds__(256) void gather_kernel(const E *__restrict__ x, int64_t n_tok, int64_t top_k, int64_t k,
                                                     const int32_t *__restrict__ pos,
                                                     const int32_t *__restrict__ n_valid, E *__restrict__ y) {
    const int64_t col = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * N;
    if (col >= k) return;
    const int64_t valid = *n_valid, pairs = n_tok * top_k;
    for (int64_t t = blockIdx.x; t < n_tok; t += gridDim.x) {
        const Pack<E, N> v = *(const Pack<E, N> *)(x + t * k + col);
        for (int64_t j = 0; j < top_k; ++j) {
            const int64_t p = pos[t * top_k + j], q = t * top_k + j;
            if (p >= 0 && p < pairs) *(Pack<E, N> *)(y + p * k + col) = v;
            if (q >= valid) {
                Pack<E, N> z;
#pragma unroll
                for (int i = 0; i < N; ++i) z.v[i] = (E)0.f;
                *(Pack<E, N> *)(y + q * k + col) = z;
            }
        }
    }
}

// Row of h of pair q, -1 for none.  pos: the row of each pair; with n_ids > 0 the id of each pair, whose row
// is the q-th and counts only where the id is in [0, n_ids); null: the q-th.
__device__ __forceinline__ int64_t row_of(const int32_t *pos, int64_t n_ids, int64_t q, int64_t pairs) {
    if (!pos) return q;
    const int64_t p = pos[q];
    if (n_ids) return p >= 0 && p < n_ids ? q : -1;
    return p >= 0 && p < pairs ? p : -1;
}

template <class E, int N>
__global__ __launch_bounds__(256) void combine_kernel(const E *__restrict__ h, int64_t n_tok, int64_t top_k, int64_t k,
                                                      const int32_t *__restrict__ pos, int64_t n_ids,
                                                      const float *__restrict__ w, const E *base, E *y) {
    const int64_t col = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * N;
    if (col >= k) return;
    const int64_t pairs = n_tok * top_k;
    for (int64_t t = blockIdx.x; t < n_tok; t += gridDim.x) {
        float acc[N], v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = 0.f;
        for (int64_t j = 0; j < top_k; ++j) {
            const int64_t q = t * top_k + j, p = row_of(pos, n_ids, q, pairs);
            if (p < 0) continue;
            const float c = w ? w[q] : 1.f;
            load_n<N>(h + p * k + col, v);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] += c * v[i];
        }
        if (base) {
            load_n<N>(base + t * k + col, v);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] += v[i];
        }
        store_n<N>(y + t * k + col, acc);
    }
}

// One workgroup per pair: dh's row and dw.  Pairs without a row have a weight gradient of zero.
template <class E, int N>
__global__ __launch_bounds__(256) void combine_backward_kernel(const E *__restrict__ dy, const E *__restrict__ h,
                                                               int64_t n_tok, int64_t top_k, int64_t k,
                                                               const int32_t *__restrict__ pos, int64_t n_ids,
                                                               const float *__restrict__ w,
                                                               const int32_t *__restrict__ n_valid,
                                                               E *__restrict__ dh, float *__restrict__ dw) {
    __shared__ float sums[4];
    const int64_t pairs = n_tok * top_k;
    for (int64_t q = blockIdx.x; q < pairs; q += gridDim.x) {
        const int64_t t = q / top_k, p = row_of(pos, n_ids, q, pairs);
        const bool ok = p >= 0;
        // dh's q-th row: the pair's own, or one past the valid places
        if (n_ids ? !ok : pos && q >= *n_valid)
            for (int64_t col = threadIdx.x * N; col < k; col += 256 * N) {
                float z[N];
#pragma unroll
                for (int i = 0; i < N; ++i) z[i] = 0.f;
                store_n<N>(dh + q * k + col, z);
            }
        float dot = 0.f;
        if (ok) {
            const float c = w ? w[q] : 1.f;
            for (int64_t col = threadIdx.x * N; col < k; col += 256 * N) {
                float d[N], v[N];
                load_n<N>(dy + t * k + col, d);
                load_n<N>(h + p * k + col, v);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    dot += d[i] * v[i];
                    d[i] *= c;
                }
                store_n<N>(dh + p * k + col, d);
            }
        }
#pragma unroll
        for (int m = 32; m; m >>= 1) dot += __shfl_xor(dot, m);
        if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = dot;
        __syncthreads();
        if (threadIdx.x == 0) dw[q] = sums[0] + sums[1] + sums[2] + sums[3];
        __syncthreads();
    }
}

dim3 grid_of(int64_t n, int64_t groups, int threads) {
    return dim3((unsigned)(n < 1 << 20 ? n : 1 << 20), (unsigned)((groups + threads - 1) / threads));
}
int threads_of(int64_t groups) { return groups >= 256 ? 256 : (int)((groups + 63) / 64 * 64); }

}  // namespace

hipError_t launch_gather_sorted(int type, const void *x, int64_t n_tok, int64_t top_k, int64_t k, const int32_t *pos,
                                const int32_t *n_valid, void *y, hipStream_t s) {
    return with_type(type, [&](auto e) -> hipError_t {
        typedef decltype(e) E;
        constexpr int N = 16 / sizeof(E);
        if (k % N == 0 && aligned16(x, y)) {
            const int th = threads_of(k / N);
            hipLaunchKernelGGL((gather_kernel<E, N>), grid_of(n_tok, k / N, th), dim3(th), 0, s, (const E *)x, n_tok,
                               top_k, k, pos, n_valid, (E *)y);
        } else {
            const int th = threads_of(k);
            hipLaunchKernelGGL((gather_kernel<E, 1>), grid_of(n_tok, k, th), dim3(th), 0, s, (const E *)x, n_tok, top_k,
                               k, pos, n_valid, (E *)y);
        }
        return hipGetLastError();
    });
}

hipError_t launch_combine(int type, const void *h, int64_t n_tok, int64_t top_k, int64_t k, const int32_t *pos,
                          int64_t n_ids, const float *w, const void *base, void *y, hipStream_t s) {
    return with_type(type, [&](auto e) -> hipError_t {
        typedef decltype(e) E;
        constexpr int N = 16 / sizeof(E);
        if (k % N == 0 && aligned16(h, base, y)) {
            const int th = threads_of(k / N);
            hipLaunchKernelGGL((combine_kernel<E, N>), grid_of(n_tok, k / N, th), dim3(th), 0, s, (const E *)h, n_tok,
                               top_k, k, pos, n_ids, w, (const E *)base, (E *)y);
        } else {
            const int th = threads_of(k);
            hipLaunchKernelGGL((combine_kernel<E, 1>), grid_of(n_tok, k, th), dim3(th), 0, s, (const E *)h, n_tok,
                               top_k, k, pos, n_ids, w, (const E *)base, (E *)y);
        }
        return hipGetLastError();
    });
}

hipError_t launch_combine_backward(int type, const void *dy, const void *h, int64_t n_tok, int64_t top_k, int64_t k,
                                   const int32_t *pos, int64_t n_ids, const float *w, const int32_t *n_valid,
                                   void *dh, float *dw, hipStream_t s) {
    return with_type(type, [&](auto e) -> hipError_t {
        typedef decltype(e) E;
        constexpr int N = 16 / sizeof(E);
        const int64_t pairs = n_tok * top_k;
        const dim3 grid((unsigned)(pairs < 1 << 20 ? pairs : 1 << 20));
        if (k % N == 0 && aligned16(dy, h, dh))
            hipLaunchKernelGGL((combine_backward_kernel<E, N>), grid, dim3(256), 0, s, (const E *)dy, (const E *)h,
                               n_tok, top_k, k, pos, n_ids, w, n_valid, (E *)dh, dw);
        else
            hipLaunchKernelGGL((combine_backward_kernel<E, 1>), grid, dim3(256), 0, s, (const E *)dy, (const E *)h,
                               n_tok, top_k, k, pos, n_ids, w, n_valid, (E *)dh, dw);
        return hipGetLastError();
    });
}

}  // namespace qmm
