// Embedding lookup: y[i] = scale * table[ids[i]], the table rows fp32, fp16, bf16 or GGUF blocks that
// are decoded on the way (embedding tables ship in the same block types as the weights), and its
// gradient: dT[v] = scale * (sum of dy[i] over the tokens with id v), over tokens sorted by id.
#include "common.hpp"
#include "launch.hpp"
#include "rowtypes.hpp"

namespace qmm {

namespace {

// Values 8g .. 8g+7 of a row of blocks, in fp32.  d * scale and dmin * min are exact (11 + 6 bits),
// their products with the codes too (at most 24 bits), so each value is rounded once.
template <int T> __device__ __forceinline__ void decode8(const uint8_t *row, int64_t g, float (&o)[8]) {
    if constexpr (T == kQ8_0) {
        const uint8_t *b = row + (g >> 2) * 34;
        const float d = h2f(ld2(b));
        const uint32_t u[2] = {ld4(b + 2 + 8 * (g & 3)), ld4(b + 6 + 8 * (g & 3))};
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = d * (float)(int8_t)(u[i >> 2] >> (8 * (i & 3)));
    } else if constexpr (T == kQ4_0) {
        const uint8_t *b = row + (g >> 2) * 18;
        const float d = h2f(ld2(b));
        const int sh = g & 2 ? 4 : 0;
        const uint32_t u[2] = {ld4(b + 2 + 8 * (g & 1)) >> sh, ld4(b + 6 + 8 * (g & 1)) >> sh};
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = d * (float)((int)((u[i >> 2] >> (8 * (i & 3))) & 15) - 8);
    } else if constexpr (T == kQ4_K || T == kQ5_K) {
        const uint8_t *b = row + (g >> 5) * Fmt<T>::BYTES;
        const int s = (int)(g & 31), j = s >> 2, at = 8 * (s & 3);
        const uint8_t *p = b + 4;
        int sc, mn;
        if (j < 4) {
            sc = p[j] & 63;
            mn = p[j + 4] & 63;
        } else {
            sc = (p[j + 4] & 15) | ((p[j - 4] >> 6) << 4);
            mn = (p[j + 4] >> 4) | ((p[j] >> 6) << 4);
        }
        const float d = h2f(ld2(b)) * (float)sc, m = h2f(ld2(b + 2)) * (float)mn;
        const uint8_t *q = b + (T == kQ5_K ? 48 : 16) + 32 * (j >> 1) + at;
        const int sh = j & 1 ? 4 : 0;
        const uint32_t u[2] = {ld4(q) >> sh, ld4(q + 4) >> sh};
        uint32_t h[2] = {0, 0};
        if constexpr (T == kQ5_K) {
            h[0] = ld4(b + 16 + at) >> j;
            h[1] = ld4(b + 20 + at) >> j;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t c = (u[i >> 2] >> (8 * (i & 3))) & 15;
            if constexpr (T == kQ5_K) c |= ((h[i >> 2] >> (8 * (i & 3))) & 1) << 4;
            o[i] = d * (float)c - m;
        }
    } else if constexpr (T == kQ6_K) {
        const uint8_t *b = row + (g >> 5) * 210;
        const int s = (int)(g & 31), half = s >> 4, part = (s >> 2) & 3, l = 8 * (s & 3);
        const float d = h2f(ld2(b + 208)) * (float)(int8_t)b[192 + (s >> 1)];
        const uint8_t *lo = b + 64 * half + 32 * (part & 1) + l, *hi = b + 128 + 32 * half + l;
        const int shl = part & 2 ? 4 : 0, shh = 2 * part;
        const uint32_t u[2] = {ld4(lo) >> shl, ld4(lo + 4) >> shl}, h[2] = {ld4(hi) >> shh, ld4(hi + 4) >> shh};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = (int)(((u[i >> 2] >> (8 * (i & 3))) & 15) | (((h[i >> 2] >> (8 * (i & 3))) & 3) << 4));
            o[i] = d * (float)(c - 32);
        }
    } else if constexpr (T == kQ3_K) {
        const uint8_t *b = row + (g >> 5) * 110;
        const int s = (int)(g & 31), half = s >> 4, part = (s >> 2) & 3, l = 8 * (s & 3), is = s >> 1;
        const uint8_t *p = b + 96;
        const int sc = ((is < 8 ? p[is] & 15 : p[is - 8] >> 4) | (((p[8 + (is & 3)] >> (2 * (is >> 2))) & 3) << 4)) - 32;
        const float d = h2f(ld2(b + 108)) * (float)sc;
        const uint8_t *lo = b + 32 + 32 * half + l, *hi = b + l;
        const int shl = 2 * part, shh = 4 * half + part;
        const uint32_t u[2] = {ld4(lo) >> shl, ld4(lo + 4) >> shl}, h[2] = {ld4(hi) >> shh, ld4(hi + 4) >> shh};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = (int)((u[i >> 2] >> (8 * (i & 3))) & 3) + (((h[i >> 2] >> (8 * (i & 3))) & 1) ? 0 : -4);
            o[i] = d * (float)c;
        }
    } else {
        static_assert(T == kIQ4_XS);
        const uint8_t *b = row + (g >> 5) * 136;
        const int s = (int)(g & 31), ib = s >> 2;
        const int ls = ((b[4 + (ib >> 1)] >> (4 * (ib & 1))) & 15) | (((ld2(b + 2) >> (2 * ib)) & 3) << 4);
        const float d = h2f(ld2(b)) * (float)(ls - 32);
        const uint8_t *q = b + 8 + 16 * ib + 8 * (s & 1);
        const int sh = s & 2 ? 4 : 0;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const uint32_t c = iq4_lookup4((ld4(q + 4 * w) >> sh) & 0x0f0f0f0fu);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[4 * w + i] = d * (float)(int8_t)(c >> (8 * i));
        }
    }
}

// One thread per 8 values, tokens and values in output order.
template <int T, class O>
__global__ __launch_bounds__(256) void embed_blocks_kernel(const uint8_t *__restrict__ table, int64_t vocab,
                                                           int64_t row_bytes, int64_t groups,
                                                           const int32_t *__restrict__ ids, int64_t total, float scale,
                                                           O *__restrict__ y) {
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
        const int64_t i = t / groups, g = t - i * groups;
        const int64_t id = ids[i];
        float o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (id >= 0 && id < vocab) {
            decode8<T>(table + id * row_bytes, g, o);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] *= scale;
        }
        store_n<8>(y + t * 8, o);
    }
}

// The same for tables of elements, N values a thread.
template <class E, class O, int N>
__global__ __launch_bounds__(256) void embed_rows_kernel(const E *__restrict__ table, int64_t vocab, int64_t k,
                                                         const int32_t *__restrict__ ids, int64_t total, float scale,
                                                         O *__restrict__ y) {
    const int64_t groups = k / N;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
        const int64_t i = t / groups, g = t - i * groups;
        const int64_t id = ids[i];
        float o[N];
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = 0.f;
        if (id >= 0 && id < vocab) {
            load_n<N>(table + id * k + g * N, o);
#pragma unroll
            for (int j = 0; j < N; ++j) o[j] *= scale;
        }
        store_n<N>(y + t * N, o);
    }
}

unsigned grid_of(int64_t threads) {
    const int64_t b = (threads + 255) / 256;
    return (unsigned)(b < 1 ? 1 : b < 65536 ? b : 65536);
}

template <int T, class O>
hipError_t embed_blocks(const uint8_t *table, int64_t vocab, int64_t k, const int32_t *ids, int64_t n, float scale, O *y,
                        hipStream_t s) {
    const int64_t total = n * (k / 8);
    hipLaunchKernelGGL((embed_blocks_kernel<T, O>), dim3(grid_of(total)), dim3(256), 0, s, table, vocab,
                       k / Fmt<T>::QK * Fmt<T>::BYTES, k / 8, ids, total, scale, y);
    return hipGetLastError();
}

template <class E, class O>
hipError_t embed_rows(const E *table, int64_t vocab, int64_t k, const int32_t *ids, int64_t n, float scale, O *y,
                      hipStream_t s) {
    // 8 values a thread where every group of them is aligned, else single values
    if (k % 8 == 0 && aligned16(table, y))
        hipLaunchKernelGGL((embed_rows_kernel<E, O, 8>), dim3(grid_of(n * (k / 8))), dim3(256), 0, s, table, vocab, k,
                           ids, n * (k / 8), scale, y);
    else
        hipLaunchKernelGGL((embed_rows_kernel<E, O, 1>), dim3(grid_of(n * k)), dim3(256), 0, s, table, vocab, k, ids,
                           n * k, scale, y);
    return hipGetLastError();
}

// ------------------------------------------------------------------------------------------------
// Gradient
// ------------------------------------------------------------------------------------------------
template <class E>
__global__ __launch_bounds__(256) void fill_zero_kernel(E *__restrict__ p, int64_t n16, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n16; i += (int64_t)gridDim.x * 256)
        ((u32x4 *)p)[i] = u32x4{0, 0, 0, 0};
    constexpr int per = 16 / sizeof(E);
    if (blockIdx.x == 0)
        for (int64_t i = n16 * per + threadIdx.x; i < n; i += 256) p[i] = (E)0.f;
}

// Chunks of kChunk sorted tokens; a workgroup sums the rows of one chunk, N columns a thread, from
// one id to the next.  An id whose tokens lie in one chunk is written at once; the others leave
// their sums in part[chunk][0] (the id began before this chunk) or part[chunk][1] (it goes on
// after it), which join_kernel adds up in chunk order: the sum's order is fixed.
constexpr int kChunk = 32;

template <class E, class O, int N>
__global__ __launch_bounds__(256) void grad_kernel(const E *__restrict__ dy, int64_t k, const int32_t *__restrict__ skeys,
                                                   const int32_t *__restrict__ order, int64_t n, int32_t vocab,
                                                   float scale, O *__restrict__ grad, float *__restrict__ part) {
    const int64_t c = blockIdx.x, e0 = c * kChunk;
    const int cnt = (int)(n - e0 < kChunk ? n - e0 : kChunk);
    const int64_t col = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * N;
    if (col >= k) return;
    int32_t cur = skeys[e0];
    bool starts = e0 == 0 || skeys[e0 - 1] != cur;
    float acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.f;
    auto flush = [&](bool ends) {
        if (starts && ends) {
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] *= scale;
            store_n<N>(grad + cur * k + col, acc);
        } else {
            store_n<N>(part + (2 * c + (starts ? 1 : 0)) * k + col, acc);
        }
    };
    for (int e = 0; e < cnt && cur < vocab; ++e) {
        const int32_t key = skeys[e0 + e];
        if (key != cur) {
            flush(true);
            cur = key;
            starts = true;
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = 0.f;
            if (key >= vocab) break;
        }
        float v[N];
        load_n<N>(dy + order[e0 + e] * k + col, v);
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] += v[j];
    }
    if (cur < vocab) flush(e0 + cnt == n || skeys[e0 + cnt] != cur);
}

template <class O, int N>
__global__ __launch_bounds__(256) void join_kernel(const float *__restrict__ part, int64_t k,
                                                   const int32_t *__restrict__ skeys, int64_t n, int32_t vocab,
                                                   float scale, O *__restrict__ grad) {
    const int64_t c = blockIdx.x, e0 = c * kChunk, e1 = e0 + kChunk;
    if (e1 >= n) return;
    const int32_t key = skeys[e1 - 1];
    // only the chunk in which an id begins that goes on after it
    if (key >= vocab || skeys[e1] != key || (skeys[e0] == key && e0 > 0 && skeys[e0 - 1] == key)) return;
    const int64_t col = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * N;
    if (col >= k) return;
    float acc[N], v[N];
    load_n<N>(part + (2 * c + 1) * k + col, acc);
    for (int64_t q = c + 1; q * kChunk < n && skeys[q * kChunk] == key; ++q) {
        load_n<N>(part + 2 * q * k + col, v);
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] += v[j];
    }
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] *= scale;
    store_n<N>(grad + key * k + col, acc);
}

template <class E, class O, int N>
hipError_t grad_n(const E *dy, int64_t n, int64_t k, const int32_t *order, const int32_t *skeys, int64_t vocab,
                  float scale, O *grad, float *part, hipStream_t s) {
    const int64_t groups = (k + N - 1) / N;
    const int threads = groups >= 256 ? 256 : (int)((groups + 63) / 64 * 64);
    const dim3 grid((unsigned)((n + kChunk - 1) / kChunk), (unsigned)((groups + threads - 1) / threads));
    hipLaunchKernelGGL((grad_kernel<E, O, N>), grid, dim3(threads), 0, s, dy, k, skeys, order, n, (int32_t)vocab, scale,
                       grad, part);
    hipLaunchKernelGGL((join_kernel<O, N>), grid, dim3(threads), 0, s, part, k, skeys, n, (int32_t)vocab, scale, grad);
    return hipGetLastError();
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

hipError_t launch_embed(int type, const void *table, int64_t vocab, int64_t k, const int32_t *ids, int64_t n,
                        float scale, int y_type, void *y, hipStream_t s) {
    return with_type(y_type, [&](auto o) -> hipError_t {
        typedef decltype(o) O;
        const uint8_t *b = (const uint8_t *)table;
        O *out = (O *)y;
        switch (type) {
            case kQ4_0: return embed_blocks<kQ4_0>(b, vocab, k, ids, n, scale, out, s);
            case kQ8_0: return embed_blocks<kQ8_0>(b, vocab, k, ids, n, scale, out, s);
            case kQ3_K: return embed_blocks<kQ3_K>(b, vocab, k, ids, n, scale, out, s);
            case kQ4_K: return embed_blocks<kQ4_K>(b, vocab, k, ids, n, scale, out, s);
            case kQ5_K: return embed_blocks<kQ5_K>(b, vocab, k, ids, n, scale, out, s);
            case kQ6_K: return embed_blocks<kQ6_K>(b, vocab, k, ids, n, scale, out, s);
            case kIQ4_XS: return embed_blocks<kIQ4_XS>(b, vocab, k, ids, n, scale, out, s);
            default:
                return with_type(type, [&](auto e) -> hipError_t {
                    typedef decltype(e) E;
                    return embed_rows((const E *)table, vocab, k, ids, n, scale, out, s);
                });
        }
    });
}

size_t embed_backward_bytes(int64_t n, int64_t k, int64_t vocab) {
    if (n == 0) return 0;
    return up256(sort_ids_bytes(n, vocab, true)) + up256((size_t)n * 4) +
           up256((size_t)((n + kChunk - 1) / kChunk) * 2 * k * 4);
}

hipError_t launch_embed_backward(int dy_type, const void *dy, int64_t n, int64_t k, const int32_t *ids, int64_t vocab,
                                 float scale, int g_type, void *grad, uint8_t *ws, hipStream_t s) {
    return with_type(g_type, [&](auto o) -> hipError_t {
        typedef decltype(o) O;
        const int64_t cells = vocab * k, n16 = aligned16(grad) ? cells * (int64_t)sizeof(O) / 16 : 0;
        hipLaunchKernelGGL(fill_zero_kernel<O>, dim3(grid_of(n16)), dim3(256), 0, s, (O *)grad, n16, cells);
        if (n == 0) return hipGetLastError();
        int32_t *order = (int32_t *)(ws + up256(sort_ids_bytes(n, vocab, true)));
        float *part = (float *)((uint8_t *)order + up256((size_t)n * 4));
        hipError_t e = launch_sort_ids(ids, n, vocab, order, nullptr, nullptr, true, ws, s);
        if (e != hipSuccess) return e;
        const int32_t *skeys = sort_ids_keys(ws, n, vocab);
        return with_type(dy_type, [&](auto i) -> hipError_t {
            typedef decltype(i) E;
            if (k % 4 == 0 && aligned16(dy, grad))
                return grad_n<E, O, 4>((const E *)dy, n, k, order, skeys, vocab, scale, (O *)grad, part, s);
            return grad_n<E, O, 1>((const E *)dy, n, k, order, skeys, vocab, scale, (O *)grad, part, s);
        });
    });
}

}  // namespace qmm
