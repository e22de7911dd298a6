// Embedding lookup: y[i] = scale * table[ids[i]], the table rows fp32, fp16, bf16 or GGUF blocks that
// are decoded on the way (embedding tables ship in the same block types as the weights), and its
// gradient: dT[v] = scale * (sum of dy[i] over the tokens with id v), over tokens sorted by id.
//
// The lookup reads each named row's bytes and writes y, a few operations a value: launch latency bounds
// a step's 8 tokens (3 us), HBM the large calls (2048 rows of 4096 Q6_K values into fp32: 11 us, 40 MB
// at 3.7 TB/s, 83 % of it the output).  A thread decodes 8 neighbouring values, so that it stores 16
// or 32 bytes and finds their scale once.  Tables of elements, 2048 rows of 4096 values into fp32: 12.5 us
// from fp32 (5.4 TB/s), 10.4 us from bf16; one value a thread, where rows are no multiple of 8 values or an
// address none of 16 bytes: 20.7 us (4092 and 4095 fp32 values).
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
// The gradient is bound by the write of the whole table (most of whose rows no token names), so it is
// written once: a launch sums the rows that have tokens and clears others beside that, which it tells
// apart by a search in the sorted ids.
//
// Sums: chunks of kChunk sorted tokens; a workgroup sums the rows of one chunk, N columns (16 bytes) a
// thread, from one id to the next, eight rows in flight.  An id whose tokens lie in one chunk is written
// at once; the others leave their sums in part[chunk][0] (the id began before this chunk) or
// part[chunk][1] (it goes on after it), which a second launch adds up in chunk order: the sum's order is
// fixed.
constexpr int kChunk = 32;

struct Grad {
    const void *dy;
    const int32_t *skeys, *order;
    void *grad;
    float *part;
    int64_t n, k, vocab;
    int64_t chunks, slices;     // workgroups of the sums or joins: chunks x slices of the columns
    int64_t row0, row1;         // table rows to clear where no token names them,
    int64_t fill_rows;          // this many a workgroup
    int64_t blocks;
    float scale;
};

template <class E, class O, int N> __device__ __forceinline__ void sum_chunk(const Grad &a, int64_t c, int64_t slice) {
    const E *dy = (const E *)a.dy;
    const int64_t e0 = c * kChunk;
    const int cnt = (int)(a.n - e0 < kChunk ? a.n - e0 : kChunk);
    const int64_t col = (slice * blockDim.x + threadIdx.x) * N;
    const int32_t vocab = (int32_t)a.vocab;
    const bool mine = col < a.k;
    const E *at = dy + (mine ? col : 0);
    int32_t cur = a.skeys[e0];
    bool starts = e0 == 0 || a.skeys[e0 - 1] != cur;
    float acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.f;
    auto flush = [&](bool ends) {
        if (!mine) return;
        if (starts && ends) {
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] *= a.scale;
            store_n<N>((O *)a.grad + cur * a.k + col, acc);
        } else {
            store_n<N>(a.part + (2 * c + (starts ? 1 : 0)) * a.k + col, acc);
        }
    };
    for (int e = 0; e < cnt && cur < vocab; e += 8) {
        float v[8][N];
#pragma unroll
        for (int u = 0; u < 8; ++u) load_n<N>(at + a.order[e0 + (e + u < cnt ? e + u : cnt - 1)] * a.k, v[u]);
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int j = 0; j < N; ++j) asm volatile("" : "+v"(v[u][j]));   // loaded here, not one by one at their use
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (e + u >= cnt || cur >= vocab) break;
            const int32_t key = a.skeys[e0 + e + u];
            if (key != cur) {
                flush(true);
                cur = key;
                starts = true;
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] = 0.f;
                if (key >= vocab) break;
            }
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += v[u][j];
        }
    }
    if (cur < vocab) flush(e0 + cnt == a.n || a.skeys[e0 + cnt] != cur);
}

// First place of the sorted keys that is >= key, by a whole wave: 64 probes a round.
__device__ __forceinline__ int64_t lower_bound(const int32_t *skeys, int64_t n, int64_t key) {
    int64_t lo = 0, hi = n;   // the answer is in [lo, hi]
    while (lo < hi) {
        const int64_t step = (hi - lo + 63) / 64, at = lo + (threadIdx.x & 63) * step;
        const int below = __popcll(__ballot(at < hi && skeys[at < hi ? at : hi - 1] < key));
        if (below == 0) return lo;
        lo += (below - 1) * step + 1;
        if (lo + step - 1 < hi) hi = lo + step - 1;
    }
    return lo;
}

constexpr int kMaxFill = 1024;

template <class O, int N> __device__ __forceinline__ void clear_rows(const Grad &a, int64_t v0, uint8_t *named) {
    const int rows = (int)(a.row1 - v0 < a.fill_rows ? a.row1 - v0 : a.fill_rows);
    for (int i = threadIdx.x; i < rows; i += blockDim.x) named[i] = 0;
    __syncthreads();
    const int64_t lo = lower_bound(a.skeys, a.n, v0), hi = lower_bound(a.skeys, a.n, v0 + rows);
    for (int64_t i = lo + threadIdx.x; i < hi; i += blockDim.x) named[a.skeys[i] - v0] = 1;
    __syncthreads();
    const int groups = (int)(a.k / N);
    float z[N];
#pragma unroll
    for (int j = 0; j < N; ++j) z[j] = 0.f;
    O *g = (O *)a.grad + v0 * a.k;
    if (groups >= (int)blockDim.x) {
        for (int r = 0; r < rows; ++r)
            if (!named[r])
                for (int i = threadIdx.x; i < groups; i += blockDim.x) store_n<N>(g + r * a.k + (int64_t)i * N, z);
    } else {
        for (int i = threadIdx.x; i < rows * groups; i += blockDim.x)
            if (!named[i / groups]) store_n<N>(g + (int64_t)i * N, z);
    }
}

// Only for a chunk in which an id begins that goes on after it.
template <class O, int N> __device__ __forceinline__ void join_chunk(const Grad &a, int64_t c, int64_t slice) {
    const int64_t e0 = c * kChunk, e1 = e0 + kChunk;
    if (e1 >= a.n) return;
    // every key that decides is loaded before any is looked at
    auto first_of = [&](int64_t q) { return a.skeys[q * kChunk < a.n ? q * kChunk : e0]; };
    int32_t key = a.skeys[e1 - 1], after = a.skeys[e1], begin = a.skeys[e0], before = a.skeys[e0 > 0 ? e0 - 1 : 0];
    int32_t next = first_of(c + 1 + (threadIdx.x & 63));
    asm volatile("" : "+v"(key), "+v"(after), "+v"(begin), "+v"(before), "+v"(next));
    key = __builtin_amdgcn_readfirstlane(key);
    if (key >= a.vocab || after != key || (begin == key && e0 > 0 && before == key)) return;
    // chunks c + 1 .. last begin with the same id
    int64_t last = c + 1;
    for (;;) {
        const uint64_t other = __ballot((last + (threadIdx.x & 63)) * kChunk >= a.n || next != key);
        if (other) {
            last += __ffsll((unsigned long long)other) - 1;
            break;
        }
        last += 64;
        next = first_of(last + (threadIdx.x & 63));
    }
    const int64_t col = (slice * blockDim.x + threadIdx.x) * N;
    if (col >= a.k) return;
    float acc[N];
    load_n<N>(a.part + (2 * c + 1) * a.k + col, acc);
    for (int64_t q = c + 1; q < last; q += 16) {   // a chunk past the last is read as the last, and left out
        float v[16][N];
#pragma unroll
        for (int u = 0; u < 16; ++u) load_n<N>(a.part + 2 * (q + u < last ? q + u : last - 1) * a.k + col, v[u]);
#pragma unroll
        for (int u = 0; u < 16; ++u)
            for (int j = 0; j < N; ++j) acc[j] += q + u < last ? v[u][j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] *= a.scale;
    store_n<N>((O *)a.grad + key * a.k + col, acc);
}

// Sums (or joins) in the first workgroups, clears in the others: N columns a thread of dy or of the
// partial sums, M of the rows it clears (16 bytes where the rows allow it).
template <class E, class O, int N, int M, bool JOIN> __global__ __launch_bounds__(256) void grad_kernel(Grad a) {
    __shared__ uint8_t named[kMaxFill];
    const int64_t first = a.chunks * a.slices;
    for (int64_t b = blockIdx.x; b < a.blocks; b += gridDim.x) {
        if (b < first) {
            if constexpr (JOIN) join_chunk<O, N>(a, b % a.chunks, b / a.chunks);
            else sum_chunk<E, O, N>(a, b % a.chunks, b / a.chunks);
        } else {
            clear_rows<O, M>(a, a.row0 + (b - first) * a.fill_rows, named);
            __syncthreads();
        }
    }
}

constexpr int64_t kMaxGrid = 1 << 22;
int threads_of(int64_t groups) { return groups >= 256 ? 256 : (int)((groups + 63) / 64 * 64); }

template <class E, class O, int N, int M, bool JOIN> hipError_t grad_part(Grad a, int64_t row0, int64_t row1, hipStream_t s) {
    const int threads = threads_of((a.k + N - 1) / N);
    a.chunks = (a.n + kChunk - 1) / kChunk;
    a.slices = a.n ? (a.k + (int64_t)N * threads - 1) / ((int64_t)N * threads) : 0;
    // about 128 KB a workgroup that clears
    a.fill_rows = 131072 / (a.k * (int64_t)sizeof(O));
    a.fill_rows = a.fill_rows < 1 ? 1 : a.fill_rows > kMaxFill ? kMaxFill : a.fill_rows;
    a.row0 = row0;
    a.row1 = row1;
    a.blocks = a.chunks * a.slices + (row1 - row0 + a.fill_rows - 1) / a.fill_rows;
    hipLaunchKernelGGL((grad_kernel<E, O, N, M, JOIN>), dim3((unsigned)(a.blocks < kMaxGrid ? a.blocks : kMaxGrid)),
                       dim3(threads), 0, s, a);
    return hipGetLastError();
}

template <class E, class O, int N, int M> hipError_t grad_n(const Grad &a, hipStream_t s) {
    // A table beyond the 256 MB cache is cleared half beside the sums and half beside the joins, which
    // would otherwise wait for its writes to drain (1 GB: 256 against 264 us); a smaller one beside the sums
    // (131 MB: 39 against 43 us).
    const int64_t half = a.n > kChunk && a.vocab * a.k * (int64_t)sizeof(O) > (256 << 20) ? a.vocab / 2 : a.vocab;
    hipError_t e = grad_part<E, O, N, M, false>(a, 0, half, s);
    if (e != hipSuccess || a.n <= kChunk) return e;
    return grad_part<float, O, N < 4 ? N : 4, M, true>(a, half, a.vocab, s);
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
    Grad a{};
    a.dy = dy;
    a.grad = grad;
    a.n = n;
    a.k = k;
    a.vocab = vocab;
    a.scale = scale;
    if (n > 0) {
        int32_t *order = (int32_t *)(ws + up256(sort_ids_bytes(n, vocab, true)));
        a.part = (float *)((uint8_t *)order + up256((size_t)n * 4));
        hipError_t e = launch_sort_ids(ids, n, vocab, order, nullptr, nullptr, true, ws, s);
        if (e != hipSuccess) return e;
        a.skeys = sort_ids_keys(ws, n, vocab);
        a.order = order;
    }
    return with_type(dy_type, [&](auto i) -> hipError_t {
        typedef decltype(i) E;
        return with_type(g_type, [&](auto o) -> hipError_t {
            typedef decltype(o) O;
            constexpr int N = 16 / sizeof(E), M = 16 / sizeof(O);
            if (k % (N > M ? N : M) == 0 && aligned16(dy, grad)) return grad_n<E, O, N, M>(a, s);
            return grad_n<E, O, 1, 1>(a, s);
        });
    });
}

}  // namespace qmm
