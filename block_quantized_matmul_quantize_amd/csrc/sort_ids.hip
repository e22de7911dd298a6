// Stable sort of indices by an int32 id: what the expert gather, the embedding gradient and the
// low-rank adapters group their rows with.  Ids outside [0, n_keys) take the key n_keys, so they
// come last.
//
// A least-significant-digit radix sort with digits of up to 11 bits: n_keys + 1 key values of up to
// 11 bits (any expert or adapter count) are one pass, a vocabulary of 2^18 two.  In a pass, each
// workgroup owns a contiguous chunk and each of its waves a contiguous part of that.  It needs the
// digits' counts over all chunks and over those before its own:
//   - up to kFused elements each workgroup counts all of them itself, so that a pass is one launch (the
//     ids, 256 KB at most, come from L2; counting them all again costs less than a launch);
//   - beyond, a launch before leaves one histogram per chunk.
// Then it counts per wave and places 64 elements at a time: lanes with equal digits find each other by
// one ballot per digit bit, a lane's rank is the number of such lanes below it.  No atomic decides an
// order, so the result is the stable one, always.
//
// Latency bounds it: 128 pairs by 128 experts 3.8 us, 16384 pairs 7.6 us (most of it counting, 64
// KB of ids in each of 16 workgroups), 16384 tokens by 131072 ids 2 x 9 us.
#include "common.hpp"
#include "launch.hpp"

namespace qmm {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kMaxBits = 11;
constexpr int64_t kFused = 65536;       // elements that every workgroup counts itself
constexpr int64_t kFusedChunk = 1024;   // and those it places: one step of its 16 waves
constexpr int64_t kMaxChunks = 128;

__device__ __forceinline__ int32_t key_of(const int32_t *ids, int64_t i, int32_t n_keys) {
    const int32_t v = ids[i];
    return (uint32_t)v < (uint32_t)n_keys ? v : n_keys;
}

struct Pass {
    const int32_t *ids;
    const int32_t *src;     // element order before this pass; null: 0, 1, 2, ...
    const int32_t *keys;    // keys in that order; null: those of ids
    int32_t *dst;           // element order after it
    int32_t *pos;           // last pass: each index's place, -1 for an id out of range
    int32_t *skeys;         // or null: the keys in the order after it
    int32_t *bounds;        // only pass, or null: first place of each key
    int32_t *table;         // [chunks][digits] histograms, or null: counted here
    int64_t n, chunk;
    int32_t n_keys, shift, bits;
};

__device__ __forceinline__ int32_t digit_of_key(const Pass &p, int32_t key) {
    return (key >> p.shift) & ((1 << p.bits) - 1);
}
__device__ __forceinline__ int32_t digit_of(const Pass &p, int64_t i) {
    return digit_of_key(p, p.keys ? p.keys[i] : key_of(p.ids, i, p.n_keys));
}

// hist[digit] += number of elements of [lo, hi), by all threads, sixteen elements a thread in flight.
// Where a whole wave has one digit (runs of one id) one lane adds for all.
__device__ __forceinline__ void count(const Pass &p, int64_t lo, int64_t hi, int32_t *hist) {
    typedef i32x4 __attribute__((aligned(4))) i32x4_a4;
    const int32_t *src = p.keys ? p.keys : p.ids;
    auto add = [&](int32_t v, bool in) {
        const uint64_t m = __ballot(in);
        if (m == 0) return;
        const int32_t d = digit_of_key(p, (uint32_t)v < (uint32_t)p.n_keys ? v : p.n_keys);
        const int32_t d0 = __builtin_amdgcn_readlane(d, __ffsll((unsigned long long)m) - 1);
        if (__ballot(in && d != d0) == 0) {
            if ((threadIdx.x & 63) == 0) atomicAdd(&hist[d0], __popcll(m));
        } else if (in) {
            atomicAdd(&hist[d], 1);
        }
    };
    int64_t i0 = lo;
    for (; i0 + 4 * kThreads <= hi; i0 += 16 * kThreads) {
        i32x4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t at = i0 + u * 4 * kThreads;
            v[u] = *(const i32x4_a4 *)(src + (at + 4 * kThreads <= hi ? at : i0) + 4 * threadIdx.x);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i0 + (u + 1) * 4 * kThreads <= hi)
#pragma unroll
                for (int q = 0; q < 4; ++q) add(v[u][q], true);
    }
    const int64_t done = lo + (hi - lo) / (4 * kThreads) * (4 * kThreads);
    for (int u = 0; u < 4; ++u) {
        const int64_t i = done + u * kThreads + threadIdx.x;
        if (done + u * kThreads < hi) add(src[i < hi ? i : done], i < hi);
    }
}

__global__ __launch_bounds__(kThreads) void count_kernel(Pass p) {
    extern __shared__ int32_t hist[];
    const int D = 1 << p.bits;
    for (int d = threadIdx.x; d < D; d += kThreads) hist[d] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * p.chunk, hi = lo + p.chunk < p.n ? lo + p.chunk : p.n;
    count(p, lo, hi, hist);
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kThreads) p.table[(int64_t)blockIdx.x * D + d] = hist[d];
}

// Exclusive scan of one value per thread over the workgroup.
__device__ __forceinline__ int32_t scan_threads(int32_t v, int32_t *wsum) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int32_t s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t u = __shfl_up(s, d);
        if (lane >= d) s += u;
    }
    if (lane == 63) wsum[wave] = s;
    __syncthreads();
    int32_t before = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) before += w < wave ? wsum[w] : 0;
    __syncthreads();
    return before + s - v;
}

__global__ __launch_bounds__(kThreads) void scatter_kernel(Pass p) {
    extern __shared__ int32_t hist[];   // [wave][digit]: counts, then the next place; [before, after][digit]
    __shared__ int32_t wsum[kWaves];
    const int D = 1 << p.bits;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool others = !p.table && gridDim.x > 1;
    for (int i = threadIdx.x; i < (kWaves + (others ? 2 : 0)) * D; i += kThreads) hist[i] = 0;
    __syncthreads();
    if (others) {
        const int64_t lo = blockIdx.x * p.chunk, hi = lo + p.chunk;
        count(p, 0, lo, hist + kWaves * D);
        if (hi < p.n) count(p, hi, p.n, hist + (kWaves + 1) * D);
    }
    // contiguous part of the chunk for each wave, a multiple of 64 elements
    const int64_t part = p.chunk / kWaves;
    const int64_t lo0 = blockIdx.x * p.chunk + wave * part;
    const int64_t lo = lo0 < p.n ? lo0 : p.n, hi = lo + part < p.n ? lo + part : p.n;
    int32_t *mine = hist + wave * D;
    for (int64_t i = lo + lane; i < hi; i += 64) atomicAdd(&mine[digit_of(p, i)], 1);
    __syncthreads();
    // first place of each digit: thread t owns digits [t * per, (t + 1) * per)
    const int per = (D + kThreads - 1) / kThreads;
    const int chunks = gridDim.x;
    int32_t total[(1 << kMaxBits) / kThreads], before[(1 << kMaxBits) / kThreads], sum = 0;
#pragma unroll
    for (int j = 0; j < (1 << kMaxBits) / kThreads; ++j) {
        const int d = threadIdx.x * per + j;
        total[j] = before[j] = 0;
        if (j < per && d < D) {
            if (!p.table) {
                for (int w = 0; w < kWaves; ++w) total[j] += hist[w * D + d];
                if (others) {
                    before[j] = hist[kWaves * D + d];
                    total[j] += before[j] + hist[(kWaves + 1) * D + d];
                }
            } else {
                for (int c = 0; c < chunks; ++c) {
                    const int32_t v = p.table[(int64_t)c * D + d];
                    total[j] += v;
                    before[j] += c < (int)blockIdx.x ? v : 0;
                }
            }
        }
        sum += total[j];
    }
    int32_t place = scan_threads(sum, wsum);
#pragma unroll
    for (int j = 0; j < (1 << kMaxBits) / kThreads; ++j) {
        const int d = threadIdx.x * per + j;
        if (j < per && d < D) {
            if (p.bounds && blockIdx.x == 0 && d <= p.n_keys) p.bounds[d] = place;
            int32_t at = place + before[j];
            for (int w = 0; w < kWaves; ++w) {
                const int32_t c = hist[w * D + d];
                hist[w * D + d] = at;
                at += c;
            }
        }
        place += total[j];
    }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 64) {
        const int64_t i = i0 + lane;
        const bool in = i < hi;
        const int32_t e = in ? (p.src ? p.src[i] : (int32_t)i) : 0;
        const int32_t key = in ? (p.keys ? p.keys[i] : key_of(p.ids, i, p.n_keys)) : 0;
        const int32_t d = (key >> p.shift) & (D - 1);
        uint64_t same = __ballot(in);
        for (int b = 0; b < p.bits; ++b) {
            const uint64_t set = __ballot((d >> b) & 1);
            same &= (d >> b) & 1 ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        int32_t at = 0;
        if (in) at = mine[d] + rank;
        // every lane has read its digit's place before the last lane of each digit moves it on
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (in && (same >> lane) == 1) mine[d] = at + 1;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (in) {
            p.dst[at] = e;
            if (p.pos) p.pos[e] = key < p.n_keys ? at : -1;
            if (p.skeys) p.skeys[at] = key;
        }
    }
}

// bounds[v] = first place whose key is >= v, by binary search in the sorted keys.
__global__ __launch_bounds__(256) void bounds_kernel(const int32_t *__restrict__ skeys, int64_t n, int64_t n_keys,
                                                     int32_t *__restrict__ bounds) {
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (v > n_keys) return;
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (skeys[mid] < v) lo = mid + 1;
        else hi = mid;
    }
    bounds[v] = (int32_t)lo;
}

struct Layout {
    int bits, passes;
    int64_t chunk, chunks;
    size_t table, tmp[2], keys[2], skeys, total;   // keys: of the passes before the last
};

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

Layout layout(int64_t n, int64_t n_keys, bool skeys) {
    Layout L{};
    int bits = 1;
    while ((n_keys >> bits) != 0) ++bits;
    L.passes = (bits + kMaxBits - 1) / kMaxBits;
    L.bits = (bits + L.passes - 1) / L.passes;
    if (n <= kFused) {
        L.chunk = kFusedChunk;
    } else {
        const int64_t c = (n + kMaxChunks - 1) / kMaxChunks;
        L.chunk = (c + kThreads - 1) / kThreads * kThreads;
    }
    L.chunks = n > 0 ? (n + L.chunk - 1) / L.chunk : 1;
    size_t off = 0;
    L.table = off;
    if (n > kFused) off += up256((size_t)L.chunks * ((size_t)4 << L.bits));
    for (int i = 0; i < 2; ++i) {
        L.tmp[i] = off;
        if (L.passes > 1 + i) off += up256((size_t)n * 4);
        L.keys[i] = off;
        if (L.passes > 1 + i) off += up256((size_t)n * 4);
    }
    L.skeys = off;
    if (skeys || L.passes > 1) off += up256((size_t)n * 4);
    L.total = off;
    return L;
}

}  // namespace

size_t sort_ids_bytes(int64_t n, int64_t n_keys, bool with_keys) { return layout(n, n_keys, with_keys).total; }

const int32_t *sort_ids_keys(const void *ws, int64_t n, int64_t n_keys) {
    return (const int32_t *)((const uint8_t *)ws + layout(n, n_keys, true).skeys);
}

hipError_t launch_sort_ids(const int32_t *ids, int64_t n, int64_t n_keys, int32_t *order, int32_t *pos,
                           int32_t *bounds, bool with_keys, uint8_t *ws, hipStream_t s) {
    const Layout L = layout(n, n_keys, with_keys);
    Pass p{};
    p.ids = ids;
    p.n = n;
    p.n_keys = (int32_t)n_keys;
    p.chunk = L.chunk;
    p.bits = L.bits;
    p.table = n > kFused ? (int32_t *)(ws + L.table) : nullptr;
    int32_t *skeys = with_keys || L.passes > 1 ? (int32_t *)(ws + L.skeys) : nullptr;
    for (int i = 0; i < L.passes; ++i) {
        const bool last = i + 1 == L.passes;
        p.shift = i * L.bits;
        p.src = i == 0 ? nullptr : p.dst;
        p.keys = i == 0 ? nullptr : p.skeys;
        p.dst = last ? order : (int32_t *)(ws + L.tmp[i & 1]);
        p.skeys = last ? skeys : (int32_t *)(ws + L.keys[i & 1]);
        p.pos = last ? pos : nullptr;
        p.bounds = L.passes == 1 ? bounds : nullptr;
        if (p.table)
            hipLaunchKernelGGL(count_kernel, dim3((unsigned)L.chunks), dim3(kThreads), (size_t)4 << L.bits, s, p);
        hipLaunchKernelGGL(scatter_kernel, dim3((unsigned)L.chunks), dim3(kThreads),
                           (size_t)(4 * (kWaves + 2)) << L.bits, s, p);
    }
    if (bounds && L.passes > 1)
        hipLaunchKernelGGL(bounds_kernel, dim3((unsigned)((n_keys + 256) / 256)), dim3(256), 0, s, skeys, n, n_keys,
                           bounds);
    return hipGetLastError();
}

}  // namespace qmm
