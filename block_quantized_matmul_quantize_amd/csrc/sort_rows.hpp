// Stable sort of row numbers by a small key, by one workgroup of 256 threads beside others that do
// something else: the counting sort of sort_ids.hip with one digit (of up to 8 bits) and four waves.
#pragma once
#include "common.hpp"

namespace qmm {

constexpr int kSortRowsKeys = 255;      // keys 0 .. n_keys, n_keys for an id out of range
constexpr int kSortRowsLds = 4 * (kSortRowsKeys + 1);   // int32 of LDS

// order [n], pos [n], bounds [n_keys + 1] as qmm_sort_ids; every thread of the workgroup calls it.
__device__ __forceinline__ void sort_rows(const int32_t *__restrict__ ids, int64_t n, int32_t n_keys, int key_bits,
                                          int32_t *__restrict__ order, int32_t *__restrict__ pos,
                                          int32_t *__restrict__ bounds, int32_t *lds) {
    constexpr int U = 8;   // steps of 64 rows whose ids are in flight together
    const int D = kSortRowsKeys + 1;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
#pragma unroll
    for (int w = 0; w < 4; ++w) lds[w * D + tid] = 0;
    __syncthreads();
    const int64_t part = (n + 255) / 256 * 64, lo = wave * part < n ? wave * part : n, hi = lo + part < n ? lo + part : n;
    int32_t *mine = lds + wave * D;
    auto each = [&](auto f) {   // f(row, key, whether there is such a row), in steps of a wave
        for (int64_t i0 = lo; i0 < hi; i0 += 64 * U) {
            int32_t id[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = i0 + 64 * u + lane;
                id[u] = ids[i < hi ? i : lo];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = i0 + 64 * u + lane;
                if (i0 + 64 * u < hi) f(i, (uint32_t)id[u] < (uint32_t)n_keys ? id[u] : n_keys, i < hi);
            }
        }
    };
    // lanes of this step with the lane's key
    auto same_of = [&](int32_t key, bool in) {
        uint64_t same = __ballot(in);
        for (int b = 0; b < key_bits; ++b) {
            const uint64_t set = __ballot((key >> b) & 1);
            same &= (key >> b) & 1 ? set : ~set;
        }
        return same;
    };
    each([&](int64_t, int32_t key, bool in) {
        const uint64_t same = same_of(key, in);
        if (in && (same >> lane) == 1) mine[key] += __popcll(same);   // one lane a key
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    });
    __syncthreads();
    // thread d: places of key d
    int32_t c[4], total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        c[w] = lds[w * D + tid];
        total += c[w];
    }
    int32_t s = total;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t u = __shfl_up(s, d);
        if (lane >= d) s += u;
    }
    __syncthreads();
    if (lane == 63) lds[wave] = s;
    __syncthreads();
    int32_t at = s - total;
#pragma unroll
    for (int w = 0; w < 3; ++w) at += w < wave ? lds[w] : 0;
    __syncthreads();
    if (tid <= n_keys) bounds[tid] = at;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        lds[w * D + tid] = at;
        at += c[w];
    }
    __syncthreads();
    each([&](int64_t i, int32_t key, bool in) {
        const uint64_t same = same_of(key, in);
        int32_t place = 0;
        if (in) place = mine[key] + __popcll(same & ((1ull << lane) - 1));
        // every lane has read its key's place before the last lane of each key moves it on
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (in && (same >> lane) == 1) mine[key] = place + 1;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (in) {
            order[place] = (int32_t)i;
            pos[i] = key < n_keys ? place : -1;
        }
    });
}

}  // namespace qmm
