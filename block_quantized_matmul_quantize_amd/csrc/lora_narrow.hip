// First half of an adapter: part[s][i][r] = sum over slice s of K of v[i][j] * m[c][r][j] (forward,
// m = A) or of v[i][j] * m[c][j][r] (backward, v = dy and m = B), c the row's adapter.
//
// The row matrix v is read once and is nearly all of the traffic (n * k against rank * k weights an
// adapter, which L2 holds), so HBM bounds the large calls and latency the small ones.  A workgroup
// takes the rows of one adapter in a window of 64 and a slice of K; its four waves take turns at 32 K
// values of all its rows, read straight into the operand registers of the matrix instructions (nothing
// is read twice within a workgroup, so LDS would serve no reuse), two or four steps in flight; one from rank
// 33 on where a tile has more than 32 rows, and from rank 65 on.  The waves' sums meet in LDS, in a fixed order.
//
// 2048 rows of 4096 fp32 values at rank 16: 10.8 us (3.1 TB/s); 8192 rows of 4096 bf16 values at rank
// 64, transposed: 20 us in runs of 256 rows (3.3 TB/s), 24 us in runs of any length; 32 rows of 64 adapters:
// 4.6 us.  At rank 64 nothing is in flight while a step is multiplied, which keeps these from a copy's rate.
#include "launch.hpp"
#include "lora_parts.hpp"
#include "sort_rows.hpp"

namespace qmm {

namespace {

struct Args {
    const void *v, *m;
    const int32_t *ids;
    float *part;
    int64_t n, k, slice;
    int32_t *order, *pos, *bounds;   // or null: the rows sorted by adapter, by one workgroup beside the others
    int32_t n_adapters, key_bits, rank, slices, lanes, parts;
};

// One 32-value step of K: operands as loaded.
template <class X, class W, int MT, int RT, bool KM> struct Step {
    Raw8<X> x[MT];
    typename std::conditional<KM, Raw8<W>, Rows8<W, RT>>::type w[KM ? RT : 1];
};

template <class X, class W, int MT, int RT, bool KM, bool XV, bool WV>
struct Narrow {
    static constexpr bool kNat = kNative<X, W>;
    typedef Step<X, W, MT, RT, KM> S;
    const X *x[MT];         // the lane's rows, at its group's first K value
    const W *w;             // KM: m[c], row r0; else m[c] at column r0
    int64_t k, rank;
    int g8, r0;

    template <bool TAIL> __device__ __forceinline__ void load(S &s, int64_t kk) const {
        const int64_t left = k - kk - g8;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if constexpr (TAIL) s.x[t] = load8<XV>(x[t] + kk, left);
            else s.x[t] = XV ? load8(x[t] + kk) : load8_any(x[t] + kk);
        }
        if constexpr (KM) {
#pragma unroll
            for (int q = 0; q < RT; ++q) {   // ranks past the last repeat it: their sums are not used
                const W *p = w + (r0 + q < rank ? q : rank - 1 - r0) * k + kk + g8;
                if constexpr (TAIL) s.w[q] = load8<WV>(p, left);
                else s.w[q] = WV ? load8(p) : load8_any(p);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (!TAIL || e < left) {
                    const W *p = w + (kk + g8 + e) * rank;
                    s.w[0].row[e] = WV ? load_row<true, RT>(p, RT) : load_any<RT>(p);
                } else {
#pragma unroll
                    for (int q = 0; q < RT; ++q) s.w[0].row[e].v[q] = (W)0.f;
                }
            }
        }
    }
    __device__ __forceinline__ void add(const S &s, f32x4 (&acc)[MT][RT]) const {
        decltype(parts_of<kNat>(s.x[0])) a[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) a[t] = parts_of<kNat>(s.x[t]);
#pragma unroll
        for (int q = 0; q < RT; ++q) {
            Raw8<W> raw;
            if constexpr (KM) raw = s.w[q];
            else raw = s.w[0].column(q);
            const auto b = parts_of<kNat>(raw);
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[t][q] = mul_acc<X>(a[t], b, acc[t][q]);
        }
    }
    // K values [lo, hi) in steps of 32 at a distance of 128
    __device__ __forceinline__ void run(int64_t lo, int64_t hi, f32x4 (&acc)[MT][RT]) const {
        // steps whose loads are in flight together: 8 to 16 KB a wave
        constexpr int U = RT >= 4 ? (RT == 8 || MT == 4 ? 1 : 2) : MT == 4 ? 2 : 4;
        int64_t kk = lo;
        for (; kk + 128 * (U - 1) + 32 <= hi; kk += 128 * U) {
            S s[U];
#pragma unroll
            for (int u = 0; u < U; ++u) load<false>(s[u], kk + 128 * u);
#pragma unroll
            for (int u = 0; u < U; ++u) add(s[u], acc);
        }
        if constexpr (U > 1)
            for (; kk + 32 <= hi; kk += 128) {
                S s;
                load<false>(s, kk);
                add(s, acc);
            }
        for (; kk < hi; kk += 128) {
            S s;
            load<true>(s, kk);
            add(s, acc);
        }
    }
};

template <class X, class W, int RT, bool KM, bool XV, bool WV>
__global__ __launch_bounds__(256, RT == 8 ? 1 : 2) void narrow_kernel(Args a) {
    constexpr int R = 16 * RT;
    __shared__ alignas(16) float red[kWindow][R];
    static_assert(sizeof(red) >= kSortRowsLds * sizeof(int32_t));
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 15, g = lane >> 4;
    if (blockIdx.x >= (unsigned)a.slices) {
        if (blockIdx.y == 0 && blockIdx.z == 0)
            sort_rows(a.ids, a.n, a.n_adapters, a.key_bits, a.order, a.pos, a.bounds, (int32_t *)&red[0][0]);
        return;
    }
    const int64_t s = slice_of_block(a.slices);
    const int64_t lo = s * a.slice, hi = lo + a.slice < a.k ? lo + a.slice : a.k;
    for (int64_t i0 = (int64_t)blockIdx.y * kWindow; i0 < a.n; i0 += (int64_t)gridDim.y * kWindow) {
        const Tiles tiles = find_tiles(a.ids, i0, a.n, a.n_adapters, a.key_bits, false);
        for (int i = blockIdx.z % a.lanes; i < tiles.count; i += a.lanes) {
            Tile t = pick_tile(tiles, i);
            if (a.parts > 1) t = part_of(t, blockIdx.z / a.lanes);
            if (t.rows <= 0) continue;
            with_groups(t, [&](auto groups) {
                constexpr int MT = decltype(groups)::value;
                Narrow<X, W, MT, RT, KM, XV, WV> op;
                op.k = a.k;
                op.rank = a.rank;
                op.g8 = 8 * g;
                // ranks past the last repeat valid ones: KM the last, else the last RT, so that a piece of ranks
                // lies within its row; of a rank that is no multiple of RT, those below `own` are another lane's
                op.r0 = KM ? (RT * m < a.rank ? RT * m : a.rank - 1) : (RT * m + RT <= a.rank ? RT * m : a.rank - RT);
                const int own = RT * m - op.r0;
#pragma unroll
                for (int u = 0; u < MT; ++u) op.x[u] = (const X *)a.v + (i0 + t.row(16 * u + m)) * a.k + op.g8;
                op.w = (const W *)a.m + (int64_t)t.key * a.rank * a.k + (KM ? op.r0 * a.k : op.r0);
                f32x4 acc[MT][RT];
#pragma unroll
                for (int u = 0; u < MT; ++u)
#pragma unroll
                    for (int q = 0; q < RT; ++q) acc[u][q] = f32x4{0.f, 0.f, 0.f, 0.f};
                op.run(lo + 32 * wave, hi, acc);
#pragma unroll 1
                for (int w = 0; w < 4; ++w) {
                    if (w == wave)
#pragma unroll
                        for (int u = 0; u < MT; ++u)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
#pragma unroll
                                for (int q = 0; q < RT; ++q) {
                                    if (!KM && !WV && q < own) continue;
                                    float *p = &red[16 * u + 4 * g + e][KM || WV ? RT * m + q : op.r0 + q];
                                    *p = w ? *p + acc[u][q][e] : acc[u][q][e];
                                }
                    __syncthreads();
                }
            });
            for (int j0 = 0; j0 < t.rows * (R / 4); j0 += 256) {
                const int j = j0 + threadIdx.x, slot = j / (R / 4), r = j % (R / 4) * 4;
                const int64_t row = i0 + t.row(slot);   // every lane takes part in the exchange
                if (slot < t.rows) *(f32x4 *)(a.part + (s * a.n + row) * R + r) = *(const f32x4 *)&red[slot][r];
            }
            __syncthreads();
        }
    }
}

int tiles_of_rank(int64_t rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }

// Slices of K: enough for 256 workgroups (2048 rows: 11.5 us, 14.4 us with 512), at most 8 partial sums a
// result (32 rows: 6.5 us in the second half, 7.0 us with 16), each of 128 values or more.
int slices_of(int64_t n, int64_t k) {
    const int64_t steps = (k + 127) / 128, windows = (n + kWindow - 1) / kWindow;
    int64_t s = 256 / windows;
    if (s > 8) s = 8;
    if (s > steps) s = steps;
    return s < 1 ? 1 : (int)s;
}

template <class X, class W, bool KM> hipError_t launch(const Args &a, bool xv, bool wv, hipStream_t st) {
    const dim3 grid = tile_grid(a.slices + (a.order ? 1 : 0), a.lanes * a.parts, a.n);
    auto go = [&](auto rt) -> hipError_t {
        constexpr int RT = decltype(rt)::value;
        if (xv && wv)
            hipLaunchKernelGGL((narrow_kernel<X, W, RT, KM, true, true>), grid, dim3(256), 0, st, a);
        else if (xv && !KM)
            hipLaunchKernelGGL((narrow_kernel<X, W, RT, KM, true, KM>), grid, dim3(256), 0, st, a);
        else
            hipLaunchKernelGGL((narrow_kernel<X, W, RT, KM, false, false>), grid, dim3(256), 0, st, a);
        return hipGetLastError();
    };
    switch (tiles_of_rank(a.rank)) {
        case 1: return go(std::integral_constant<int, 1>{});
        case 2: return go(std::integral_constant<int, 2>{});
        case 4: return go(std::integral_constant<int, 4>{});
        default: return go(std::integral_constant<int, 8>{});
    }
}

}  // namespace

int lora_padded_rank(int64_t rank) { return 16 * tiles_of_rank(rank); }
// One workgroup's sort hides beside the others' product: 2048 rows 6.6 us against 8.4 us in two launches;
// 8192 rows of 64 values take it 19.6 us, against 10.7 us.
bool lora_narrow_sorts(int64_t n, int64_t n_adapters) { return n <= 2048 && n_adapters <= kSortRowsKeys; }
int lora_narrow_slices(int64_t n, int64_t k) { return slices_of(n, k); }

hipError_t launch_lora_narrow(int x_type, int w_type, bool by_row, const void *v, int64_t n, int64_t k, const void *m,
                              int64_t rank, int64_t n_adapters, const int32_t *ids, float *part, int32_t *order, int32_t *pos,
                              int32_t *bounds, hipStream_t s) {
    Args a{};
    a.v = v;
    a.m = m;
    a.ids = ids;
    a.part = part;
    a.n = n;
    a.k = k;
    a.rank = (int32_t)rank;
    a.n_adapters = (int32_t)n_adapters;
    a.key_bits = key_bits_of(n_adapters);
    a.slices = slices_of(n, k);
    a.slice = ((k + a.slices - 1) / a.slices + 127) / 128 * 128;
    const int64_t windows = (n + kWindow - 1) / kWindow;
    a.order = order;
    a.pos = pos;
    a.bounds = bounds;
    a.lanes = tile_lanes(windows * a.slices, n, n_adapters);
    a.parts = tile_parts(windows * a.slices, a.lanes, n, n_adapters);
    return with_lora_types(x_type, w_type, [&](auto x, auto w) -> hipError_t {
        typedef decltype(x) X;
        typedef decltype(w) W;
        const bool xv = k % 8 == 0 && aligned16(v);
        const int rt = tiles_of_rank(rank);
        const size_t piece = rt * sizeof(W) < 16 ? rt * sizeof(W) : 16;
        if (by_row) return launch<X, W, true>(a, xv && aligned16(m), xv && aligned16(m), s);
        return launch<X, W, false>(a, xv, rank % rt == 0 && (uintptr_t)m % piece == 0, s);
    });
}

}  // namespace qmm
