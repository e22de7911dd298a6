// First half of an adapter: part[s][i][r] = sum over slice s of K of v[i][j] * m[c][r][j] (forward,
// m = A) or of v[i][j] * m[c][j][r] (backward, v = dy and m = B), c the row's adapter.
//
// The row matrix v is read once and is nearly all of the traffic (n * k against rank * k weights an
// adapter, which L2 holds), so HBM bounds the large calls and latency the small ones.  A workgroup
// takes the rows of one adapter in a window of 64 and a slice of K; its four waves take 16 rows each,
// or, where there are fewer rows, turns at 32 K values of them, read straight into the operand
// registers of the matrix instructions: a wave has 16 rows, so there is no reuse that LDS would serve.
#include "launch.hpp"
#include "lora_parts.hpp"

namespace qmm {

namespace {

struct Args {
    const void *v, *m;
    const int32_t *ids;
    float *part;
    int64_t n, k, slice;
    int32_t n_adapters, key_bits, rank, slices, lanes;
};

// One 32-value step of K: operands as loaded.
template <class X, class W, int RT, bool KM> struct Step {
    Raw8<X> x;
    typename std::conditional<KM, Raw8<W>, Rows8<W, RT>>::type w[KM ? RT : 1];
};

template <class X, class W, int RT, bool KM, bool XV, bool WV>
struct Narrow {
    static constexpr bool kNat = kNative<X, W>;
    const X *x;             // the lane's row, at its group's first K value
    const W *w;             // KM: m[c], row RT * (lane % 16); else m[c] at column RT * (lane % 16)
    int64_t k, rank;
    int g8, r0;

    template <bool TAIL> __device__ __forceinline__ void load(Step<X, W, RT, KM> &s, int64_t kk) const {
        const int64_t left = k - kk - g8;
        if constexpr (TAIL) s.x = load8<XV>(x + kk, left);
        else s.x = load8(x + kk);
        if constexpr (KM) {
#pragma unroll
            for (int q = 0; q < RT; ++q) {   // ranks past the last repeat it: their sums are not used
                const W *p = w + (r0 + q < rank ? q : rank - 1 - r0) * k + kk + g8;
                if constexpr (TAIL) s.w[q] = load8<WV>(p, left);
                else s.w[q] = load8(p);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (!TAIL || e < left) {
                    s.w[0].row[e] = load_row<WV, RT>(w + (kk + g8 + e) * rank, (int)(rank - r0));
                } else {
#pragma unroll
                    for (int q = 0; q < RT; ++q) s.w[0].row[e].v[q] = (W)0.f;
                }
            }
        }
    }
    __device__ __forceinline__ void add(const Step<X, W, RT, KM> &s, f32x4 (&acc)[RT]) const {
        const auto a = parts_of<kNat>(s.x);
#pragma unroll
        for (int q = 0; q < RT; ++q) {
            Raw8<W> raw;
            if constexpr (KM) raw = s.w[q];
            else raw = s.w[0].column(q);
            acc[q] = mul_acc<X>(a, parts_of<kNat>(raw), acc[q]);
        }
    }
    // K values [lo, hi) in steps of 32 at a distance
    __device__ __forceinline__ void run(int64_t lo, int64_t hi, int distance, f32x4 (&acc)[RT]) const {
        // steps whose loads are in flight together
        constexpr int U = RT <= 2 ? 4 : 2;
        int64_t kk = lo;
        if constexpr (XV && (WV || !KM)) {
            for (; kk + distance * (U - 1) + 32 <= hi; kk += distance * U) {
                Step<X, W, RT, KM> s[U];
#pragma unroll
                for (int u = 0; u < U; ++u) load<false>(s[u], kk + distance * u);
#pragma unroll
                for (int u = 0; u < U; ++u) add(s[u], acc);
            }
            for (; kk + 32 <= hi; kk += distance) {
                Step<X, W, RT, KM> s;
                load<false>(s, kk);
                add(s, acc);
            }
        }
        for (; kk < hi; kk += distance) {
            Step<X, W, RT, KM> s;
            load<true>(s, kk);
            add(s, acc);
        }
    }
};

template <class X, class W, int RT, bool KM, bool XV, bool WV>
__global__ __launch_bounds__(256) void narrow_kernel(Args a) {
    constexpr int R = 16 * RT;
    __shared__ alignas(16) float red[3][16][R];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 15, g = lane >> 4;
    const int64_t s = slice_of_block();
    const int64_t lo = s * a.slice, hi = lo + a.slice < a.k ? lo + a.slice : a.k;
    for (int64_t i0 = (int64_t)blockIdx.z * kWindow; i0 < a.n; i0 += (int64_t)gridDim.z * kWindow) {
        const Tiles tiles = find_tiles(a.ids, i0, a.n, a.n_adapters, a.key_bits, false);
        for (int i = blockIdx.y; i < tiles.count; i += gridDim.y) {
            const Tile t = pick_tile(tiles, i);
            const int groups = t.groups(), slot0 = 16 * (wave % groups), turn = wave / groups, turns = 4 / groups;
            Narrow<X, W, RT, KM, XV, WV> op;
            op.k = a.k;
            op.rank = a.rank;
            op.g8 = 8 * g;
            op.r0 = RT * m < a.rank ? RT * m : a.rank - 1;
            if (WV && !KM && op.r0 + RT > a.rank) op.r0 = a.rank - RT;
            op.x = (const X *)a.v + (i0 + t.row(slot0 + m)) * a.k + op.g8;
            op.w = (const W *)a.m + (int64_t)t.key * a.rank * a.k + (KM ? op.r0 * a.k : op.r0);
            f32x4 acc[RT];
#pragma unroll
            for (int q = 0; q < RT; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (slot0 < t.rows) op.run(lo + 32 * turn, hi, 32 * turns, acc);
            if (turns > 1) {   // the waves of a group meet in LDS, in a fixed order
                if (turn > 0)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int q = 0; q < RT; ++q) red[wave - groups][4 * g + e][RT * m + q] = acc[q][e];
                __syncthreads();
                if (turn == 0)
                    for (int w = groups; w < 4; w += groups)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int q = 0; q < RT; ++q) acc[q][e] += red[w - groups + wave][4 * g + e][RT * m + q];
                __syncthreads();
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int slot = slot0 + 4 * g + e;
                const int64_t row = i0 + t.row(slot);
                if (turn == 0 && slot < t.rows) {
                    Piece<float, RT> o;
#pragma unroll
                    for (int q = 0; q < RT; ++q) o.v[q] = acc[q][e];
                    *(Piece<float, RT> *)(a.part + (s * a.n + row) * R + RT * m) = o;
                }
            }
        }
    }
}

int tiles_of_rank(int64_t rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }

// Slices of K: enough for two waves of 16 rows on each of the 1024 SIMD units, at most 16 partial sums
// a result, each of 128 values or more.
int slices_of(int64_t n, int64_t k) {
    const int64_t steps = (k + 127) / 128, groups = (n + 15) / 16;
    int64_t s = 2048 / groups;
    if (s > 16) s = 16;
    if (s > steps) s = steps;
    return s < 1 ? 1 : (int)s;
}

template <class X, class W, bool KM> hipError_t launch(const Args &a, bool xv, bool wv, hipStream_t st) {
    const dim3 grid = tile_grid(a.slices, a.lanes, a.n);
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
int lora_narrow_slices(int64_t n, int64_t k) { return slices_of(n, k); }

hipError_t launch_lora_narrow(int x_type, int w_type, bool by_row, const void *v, int64_t n, int64_t k, const void *m,
                              int64_t rank, int64_t n_adapters, const int32_t *ids, float *part, hipStream_t s) {
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
    a.lanes = tile_lanes(windows * a.slices, n, n_adapters);
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
