// Second half of an adapter: out[i][j] = base[i][j] + sum over r of h[i][r] * m[c][j][r] (forward,
// m = B) or * m[c][r][j] (backward, m = A), where h[i][r] = scale[c] * sum of the first half's slices;
// rows without an adapter get base, or zeros.
//
// It reads base and writes out, 8 bytes an fp32 result, against a few operations for each: HBM bounds
// it.  A workgroup takes the rows of one adapter in a window of 64 and a slice of the columns; each of
// its four waves 16 rows, or, where there are fewer, its share of the columns.  A wave adds up the
// slices of its rows' h and keeps their bf16 parts in registers for all its columns.  Lane l % 16 owns
// four neighbouring columns of a row, so that base is read and out written 256 (fp32) or 128 bytes a
// row at a time, straight from the accumulators: column q of the lanes' pieces is one matrix
// instruction's 16 columns.  No wave waits for another.
#include "launch.hpp"
#include "lora_parts.hpp"

namespace qmm {

namespace {

constexpr int kPiece = 4;   // neighbouring columns of a lane: 16 bytes of fp32, 8 of the other types

struct Args {
    const float *part;
    const void *m, *base;
    void *out;
    const int32_t *ids;
    const float *scale;
    int64_t n, cols, slice;
    int32_t n_adapters, key_bits, rank, padded, parts, slices, lanes;
};

template <class X, class W, int KS, bool KM, bool OV, bool WV>
__global__ __launch_bounds__(256, KS == 1 ? 4 : KS == 2 ? 3 : 2) void wide_kernel(Args a) {
    constexpr int R = 32 * KS;                        // K of the product
    constexpr int V = kPiece;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 15, g = lane >> 4;
    const int64_t slice = slice_of_block();
    const int64_t lo = slice * a.slice, hi = lo + a.slice < a.cols ? lo + a.slice : a.cols;
    for (int64_t i0 = (int64_t)blockIdx.z * kWindow; i0 < a.n; i0 += (int64_t)gridDim.z * kWindow) {
        const Tiles tiles = find_tiles(a.ids, i0, a.n, a.n_adapters, a.key_bits, true);
        for (int i = blockIdx.y; i < tiles.count; i += gridDim.y) {
            const Tile t = pick_tile(tiles, i);
            const bool some = t.key < a.n_adapters;
            const int groups = t.groups(), slot0 = 16 * (wave % groups), turns = 4 / groups;
            int64_t c0 = lo + wave / groups * (16 * V);
            if (slot0 >= t.rows || c0 >= hi) continue;
            int64_t row[4];
            bool live[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int slot = slot0 + 4 * g + e;
                live[e] = slot < t.rows;
                row[e] = (i0 + t.row(slot)) * a.cols;   // slots past the last: row of slot 0, not stored
            }
            const X *base = (const X *)a.base;
            const W *w = (const W *)a.m + (int64_t)t.key * a.rank * a.cols;
            // a lane's columns: all V, or some, or none at the end (nothing of those is stored)
            auto col_of = [&](int64_t at) { return at + V * m < hi ? at + V * m : OV ? hi - V : hi - 1; };
            auto width_of = [&](int64_t col) { return OV || hi - col >= V ? V : (int)(hi - col); };
            Piece<X, V> b[4];
            auto load_base = [&](int64_t at) {
                const int64_t col = col_of(at);
#pragma unroll
                for (int e = 0; e < 4; ++e) b[e] = load_row<OV, V>(base + row[e] + col, width_of(col));
            };
            if (base) load_base(c0);
            Frag<3> h[KS];
            if (some) {
                const float c = a.scale ? a.scale[t.key] : 1.f;
                const float *p = a.part + (i0 + t.row(slot0 + m)) * a.padded;
                const int64_t next = a.n * a.padded;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const int r0 = 32 * s + 8 * g;
                    const float *q = p + (r0 < a.padded ? r0 : 0);
                    f32x4 u0 = *(const f32x4 *)q, u1 = *(const f32x4 *)(q + 4);
#pragma unroll 4
                    for (int i = 1; i < a.parts; ++i) {
                        u0 += *(const f32x4 *)(q + i * next);
                        u1 += *(const f32x4 *)(q + i * next + 4);
                    }
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)   // ranks past the last hold nothing of use
                        v[e] = r0 + e < a.rank ? (e < 4 ? u0[e & 3] : u1[e & 3]) * c : 0.f;
                    h[s] = split8<3>(v);
                }
            }
            for (; c0 < hi; c0 += turns * 16 * V) {
                const int64_t col = col_of(c0);
                const int nw = width_of(col);
                f32x4 acc[V];
#pragma unroll
                for (int q = 0; q < V; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (some) {
#pragma unroll
                    for (int s = 0; s < KS; ++s) {
                        const int r0 = 32 * s + 8 * g;
                        Raw8<W> raw[V];
                        if constexpr (KM) {
#pragma unroll
                            for (int q = 0; q < V; ++q) {
                                const W *p = w + (col + (OV || q < nw ? q : nw - 1)) * a.rank;
                                if constexpr (WV) raw[q] = load8(p + (r0 < a.rank ? r0 : 0));
                                else raw[q] = load8<false>(p + r0, a.rank - r0);
                            }
                            if (WV && a.rank < R && r0 >= a.rank)
#pragma unroll
                                for (int q = 0; q < V; ++q) raw[q] = Raw8<W>{};
                        } else {
                            Rows8<W, V> rows;
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                rows.row[e] = load_row<OV, V>(w + (r0 + e < a.rank ? r0 + e : 0) * a.cols + col, nw);
                            if (a.rank < R)
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    if (r0 + e >= a.rank)
#pragma unroll
                                        for (int q = 0; q < V; ++q) rows.row[e].v[q] = (W)0.f;
#pragma unroll
                            for (int q = 0; q < V; ++q) raw[q] = rows.column(q);
                        }
#pragma unroll
                        for (int q = 0; q < V; ++q) acc[q] = mul_acc<bf16_t>(h[s], parts_of<false>(raw[q]), acc[q]);
                    }
                }
                if (base)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int q = 0; q < V; ++q) acc[q][e] = (float)b[e].v[q] + acc[q][e];
                const bool in = c0 + V * m < hi;
                const int64_t at = c0 + turns * 16 * V;
                if (base && at < hi) load_base(at);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (!live[e] || !in) continue;
                    Piece<X, V> o;
#pragma unroll
                    for (int q = 0; q < V; ++q) o.v[q] = (X)acc[q][e];
                    X *p = (X *)a.out + row[e] + col;
                    if constexpr (OV) {
                        *(Piece<X, V> *)p = o;
                    } else {
#pragma unroll
                        for (int q = 0; q < V; ++q)
                            if (q < nw) p[q] = o.v[q];
                    }
                }
            }
        }
    }
}

template <class X, class W, bool KM> hipError_t launch(const Args &a, bool ov, bool wv, hipStream_t st) {
    const dim3 grid = tile_grid(a.slices, a.lanes, a.n);
    auto go = [&](auto ks) -> hipError_t {
        constexpr int KS = decltype(ks)::value;
        if (ov && wv)
            hipLaunchKernelGGL((wide_kernel<X, W, KS, KM, true, true>), grid, dim3(256), 0, st, a);
        else if (ov)
            hipLaunchKernelGGL((wide_kernel<X, W, KS, KM, true, !KM>), grid, dim3(256), 0, st, a);
        else
            hipLaunchKernelGGL((wide_kernel<X, W, KS, KM, false, false>), grid, dim3(256), 0, st, a);
        return hipGetLastError();
    };
    if (a.rank <= 32) return go(std::integral_constant<int, 1>{});
    if (a.rank <= 64) return go(std::integral_constant<int, 2>{});
    return go(std::integral_constant<int, 4>{});
}

}  // namespace

hipError_t launch_lora_wide(int x_type, int w_type, bool by_row, const float *part, int parts, int64_t n, int64_t cols,
                            const void *m, int64_t rank, int64_t n_adapters, const int32_t *ids, const float *scale,
                            const void *base, void *out, hipStream_t s) {
    Args a{};
    a.part = part;
    a.parts = parts;
    a.n = n;
    a.cols = cols;
    a.m = m;
    a.rank = (int32_t)rank;
    a.padded = lora_padded_rank(rank);
    a.n_adapters = (int32_t)n_adapters;
    a.key_bits = key_bits_of(n_adapters);
    a.ids = ids;
    a.scale = scale;
    a.base = base;
    a.out = out;
    const int64_t windows = (n + kWindow - 1) / kWindow;
    // columns of a workgroup: 4 steps of 16 pieces, or 8 or 16 as long as there are 1024 workgroups
    a.slice = 64 * kPiece;
    while (a.slice < 256 * kPiece && windows * ((cols + 2 * a.slice - 1) / (2 * a.slice)) >= 1024) a.slice *= 2;
    a.slices = (int32_t)((cols + a.slice - 1) / a.slice);
    a.lanes = tile_lanes(windows * a.slices, n, n_adapters);
    return with_lora_types(x_type, w_type, [&](auto x, auto w) -> hipError_t {
        typedef decltype(x) X;
        typedef decltype(w) W;
        const bool ov = cols % kPiece == 0 && aligned16(base, out);
        if (!by_row) return launch<X, W, true>(a, ov, rank % 8 == 0 && aligned16(m), s);
        return launch<X, W, false>(a, ov && aligned16(m), true, s);
    });
}

}  // namespace qmm
