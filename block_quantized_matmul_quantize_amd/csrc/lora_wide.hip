// Second half of an adapter: out[i][j] = base[i][j] + sum over r of h[i][r] * m[c][j][r] (forward,
// m = B) or * m[c][r][j] (backward, m = A), where h[i][r] = scale[c] * sum of the first half's slices;
// rows without an adapter get base, or zeros.
//
// It reads base and writes out, 8 bytes an fp32 result, against a few operations for each: HBM bounds
// it.  A workgroup takes a tile of up to 32 rows of one adapter and a slice of the columns; it adds up
// the slices of h once, splits them into bf16 parts in LDS, from where every wave takes them into
// registers for all its columns.  Lane l % 16 owns 16 bytes of neighbouring columns of a row, so that
// base is read and out written 256 bytes a row at a time, straight from the accumulators: column q of
// the lanes' pieces is one matrix instruction's 16 columns.
#include "launch.hpp"
#include "lora_parts.hpp"

namespace qmm {

namespace {

struct Args {
    const float *part;
    const void *m, *base;
    void *out;
    float *h;               // or null: receives the summed h, scaled where scale_h
    const int32_t *ids;
    const float *scale;
    int64_t n, cols, slice, h_stride;
    int32_t n_adapters, key_bits, rank, padded, parts, slices, lanes, scale_h;
};

template <class X, class W, int KS, bool KM, bool OV, bool WV>
__global__ __launch_bounds__(256) void wide_kernel(Args a) {
    constexpr int R = 32 * KS;                        // K of the product
    constexpr int V = 16 / (int)sizeof(X);            // columns of a lane's piece
    constexpr int kStride = R + 8;                    // keeps 16-byte pieces, and rows off the same banks
    __shared__ alignas(16) uint16_t hs[3][kTileRows][kStride];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 15, g = lane >> 4;
    const int64_t slice = blockIdx.x;
    for (int64_t i0 = (int64_t)blockIdx.z * kWindow; i0 < a.n; i0 += (int64_t)gridDim.z * kWindow) {
        const Tiles tiles = find_tiles(a.ids, i0, a.n, a.n_adapters, a.key_bits, true);
        const int64_t lo = slice * a.slice, hi = lo + a.slice < a.cols ? lo + a.slice : a.cols;
        for (int i = blockIdx.y; i < tiles.count; i += gridDim.y) {
            const Tile t = pick_tile(tiles, i);
            const bool some = t.key < a.n_adapters;
            if (some || (a.h && slice == 0)) {
                const float c = some && a.scale ? a.scale[t.key] : 1.f;
                for (int j = threadIdx.x; j < kTileRows * R; j += 256) {
                    const int slot = j / R, r = j % R;
                    const int64_t row = i0 + t.row(slot);
                    float v = 0.f;
                    if (some && slot < t.rows && r < a.rank)
                        for (int p = 0; p < a.parts; ++p) v += a.part[((int64_t)p * a.n + row) * a.padded + r];
                    if (a.h && slice == 0 && slot < t.rows && r < a.rank) a.h[row * a.h_stride + r] = a.scale_h ? v * c : v;
                    v *= c;
                    const float mid = rest_of(v);
                    const uint32_t mb = __float_as_uint(mid);
                    hs[0][slot][r] = (uint16_t)(__float_as_uint(v) >> 16);
                    hs[1][slot][r] = (uint16_t)(mb >> 16);
                    hs[2][slot][r] = (uint16_t)(__float_as_uint(mid - __uint_as_float(mb & 0xffff0000u)) >> 16);
                }
            }
            __syncthreads();
            auto columns = [&](auto mt) {
                constexpr int MT = decltype(mt)::value;
                Frag<3> h[MT][KS];
                int64_t row[MT][4];
                bool live[MT][4];
#pragma unroll
                for (int u = 0; u < MT; ++u) {
#pragma unroll
                    for (int s = 0; s < KS; ++s)
#pragma unroll
                        for (int p = 0; p < 3; ++p) h[u][s].p[p] = *(const u32x4 *)&hs[p][16 * u + m][32 * s + 8 * g];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int slot = 16 * u + 4 * g + e;
                        live[u][e] = slot < t.rows;
                        row[u][e] = (i0 + t.row(slot)) * a.cols;
                    }
                }
                const W *w = (const W *)a.m + (int64_t)t.key * a.rank * a.cols;
                for (int64_t c0 = lo + wave * (16 * V); c0 < hi; c0 += 4 * 16 * V) {
                    const int64_t col = c0 + V * m;
                    const int64_t left = hi - col;          // columns of the piece: V or more, or some, or none
                    // pieces past the end load the last columns' weights; nothing of them is stored
                    const int64_t cw = left > 0 ? col : (OV ? hi - V : hi - 1);
                    Piece<X, V> base[MT][4];
                    if (a.base) {
#pragma unroll
                        for (int u = 0; u < MT; ++u)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (live[u][e] && left > 0)
                                    base[u][e] = load_row<OV, V>((const X *)a.base + row[u][e] + col,
                                                                 left < V ? (int)left : V);
                    }
                    f32x4 acc[MT][V];
#pragma unroll
                    for (int u = 0; u < MT; ++u)
#pragma unroll
                        for (int q = 0; q < V; ++q) acc[u][q] = f32x4{0.f, 0.f, 0.f, 0.f};
                    if (some) {
#pragma unroll
                        for (int s = 0; s < KS; ++s) {
                            const int r0 = 32 * s + 8 * g;
                            if constexpr (KM) {
#pragma unroll
                                for (int q = 0; q < V; ++q) {
                                    const int64_t cq = OV || q < left ? cw + q : hi - 1;
                                    const auto f = parts_of<false>(load8<WV>(w + cq * a.rank + r0, a.rank - r0));
#pragma unroll
                                    for (int u = 0; u < MT; ++u) acc[u][q] = mul_acc<bf16_t>(h[u][s], f, acc[u][q]);
                                }
                            } else {
                                Rows8<W, V> rows;
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    if (r0 + e < a.rank)
                                        rows.row[e] = load_row<OV, V>(w + (r0 + e) * a.cols + cw,
                                                                      left < V && left > 0 ? (int)left : left > 0 ? V : 1);
                                    else
#pragma unroll
                                        for (int q = 0; q < V; ++q) rows.row[e].v[q] = (W)0.f;
                                }
#pragma unroll
                                for (int q = 0; q < V; ++q) {
                                    const auto f = parts_of<false>(rows.column(q));
#pragma unroll
                                    for (int u = 0; u < MT; ++u) acc[u][q] = mul_acc<bf16_t>(h[u][s], f, acc[u][q]);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int u = 0; u < MT; ++u)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (!live[u][e] || left <= 0) continue;
                            Piece<X, V> o;
#pragma unroll
                            for (int q = 0; q < V; ++q)
                                o.v[q] = (X)(a.base ? (float)base[u][e].v[q] + acc[u][q][e] : acc[u][q][e]);
                            X *p = (X *)a.out + row[u][e] + col;
                            if constexpr (OV) {
                                *(Piece<X, V> *)p = o;
                            } else {
#pragma unroll
                                for (int q = 0; q < V; ++q)
                                    if (q < left) p[q] = o.v[q];
                            }
                        }
                }
            };
            if (t.rows > 16) columns(std::integral_constant<int, 2>{});
            else columns(std::integral_constant<int, 1>{});
            __syncthreads();
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
                            const void *base, void *out, float *h, int64_t h_stride, bool scale_h, hipStream_t s) {
    Args a{};
    a.part = part;
    a.parts = parts;
    a.n = n;
    a.cols = out ? cols : 0;   // without an output only h is finished
    a.m = m;
    a.rank = (int32_t)rank;
    a.padded = lora_padded_rank(rank);
    a.n_adapters = (int32_t)n_adapters;
    a.key_bits = key_bits_of(n_adapters);
    a.ids = ids;
    a.scale = scale;
    a.base = base;
    a.out = out;
    a.h = h;
    a.h_stride = h_stride;
    a.scale_h = scale_h;
    const int64_t windows = (n + kWindow - 1) / kWindow, tiles = (n + kTileRows - 1) / kTileRows;
    return with_lora_types(x_type, w_type, [&](auto x, auto w) -> hipError_t {
        typedef decltype(x) X;
        typedef decltype(w) W;
        constexpr int V = 16 / (int)sizeof(X);
        // columns of a workgroup: four waves' 16 pieces, 1 to 4 times, as long as there are 1024 workgroups
        int64_t step = 64 * V;
        while (step < 256 * V && tiles * ((a.cols + 2 * step - 1) / (2 * step)) >= 1024) step *= 2;
        Args b = a;
        b.slice = step;
        b.slices = (int32_t)(a.cols > 0 ? (a.cols + step - 1) / step : 1);
        b.lanes = tile_lanes(windows * b.slices, n, n_adapters);
        const bool ov = cols % V == 0 && aligned16(base, out);
        // a wide piece of W is V elements of a row: 8 or 16 bytes
        if (!by_row) return launch<X, W, true>(b, ov, rank % 8 == 0 && aligned16(m), s);
        return launch<X, W, false>(b, ov && aligned16(m), true, s);
    });
}

}  // namespace qmm
