// Second half of an adapter: out[i][j] = base[i][j] + sum over r of h[i][r] * m[c][j][r] (forward,
// m = B) or * m[c][r][j] (backward, m = A), where h[i][r] = scale[c] * sum of the first half's slices;
// rows without an adapter get base, or zeros.
//
// It reads base and writes out, 8 bytes an fp32 result, against a few operations for each: HBM bounds
// it.  A workgroup takes the rows of one adapter in a window of 64 and a slice of the columns; it adds
// up the slices of its rows' h and leaves their bf16 parts in LDS.  A wave takes 64 columns at a time for
// all the rows, 16 or 32 of them together: it loads the adapter's part for them once.
// Lane l % 16 owns four neighbouring columns of a row, so that base is read and out written 256 (fp32)
// or 128 bytes a row at a time, straight from the accumulators: column q of the lanes' pieces is one
// matrix instruction's 16 columns.
//
// 2048 rows into 14336 fp32 columns at rank 16: 46 us (5.1 TB/s, a copy's rate); 8192 rows into 4096
// bf16 columns at rank 64: 31 us, backward 33 (runs of 256 rows) to 45 us (runs of any length); 32 rows
// of 64 adapters into 4096 columns: 5.2 us.
//
// Beyond rank 32 registers bound it too: the parts of all ranks and of a lane's four columns are held at
// once, and with two waves a SIMD (256 registers) 53 of the 75 instances spill some.  Vector registers
// spilled: up to 13 at ranks up to 32; at ranks 33-64 forward up to 34 and backward 44-64 (bf16 matrices
// 4-16); at ranks 65-128 forward 67-85 and backward 124-144 with fp16 matrices, 0-25 and 57-77 with bf16 ones,
// none with fp32 ones, which have one wave a SIMD.  4096 rows into 4096 columns, backward, by the types of the
// rows and matrices: rank 64 bf16 20, fp16 34, fp32 / bf16 31, fp32 / fp16 50, fp32 46 us; rank 128 40, 65, 54,
// 79, 67 us.  Forward: rank 64 21, 25, 29, 34, 35 us; rank 128 32, 55, 39, 66, 72 us.
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
    int32_t n_adapters, key_bits, rank, padded, parts, slices, lanes, row_parts;
};

template <int R> struct Stage {
    uint16_t v[3][kWindow][R + 8];   // keeps 16-byte pieces, and rows off the same banks
    __device__ __forceinline__ void put(int slot, int r, const float (&x)[4]) {
        uint32_t p[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float mid = rest_of(x[i]);
            p[0][i] = __float_as_uint(x[i]);
            p[1][i] = __float_as_uint(mid);
            p[2][i] = __float_as_uint(mid - __uint_as_float(p[1][i] & 0xffff0000u));
        }
#pragma unroll
        for (int j = 0; j < 3; ++j)
            *(u32x2 *)&v[j][slot][r] = u32x2{high_halves(p[j][0], p[j][1]), high_halves(p[j][2], p[j][3])};
    }
    __device__ __forceinline__ Frag<3> get(int slot, int r) const {
        Frag<3> f;
#pragma unroll
        for (int p = 0; p < 3; ++p) f.p[p] = *(const u32x4 *)&v[p][slot][r];
        return f;
    }
};

template <class X, class W, int KS, bool KM, bool OV, bool WV>
__global__ __launch_bounds__(256, KS == 4 && sizeof(W) == 4 ? 1 : 2) void wide_kernel(Args a) {
    constexpr int R = 32 * KS;                        // K of the product
    constexpr int V = kPiece;
    __shared__ alignas(16) Stage<R> stage;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 15, g = lane >> 4;
    const int64_t slice = slice_of_block(a.slices);
    const int64_t lo = slice * a.slice, hi = lo + a.slice < a.cols ? lo + a.slice : a.cols;
    for (int64_t i0 = (int64_t)blockIdx.y * kWindow; i0 < a.n; i0 += (int64_t)gridDim.y * kWindow) {
        const Tiles tiles = find_tiles(a.ids, i0, a.n, a.n_adapters, a.key_bits, true);
        for (int i = blockIdx.z % a.lanes; i < tiles.count; i += a.lanes) {
            Tile t = pick_tile(tiles, i);
            if (a.row_parts > 1) t = part_of(t, blockIdx.z / a.lanes);
            if (t.rows <= 0) continue;
            const bool some = t.key < a.n_adapters;
            with_groups(t, [&](auto groups) {
                // groups of 16 rows, and at a time (fp32 matrices and 128 ranks need the registers: 31.5 us with 1,
                // 44.5 with 2, for 4096 fp32 rows at rank 16; 25.4 and 38.6 for as many bf16 rows at rank 128)
                constexpr int G = decltype(groups)::value, MT = G < 2 || sizeof(W) == 4 || KS == 4 ? 1 : 2;
                const X *base = (const X *)a.base;
                const W *w = (const W *)a.m + (int64_t)t.key * a.rank * a.cols;
                int32_t row[G][4];
#pragma unroll
                for (int u = 0; u < G; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e)   // slots past the last: row of slot 0, not stored
                        row[u][e] = (int32_t)i0 + t.row(16 * u + 4 * g + e);
                // a lane's columns: all V, or some, or none at the end (nothing of those is stored)
                auto col_of = [&](int64_t at) { return at + V * m < hi ? at + V * m : OV ? hi - V : hi - 1; };
                auto width_of = [&](int64_t col) { return OV || hi - col >= V ? V : (int)(hi - col); };
                Piece<X, V> b[MT][4];
                auto load_base = [&](int64_t at, int u0) {
                    const int64_t col = col_of(at);
                    if (OV || at + 16 * V <= hi) {
#pragma unroll
                        for (int u = 0; u < MT; ++u)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const X *p = base + row[u0 + u][e] * a.cols + col;
                                b[u][e] = OV ? load_row<true, V>(p, V) : load_any<V>(p);
                            }
                    } else {   // the last columns
#pragma unroll
                        for (int u = 0; u < MT; ++u)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                b[u][e] = load_row<false, V>(base + row[u0 + u][e] * a.cols + col, width_of(col));
                    }
                };
                int64_t c0 = lo + wave * (16 * V);
                if (base && c0 < hi) load_base(c0, 0);
                // the adapter's part for 32 ranks from 32 * s and the columns of a step
                auto load_w = [&](int64_t at, int s, Raw8<W> (&raw)[V]) {
                    const int64_t col = col_of(at);
                    const int nw = width_of(col), r0 = 32 * s + 8 * g;
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
                };
                // up to 32 ranks of the first step before h is there, so that one latency covers both
                Raw8<W> raw[V];
                if (KS == 1 && some && c0 < hi) load_w(c0, 0, raw);
                if (some) {
                    const float c = a.scale ? a.scale[t.key] : 1.f;
                    const int64_t next = a.n * a.padded;
#pragma unroll
                    for (int u = 0; u < G * KS / 2 || u == 0; ++u) {
                        const int j = 256 * u + threadIdx.x, slot = j / (R / 4), r = j % (R / 4) * 4;
                        const float *p = a.part + (i0 + t.row(slot)) * a.padded + (r < a.padded ? r : 0);
                        f32x4 sum = *(const f32x4 *)p;
                        for (int s0 = 1; s0 < a.parts; s0 += 8) {   // a slice past the last is read as the first, and left out
                            f32x4 q[8];
#pragma unroll
                            for (int s = 0; s < 8; ++s) q[s] = *(const f32x4 *)(p + (s0 + s < a.parts ? s0 + s : 0) * next);
#pragma unroll
                            for (int s = 0; s < 8; ++s) sum += s0 + s < a.parts ? q[s] : f32x4{0.f, 0.f, 0.f, 0.f};
                        }
                        float v[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) v[q] = r + q < a.rank ? sum[q] * c : 0.f;   // no other rank is of use
                        stage.put(slot, r, v);
                    }
                    __syncthreads();
                }
                for (; c0 < hi; c0 += 64 * V) {
                    const int64_t col = col_of(c0), at = c0 + 64 * V;
                    const int nw = width_of(col);
                    const bool in = c0 + V * m < hi;
                    decltype(parts_of<false>(raw[0])) f[KS][V];
                    if (some) {
#pragma unroll
                        for (int s = 0; s < KS; ++s) {
                            if constexpr (KS > 1) load_w(c0, s, raw);
#pragma unroll
                            for (int q = 0; q < V; ++q) f[s][q] = parts_of<false>(raw[q]);
                        }
                        if (KS == 1 && at < hi) load_w(at, 0, raw);
                    }
#pragma unroll
                    for (int u0 = 0; u0 < G; u0 += MT) {
                        f32x4 acc[MT][V];
#pragma unroll
                        for (int u = 0; u < MT; ++u)
#pragma unroll
                            for (int q = 0; q < V; ++q) acc[u][q] = f32x4{0.f, 0.f, 0.f, 0.f};
                        if (some)
#pragma unroll
                            for (int s = 0; s < KS; ++s)
#pragma unroll
                                for (int u = 0; u < MT; ++u) {
                                    const Frag<3> h = stage.get(16 * (u0 + u) + m, 32 * s + 8 * g);
#pragma unroll
                                    for (int q = 0; q < V; ++q) acc[u][q] = mul_acc<bf16_t>(h, f[s][q], acc[u][q]);
                                }
                        if (base)
#pragma unroll
                            for (int u = 0; u < MT; ++u)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
#pragma unroll
                                    for (int q = 0; q < V; ++q) acc[u][q][e] = (float)b[u][e].v[q] + acc[u][q][e];
                        if (base && u0 + MT < G) load_base(c0, u0 + MT);
                        else if (base && at < hi) load_base(at, 0);
#pragma unroll
                        for (int u = 0; u < MT; ++u)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if (16 * (u0 + u) + 4 * g + e >= t.rows || !in) continue;
                                Piece<X, V> o;
#pragma unroll
                                for (int q = 0; q < V; ++q) o.v[q] = (X)acc[u][q][e];
                                X *p = (X *)a.out + row[u0 + u][e] * a.cols + col;
                                if constexpr (OV) {
                                    *(Piece<X, V> *)p = o;
                                } else if (nw == V) {
                                    __builtin_memcpy(p, &o, sizeof(o));
                                } else {
#pragma unroll
                                    for (int q = 0; q < V; ++q)
                                        if (q < nw) p[q] = o.v[q];
                                }
                            }
                    }
                }
                if (some) __syncthreads();
            });
        }
    }
}

template <class X, class W, bool KM> hipError_t launch(const Args &a, bool ov, bool wv, hipStream_t st) {
    const dim3 grid = tile_grid(a.slices, a.lanes * a.row_parts, a.n);
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
    // columns of a workgroup: one step of its four waves, or 2 or 4 as long as there are 512 workgroups
    a.slice = 64 * kPiece;
    while (a.slice < 256 * kPiece && windows * ((cols + 2 * a.slice - 1) / (2 * a.slice)) >= 512) a.slice *= 2;
    a.slices = (int32_t)((cols + a.slice - 1) / a.slice);
    a.lanes = tile_lanes(windows * a.slices, n, n_adapters);
    a.row_parts = tile_parts(windows * a.slices, a.lanes, n, n_adapters);
    return with_lora_types(x_type, w_type, [&](auto x, auto w) -> hipError_t {
        typedef decltype(x) X;
        typedef decltype(w) W;
        const bool ov = cols % kPiece == 0 && aligned16(base, out);
        if (!by_row) return launch<X, W, true>(a, ov, rank % 8 == 0 && aligned16(m), s);
        return launch<X, W, false>(a, ov && aligned16(m), true, s);
    });
}

}  // namespace qmm
