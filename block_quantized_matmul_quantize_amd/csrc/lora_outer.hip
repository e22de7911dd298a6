// Gradients of the adapters' matrices: da[c][r][j] = sum of dh[i][r] * x[i][j] and db[c][o][r] =
// scale[c] * sum of dy[i][o] * h[i][r] over the rows i of adapter c, both in one launch.
//
// A workgroup takes 64 or 128 columns of x (or dy) for all ranks of one adapter; its four waves take
// turns at 32 places of the rows sorted by adapter.  x and dy are read once; K of the products is the
// row, so every lane reads 8 rows of 4 or 8 neighbouring columns and is itself the transpose that the
// operand needs, without LDS.  h and dh come as bf16 parts [place / 32][3][rank][place % 32], operands
// as they are and one stretch of memory a step, from L2, once for each block of columns.  The waves add
// their sums up in LDS in a fixed order.  An adapter with many rows and few columns is split over
// several workgroups, whose sums a second launch adds up.
//
// 8192 rows of 4 adapters, x and dy of 4096 bf16 values (134 MB): 24 us at rank 16 (5.6 TB/s), 46 us at
// rank 64, where the parts of h and dh, read once for each block of columns, are 200 MB from L2 beside
// it (with 64 columns a block instead of 128: 70 us), 70 us for 4096 rows at rank 128.
#include "launch.hpp"
#include "lora_parts.hpp"

namespace qmm {

namespace {

struct Job {
    const void *v;
    const uint16_t *h;      // bf16 parts [place / 32][3][padded rank][place % 32]
    float *out;
    const float *scale;     // or null
    int64_t cols, slices;
    int32_t by_row;         // out [rank][cols], else [cols][rank]
};
struct Args {
    Job job[2];
    const int32_t *order, *bounds;
    float *part;            // [splits][n_adapters * rank * (all columns)], where splits > 1
    int64_t items, out_total;
    int32_t rank, splits, n_adapters, spread;
};

template <class X, int RT> constexpr int kCols = sizeof(X) == 4 || RT == 8 ? 4 : 8;   // a lane's columns

template <class X, int RT, bool VV>
__global__ __launch_bounds__(256) void outer_kernel(Args a) {
    constexpr int V = kCols<X, RT>, C = 16 * V, R = 16 * RT;
    __shared__ float sum[R][C + 4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 15, g = lane >> 4;
    for (int64_t b = blockIdx.x; b < a.items; b += gridDim.x) {
        // neighbouring blocks of columns on one die: they share h in its L2, and spread over its channels
        const int64_t item = xcd_remap(b, a.items);
        // (adapter, job, block of columns, split of the rows)
        const int64_t per = (a.job[0].slices + a.job[1].slices) * a.splits;
        const int64_t c = item / per;
        int64_t u = item - c * per;
        const int split = (int)(u % a.splits);
        u /= a.splits;
        const int which = u < a.job[0].slices ? 0 : 1;
        const Job &job = a.job[which];
        // spread: a block of columns for each wave
        const int64_t block = which ? u - a.job[0].slices : u;
        const int64_t col0 = (a.spread ? 4 * block + wave : block) * C;
        const int64_t lo = a.bounds[c], hi = a.bounds[c + 1];
        const X *v = (const X *)job.v;
        // columns and ranks past the last repeat valid ones: their sums are not used
        const int64_t left = job.cols - col0 - V * m;
        const int64_t col = left >= V || (!VV && left > 0) ? col0 + V * m : VV ? job.cols - V : job.cols - 1;
        const int nc = left >= V ? V : left > 0 ? (int)left : VV ? V : 1;
        const bool whole = __ballot(nc != V) == 0;
        f32x4 acc[RT][V];
#pragma unroll
        for (int p = 0; p < RT; ++p)
#pragma unroll
            for (int q = 0; q < V; ++q) acc[p][q] = f32x4{0.f, 0.f, 0.f, 0.f};
        // steps at multiples of 32 places; an adapter without rows has none (its lo may be past the last row)
        const int64_t step = a.spread ? 32 : (int64_t)a.splits * 4 * 32;
        const int64_t start = lo < hi && col0 < job.cols ? lo / 32 * 32 + (a.spread ? 0 : (split * 4 + wave) * 32) : hi;
        auto rows_of = [&](int64_t p0) {   // lane l: row of place p0 + l % 32 (of a place of the adapter, at the ends)
            const int64_t at = p0 + (lane & 31);
            return a.order[at < lo ? lo : at < hi ? at : hi - 1];
        };
        int32_t rows = start < hi ? rows_of(start) : 0;
        for (int64_t p0 = start; p0 < hi; p0 += step) {
            Rows8<X, V> xs;
            Frag<3> hf[RT];
            const X *at_row[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) at_row[e] = v + (int64_t)__shfl(rows, 8 * g + e) * job.cols + col;
            if (VV || whole) {
#pragma unroll
                for (int e = 0; e < 8; ++e) xs.row[e] = VV ? load_row<true, V>(at_row[e], V) : load_any<V>(at_row[e]);
            } else {   // the last block of columns
#pragma unroll
                for (int e = 0; e < 8; ++e) xs.row[e] = load_row<false, V>(at_row[e], nc);
            }
            rows = rows_of(p0 + step);   // the next step's, in flight during this one
#pragma unroll
            for (int p = 0; p < RT; ++p)
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    hf[p].p[j] = *(const u32x4 *)(job.h + 3 * R * p0 + (j * R + 16 * p + m) * 32 + 8 * g);
            if (p0 < lo || p0 + 32 > hi) {   // places of other adapters
                u32x4 keep;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int64_t place = p0 + 8 * g + e;
                    const bool mine = place >= lo && place < hi;
                    const uint32_t half = mine ? 0xffffu : 0;
                    keep[e / 2] = e & 1 ? keep[e / 2] | half << 16 : half;
                    if (!mine)
#pragma unroll
                        for (int q = 0; q < V; ++q) xs.row[e].v[q] = (X)0.f;
                }
#pragma unroll
                for (int p = 0; p < RT; ++p)
#pragma unroll
                    for (int j = 0; j < 3; ++j) hf[p].p[j] &= keep;
            }
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const auto xf = parts_of<false>(xs.column(q));
#pragma unroll
                for (int p = 0; p < RT; ++p) acc[p][q] = mul_acc<bf16_t>(hf[p], xf, acc[p][q]);
            }
        }
        // acc[p][q] element e: rank 16 * p + 4g + e, column col0 + V * m + q
        if (a.spread) {
            const float scale = job.scale ? job.scale[c] : 1.f;
            float *out = job.out + c * a.rank * job.cols;
#pragma unroll
            for (int p = 0; p < RT; ++p) {
                const int r = 16 * p + 4 * g;
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const int64_t k = col0 + V * m + q;
                    if (k >= job.cols) continue;
                    f32x4 o = acc[p][q] * scale;
                    if (!job.by_row && r + 4 <= a.rank) {
                        __builtin_memcpy(out + k * a.rank + r, &o, sizeof(o));
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (r + e < a.rank) out[job.by_row ? (r + e) * job.cols + k : k * a.rank + r + e] = o[e];
                    }
                }
            }
            continue;
        }
        for (int w = 0; w < 4; ++w) {
            if (wave == w) {
#pragma unroll
                for (int p = 0; p < RT; ++p)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float *s = &sum[16 * p + 4 * g + e][V * m];
#pragma unroll
                        for (int q = 0; q < V; ++q) s[q] = w ? s[q] + acc[p][q][e] : acc[p][q][e];
                    }
            }
            __syncthreads();
        }
        const float scale = job.scale ? job.scale[c] : 1.f;
        const int64_t cols = job.cols - col0 < C ? job.cols - col0 : C;
        const int64_t first = which ? (int64_t)a.n_adapters * a.rank * a.job[0].cols : 0;
        float *out = a.splits > 1 ? a.part + split * a.out_total + first : job.out;
        if (job.by_row) {
            for (int j = threadIdx.x; j < a.rank * C; j += 256) {
                const int r = j / C, k = j % C;
                if (k < cols) out[(c * a.rank + r) * job.cols + col0 + k] = sum[r][k] * scale;
            }
        } else {
            out += (c * job.cols + col0) * a.rank;
            for (int k = threadIdx.x / R; k < cols; k += 256 / R) {
                const int r = threadIdx.x % R;
                if (r < a.rank) out[k * a.rank + r] = sum[r][k] * scale;
            }
        }
        __syncthreads();
    }
}

__global__ __launch_bounds__(256) void join_kernel(const float *__restrict__ part, int splits, int64_t n0, int64_t total,
                                                   float *__restrict__ out0, float *__restrict__ out1) {
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
        float s = 0.f;
#pragma unroll 4
        for (int p = 0; p < splits; ++p) s += part[p * total + t];
        (t < n0 ? out0[t] : out1[t - n0]) = s;
    }
}


// Workgroups an adapter's rows are split over: 256 in all, while each wave keeps two steps of the
// average adapter's rows.  This rule and the next go by the average: the host does not know the segments.
// Where one adapter of a large pool has all the rows, its few workgroups walk them alone (2048 rows at rank
// 16, 4096 bf16 columns: 62 us in a pool of 64, 11 + 3 us in a pool of one).
int splits_of(int64_t n, int64_t n_adapters, int64_t blocks) {
    int64_t s = 256 / (blocks * n_adapters), most = n / n_adapters / 256;
    if (s > most) s = most;
    return s < 1 ? 1 : s > 16 ? 16 : (int)s;
}
// With few rows an adapter the four waves of a workgroup take a block of columns each instead of steps of
// rows that are not there (157 rows of 57 adapters at rank 64, 4625 columns: 36-41 us, 51 us with steps; from
// 64 rows an adapter on, every wave has a step or two of its own).
bool spread_of(int64_t n, int64_t n_adapters) { return n / n_adapters < 64; }
int rank_tiles(int64_t rank) { return lora_padded_rank(rank) / 16; }
int64_t block_cols(int x_type, int rt) { return x_type == kF32 || rt == 8 ? 64 : 128; }
int64_t blocks_of(int x_type, int64_t rank, int64_t cols) {
    const int64_t c = block_cols(x_type, rank_tiles(rank));
    return (cols + c - 1) / c;
}

}  // namespace

size_t lora_outer_bytes(int64_t n, int64_t k, int64_t rows, int64_t rank, int64_t n_adapters) {
    // for any element type, and either gradient alone: no workgroup count is below the widest blocks'
    size_t most = 0;
    for (int which = 1; which < 4; ++which) {
        const int64_t c = (which & 1 ? k : 0) + (which & 2 ? rows : 0);
        const int64_t blocks = (which & 1 ? blocks_of(kBF16, rank, k) : 0) + (which & 2 ? blocks_of(kBF16, rank, rows) : 0);
        const int s = spread_of(n, n_adapters) ? 1 : splits_of(n, n_adapters, blocks);
        const size_t bytes = s > 1 ? (size_t)s * n_adapters * rank * c * 4 : 0;
        if (bytes > most) most = bytes;
    }
    return most;
}

hipError_t launch_lora_outer(int x_type, const void *x, const uint16_t *parts_dh, int64_t k, float *da, const void *dy,
                             const uint16_t *parts_h, int64_t rows, const float *scale, float *db, int64_t n,
                             int64_t rank, int64_t n_adapters, const int32_t *order, const int32_t *bounds, float *part,
                             hipStream_t s) {
    Args a{};
    a.job[0] = Job{x, parts_dh, da, nullptr, da ? k : 0, 0, 1};
    a.job[1] = Job{dy, parts_h, db, scale, db ? rows : 0, 0, 0};
    a.order = order;
    a.bounds = bounds;
    a.part = part;
    a.rank = (int32_t)rank;
    a.n_adapters = (int32_t)n_adapters;
    const int rt = rank_tiles(rank);
    int64_t blocks = 0;
    a.spread = spread_of(n, n_adapters);
    for (Job &j : a.job) {
        j.slices = blocks_of(x_type, rank, j.cols);
        if (a.spread) j.slices = (j.slices + 3) / 4;
        blocks += j.slices;
    }
    a.splits = a.spread ? 1 : splits_of(n, n_adapters, blocks);
    a.items = n_adapters * blocks * a.splits;
    a.out_total = n_adapters * rank * (a.job[0].cols + a.job[1].cols);
    hipError_t e = with_type(x_type, [&](auto t) -> hipError_t {
        typedef decltype(t) X;
        const dim3 grid((unsigned)(a.items < 1 << 22 ? a.items : 1 << 22));
        auto go = [&](auto r) -> hipError_t {
            constexpr int RT = decltype(r)::value;
            constexpr int V = kCols<X, RT>;
            const bool vv = a.job[0].cols % V == 0 && a.job[1].cols % V == 0 && aligned16(da ? x : nullptr, db ? dy : nullptr);
            if (vv) hipLaunchKernelGGL((outer_kernel<X, RT, true>), grid, dim3(256), 0, s, a);
            else hipLaunchKernelGGL((outer_kernel<X, RT, false>), grid, dim3(256), 0, s, a);
            return hipGetLastError();
        };
        switch (rt) {
            case 1: return go(std::integral_constant<int, 1>{});
            case 2: return go(std::integral_constant<int, 2>{});
            case 4: return go(std::integral_constant<int, 4>{});
            default: return go(std::integral_constant<int, 8>{});
        }
    });
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t n0 = n_adapters * rank * a.job[0].cols, b = (a.out_total + 255) / 256;
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)(b < 65536 ? b : 65536)), dim3(256), 0, s, part, a.splits, n0,
                       a.out_total, da, db);
    return hipGetLastError();
}

}  // namespace qmm
