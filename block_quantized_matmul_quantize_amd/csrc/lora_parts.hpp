// What the adapter kernels (lora_narrow.hip, lora_wide.hip, lora_outer.hip) have in common: the rows of
// a window that share an adapter, and products of fp32 / fp16 / bf16 operands on the bf16 matrix unit.
#pragma once
#include <type_traits>

#include "common.hpp"
#include "rowtypes.hpp"

namespace qmm {

// ------------------------------------------------------------------------------------------------
// Rows that share an adapter
// ------------------------------------------------------------------------------------------------
// A window is 64 consecutive rows, a lane each.  The rows of one adapter in it are a tile; rows without
// an adapter (key n_adapters) form a tile of their own, or none.  Found by one ballot per key bit from
// 256 bytes of ids, so every wave does it for itself: no sort is launched before the forward pass, and
// a step of single tokens (each row its own adapter) spreads over as many workgroups as it has tiles.
//
// So rows of one request should be neighbours.  In random order a window of many adapters has tiles of one or
// two rows, each a product of 16 that reads its adapter again: 2048 rows of 64 adapters at rank 16,
// 4096 -> 14336 columns, take 63 + 420 us forward, 11 + 46 us in runs of 256; backward 216 + 121 us for the two
// products, 39 + 16 us in runs.  (The gradients of A and B take the rows sorted.)
constexpr int kWindow = 64;

struct Tiles {
    int32_t key;    // the lane's row: its adapter
    int tile, slot; // its tile (-1: none) and place in it
    int count;      // tiles of the window
};

// lowest set bit (v != 0)
__device__ __forceinline__ int lowest(uint64_t v) { return __ffsll((unsigned long long)v) - 1; }

__device__ __forceinline__ Tiles find_tiles(const int32_t *__restrict__ ids, int64_t i0, int64_t n, int32_t n_adapters,
                                            int key_bits, bool with_none) {
    const int lane = threadIdx.x & 63;
    Tiles t;
    const bool row = i0 + lane < n;
    const int32_t id = row ? ids[i0 + lane] : -1;
    t.key = (uint32_t)id < (uint32_t)n_adapters ? id : n_adapters;
    const bool in = row && (with_none || t.key < n_adapters);
    uint64_t same = __ballot(in);
    for (int b = 0; b < key_bits; ++b) {
        const uint64_t set = __ballot((t.key >> b) & 1);
        same &= (t.key >> b) & 1 ? set : ~set;
    }
    t.slot = __popcll(same & ((1ull << lane) - 1));
    const uint64_t first = __ballot(in && t.slot == 0);
    t.tile = in ? __popcll(first & ((1ull << lowest(same)) - 1)) : -1;
    t.count = __popcll(first);
    return t;
}

struct Tile {
    int32_t key;    // adapter
    int rows;       // 1 .. 64
    int slot0;      // first slot
    int at;         // lane l: row of slot l within the window
    __device__ __forceinline__ int row(int slot) const { return __shfl(at, slot0 + (slot < rows ? slot : 0)); }
};
__device__ __forceinline__ Tile pick_tile(const Tiles &t, int i) {
    const uint64_t m = __ballot(t.tile == i);
    Tile r;
    r.rows = __popcll(m);
    r.slot0 = 0;
    r.key = __builtin_amdgcn_readlane(t.key, lowest(m));
    // each row's lane number goes to the lane of its slot; the other lanes push to lane 63, which is a
    // slot only where there are no other lanes
    r.at = __builtin_amdgcn_ds_permute((t.tile == i ? t.slot : 63) * 4, (int)(threadIdx.x & 63));
    return r;
}

// One of four parts of a tile, 16 slots each (without rows where the tile has fewer).
__device__ __forceinline__ Tile part_of(const Tile &t, int part) {
    Tile r = t;
    r.slot0 = 16 * part;
    r.rows = t.rows - r.slot0 < 16 ? t.rows - r.slot0 : 16;
    return r;
}
// Calls f(number of 16-row groups, 1, 2 or 4): a wave takes all of them, so that its operand of the
// adapter's matrix, once loaded, serves every row of the tile.
template <class F> __device__ __forceinline__ void with_groups(const Tile &t, F f) {
    if (t.rows <= 16) f(std::integral_constant<int, 1>{});
    else if (t.rows <= 32) f(std::integral_constant<int, 2>{});
    else f(std::integral_constant<int, 4>{});
}

// Host: bits of a key, and tiles that a window can have.
inline int key_bits_of(int64_t n_adapters) {
    int b = 1;
    while (n_adapters >> b) ++b;
    return b;
}
inline int64_t tiles_of_window(int64_t n, int64_t n_adapters) {
    const int64_t most = n_adapters + 1 < kWindow ? n_adapters + 1 : kWindow;
    return n < most ? n : most;
}
// Workgroups that share a window's tiles: one for each tile there can be as long as the launch stays
// at about 1024 workgroups, else 2 (runs of rows of one request give a window one or two tiles); those
// that find no tile end after reading the ids, but hold a place on a compute unit until then.
inline int tile_lanes(int64_t others, int64_t n, int64_t n_adapters) {
    const int64_t most = tiles_of_window(n, n_adapters), fit = 1024 / others;
    const int64_t least = most < 2 ? most : 2;
    return (int)(fit > most ? most : fit < least ? least : fit);
}
// Workgroups that a tile's rows are spread over: a small call, which latency bounds, has each take 16 rows,
// if adapters have that many (300 rows of 2 adapters into 2048 columns: 8.7 against 13.7 us; 32 rows of 64
// adapters: 14.2 against 7.0 us).
inline int tile_parts(int64_t others, int lanes, int64_t n, int64_t n_adapters) {
    return others * lanes * 4 <= 1024 && n_adapters * 16 <= n ? 4 : 1;
}
// Slices of the other dimension x windows (the kernels step through what exceeds the grid) x workgroups
// of a window, which come last: workgroups go round the compute units in order, so that those without a
// tile, were they every other one, would leave every other unit idle (measured: 2.9 times slower).
inline dim3 tile_grid(int64_t slices, int lanes, int64_t n) {
    const int64_t windows = (n + kWindow - 1) / kWindow;
    return dim3((unsigned)slices, (unsigned)(windows < 65535 ? windows : 65535), (unsigned)lanes);
}
// The slice of a workgroup: turned by one from window to window.  Workgroups go round the eight dies, so
// with 8 slices each die would otherwise see one range of columns only, and rows a multiple of 4 KB
// apart would share few of its L2 channels.
__device__ __forceinline__ int64_t slice_of_block(int64_t slices) { return (blockIdx.x + blockIdx.y) % slices; }
// Host: calls f(values of the element types of x and of the adapters).
template <class F> hipError_t with_lora_types(int x_type, int w_type, F f) {
    return with_type(x_type, [&](auto x) -> hipError_t {
        return with_type(w_type, [&](auto w) -> hipError_t {
            if constexpr (sizeof(x) == 4 || std::is_same<decltype(x), decltype(w)>::value) return f(x, w);
            else return hipErrorInvalidValue;
        });
    });
}

// ------------------------------------------------------------------------------------------------
// Products
// ------------------------------------------------------------------------------------------------
// fp32 operands keep all their 24 bits: a value is the sum of three bf16 numbers, each the next eight
// significant bits (truncated, so every step is exact), and a product of two values the sum of the
// products of their parts, accumulated in fp32.  fp16 is the sum of two such parts (8 + 3 bits), bf16
// one.  Only the product of two third parts (below 2^-30 of the whole) is left out.  Where both
// operands are the same 16-bit type, one instruction of that type does it.
template <class T> constexpr int kParts = std::is_same<T, float>::value ? 3 : std::is_same<T, f16_t>::value ? 2 : 1;
template <class X, class W> constexpr bool kNative = sizeof(X) == 2 && std::is_same<X, W>::value;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// 16x16x32: A lane l holds row l % 16, B lane l column l % 16, each the 8 K values of lane group l / 16;
// C lane l holds C[4 * (l / 16) + e][l % 16], e = 0..3.
template <class T> __device__ __forceinline__ f32x4 mfma32(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (std::is_same<T, f16_t>::value)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
}

// {high 16 bits of a, of b} and {low 16 bits of a, of b}, a's in the low half
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_perm(b, a, 0x07060302u);
}
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_perm(b, a, 0x05040100u);
}

template <int P> struct Frag { u32x4 p[P]; };

// What is left of v after its top eight significant bits; 0 for an infinity, which its first part holds whole.
__device__ __forceinline__ float rest_of(float v) {
    const float r = v - __uint_as_float(__float_as_uint(v) & 0xffff0000u);
    return __builtin_isinf(v) ? 0.f : r;
}
template <int P> __device__ __forceinline__ Frag<P> split8(const float (&v)[8]) {
    Frag<P> f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = v[2 * i], b = v[2 * i + 1];
        f.p[0][i] = high_halves(__float_as_uint(a), __float_as_uint(b));
        if constexpr (P > 1) {
            const float ra = rest_of(a), rb = rest_of(b);
            f.p[1][i] = high_halves(__float_as_uint(ra), __float_as_uint(rb));
            if constexpr (P > 2) {
                const float la = ra - __uint_as_float(__float_as_uint(ra) & 0xffff0000u);
                const float lb = rb - __uint_as_float(__float_as_uint(rb) & 0xffff0000u);
                f.p[2][i] = high_halves(__float_as_uint(la), __float_as_uint(lb));
            }
        }
    }
    return f;
}

// Eight elements as loaded: fp32 values, or 16-bit ones packed in order.
template <class T> struct Raw8 { u32x4 v; };
template <> struct Raw8<float> { float v[8]; };

template <class T> __device__ __forceinline__ uint32_t bits16(T v) { return (uint32_t)__builtin_bit_cast(uint16_t, v); }

// As parts, or (16-bit types of a native product) as they are.
template <bool NATIVE, class T> __device__ __forceinline__ auto parts_of(const Raw8<T> &r) {
    if constexpr (std::is_same<T, float>::value) {
        return split8<3>(r.v);
    } else if constexpr (std::is_same<T, f16_t>::value && !NATIVE) {
        float v[8];
        const f16x8 h = __builtin_bit_cast(f16x8, r.v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
        return split8<2>(v);
    } else {
        return Frag<1>{{r.v}};
    }
}

template <class T, int PA, int PB> __device__ __forceinline__ f32x4 mul_acc(const Frag<PA> &a, const Frag<PB> &b, f32x4 c) {
#pragma unroll
    for (int s = (PA - 1) + (PB - 1) < 3 ? PA + PB - 2 : 3; s >= 0; --s)   // the smallest first
#pragma unroll
        for (int i = 0; i < PA; ++i)
            if (s - i >= 0 && s - i < PB) c = mfma32<T>(a.p[i], b.p[s - i], c);
    return c;
}

// ------------------------------------------------------------------------------------------------
// Loads
// ------------------------------------------------------------------------------------------------
// N elements as aligned pieces of up to 16 bytes.
template <class T, int N> struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Piece { T v[N]; };

// Eight elements of a row that begins at p, `left` of which belong to it (the others become 0).
// VEC: aligned, and all or none.
template <bool VEC, class T> __device__ __forceinline__ Raw8<T> load8(const T *p, int64_t left) {
    Raw8<T> r;
    if constexpr (VEC) {
        if (left > 0) {
            const Piece<T, 8> u = *(const Piece<T, 8> *)p;
            r = __builtin_bit_cast(Raw8<T>, u);
        } else {
            r = Raw8<T>{};
        }
    } else {
        T u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = i < left ? p[i] : (T)0.f;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) r.v[i] = u[i];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) r.v[i] = bits16(u[2 * i]) | (bits16(u[2 * i + 1]) << 16);
        }
    }
    return r;
}

// N elements at any multiple of their size: still 16 bytes a load, which gfx950 takes at any address.
template <int N, class T> __device__ __forceinline__ Piece<T, N> load_any(const T *p) {
    Piece<T, N> r;
    __builtin_memcpy(&r, p, sizeof(r));
    return r;
}
template <class T> __device__ __forceinline__ Raw8<T> load8_any(const T *p) {
    return __builtin_bit_cast(Raw8<T>, load_any<8>(p));
}
// Eight aligned elements, all the row's own.
template <class T> __device__ __forceinline__ Raw8<T> load8(const T *p) {
    return __builtin_bit_cast(Raw8<T>, *(const Piece<T, 8> *)p);
}

// A block of 8 rows (K values) x N columns, N elements of a row together; column q's 8 K values are an
// operand.  So [K][columns] matrices need no transpose in memory: a lane reads its 8 rows itself.
template <class T, int N> struct Rows8 {
    Piece<T, N> row[8];
    __device__ __forceinline__ Raw8<T> column(int q) const {
        Raw8<T> r;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r.v[e] = row[e].v[q];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (N == 1) {
                    r.v[i] = bits16(row[2 * i].v[0]) | (bits16(row[2 * i + 1].v[0]) << 16);
                } else {
                    typedef uint32_t Words __attribute__((ext_vector_type(N / 2)));
                    const Words a = __builtin_bit_cast(Words, row[2 * i]), b = __builtin_bit_cast(Words, row[2 * i + 1]);
                    r.v[i] = q & 1 ? high_halves(a[q / 2], b[q / 2]) : low_halves(a[q / 2], b[q / 2]);
                }
            }
        }
        return r;
    }
};

// N elements at p, of which the first `left` (at least 1) are the row's own: the others repeat the last.
template <bool VEC, int N, class T> __device__ __forceinline__ Piece<T, N> load_row(const T *p, int left) {
    if constexpr (VEC || N == 1) {
        return *(const Piece<T, N> *)p;
    } else {
        if (left >= N) return load_any<N>(p);
        Piece<T, N> r;
#pragma unroll
        for (int q = 0; q < N; ++q) r.v[q] = p[q < left ? q : left - 1];
        return r;
    }
}

}  // namespace qmm
