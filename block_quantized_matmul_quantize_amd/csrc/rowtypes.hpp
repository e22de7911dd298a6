// Element types of the row operators (embedding, expert gather / combine, low-rank adapters): fp32,
// fp16 and bf16 rows, read and written 16 bytes or one element at a time, computed on in fp32 and
// rounded to nearest even once, at the store.
#pragma once
#include "common.hpp"

namespace qmm {

constexpr int kF32 = 0, kF16 = 1, kBF16 = 30;   // GGUF type ids

typedef _Float16 f16_t;
typedef __bf16 bf16_t;

template <int T> struct Elem;
template <> struct Elem<kF32> { typedef float type; };
template <> struct Elem<kF16> { typedef f16_t type; };
template <> struct Elem<kBF16> { typedef bf16_t type; };

// N consecutive elements as one aligned value, so that a load or store is one instruction.
template <class T, int N> struct alignas(sizeof(T) * N) Pack { T v[N]; };

template <int N, class T> __device__ __forceinline__ void load_n(const T *p, float (&o)[N]) {
    const Pack<T, N> u = *(const Pack<T, N> *)p;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = (float)u.v[i];
}
template <int N, class T> __device__ __forceinline__ void store_n(T *p, const float (&o)[N]) {
    Pack<T, N> u;
#pragma unroll
    for (int i = 0; i < N; ++i) u.v[i] = (T)o[i];
    *(Pack<T, N> *)p = u;
}

// Host: calls f(a value of the element type of `type`).
template <class F> hipError_t with_type(int type, F f) {
    switch (type) {
        case kF32: return f(float());
        case kF16: return f(f16_t());
        case kBF16: return f(bf16_t());
        default: return hipErrorInvalidValue;
    }
}

inline int elem_bytes(int type) { return type == kF32 ? 4 : type == kF16 || type == kBF16 ? 2 : 0; }
// Every pointer at a multiple of 16 bytes (null ones too).
template <class... P> bool aligned16(P... p) { return (((uintptr_t)p | ... | 0) & 15) == 0; }

}  // namespace qmm
