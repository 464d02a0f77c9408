// Loads and stores of several adjacent elements, the activations' functions, and lane
// reductions for the bandwidth-bound kernels of a block.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"

namespace retn {
namespace {

// V adjacent elements as they lie in memory.  The type is aligned like one element only:
// gfx950 takes wide global loads and stores at any element's address, so rows of any
// stride and width go through the same code.
template <typename T, int V>
struct __attribute__((packed, aligned(sizeof(T)))) Raw {
    T v[V];
};
// They are moved as vectors of words, which the compiler keeps whole.  (As structures of
// elements it splits them to share pieces with the element-wise loads of a cut pack.)
template <int BYTES>
struct Words {
    typedef uint32_t type __attribute__((ext_vector_type(BYTES / 4)));
};
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> raw_load(const T* p) {
    if constexpr (sizeof(T) * V >= 4) {
        typedef typename Words<sizeof(T) * V>::type W;
        typedef W At __attribute__((aligned(sizeof(T))));
        return __builtin_bit_cast(Raw<T, V>, static_cast<W>(*reinterpret_cast<const At*>(p)));
    } else {
        return *reinterpret_cast<const Raw<T, V>*>(p);
    }
}
template <typename T, int V>
__device__ __forceinline__ void raw_store(T* p, const Raw<T, V>& r) {
    if constexpr (sizeof(T) * V >= 4) {
        typedef typename Words<sizeof(T) * V>::type W;
        typedef W At __attribute__((aligned(sizeof(T))));
        *reinterpret_cast<At*>(p) = __builtin_bit_cast(W, r);
    } else {
        *reinterpret_cast<Raw<T, V>*>(p) = r;
    }
}
template <typename T>
__device__ __forceinline__ float up(T x) {
    return io<T>::load(&x);
}
template <typename T>
__device__ __forceinline__ T down(float x) {
    T r;
    io<T>::store(&r, x);
    return r;
}
// Loads and stores past the caches, for what is used once: large outputs (kStreamBytes) of the
// normalisation and of the backward passes, which the caches would not hold until they are
// read again.  Measured per kernel: normalisation of 16384 x 2048 bf16 38 us with plain
// stores, 32 us with these, 30 us with loads too; convolution's gradient 33.6 and 32.2 us,
// scan's 417 and 408 us; rotary positions got slower (51 and 56 us) and keep plain ones.
constexpr size_t kStreamBytes = static_cast<size_t>(8) << 20;
template <typename T, int V>
__device__ __forceinline__ void store_stream(T* p, const Raw<T, V>& r) {
    typedef typename Words<sizeof(T) * V>::type W;
    typedef W At __attribute__((aligned(sizeof(T))));
    asm volatile("");       // on both sides: else the compiler joins it with a plain store beside it
    __builtin_nontemporal_store(__builtin_bit_cast(W, r), reinterpret_cast<At*>(p));
    asm volatile("");
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_stream(const T* p) {
    typedef typename Words<sizeof(T) * V>::type W;
    typedef W At __attribute__((aligned(sizeof(T))));
    asm volatile("");
    return __builtin_bit_cast(Raw<T, V>, static_cast<W>(__builtin_nontemporal_load(reinterpret_cast<const At*>(p))));
}
// The first `left` of V elements, zeros behind them (left >= V: one wide load).
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> raw_load_n(const T* p, int left) {
    if (left >= V) return raw_load<T, V>(p);
    Raw<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = i < left ? p[i] : T(0);
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void raw_store_n(T* p, const Raw<T, V>& r, int left) {
    if (left >= V) {
        raw_store<T, V>(p, r);
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < left) p[i] = r.v[i];
}
template <typename T, int V>
__device__ __forceinline__ void store_n(T* p, const float* x, int left, bool stream = false) {
    Raw<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = down<T>(x[i]);
    if constexpr (V * sizeof(T) >= 8) {
        if (stream && left >= V) {
            store_stream(p, r);
            return;
        }
    }
    raw_store_n(p, r, left);
}
template <typename T>
constexpr int kPack = 16 / static_cast<int>(sizeof(T));   // elements of a 16-byte access

__device__ __forceinline__ float rcp(float x) { return __builtin_amdgcn_rcpf(x); }
// 1 / (1 + e^-x).  The exponent's rounding is relative to x (|x| 2^-24 of e^-x), which the
// bounded x of a gate keeps near the rounding of its own type.
__device__ __forceinline__ float sigmoid_f(float x) { return rcp(1.f + __builtin_amdgcn_exp2f(x * -kLog2e)); }
// log(1 + e^x).  With w = 1 + e rounded, the logarithm of w lacks log(1 + c / w), c = e - (w - 1)
// being what the rounding lost (all of e, where e is small).  Where e^x overflows the sum is
// no number and the maximum takes x, which softplus then is; a NaN stays one.
__device__ __forceinline__ float softplus_f(float x) {
    const float e = __builtin_amdgcn_exp2f(x * kLog2e);
    const float w = 1.f + e, c = e - (w - 1.f);
    return fmaxf(fmaf(c, rcp(w), __builtin_amdgcn_logf(w) * 0.693147180559945f), x);
}

// Exchange with the lane whose number differs in the bits of MASK, for the masks that one
// vector instruction reaches: 1, 2 (quads), 7 (half rows mirrored), 8 (rows rotated).
template <int MASK>
__device__ __forceinline__ float lane_xor(float x) {
    constexpr int ctrl = MASK == 1 ? 0xB1 : MASK == 2 ? 0x4E : MASK == 7 ? 0x141 : 0x128;
    static_assert(MASK == 1 || MASK == 2 || MASK == 7 || MASK == 8, "one instruction");
    const int v = __float_as_int(x);
    return __int_as_float(__builtin_amdgcn_update_dpp(v, v, ctrl, 0xF, 0xF, true));
}
// a of the lower half of each 32 (16) lanes beside b of the upper, summed over the halves:
// lanes 0..31 get a(l) + a(l + 32), lanes 32..63 b(l - 32) + b(l).
__device__ __forceinline__ float halves_sum32(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float halves_sum16(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Sums over partner lanes that differ in bit 3 (lane ^ 8) or, mirrored, in bit 2 (lane ^ 7):
// of a where the bit is clear, of b where it is set.  The second addition writes only the
// banks (four lanes) with the bit set, which takes the place of two selects; the leading
// wait covers the two slots between writing a register and reading it across lanes.
__device__ __forceinline__ float pair_sum8(float a, float b) {
    float r;
    asm("s_nop 1\n\t"
        "v_add_f32_dpp %0, %1, %1 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %0, %2, %2 row_ror:8 row_mask:0xf bank_mask:0xc"
        : "=&v"(r)
        : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ float pair_sum7(float a, float b) {
    float r;
    asm("s_nop 1\n\t"
        "v_add_f32_dpp %0, %1, %1 row_half_mirror row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %0, %2, %2 row_half_mirror row_mask:0xf bank_mask:0xa"
        : "=&v"(r)
        : "v"(a), "v"(b));
    return r;
}
// The sum over a wave's 64 lanes, in every lane.
__device__ __forceinline__ float wave_sum(float x) {
    x += lane_xor<1>(x);
    x += lane_xor<2>(x);
    x += lane_xor<7>(x);
    x += lane_xor<8>(x);
    x = halves_sum16(x, x);
    return halves_sum32(x, x);
}

}  // namespace
}  // namespace retn
