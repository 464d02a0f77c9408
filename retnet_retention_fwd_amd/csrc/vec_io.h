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
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> raw_load(const T* p) {
    return *reinterpret_cast<const Raw<T, V>*>(p);
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
        *reinterpret_cast<Raw<T, V>*>(p) = r;
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < left) p[i] = r.v[i];
}
template <typename T, int V>
__device__ __forceinline__ void store_n(T* p, const float* x, int left) {
    Raw<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = down<T>(x[i]);
    raw_store_n(p, r, left);
}
template <typename T>
constexpr int kPack = 16 / static_cast<int>(sizeof(T));   // elements of a 16-byte access

// e^x to a few units in the last place: the rounding of x log2(e) is carried along (alone
// it costs |x| 2^-24).  Results under the normal range may flush to zero.
__device__ __forceinline__ float exp_acc(float x) {
    x = x < -126.f ? -126.f : x;
    const float t = x * 1.44269502162933349609f;                 // log2(e), upper part
    const float lo = fmaf(x, 1.44269502162933349609f, -t) + x * 1.92596299112661746887e-8f;
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, lo * 0.693147180559945f, e);
}
__device__ __forceinline__ float rcp(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ float sigmoid_f(float x) { return rcp(1.f + exp_acc(x < -80.f ? 80.f : -x)); }
// log(1 + e^x), x itself above 20 (the difference there is below half a unit of x).  The
// logarithm of w = 1 + e is divided by (w - 1) / e, which takes out the rounding of w.
__device__ __forceinline__ float softplus_f(float x) {
    const float e = exp_acc(x > 20.f ? 20.f : x);
    const float w = 1.f + e, d = w - 1.f;
    const float l = d > 0.f ? __builtin_amdgcn_logf(w) * 0.693147180559945f * (e * rcp(d)) : e;
    return x <= 20.f ? l : x;
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
// The sum over two partner lanes, kept as a where the lane's bit is clear, as b where set.
template <int MASK>
__device__ __forceinline__ float pair_sum(float a, float b, bool bit) {
    const float keep = bit ? b : a, send = bit ? a : b;
    return keep + lane_xor<MASK>(send);
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
