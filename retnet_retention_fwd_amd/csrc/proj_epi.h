// What the products of proj.hip and proj_small.hip share: a fragment's products, and what happens
// to the sums (bias, activation, residual, the gated product and its gradients).
#pragma once

#include "act.h"
#include "cdna4.h"
#include "proj.h"
#include "vec_io.h"

namespace retn {
namespace {

// c += a b over one fragment: 16 x 16 sums, 32 (bf16) or 16 (fp32) elements of the reduction.
// Lane (g, l) = (lane / 16, lane % 16) brings row l of a and column l of b, 16 bytes of the
// reduction from 16 g on, and holds columns ... of c as the matrix instructions do; which
// elements meet in one instruction is the same for both operands, so any order will do.
template <typename T>
__device__ __forceinline__ f32x4_t frag_mul(u16x8_t a, u16x8_t b, f32x4_t c) {
    if constexpr (sizeof(T) == 2) {
        return mfma16(a, b, c);
    } else {
        const f32x4_t x = __builtin_bit_cast(f32x4_t, a), y = __builtin_bit_cast(f32x4_t, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[j], y[j], c, 0, 0, 0);
        return c;
    }
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, int left, float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        const Raw<T, 8> r = raw_load_n<T, 8>(p, left);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = up(r.v[i]);
    } else {
        const Raw<T, 4> r = raw_load_n<T, 4>(p, left), q = raw_load_n<T, 4>(p + 4, left - 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = r.v[i];
            v[i + 4] = q.v[i];
        }
    }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8], int left) {
    if constexpr (sizeof(T) == 2) {
        store_n<T, 8>(p, v, left);
    } else {
        const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
        store_n<T, 4>(p, lo, left);
        store_n<T, 4>(p + 4, hi, left - 4);
    }
}

// Waits for a loaded value here.  (Loads and stores count on one counter in their order, so a wait
// behind stores, or in a loop with them, is one for the stores as well.)
template <typename V>
__device__ __forceinline__ void arrived(V& v) {
    asm volatile("" : "+v"(v));
}
// What a lane's eight columns n .. n + 7 have in every row.
template <typename T, int KIND>
struct Columns {
    float bias[KIND == kProjLinear ? 8 : 1];
    __device__ __forceinline__ void load(const ProjEpi& e, int n, int left) {
        if constexpr (KIND == kProjLinear) {
#pragma unroll
            for (int i = 0; i < 8; ++i) bias[i] = 0.f;
            if (e.bias == nullptr || left <= 0) return;
            if (e.bias_f32)
                load8<float>(static_cast<const float*>(e.bias) + n, left, bias);
            else
                load8<T>(static_cast<const T*>(e.bias) + n, left, bias);
#pragma unroll
            for (int i = 0; i < 8; ++i) arrived(bias[i]);
        }
    }
};
// Eight adjacent elements as they lie in memory.
template <typename T>
struct Eight {
    static constexpr int V = kPack<T>;
    Raw<T, V> r[8 / V];
    __device__ __forceinline__ void load(const T* p, int left) {
#pragma unroll
        for (int i = 0; i < 8 / V; ++i) r[i] = raw_load_n<T, V>(p + i * V, left - i * V);
    }
    __device__ __forceinline__ void open(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = up(r[i / V].v[i % V]);
    }
    __device__ __forceinline__ void wait() {
#pragma unroll
        for (int i = 0; i < 8 / V; ++i) {
            u32x4_t w = __builtin_bit_cast(u32x4_t, r[i]);
            arrived(w);
            r[i] = __builtin_bit_cast(decltype(Raw<T, V>{}), w);
        }
    }
};
// What R rows m[r] read besides the sums: the residual, or gate and up.
template <typename T, int KIND, int R>
struct Reads {
    static constexpr int N = KIND == kProjGated ? 0 : KIND == kProjGatedBwd ? 2 : 1;
    Eight<T> x[N > 0 ? R : 1], u[N > 1 ? R : 1];
    __device__ __forceinline__ void wait(const ProjEpi& e) {
        if constexpr (N > 0) {
            if (KIND == kProjLinear && e.res == nullptr) return;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                x[r].wait();
                if constexpr (N > 1) u[r].wait();
            }
        }
    }
    __device__ __forceinline__ void load(const ProjEpi& e, const ProjGroup& g, const int (&m)[R], int n) {
        if constexpr (N > 0) {
            if (n >= g.N || (KIND == kProjLinear && e.res == nullptr)) return;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (m[r] >= g.M) continue;
                if constexpr (KIND == kProjLinear) {
                    x[r].load(static_cast<const T*>(e.res) + static_cast<size_t>(m[r]) * g.N + n, g.N - n);
                } else {
                    const size_t at = static_cast<size_t>(m[r]) * e.gate_ld + n;
                    x[r].load(static_cast<const T*>(e.gate) + at, e.gate_n - n);
                    u[r].load(static_cast<const T*>(e.up) + at, e.gate_n - n);
                }
            }
        }
    }
};
// Columns of a padded product past gate's and up's are zero also where an infinite operand met the
// zeros there: the next product reads them.
__device__ __forceinline__ void no_padding(float (&v)[8], int left) {
    if (left >= 8) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? v[i] : 0.f;
}
// What a product stores is rounded to T once.  In bf16 that holds for the gated product (kind gated: c) and for the
// gradients and the product behind the gate (kind gated backward: ggate, gup, prod) too, which the next product reads: the
// matrix instructions take bf16 operands, and two parts of each value instead would double that product's
// instructions.  Relative to 64 bits the block's outputs are then off by 1.9e-3 and its gradients by 2.3e-3, of which
// the rounding of the outputs themselves is 1.7e-3.  All else (sums, activations, slopes) stays in fp32.
//
// R rows m[r] of eight adjacent columns n .. n + 7 (`v`, and `w`: the second projection's sums).
template <typename T, int KIND, int R>
__device__ __forceinline__ void finish(const ProjEpi& e, const ProjGroup& g, const Columns<T, KIND>& cols,
                                       const Reads<T, KIND, R>& reads, const int (&m)[R], int n, float (&v)[R][8],
                                       float (&w)[R][8]) {
    const int left = g.N - n;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (m[r] >= g.M) continue;
        const size_t ca = static_cast<size_t>(m[r]) * g.ldc + n;
        T* const c = static_cast<T*>(g.c) + ca;
        if constexpr (KIND == kProjLinear) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[r][i] += cols.bias[i];
            if (e.pre != nullptr) store8<T>(static_cast<T*>(e.pre) + static_cast<size_t>(m[r]) * g.N + n, v[r], left);
            act_values(v[r], e.act);
            if (e.res != nullptr) {
                float x[8];
                reads.x[r].open(x);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[r][i] += x[i];
            }
            store8<T>(c, v[r], left);
        } else if constexpr (KIND == kProjGated) {
            no_padding(v[r], e.gate_n - n);
            no_padding(w[r], e.gate_n - n);
            const size_t ga = static_cast<size_t>(m[r]) * e.gate_ld + n;
            if (e.gate != nullptr) store8<T>(static_cast<T*>(e.gate) + ga, v[r], e.gate_n - n);
            if (e.up != nullptr) store8<T>(static_cast<T*>(e.up) + ga, w[r], e.gate_n - n);
            act_values(v[r], e.act);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[r][i] *= w[r][i];
            store8<T>(c, v[r], left);
        } else {
            float x[8], u[8], h[8], a[8];
            reads.x[r].open(x);
            reads.u[r].open(u);
            no_padding(v[r], e.gate_n - n);
            act_slopes(x, a, e.act);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[i] = a[i] * u[i];
                x[i] *= v[r][i] * u[i];
                v[r][i] *= a[i];
            }
            if (e.ggate != nullptr) store8<T>(static_cast<T*>(e.ggate) + ca, x, left);
            if (e.gup != nullptr) store8<T>(static_cast<T*>(e.gup) + ca, v[r], left);
            if (e.prod != nullptr) store8<T>(static_cast<T*>(e.prod) + ca, h, left);
        }
    }
}

}  // namespace
}  // namespace retn
