// What the scan's forward and backward kernels share: lane layout, staging, reductions.
//
// Lanes.  LPC adjacent lanes hold one channel's states, SPL each (4 LPC >= S states): lane
// = LPC c + q' for channel c of the wave.  A wave of 64 channels-by-state-groups walks over
// tokens with its states in registers; x, dt and the gates are staged once per (token,
// channel) in LDS, so their transcendental functions are not repeated in the LPC lanes.
// With LPC = 4 the state group of a lane is q' with its two bits flipped in odd channels:
// then lane ^ 7, which one DPP instruction reaches, is the neighbouring channel's lane of
// the same state group, and sums over channels as well as over a channel's states run on
// DPP and permlane-swap instructions without LDS.
#pragma once

#include "block.h"
#include "cdna4.h"
#include "launch.h"
#include "vec_io.h"

namespace retn {
namespace {

constexpr int kScanThreads = 256;

template <int LPC>
__device__ __forceinline__ int state_group(int lane) {
    const int q = lane & (LPC - 1);
    return LPC == 4 ? q ^ ((lane & 4) ? 3 : 0) : q;
}

// Sums over the LPC lanes of a channel of LPC values each; the lane keeps the sum of value
// `kept(lane)`.  Mask 7 comes before 1 and 2: its partner then differs in them, later
// partners agree in what has been kept.
template <int LPC>
__device__ __forceinline__ float state_sum(const float* v, int lane) {
    float t[LPC];
#pragma unroll
    for (int i = 0; i < LPC; ++i) t[i] = v[i];
    if (LPC >= 16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = pair_sum<8>(t[i], t[(i + 8) & (LPC - 1)], lane & 8);
    }
    if (LPC >= 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = pair_sum<7>(t[i], t[(i + 4) & (LPC - 1)], lane & 4);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) t[i] = pair_sum<2>(t[i], t[i + 2], lane & 2);
    return pair_sum<1>(t[0], t[1], lane & 1);
}
// The value that state_sum leaves in a lane is number lane & (LPC - 1).

// One token's dt and its factors for the tile's rows behind `rows`: dt = u = 0 keeps the state.
__device__ __forceinline__ float step_size(float raw, bool softplus) { return softplus ? softplus_f(raw) : raw; }

__device__ __forceinline__ int scan_length(const int* lengths, int b, int N) {
    if (lengths == nullptr) return N;
    const int n = lengths[b];
    return n < 0 ? 0 : n < N ? n : N;
}

// The workgroup's place: channel block (of one group), segment, sequence.
struct ScanPlace {
    int g, c0, cend, seg, b;
};
template <int CH>
__device__ __forceinline__ ScanPlace scan_place(const ScanArgs& a, int nblk, int nseg, unsigned id) {
    const int per = nblk / a.G, dg = a.D / a.G, blk = id % nblk;
    const unsigned bs = id / nblk;
    ScanPlace p;
    p.g = blk / per;
    p.c0 = p.g * dg + blk % per * CH;
    p.cend = (p.g + 1) * dg;
    p.seg = bs % nseg;
    p.b = bs / nseg;
    return p;
}

// B and C of a tile's tokens, [TT][SP] in LDS, zeros behind the last state and token.
template <typename T, int TT, int SP>
struct StateRows {
    static constexpr int kPer = (TT * SP + kScanThreads - 1) / kScanThreads;
    T raw[kPer];
    __device__ __forceinline__ void load(const T* p, long long ld, int rows, int S) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = threadIdx.x + k * kScanThreads, t = i / SP, n = i % SP;
            raw[k] = t < rows && n < S ? p[t * ld + n] : T(0);
        }
    }
    __device__ __forceinline__ void store(float* lds) const {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = threadIdx.x + k * kScanThreads;
            if (TT * SP % kScanThreads == 0 || i < TT * SP) lds[i] = up(raw[k]);
        }
    }
};

template <int SPL>
__device__ __forceinline__ void lds_states(const float* p, float (&out)[SPL]) {
    if (SPL % 4 == 0) {
#pragma unroll
        for (int i = 0; i < SPL; i += 4) {
            const f32v4 v = *reinterpret_cast<const f32v4*>(p + i);
            out[i] = v.x;
            out[i + 1] = v.y;
            out[i + 2] = v.z;
            out[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < SPL; ++i) out[i] = p[i];
    }
}

// S states of a channel: a lane's SPL of them, from n0, zeros behind the last one.
template <int SPL>
__device__ __forceinline__ void load_state(const float* p, int n0, int S, bool on, float (&h)[SPL]) {
#pragma unroll
    for (int i = 0; i < SPL; ++i) h[i] = on && n0 + i < S ? p[n0 + i] : 0.f;
}
template <int SPL>
__device__ __forceinline__ void store_state(float* p, int n0, int S, const float (&h)[SPL]) {
    if (SPL % 4 == 0 && S % 4 == 0) {
#pragma unroll
        for (int i = 0; i < SPL; i += 4)
            if (n0 + i < S) *reinterpret_cast<Raw<float, 4>*>(p + n0 + i) = Raw<float, 4>{{h[i], h[i + 1], h[i + 2], h[i + 3]}};
        return;
    }
#pragma unroll
    for (int i = 0; i < SPL; ++i)
        if (n0 + i < S) p[n0 + i] = h[i];
}

}  // namespace
}  // namespace retn
