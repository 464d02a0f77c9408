// What the scan's forward and backward kernels share.
//
// Walks without channel sums (the forward, the backward's first passes) give a lane a
// channel with all of its S states in registers: nothing is exchanged between lanes, x, dt
// and the gates are read where they are used, and B and C, the same for all lanes, come
// through scalar loads as scalar operands (WaveRows).  A wave is 64 channels of one group
// of one sequence's segment, and needs no other wave: no LDS, no barriers.
#pragma once

#include "block.h"
#include "cdna4.h"
#include "launch.h"
#include "vec_io.h"

namespace retn {
namespace {

constexpr int kScanThreads = 256;
constexpr int kAhead = 8;      // tokens whose loads are issued together, a block ahead

// One token's dt.
__device__ __forceinline__ float step_size(float raw, bool softplus) { return softplus ? softplus_f(raw) : raw; }

__device__ __forceinline__ int scan_length(const int* lengths, int b, int N) {
    if (lengths == nullptr) return N;
    const int n = __builtin_amdgcn_readfirstlane(lengths[b]);   // b is the same for all lanes
    return n < 0 ? 0 : n < N ? n : N;
}

// A wave's or workgroup's place: channel block (of one group), segment, sequence.
struct ScanPlace {
    int g, c0, cend, seg, b, blk;
    int t_begin, t_full, t_end;   // the segment's tokens, all and those of the sequence
};
template <int CH>
__device__ __forceinline__ ScanPlace scan_place(const ScanArgs& a, int nblk, int nseg, int seg, unsigned id) {
    const int per = nblk / a.G, dg = a.D / a.G;
    const unsigned bs = id / nblk;
    ScanPlace p;
    p.blk = static_cast<int>(id % nblk);
    p.g = p.blk / per;
    p.c0 = p.g * dg + p.blk % per * CH;
    p.cend = (p.g + 1) * dg;
    p.seg = bs % nseg;
    p.b = bs / nseg;
    const int n = scan_length(a.lengths, p.b, a.N);
    p.t_begin = p.seg * seg;
    p.t_full = p.t_begin + seg < a.N ? p.t_begin + seg : a.N;
    p.t_end = p.t_full < n ? p.t_full : n;
    return p;
}
// The place of this wave among all waves of a launch of waves (not of workgroups).
__device__ __forceinline__ unsigned wave_id() {
    return __builtin_amdgcn_readfirstlane(blockIdx.x * (kScanThreads / 64) + (threadIdx.x >> 6));
}

// The S values of B or C of one token, as scalars.  SCALAR: S = SP and every row starts at a
// multiple of 4 bytes, so they come by scalar loads from constant memory; else a lane loads
// each and they are read across (S extra vector instructions a token).
template <typename T, int SP, bool SCALAR>
struct WaveRow;
template <int SP>
struct WaveRow<float, SP, true> {
    float v[SP];
    __device__ __forceinline__ void load(const float* p, int) {
        const auto* c = reinterpret_cast<const __attribute__((address_space(4))) float*>(reinterpret_cast<uintptr_t>(p));
#pragma unroll
        for (int i = 0; i < SP; ++i) v[i] = c[i];
    }
    __device__ __forceinline__ float get(int i) const { return v[i]; }
};
template <int SP>
struct WaveRow<bf16_t, SP, true> {
    uint32_t v[SP / 2];
    __device__ __forceinline__ void load(const bf16_t* p, int) {
        const auto* c = reinterpret_cast<const __attribute__((address_space(4))) uint32_t*>(reinterpret_cast<uintptr_t>(p));
#pragma unroll
        for (int i = 0; i < SP / 2; ++i) v[i] = c[i];
    }
    __device__ __forceinline__ float get(int i) const {
        return __uint_as_float(i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
    }
};
template <typename T, int SP>
struct WaveRow<T, SP, false> {
    float v;
    __device__ __forceinline__ void load(const T* p, int S) {
        const int lane = threadIdx.x & 63;
        v = lane < S ? up(p[lane]) : 0.f;
    }
    __device__ __forceinline__ float get(int i) const {
        return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i));
    }
};
// Scalar loads return in any order, so the only wait for one is the wait for all of them.
// Behind this point the rows loaded so far are there, and the next rows' loads, issued right
// behind it, have a whole token's work to arrive.
template <bool SCALAR>
__device__ __forceinline__ void rows_arrived() {
    if (!SCALAR) return;
    __builtin_amdgcn_s_waitcnt(0xC07F);      // lgkmcnt(0), nothing else
    __builtin_amdgcn_sched_barrier(0);
}
template <bool SCALAR>
__device__ __forceinline__ void rows_issued() {
    if (SCALAR) __builtin_amdgcn_sched_barrier(0);
}

// An element of a row that is the same for all lanes: a scalar address and the lane's byte
// offset, which one load instruction adds.
template <typename T>
__device__ __forceinline__ T row_at(const T* row, uint32_t byte) {
    return *reinterpret_cast<const T*>(reinterpret_cast<const char*>(row) + byte);
}
// A stride whose multiples the compiler does not keep (eight of each tensor's would crowd the
// scalar registers): rows are stepped through by adding it.
__device__ __forceinline__ long long stepped(long long ld) {
    asm volatile("" : "+s"(ld));
    return ld;
}
template <typename T>
__device__ __forceinline__ void row_put(T* row, uint32_t byte, T v) {
    *reinterpret_cast<T*>(reinterpret_cast<char*>(row) + byte) = v;
}

// S states of a channel, zeros behind the last one.
template <int SP>
__device__ __forceinline__ void load_state(const float* p, int S, bool on, float (&h)[SP]) {
#pragma unroll
    for (int i = 0; i < SP; i += 4) {
        Raw<float, 4> r = {};
        if (on && i < S) r = raw_load_n<float, 4>(p + i, S - i);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i + j] = r.v[j];
    }
}
template <int SP>
__device__ __forceinline__ void store_state(float* p, int S, const float (&h)[SP]) {
#pragma unroll
    for (int i = 0; i < SP; i += 4)
        if (i < S) raw_store_n<float, 4>(p + i, Raw<float, 4>{{h[i], h[i + 1], h[i + 2], h[i + 3]}}, S - i);
}

// Entry states of a sequence's segments.  Along the walk (from the last segment to the first
// with BACK) segment k takes e_k in and leaves e_(k+1) = exp(A sum_k dt) e_k + own_k, own_k
// being what it makes of a zero state: `at` holds own and gets e.  A lane takes a (channel,
// state) pair.  WAVES = 1: it walks all segments, for there are few of them and many pairs.
// Otherwise the waves of a workgroup share 64 pairs' segments: each composes its own from
// zero, then all of those before it, then walks its own again.  First passes and composition,
// S = 16, bf16, in us with 1 and 16 waves: forward, 16 segments of 524288 pairs 67 and 99,
// 32 of 131072 67 and 77, 64 of 65536 30 and 32, 128 of 16384 32 and 23, 1024 of 2048 112 and
// 39; backward, 32 of 65536 46 and 50, 64 of 32768 76 and 70.
constexpr int kComposeWaves = 16;
template <int WAVES>
struct ComposeSums {
    float own[WAVES][64], dt[WAVES][64];
};
template <int WAVES, bool BACK>
__device__ __forceinline__ void compose(float* at, const float* sum, size_t ds, int D, int nseg, float A2, float init,
                                        ComposeSums<WAVES>& sums) {
    constexpr int U = WAVES > 1 ? 8 : 16;      // segments whose loads are in flight together
    const int lane = threadIdx.x & 63, wave = WAVES > 1 ? threadIdx.x >> 6 : 0;
    const int each = (nseg + WAVES - 1) / WAVES, k0 = wave * each;
    const int k1 = k0 + each < nseg ? k0 + each : nseg;
    float own[U], dt[U];
    auto fetch = [&](int k) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int kk = k + i, s = BACK ? nseg - 1 - kk : kk;
            // (the last segment of the walk has nothing to hand on, and its slot may be unset)
            const bool hands = kk < k1 && kk < nseg - 1;
            own[i] = hands ? at[s * ds] : 0.f;
            dt[i] = hands ? sum[static_cast<size_t>(s) * D] : 0.f;
        }
    };
    float e = init;
    if constexpr (WAVES > 1) {
        float h = 0.f, total = 0.f;
        for (int k = k0; k < k1; k += U) {
            fetch(k);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                h = fmaf(exp2_fast(A2 * dt[i]), h, own[i]);
                total += dt[i];
            }
        }
        sums.own[wave][lane] = h;
        sums.dt[wave][lane] = total;
        __syncthreads();
        for (int w = 0; w < wave; ++w) e = fmaf(exp2_fast(A2 * sums.dt[w][lane]), e, sums.own[w][lane]);
    }
    for (int k = k0; k < k1; k += U) {
        fetch(k);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (k + i >= k1) break;
            at[(BACK ? nseg - 1 - k - i : k + i) * ds] = e;
            e = fmaf(exp2_fast(A2 * dt[i]), e, own[i]);
        }
    }
}
inline int compose_waves(int nseg) { return nseg > 3 * kComposeWaves ? kComposeWaves : 1; }

// Whether B's and C's rows can be read by scalar loads (WaveRow).
inline bool scalar_rows(const ScanArgs& a, int SP) {
    if (a.S != SP) return false;
    const size_t es = a.bf16 ? 2 : 4;
    auto even = [&](const void* p, long long ld) {
        return (reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * es)) % 4 == 0;
    };
    return even(a.Bm, a.ldb) && even(a.Cm, a.ldc);
}

}  // namespace
}  // namespace retn
