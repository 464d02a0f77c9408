// What the scan's forward and backward kernels share.
//
// Walks without channel sums (the forward, the backward's first passes) give a lane a
// channel with all of its S states in registers: nothing is exchanged between lanes, x, dt
// and the gates are read where they are used, the products of B (or C) with a lane's value are
// added by the matrix cores (MatRows), and the read-out takes C, the same for all lanes, as
// scalar operands (WaveRow).  A wave is 64 channels of one group of one sequence's segment,
// and needs no other wave: no LDS, no barriers.
#pragma once

#include "block.h"
#include "cdna4.h"
#include "launch.h"
#include "vec_io.h"

#include <utility>

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

// The S values of C of one token for the forward's read-out.  SCALAR: S = SP and every row
// starts at a multiple of 4 bytes, so they come by scalar loads from constant memory, as
// operands of the multiply-adds.  Otherwise lane l of register q loads state 16 q + l % 16 and a
// state is read from its lane of each sixteen, which costs an instruction a state more.
template <typename T, int SP, bool SCALAR>
struct WaveRow {
    static constexpr int kRegs = SP > 16 ? SP / 16 : 1;
    T raw[kRegs];
    __device__ __forceinline__ void load(const T* row, int S) {
        const int l = static_cast<int>(opaque(threadIdx.x & 15));
#pragma unroll
        for (int q = 0; q < kRegs; ++q) raw[q] = row_at(row, static_cast<uint32_t>(16 * q + l < S ? 16 * q + l : 0) * sizeof(T));
    }
    template <int I>
    __device__ __forceinline__ float get(int S) const {
        const float v = 16 * (I / 16) + static_cast<int>(threadIdx.x & 15) < S ? up(raw[I / 16]) : 0.f;
        return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x150 + I % 16, 0xf, 0xf, true));   // row_newbcast
    }
};
template <int SP>
struct WaveRow<float, SP, true> {
    float v[SP];
    __device__ __forceinline__ void load(const float* p, int) {
        const auto* c = reinterpret_cast<const __attribute__((address_space(4))) float*>(reinterpret_cast<uintptr_t>(p));
#pragma unroll
        for (int i = 0; i < SP; ++i) v[i] = c[i];
    }
    template <int I>
    __device__ __forceinline__ float get(int) const {
        return v[I];
    }
};
template <int SP>
struct WaveRow<bf16_t, SP, true> {
    uint32_t v[SP / 2];
    __device__ __forceinline__ void load(const bf16_t* p, int) {
        const auto* c = reinterpret_cast<const __attribute__((address_space(4))) uint32_t*>(reinterpret_cast<uintptr_t>(p));
#pragma unroll
        for (int i = 0; i < SP / 2; ++i) v[i] = c[i];
    }
    template <int I>
    __device__ __forceinline__ float get(int) const {
        return __uint_as_float(I & 1 ? v[I / 2] & 0xffff0000u : v[I / 2] << 16);
    }
};

// f(0), .., f(N - 1), each with its number as a constant.
template <typename F, int... K>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, K...>) {
    (f(std::integral_constant<int, K>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
    each_of(static_cast<F&&>(f), std::make_integer_sequence<int, N>{});
}

// Rows of B or C for the matrix cores: lane l of a register holds state l % SP of its token
// l / SP, zero behind the last state.
template <typename T, int SP>
struct MatRows {
    static constexpr int kTok = 64 / SP;       // tokens of a register
    static __device__ __forceinline__ uint32_t lane_at(long long ld, int S) {
        const uint32_t l = threadIdx.x & 63, s = l % SP;
        return (l / SP * static_cast<uint32_t>(ld) + (s < static_cast<uint32_t>(S) ? s : 0)) * sizeof(T);
    }
    static __device__ __forceinline__ float value(T raw, int S) {
        return static_cast<int>((threadIdx.x & 63) % SP) < S ? up(raw) : 0.f;
    }
};
// The same of a block of kAhead tokens.
template <typename T, int SP>
struct MatBlock {
    using R = MatRows<T, SP>;
    static constexpr int kTok = R::kTok < kAhead ? R::kTok : kAhead, kRegs = kAhead / kTok;
    T raw[kRegs];
    __device__ __forceinline__ void load(const T* rows, long long ld, uint32_t lane) {
#pragma unroll
        for (int r = 0; r < kRegs; ++r) raw[r] = row_at(rows + r * kTok * ld, lane);
    }
    __device__ __forceinline__ void values(int S, float (&v)[kRegs]) const {
#pragma unroll
        for (int r = 0; r < kRegs; ++r) v[r] = R::value(raw[r], S);
    }
};
// One token's outer product: h[state] = B[state] u + decayed[state], for the lane's channel u.
// The 4x4 matrix instruction has 16 blocks of four lanes: a block's column is a lane, its rows
// are four of the lane's states, and the four B of its rows come from one block of the B
// register, the same for all blocks.  K = 1: no channel and no state meets another's values.
// Any S and alignment run alike.  Against B by scalar operands where S and alignment allowed it,
// read across lanes elsewhere, forward of 4 x 2048 x 2048 channels: bf16 16 states 128 and 128
// us, 13 states 137 and 226, fp32 133 and 146; 32 x 512 x 1024 channels 124 and 132.
template <int SP, int TOK, int J>
__device__ __forceinline__ f32v4 outer(float row, float u, f32v4 decayed) {
    return __builtin_amdgcn_mfma_f32_4x4x1f32(row, u, decayed, 4, TOK * (SP / 4) + J, 0);
}

// Scalar loads return in any order, so the only wait for one is the wait for all of them.
// Behind this point the rows loaded so far are there, and the next rows' loads, issued right
// behind it, have a whole token's work to arrive.
__device__ __forceinline__ void rows_arrived() {
    __builtin_amdgcn_s_waitcnt(0xC07F);      // lgkmcnt(0), nothing else
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void rows_issued() {
    __builtin_amdgcn_sched_barrier(0);
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

// A state carried over tokens of log2 decay x in all: 2^x e + own.  Where tokens grow (A dt > 0) the
// factor of many can overflow although none of theirs does: it is then applied in two halves, and
// a state of zero stays zero, as token by token.
__device__ __forceinline__ float carry(float x, float e, float own) {
    const bool far = x > 127.f;
    const float f = exp2_fast(far ? 0.5f * x : x);
    return e != 0.f ? fmaf(f, far ? f * e : e, own) : own;
}

// Entry states of a sequence's segments.  Along the walk (from the last segment to the first
// with BACK) segment k takes e_k in and leaves e_(k+1) = exp(A sum_k dt) e_k + own_k, own_k
// being what it makes of a zero state: `at` holds own and gets e.  A lane takes a (channel,
// state) pair.  WAVES = 1: it walks all segments, for there are few of them and many pairs.
// Otherwise the waves of a workgroup share 64 pairs' segments: each composes its own from
// zero, then all of those before it, then walks its own again, which reads them twice.  First
// passes and composition, bf16, in us with 1 and 16 waves: forward, 16 segments of 524288 pairs 67 and
// 99, 32 of 131072 67 and 77, 128 of 131072 84 and 121, 64 of 65536 30 and 32, 128 of 32768 116
// and 112, 128 of 16384 32 and 23, 1024 of 2048 112 and 39; backward, 32 of 65536 46 and
// 50, 64 of 32768 76 and 70.
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
    float own[U], dt[U];                       // (dt: then its log2 decay)
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
    // the fetched segments' factors; whether a lane of the wave has one beyond fp32
    auto decays = [&]() {
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i) most = fmaxf(most, dt[i] *= A2);
        return __any(most > 127.f);
    };
    float e = init;
    if constexpr (WAVES > 1) {
        float h = 0.f, total = 0.f;
        for (int k = k0; k < k1; k += U) {
            fetch(k);
#pragma unroll
            for (int i = 0; i < U; ++i) total += dt[i];
            if (decays()) {
#pragma unroll
                for (int i = 0; i < U; ++i) h = carry(dt[i], h, own[i]);
            } else {
#pragma unroll
                for (int i = 0; i < U; ++i) h = fmaf(exp2_fast(dt[i]), h, own[i]);
            }
        }
        sums.own[wave][lane] = h;
        sums.dt[wave][lane] = total;
        __syncthreads();
        for (int w = 0; w < wave; ++w) e = carry(A2 * sums.dt[w][lane], e, sums.own[w][lane]);
    }
    for (int k = k0; k < k1; k += U) {
        fetch(k);
        auto walk = [&](auto next) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (k + i >= k1) break;
                at[(BACK ? nseg - 1 - k - i : k + i) * ds] = e;
                e = next(dt[i], e, own[i]);
            }
        };
        if (decays())
            walk(carry);
        else
            walk([](float x, float e, float own) { return fmaf(exp2_fast(x), e, own); });
    }
}
inline int compose_waves(int nseg, size_t pairs) { return nseg > 48 && pairs <= 32768 ? kComposeWaves : 1; }

// Whether C's rows can be read by scalar loads (WaveRow).
inline bool scalar_rows(const ScanArgs& a, int SP) {
    if (a.S != SP) return false;
    const size_t es = a.bf16 ? 2 : 4;
    return (reinterpret_cast<uintptr_t>(a.Cm) | static_cast<uintptr_t>(a.ldc * es)) % 4 == 0;
}

}  // namespace
}  // namespace retn
