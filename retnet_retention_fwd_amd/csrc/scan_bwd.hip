// Backward of the selective scan.  With g_t = gy_t silu(z_t) and the adjoint state
//     w_t = C_t g_t + exp(dt_(t+1) A) w_(t+1)   (+ grad_state_out behind the last token),
// the gradients are
//     du_t = sum_n w_t B_t,   q_t[n] = w_t h_(t-1) exp(dt_t A),
//     dx = du dt + D g,       ddt = du x + sum_n q A  (times sigmoid(raw + bias)),
//     dA = sum_t q dt,        dB_t = sum_channels w dt x,   dC_t = sum_channels g h_t,
//     dD = sum g x,           dz = gy (C.h + D x) silu'(z).
//
// Bound by the vector ALUs, like the forward.  A first pass walks forward (a lane a channel,
// scan.h) and keeps the state in front of every 16th token; the main pass takes tiles of 16
// tokens from the last to the first.  It recomputes the states in front of the tile's parts of
// four tokens, then the states and decays of a part into registers, and walks back through
// them: no state but one in 16 is ever in memory, and an exponential is taken 2.75 times per
// (token, channel, state), 3.75 times with the segments' walk back.
//
// dB and dC sum over channels, so the main pass spreads a channel's states over LPC lanes, four
// each: few enough to keep a part of them, and lanes of the same states are then the ones to
// sum over.  A wave sums its channels' terms in registers (permlane swaps and DPP), a
// workgroup its waves' in LDS, a second kernel the workgroups' in a fixed order.  Everything
// that is per (token, channel) is computed once for the tile and kept in LDS.  The parameters'
// sums over tokens stay in registers until the end of a segment.
//
// Segments, where channels are few: the first pass walks each from a zero state, a second
// one walks the adjoint back through each from zero, and a small kernel composes both into
// the states that enter the segments from either side.
//
// Measured, S = 16, bf16, gated: 4 x 2048 x 2048 channels 374 us, of which first passes 101,
// composition 10, main pass 250 (vector ALUs busy 92%; 51 KB of LDS and 168 registers leave
// three workgroups a CU, and parts of eight tokens do not fit those registers), sums 12.

#include "scan.h"

namespace retn {

namespace {

constexpr int kTile = 16;      // tokens of a tile, and between kept states
constexpr int kPart = 4;       // tokens whose states and decays are in registers together
constexpr size_t kWantWaves = 2048;   // of either first pass: two a SIMD
constexpr int SPL = 4;         // states of a lane in the main pass

// The state in front of each tile, its segment walked from zero, and the sum of dt from the
// segment's first token to there; the end state and whole sum of dt go to the segment's slot.
template <typename T, int SP, bool ALL>
__device__ __forceinline__ void keep_states(const ScanArgs& a, const ScanPlan& pl, int nblk, unsigned id) {
    const ScanPlace p = scan_place<64>(a, nblk, pl.nseg, pl.seg, id);
    const int c = p.c0 + (threadIdx.x & 63), S = ALL ? SP : a.S;
    const bool on = c < p.cend;
    const int ch = on ? c : p.cend - 1;
    using Block = MatBlock<T, SP>;
    float A2[SP], dsum = 0.f;
    f32v4 h[SP / 4];
    load_state<SP>(a.A + static_cast<size_t>(ch) * S, S, true, A2);
#pragma unroll
    for (int i = 0; i < SP; ++i) {
        A2[i] *= kLog2e;
        h[i / 4][i % 4] = 0.f;
    }
    const int tiles = (a.N + kTile - 1) / kTile;
    const float bias = a.bias != nullptr ? a.bias[ch] : 0.f;
    const size_t tok0 = static_cast<size_t>(p.b) * a.N;
    const T* xp = static_cast<const T*>(a.x) + tok0 * a.ldx;
    const T* dp = static_cast<const T*>(a.dt) + tok0 * a.lddt;
    const uint32_t lane_at = static_cast<uint32_t>(ch) * sizeof(T);
    const T* Bp = static_cast<const T*>(a.Bm) + tok0 * a.ldb + p.g * S;
    const uint32_t row_lane = MatRows<T, SP>::lane_at(a.ldb, S), row_one = MatRows<T, SP>::lane_at(0, S);
    auto step = [&](float dt, float x, float B, auto tok) __attribute__((always_inline)) {
        const float u = dt * x;
        each<SP / 4>([&](auto j) __attribute__((always_inline)) {
            f32v4 d;
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = exp2_fast(dt * A2[4 * j + i]) * h[j][i];
            h[j] = outer<SP, tok, j>(B, u, d);
        });
        dsum += dt;
    };
    auto put = [&](float* to) {
        float v[SP];
#pragma unroll
        for (int i = 0; i < SP; ++i) v[i] = h[i / 4][i % 4];
        store_state<SP>(to, S, v);
    };
    auto keep = [&](int t) {
        if (!on) return;
        const size_t at = (static_cast<size_t>(p.b) * tiles + t / kTile) * a.D + ch;
        put(a.workspace + pl.off_ckpt + at * S);
        a.workspace[pl.off_cum + at] = dsum;
    };
    T rx[kAhead], rdt[kAhead];
    Block rB;
    auto fetch = [&](int t0) {
        const long long ldx = stepped(a.ldx), lddt = stepped(a.lddt);
        const uint32_t at = opaque(lane_at);   // added last, by the load itself
        const T* xr = xp + t0 * ldx;
        const T* dr = dp + t0 * lddt;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            rx[k] = row_at(xr, at);
            rdt[k] = row_at(dr, at);
            xr += ldx;
            dr += lddt;
        }
        rB.load(Bp + t0 * a.ldb, a.ldb, row_lane);
    };
    int t = p.t_begin;
    if (t + kAhead <= p.t_end) fetch(t);
    for (; t + kAhead <= p.t_end; t += kAhead) {
        if (t % kTile == 0) keep(t);
        float x[kAhead], dt[kAhead], B[Block::kRegs];
        rB.values(S, B);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            x[k] = up(rx[k]);
            dt[k] = up(rdt[k]) + bias;
        }
        if (t + 2 * kAhead <= p.t_end) fetch(t + kAhead);
        if (a.softplus) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) dt[k] = softplus_f(dt[k]);
        }
        each<kAhead>([&](auto k) __attribute__((always_inline)) {
            step(dt[k], x[k], B[k / Block::kTok], std::integral_constant<int, k % Block::kTok>{});
        });
    }
    for (; t < p.t_end; ++t) {
        if (t % kTile == 0) keep(t);
        const size_t tt = t;
        const float B = MatRows<T, SP>::value(row_at(Bp + tt * a.ldb, row_one), S);
        step(step_size(up(row_at(dp + tt * a.lddt, lane_at)) + bias, a.softplus), up(row_at(xp + tt * a.ldx, lane_at)), B,
             std::integral_constant<int, 0>{});
    }
    if (!on || pl.nseg == 1) return;
    const size_t slot = (static_cast<size_t>(p.b) * pl.nseg + p.seg) * a.D + ch;
    put(a.workspace + pl.off_end + slot * S);
    a.workspace[pl.off_dt + slot] = dsum;
}

// The adjoint that leaves each segment but the first at its front, from zero behind its end.
template <typename T, int SP, bool ALL>
__device__ __forceinline__ void walk_back(const ScanArgs& a, const ScanPlan& pl, int nblk, unsigned id) {
    ScanPlace p = scan_place<64>(a, nblk, pl.nseg - 1, pl.seg, id);
    p.seg += 1;                                // the place of the segment behind
    p.t_begin = p.seg * pl.seg;
    p.t_full = p.t_begin + pl.seg < a.N ? p.t_begin + pl.seg : a.N;
    const int n = scan_length(a.lengths, p.b, a.N);
    p.t_end = p.t_full < n ? p.t_full : n;
    const int c = p.c0 + (threadIdx.x & 63), S = ALL ? SP : a.S;
    const bool on = c < p.cend;
    const int ch = on ? c : p.cend - 1;
    using Block = MatBlock<T, SP>;
    float A2[SP];
    f32v4 w[SP / 4];
    load_state<SP>(a.A + static_cast<size_t>(ch) * S, S, true, A2);
#pragma unroll
    for (int i = 0; i < SP; ++i) {
        A2[i] *= kLog2e;
        w[i / 4][i % 4] = 0.f;
    }
    const float bias = a.bias != nullptr ? a.bias[ch] : 0.f;
    const size_t tok0 = static_cast<size_t>(p.b) * a.N;
    const T* dp = static_cast<const T*>(a.dt) + tok0 * a.lddt;
    const T* zp = static_cast<const T*>(a.z) + tok0 * a.ldz;
    const T* gp = static_cast<const T*>(a.gy) + tok0 * a.D;
    const uint32_t lane_at = static_cast<uint32_t>(ch) * sizeof(T);
    const T* Cp = static_cast<const T*>(a.Cm) + tok0 * a.ldc + p.g * S;
    const bool gated = a.z != nullptr;
    const uint32_t row_lane = MatRows<T, SP>::lane_at(a.ldc, S), row_one = MatRows<T, SP>::lane_at(0, S);
    auto step = [&](float dt, float g, float C, auto tok) __attribute__((always_inline)) {
        each<SP / 4>([&](auto j) __attribute__((always_inline)) {
            w[j] = outer<SP, tok, j>(C, g, w[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[j][i] *= exp2_fast(dt * A2[4 * j + i]);
        });
    };
    const int blocks = p.t_end > p.t_begin ? (p.t_end - p.t_begin) / kAhead : 0;
    for (int t = p.t_end - 1; t >= p.t_begin + blocks * kAhead; --t) {
        const size_t tt = t;
        const float C = MatRows<T, SP>::value(row_at(Cp + tt * a.ldc, row_one), S);
        float g = up(row_at(gp + tt * a.D, lane_at));
        if (gated) {
            const float z = up(row_at(zp + tt * a.ldz, lane_at));
            g *= z * sigmoid_f(z);
        }
        step(step_size(up(row_at(dp + tt * a.lddt, lane_at)) + bias, a.softplus), g, C, std::integral_constant<int, 0>{});
    }
    T rdt[kAhead], rz[kAhead] = {}, rg[kAhead];
    Block rC;
    auto fetch = [&](int t0) {
        const long long lddt = stepped(a.lddt), ldg = stepped(a.D), ldz = stepped(a.ldz);
        const uint32_t at = opaque(lane_at);
        const T* dr = dp + t0 * lddt;
        const T* gr = gp + t0 * ldg;
        const T* zr = zp + t0 * ldz;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            rdt[k] = row_at(dr, at);
            rg[k] = row_at(gr, at);
            dr += lddt;
            gr += ldg;
        }
        if (gated) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                rz[k] = row_at(zr, at);
                zr += ldz;
            }
        }
        rC.load(Cp + t0 * a.ldc, a.ldc, row_lane);
    };
    if (blocks > 0) fetch(p.t_begin + (blocks - 1) * kAhead);
    for (int blk = blocks - 1; blk >= 0; --blk) {
        const int t = p.t_begin + blk * kAhead;
        float dt[kAhead], g[kAhead], z[kAhead], C[Block::kRegs];
        rC.values(S, C);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            dt[k] = up(rdt[k]) + bias;
            g[k] = up(rg[k]);
            z[k] = up(rz[k]);
        }
        if (blk > 0) fetch(t - kAhead);
        if (a.softplus) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) dt[k] = softplus_f(dt[k]);
        }
        if (gated) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) g[k] *= z[k] * sigmoid_f(z[k]);
        }
        each<kAhead>([&](auto i) __attribute__((always_inline)) {
            constexpr int k = kAhead - 1 - i;
            step(dt[k], g[k], C[k / Block::kTok], std::integral_constant<int, k % Block::kTok>{});
        });
    }
    if (!on) return;
    const size_t slot = (static_cast<size_t>(p.b) * pl.nseg + p.seg) * a.D + ch;
    float out[SP];
#pragma unroll
    for (int i = 0; i < SP; ++i) out[i] = w[i / 4][i % 4];
    store_state<SP>(a.workspace + pl.off_rev + slot * S, S, out);
}

// Both walks in one launch: neither needs the other, and together they bring each SIMD the
// waves that keep its vector ALU busy (22 us less than one behind the other in a training step's
// backward, where they take 101 us together).
// ALL: S = SP; its rows are then stored without tests (4 x 2048 x 512 channels, S = 64: 133 us against 165).
template <typename T, int SP, bool ALL>
__global__ __launch_bounds__(kScanThreads, SP <= 16 ? 4 : 2) void scan_first_kernel(ScanArgs a, ScanPlan pl) {
    const unsigned id = wave_id();
    const int nblk = a.G * ((a.D / a.G + 63) / 64);
    const unsigned one = static_cast<unsigned>(nblk) * a.B, forward = one * pl.nseg;
    if (id < forward)
        keep_states<T, SP, ALL>(a, pl, nblk, id);
    else if (id - forward < one * (pl.nseg - 1))
        walk_back<T, SP, ALL>(a, pl, nblk, id - forward);
}

// Entry states (in place of the end states) and, behind each segment, the adjoint (in place
// of the one that it lets out of its front).
template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void scan_compose_both_kernel(ScanArgs a, ScanPlan pl) {
    __shared__ ComposeSums<WAVES> sums;
    const size_t ds = static_cast<size_t>(a.D) * a.S, id = static_cast<size_t>(blockIdx.x) * 64 + (threadIdx.x & 63);
    // The last workgroup's idle lanes walk no segment: the walk is in place, and a pair has one owner.
    const bool live = id < ds * a.B;
    const size_t in = live ? id : 0;
    const int nseg = live ? pl.nseg : 0;
    const size_t b = in / ds, e = in % ds;
    const float A2 = a.A[e] * kLog2e;
    const float* sum = a.workspace + pl.off_dt + b * pl.nseg * a.D + e / a.S;
    compose<WAVES, false>(a.workspace + pl.off_end + b * pl.nseg * ds + e, sum, ds, a.D, nseg, A2,
                          a.state_in != nullptr ? a.state_in[in] : 0.f, sums);
    __syncthreads();
    compose<WAVES, true>(a.workspace + pl.off_rev + b * pl.nseg * ds + e, sum, ds, a.D, nseg, A2,
                         a.gstate_out != nullptr ? a.gstate_out[in] : 0.f, sums);
}

// Lanes of the main pass: LPC adjacent lanes hold one channel's states.  With LPC = 4 the state
// group of a lane is its number's low two bits, flipped in odd channels: then lane ^ 7, which
// one DPP instruction reaches, is the neighbouring channel's lane of the same state group.
template <int LPC>
__device__ __forceinline__ int state_group(int lane) {
    const int q = lane & (LPC - 1);
    return LPC == 4 ? q ^ ((lane & 4) ? 3 : 0) : q;
}
// The sum over a channel's LPC lanes, in each of them.
template <int LPC>
__device__ __forceinline__ float state_sum(float x) {
    x += lane_xor<1>(x);
    x += lane_xor<2>(x);
    if (LPC >= 8) x += lane_xor<7>(x);
    if (LPC >= 16) x += lane_xor<8>(x);
    return x;
}
// Sums over a wave's channels (the lanes that share a state group) for four tokens, in steps:
// tokens 3 and 2 and tokens 1 and 0 are summed over the two halves of the wave as soon as
// both are there (pair), then all over rows of 16 and down to the channels' last bits (join).
// Afterwards a lane holds token 2 b4 + b5 (its number's bits), and of the SPL states with 16
// (8, 4) channels a wave: state 2 b3 + b2 (2 b3 and the one behind it, all).
__device__ __forceinline__ void channel_pair(const float (&lo)[SPL], const float (&hi)[SPL], float (&r)[SPL]) {
#pragma unroll
    for (int i = 0; i < SPL; ++i) r[i] = halves_sum32(lo[i], hi[i]);
}
template <int LPC>
__device__ __forceinline__ void channel_join(const float (&lo)[SPL], const float (&hi)[SPL], float (&out)[LPC / 4]) {
    float r[SPL];
#pragma unroll
    for (int i = 0; i < SPL; ++i) r[i] = halves_sum16(lo[i], hi[i]);
    if (LPC == 16) {
#pragma unroll
        for (int i = 0; i < LPC / 4; ++i) out[i] = r[i & 3];
        return;
    }
    const float s0 = pair_sum8(r[0], r[2]), s1 = pair_sum8(r[1], r[3]);
    if (LPC == 8) {
        out[0] = s0;
        out[LPC / 4 - 1] = s1;
    } else {
        out[0] = pair_sum7(s0, s1);
    }
}

// B and C of a tile's tokens, [kTile][SP] in LDS, zeros behind the last state and token.
template <typename T, int SP>
struct StateRows {
    static constexpr int kPer = kTile * SP / kScanThreads;
    T raw[kPer];
    // (what lies behind is read from the last token or state there is, and not used)
    __device__ __forceinline__ void load(const T* p, long long ld, int rows, int S, int tid) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = tid + k * kScanThreads, t = i / SP, n = i % SP;
            const uint32_t at = static_cast<uint32_t>(t < rows ? t : rows - 1) * static_cast<uint32_t>(ld) + (n < S ? n : S - 1);
            raw[k] = row_at(p, at * static_cast<uint32_t>(sizeof(T)));
        }
    }
    __device__ __forceinline__ void store(float* lds, int rows, int S, int tid) const {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = tid + k * kScanThreads;
            lds[i] = i / SP < rows && i % SP < S ? up(raw[k]) : 0.f;
        }
    }
};

// What was read from LDS before is read again behind this point: kept in registers over the
// parts of a tile it would crowd out the states.
__device__ __forceinline__ void reload() { asm volatile("" ::: "memory"); }

// A pack at a byte offset from an address that is the same for the whole workgroup; `left` of
// its elements are there.
template <typename T, bool WHOLE>
__device__ __forceinline__ Raw<T, 4> pack_at(const T* base, uint32_t byte, int left) {
    return raw_load_n<T, 4>(reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + byte), WHOLE ? 4 : left);
}
template <typename T, bool WHOLE>
__device__ __forceinline__ void pack_put(T* base, uint32_t byte, const float (&v)[4], int left, bool stream = false) {
    store_n<T, 4>(reinterpret_cast<T*>(reinterpret_cast<char*>(base) + byte), v, WHOLE ? 4 : left, stream);
}

// WHOLE: a group's channels and the states are multiples of 4, so that every pack is whole.
// Idle threads then repeat the loads of others and drop them, which keeps the loads free of
// branches.
template <typename T, int LPC, bool WHOLE>
__global__ __launch_bounds__(kScanThreads, LPC == 16 || (LPC == 4 && sizeof(T) == 4) ? 2 : 3)   // what LDS allows
    void scan_bwd_kernel(ScanArgs a, ScanPlan pl) {
    constexpr int CH = kScanThreads / LPC, SP = LPC * SPL, CQ = CH / 4, KEPT = LPC / 4, ES = sizeof(T);
    constexpr int PACKS = kTile * CQ;     // packs of 4 channels of a tile: one a thread at most
    static_assert(PACKS <= kScanThreads && kPart == 4, "one pack a thread, parts of four tokens");
    __shared__ float sdt[kTile][CH], su[kTile][CH], sg[kTile][CH], sdu[kTile][CH], sda[kTile][CH], sy[kTile][CH];
    __shared__ __attribute__((aligned(16))) float sB[kTile * SP], sC[kTile * SP];
    __shared__ float rB[4][kTile * SP], rC[4][kTile * SP];   // each wave's sums over its channels
    __shared__ Raw<T, 4> sx[PACKS], sraw[PACKS], sz[PACKS], sgy[PACKS];   // x, dt, z, gy as they came
    __shared__ float sbias[CH], sskip[CH];
    __shared__ f32v4 sgD[PACKS], sgbias[PACKS];               // each pack's sums over tokens
    const int tid = threadIdx.x, lane = tid & 63;
    const ScanPlace p = scan_place<CH>(a, pl.nblk, pl.nseg, pl.seg, blockIdx.x);
    const int cl = tid / LPC, n0 = state_group<LPC>(lane) * SPL;
    const size_t slot = ((static_cast<size_t>(p.b) * pl.nseg + p.seg) * a.D + p.c0) * a.S;
    const size_t bd = (static_cast<size_t>(p.b) * a.D + p.c0) * a.S;
    const int tiles = (a.N + kTile - 1) / kTile;
    // a lane's SPL of a channel's S states, from the block's first channel
    struct Lane {
        int cl, n0, left;          // channel of the block, first state, states from it on (<= 0: none)
        uint32_t at;               // byte offset in the block's states
    };
    auto lane_place = [&]() {
        const int id = static_cast<int>(opaque(tid)), c = id / LPC, n = state_group<LPC>(id) * SPL;
        return Lane{c, n, p.c0 + c < p.cend ? a.S - n : 0, (static_cast<uint32_t>(c) * a.S + n) * 4};
    };
    auto load_lane = [&](const float* s, float (&v)[SPL]) {
        const Lane l = lane_place();
        const Raw<float, SPL> r = pack_at<float, WHOLE>(s, l.left > 0 ? l.at : 0, l.left);
#pragma unroll
        for (int i = 0; i < SPL; ++i) v[i] = l.left > 0 ? r.v[i] : 0.f;
    };
    float A2[SPL], w[SPL] = {}, gA[SPL] = {};
    load_lane(a.A + static_cast<size_t>(p.c0) * a.S, A2);
#pragma unroll
    for (int i = 0; i < SPL; ++i) A2[i] *= kLog2e;
    const float* entry = pl.nseg > 1 ? a.workspace + pl.off_end + slot : a.state_in != nullptr ? a.state_in + bd : nullptr;
    const float* last = pl.nseg > 1 ? a.workspace + pl.off_rev + slot : a.gstate_out != nullptr ? a.gstate_out + bd : nullptr;
    if (last != nullptr) load_lane(last, w);
    // This thread's pack of 4 channels of a tile's row: worked out again wherever it is used
    // (`opaque`), since what is derived from it would otherwise sit in registers throughout.
    struct Pack {
        int id, ur, cq, left;      // left: channels from the pack's first one on, <= 0: idle
        __device__ __forceinline__ uint32_t off(long long ld) const {     // byte offset in the tile, rows ld apart
            return (static_cast<uint32_t>(ur) * static_cast<uint32_t>(ld) + 4 * cq) * ES;
        }
        __device__ __forceinline__ uint32_t from(long long ld, int rows) const {   // the same, of a pack that is there
            const int r = ur < rows ? ur : 0, c = left > 0 ? 4 * cq : 0;
            return (static_cast<uint32_t>(r) * static_cast<uint32_t>(ld) + c) * ES;
        }
    };
    auto pack = [&]() {
        const int id = static_cast<int>(opaque(tid)), ur = id / CQ, cq = id % CQ;
        return Pack{id, ur, cq, ur < kTile ? p.cend - p.c0 - 4 * cq : 0};
    };
    if (tid < PACKS) sgD[tid] = sgbias[tid] = f32v4{0.f, 0.f, 0.f, 0.f};
    if (tid < CH) {
        const bool in = p.c0 + tid < p.cend;
        sbias[tid] = in && a.bias != nullptr ? a.bias[p.c0 + tid] : 0.f;
        sskip[tid] = in && a.Dskip != nullptr ? a.Dskip[p.c0 + tid] : 0.f;
    }
    const size_t tok0 = static_cast<size_t>(p.b) * a.N;
    const T* const gy = static_cast<const T*>(a.gy) + p.c0;
    T* const gx = static_cast<T*>(a.gx) + p.c0;
    T* const gdt = static_cast<T*>(a.gdt) + p.c0;
    T* const gz = static_cast<T*>(a.gz) + p.c0;
    // gradient rows behind the sequence's last token are zero
    const int behind = p.t_end > p.t_begin ? p.t_end : p.t_begin;
    for (int t0 = behind; t0 < p.t_full; t0 += kTile) {
        const float zero[4] = {};
        const size_t at = (tok0 + t0) * a.D;
        const Pack k = pack();
        if (t0 + k.ur >= p.t_full || k.left <= 0) continue;
        pack_put<T, WHOLE>(gx + at, k.off(a.D), zero, k.left);
        pack_put<T, WHOLE>(gdt + at, k.off(a.D), zero, k.left);
        if (a.gz != nullptr) pack_put<T, WHOLE>(gz + at, k.off(a.D), zero, k.left);
    }
    const size_t tokens = static_cast<size_t>(a.B) * a.N;   // partial sums [2][block][B N][S]
    float* const pB = a.workspace + pl.off_bc + (static_cast<size_t>(p.blk) * tokens + tok0) * a.S;
    float* const pC = pB + static_cast<size_t>(pl.nblk) * tokens * a.S;
    for (size_t e = static_cast<size_t>(behind) * a.S + tid; e < static_cast<size_t>(p.t_full) * a.S; e += kScanThreads)
        pB[e] = pC[e] = 0.f;

    Raw<T, 4> rx = {}, rdt = {}, rz = {}, rg = {};
    StateRows<T, SP> nB, nC;
    float kept[SPL], cum;
    const int ntile = p.t_end > p.t_begin ? (p.t_end - p.t_begin + kTile - 1) / kTile : 0;
    auto fetch = [&](int t0) {
        const int rows = p.t_end - t0;
        const size_t t = tok0 + t0;
        const Pack k = pack();
        if (WHOLE || (k.ur < rows && k.left > 0)) {
            rx = pack_at<T, WHOLE>(static_cast<const T*>(a.x) + t * a.ldx + p.c0, k.from(a.ldx, rows), k.left);
            rdt = pack_at<T, WHOLE>(static_cast<const T*>(a.dt) + t * a.lddt + p.c0, k.from(a.lddt, rows), k.left);
            if (a.z != nullptr)
                rz = pack_at<T, WHOLE>(static_cast<const T*>(a.z) + t * a.ldz + p.c0, k.from(a.ldz, rows), k.left);
            rg = pack_at<T, WHOLE>(gy + t * a.D, k.from(a.D, rows), k.left);
        }
        nB.load(static_cast<const T*>(a.Bm) + t * a.ldb + p.g * a.S, a.ldb, rows, a.S, k.id);
        nC.load(static_cast<const T*>(a.Cm) + t * a.ldc + p.g * a.S, a.ldc, rows, a.S, k.id);
        const size_t at = (static_cast<size_t>(p.b) * tiles + t0 / kTile) * a.D + p.c0;
        load_lane(a.workspace + pl.off_ckpt + at * a.S, kept);
        const Lane l = lane_place();
        cum = (a.workspace + pl.off_cum + at)[l.left > 0 ? l.cl : 0];
    };
    if (ntile > 0) fetch(p.t_begin + (ntile - 1) * kTile);
    __syncthreads();
    for (int tile = ntile - 1; tile >= 0; --tile) {
        const int t0 = p.t_begin + tile * kTile, rows = p.t_end - t0 < kTile ? p.t_end - t0 : kTile;
        // the state in front of the tile: what its segment made of zero, and what entered it
        float h0[SPL];
#pragma unroll
        for (int i = 0; i < SPL; ++i) h0[i] = kept[i];
        if (entry != nullptr) {
            float e[SPL];
            load_lane(entry, e);
#pragma unroll
            for (int i = 0; i < SPL; ++i) h0[i] = carry(cum * A2[i], e[i], h0[i]);
        }
        const Pack k = pack();
        if (k.ur < kTile) {
            f32v4 d, u, g;
            const f32v4 bias = *reinterpret_cast<const f32v4*>(&sbias[4 * k.cq]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float dt = step_size(up(rdt.v[i]) + bias[i], a.softplus);
                const bool there = k.ur < rows && i < k.left;
                float gi = up(rg.v[i]);
                if (a.z != nullptr) {
                    const float z = up(rz.v[i]);
                    gi *= z * sigmoid_f(z);
                }
                d[i] = there ? dt : 0.f;
                u[i] = there ? dt * up(rx.v[i]) : 0.f;
                g[i] = there ? gi : 0.f;
            }
            *reinterpret_cast<f32v4*>(&sdt[k.ur][4 * k.cq]) = d;
            *reinterpret_cast<f32v4*>(&su[k.ur][4 * k.cq]) = u;
            *reinterpret_cast<f32v4*>(&sg[k.ur][4 * k.cq]) = g;
            sx[k.id] = rx;
            sraw[k.id] = rdt;
            sz[k.id] = rz;
            sgy[k.id] = rg;
        }
        nB.store(sB, rows, a.S, k.id);
        nC.store(sC, rows, a.S, k.id);
        __syncthreads();
        if (tile > 0) fetch(t0 - kTile);
        // the states in front of the tile's parts
        float hp[kTile / kPart][SPL];
#pragma unroll
        for (int i = 0; i < SPL; ++i) hp[0][i] = h0[i];
#pragma unroll
        for (int t = 0; t < kTile - kPart; ++t) {
            const float dt = sdt[t][cl], u = su[t][cl];
            const f32v4 Bv = *reinterpret_cast<const f32v4*>(sB + t * SP + n0);
#pragma unroll
            for (int i = 0; i < SPL; ++i) h0[i] = fmaf(exp2_fast(dt * A2[i]), h0[i], u * Bv[i]);
            if (t % kPart == kPart - 1) {
#pragma unroll
                for (int i = 0; i < SPL; ++i) hp[t / kPart + 1][i] = h0[i];
                reload();
            }
        }
        float tA[SPL] = {};
#pragma unroll
        for (int tb = kTile - kPart; tb >= 0; tb -= kPart) {
            // forward through the part: its decays and the states before its tokens stay in
            // registers; y and dC need only what is known here
            const int id = static_cast<int>(opaque(tid)), row = tb + 2 * ((id >> 4) & 1) + ((id >> 5) & 1);
            const int s0 = state_group<LPC>(id) * SPL +
                           (LPC == 16 ? 0 : LPC == 8 ? (id >> 3 & 1) * 2 : (id >> 3 & 1) * 2 + (id >> 2 & 1));
            float da[kPart][SPL], hs[kPart][SPL], v[2][SPL], c[2][SPL], o[KEPT], h[SPL];
#pragma unroll
            for (int i = 0; i < SPL; ++i) h[i] = hp[tb / kPart][i];
#pragma unroll
            for (int t = 0; t < kPart; ++t) {
                const float dt = sdt[tb + t][cl], u = su[tb + t][cl], gt = sg[tb + t][cl];
                const f32v4 Bv = *reinterpret_cast<const f32v4*>(sB + (tb + t) * SP + n0);
                const f32v4 Cv = *reinterpret_cast<const f32v4*>(sC + (tb + t) * SP + n0);
                float y = 0.f;
#pragma unroll
                for (int i = 0; i < SPL; ++i) {
                    hs[t][i] = h[i];
                    da[t][i] = exp2_fast(dt * A2[i]);
                    h[i] = fmaf(da[t][i], h[i], u * Bv[i]);
                    y = fmaf(Cv[i], h[i], y);
                    v[t & 1][i] = gt * h[i];
                }
                y = state_sum<LPC>(y);
                if ((lane & (LPC - 1)) == 0) sy[tb + t][cl] = y;
                if (t & 1) channel_pair(v[0], v[1], c[t / 2]);
            }
            channel_join<LPC>(c[0], c[1], o);
#pragma unroll
            for (int k = 0; k < KEPT; ++k) rC[id >> 6][row * SP + s0 + k] = o[k];
            // and back
            reload();
#pragma unroll
            for (int t = kPart - 1; t >= 0; --t) {
                const float dt = sdt[tb + t][cl], u = su[tb + t][cl], gt = sg[tb + t][cl];
                const f32v4 Bv = *reinterpret_cast<const f32v4*>(sB + (tb + t) * SP + n0);
                const f32v4 Cv = *reinterpret_cast<const f32v4*>(sC + (tb + t) * SP + n0);
                float du = 0.f, dA = 0.f;
#pragma unroll
                for (int i = 0; i < SPL; ++i) {
                    const float adj = fmaf(Cv[i], gt, w[i]);
                    du = fmaf(adj, Bv[i], du);
                    v[t & 1][i] = adj * u;
                    w[i] = adj * da[t][i];
                    const float q = w[i] * hs[t][i];
                    dA = fmaf(A2[i], q, dA);
                    tA[i] = fmaf(dt, q, tA[i]);
                }
                du = state_sum<LPC>(du);
                dA = state_sum<LPC>(dA);
                if ((lane & (LPC - 1)) == 0) {
                    sdu[tb + t][cl] = du;
                    sda[tb + t][cl] = dA;
                }
                if (t % 2 == 0) channel_pair(v[0], v[1], c[t / 2]);
            }
            channel_join<LPC>(c[0], c[1], o);
#pragma unroll
            for (int k = 0; k < KEPT; ++k) rB[id >> 6][row * SP + s0 + k] = o[k];
            reload();
        }
#pragma unroll
        for (int i = 0; i < SPL; ++i) gA[i] += tA[i];
        __syncthreads();
        const Pack k2 = pack();
        for (int e = k2.id; e < rows * SP; e += kScanThreads) {
            const int t = e / SP, s = e % SP;
            if (s >= a.S) continue;
            float* const rowB = pB + static_cast<size_t>(t0) * a.S;
            float* const rowC = pC + static_cast<size_t>(t0) * a.S;
            const uint32_t at = static_cast<uint32_t>(t * a.S + s);
            rowB[at] = (rB[0][e] + rB[1][e]) + (rB[2][e] + rB[3][e]);
            rowC[at] = (rC[0][e] + rC[1][e]) + (rC[2][e] + rC[3][e]);
        }
        if (k2.ur < rows && k2.left > 0) {
            const f32v4 du = *reinterpret_cast<const f32v4*>(&sdu[k2.ur][4 * k2.cq]);
            const f32v4 dA = *reinterpret_cast<const f32v4*>(&sda[k2.ur][4 * k2.cq]);
            const f32v4 ys = *reinterpret_cast<const f32v4*>(&sy[k2.ur][4 * k2.cq]);
            const f32v4 d = *reinterpret_cast<const f32v4*>(&sdt[k2.ur][4 * k2.cq]);
            const f32v4 g = *reinterpret_cast<const f32v4*>(&sg[k2.ur][4 * k2.cq]);
            const f32v4 bias = *reinterpret_cast<const f32v4*>(&sbias[4 * k2.cq]);
            const f32v4 skip = *reinterpret_cast<const f32v4*>(&sskip[4 * k2.cq]);
            const Raw<T, 4> cx = sx[k2.id], cdt = sraw[k2.id], cz = sz[k2.id], cg = sgy[k2.id];
            f32v4 gD = sgD[k2.id], gbias = sgbias[k2.id];
            float ox[4], odt[4], oz[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = up(cx.v[i]);
                ox[i] = fmaf(du[i], d[i], g[i] * skip[i]);
                odt[i] = fmaf(du[i], x, dA[i] * (1.f / kLog2e));     // summed with A log2(e)
                if (a.softplus) odt[i] *= sigmoid_f(up(cdt.v[i]) + bias[i]);
                gD[i] = fmaf(g[i], x, gD[i]);
                gbias[i] += odt[i];
                if (a.z != nullptr) {
                    const float z = up(cz.v[i]), s = sigmoid_f(z);
                    oz[i] = up(cg.v[i]) * fmaf(skip[i], x, ys[i]) * fmaf(z * s, 1.f - s, s);
                }
            }
            sgD[k2.id] = gD;
            sgbias[k2.id] = gbias;
            const size_t at = (tok0 + t0) * a.D;
            pack_put<T, WHOLE>(gx + at, k2.off(a.D), ox, k2.left, a.stream);
            pack_put<T, WHOLE>(gdt + at, k2.off(a.D), odt, k2.left, a.stream);
            if (a.gz != nullptr) pack_put<T, WHOLE>(gz + at, k2.off(a.D), oz, k2.left, a.stream);
        }
    }
    // [B nseg][S + 2][D] partial sums of the parameters' gradients
    float* const par = a.workspace + pl.off_par + static_cast<size_t>(blockIdx.x / pl.nblk) * (a.S + 2) * a.D;
    const Lane l = lane_place();
    if (l.left > 0) {
#pragma unroll
        for (int i = 0; i < SPL; ++i)
            if (i < l.left) par[static_cast<size_t>(l.n0 + i) * a.D + p.c0 + l.cl] = gA[i];
        if (p.seg == 0 && a.gstate_in != nullptr) pack_put<float, WHOLE>(a.gstate_in + bd, l.at, w, l.left);
    }
    __syncthreads();
    if (tid < CH && p.c0 + tid < p.cend) {
        float s = 0.f, b = 0.f;
#pragma unroll
        for (int r = 0; r < kTile; ++r) {
            s += sgD[r * CQ + tid / 4][tid % 4];
            b += sgbias[r * CQ + tid / 4][tid % 4];
        }
        par[static_cast<size_t>(a.S) * a.D + p.c0 + tid] = s;
        par[static_cast<size_t>(a.S + 1) * a.D + p.c0 + tid] = b;
    }
}

// dB and dC [B, N, G, S]: the sums over a group's channel blocks, in order.
template <typename T>
__global__ __launch_bounds__(kScanThreads) void scan_bc_kernel(ScanArgs a, ScanPlan pl) {
    const size_t tokens = static_cast<size_t>(a.B) * a.N, one = tokens * a.G * a.S;
    const size_t id = static_cast<size_t>(blockIdx.x) * kScanThreads + threadIdx.x;
    if (id >= 2 * one) return;
    const size_t e = id < one ? id : id - one, s = e % a.S, g = e / a.S % a.G, tok = e / a.S / a.G;
    const int per = pl.nblk / a.G;
    const float* in = a.workspace + pl.off_bc + ((id < one ? 0 : pl.nblk) + g * per) * tokens * a.S + tok * a.S + s;
    float t = 0.f;
#pragma unroll 8
    for (int k = 0; k < per; ++k) t += in[k * tokens * a.S];
    static_cast<T*>(id < one ? a.gB : a.gC)[e] = down<T>(t);
}

template <typename T, int SP>
hipError_t first_passes(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
    const dim3 block(kScanThreads);
    constexpr unsigned wpg = kScanThreads / 64;
    const unsigned waves = static_cast<unsigned>(a.G * ((a.D / a.G + 63) / 64)) * a.B;
    ProfScope prof(kProfScanPre, st);
    const dim3 grid((waves * (2 * p.nseg - 1) + wpg - 1) / wpg);
    if (a.S == SP)
        hipLaunchKernelGGL((scan_first_kernel<T, SP, true>), grid, block, 0, st, a, p);
    else
        hipLaunchKernelGGL((scan_first_kernel<T, SP, false>), grid, block, 0, st, a, p);
    if (p.nseg > 1) {
        const size_t n = static_cast<size_t>(a.B) * a.D * a.S;
        const int waves = compose_waves(p.nseg, n);
        hipLaunchKernelGGL(waves > 1 ? scan_compose_both_kernel<kComposeWaves> : scan_compose_both_kernel<1>,
                           dim3(static_cast<unsigned>((n + 63) / 64)), dim3(64 * waves), 0, st, a, p);
    }
    return hipGetLastError();
}

template <typename T, int SP>
hipError_t bwd_states(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
    constexpr int LPC = SP <= 16 ? 4 : SP / 4;
    const dim3 block(kScanThreads);
    const unsigned wgs = static_cast<unsigned>(p.nblk) * a.B;
    if (wgs > 0) {
        hipError_t e = first_passes<T, SP>(a, p, st);
        if (e != hipSuccess) return e;
        {
            ProfScope prof(kProfSelScan, st);
            if (a.D / a.G % 4 == 0 && a.S % 4 == 0)
                hipLaunchKernelGGL((scan_bwd_kernel<T, LPC, true>), dim3(wgs * p.nseg), block, 0, st, a, p);
            else
                hipLaunchKernelGGL((scan_bwd_kernel<T, LPC, false>), dim3(wgs * p.nseg), block, 0, st, a, p);
        }
        const size_t n = 2 * static_cast<size_t>(a.B) * a.N * a.G * a.S;
        if (n > 0) {
            ProfScope prof(kProfReduce, st);
            hipLaunchKernelGGL((scan_bc_kernel<T>), dim3(static_cast<unsigned>((n + kScanThreads - 1) / kScanThreads)), block,
                               0, st, a, p);
        }
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const ColReduceArgs c{a.workspace + p.off_par, a.B * p.nseg, a.S + 2, a.S, a.D, a.gA, a.gD, a.gbias, false};
    return launch_col_reduce(c, st);
}

template <typename T>
hipError_t bwd_typed(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
    if (a.S <= 16) return bwd_states<T, 16>(a, p, st);
    return a.S <= 32 ? bwd_states<T, 32>(a, p, st) : bwd_states<T, 64>(a, p, st);
}

}  // namespace

ScanPlan scan_bwd_plan(int B, int N, int D, int G, int S) {
    ScanPlan p{};
    const int ch = S <= 16 ? 64 : S <= 32 ? 32 : 16;       // channels of a workgroup of the main pass
    p.nblk = G * ((D / G + ch - 1) / ch);
    // Segments: as many as bring the chip two waves of either first pass a SIMD, of a tile at
    // least.
    const size_t waves = static_cast<size_t>(G) * ((D / G + 63) / 64) * (B > 0 ? B : 1);
    const int most = N / kTile > 1 ? N / kTile : 1;
    int want = waves >= 2048 ? 1 : static_cast<int>((kWantWaves + waves - 1) / waves);
    if (want > most) want = most;
    const int steps = (N + kTile - 1) / kTile, per = (steps + want - 1) / want;
    p.seg = per > 0 ? per * kTile : kTile;
    p.nseg = N > 0 ? (N - 1) / p.seg + 1 : 1;
    const size_t bs = static_cast<size_t>(B) * p.nseg * D, tiles = (static_cast<size_t>(N) + kTile - 1) / kTile;
    size_t at = 0;
    auto take = [&](size_t floats) {
        const size_t here = at;
        at += (floats + 3) / 4 * 4;
        return here;
    };
    p.off_end = take(p.nseg > 1 ? bs * S : 0);
    p.off_rev = take(p.nseg > 1 ? bs * S : 0);
    p.off_dt = take(p.nseg > 1 ? bs : 0);
    p.off_ckpt = take(B * tiles * D * S);
    p.off_cum = take(B * tiles * D);
    p.off_bc = take(2 * static_cast<size_t>(p.nblk) * B * N * S);
    p.off_par = take(static_cast<size_t>(B) * p.nseg * (S + 2) * D);
    p.total = at;
    return p;
}

hipError_t launch_scan_bwd(const ScanArgs& args, const ScanPlan& p, hipStream_t st) {
    ScanArgs a = args;
    a.stream = static_cast<size_t>(a.B) * a.N * a.D * (a.bf16 ? 2 : 4) >= kStreamBytes;
    return a.bf16 ? bwd_typed<bf16_t>(a, p, st) : bwd_typed<float>(a, p, st);
}

}  // namespace retn
