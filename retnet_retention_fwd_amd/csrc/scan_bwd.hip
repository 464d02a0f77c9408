// Backward of the selective scan.  With g_t = gy_t silu(z_t) and the adjoint state
//     w_t = C_t g_t + exp(dt_(t+1) A) w_(t+1)   (+ grad_state_out behind the last token),
// the gradients are
//     du_t = sum_n w_t B_t,   q_t[n] = w_t h_(t-1) exp(dt_t A),
//     dx = du dt + D g,       ddt = du x + sum_n q A  (times sigmoid(raw + bias)),
//     dA = sum_t q dt,        dB_t = sum_channels w dt x,   dC_t = sum_channels g h_t,
//     dD = sum g x,           dz = gy (C.h + D x) silu'(z).
//
// Bound by the vector ALUs, like the forward.  A first pass walks forward and keeps the
// state in front of every 16th token; the main pass takes tiles of 16 tokens from the last
// to the first, recomputes the tile's states and decays into registers and walks back
// through them.  So no state but one in 16 is ever in memory and an exponential is taken
// twice per (token, channel, state) in all.  dB and dC sum over channels: over a wave's in
// registers (two instructions a value, scan.h), over a workgroup's in LDS, over workgroups
// by a second kernel in a fixed order; the parameters' sums over tokens stay in registers
// until the end of a segment.
//
// Segments, where channels are few: the first pass walks each from a zero state, a second
// one walks the adjoint back through each from zero, and a small kernel composes both into
// the states that enter the segments from either side.

#include "scan.h"

namespace retn {

namespace {

constexpr int kTile = 16;      // tokens of a tile, and between kept states
constexpr int SPL = 4;

// The state in front of each tile, its segment walked from zero, and the sum of dt from the
// segment's first token to there; the end state and whole sum of dt go to the segment's slot.
template <typename T, int LPC>
__global__ __launch_bounds__(kScanThreads) void scan_keep_kernel(ScanArgs a, ScanPlan pl) {
    constexpr int CH = kScanThreads / LPC, SP = LPC * SPL, CQ = CH / 4, TT = 2 * kTile;
    constexpr int UNITS = TT * CQ, NU = (UNITS + kScanThreads - 1) / kScanThreads;
    __shared__ float sdt[TT][CH], su[TT][CH];
    __shared__ __attribute__((aligned(16))) float sB[TT * SP];
    const int tid = threadIdx.x, lane = tid & 63;
    const ScanPlace p = scan_place<CH>(a, pl.nblk, pl.nseg, blockIdx.x);
    const int n = scan_length(a.lengths, p.b, a.N);
    const int t_begin = p.seg * pl.seg, t_full = t_begin + pl.seg < a.N ? t_begin + pl.seg : a.N;
    const int t_end = t_full < n ? t_full : n;
    const int cl = tid / LPC, ch = p.c0 + cl, n0 = state_group<LPC>(lane) * SPL;
    const bool on = ch < p.cend;
    float A2[SPL], h[SPL], dsum = 0.f;
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        A2[i] = on && n0 + i < a.S ? a.A[static_cast<size_t>(ch) * a.S + n0 + i] * kLog2e : 0.f;
        h[i] = 0.f;
    }
    const size_t slot = (static_cast<size_t>(p.b) * pl.nseg + p.seg) * a.D + ch;
    const int tiles = (a.N + kTile - 1) / kTile;
    const int cq = tid % CQ, uc = p.c0 + 4 * cq, left = p.cend - uc;
    float bias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[i] = a.bias != nullptr && i < left ? a.bias[uc + i] : 0.f;
    Raw<T, 4> rx[NU], rdt[NU];
    StateRows<T, TT, SP> rB;
    const size_t tok0 = static_cast<size_t>(p.b) * a.N;
    auto fetch = [&](int t0) {
        const int rows = t_end - t0;
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            const int r = (tid + k * kScanThreads) / CQ;
            rx[k] = rdt[k] = Raw<T, 4>{};
            if (r < rows && r < TT && left > 0) {
                const size_t t = tok0 + t0 + r;
                rx[k] = raw_load_n<T, 4>(static_cast<const T*>(a.x) + t * a.ldx + uc, left);
                rdt[k] = raw_load_n<T, 4>(static_cast<const T*>(a.dt) + t * a.lddt + uc, left);
            }
        }
        rB.load(static_cast<const T*>(a.Bm) + (tok0 + t0) * a.ldb + p.g * a.S, a.ldb, rows, a.S);
    };
    auto keep = [&](int t) {
        if (!on) return;
        const size_t at = (static_cast<size_t>(p.b) * tiles + t / kTile) * a.D + ch;
        store_state<SPL>(a.workspace + pl.off_ckpt + at * a.S, n0, a.S, h);
        if (n0 == 0) a.workspace[pl.off_cum + at] = dsum;
    };
    if (t_begin < t_end) fetch(t_begin);
    for (int t0 = t_begin; t0 < t_end; t0 += TT) {
        const int rows = t_end - t0 < TT ? t_end - t0 : TT;
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            const int r = (tid + k * kScanThreads) / CQ;
            if (UNITS % kScanThreads == 0 || r < TT) {
                f32v4 d, u;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    d[i] = r < rows ? step_size(up(rdt[k].v[i]) + bias[i], a.softplus) : 0.f;
                    u[i] = d[i] * up(rx[k].v[i]);
                }
                *reinterpret_cast<f32v4*>(&sdt[r][4 * cq]) = d;
                *reinterpret_cast<f32v4*>(&su[r][4 * cq]) = u;
            }
        }
        rB.store(sB);
        __syncthreads();
        if (t0 + TT < t_end) fetch(t0 + TT);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (t0 + half * kTile >= t_end) break;
            keep(t0 + half * kTile);
#pragma unroll
            for (int j = 0; j < kTile; ++j) {
                const int t = half * kTile + j;
                const float dt = sdt[t][cl], u = su[t][cl];
                float Bv[SPL];
                lds_states<SPL>(sB + t * SP + n0, Bv);
                dsum += dt;
#pragma unroll
                for (int i = 0; i < SPL; ++i) h[i] = fmaf(exp2_fast(dt * A2[i]), h[i], u * Bv[i]);
            }
        }
        __syncthreads();
    }
    if (!on || pl.nseg == 1) return;
    store_state<SPL>(a.workspace + pl.off_end + slot * a.S, n0, a.S, h);
    if (n0 == 0) a.workspace[pl.off_dt + slot] = dsum;
}

// The adjoint that leaves each segment but the first at its front, from zero behind its end.
template <typename T, int LPC>
__global__ __launch_bounds__(kScanThreads) void scan_rev_kernel(ScanArgs a, ScanPlan pl) {
    constexpr int CH = kScanThreads / LPC, SP = LPC * SPL, CQ = CH / 4, TT = 2 * kTile;
    constexpr int UNITS = TT * CQ, NU = (UNITS + kScanThreads - 1) / kScanThreads;
    __shared__ float sdt[TT][CH], sg[TT][CH];
    __shared__ __attribute__((aligned(16))) float sC[TT * SP];
    const int tid = threadIdx.x, lane = tid & 63;
    ScanPlace p = scan_place<CH>(a, pl.nblk, pl.nseg - 1, blockIdx.x);
    p.seg += 1;
    const int n = scan_length(a.lengths, p.b, a.N);
    const int t_begin = p.seg * pl.seg, t_full = t_begin + pl.seg < a.N ? t_begin + pl.seg : a.N;
    const int t_end = t_full < n ? t_full : n;
    const int cl = tid / LPC, ch = p.c0 + cl, n0 = state_group<LPC>(lane) * SPL;
    const bool on = ch < p.cend;
    float A2[SPL], w[SPL];
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        A2[i] = on && n0 + i < a.S ? a.A[static_cast<size_t>(ch) * a.S + n0 + i] * kLog2e : 0.f;
        w[i] = 0.f;
    }
    const int cq = tid % CQ, uc = p.c0 + 4 * cq, left = p.cend - uc;
    float bias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[i] = a.bias != nullptr && i < left ? a.bias[uc + i] : 0.f;
    Raw<T, 4> rdt[NU], rz[NU], rg[NU];
    StateRows<T, TT, SP> rC;
    const size_t tok0 = static_cast<size_t>(p.b) * a.N;
    const int ntile = t_end > t_begin ? (t_end - t_begin + TT - 1) / TT : 0;
    auto fetch = [&](int t0) {
        const int rows = t_end - t0;
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            const int r = (tid + k * kScanThreads) / CQ;
            rdt[k] = rz[k] = rg[k] = Raw<T, 4>{};
            if (r < rows && r < TT && left > 0) {
                const size_t t = tok0 + t0 + r;
                rdt[k] = raw_load_n<T, 4>(static_cast<const T*>(a.dt) + t * a.lddt + uc, left);
                if (a.z != nullptr) rz[k] = raw_load_n<T, 4>(static_cast<const T*>(a.z) + t * a.ldz + uc, left);
                rg[k] = raw_load_n<T, 4>(static_cast<const T*>(a.gy) + t * a.D + uc, left);
            }
        }
        rC.load(static_cast<const T*>(a.Cm) + (tok0 + t0) * a.ldc + p.g * a.S, a.ldc, rows, a.S);
    };
    if (ntile > 0) fetch(t_begin + (ntile - 1) * TT);
    for (int tile = ntile - 1; tile >= 0; --tile) {
        const int t0 = t_begin + tile * TT, rows = t_end - t0 < TT ? t_end - t0 : TT;
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            const int r = (tid + k * kScanThreads) / CQ;
            if (UNITS % kScanThreads == 0 || r < TT) {
                f32v4 d, g;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    d[i] = r < rows ? step_size(up(rdt[k].v[i]) + bias[i], a.softplus) : 0.f;
                    g[i] = up(rg[k].v[i]);
                    if (a.z != nullptr) {
                        const float z = up(rz[k].v[i]);
                        g[i] *= z * sigmoid_f(z);
                    }
                }
                *reinterpret_cast<f32v4*>(&sdt[r][4 * cq]) = d;
                *reinterpret_cast<f32v4*>(&sg[r][4 * cq]) = g;
            }
        }
        rC.store(sC);
        __syncthreads();
        if (tile > 0) fetch(t0 - TT);
#pragma unroll
        for (int t = TT - 1; t >= 0; --t) {
            const float dt = sdt[t][cl], g = sg[t][cl];
            float Cv[SPL];
            lds_states<SPL>(sC + t * SP + n0, Cv);
#pragma unroll
            for (int i = 0; i < SPL; ++i) w[i] = exp2_fast(dt * A2[i]) * fmaf(Cv[i], g, w[i]);
        }
        __syncthreads();
    }
    if (!on) return;
    const size_t slot = (static_cast<size_t>(p.b) * pl.nseg + p.seg) * a.D + ch;
    store_state<SPL>(a.workspace + pl.off_rev + slot * a.S, n0, a.S, w);
}

// Entry states (in place of the end states) and, behind each segment, the adjoint (in place
// of the one that the next segment lets out of its front).
__global__ __launch_bounds__(kScanThreads) void scan_compose_both_kernel(ScanArgs a, ScanPlan pl) {
    const size_t ds = static_cast<size_t>(a.D) * a.S, id = static_cast<size_t>(blockIdx.x) * kScanThreads + threadIdx.x;
    if (id >= ds * a.B) return;
    const size_t b = id / ds, e = id % ds;
    const float A2 = a.A[e] * kLog2e;
    float* end = a.workspace + pl.off_end + b * pl.nseg * ds + e;
    float* rev = a.workspace + pl.off_rev + b * pl.nseg * ds + e;
    const float* sum = a.workspace + pl.off_dt + b * pl.nseg * a.D + e / a.S;
    float h = a.state_in != nullptr ? a.state_in[id] : 0.f;
    for (int s = 0; s < pl.nseg; ++s) {
        const float own = end[s * ds];
        end[s * ds] = h;
        h = fmaf(exp2_fast(A2 * sum[static_cast<size_t>(s) * a.D]), h, own);
    }
    float w = a.gstate_out != nullptr ? a.gstate_out[id] : 0.f;
    for (int s = pl.nseg - 1; s >= 0; --s) {
        const float own = s > 0 ? rev[s * ds] : 0.f;
        rev[s * ds] = w;
        w = fmaf(exp2_fast(A2 * sum[static_cast<size_t>(s) * a.D]), w, own);
    }
}

// Sums over a wave's channels (the lanes that share a state group) of v[token][state] for
// four tokens; afterwards a lane holds token 2 b5 + b4 (its number's bits), and of the SPL
// states with 16 (8, 4) channels a wave: state 2 b3 + b2 (2 b3 and the one behind it, all).
template <int LPC>
__device__ __forceinline__ void channel_sum(const float (&v)[4][SPL], int lane, float (&out)[LPC / 4]) {
    float r[SPL];
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        const float lo = halves_sum32(v[0][i], v[2][i]), hi = halves_sum32(v[1][i], v[3][i]);
        r[i] = halves_sum16(lo, hi);
    }
    if (LPC == 16) {
#pragma unroll
        for (int i = 0; i < LPC / 4; ++i) out[i] = r[i & 3];
        return;
    }
    const float s0 = pair_sum<8>(r[0], r[2], lane & 8), s1 = pair_sum<8>(r[1], r[3], lane & 8);
    if (LPC == 8) {
        out[0] = s0;
        out[LPC / 4 - 1] = s1;
    } else {
        out[0] = pair_sum<7>(s0, s1, lane & 4);
    }
}

template <typename T, int LPC>
__global__ __launch_bounds__(kScanThreads, 2) void scan_bwd_kernel(ScanArgs a, ScanPlan pl) {
    constexpr int CH = kScanThreads / LPC, SP = LPC * SPL, CQ = CH / 4, KEPT = LPC / 4;
    constexpr int UNITS = kTile * CQ;     // packs of 4 channels of a tile: one a thread at most
    static_assert(UNITS <= kScanThreads, "one pack a thread");
    __shared__ float sdt[kTile][CH], su[kTile][CH], sg[kTile][CH], sdu[kTile][CH], sda[kTile][CH], sy[kTile][CH];
    __shared__ __attribute__((aligned(16))) float sB[kTile * SP], sC[kTile * SP];
    __shared__ float rB[4][kTile * SP], rC[4][kTile * SP];   // each wave's sums over its channels
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const ScanPlace p = scan_place<CH>(a, pl.nblk, pl.nseg, blockIdx.x);
    const int n = scan_length(a.lengths, p.b, a.N);
    const int t_begin = p.seg * pl.seg, t_full = t_begin + pl.seg < a.N ? t_begin + pl.seg : a.N;
    const int t_end = t_full < n ? t_full : n;
    const int cl = tid / LPC, ch = p.c0 + cl, n0 = state_group<LPC>(lane) * SPL;
    const bool on = ch < p.cend;
    const size_t slot = (static_cast<size_t>(p.b) * pl.nseg + p.seg) * a.D + ch;
    const size_t bd = static_cast<size_t>(p.b) * a.D + ch;
    const int tiles = (a.N + kTile - 1) / kTile;
    float An[SPL], A2[SPL], entry[SPL], w[SPL], gA[SPL];
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        An[i] = on && n0 + i < a.S ? a.A[static_cast<size_t>(ch) * a.S + n0 + i] : 0.f;
        A2[i] = An[i] * kLog2e;
        gA[i] = entry[i] = w[i] = 0.f;
    }
    if (pl.nseg > 1) {
        load_state<SPL>(a.workspace + pl.off_end + slot * a.S, n0, a.S, on, entry);
        load_state<SPL>(a.workspace + pl.off_rev + slot * a.S, n0, a.S, on, w);
    } else {
        if (a.state_in != nullptr) load_state<SPL>(a.state_in + bd * a.S, n0, a.S, on, entry);
        if (a.gstate_out != nullptr) load_state<SPL>(a.gstate_out + bd * a.S, n0, a.S, on, w);
    }
    const int cq = tid % CQ, ur = tid / CQ, uc = p.c0 + 4 * cq, left = ur < kTile ? p.cend - uc : 0;
    float bias[4], skip[4], gD[4] = {}, gbias[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bias[i] = a.bias != nullptr && i < left ? a.bias[uc + i] : 0.f;
        skip[i] = a.Dskip != nullptr && i < left ? a.Dskip[uc + i] : 0.f;
    }
    const size_t tok0 = static_cast<size_t>(p.b) * a.N;
    // gradient rows behind the sequence's last token are zero
    for (int t = (t_end > t_begin ? t_end : t_begin) + ur; t < t_full && left > 0; t += kScanThreads / CQ) {
        const float zero[4] = {};
        const size_t at = (tok0 + t) * a.D + uc;
        store_n<T, 4>(static_cast<T*>(a.gx) + at, zero, left);
        store_n<T, 4>(static_cast<T*>(a.gdt) + at, zero, left);
        if (a.gz != nullptr) store_n<T, 4>(static_cast<T*>(a.gz) + at, zero, left);
    }
    float* part = a.workspace + pl.off_bc;                 // [2][block][B N][S]
    const size_t tokens = static_cast<size_t>(a.B) * a.N;
    const int blk = blockIdx.x % pl.nblk;
    float* pB = part + (static_cast<size_t>(blk) * tokens + tok0) * a.S;
    float* pC = pB + static_cast<size_t>(pl.nblk) * tokens * a.S;
    for (size_t t = static_cast<size_t>(t_end > t_begin ? t_end : t_begin) * a.S + tid; t < static_cast<size_t>(t_full) * a.S;
         t += kScanThreads)
        pB[t] = pC[t] = 0.f;

    Raw<T, 4> rx = {}, rdt = {}, rz = {}, rg = {};
    StateRows<T, kTile, SP> nB, nC;
    const int ntile = t_end > t_begin ? (t_end - t_begin + kTile - 1) / kTile : 0;
    auto fetch = [&](int t0) {
        const int rows = t_end - t0;
        rx = rdt = rz = rg = Raw<T, 4>{};
        if (ur < rows && left > 0) {
            const size_t t = tok0 + t0 + ur;
            rx = raw_load_n<T, 4>(static_cast<const T*>(a.x) + t * a.ldx + uc, left);
            rdt = raw_load_n<T, 4>(static_cast<const T*>(a.dt) + t * a.lddt + uc, left);
            if (a.z != nullptr) rz = raw_load_n<T, 4>(static_cast<const T*>(a.z) + t * a.ldz + uc, left);
            rg = raw_load_n<T, 4>(static_cast<const T*>(a.gy) + t * a.D + uc, left);
        }
        nB.load(static_cast<const T*>(a.Bm) + (tok0 + t0) * a.ldb + p.g * a.S, a.ldb, rows, a.S);
        nC.load(static_cast<const T*>(a.Cm) + (tok0 + t0) * a.ldc + p.g * a.S, a.ldc, rows, a.S);
    };
    if (ntile > 0) fetch(t_begin + (ntile - 1) * kTile);
    for (int tile = ntile - 1; tile >= 0; --tile) {
        const int t0 = t_begin + tile * kTile, rows = t_end - t0 < kTile ? t_end - t0 : kTile;
        // the state in front of the tile
        float h0[SPL];
        {
            const size_t at = (static_cast<size_t>(p.b) * tiles + t0 / kTile) * a.D + ch;
            load_state<SPL>(a.workspace + pl.off_ckpt + at * a.S, n0, a.S, on, h0);
            const float cum = on ? a.workspace[pl.off_cum + at] : 0.f;
#pragma unroll
            for (int i = 0; i < SPL; ++i) h0[i] = fmaf(exp2_fast(cum * A2[i]), entry[i], h0[i]);
        }
        const Raw<T, 4> cx = rx, cz = rz, cg = rg, cdt = rdt;
        f32v4 d = {0.f, 0.f, 0.f, 0.f}, g = d;
        if (ur < kTile) {
            f32v4 u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                d[i] = ur < rows ? step_size(up(cdt.v[i]) + bias[i], a.softplus) : 0.f;
                u[i] = d[i] * up(cx.v[i]);
                g[i] = up(cg.v[i]);
                if (a.z != nullptr) {
                    const float z = up(cz.v[i]);
                    g[i] *= z * sigmoid_f(z);
                }
            }
            *reinterpret_cast<f32v4*>(&sdt[ur][4 * cq]) = d;
            *reinterpret_cast<f32v4*>(&su[ur][4 * cq]) = u;
            *reinterpret_cast<f32v4*>(&sg[ur][4 * cq]) = g;
        }
        nB.store(sB);
        nC.store(sC);
        __syncthreads();
        if (tile > 0) fetch(t0 - kTile);
        // forward through the tile: decays and states stay in registers
        float da[kTile][SPL], hs[kTile][SPL], py[kTile];
#pragma unroll
        for (int t = 0; t < kTile; ++t) {
            const float dt = sdt[t][cl], u = su[t][cl];
            float Bv[SPL], Cv[SPL];
            lds_states<SPL>(sB + t * SP + n0, Bv);
            lds_states<SPL>(sC + t * SP + n0, Cv);
            py[t] = 0.f;
#pragma unroll
            for (int i = 0; i < SPL; ++i) {
                da[t][i] = exp2_fast(dt * A2[i]);
                hs[t][i] = fmaf(da[t][i], t > 0 ? hs[t > 0 ? t - 1 : 0][i] : h0[i], u * Bv[i]);
                py[t] = fmaf(Cv[i], hs[t][i], py[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < kTile; t += LPC) sy[t + (lane & (LPC - 1))][cl] = state_sum<LPC>(py + t, lane);
        // and back
        float pu[kTile], pa[kTile], tA[SPL] = {};
#pragma unroll
        for (int tb = kTile - 4; tb >= 0; tb -= 4) {
            float vB[4][SPL], vC[4][SPL];
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                const int t = tb + j;
                const float dt = sdt[t][cl], u = su[t][cl], gt = sg[t][cl];
                float Bv[SPL], Cv[SPL];
                lds_states<SPL>(sB + t * SP + n0, Bv);
                lds_states<SPL>(sC + t * SP + n0, Cv);
                pu[t] = pa[t] = 0.f;
#pragma unroll
                for (int i = 0; i < SPL; ++i) {
                    const float adj = fmaf(Cv[i], gt, w[i]);
                    pu[t] = fmaf(adj, Bv[i], pu[t]);
                    vB[j][i] = adj * u;
                    vC[j][i] = gt * hs[t][i];
                    w[i] = adj * da[t][i];
                    const float q = w[i] * (t > 0 ? hs[t > 0 ? t - 1 : 0][i] : h0[i]);
                    pa[t] = fmaf(An[i], q, pa[t]);
                    tA[i] = fmaf(dt, q, tA[i]);
                }
            }
            float oB[KEPT], oC[KEPT];
            channel_sum<LPC>(vB, lane, oB);
            channel_sum<LPC>(vC, lane, oC);
            const int t = tb + 2 * (lane >> 5) + ((lane >> 4) & 1);
            const int s0 = n0 + (LPC == 16 ? 0 : LPC == 8 ? ((lane >> 3) & 1) * 2 : ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1));
#pragma unroll
            for (int k = 0; k < KEPT; ++k) {
                rB[wave][t * SP + s0 + k] = oB[k];
                rC[wave][t * SP + s0 + k] = oC[k];
            }
        }
#pragma unroll
        for (int i = 0; i < SPL; ++i) gA[i] += tA[i];
#pragma unroll
        for (int t = 0; t < kTile; t += LPC) {
            sdu[t + (lane & (LPC - 1))][cl] = state_sum<LPC>(pu + t, lane);
            sda[t + (lane & (LPC - 1))][cl] = state_sum<LPC>(pa + t, lane);
        }
        __syncthreads();
        for (int e = tid; e < rows * SP; e += kScanThreads) {
            const int t = e / SP, s = e % SP;
            if (s >= a.S) continue;
            const size_t at = static_cast<size_t>(t0 + t) * a.S + s;
            pB[at] = (rB[0][e] + rB[1][e]) + (rB[2][e] + rB[3][e]);
            pC[at] = (rC[0][e] + rC[1][e]) + (rC[2][e] + rC[3][e]);
        }
        if (ur < rows && left > 0) {
            const f32v4 du = *reinterpret_cast<const f32v4*>(&sdu[ur][4 * cq]);
            const f32v4 dA = *reinterpret_cast<const f32v4*>(&sda[ur][4 * cq]);
            const f32v4 ys = *reinterpret_cast<const f32v4*>(&sy[ur][4 * cq]);
            float ox[4], odt[4], oz[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = up(cx.v[i]);
                ox[i] = fmaf(du[i], d[i], g[i] * skip[i]);
                odt[i] = fmaf(du[i], x, dA[i]);
                if (a.softplus) odt[i] *= sigmoid_f(up(cdt.v[i]) + bias[i]);
                gD[i] = fmaf(g[i], x, gD[i]);
                gbias[i] += odt[i];
                if (a.z != nullptr) {
                    const float z = up(cz.v[i]), s = sigmoid_f(z);
                    oz[i] = up(cg.v[i]) * fmaf(skip[i], x, ys[i]) * fmaf(z * s, 1.f - s, s);
                }
            }
            const size_t at = (tok0 + t0 + ur) * a.D + uc;
            store_n<T, 4>(static_cast<T*>(a.gx) + at, ox, left);
            store_n<T, 4>(static_cast<T*>(a.gdt) + at, odt, left);
            if (a.gz != nullptr) store_n<T, 4>(static_cast<T*>(a.gz) + at, oz, left);
        }
    }
    // [B nseg][S + 2][D] partial sums of the parameters' gradients
    float* par = a.workspace + pl.off_par + static_cast<size_t>(blockIdx.x / pl.nblk) * (a.S + 2) * a.D;
    if (on) {
#pragma unroll
        for (int i = 0; i < SPL; ++i)
            if (n0 + i < a.S) par[static_cast<size_t>(n0 + i) * a.D + ch] = gA[i];
        if (p.seg == 0 && a.gstate_in != nullptr) store_state<SPL>(a.gstate_in + bd * a.S, n0, a.S, w);
    }
    __syncthreads();
    if (ur < kTile) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sdu[ur][4 * cq + i] = gD[i];
            sda[ur][4 * cq + i] = gbias[i];
        }
    }
    __syncthreads();
    if (tid < CH && p.c0 + tid < p.cend) {
        float s = 0.f, b = 0.f;
#pragma unroll
        for (int r = 0; r < kTile; ++r) {
            s += sdu[r][tid];
            b += sda[r][tid];
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

template <typename T, int LPC>
hipError_t bwd_cfg(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
    const dim3 block(kScanThreads);
    const unsigned wgs = static_cast<unsigned>(p.nblk) * a.B;
    if (wgs > 0) {
        {
            ProfScope prof(kProfScanPre, st);
            hipLaunchKernelGGL((scan_keep_kernel<T, LPC>), dim3(wgs * p.nseg), block, 0, st, a, p);
        }
        if (p.nseg > 1) {
            ProfScope prof(kProfScanPre, st);
            hipLaunchKernelGGL((scan_rev_kernel<T, LPC>), dim3(wgs * (p.nseg - 1)), block, 0, st, a, p);
            const size_t n = static_cast<size_t>(a.B) * a.D * a.S;
            hipLaunchKernelGGL(scan_compose_both_kernel, dim3(static_cast<unsigned>((n + kScanThreads - 1) / kScanThreads)),
                               block, 0, st, a, p);
        }
        {
            ProfScope prof(kProfSelScan, st);
            hipLaunchKernelGGL((scan_bwd_kernel<T, LPC>), dim3(wgs * p.nseg), block, 0, st, a, p);
        }
        const size_t n = 2 * static_cast<size_t>(a.B) * a.N * a.G * a.S;
        if (n > 0) {
            ProfScope prof(kProfReduce, st);
            hipLaunchKernelGGL((scan_bc_kernel<T>), dim3(static_cast<unsigned>((n + kScanThreads - 1) / kScanThreads)), block,
                               0, st, a, p);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const ColReduceArgs c{a.workspace + p.off_par, a.B * p.nseg, a.S + 2, a.S, a.D, a.gA, a.gD, a.gbias, false};
    return launch_col_reduce(c, st);
}

template <typename T>
hipError_t bwd_typed(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
    return p.cfg == 0 ? bwd_cfg<T, 4>(a, p, st) : p.cfg == 1 ? bwd_cfg<T, 8>(a, p, st) : bwd_cfg<T, 16>(a, p, st);
}

}  // namespace

ScanPlan scan_bwd_plan(int B, int N, int D, int G, int S) {
    ScanPlan p{};
    p.cfg = S <= 16 ? 0 : S <= 32 ? 1 : 2;
    p.ch = p.cfg == 0 ? 64 : p.cfg == 1 ? 32 : 16;
    p.nblk = G * ((D / G + p.ch - 1) / p.ch);
    const size_t wgs = static_cast<size_t>(p.nblk) * (B > 0 ? B : 1);
    // Segments: as many as bring the chip two workgroups a CU, of 8 tiles at least.
    const int most = N / (8 * kTile) > 1 ? N / (8 * kTile) : 1;
    int want = wgs >= 256 ? 1 : static_cast<int>((512 + wgs - 1) / wgs);
    if (want > most) want = most;
    const int steps = (N + 2 * kTile - 1) / (2 * kTile);   // the first passes take two tiles a step
    const int per = (steps + want - 1) / want;
    p.seg = per > 0 ? per * 2 * kTile : 2 * kTile;
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

hipError_t launch_scan_bwd(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
    return a.bf16 ? bwd_typed<bf16_t>(a, p, st) : bwd_typed<float>(a, p, st);
}

}  // namespace retn
