// Selective scan: per channel d and state n,
//     h_t[n] = exp(dt_t A[n]) h_(t-1)[n] + dt_t x_t B_t[n],
//     y_t = (sum_n C_t[n] h_t[n] + D x_t) silu(z_t),      dt = softplus(raw + bias)
//
// Bound by the vector ALUs: an exponential and four multiply-adds per (token, channel,
// state), where HBM moves eight bytes per (token, channel).  The states stay in registers
// (scan.h has the lane layout), tokens come in tiles of 32 that are staged in LDS: dt and
// dt x once per (token, channel), B and C once per token.  The next tile's global loads are
// in flight while a tile is walked; y goes back through LDS so that its gating and its
// store run on packs of channels.
//
// Few channels leave most of the chip idle, so a sequence is then cut into segments: a
// first pass walks every segment but the last from a zero state, keeping its end state
// and the sum of its dt (the segment's whole decay is exp(A sum dt)), a small kernel
// composes the entry states, and the main pass walks all segments at once.

#include "scan.h"

namespace retn {

namespace {

constexpr int kTile = 32;      // tokens of a tile

// STATE: the first pass of a segmented sequence, no y.
template <typename T, int LPC, int SPL, bool STATE>
__global__ __launch_bounds__(kScanThreads) void scan_fwd_kernel(ScanArgs a, ScanPlan pl) {
    constexpr int CH = kScanThreads / LPC, SP = LPC * SPL, CQ = CH / 4;   // channels, states, packs of 4 channels
    constexpr int UNITS = kTile * CQ, NU = (UNITS + kScanThreads - 1) / kScanThreads;
    static_assert(UNITS % kScanThreads == 0 || NU == 1, "units fill the workgroup or run in one pass");
    __shared__ float sdt[kTile][CH], su[kTile][CH], sy[STATE ? 1 : kTile][CH];
    __shared__ __attribute__((aligned(16))) float sB[kTile * SP], sC[STATE ? 4 : kTile * SP];
    const int tid = threadIdx.x, lane = tid & 63;
    const ScanPlace p = scan_place<CH>(a, pl.nblk, STATE ? pl.nseg - 1 : pl.nseg, blockIdx.x);
    const int n = scan_length(a.lengths, p.b, a.N);
    const int t_begin = p.seg * pl.seg, t_full = t_begin + pl.seg < a.N ? t_begin + pl.seg : a.N;
    const int t_end = t_full < n ? t_full : n;
    // this lane's channel and states
    const int cl = tid / LPC, ch = p.c0 + cl, n0 = state_group<LPC>(lane) * SPL;
    const bool on = ch < p.cend;
    float A2[SPL], h[SPL];
#pragma unroll
    for (int i = 0; i < SPL; ++i)
        A2[i] = on && n0 + i < a.S ? a.A[static_cast<size_t>(ch) * a.S + n0 + i] * kLog2e : 0.f;
    const size_t bd = static_cast<size_t>(p.b) * a.D + ch;
    const size_t slot = (static_cast<size_t>(p.b) * pl.nseg + p.seg) * a.D + ch;   // (sequence, segment, channel)
    if (STATE || (pl.nseg == 1 && a.state_in == nullptr)) {
#pragma unroll
        for (int i = 0; i < SPL; ++i) h[i] = 0.f;
    } else if (pl.nseg == 1) {
        load_state<SPL>(a.state_in + bd * a.S, n0, a.S, on, h);
    } else {
        load_state<SPL>(a.workspace + pl.off_end + slot * a.S, n0, a.S, on, h);
    }
    float dsum = 0.f;

    // this thread's packs of 4 channels: all of its tokens in the same channels
    const int cq = tid % CQ, uc = p.c0 + 4 * cq, left = p.cend - uc;
    float bias[4], skip[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bias[i] = a.bias != nullptr && i < left ? a.bias[uc + i] : 0.f;
        skip[i] = a.Dskip != nullptr && i < left ? a.Dskip[uc + i] : 0.f;
    }
    Raw<T, 4> rx[NU], rdt[NU], rz[NU], cx[NU], cz[NU];
    StateRows<T, kTile, SP> rB, rC;
    const size_t tok0 = static_cast<size_t>(p.b) * a.N;
    auto fetch = [&](int t0) {
        const int rows = t_end - t0;
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            const int r = (tid + k * kScanThreads) / CQ;
            rx[k] = rdt[k] = rz[k] = Raw<T, 4>{};
            if (r < rows && r < kTile && left > 0) {
                const size_t t = tok0 + t0 + r;
                rx[k] = raw_load_n<T, 4>(static_cast<const T*>(a.x) + t * a.ldx + uc, left);
                rdt[k] = raw_load_n<T, 4>(static_cast<const T*>(a.dt) + t * a.lddt + uc, left);
                if (!STATE && a.z != nullptr) rz[k] = raw_load_n<T, 4>(static_cast<const T*>(a.z) + t * a.ldz + uc, left);
            }
        }
        rB.load(static_cast<const T*>(a.Bm) + (tok0 + t0) * a.ldb + p.g * a.S, a.ldb, rows, a.S);
        if (!STATE) rC.load(static_cast<const T*>(a.Cm) + (tok0 + t0) * a.ldc + p.g * a.S, a.ldc, rows, a.S);
    };
    if (t_begin < t_end) fetch(t_begin);
    for (int t0 = t_begin; t0 < t_end; t0 += kTile) {
        const int rows = t_end - t0 < kTile ? t_end - t0 : kTile;
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            const int r = (tid + k * kScanThreads) / CQ;
            if (UNITS % kScanThreads == 0 || r < kTile) {
                f32v4 d, u;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float v = r < rows ? step_size(up(rdt[k].v[i]) + bias[i], a.softplus) : 0.f;
                    d[i] = v;
                    u[i] = v * up(rx[k].v[i]);
                }
                *reinterpret_cast<f32v4*>(&sdt[r][4 * cq]) = d;
                *reinterpret_cast<f32v4*>(&su[r][4 * cq]) = u;
            }
            cx[k] = rx[k];
            cz[k] = rz[k];
        }
        rB.store(sB);
        if (!STATE) rC.store(sC);
        __syncthreads();
        if (t0 + kTile < t_end) fetch(t0 + kTile);
#pragma unroll
        for (int tb = 0; tb < kTile; tb += LPC) {
            float part[LPC];
#pragma unroll
            for (int j = 0; j < LPC; ++j) {
                const int t = tb + j;
                const float dt = sdt[t][cl], u = su[t][cl];
                float Bv[SPL], Cv[SPL];
                lds_states<SPL>(sB + t * SP + n0, Bv);
                if (!STATE) lds_states<SPL>(sC + t * SP + n0, Cv);
                if (STATE) dsum += dt;
                float y = 0.f;
#pragma unroll
                for (int i = 0; i < SPL; ++i) {
                    h[i] = fmaf(exp2_fast(dt * A2[i]), h[i], u * Bv[i]);
                    if (!STATE) y = fmaf(Cv[i], h[i], y);
                }
                part[j] = y;
            }
            if (!STATE) sy[tb + (lane & (LPC - 1))][cl] = state_sum<LPC>(part, lane);
        }
        __syncthreads();
        if (!STATE) {
#pragma unroll
            for (int k = 0; k < NU; ++k) {
                const int r = (tid + k * kScanThreads) / CQ;
                if (r >= rows || left <= 0) continue;
                const f32v4 s = *reinterpret_cast<const f32v4*>(&sy[r][4 * cq]);
                float o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[i] = fmaf(skip[i], up(cx[k].v[i]), s[i]);
                    if (a.z != nullptr) {
                        const float z = up(cz[k].v[i]);
                        o[i] *= z * sigmoid_f(z);
                    }
                }
                store_n<T, 4>(static_cast<T*>(a.y) + (tok0 + t0 + r) * a.D + uc, o, left);
            }
        }
    }
    if (!on) return;
    if (STATE) {
        store_state<SPL>(a.workspace + pl.off_end + slot * a.S, n0, a.S, h);
        if (n0 == 0) a.workspace[pl.off_dt + slot] = dsum;
    } else if (p.seg == pl.nseg - 1 && a.state_out != nullptr) {
        store_state<SPL>(a.state_out + bd * a.S, n0, a.S, h);
    }
}

// Entry states of a sequence's segments in place of their predecessors' end states.
__global__ __launch_bounds__(kScanThreads) void scan_compose_kernel(ScanArgs a, ScanPlan pl) {
    const size_t ds = static_cast<size_t>(a.D) * a.S, id = static_cast<size_t>(blockIdx.x) * kScanThreads + threadIdx.x;
    if (id >= ds * a.B) return;
    const size_t b = id / ds, e = id % ds;
    const float A2 = a.A[e] * kLog2e;
    float* end = a.workspace + pl.off_end + b * pl.nseg * ds + e;
    const float* sum = a.workspace + pl.off_dt + b * pl.nseg * a.D + e / a.S;
    float h = a.state_in != nullptr ? a.state_in[id] : 0.f;
    for (int s = 0; s < pl.nseg - 1; ++s) {
        const float own = end[s * ds];
        end[s * ds] = h;
        h = fmaf(exp2_fast(A2 * sum[static_cast<size_t>(s) * a.D]), h, own);
    }
    end[(pl.nseg - 1) * ds] = h;
}

// One token.  LPC lanes of 4 states per channel; the state is read and written once.
template <typename T, int LPC>
__global__ __launch_bounds__(kScanThreads) void scan_step_kernel(ScanArgs a) {
    const size_t id = static_cast<size_t>(blockIdx.x) * kScanThreads + threadIdx.x, bd = id / LPC;
    const bool live = bd < static_cast<size_t>(a.B) * a.D;     // whole channels: their lanes agree
    const size_t b = live ? bd / a.D : 0;
    const int d = live ? static_cast<int>(bd % a.D) : 0, n0 = static_cast<int>(id % LPC) * 4, g = d / (a.D / a.G);
    const float x = live ? up(static_cast<const T*>(a.x)[b * a.ldx + d]) : 0.f;
    float dt = live ? up(static_cast<const T*>(a.dt)[b * a.lddt + d]) : 0.f;
    if (a.bias != nullptr) dt += a.bias[d];
    dt = step_size(dt, a.softplus);
    const float u = dt * x;
    const T* Bp = static_cast<const T*>(a.Bm) + b * a.ldb + g * a.S + n0;
    const T* Cp = static_cast<const T*>(a.Cm) + b * a.ldc + g * a.S + n0;
    const int left = live ? a.S - n0 : 0;
    float y = 0.f;
    if (left > 0) {
        float* hp = a.state_out + bd * a.S + n0;
        const Raw<float, 4> h = raw_load_n<float, 4>(hp, left);
        const Raw<float, 4> A = raw_load_n<float, 4>(a.A + static_cast<size_t>(d) * a.S + n0, left);
        const Raw<T, 4> Br = raw_load_n<T, 4>(Bp, left), Cr = raw_load_n<T, 4>(Cp, left);
        Raw<float, 4> o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o.v[i] = fmaf(exp2_fast(dt * (A.v[i] * kLog2e)), h.v[i], u * up(Br.v[i]));
            y = fmaf(i < left ? up(Cr.v[i]) : 0.f, o.v[i], y);
        }
        raw_store_n<float, 4>(hp, o, left);
    }
    if (LPC >= 2) y += lane_xor<1>(y);
    if (LPC >= 4) y += lane_xor<2>(y);
    if (LPC >= 8) y += lane_xor<7>(y);
    if (LPC >= 16) y += lane_xor<8>(y);
    if (!live || n0 != 0) return;
    if (a.Dskip != nullptr) y = fmaf(a.Dskip[d], x, y);
    if (a.z != nullptr) {
        const float z = up(static_cast<const T*>(a.z)[b * a.ldz + d]);
        y *= z * sigmoid_f(z);
    }
    static_cast<T*>(a.y)[bd] = down<T>(y);
}

template <typename T, int LPC, int SPL>
hipError_t fwd_cfg(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
    const dim3 block(kScanThreads);
    if (p.nseg > 1) {
        {
            ProfScope prof(kProfScanPre, st);
            hipLaunchKernelGGL((scan_fwd_kernel<T, LPC, SPL, true>),
                               dim3(static_cast<unsigned>(p.nblk) * (p.nseg - 1) * a.B), block, 0, st, a, p);
        }
        const size_t n = static_cast<size_t>(a.B) * a.D * a.S;
        ProfScope prof(kProfScanPre, st);
        hipLaunchKernelGGL(scan_compose_kernel, dim3(static_cast<unsigned>((n + kScanThreads - 1) / kScanThreads)), block, 0,
                           st, a, p);
    }
    ProfScope prof(kProfSelScan, st);
    hipLaunchKernelGGL((scan_fwd_kernel<T, LPC, SPL, false>), dim3(static_cast<unsigned>(p.nblk) * p.nseg * a.B), block, 0,
                       st, a, p);
    return hipGetLastError();
}

template <typename T>
hipError_t fwd_typed(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
    return p.cfg == 0 ? fwd_cfg<T, 4, 4>(a, p, st) : p.cfg == 1 ? fwd_cfg<T, 8, 4>(a, p, st) : fwd_cfg<T, 16, 4>(a, p, st);
}

template <typename T>
hipError_t step_typed(const ScanArgs& a, hipStream_t st) {
    const int lanes = (a.S + 3) / 4, lpc = lanes <= 1 ? 1 : lanes <= 2 ? 2 : lanes <= 4 ? 4 : lanes <= 8 ? 8 : 16;
    const size_t n = static_cast<size_t>(a.B) * a.D * lpc;
    const dim3 grid(static_cast<unsigned>((n + kScanThreads - 1) / kScanThreads)), block(kScanThreads);
    ProfScope prof(kProfSelScan, st);
    switch (lpc) {
        case 1: hipLaunchKernelGGL((scan_step_kernel<T, 1>), grid, block, 0, st, a); break;
        case 2: hipLaunchKernelGGL((scan_step_kernel<T, 2>), grid, block, 0, st, a); break;
        case 4: hipLaunchKernelGGL((scan_step_kernel<T, 4>), grid, block, 0, st, a); break;
        case 8: hipLaunchKernelGGL((scan_step_kernel<T, 8>), grid, block, 0, st, a); break;
        default: hipLaunchKernelGGL((scan_step_kernel<T, 16>), grid, block, 0, st, a); break;
    }
    return hipGetLastError();
}

}  // namespace

ScanPlan scan_fwd_plan(int B, int N, int D, int G, int S) {
    ScanPlan p{};
    p.cfg = S <= 16 ? 0 : S <= 32 ? 1 : 2;
    p.ch = p.cfg == 0 ? 64 : p.cfg == 1 ? 32 : 16;
    p.nblk = G * ((D / G + p.ch - 1) / p.ch);
    // Segments: as many as bring the chip four workgroups a CU, of four tiles at least.
    const size_t wgs = static_cast<size_t>(p.nblk) * (B > 0 ? B : 1);
    const int most = N / (4 * kTile) > 1 ? N / (4 * kTile) : 1;
    int want = wgs >= 512 ? 1 : static_cast<int>((1024 + wgs - 1) / wgs);
    if (want > most) want = most;
    const int tiles = (N + kTile - 1) / kTile;
    const int per = want > 0 ? (tiles + want - 1) / want : tiles;
    p.seg = per > 0 ? per * kTile : kTile;
    p.nseg = N > 0 ? (N - 1) / p.seg + 1 : 1;
    const size_t bs = static_cast<size_t>(B) * p.nseg * D;
    p.off_end = 0;
    p.off_dt = bs * S;
    p.total = p.nseg > 1 ? p.off_dt + bs : 0;
    return p;
}

hipError_t launch_scan_fwd(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
    return a.bf16 ? fwd_typed<bf16_t>(a, p, st) : fwd_typed<float>(a, p, st);
}
hipError_t launch_scan_step(const ScanArgs& a, hipStream_t st) {
    return a.bf16 ? step_typed<bf16_t>(a, st) : step_typed<float>(a, st);
}

}  // namespace retn
