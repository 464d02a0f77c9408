// Selective scan: per channel d and state n,
//     h_t[n] = exp(dt_t A[n]) h_(t-1)[n] + dt_t x_t B_t[n],
//     y_t = (sum_n C_t[n] h_t[n] + D x_t) silu(z_t),      dt = softplus(raw + bias)
//
// Bound by the vector ALUs: an exponential and four products per (token, channel,
// state), where HBM moves eight bytes per (token, channel).  A lane walks over the tokens of
// one channel with all of its states in registers (scan.h).
//
// Few channels leave most of the chip idle, so a sequence is cut into segments: a first
// pass walks every segment but the last from a zero state, keeping its end state and the
// sum of its dt (the segment's whole decay is exp(A sum dt)), a small kernel composes the
// entry states, and the main pass walks all segments at once.
//
// Measured, S = 16, bf16, gated: 4 x 2048 x 2048 channels 125 us (first pass 50, composition 9,
// main pass 66), 1 x 16384 x 2048 230 us (95, 11 and 123); the vector ALUs are busy 65-75% of the
// first pass and 72-80% of the main pass, and issue matrix instructions in much of the rest.  An
// exponential costs as much issue time as three multiply-adds, so the pass cannot be much
// shorter than its instructions.

#include "scan.h"

namespace retn {

namespace {

// STATE: the first pass of a segmented sequence, no y.  (With the register limits the matrix
// instructions' states are in vector registers; without, they move to accumulation
// registers and back for every product: 153 us where these take 128.)
template <typename T, int SP, bool SCALAR, bool STATE>
__global__ __launch_bounds__(kScanThreads, SP <= 16 ? 4 : 2) void scan_fwd_kernel(ScanArgs a, ScanPlan pl) {
    const unsigned id = wave_id();
    const int nseg = STATE ? pl.nseg - 1 : pl.nseg;
    if (id >= static_cast<unsigned>(pl.nblk) * nseg * a.B) return;
    const ScanPlace p = scan_place<64>(a, pl.nblk, nseg, pl.seg, id);
    const int c = p.c0 + (threadIdx.x & 63), S = SCALAR ? SP : a.S;
    const bool on = c < p.cend;
    const int ch = on ? c : p.cend - 1;        // idle lanes repeat the last channel and store nothing
    using Rows = MatRows<T, SP>;
    using Block = MatBlock<T, SP>;
    using Read = WaveRow<T, SP, SCALAR>;
    float A2[SP], first[SP];
    f32v4 h[SP / 4];
    load_state<SP>(a.A + static_cast<size_t>(ch) * S, S, true, A2);
#pragma unroll
    for (int i = 0; i < SP; ++i) A2[i] *= kLog2e;
    const size_t bd = static_cast<size_t>(p.b) * a.D + ch;
    const size_t slot = (static_cast<size_t>(p.b) * pl.nseg + p.seg) * a.D + ch;   // (sequence, segment, channel)
    const float* from = STATE ? nullptr : pl.nseg > 1 ? a.workspace + pl.off_end + slot * S
                        : a.state_in != nullptr       ? a.state_in + bd * S
                                                      : nullptr;
    load_state<SP>(from, S, from != nullptr, first);
#pragma unroll
    for (int i = 0; i < SP; ++i) h[i / 4][i % 4] = first[i];
    const float bias = a.bias != nullptr ? a.bias[ch] : 0.f, skip = a.Dskip != nullptr ? a.Dskip[ch] : 0.f;
    float dsum = 0.f;
    const size_t tok0 = static_cast<size_t>(p.b) * a.N;
    // rows of the sequence, the same for all lanes; a lane adds its channel
    const T* xp = static_cast<const T*>(a.x) + tok0 * a.ldx;
    const T* dp = static_cast<const T*>(a.dt) + tok0 * a.lddt;
    const T* zp = static_cast<const T*>(a.z) + tok0 * a.ldz;
    const T* Bp = static_cast<const T*>(a.Bm) + tok0 * a.ldb + p.g * S;
    const T* Cp = static_cast<const T*>(a.Cm) + tok0 * a.ldc + p.g * S;
    T* yp = static_cast<T*>(a.y) + tok0 * a.D;
    const uint32_t at = static_cast<uint32_t>(ch) * sizeof(T);
    const bool gated = !STATE && a.z != nullptr;
    if (!STATE && a.zero_behind && on) {
        // this segment's rows behind the sequence's last token
        for (int t = p.t_begin > p.t_end ? p.t_begin : p.t_end; t < p.t_full; ++t)
            row_put(yp + static_cast<size_t>(t) * a.D, at, T(0));
    }

    // one token's step of all states; its read-out
    auto step = [&](float dt, float x, float B, auto tok, const Read& C) __attribute__((always_inline)) {
        const float u = dt * x;
        float y0 = skip * x, y1 = 0.f;
        each<SP / 4>([&](auto j) __attribute__((always_inline)) {
            f32v4 d;
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = exp2_fast(dt * A2[4 * j + i]) * h[j][i];
            h[j] = outer<SP, tok, j>(B, u, d);
        });
        if constexpr (!STATE) {
            each<SP>([&](auto i) __attribute__((always_inline)) {
                (i & 1 ? y1 : y0) = fmaf(C.template get<i>(S), h[i / 4][i % 4], i & 1 ? y1 : y0);
            });
        }
        dsum += dt;
        return y0 + y1;
    };
    auto gate = [&](float z) { return z * sigmoid_f(z); };

    T rx[kAhead], rdt[kAhead], rz[kAhead] = {};
    Block rB;
    Read rC[kAhead];                           // not SCALAR
    const uint32_t row_lane = Rows::lane_at(a.ldb, S), row_one = Rows::lane_at(0, S);
    auto fetch = [&](int t0) {
        const long long ldx = stepped(a.ldx), lddt = stepped(a.lddt), ldz = stepped(a.ldz);
        const uint32_t lane = opaque(at);      // added last, by the load itself
        const T* xr = xp + t0 * ldx;
        const T* dr = dp + t0 * lddt;
        const T* zr = zp + t0 * ldz;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            rx[k] = row_at(xr, lane);
            rdt[k] = row_at(dr, lane);
            xr += ldx;
            dr += lddt;
        }
        if (gated) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                rz[k] = row_at(zr, lane);
                zr += ldz;
            }
        }
        rB.load(Bp + t0 * a.ldb, a.ldb, row_lane);
        if (!STATE && !SCALAR) {
            const long long ldc = stepped(a.ldc);
            const T* cr = Cp + t0 * ldc;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                rC[k].load(cr, S);
                cr += ldc;
            }
        }
    };
    int t = p.t_begin;
    if (t + kAhead <= p.t_end) fetch(t);
    for (; t + kAhead <= p.t_end; t += kAhead) {
        // the block's steps and, behind them, its gates are taken together, so that the tokens
        // between them are straight code
        float x[kAhead], dt[kAhead], z[kAhead], y[kAhead];
        float B[Block::kRegs];
        rB.values(S, B);
        Read C[SCALAR ? 2 : kAhead];
        const long long ldc = stepped(a.ldc);
        const T* Ct = Cp + t * ldc;
        if (!STATE && SCALAR) C[0].load(Ct, S);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            x[k] = up(rx[k]);
            dt[k] = up(rdt[k]) + bias;
            z[k] = up(rz[k]);
            if (!STATE && !SCALAR) C[k] = rC[k];
        }
        if (t + 2 * kAhead <= p.t_end) fetch(t + kAhead);
        if (a.softplus) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) dt[k] = softplus_f(dt[k]);
        }
        each<kAhead>([&](auto k) __attribute__((always_inline)) {
            if (!STATE && SCALAR) {
                rows_arrived();
                if (k + 1 < kAhead) C[(k + 1) & 1].load(Ct += ldc, S);
                rows_issued();
            }
            y[k] = step(dt[k], x[k], B[k / Block::kTok], std::integral_constant<int, k % Block::kTok>{}, C[SCALAR ? k & 1 : k]);
        });
        if (STATE) continue;
        if (gated) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) y[k] *= gate(z[k]);
        }
        if (on) {
            const long long ldy = stepped(a.D);
            const uint32_t lane = opaque(at);
            T* yr = yp + t * ldy;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                row_put(yr, lane, down<T>(y[k]));
                yr += ldy;
            }
        }
    }
    for (; t < p.t_end; ++t) {
        Read C;
        if (!STATE) C.load(Cp + static_cast<size_t>(t) * a.ldc, S);
        const size_t tt = t;
        const float B = Rows::value(row_at(Bp + tt * a.ldb, row_one), S);   // every token's lanes: this one
        float y = step(step_size(up(row_at(dp + tt * a.lddt, at)) + bias, a.softplus), up(row_at(xp + tt * a.ldx, at)), B,
                       std::integral_constant<int, 0>{}, C);
        if (STATE) continue;
        if (gated) y *= gate(up(row_at(zp + tt * a.ldz, at)));
        if (on) row_put(yp + tt * a.D, at, down<T>(y));
    }
    if (!on) return;
#pragma unroll
    for (int i = 0; i < SP; ++i) first[i] = h[i / 4][i % 4];
    if (STATE) {
        store_state<SP>(a.workspace + pl.off_end + slot * S, S, first);
        a.workspace[pl.off_dt + slot] = dsum;
    } else if (p.seg == pl.nseg - 1 && a.state_out != nullptr) {
        store_state<SP>(a.state_out + bd * S, S, first);
    }
}

// Entry states of the segments in place of their end states.
template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void scan_compose_kernel(ScanArgs a, ScanPlan pl) {
    __shared__ ComposeSums<WAVES> sums;
    const size_t ds = static_cast<size_t>(a.D) * a.S, id = static_cast<size_t>(blockIdx.x) * 64 + (threadIdx.x & 63);
    // The last workgroup's idle lanes walk no segment: the walk is in place, and a pair has one owner.
    const bool live = id < ds * a.B;
    const size_t in = live ? id : 0;
    const int nseg = live ? pl.nseg : 0;
    const size_t b = in / ds, e = in % ds;
    compose<WAVES, false>(a.workspace + pl.off_end + b * pl.nseg * ds + e,
                          a.workspace + pl.off_dt + b * pl.nseg * a.D + e / a.S, ds, a.D, nseg, a.A[e] * kLog2e,
                          a.state_in != nullptr ? a.state_in[in] : 0.f, sums);
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

template <typename T, int SP, bool SCALAR>
hipError_t fwd_cfg(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
    const dim3 block(kScanThreads);
    constexpr unsigned wpg = kScanThreads / 64;
    const unsigned waves = static_cast<unsigned>(p.nblk) * a.B;
    if (p.nseg > 1) {
        ProfScope prof(kProfScanPre, st);
        hipLaunchKernelGGL((scan_fwd_kernel<T, SP, SCALAR, true>), dim3((waves * (p.nseg - 1) + wpg - 1) / wpg), block, 0, st,
                           a, p);
        const size_t n = static_cast<size_t>(a.B) * a.D * a.S;
        const int waves = compose_waves(p.nseg, n);
        hipLaunchKernelGGL(waves > 1 ? scan_compose_kernel<kComposeWaves> : scan_compose_kernel<1>,
                           dim3(static_cast<unsigned>((n + 63) / 64)), dim3(64 * waves), 0, st, a, p);
    }
    ProfScope prof(kProfSelScan, st);
    hipLaunchKernelGGL((scan_fwd_kernel<T, SP, SCALAR, false>), dim3((waves * p.nseg + wpg - 1) / wpg), block, 0, st, a, p);
    return hipGetLastError();
}

template <typename T, int SP>
hipError_t fwd_states(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
    return scalar_rows(a, SP) ? fwd_cfg<T, SP, true>(a, p, st) : fwd_cfg<T, SP, false>(a, p, st);
}

template <typename T>
hipError_t fwd_typed(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
    if (a.S <= 8) return fwd_states<T, 8>(a, p, st);
    if (a.S <= 16) return fwd_states<T, 16>(a, p, st);
    return a.S <= 32 ? fwd_states<T, 32>(a, p, st) : fwd_states<T, 64>(a, p, st);
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
    p.nblk = G * ((D / G + 63) / 64);
    // Segments: as many as bring the chip four waves a SIMD, of 16 tokens at least (a wave takes
    // 0.4 us a token where it has its SIMD to itself: 512 tokens of 2048 channels run 50 us
    // in segments of 64 tokens, 26 us in segments of 16).  Below 64 tokens the launches of a
    // cut cost more than it saves (32 tokens of 2048 channels 18 us whole, 24 us cut).
    const size_t waves = static_cast<size_t>(p.nblk) * (B > 0 ? B : 1);
    int want = waves >= 2048 ? 1 : static_cast<int>((4096 + waves - 1) / waves);
    const int most = N >= 64 ? N / 16 : 1;
    if (want > most) want = most;
    const int steps = (N + kAhead - 1) / kAhead, per = (steps + want - 1) / want;
    p.seg = per > 0 ? per * kAhead : kAhead;
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
