// Rotary positions: pair i of a head's first `rot` elements turns by its token's angle,
//     (a, b) -> (a c - b s, a s + b c),   (c, s) = table[position][i],
// where the pair is (2i, 2i+1) or (i, i + rot/2); the other elements pass; everything is
// scaled.  The backward is the transpose, (c, s) -> (c, -s).
//
// Bound by HBM: every element of q and k is read and written once.  A thread takes one
// 16-byte pack (or one in each half) of a token's head and walks over that token's heads
// with the cosines and sines in registers, so the table is read once per token and not
// once per head; four heads' loads are in flight at a time.  Reading and writing with
// strides, the pass also turns token-major projections into the operators' [B,H,N,d].
//
// Measured: 277 MB of bf16 q and k (16384 tokens, 16 heads of 128) in 56 us (4.9 TB/s), 68 MB
// of gradients in 14.1 us; one token of 128 sequences is one launch (4 us on the device).

#include "block.h"
#include "launch.h"
#include "vec_io.h"

namespace retn {

namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 4;               // heads whose loads are issued together
constexpr size_t kWantThreads = 1 << 17;   // 8 waves of 64 for each of 256 CUs
constexpr size_t kMostGroups = 1 << 23;    // of one launch, which takes 2^32 threads at most

// V elements a side: interleaved, V adjacent elements (V / 2 pairs); halves, V pairs with
// one pack in each half.  V = 0: one pair a thread, any sizes.
template <typename T, bool INTER, int V>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a, size_t tok0, int units, int heads_per) {
    constexpr int E = V > 0 ? V : (INTER ? 2 : 1);   // adjacent elements of a pack
    constexpr int PAIRS = INTER ? E / 2 : E;
    const int tpb = kThreads / units;                // tokens of a workgroup
    const int u = threadIdx.x % units;
    const size_t tok = tok0 + static_cast<size_t>(blockIdx.x) * tpb + threadIdx.x / units;
    if (threadIdx.x >= tpb * units || tok >= static_cast<size_t>(a.B) * a.N) return;
    const int b = static_cast<int>(tok / a.N), n = static_cast<int>(tok % a.N);
    // a unit rotates, or copies elements behind the rotated part
    const int half = a.rot / 2;
    const int turning = INTER ? a.rot / E : half / E;
    const bool turns = u < turning;
    const bool one = V == 0 && INTER;                // the scalar form copies single elements
    const int e0 = turns ? u * E : a.rot + (u - turning) * (one ? 1 : E);
    float c[PAIRS], s[PAIRS];
    if (turns) {
        const long long p = a.pos != nullptr ? a.pos[a.pos_batched ? tok : static_cast<size_t>(n)] : a.first + n;
        const bool known = p >= 0 && p < a.table_len;
        const float nan = __builtin_nanf("");
        const float* t = a.table + (known ? p : 0) * a.rot + 2 * (INTER ? u * PAIRS : e0);
        const Raw<float, 2 * PAIRS> r = raw_load<float, 2 * PAIRS>(t);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            c[i] = known ? r.v[2 * i] : nan;
            s[i] = known ? (a.transpose ? -r.v[2 * i + 1] : r.v[2 * i + 1]) : nan;
        }
    }
    const int heads = a.q.H + a.k.H, h1 = blockIdx.y * heads_per;
    const int h2 = h1 + heads_per < heads ? h1 + heads_per : heads;
    const bool both = turns && !INTER;               // a second pack, in the other half
    for (int h = h1; h < h2; h += kInFlight) {
        Raw<T, E> lo[kInFlight], hi[kInFlight];
#pragma unroll
        for (int j = 0; j < kInFlight; ++j) {
            if (h + j >= h2) break;
            const bool isk = h + j >= a.q.H;
            const RotaryView& w = isk ? a.k : a.q;
            const T* p = static_cast<const T*>(w.in) + b * w.in_b + (h + j - (isk ? a.q.H : 0)) * w.in_h + n * w.in_n + e0;
            lo[j].v[0] = T(0);
            if (one && !turns)
                lo[j].v[0] = p[0];
            else
                lo[j] = raw_load<T, E>(p);
            if (both) hi[j] = raw_load<T, E>(p + half);
        }
#pragma unroll
        for (int j = 0; j < kInFlight; ++j) {
            if (h + j >= h2) break;
            const bool isk = h + j >= a.q.H;
            const RotaryView& w = isk ? a.k : a.q;
            T* p = static_cast<T*>(w.out) + b * w.out_b + (h + j - (isk ? a.q.H : 0)) * w.out_h + n * w.out_n + e0;
            const float m = w.scale;
            if (!turns) {
                if (one) {
                    p[0] = down<T>(up(lo[j].v[0]) * m);
                } else {
                    float o[E];
#pragma unroll
                    for (int i = 0; i < E; ++i) o[i] = up(lo[j].v[i]) * m;
                    store_n<T, E>(p, o, E);
                }
                continue;
            }
            float o[E], o2[E];
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                const float x = up(INTER ? lo[j].v[2 * i] : lo[j].v[i]);
                const float y = up(INTER ? lo[j].v[2 * i + 1] : hi[j].v[i]);
                const float rx = (x * c[i] - y * s[i]) * m, ry = (x * s[i] + y * c[i]) * m;
                if (INTER) {
                    o[2 * i] = rx;
                    o[2 * i + 1] = ry;
                } else {
                    o[i] = rx;
                    o2[i] = ry;
                }
            }
            store_n<T, E>(p, o, E);
            if (both) store_n<T, E>(p + half, o2, E);
        }
    }
}

// table[i][j] = magnitude (cos, sin)((first + i) freq[j]): the angle is formed and reduced
// modulo 2 pi in fp64 (far positions reach millions of radians), the functions are fp64 too.
__global__ __launch_bounds__(kThreads) void rotary_table_kernel(float* table, const double* freq, int pairs, long long first,
                                                                 long long count, float magnitude) {
    const size_t e = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (e >= static_cast<size_t>(count) * pairs) return;
    const double ang = static_cast<double>(first + static_cast<long long>(e / pairs)) * freq[e % pairs];
    double s, c;
    sincos(ang, &s, &c);
    table[2 * e] = static_cast<float>(c * magnitude);
    table[2 * e + 1] = static_cast<float>(s * magnitude);
}

template <typename T, bool INTER>
hipError_t launch_typed(const RotaryArgs& a, hipStream_t st) {
    constexpr int V = kPack<T>;
    const int rest = a.d - a.rot;
    const bool packs = INTER ? a.rot % V == 0 && rest % V == 0 : a.rot / 2 % V == 0 && rest % V == 0;
    // elements that a unit of the rotated part and of the rest takes
    const int units = packs ? (INTER ? a.rot / V : a.rot / 2 / V) + rest / V : a.rot / 2 + rest;
    const size_t tokens = static_cast<size_t>(a.B) * a.N;
    const int heads = a.q.H + a.k.H;
    // as many heads a thread as leave enough threads to fill the chip
    int per = 16;
    while (per > 1 && tokens * units * ((heads + per - 1) / per) < kWantThreads) per /= 2;
    const int tpb = kThreads / units;
    const size_t groups = (tokens + tpb - 1) / tpb;
    ProfScope prof(kProfRotary, st);
    // (one launch, unless there are more than 8M workgroups: heads without packs, a token each)
    for (size_t g = 0; g < groups; g += kMostGroups) {
        const size_t now = groups - g < kMostGroups ? groups - g : kMostGroups;
        const dim3 grid(static_cast<unsigned>(now), (heads + per - 1) / per), block(kThreads);
        if (packs)
            hipLaunchKernelGGL((rotary_kernel<T, INTER, V>), grid, block, 0, st, a, g * tpb, units, per);
        else
            hipLaunchKernelGGL((rotary_kernel<T, INTER, 0>), grid, block, 0, st, a, g * tpb, units, per);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, hipStream_t st) {
    if (a.bf16) return a.interleaved ? launch_typed<bf16_t, true>(a, st) : launch_typed<bf16_t, false>(a, st);
    return a.interleaved ? launch_typed<float, true>(a, st) : launch_typed<float, false>(a, st);
}

hipError_t launch_rotary_table(float* table, const double* freq, int pairs, long long first, long long count,
                               float magnitude, hipStream_t st) {
    const size_t n = static_cast<size_t>(count) * pairs;
    ProfScope prof(kProfRotary, st);
    hipLaunchKernelGGL(rotary_table_kernel, dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                       st, table, freq, pairs, first, count, magnitude);
    return hipGetLastError();
}

}  // namespace retn
