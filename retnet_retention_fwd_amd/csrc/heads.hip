// Root-mean-square norm of each head's row of queries and keys with rotary positions:
//     r = 1 / sqrt(mean(x^2) + eps),   out = scale turn(x r w)
// and the gradient: with g = scale turn^T(grad), xh = x r, v = g w,
//     gx = r (v - xh mean(v xh)),   gw = sum over all rows of g xh.
//
// Bound by HBM: each row is read once (twice for the gradient: x and grad) and written once.  A
// row lies over a group of LG lanes, a power of two, each with one 16-byte pack, or one in each
// half of the rotated part where pairs are (i, i + rot/2), so that a lane holds both elements
// of its pairs and the row's sum is a few lane exchanges.  A lane walks over the heads of its
// token with the cosines, the sines and both weights in registers, four heads' loads in flight.
// Heads whose parts are not whole packs take single pairs, four a lane of a whole wave.

#include "common.h"
#include "launch.h"
#include "proj.h"
#include "vec_io.h"

#include <algorithm>
#include <type_traits>

namespace retn {
namespace {

constexpr int kThreads = 256;
constexpr size_t kWantThreads = 1 << 17;   // 8 waves of 64 for each of 256 CUs
constexpr int kMaxBlocks = 1024;           // of the gradient: each leaves 2 d partial sums
constexpr size_t kMostGroups = 1 << 22;    // of one launch

// The sum over aligned groups of lg lanes (a power of two), in every lane.
__device__ __forceinline__ float group_sum(float x, int lg) {
    if (lg >= 2) x += lane_xor<1>(x);
    if (lg >= 4) x += lane_xor<2>(x);
    if (lg >= 8) x += lane_xor<7>(x);
    if (lg >= 16) x += lane_xor<8>(x);
    if (lg >= 32) x = halves_sum16(x, x);
    if (lg >= 64) x = halves_sum32(x, x);
    return x;
}

// A lane's part of a row: S units, in each E adjacent elements (lo) and, turning in halves, E more
// (hi), rot / 2 elements on.
template <int E, int S>
struct Part {
    float lo[S][E], hi[S][E];
};

// E: adjacent elements of a unit, S: units of a lane.  S = 1: packs; S = 4: single pairs, where a
// unit behind the rotated part is one element.
template <typename T, typename W, bool INTER, int E, int S, bool BWD>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadsArgs a, size_t tok0, size_t tokens, int lg, int heads_per) {
    constexpr bool kOne = S > 1;                     // single elements behind the rotated part
    constexpr int kPairs = INTER ? E / 2 : E;
    constexpr int kFly = kOne ? 1 : BWD ? 2 : 4;     // heads whose loads are in flight together
    const int sub = threadIdx.x & (lg - 1), rows = kThreads / lg;
    const int half = a.rot / 2, turning = INTER ? a.rot / E : half / E;
    const int rest_e = kOne ? 1 : E, units = turning + (a.d - a.rot) / rest_e;
    int e0[S];
    bool turns[S], live[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int u = sub + s * lg;
        live[s] = u < units;
        turns[s] = u < turning;
        e0[s] = turns[s] ? u * E : a.rot + (u - turning) * rest_e;
    }
    // elements s, i of a unit exist: behind the rotated part of single pairs only the first
    auto has = [&](int s, int i) { return live[s] && (!kOne || turns[s] || i == 0); };
    auto load = [&](const T* p, Part<E, S>& v) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if constexpr (kOne) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    v.lo[s][i] = has(s, i) ? up(p[e0[s] + i]) : 0.f;
                    v.hi[s][i] = !INTER && turns[s] && live[s] ? up(p[e0[s] + half + i]) : 0.f;
                }
            } else {
                Raw<T, E> x{}, y{};
                if (live[s]) x = raw_load<T, E>(p + e0[s]);
                if (!INTER && turns[s]) y = raw_load<T, E>(p + e0[s] + half);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    v.lo[s][i] = up(x.v[i]);
                    v.hi[s][i] = up(y.v[i]);
                }
            }
        }
    };
    auto store = [&](T* p, const Part<E, S>& v) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if constexpr (kOne) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    if (has(s, i)) p[e0[s] + i] = down<T>(v.lo[s][i]);
                    if (!INTER && turns[s] && live[s]) p[e0[s] + half + i] = down<T>(v.hi[s][i]);
                }
            } else {
                if (live[s]) store_n<T, E>(p + e0[s], v.lo[s], E);
                if (!INTER && turns[s]) store_n<T, E>(p + e0[s] + half, v.hi[s], E);
            }
        }
    };
    // the weights of q and k, in the places of the elements
    Part<E, S> w[2];
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        const W* p = static_cast<const W*>(o ? a.k.w : a.q.w);
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < E; ++i) {
                w[o].lo[s][i] = p == nullptr ? 1.f : has(s, i) ? up(p[e0[s] + i]) : 0.f;
                w[o].hi[s][i] = INTER || !turns[s] || !live[s] ? 0.f : p == nullptr ? 1.f : up(p[e0[s] + half + i]);
            }
    }
    Part<E, S> gw[2];
    if constexpr (BWD) {
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < E; ++i) gw[o].lo[s][i] = gw[o].hi[s][i] = 0.f;
    }
    const int heads = a.q.H + a.k.H, h1 = blockIdx.y * heads_per, h2 = min(h1 + heads_per, heads);
    const float inv_d = 1.f / a.d;

    // one trip a workgroup in the forward; the gradient's workgroups walk over the tokens
    for (size_t tok = tok0 + static_cast<size_t>(blockIdx.x) * rows + threadIdx.x / lg; tok < tokens;
         tok += static_cast<size_t>(gridDim.x) * rows) {
        const int b = static_cast<int>(tok / a.N), n = static_cast<int>(tok % a.N);
        float c[S][kPairs], sn[S][kPairs];
        {
            const long long p = a.pos != nullptr ? a.pos[a.pos_batched ? tok : static_cast<size_t>(n)] : a.first + n;
            const bool known = p >= 0 && p < a.table_len;
            const float nan = __builtin_nanf("");
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const float* t = a.table + (known ? p : 0) * a.rot + 2 * (INTER ? e0[s] / 2 : e0[s]);
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    c[s][i] = 1.f;
                    sn[s][i] = 0.f;
                    if (turns[s]) {
                        c[s][i] = known ? t[2 * i] : nan;
                        sn[s][i] = known ? (BWD ? -t[2 * i + 1] : t[2 * i + 1]) : nan;
                    }
                }
            }
        }
        auto turn = [&](Part<E, S>& v, float m) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if (!turns[s]) {
#pragma unroll
                    for (int i = 0; i < E; ++i) v.lo[s][i] *= m;
                    continue;
                }
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    float& x = INTER ? v.lo[s][2 * i] : v.lo[s][i];
                    float& y = INTER ? v.lo[s][2 * i + 1] : v.hi[s][i];
                    const float rx = (x * c[s][i] - y * sn[s][i]) * m, ry = (x * sn[s][i] + y * c[s][i]) * m;
                    x = rx;
                    y = ry;
                }
            }
        };
        // head h of q (o = 0) or k (o = 1)
        auto one = [&](auto o, const HeadsView& v, int h, Part<E, S>& x, Part<E, S>& g) {
            const Part<E, S>& ww = w[o()];
            float ss = 0.f;
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    ss = fmaf(x.lo[s][i], x.lo[s][i], ss);
                    if (!INTER) ss = fmaf(x.hi[s][i], x.hi[s][i], ss);
                }
            // (the hardware's root is off by one step of fp32 at most)
            const float r = __builtin_amdgcn_rsqf(fmaf(group_sum(ss, lg), inv_d, a.eps));
            T* const out = static_cast<T*>(v.out) + b * v.o_b + h * v.o_h + n * v.o_n;
            if constexpr (!BWD) {
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        x.lo[s][i] *= r * ww.lo[s][i];
                        if (!INTER) x.hi[s][i] *= r * ww.hi[s][i];
                    }
                turn(x, v.scale);
                store(out, x);
            } else {
                turn(g, v.scale);
                float dot = 0.f;
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        x.lo[s][i] *= r;
                        gw[o()].lo[s][i] = fmaf(g.lo[s][i], x.lo[s][i], gw[o()].lo[s][i]);
                        g.lo[s][i] *= ww.lo[s][i];
                        dot = fmaf(g.lo[s][i], x.lo[s][i], dot);
                        if (!INTER) {
                            x.hi[s][i] *= r;
                            gw[o()].hi[s][i] = fmaf(g.hi[s][i], x.hi[s][i], gw[o()].hi[s][i]);
                            g.hi[s][i] *= ww.hi[s][i];
                            dot = fmaf(g.hi[s][i], x.hi[s][i], dot);
                        }
                    }
                const float mean = group_sum(dot, lg) * inv_d;
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        g.lo[s][i] = r * (g.lo[s][i] - x.lo[s][i] * mean);
                        if (!INTER) g.hi[s][i] = r * (g.hi[s][i] - x.hi[s][i] * mean);
                    }
                store(out, g);
            }
        };
        auto walk = [&](auto o, const HeadsView& v, int from, int to) {
            for (int h = from; h < to; h += kFly) {
                Part<E, S> x[kFly], g[BWD ? kFly : 1];
#pragma unroll
                for (int j = 0; j < kFly; ++j) {
                    if (h + j >= to) break;
                    load(static_cast<const T*>(v.x) + b * v.x_b + (h + j) * v.x_h + n * v.x_n, x[j]);
                    if constexpr (BWD) load(static_cast<const T*>(v.gy) + b * v.g_b + (h + j) * v.g_h + n * v.g_n, g[j]);
                }
#pragma unroll
                for (int j = 0; j < kFly; ++j) {
                    if (h + j >= to) break;
                    one(o, v, h + j, x[j], g[BWD ? j : 0]);
                }
            }
        };
        walk(std::integral_constant<int, 0>(), a.q, h1, min(h2, a.q.H));
        walk(std::integral_constant<int, 1>(), a.k, max(h1 - a.q.H, 0), h2 - a.q.H);
    }

    if constexpr (BWD) {
        if (a.part == nullptr) return;
        // the workgroup's rows together, in their order: part[block][q or k][d]
        __shared__ float sums[kThreads];
        float* const out = a.part + (static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 2 * a.d;
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < E; ++i)
#pragma unroll
                    for (int z = 0; z < (INTER ? 1 : 2); ++z) {
                        __syncthreads();
                        sums[threadIdx.x] = z ? gw[o].hi[s][i] : gw[o].lo[s][i];
                        __syncthreads();
                        if (threadIdx.x >= static_cast<unsigned>(lg)) continue;
                        if (z ? !(turns[s] && live[s]) : !has(s, i)) continue;
                        float t = 0.f;
                        for (int k = threadIdx.x; k < kThreads; k += lg) t += sums[k];
                        out[o * a.d + e0[s] + i + (z ? half : 0)] = t;
                    }
    }
}

struct HeadsPlan {
    bool packs;
    int lg, per, rows;
    size_t groups, blocks;
};
HeadsPlan heads_plan(const HeadsArgs& a) {
    HeadsPlan p;
    const int V = a.bf16 ? 8 : 4, rest = a.d - a.rot;
    const int part = a.interleaved ? a.rot : a.rot / 2;
    p.packs = part % V == 0 && rest % V == 0;
    const int units = part / V + rest / V;
    p.lg = p.packs ? 1 : 64;
    while (p.packs && p.lg < units) p.lg *= 2;
    p.rows = kThreads / p.lg;
    const size_t tokens = static_cast<size_t>(a.B) * a.N;
    const int heads = a.q.H + a.k.H;
    // as many heads a thread as leave enough threads to fill the chip
    p.per = 16;
    while (p.per > 1 && tokens * p.lg * ((heads + p.per - 1) / p.per) < kWantThreads) p.per /= 2;
    while (a.backward && (heads + p.per - 1) / p.per > kMaxBlocks) p.per *= 2;
    p.groups = heads == 0 ? 0 : (tokens + p.rows - 1) / p.rows;
    const size_t ys = (heads + p.per - 1) / p.per;
    p.blocks = std::max<size_t>(1, std::min<size_t>(p.groups, kMaxBlocks / std::max<size_t>(ys, 1)));
    return p;
}

template <typename T, typename W, bool INTER, bool BWD>
hipError_t launch_typed(const HeadsArgs& a, hipStream_t st) {
    const HeadsPlan p = heads_plan(a);
    const size_t tokens = static_cast<size_t>(a.B) * a.N;
    const unsigned ys = static_cast<unsigned>((a.q.H + a.k.H + p.per - 1) / p.per);
    constexpr int V = kPack<T>;
    const size_t step = BWD ? p.groups : kMostGroups;
    {
        ProfScope prof(kProfHeads, st);
        for (size_t g = 0; g < p.groups; g += step) {
            const size_t now = BWD ? p.blocks : std::min(p.groups - g, step);
            const size_t end = std::min(tokens, (g + step) * p.rows);
            const dim3 grid(static_cast<unsigned>(now), ys), block(kThreads);
            if (p.packs)
                hipLaunchKernelGGL((heads_kernel<T, W, INTER, V, 1, BWD>), grid, block, 0, st, a, g * p.rows, end, p.lg, p.per);
            else
                hipLaunchKernelGGL((heads_kernel<T, W, INTER, INTER ? 2 : 1, 4, BWD>), grid, block, 0, st, a, g * p.rows, end,
                                   p.lg, p.per);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    if (!BWD || a.part == nullptr) return hipSuccess;
    ColReduceArgs c{};
    c.in = a.part;
    c.P = p.groups == 0 ? 0 : static_cast<int>(p.blocks * ys);
    c.rows = 2;
    c.K = 0;
    c.D = a.d;
    c.out1 = a.q.gw;
    c.out2 = a.k.gw;
    c.out_bf16 = sizeof(W) == 2;
    return launch_col_reduce(c, st);
}

template <typename T, typename W>
hipError_t launch_way(const HeadsArgs& a, hipStream_t st) {
    if (a.backward) return a.interleaved ? launch_typed<T, W, true, true>(a, st) : launch_typed<T, W, false, true>(a, st);
    return a.interleaved ? launch_typed<T, W, true, false>(a, st) : launch_typed<T, W, false, false>(a, st);
}

}  // namespace

size_t heads_partial_bytes(int d) { return static_cast<size_t>(kMaxBlocks) * 2 * d * sizeof(float); }

hipError_t launch_heads(const HeadsArgs& a, hipStream_t st) {
    if (!a.bf16) return launch_way<float, float>(a, st);
    return a.w_bf16 ? launch_way<bf16_t, bf16_t>(a, st) : launch_way<bf16_t, float>(a, st);
}

}  // namespace retn
