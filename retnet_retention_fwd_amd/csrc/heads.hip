// Root-mean-square norm of each head's row of queries and keys with rotary positions:
//     r = 1 / sqrt(mean(x^2) + eps),   out = scale turn(x r w)
// and the gradient: with g = scale turn^T(grad), xh = x r, v = g w,
//     gx = r (v - xh mean(v xh)),   gw = sum over all rows of g xh.
//
// Bound by HBM: each row is read once (twice for the gradient: x and grad) and written once.  A
// row lies over a group of LG lanes, a power of two, each with one 16-byte pack, or one in each
// half of the rotated part (and of what is behind it) where pairs are (i, i + rot/2), so that a
// lane holds both elements of its pairs and the row's sum is a few lane exchanges.  A lane walks over the heads of its
// token with the cosines, the sines and both weights in registers, four heads' loads in flight.
// Heads whose parts are not whole packs take single pairs, four a lane of a whole wave.
//
// Measured: 277 MB of bf16 q and k (16384 tokens, 16 + 16 heads of 128) in 56 to 59 us (4.7 to 4.9 TB/s); gradients
// of 4 x 2048 tokens, 8 + 8 heads of 128, half of them turning (101 MB), in 32 us and 4 for the
// weights' sums: there the vector ALUs' work and the loads' latency count, at two waves a SIMD.

#include "common.h"
#include "launch.h"
#include "proj.h"
#include "vec_io.h"

#include <algorithm>

namespace retn {
namespace {

constexpr int kThreads = 256;
constexpr size_t kWantThreads = 1 << 18;   // 16 waves of 64 for each of 256 CUs
constexpr int kMaxBlocks = 1024;           // of the gradient: each leaves d partial sums
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
// The same as it lies in memory.
template <typename T, int E, int S>
struct Packs {
    Raw<T, E> lo[S], hi[S];
};

// E: adjacent elements of a unit, S: units of a lane.  S = 1: packs; S = 4: single pairs, where a
// unit behind the rotated part is one element.
// A workgroup takes heads of q or of k: blockIdx.y counts through q's, then k's, heads_per each.
template <typename T, typename W, bool INTER, int E, int S, bool BWD>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadsArgs a, size_t tok0, size_t tokens, int lg, int heads_per) {
    constexpr bool kOne = S > 1;                     // single elements behind the rotated part
    constexpr int kPairs = INTER ? E / 2 : E;
    constexpr int kFly = kOne ? 1 : BWD && !INTER ? 2 : 4;     // heads whose loads are in flight together
    const int yq = (a.q.H + heads_per - 1) / heads_per;
    const bool isk = static_cast<int>(blockIdx.y) >= yq;
    const HeadsView v = isk ? a.k : a.q;
    const int h1 = (static_cast<int>(blockIdx.y) - (isk ? yq : 0)) * heads_per, h2 = min(h1 + heads_per, v.H);
    const int sub = threadIdx.x & (lg - 1), rows = kThreads / lg;
    const int turning = INTER ? a.rot / E : a.rot / 2 / E;
    const int rest_e = kOne ? 1 : E, rest = (a.d - a.rot) / rest_e;   // units behind the rotated part,
    const int behind = INTER ? rest : (rest + 1) / 2;                 // in halves too, the second may be one less
    int e0[S], ho[S];                                // first element of a unit, way to its second one
    bool turns[S], live[S], two[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int u = sub + s * lg;
        live[s] = u < turning + behind;
        turns[s] = u < turning;
        e0[s] = turns[s] ? u * E : a.rot + (u - turning) * rest_e;
        ho[s] = turns[s] ? a.rot / 2 : behind * rest_e;
        two[s] = !INTER && live[s] && (turns[s] || u - turning + behind < rest);
    }
    // elements s, i of a unit exist: behind the rotated part of single pairs only the first
    auto has = [&](int s, int i) { return live[s] && (!kOne || turns[s] || i == 0); };
    auto load = [&](const T* p, Packs<T, E, S>& v) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            v.lo[s] = v.hi[s] = Raw<T, E>{};
            if constexpr (kOne) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    if (has(s, i)) v.lo[s].v[i] = p[e0[s] + i];
                    if (two[s]) v.hi[s].v[i] = p[e0[s] + ho[s] + i];
                }
            } else {
                if (live[s]) v.lo[s] = raw_load<T, E>(p + e0[s]);
                if (two[s]) v.hi[s] = raw_load<T, E>(p + e0[s] + ho[s]);
            }
        }
    };
    auto open = [&](const Packs<T, E, S>& r, Part<E, S>& v) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < E; ++i) {
                v.lo[s][i] = up(r.lo[s].v[i]);
                v.hi[s][i] = INTER ? 0.f : up(r.hi[s].v[i]);
            }
    };
    auto store = [&](T* p, const Part<E, S>& v) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if constexpr (kOne) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    if (has(s, i)) p[e0[s] + i] = down<T>(v.lo[s][i]);
                    if (two[s]) p[e0[s] + ho[s] + i] = down<T>(v.hi[s][i]);
                }
            } else {
                if (live[s]) store_n<T, E>(p + e0[s], v.lo[s], E);
                if (two[s]) store_n<T, E>(p + e0[s] + ho[s], v.hi[s], E);
            }
        }
    };
    // the weights, in the places of the elements
    Part<E, S> w, gw;
    {
        const W* p = static_cast<const W*>(v.w);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            Raw<W, E> lo{}, hi{};
            if (p != nullptr) {
                if constexpr (kOne) {
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        if (has(s, i)) lo.v[i] = p[e0[s] + i];
                } else if (live[s]) {
                    lo = raw_load<W, E>(p + e0[s]);
                }
                if (two[s]) hi = raw_load<W, E>(p + e0[s] + ho[s]);
            }
#pragma unroll
            for (int i = 0; i < E; ++i) {
                w.lo[s][i] = p == nullptr ? 1.f : up(lo.v[i]);
                w.hi[s][i] = p == nullptr ? 1.f : up(hi.v[i]);
                gw.lo[s][i] = gw.hi[s][i] = 0.f;
            }
        }
    }
    const float inv_d = 1.f / a.d;

    // one trip a workgroup in the forward; the gradient's workgroups walk over the tokens
    for (size_t tok = tok0 + static_cast<size_t>(blockIdx.x) * rows + threadIdx.x / lg; tok < tokens;
         tok += static_cast<size_t>(gridDim.x) * rows) {
        const unsigned t32 = static_cast<unsigned>(tok);            // (below 2^31)
        const int b = t32 / static_cast<unsigned>(a.N), n = t32 % static_cast<unsigned>(a.N);
        float c[S][kPairs], sn[S][kPairs];
        {
            const long long p = a.pos != nullptr ? a.pos[a.pos_batched ? tok : static_cast<size_t>(n)] : a.first + n;
            const bool known = p >= 0 && p < a.table_len;
            const float nan = __builtin_nanf("");
#pragma unroll
            for (int s = 0; s < S; ++s) {
                Raw<float, 2 * kPairs> t{};
                if (turns[s]) t = raw_load<float, 2 * kPairs>(a.table + (known ? p : 0) * a.rot + 2 * (INTER ? e0[s] / 2 : e0[s]));
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    c[s][i] = known ? t.v[2 * i] : nan;
                    sn[s][i] = known ? (BWD ? -t.v[2 * i + 1] : t.v[2 * i + 1]) : nan;
                }
            }
        }
        auto turn = [&](Part<E, S>& v, float m) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if (!turns[s]) {
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        v.lo[s][i] *= m;
                        v.hi[s][i] *= m;
                    }
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
        auto one = [&](int h, Part<E, S>& x, Part<E, S>& g) {
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
                        x.lo[s][i] *= r * w.lo[s][i];
                        if (!INTER) x.hi[s][i] *= r * w.hi[s][i];
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
                        gw.lo[s][i] = fmaf(g.lo[s][i], x.lo[s][i], gw.lo[s][i]);
                        g.lo[s][i] *= w.lo[s][i];
                        dot = fmaf(g.lo[s][i], x.lo[s][i], dot);
                        if (!INTER) {
                            x.hi[s][i] *= r;
                            gw.hi[s][i] = fmaf(g.hi[s][i], x.hi[s][i], gw.hi[s][i]);
                            g.hi[s][i] *= w.hi[s][i];
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
        for (int h = h1; h < h2; h += kFly) {
            Packs<T, E, S> x[kFly], g[BWD ? kFly : 1];
#pragma unroll
            for (int j = 0; j < kFly; ++j) {
                if (h + j >= h2) break;
                load(static_cast<const T*>(v.x) + b * v.x_b + (h + j) * v.x_h + n * v.x_n, x[j]);
                if constexpr (BWD) load(static_cast<const T*>(v.gy) + b * v.g_b + (h + j) * v.g_h + n * v.g_n, g[j]);
            }
#pragma unroll
            for (int j = 0; j < kFly; ++j) {
                if (h + j >= h2) break;
                Part<E, S> xf, gf;
                open(x[j], xf);
                if constexpr (BWD) open(g[j], gf);
                one(h + j, xf, gf);
            }
        }
    }

    if constexpr (BWD) {
        if (a.part == nullptr) return;
        // the workgroup's rows together: a wave's by lane exchanges, then the waves' in their order
        __shared__ float sums[kThreads / 64][256];
        const int wave = threadIdx.x >> 6;
        auto put = [&](float t, bool on, int e) {
            for (int m = lg; m < 64; m *= 2) t += __shfl_xor(t, m, 64);
            if (on && (threadIdx.x & 63) < static_cast<unsigned>(lg)) sums[wave][e] = t;
        };
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < E; ++i) {
                put(gw.lo[s][i], has(s, i), e0[s] + i);
                if (!INTER) put(gw.hi[s][i], two[s], e0[s] + ho[s] + i);
            }
        __syncthreads();
        float* const out = a.part + (static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * a.d;
        for (int e = threadIdx.x; e < a.d; e += kThreads) out[e] = (sums[0][e] + sums[1][e]) + (sums[2][e] + sums[3][e]);
    }
}

// The weights' gradients from the workgroups' sums: rows 0 .. P[0] - 1 of q, P[1] behind them of k.
template <typename W>
__global__ __launch_bounds__(1024) void heads_sum_kernel(const float* part, int P0, int P1, int d, void* gq, void* gk) {
    __shared__ float sums[16][64];
    const int c = threadIdx.x & 63, g = threadIdx.x >> 6, col = blockIdx.x * 64 + c;
    const bool isk = blockIdx.y != 0;
    const float* in = part + (isk ? static_cast<size_t>(P0) * d : 0);
    const int P = isk ? P1 : P0;
    W* const out = static_cast<W*>(isk ? gk : gq);
    float s = 0.f;
    if (col < d) {
#pragma unroll 8
        for (int p = g; p < P; p += 16) s += in[static_cast<size_t>(p) * d + col];
    }
    sums[g][c] = s;
    __syncthreads();
    if (g != 0 || col >= d || out == nullptr) return;
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sums[i][c];
    out[col] = down<W>(t);
}

struct HeadsPlan {
    bool packs;
    int lg, per, rows, yq, yk;
    size_t groups, blocks;
};
HeadsPlan heads_plan(const HeadsArgs& a) {
    HeadsPlan p;
    const int V = a.bf16 ? 8 : 4, rest = a.d - a.rot;
    const int part = a.interleaved ? a.rot : a.rot / 2;
    p.packs = part % V == 0 && rest % V == 0;
    const int units = part / V + (a.interleaved ? rest / V : (rest / V + 1) / 2);
    p.lg = p.packs ? 1 : 64;
    while (p.packs && p.lg < units) p.lg *= 2;
    p.rows = kThreads / p.lg;
    const size_t tokens = static_cast<size_t>(a.B) * a.N;
    auto cut = [&](int per) {
        p.per = per;
        p.yq = (a.q.H + per - 1) / per;
        p.yk = (a.k.H + per - 1) / per;
    };
    // as many heads a thread as leave enough threads to fill the chip
    cut(16);
    while (p.per > 1 && tokens * p.lg * (p.yq + p.yk) < kWantThreads) cut(p.per / 2);
    while (a.backward && p.yq + p.yk > kMaxBlocks) cut(p.per * 2);
    p.groups = p.yq + p.yk == 0 ? 0 : (tokens + p.rows - 1) / p.rows;
    p.blocks = std::max<size_t>(1, std::min<size_t>(p.groups, kMaxBlocks / std::max(1, p.yq + p.yk)));
    return p;
}

template <typename T, typename W, bool INTER, bool BWD>
hipError_t launch_typed(const HeadsArgs& a, hipStream_t st) {
    const HeadsPlan p = heads_plan(a);
    const size_t tokens = static_cast<size_t>(a.B) * a.N;
    const unsigned ys = static_cast<unsigned>(p.yq + p.yk);
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
    const int blocks = p.groups == 0 ? 0 : static_cast<int>(p.blocks);
    ProfScope prof(kProfReduce, st);
    hipLaunchKernelGGL((heads_sum_kernel<W>), dim3((a.d + 63) / 64, 2), dim3(1024), 0, st, a.part, blocks * p.yq, blocks * p.yk,
                       a.d, a.q.gw, a.k.gw);
    return hipGetLastError();
}

template <typename T, typename W>
hipError_t launch_way(const HeadsArgs& a, hipStream_t st) {
    if (a.backward) return a.interleaved ? launch_typed<T, W, true, true>(a, st) : launch_typed<T, W, false, true>(a, st);
    return a.interleaved ? launch_typed<T, W, true, false>(a, st) : launch_typed<T, W, false, false>(a, st);
}

}  // namespace

size_t heads_partial_bytes(int d) { return static_cast<size_t>(kMaxBlocks) * d * sizeof(float); }

hipError_t launch_heads(const HeadsArgs& a, hipStream_t st) {
    if (!a.bf16) return launch_way<float, float>(a, st);
    return a.w_bf16 ? launch_way<bf16_t, bf16_t>(a, st) : launch_way<bf16_t, float>(a, st);
}

}  // namespace retn
