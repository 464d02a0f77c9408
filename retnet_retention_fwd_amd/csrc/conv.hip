// Short causal convolution of each channel over its last K tokens (K = 2, 3, 4), the step
// in front of the selective scan, with an optional silu behind it.  With the incoming state
// xs = [state_in (K-1 rows) ; x (N rows)]:
//     pre_t = bias + sum_j w_j xs_(t+j),   y = pre or silu(pre),   state_out = xs_(N .. N+K-2)
//     dpre = gy silu'(pre),   dxs_i = sum_j w_j dpre_(i-j)  (+ grad_state_out_(i-N)),
//     dw_j = sum_t dpre_t xs_(t+j),   dbias = sum_t dpre_t
//
// Bound by HBM: a few operations per element.  A thread owns one 16-byte pack of channels
// and walks over tokens with the last K rows in registers, so a row is read once (plus K-1
// rows where a walk begins); neighbouring lanes own neighbouring channels.  The backward
// walks in the same direction: behind token s it knows dpre_(s-K+1 .. s), which is what row
// s-K+1 of the gradient needs, so it reads x and gy once too and keeps its channels' weight
// sums in registers until the end of the walk.

#include "block.h"
#include "launch.h"
#include "vec_io.h"

namespace retn {

namespace {

constexpr int kThreads = 256;
constexpr int kWalkBwd = 32;    // tokens of a backward walk
constexpr int kAhead = 8;       // rows loaded together

__device__ __forceinline__ int length_of(const int* lengths, int b, int N) {
    if (lengths == nullptr) return N;
    const int n = lengths[b];
    return n < 0 ? 0 : n < N ? n : N;
}

// Weights [D, K] of V adjacent channels, zeros behind the last channel.
template <typename W, int V, int K>
__device__ __forceinline__ void load_weights(const W* w, int c, int D, float (&out)[K][V]) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < K; ++j) out[j][i] = c + i < D ? up(w[static_cast<size_t>(c + i) * K + j]) : 0.f;
}

// Row t of xs without the K-1 state rows counted: t < 0 is a state row.
template <typename T, int V, int K>
__device__ __forceinline__ Raw<T, V> row(const ConvArgs& a, int b, long long t, int c) {
    if (t >= 0) return raw_load_n<T, V>(static_cast<const T*>(a.x) + (static_cast<size_t>(b) * a.N + t) * a.ldx + c, a.D - c);
    if (a.state_in == nullptr) return Raw<T, V>{};
    return raw_load_n<T, V>(static_cast<const T*>(a.state_in) + (static_cast<size_t>(b) * (K - 1) + K - 1 + t) * a.D + c,
                            a.D - c);
}

template <typename T, typename W, int K, int TT>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(ConvArgs a, int packs, int tiles) {
    constexpr int V = kPack<T>;
    const size_t id = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int c = static_cast<int>(id % packs) * V;
    const size_t bt = id / packs;
    const int b = static_cast<int>(bt / tiles), tile = static_cast<int>(bt % tiles);
    if (b >= a.B) return;
    const int n = length_of(a.lengths, b, a.N), t0 = tile * TT, left = a.D - c;
    const bool last = tile == (n > 0 ? (n - 1) / TT : 0);
    if (t0 >= n && !last) return;
    Raw<T, V> xs[TT + K - 1];
#pragma unroll
    for (int i = 0; i < TT + K - 1; ++i) {
        xs[i] = Raw<T, V>{};
        if (t0 + i - (K - 1) < n) xs[i] = row<T, V, K>(a, b, t0 + i - (K - 1), c);
    }
    float w[K][V], bias[V];
    load_weights<W, V, K>(static_cast<const W*>(a.w), c, a.D, w);
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = a.b != nullptr && i < left ? up(static_cast<const W*>(a.b)[c + i]) : 0.f;
    T* y = static_cast<T*>(a.y) + (static_cast<size_t>(b) * a.N + t0) * a.D + c;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        if (t0 + t >= n) continue;
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            o[i] = bias[i];
#pragma unroll
            for (int j = 0; j < K; ++j) o[i] = fmaf(w[j][i], up(xs[t + j].v[i]), o[i]);
            if (a.silu) o[i] *= sigmoid_f(o[i]);
        }
        store_n<T, V>(y + static_cast<size_t>(t) * a.D, o, left);
    }
    if (last && a.state_out != nullptr) {
        T* s = static_cast<T*>(a.state_out) + static_cast<size_t>(b) * (K - 1) * a.D + c;
#pragma unroll
        for (int r = 0; r < K - 1; ++r)
            raw_store_n<T, V>(s + static_cast<size_t>(r) * a.D, row<T, V, K>(a, b, static_cast<long long>(n) + r - (K - 1), c),
                              left);
    }
}

// One token: the state's rows move up by one, the new row comes last.
template <typename T, typename W, int K>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(ConvArgs a, int packs) {
    constexpr int V = kPack<T>;
    const size_t id = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int c = static_cast<int>(id % packs) * V, b = static_cast<int>(id / packs);
    if (b >= a.B) return;
    const int left = a.D - c;
    T* s = static_cast<T*>(a.state_out) + static_cast<size_t>(b) * (K - 1) * a.D + c;
    Raw<T, V> xs[K];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) xs[j] = raw_load_n<T, V>(s + static_cast<size_t>(j) * a.D, left);
    xs[K - 1] = raw_load_n<T, V>(static_cast<const T*>(a.x) + b * a.ldx + c, left);
    float w[K][V], o[V];
    load_weights<W, V, K>(static_cast<const W*>(a.w), c, a.D, w);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        o[i] = a.b != nullptr && i < left ? up(static_cast<const W*>(a.b)[c + i]) : 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) o[i] = fmaf(w[j][i], up(xs[j].v[i]), o[i]);
        if (a.silu) o[i] *= sigmoid_f(o[i]);
    }
    store_n<T, V>(static_cast<T*>(a.y) + static_cast<size_t>(b) * a.D + c, o, left);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) raw_store_n<T, V>(s + static_cast<size_t>(j) * a.D, xs[j + 1], left);
}

// `wide` lanes own packs, kThreads / wide walks of kWalkBwd tokens share a workgroup, which
// adds their weight sums through LDS and leaves them as [workgroup][K+1][D].
template <typename T, typename W, int K>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(ConvArgs a, int wide, int tiles, int across) {
    constexpr int V = kPack<T>;
    __shared__ float sums[kThreads * V];
    const int lane = threadIdx.x % wide, walk = threadIdx.x / wide, walks = kThreads / wide;
    const int blk = blockIdx.x % across, bt = blockIdx.x / across;   // channels, then (sequence, tile)
    const int c = (blk * wide + lane) * V, left = a.D - c;
    const int b = bt / tiles, t0 = (bt % tiles * walks + walk) * kWalkBwd;
    const int n = length_of(a.lengths, b, a.N);
    float gw[K][V] = {}, gb[V] = {};
    if (left > 0 && (t0 < a.N || t0 == 0)) {
        float w[K][V], bias[V];
        load_weights<W, V, K>(static_cast<const W*>(a.w), c, a.D, w);
#pragma unroll
        for (int i = 0; i < V; ++i) bias[i] = a.b != nullptr && i < left ? up(static_cast<const W*>(a.b)[c + i]) : 0.f;
        float xs[K][V], dp[K][V];      // rows s-K+1 .. s of xs and of dpre
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) xs[j][i] = dp[j][i] = 0.f;
#pragma unroll
        for (int j = 1; j < K; ++j) {  // the rows before t0, moved down by the first step
            Raw<T, V> r = {};
            if (t0 - K + j < n) r = row<T, V, K>(a, b, t0 - K + j, c);
#pragma unroll
            for (int i = 0; i < V; ++i) xs[j][i] = up(r.v[i]);
        }
        const T* gy = static_cast<const T*>(a.gy) + static_cast<size_t>(b) * a.N * a.D + c;
        T* gx = static_cast<T*>(a.y) + static_cast<size_t>(b) * a.N * a.D + c;
        const int end = (t0 + kWalkBwd < a.N ? t0 + kWalkBwd : a.N);   // rows of gx that are this walk's
        for (int s0 = t0; s0 < end + K - 1; s0 += kAhead) {
            Raw<T, V> rx[kAhead], rg[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                rx[k] = rg[k] = Raw<T, V>{};
                if (s0 + k < n && s0 + k < end + K - 1) {
                    rx[k] = row<T, V, K>(a, b, s0 + k, c);
                    rg[k] = raw_load_n<T, V>(gy + static_cast<size_t>(s0 + k) * a.D, left);
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int s = s0 + k, i0 = s - (K - 1);
                if (s >= end + K - 1) break;
                const bool on = s < n, mine = s < end;
                float gx_row[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
#pragma unroll
                    for (int j = 0; j + 1 < K; ++j) {
                        xs[j][i] = xs[j + 1][i];
                        dp[j][i] = dp[j + 1][i];
                    }
                    xs[K - 1][i] = up(rx[k].v[i]);
                    float pre = bias[i];
#pragma unroll
                    for (int j = 0; j < K; ++j) pre = fmaf(w[j][i], xs[j][i], pre);
                    float g = up(rg[k].v[i]);
                    if (a.silu) {
                        const float sg = sigmoid_f(pre);
                        g *= fmaf(pre * sg, 1.f - sg, sg);
                    }
                    g = on ? g : 0.f;
                    dp[K - 1][i] = g;
                    if (mine) {
                        gb[i] += g;
#pragma unroll
                        for (int j = 0; j < K; ++j) gw[j][i] = fmaf(g, xs[j][i], gw[j][i]);
                    }
                    float r = 0.f;
#pragma unroll
                    for (int j = 0; j < K; ++j) r = fmaf(w[j][i], dp[K - 1 - j][i], r);
                    gx_row[i] = r;
                }
                // row i0 of the gradient of xs: a token's, or (t0 = 0) a state row's
                if (i0 < t0 && t0 > 0) continue;
                if (a.gstate_out != nullptr && s >= n && i0 < n) {
                    const Raw<T, V> r = raw_load_n<T, V>(
                        static_cast<const T*>(a.gstate_out) + (static_cast<size_t>(b) * (K - 1) + s - n) * a.D + c, left);
#pragma unroll
                    for (int i = 0; i < V; ++i) gx_row[i] += up(r.v[i]);
                }
                if (i0 >= 0) {
                    if (i0 < end) store_n<T, V>(gx + static_cast<size_t>(i0) * a.D, gx_row, left);
                } else if (a.gstate_in != nullptr) {
                    store_n<T, V>(static_cast<T*>(a.gstate_in) + (static_cast<size_t>(b) * (K - 1) + s) * a.D + c, gx_row, left);
                }
            }
        }
    }
    if (a.workspace == nullptr) return;
    float* out = a.workspace + static_cast<size_t>(bt) * (K + 1) * a.D;
#pragma unroll
    for (int j = 0; j <= K; ++j) {
#pragma unroll
        for (int i = 0; i < V; ++i) sums[threadIdx.x * V + i] = j < K ? gw[j < K ? j : 0][i] : gb[i];
        __syncthreads();
        for (int e = threadIdx.x; e < wide * V; e += kThreads) {
            const int col = blk * wide * V + e;
            float t = 0.f;
            for (int k = 0; k < walks; ++k) t += sums[k * wide * V + e];
            if (col < a.D) out[static_cast<size_t>(j) * a.D + col] = t;
        }
        __syncthreads();
    }
}

int packs_of(int D, bool bf16) { return bf16 ? (D + 7) / 8 : (D + 3) / 4; }
// Lanes across the channels: enough for all of them up to a wave.
int bwd_wide(int D, bool bf16) {
    int w = 8;
    while (w < 64 && w < packs_of(D, bf16)) w *= 2;
    return w;
}
int bwd_tiles(int N, int D, bool bf16) {
    const int tokens = kThreads / bwd_wide(D, bf16) * kWalkBwd;
    return N > 0 ? (N - 1) / tokens + 1 : 1;
}

template <typename T, typename W, int K>
hipError_t fwd_k(const ConvArgs& a, hipStream_t st) {
    const int packs = packs_of(a.D, a.bf16);
    const dim3 block(kThreads);
    ProfScope prof(kProfConv, st);
    // 16 tokens a thread while that leaves 4 waves a SIMD, else 4: a walk of 16 reads 3/16
    // more rows than it writes, a walk of 4 fills the chip with a sixteenth of the work
    const size_t want = static_cast<size_t>(1024) * 4 * 64;
    if (static_cast<size_t>(a.B) * packs * ((a.N + 15) / 16) >= want) {
        const int tiles = (a.N + 15) / 16;
        const size_t n = static_cast<size_t>(a.B) * tiles * packs;
        hipLaunchKernelGGL((conv_fwd_kernel<T, W, K, 16>), dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads)), block,
                           0, st, a, packs, tiles);
    } else {
        const int tiles = a.N > 0 ? (a.N - 1) / 4 + 1 : 1;
        const size_t n = static_cast<size_t>(a.B) * tiles * packs;
        hipLaunchKernelGGL((conv_fwd_kernel<T, W, K, 4>), dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads)), block, 0,
                           st, a, packs, tiles);
    }
    return hipGetLastError();
}

template <typename T, typename W, int K>
hipError_t step_k(const ConvArgs& a, hipStream_t st) {
    const int packs = packs_of(a.D, a.bf16);
    const size_t n = static_cast<size_t>(a.B) * packs;
    ProfScope prof(kProfConv, st);
    hipLaunchKernelGGL((conv_step_kernel<T, W, K>), dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads)), dim3(kThreads),
                       0, st, a, packs);
    return hipGetLastError();
}

template <typename T, typename W, int K>
hipError_t bwd_k(const ConvArgs& a, hipStream_t st) {
    const int wide = bwd_wide(a.D, a.bf16), tiles = bwd_tiles(a.N, a.D, a.bf16), packs = packs_of(a.D, a.bf16);
    if (a.B > 0) {
        ProfScope prof(kProfConv, st);
        const int across = (packs + wide - 1) / wide;
        hipLaunchKernelGGL((conv_bwd_kernel<T, W, K>), dim3(static_cast<unsigned>(across) * a.B * tiles), dim3(kThreads), 0,
                           st, a, wide, tiles, across);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.gw == nullptr && a.gb == nullptr) return hipSuccess;
    const ColReduceArgs c{a.workspace, a.B * tiles, K + 1, K, a.D, a.gw, a.gb, nullptr, a.w_bf16};
    return launch_col_reduce(c, st);
}

enum Way { kFwd, kStep, kBwd };
template <typename T, typename W, int K>
hipError_t go_k(const ConvArgs& a, Way way, hipStream_t st) {
    return way == kFwd ? fwd_k<T, W, K>(a, st) : way == kStep ? step_k<T, W, K>(a, st) : bwd_k<T, W, K>(a, st);
}
template <typename T, typename W>
hipError_t go_typed(const ConvArgs& a, Way way, hipStream_t st) {
    return a.K == 2 ? go_k<T, W, 2>(a, way, st) : a.K == 3 ? go_k<T, W, 3>(a, way, st) : go_k<T, W, 4>(a, way, st);
}
hipError_t go(const ConvArgs& a, Way way, hipStream_t st) {
    if (!a.bf16) return go_typed<float, float>(a, way, st);
    return a.w_bf16 ? go_typed<bf16_t, bf16_t>(a, way, st) : go_typed<bf16_t, float>(a, way, st);
}

}  // namespace

size_t conv_bwd_workspace(int B, int N, int D, int K, bool bf16) {
    return static_cast<size_t>(B) * bwd_tiles(N, D, bf16) * (K + 1) * D * sizeof(float);
}
hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t st) { return go(a, kFwd, st); }
hipError_t launch_conv_step(const ConvArgs& a, hipStream_t st) { return go(a, kStep, st); }
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t st) { return go(a, kBwd, st); }

}  // namespace retn
