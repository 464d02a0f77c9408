// Short causal convolution of each channel over its last K tokens (K = 2, 3, 4), the step
// in front of the selective scan, with an optional silu behind it.  With the incoming state
// xs = [state_in (K-1 rows) ; x (N rows)]:
//     pre_t = bias + sum_j w_j xs_(t+j),   y = pre or silu(pre),   state_out = xs_(N .. N+K-2)
//     dpre = gy silu'(pre),   dxs_i = sum_j w_j dpre_(i-j)  (+ grad_state_out_(i-N)),
//     dw_j = sum_t dpre_t xs_(t+j),   dbias = sum_t dpre_t
//
// Bound by HBM: a few operations per element.  A thread owns four adjacent channels and walks
// over tokens with the last K rows in registers, so a row is read once (plus K-1 rows where
// a walk begins); neighbouring lanes own neighbouring channels.  Four rows are in flight
// while four are worked on, and few registers a thread keep many waves in flight (with eight
// channels a thread the training gradient took 70 us instead).  The backward walks in the
// same direction: behind token s it knows dpre_(s-K+1 .. s), which is what row s-K+1 of the
// gradient needs, so it reads x and gy once too and keeps its channels' weight sums in
// registers until the end of the walk.
//
// Measured, bf16: forward of 2 x 8191 x 2048 channels 29.5 us for 134 MB (4.6 TB/s), 23 us for the
// 110 MB of padded sequences with 64% of these tokens, the zeros behind them written; backward
// of 4 x 2048 x 2048 31 us for 101 MB (3.3 TB/s; the launch of the sums is 4 of them; the vector ALUs
// are 55% busy with silu and its derivative).  Its walks of 32 tokens bring two waves a SIMD where
// registers allow three: walks of 24, 22 and 16 tokens bring more, read more rows twice and leave
// more partial sums, and take 33.7, 34.2 and 36.4 us (fp32 53 us with 32 tokens, 57 to 65 with those).

#include "block.h"
#include "launch.h"
#include "vec_io.h"

namespace retn {

namespace {

constexpr int kThreads = 256;
constexpr int V = 4;            // channels of a thread
constexpr int kRows = 4;        // rows loaded together
constexpr int kWalkBwd = 32;    // tokens of a backward walk

__device__ __forceinline__ int length_of(const int* lengths, int b, int N) {
    if (lengths == nullptr) return N;
    const int n = lengths[b];
    return n < 0 ? 0 : n < N ? n : N;
}

// Weights [D, K] of V adjacent channels, zeros behind the last channel.
template <typename W, int K>
__device__ __forceinline__ void load_weights(const W* w, int c, int D, float (&out)[K][V]) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < K; ++j) out[j][i] = c + i < D ? up(w[static_cast<size_t>(c + i) * K + j]) : 0.f;
}
template <typename W>
__device__ __forceinline__ void load_bias(const W* b, int c, int D, float (&out)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = b != nullptr && c + i < D ? up(b[c + i]) : 0.f;
}

// V channels of a row; WHOLE: the channels are a multiple of V, so no pack is cut.
template <typename T, bool WHOLE>
__device__ __forceinline__ Raw<T, V> pack(const T* p, int left) {
    return raw_load_n<T, V>(p, WHOLE ? V : left);
}
template <typename T, bool WHOLE>
__device__ __forceinline__ void put(T* p, const float (&v)[V], int left, bool stream) {
    store_n<T, V>(p, v, WHOLE ? V : left, stream);
}

// Row t of xs without the K-1 state rows counted: t < 0 is a state row.
template <typename T, int K, bool WHOLE>
__device__ __forceinline__ Raw<T, V> row(const ConvArgs& a, int b, long long t, int c) {
    if (t >= 0) return pack<T, WHOLE>(static_cast<const T*>(a.x) + (static_cast<size_t>(b) * a.N + t) * a.ldx + c, a.D - c);
    if (a.state_in == nullptr) return Raw<T, V>{};
    return pack<T, WHOLE>(static_cast<const T*>(a.state_in) + (static_cast<size_t>(b) * (K - 1) + K - 1 + t) * a.D + c, a.D - c);
}

template <typename T, typename W, int K, bool WHOLE>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(ConvArgs a, int packs, int tiles, int walk) {
    const size_t id = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int c = static_cast<int>(id % packs) * V;
    const size_t bt = id / packs;
    const int b = static_cast<int>(bt / tiles), tile = static_cast<int>(bt % tiles);
    if (b >= a.B) return;
    const int n = length_of(a.lengths, b, a.N), t0 = tile * walk, left = a.D - c;
    const bool last = tile == (n > 0 ? (n - 1) / walk : 0);
    if (a.zero_behind) {
        // this walk's rows behind the sequence's last token
        const int end = t0 + walk < a.N ? t0 + walk : a.N;
        const float zero[V] = {};
        for (int t = t0 > n ? t0 : n; t < end; ++t)
            put<T, WHOLE>(static_cast<T*>(a.y) + (static_cast<size_t>(b) * a.N + t) * a.D + c, zero, left, false);
    }
    if (t0 < n) {
        const int end = t0 + walk < n ? t0 + walk : n;
        const T* x = static_cast<const T*>(a.x) + static_cast<size_t>(b) * a.N * a.ldx + c;
        T* y = static_cast<T*>(a.y) + (static_cast<size_t>(b) * a.N + t0) * a.D + c;
        Raw<T, V> next[kRows];
        // rows behind the walk's end are not needed: the last one is read again instead
        auto fetch = [&](int t) {
#pragma unroll
            for (int k = 0; k < kRows; ++k)
                next[k] = pack<T, WHOLE>(x + static_cast<size_t>(t + k < end ? t + k : end - 1) * a.ldx, left);
        };
        fetch(t0);
        float w[K][V], bias[V], xs[K + kRows - 1][V];
        load_weights<W, K>(static_cast<const W*>(a.w), c, a.D, w);
        load_bias<W>(static_cast<const W*>(a.b), c, a.D, bias);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const Raw<T, V> r = row<T, K, WHOLE>(a, b, static_cast<long long>(t0) - (K - 1) + j, c);
#pragma unroll
            for (int i = 0; i < V; ++i) xs[j][i] = up(r.v[i]);
        }
        for (int t = t0; t < end; t += kRows) {
#pragma unroll
            for (int k = 0; k < kRows; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) xs[K - 1 + k][i] = up(next[k].v[i]);
            if (t + kRows < end) fetch(t + kRows);
            float o[kRows][V];
#pragma unroll
            for (int k = 0; k < kRows; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    o[k][i] = bias[i];
#pragma unroll
                    for (int j = 0; j < K; ++j) o[k][i] = fmaf(w[j][i], xs[k + j][i], o[k][i]);
                }
            if (a.silu) {
#pragma unroll
                for (int k = 0; k < kRows; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) o[k][i] *= sigmoid_f(o[k][i]);
            }
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                if (t + k < end) put<T, WHOLE>(y, o[k], left, false);
                y += a.D;
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) xs[j][i] = xs[j + kRows][i];
        }
    }
    if (last && a.state_out != nullptr) {
        T* s = static_cast<T*>(a.state_out) + static_cast<size_t>(b) * (K - 1) * a.D + c;
#pragma unroll
        for (int r = 0; r < K - 1; ++r)
            raw_store_n<T, V>(s + static_cast<size_t>(r) * a.D,
                              row<T, K, WHOLE>(a, b, static_cast<long long>(n) + r - (K - 1), c), left);
    }
}

// One token: the state's rows move up by one, the new row comes last.
template <typename T, typename W, int K>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(ConvArgs a, int packs) {
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
    load_weights<W, K>(static_cast<const W*>(a.w), c, a.D, w);
    load_bias<W>(static_cast<const W*>(a.b), c, a.D, o);
#pragma unroll
    for (int i = 0; i < V; ++i) {
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
template <typename T, typename W, int K, bool WHOLE>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(ConvArgs a, int wide, int tiles, int across) {
    __shared__ float sums[kThreads * V];
    const int lane = threadIdx.x % wide, walk = threadIdx.x / wide, walks = kThreads / wide;
    const int blk = blockIdx.x % across, bt = blockIdx.x / across;   // channels, then (sequence, tile)
    const int c = (blk * wide + lane) * V, left = a.D - c;
    const int b = bt / tiles, t0 = (bt % tiles * walks + walk) * kWalkBwd;
    const int n = length_of(a.lengths, b, a.N);
    float gw[K][V] = {}, gb[V] = {};
    if (left > 0 && (t0 < a.N || t0 == 0)) {
        const T* x = static_cast<const T*>(a.x) + static_cast<size_t>(b) * a.N * a.ldx + c;
        const T* gy = static_cast<const T*>(a.gy) + static_cast<size_t>(b) * a.N * a.D + c;
        T* gx = static_cast<T*>(a.y) + static_cast<size_t>(b) * a.N * a.D + c;
        const int end = t0 + kWalkBwd < a.N ? t0 + kWalkBwd : a.N;   // rows of gx that are this walk's
        const int stop = end + K - 1;                                // it needs dpre up to here
        const int there = stop < n ? stop : n;                       // rows that are read
        Raw<T, V> nx[kRows], ng[kRows];
        // rows behind the last one are worth zero: the last is read again instead
        auto fetch = [&](int s) {
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const size_t t = s + k < there ? s + k : there - 1;
                nx[k] = pack<T, WHOLE>(x + t * a.ldx, left);
                ng[k] = pack<T, WHOLE>(gy + t * a.D, left);
            }
        };
        if (t0 < there) fetch(t0);
        float w[K][V], bias[V];
        load_weights<W, K>(static_cast<const W*>(a.w), c, a.D, w);
        load_bias<W>(static_cast<const W*>(a.b), c, a.D, bias);
        float xs[K][V], dp[K][V];      // rows s-K+1 .. s of xs and of dpre
#pragma unroll
        for (int j = 0; j < K; ++j) {
            // the rows before t0, moved down by the first step
            Raw<T, V> r = {};
            if (j > 0 && t0 - K + j < n) r = row<T, K, WHOLE>(a, b, t0 - K + j, c);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                xs[j][i] = up(r.v[i]);
                dp[j][i] = 0.f;
            }
        }
        for (int s0 = t0; s0 < stop; s0 += kRows) {
            float px[kRows][V], pg[kRows][V];
#pragma unroll
            for (int k = 0; k < kRows; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    px[k][i] = s0 + k < there ? up(nx[k].v[i]) : 0.f;
                    pg[k][i] = s0 + k < there ? up(ng[k].v[i]) : 0.f;
                }
            if (s0 + kRows < there) fetch(s0 + kRows);
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int s = s0 + k, i0 = s - (K - 1);
                const bool mine = s < end;       // its weight sums are this walk's too
                float gx_row[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
#pragma unroll
                    for (int j = 0; j + 1 < K; ++j) {
                        xs[j][i] = xs[j + 1][i];
                        dp[j][i] = dp[j + 1][i];
                    }
                    xs[K - 1][i] = px[k][i];
                    float g = pg[k][i];
                    if (a.silu) {
                        float pre = bias[i];
#pragma unroll
                        for (int j = 0; j < K; ++j) pre = fmaf(w[j][i], xs[j][i], pre);
                        const float sg = sigmoid_f(pre);
                        g *= fmaf(pre * sg, 1.f - sg, sg);
                    }
                    g = s < there ? g : 0.f;
                    dp[K - 1][i] = g;
                    const float gm = mine ? g : 0.f;
                    gb[i] += gm;
#pragma unroll
                    for (int j = 0; j < K; ++j) gw[j][i] = fmaf(gm, xs[j][i], gw[j][i]);
                    float r = 0.f;
#pragma unroll
                    for (int j = 0; j < K; ++j) r = fmaf(w[j][i], dp[K - 1 - j][i], r);
                    gx_row[i] = r;
                }
                // row i0 of the gradient of xs: a token's, or (t0 = 0) a state row's
                if (s >= stop || (i0 < t0 && t0 > 0)) continue;
                if (a.gstate_out != nullptr && s >= n && i0 < n) {
                    const Raw<T, V> r = pack<T, WHOLE>(
                        static_cast<const T*>(a.gstate_out) + (static_cast<size_t>(b) * (K - 1) + s - n) * a.D + c, left);
#pragma unroll
                    for (int i = 0; i < V; ++i) gx_row[i] += up(r.v[i]);
                }
                if (i0 >= 0) {
                    put<T, WHOLE>(gx + static_cast<size_t>(i0) * a.D, gx_row, left, a.stream);
                } else if (a.gstate_in != nullptr) {
                    put<T, WHOLE>(static_cast<T*>(a.gstate_in) + (static_cast<size_t>(b) * (K - 1) + s) * a.D + c, gx_row, left,
                                  false);
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

int packs_of(int D) { return (D + V - 1) / V; }
// Lanes across the channels: enough for all of them up to a wave.
int bwd_wide(int D) {
    int w = 8;
    while (w < 64 && w < packs_of(D)) w *= 2;
    return w;
}
int bwd_tiles(int N, int D) {
    const int tokens = kThreads / bwd_wide(D) * kWalkBwd;
    return N > 0 ? (N - 1) / tokens + 1 : 1;
}

template <typename T, typename W, int K>
hipError_t fwd_k(const ConvArgs& a, hipStream_t st) {
    const int packs = packs_of(a.D);
    // A walk of w tokens reads K-1 rows more than it writes: the longest one, up to 32, that
    // leaves kWantWaves waves, down to 4.
    constexpr size_t kWantWaves = 4096;
    int walk = 32;
    while (walk > 4 && static_cast<size_t>(a.B) * packs * ((a.N + walk - 1) / walk) < kWantWaves * 64) walk /= 2;
    const int tiles = a.N > 0 ? (a.N - 1) / walk + 1 : 1;
    const size_t n = static_cast<size_t>(a.B) * tiles * packs;
    const dim3 grid(static_cast<unsigned>((n + kThreads - 1) / kThreads)), block(kThreads);
    ProfScope prof(kProfConv, st);
    if (a.D % V == 0)
        hipLaunchKernelGGL((conv_fwd_kernel<T, W, K, true>), grid, block, 0, st, a, packs, tiles, walk);
    else
        hipLaunchKernelGGL((conv_fwd_kernel<T, W, K, false>), grid, block, 0, st, a, packs, tiles, walk);
    return hipGetLastError();
}

template <typename T, typename W, int K>
hipError_t step_k(const ConvArgs& a, hipStream_t st) {
    const int packs = packs_of(a.D);
    const size_t n = static_cast<size_t>(a.B) * packs;
    ProfScope prof(kProfConv, st);
    hipLaunchKernelGGL((conv_step_kernel<T, W, K>), dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads)), dim3(kThreads),
                       0, st, a, packs);
    return hipGetLastError();
}

template <typename T, typename W, int K>
hipError_t bwd_k(const ConvArgs& a, hipStream_t st) {
    const int wide = bwd_wide(a.D), tiles = bwd_tiles(a.N, a.D), packs = packs_of(a.D);
    if (a.B > 0) {
        ProfScope prof(kProfConv, st);
        const int across = (packs + wide - 1) / wide;
        const dim3 grid(static_cast<unsigned>(across) * a.B * tiles), block(kThreads);
        if (a.D % V == 0)
            hipLaunchKernelGGL((conv_bwd_kernel<T, W, K, true>), grid, block, 0, st, a, wide, tiles, across);
        else
            hipLaunchKernelGGL((conv_bwd_kernel<T, W, K, false>), grid, block, 0, st, a, wide, tiles, across);
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
hipError_t go(const ConvArgs& args, Way way, hipStream_t st) {
    ConvArgs a = args;
    a.stream = static_cast<size_t>(a.B) * a.N * a.D * (a.bf16 ? 2 : 4) >= kStreamBytes;
    if (!a.bf16) return go_typed<float, float>(a, way, st);
    return a.w_bf16 ? go_typed<bf16_t, bf16_t>(a, way, st) : go_typed<bf16_t, float>(a, way, st);
}

}  // namespace

size_t conv_bwd_workspace(int B, int N, int D, int K) {
    return static_cast<size_t>(B) * bwd_tiles(N, D) * (K + 1) * D * sizeof(float);
}
hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t st) { return go(a, kFwd, st); }
hipError_t launch_conv_step(const ConvArgs& a, hipStream_t st) { return go(a, kStep, st); }
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t st) { return go(a, kBwd, st); }

}  // namespace retn
