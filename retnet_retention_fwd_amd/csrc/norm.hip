// Layer normalisation, forward and backward, and the column sums that finish the gradients
// of weights (also the convolution's and the scan's).
//
//     y = (x - mean) rstd w + b,      rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//     dx = rstd (v - mean(v) - xh mean(v xh)),   v = gy w,   xh = (x - mean) rstd
//     dw = sum over rows of gy xh,    db = sum over rows of gy
//
// Bound by HBM: forward reads and writes a row once, backward reads two and writes one.  A
// row stays in the registers of one wave (up to 1024 columns) or of one workgroup, so the
// mean is known before the squared deviations are summed: no cancellation, one read.  The
// waves walk over rows with the weights in registers; in the backward each keeps its
// columns' sums of gy xh and gy over all of its rows, the workgroup adds its waves' sums
// through LDS, and a second launch adds the workgroups' partial sums in a fixed order.
//
// Measured: forward, 16384 x 2048 bf16, 134 MB in 30 us (4.4 TB/s; a large copy reaches
// 5.1); backward, 8200 x 1111 f32, 109 MB in 26 us, 22 of them this kernel and 5 the column
// sums (profiled); backward, 16384 x 2048 and 4096 x 8192 bf16, 201 MB in 54 us (49 and 5), which
// wait 62% of the waves' time: a workgroup has one row ahead in flight, and leaves and reads
// again 13 to 17 MB of partial sums.

#include "block.h"
#include "launch.h"
#include "vec_io.h"

namespace retn {

namespace {

constexpr int kThreads = 256;

// Threads of a workgroup whose rows take TPR threads each.
constexpr int threads_of(int tpr) { return tpr > kThreads ? tpr : kThreads; }

// Sums of two values over the TPR threads that share a row (red: 4 TPR / 64 floats).
template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* red, int& slot) {
    a = wave_sum(a);
    b = wave_sum(b);
    if (TPR > 64) {
        // two sets of slots in turn: the next call writes one that nobody still reads
        constexpr int WV = TPR / 64;
        float* r = red + slot * 2 * WV;
        slot ^= 1;
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            r[wave] = a;
            r[WV + wave] = b;
        }
        __syncthreads();
        a = b = 0.f;
#pragma unroll
        for (int i = 0; i < WV; ++i) {
            a += r[i];
            b += r[WV + i];
        }
    }
}

template <typename T, typename W, int F, int TPR>
__global__ __launch_bounds__(kThreads) void norm_fwd_kernel(NormArgs a) {
    constexpr int V = kPack<T>, P = F / V, RPB = kThreads / TPR;
    __shared__ float red[16];
    int slot = 0;
    const int l = threadIdx.x % TPR, D = a.D;
    const T* x = static_cast<const T*>(a.x);
    const W* w = static_cast<const W*>(a.w);
    const W* b = static_cast<const W*>(a.b);
    T* y = static_cast<T*>(a.y);
    Raw<W, V> wr[P], br[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int e = (p * TPR + l) * V;
        if (e < D && w != nullptr) wr[p] = raw_load_n<W, V>(w + e, D - e);
        if (e < D && b != nullptr) br[p] = raw_load_n<W, V>(b + e, D - e);
    }
    const float inv = 1.f / static_cast<float>(D);
    // the next row is in flight while one is worked on
    Raw<T, V> next[P];
    auto fetch = [&](size_t r) {
        const T* xr = x + (r < a.rows ? r : a.rows - 1) * D;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * TPR + l) * V;
            next[p] = Raw<T, V>{};
            if (a.stream && e + V <= D)
                next[p] = load_stream<T, V>(xr + e);
            else if (e < D)
                next[p] = raw_load_n<T, V>(xr + e, D - e);
        }
    };
    const size_t stride = static_cast<size_t>(gridDim.x) * RPB;
    fetch(static_cast<size_t>(blockIdx.x) * RPB + threadIdx.x / TPR);
    // a workgroup's rows share their trips, so the barriers of row_sum2 are uniform
    for (size_t r0 = static_cast<size_t>(blockIdx.x) * RPB; r0 < a.rows; r0 += stride) {
        const size_t r = r0 + threadIdx.x / TPR;
        const bool live = r < a.rows;
        float v[P][V];
        float s = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[p][i] = up(next[p].v[i]);
                s += v[p][i];
            }
        }
        if (r0 + stride < a.rows) fetch(r + stride);
        float none = 0.f, q = 0.f;
        row_sum2<TPR>(s, none, red, slot);
        const float mean = s * inv;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * TPR + l) * V;
            // only the pack that the row ends in is masked element by element
            if (e + V <= D) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    v[p][i] -= mean;
                    q = fmaf(v[p][i], v[p][i], q);
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    v[p][i] -= mean;
                    if (e + i < D) q = fmaf(v[p][i], v[p][i], q);
                }
            }
        }
        none = 0.f;
        row_sum2<TPR>(q, none, red, slot);
        const float rstd = 1.f / sqrtf(fmaf(q, inv, a.eps));
        if (!live) continue;   // only where a wave has a row of its own: no barrier follows
        if (l == 0) {
            if (a.mean != nullptr) a.mean[r] = mean;
            if (a.rstd != nullptr) a.rstd[r] = rstd;
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * TPR + l) * V;
            if (e >= D) continue;
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                o[i] = v[p][i] * rstd;
                if (w != nullptr) o[i] *= up(wr[p].v[i]);
                if (b != nullptr) o[i] += up(br[p].v[i]);
            }
            store_n<T, V>(y + r * D + e, o, D - e, a.stream);
        }
    }
}

template <typename T, typename W, int F, int TPR>
__global__ __launch_bounds__(threads_of(TPR)) void norm_bwd_kernel(NormArgs a) {
    constexpr int V = kPack<T>, P = F / V, RPB = threads_of(TPR) / TPR;
    __shared__ float red[TPR / 16];
    __shared__ float col[RPB > 1 ? RPB * F * 64 : 1];
    int slot = 0;
    const int l = threadIdx.x % TPR, D = a.D;
    const T* x = static_cast<const T*>(a.x);
    const T* gy = static_cast<const T*>(a.gy);
    const W* w = static_cast<const W*>(a.w);
    T* gx = static_cast<T*>(a.y);
    Raw<W, V> wr[P];
    float gw[P][V], gb[P][V];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int e = (p * TPR + l) * V;
        wr[p] = Raw<W, V>{};       // zeros behind the last column, where the gradient is zero too
        if (e < D && w != nullptr) wr[p] = raw_load_n<W, V>(w + e, D - e);
#pragma unroll
        for (int i = 0; i < V; ++i) gw[p][i] = gb[p][i] = 0.f;
    }
    const float inv = 1.f / static_cast<float>(D);
    // the next row is in flight while one is worked on
    Raw<T, V> rx[P], rg[P];
    float mean = 0.f, rstd = 0.f;
    auto fetch = [&](size_t r) {
        const bool there = r < a.rows;
        const T* xr = x + (there ? r : 0) * D;
        const T* gr = gy + (there ? r : 0) * D;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * TPR + l) * V;
            rx[p] = rg[p] = Raw<T, V>{};
            if (there && e < D) {
                rx[p] = raw_load_n<T, V>(xr + e, D - e);
                rg[p] = raw_load_n<T, V>(gr + e, D - e);
            }
        }
        mean = there ? a.mean[r] : 0.f;
        rstd = there ? a.rstd[r] : 0.f;
    };
    const size_t stride = static_cast<size_t>(gridDim.x) * RPB;
    fetch(static_cast<size_t>(blockIdx.x) * RPB + threadIdx.x / TPR);
    for (size_t r0 = static_cast<size_t>(blockIdx.x) * RPB; r0 < a.rows; r0 += stride) {
        const size_t r = r0 + threadIdx.x / TPR;
        const bool live = r < a.rows;
        const float scale = rstd;
        float xh[P][V], v[P][V], s = 0.f, sx = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float g = up(rg[p].v[i]);      // zero behind the last column
                xh[p][i] = (up(rx[p].v[i]) - mean) * rstd;
                gw[p][i] = fmaf(g, xh[p][i], gw[p][i]);
                gb[p][i] += g;
                v[p][i] = w != nullptr ? g * up(wr[p].v[i]) : g;
                s += v[p][i];
                sx = fmaf(v[p][i], xh[p][i], sx);
            }
        }
        if (r0 + stride < a.rows) fetch(r + stride);
        row_sum2<TPR>(s, sx, red, slot);
        if (!live) continue;
        const float m1 = s * inv, m2 = sx * inv;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * TPR + l) * V;
            if (e >= D) continue;
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = scale * (v[p][i] - fmaf(xh[p][i], m2, m1));
            store_n<T, V>(gx + r * D + e, o, D - e, a.stream);
        }
    }
    if (a.workspace == nullptr) return;
    // [workgroup][2][D] partial sums
    float* out = a.workspace + static_cast<size_t>(blockIdx.x) * 2 * D;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (RPB == 1) {
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int e = (p * TPR + l) * V;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (e + i < D) out[which * D + e + i] = which ? gb[p][i] : gw[p][i];
            }
        } else {
            __syncthreads();
            float* c = col + (threadIdx.x / TPR) * F * 64;
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < V; ++i) c[(p * TPR + l) * V + i] = which ? gb[p][i] : gw[p][i];
            __syncthreads();
            for (int e = threadIdx.x; e < D; e += kThreads) {
                float t = 0.f;
#pragma unroll
                for (int g = 0; g < RPB; ++g) t += col[g * F * 64 + e];
                out[which * D + e] = t;
            }
        }
    }
}

// Rows wider than a workgroup's registers: a workgroup per row, the row read again (from the
// caches) for each of its sums.
template <typename T, typename W>
__global__ __launch_bounds__(kThreads) void norm_fwd_wide_kernel(NormArgs a) {
    __shared__ float red[16];
    int slot = 0;
    const int D = a.D;
    const float inv = 1.f / static_cast<float>(D);
    const W* w = static_cast<const W*>(a.w);
    const W* b = static_cast<const W*>(a.b);
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * D;
        T* y = static_cast<T*>(a.y) + r * D;
        float s = 0.f, q = 0.f, none = 0.f;
        for (int e = threadIdx.x; e < D; e += kThreads) s += up(x[e]);
        row_sum2<kThreads>(s, none, red, slot);
        const float mean = s * inv;
        for (int e = threadIdx.x; e < D; e += kThreads) {
            const float c = up(x[e]) - mean;
            q = fmaf(c, c, q);
        }
        none = 0.f;
        row_sum2<kThreads>(q, none, red, slot);
        const float rstd = 1.f / sqrtf(fmaf(q, inv, a.eps));
        if (threadIdx.x == 0) {
            if (a.mean != nullptr) a.mean[r] = mean;
            if (a.rstd != nullptr) a.rstd[r] = rstd;
        }
        for (int e = threadIdx.x; e < D; e += kThreads) {
            float o = (up(x[e]) - mean) * rstd;
            if (w != nullptr) o *= up(w[e]);
            if (b != nullptr) o += up(b[e]);
            y[e] = down<T>(o);
        }
    }
}

template <typename T, typename W>
__global__ __launch_bounds__(kThreads) void norm_bwd_wide_kernel(NormArgs a) {
    __shared__ float red[16];
    int slot = 0;
    const int D = a.D;
    const float inv = 1.f / static_cast<float>(D);
    const W* w = static_cast<const W*>(a.w);
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * D;
        const T* gy = static_cast<const T*>(a.gy) + r * D;
        T* gx = static_cast<T*>(a.y) + r * D;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s = 0.f, sx = 0.f;
        for (int e = threadIdx.x; e < D; e += kThreads) {
            const float v = w != nullptr ? up(gy[e]) * up(w[e]) : up(gy[e]);
            s += v;
            sx = fmaf(v, (up(x[e]) - mean) * rstd, sx);
        }
        row_sum2<kThreads>(s, sx, red, slot);
        const float m1 = s * inv, m2 = sx * inv;
        for (int e = threadIdx.x; e < D; e += kThreads) {
            const float v = w != nullptr ? up(gy[e]) * up(w[e]) : up(gy[e]);
            gx[e] = down<T>(rstd * (v - fmaf((up(x[e]) - mean) * rstd, m2, m1)));
        }
    }
}

// Column sums of a range of rows, one column a thread: partial sums as norm_bwd_kernel's.
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_bwd_cols_kernel(NormArgs a, int chunks) {
    const int col = blockIdx.x * kThreads + threadIdx.x;
    if (col >= a.D) return;
    const size_t per = (a.rows + chunks - 1) / chunks, lo = blockIdx.y * per;
    const size_t hi = lo + per < a.rows ? lo + per : a.rows;
    float gw = 0.f, gb = 0.f;
    for (size_t r = lo; r < hi; ++r) {
        const float g = up(static_cast<const T*>(a.gy)[r * a.D + col]);
        gw = fmaf(g, (up(static_cast<const T*>(a.x)[r * a.D + col]) - a.mean[r]) * a.rstd[r], gw);
        gb += g;
    }
    float* out = a.workspace + static_cast<size_t>(blockIdx.y) * 2 * a.D;
    out[col] = gw;
    out[a.D + col] = gb;
}

constexpr int kRedCols = 64, kRedGroups = 16;
template <typename O>
__global__ __launch_bounds__(kRedCols* kRedGroups) void col_reduce_kernel(ColReduceArgs a) {
    __shared__ float part[kRedGroups][kRedCols];
    const int c = threadIdx.x % kRedCols, g = threadIdx.x / kRedCols;
    const size_t C = static_cast<size_t>(a.rows) * a.D, at = static_cast<size_t>(blockIdx.x) * kRedCols + c;
    float s = 0.f;
    if (at < C) {
#pragma unroll 8
        for (int p = g; p < a.P; p += kRedGroups) s += a.in[p * C + at];
    }
    part[g][c] = s;
    __syncthreads();
    if (g != 0 || at >= C) return;
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kRedGroups; ++i) t += part[i][c];
    const int j = static_cast<int>(at / a.D), d = static_cast<int>(at % a.D);
    if (j < a.K) {
        if (a.out0 != nullptr) static_cast<O*>(a.out0)[static_cast<size_t>(d) * a.K + j] = down<O>(t);
    } else {
        O* o = static_cast<O*>(j == a.K ? a.out1 : a.out2);
        if (o != nullptr) o[d] = down<O>(t);
    }
}

constexpr int kGroupF = 64;                                 // floats of a row per thread, forward
constexpr int kMaxBlocks = 2048;                            // forward workgroups: 8 per CU
constexpr int kWideBwd = 16 * 1024;                         // columns above which rows are read again
constexpr int kWideChunks = 64;

// Workgroups of the backward: each leaves 2 D partial sums, so few; enough to fill the chip
// (for 16384 rows of 2048: 61 us with 512 of them, 55 us with 768 or 1024).
int bwd_blocks(size_t rows, int D) {
    if (D > kWideBwd) return kWideChunks;
    const size_t rpb = D <= 1024 ? 4 : 1, most = D <= 1024 ? 512 : D <= 2048 ? 768 : D <= 4096 ? 512 : 256;
    const size_t n = (rows + rpb - 1) / rpb;
    return static_cast<int>(n < most ? n : most);
}

template <typename T, typename W>
hipError_t fwd_typed(const NormArgs& a, hipStream_t st) {
    const int D = a.D;
    const bool wave = D <= 1024;
    const size_t need = wave ? (a.rows + 3) / 4 : a.rows;
    const dim3 grid(static_cast<unsigned>(need < kMaxBlocks ? need : kMaxBlocks)), block(kThreads);
    ProfScope prof(kProfNorm, st);
    if (D <= 512)
        hipLaunchKernelGGL((norm_fwd_kernel<T, W, 8, 64>), grid, block, 0, st, a);
    else if (D <= 1024)
        hipLaunchKernelGGL((norm_fwd_kernel<T, W, 16, 64>), grid, block, 0, st, a);
    else if (D <= 8 * kThreads)
        hipLaunchKernelGGL((norm_fwd_kernel<T, W, 8, kThreads>), grid, block, 0, st, a);
    else if (D <= 16 * kThreads)
        hipLaunchKernelGGL((norm_fwd_kernel<T, W, 16, kThreads>), grid, block, 0, st, a);
    else if (D <= 32 * kThreads)
        hipLaunchKernelGGL((norm_fwd_kernel<T, W, 32, kThreads>), grid, block, 0, st, a);
    else if (D <= kGroupF * kThreads)
        hipLaunchKernelGGL((norm_fwd_kernel<T, W, kGroupF, kThreads>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((norm_fwd_wide_kernel<T, W>), grid, block, 0, st, a);
    return hipGetLastError();
}

template <typename T, typename W>
hipError_t bwd_typed(const NormArgs& a, hipStream_t st) {
    const int D = a.D, blocks = bwd_blocks(a.rows, D);
    const dim3 grid(blocks), block(kThreads);
    if (a.rows > 0) {
        ProfScope prof(kProfNorm, st);
        if (D <= 512)
            hipLaunchKernelGGL((norm_bwd_kernel<T, W, 8, 64>), grid, block, 0, st, a);
        else if (D <= 1024)
            hipLaunchKernelGGL((norm_bwd_kernel<T, W, 16, 64>), grid, block, 0, st, a);
        else if (D <= 2048)
            hipLaunchKernelGGL((norm_bwd_kernel<T, W, 8, 256>), grid, block, 0, st, a);
        else if (D <= 4096)
            hipLaunchKernelGGL((norm_bwd_kernel<T, W, 8, 512>), grid, dim3(512), 0, st, a);
        else if (D <= 8192)
            hipLaunchKernelGGL((norm_bwd_kernel<T, W, 8, 1024>), grid, dim3(1024), 0, st, a);
        else if (D <= kWideBwd)
            hipLaunchKernelGGL((norm_bwd_kernel<T, W, 16, 1024>), grid, dim3(1024), 0, st, a);
        else {
            const dim3 rows(static_cast<unsigned>(a.rows < kMaxBlocks ? a.rows : kMaxBlocks));
            hipLaunchKernelGGL((norm_bwd_wide_kernel<T, W>), rows, block, 0, st, a);
            if (a.workspace != nullptr)
                hipLaunchKernelGGL((norm_bwd_cols_kernel<T>), dim3((D + kThreads - 1) / kThreads, kWideChunks), block, 0,
                                   st, a, kWideChunks);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.gw == nullptr && a.gb == nullptr) return hipSuccess;
    const ColReduceArgs c{a.workspace, a.rows > 0 ? blocks : 0, 2, 1, D, a.gw, a.gb, nullptr, a.w_bf16};
    return launch_col_reduce(c, st);
}

}  // namespace

hipError_t launch_col_reduce(const ColReduceArgs& a, hipStream_t st) {
    const size_t C = static_cast<size_t>(a.rows) * a.D;
    const dim3 grid(static_cast<unsigned>((C + kRedCols - 1) / kRedCols)), block(kRedCols * kRedGroups);
    ProfScope prof(kProfReduce, st);
    if (a.out_bf16)
        hipLaunchKernelGGL((col_reduce_kernel<bf16_t>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((col_reduce_kernel<float>), grid, block, 0, st, a);
    return hipGetLastError();
}

size_t norm_bwd_workspace(size_t rows, int D) {
    return static_cast<size_t>(bwd_blocks(rows, D)) * 2 * D * sizeof(float);
}

hipError_t launch_norm_fwd(const NormArgs& args, hipStream_t st) {
    NormArgs a = args;
    a.stream = a.rows * a.D * (a.bf16 ? 2 : 4) >= kStreamBytes;
    if (!a.bf16) return fwd_typed<float, float>(a, st);
    return a.w_bf16 ? fwd_typed<bf16_t, bf16_t>(a, st) : fwd_typed<bf16_t, float>(a, st);
}

hipError_t launch_norm_bwd(const NormArgs& args, hipStream_t st) {
    NormArgs a = args;
    a.stream = a.rows * a.D * (a.bf16 ? 2 : 4) >= kStreamBytes;
    if (!a.bf16) return bwd_typed<float, float>(a, st);
    return a.w_bf16 ? bwd_typed<bf16_t, bf16_t>(a, st) : bwd_typed<bf16_t, float>(a, st);
}

}  // namespace retn
