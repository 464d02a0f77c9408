// Products of few rows (the tokens of a decoding batch): C = A W^T with at most 32 rows.
//
// Bound by the weights' bytes and by latency: every weight is used for one block of rows only, so
// it goes from memory straight into the matrix instructions' registers, past LDS.  A workgroup
// owns 16 columns, and its waves share the reduction: a wave takes every nw-th piece of 64 bytes
// of the rows, eight pieces (four for two blocks of rows) at a time with all their loads in flight while it has
// that many left, then one at a time; the waves' sums are added in LDS in their order.  A wave's share is short
// where the reduction is: of 1024 bf16 elements over eight waves, or 2048 over sixteen, it is four pieces, which one
// block of rows takes singly.  Rows and widths of any alignment are read as they lie.
//
// Measured: one token through the gated block of 1024 x 4096, 17 MB of weights in 6.1 us and 8 MB in 7.7
// (64 workgroups of 16 waves on 256 CUs); 16 rows of 4096 x 4096 in 12.4 us with weights that no cache holds (2.7 TB/s).

#include "common.h"
#include "launch.h"
#include "proj_epi.h"

#include <algorithm>

namespace retn {
namespace {

constexpr int kMaxWaves = 16;

// 16 bytes of a row from element k on: whole, or cut at the row's end.
template <typename T, bool CUT>
__device__ __forceinline__ u16x8_t piece(const T* row, int k, int K) {
    constexpr int V = kPack<T>;
    if constexpr (CUT) return __builtin_bit_cast(u16x8_t, raw_load_n<T, V>(row + k, K - k));
    return __builtin_bit_cast(u16x8_t, raw_load<T, V>(row + k));
}

// MT blocks of 16 rows.
template <typename T, int MT, int KIND>
__global__ __launch_bounds__(64 * kMaxWaves) void proj_small_kernel(const ProjArgs p) {
    constexpr bool PAIRS = KIND == kProjGated;
    constexpr int kOf = PAIRS ? 2 : 1, kStep = 64 / static_cast<int>(sizeof(T)), V = kPack<T>;
    constexpr int kFly = MT == 1 ? 8 : 4;            // pieces whose loads are in flight together
    extern __shared__ __attribute__((aligned(16))) float sums[];    // [wave][projection][block][16][16]
    const ProjGroup& g = p.g[0];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
    const int l16 = lane & 15, g4 = lane >> 4, n0 = blockIdx.x * 16, K = p.red_rows;
    const int col = min(n0 + l16, g.bn - 1);         // (a column past the last is computed again and not stored)
    const T* w[kOf];
    w[0] = static_cast<const T*>(g.b) + static_cast<size_t>(col) * g.ldb;
    if constexpr (PAIRS) w[1] = static_cast<const T*>(g.b2) + static_cast<size_t>(col) * g.ldb;
    const T* x[MT];
    bool row[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        row[i] = i * 16 + l16 < g.M;
        x[i] = static_cast<const T*>(g.a) + static_cast<size_t>(row[i] ? i * 16 + l16 : 0) * g.lda;
    }
    f32x4_t acc[kOf][MT];
#pragma unroll
    for (int o = 0; o < kOf; ++o)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[o][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const u16x8_t none = {0, 0, 0, 0, 0, 0, 0, 0};
    // the products of pieces s, s + nw, ... (COUNT of them)
    auto pieces = [&](int s, auto count, auto cut) {
        constexpr int COUNT = count();
        constexpr bool CUT = cut();
        u16x8_t wf[COUNT][kOf], xf[COUNT][MT];
#pragma unroll
        for (int c = 0; c < COUNT; ++c) {
            const int k = (s + c * nw) * kStep + V * g4;
#pragma unroll
            for (int o = 0; o < kOf; ++o) wf[c][o] = piece<T, CUT>(w[o], k, K);
        }
#pragma unroll
        for (int c = 0; c < COUNT; ++c) {
            const int k = (s + c * nw) * kStep + V * g4;
#pragma unroll
            for (int i = 0; i < MT; ++i) xf[c][i] = row[i] ? piece<T, CUT>(x[i], k, K) : none;
        }
#pragma unroll
        for (int c = 0; c < COUNT; ++c)
#pragma unroll
            for (int o = 0; o < kOf; ++o)
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[o][i] = frag_mul<T>(wf[c][o], xf[c][i], acc[o][i]);
    };
    const int full = K / kStep;
    int s = wave;
    for (; s + (kFly - 1) * nw < full; s += kFly * nw)
        pieces(s, std::integral_constant<int, kFly>(), std::integral_constant<bool, false>());
    for (; s < full; s += nw) pieces(s, std::integral_constant<int, 1>(), std::integral_constant<bool, false>());
    if (s == full && full * kStep < K) pieces(s, std::integral_constant<int, 1>(), std::integral_constant<bool, true>());

    // lane (l16, g4) holds row l16 and columns 4 g4 .. 4 g4 + 3 of a block
    constexpr int kBlock = kOf * MT * 256;
#pragma unroll
    for (int o = 0; o < kOf; ++o)
#pragma unroll
        for (int i = 0; i < MT; ++i)
            *reinterpret_cast<f32x4_t*>(sums + wave * kBlock + (o * MT + i) * 256 + l16 * 16 + 4 * g4) = acc[o][i];
    __syncthreads();
    for (int q = threadIdx.x; q < kBlock / 4; q += blockDim.x) {
        f32x4_t t = *reinterpret_cast<const f32x4_t*>(sums + 4 * q);
        for (int v = 1; v < nw; ++v) t += *reinterpret_cast<const f32x4_t*>(sums + v * kBlock + 4 * q);
        *reinterpret_cast<f32x4_t*>(sums + 4 * q) = t;
    }
    __syncthreads();
    if (threadIdx.x >= MT * 32) return;
    const int r = threadIdx.x >> 1, n = n0 + (threadIdx.x & 1) * 8;
    if (r >= g.M || n >= g.N) return;
    float v[1][8], u[1][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[0][i] = sums[r * 16 + (threadIdx.x & 1) * 8 + i];
        u[0][i] = PAIRS ? sums[MT * 256 + r * 16 + (threadIdx.x & 1) * 8 + i] : 0.f;
    }
    Columns<T, KIND> cols;
    cols.load(p.e, n, g.N - n);
    const int m[1] = {r};
    Reads<T, KIND, 1> reads;
    reads.load(p.e, g, m, n);
    finish<T, KIND, 1>(p.e, g, cols, reads, m, n, v, u);
}

template <typename T, int MT, int KIND>
hipError_t launch_rows(const ProjArgs& a, hipStream_t st) {
    constexpr int kStep = 64 / static_cast<int>(sizeof(T));
    // waves of a workgroup, with more than two pieces each (all of one wave's where there are four or less);
    // more than eight waves where few workgroups share the chip
    const int pieces = (a.red_rows + kStep - 1) / kStep, groups = (a.g[0].N + 15) / 16;
    int nw = 1;
    while (nw < (groups <= 256 ? kMaxWaves : 8) && nw * 4 < pieces) nw *= 2;
    const size_t lds = static_cast<size_t>(nw) * (KIND == kProjGated ? 2 : 1) * MT * 256 * sizeof(float);
    if (lds > 65536) return hipErrorInvalidValue;
    ProfScope prof(kProfProj, st);
    hipLaunchKernelGGL((proj_small_kernel<T, MT, KIND>), dim3(groups), dim3(64 * nw), lds, st, a);
    return hipGetLastError();
}
template <typename T, int KIND>
hipError_t launch_blocks(const ProjArgs& a, hipStream_t st) {
    if (a.g[0].M <= 16) return launch_rows<T, 1, KIND>(a, st);
    return launch_rows<T, 2, KIND>(a, st);
}

}  // namespace

// One block of rows always (16 rows of 4096 x 4096: 12 us; a cut tile takes 18 for any number up to 128).  Two blocks
// up to 4096 columns, as every workgroup reads all rows again: 32 rows of N columns x K, here and with a cut tile,
// in us, bf16: 1024 x 1024 5 and 11, 4096 x 1024 6 and 14, 4096 x 4096 15 and 19; 16384 x 2048 27 and 23, 16384 x 8192 95 and
// 79.  The border is by columns alone and coarse: up to it, reductions of 8192 are faster with a tile (2048 x 8192 26 and
// 20, 4096 x 8192 28 and 24); beyond it short ones would be faster here (8192 x 2048 16 and 19), and fp32 at any size (16384 x
// 8192 210 and 276).
bool proj_small(int M, int N) { return M <= 16 || (M <= 32 && N <= 4096); }

hipError_t launch_proj_small(const ProjArgs& a, ProjKind kind, bool bf16, hipStream_t st) {
    if (a.g[0].M > 32 || a.g[0].N == 0) return hipErrorInvalidValue;
    if (kind == kProjGated) return bf16 ? launch_blocks<bf16_t, kProjGated>(a, st) : launch_blocks<float, kProjGated>(a, st);
    return bf16 ? launch_blocks<bf16_t, kProjLinear>(a, st) : launch_blocks<float, kProjLinear>(a, st);
}

}  // namespace retn
