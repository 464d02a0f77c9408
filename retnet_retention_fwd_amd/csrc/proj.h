// Arguments and launchers of the projections of a block: the matrix product with bias,
// activation and residual in its epilogue, and the gated feed-forward block, with their
// gradients (proj.hip, proj_small.hip), and of the head norms with rotary positions
// (heads.hip).  Every argument has been validated (proj_api.cpp) before a launcher sees it.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "block.h"

namespace retn {

// One matrix product of a launch, C[M, N] = A B with the reduction over `red` elements (of
// each phase).  An operand is reduction-major (its rows are indexed by the output, the
// reduction adjacent) or output-major (its rows are indexed by the reduction).
struct ProjGroup {
    const void *a, *b;         // operands of the first phase
    const void *a2, *b2;       // of the second (two phases); or b2: the second projection (gated)
    void* c;                   // output, ldc elements between rows
    long long ldc;
    int lda, ldb;              // elements between rows: multiples of 16 bytes, as are the pointers
    int M, N;                  // N also counts zero columns that a padded C takes,
    int bn;                    // this does not: B's columns
    int tiles_n, end;          // set by the launcher: column tiles, exclusive last tile
};

// What happens to a product's sums.
struct ProjEpi {
    const void* bias;          // [N], may be null
    bool bias_f32;
    int act;                   // a retn_activation
    const void* res;           // [M, N] contiguous, may be null
    void* pre;                 // [M, N] contiguous: the sums with bias before the activation; may be null
    // gated forward: the two projections [M, gate_ld], may be null; backward: read
    void *gate, *up;
    long long gate_ld;
    int gate_n;                // columns that gate and up have
    // gated backward: gradients of gate and up, and the product act(gate) up, [M, ldc]
    void *ggate, *gup, *prod;
};

enum ProjKind { kProjLinear = 0, kProjGated = 1, kProjGatedBwd = 2 };

struct ProjArgs {
    ProjGroup g[3];
    int ngroups;
    int red, red_rows, phases; // elements of the reduction; red counts zeros that pad rows to 16 bytes
    ProjEpi e;
    int steps, tiles, band;    // set by the launcher: steps of a tile, tiles, rows of tiles walked together
    int tiles1, splits1, splits2;   // set by the launcher: the first tiles1 are cut in splits1 parts, the others in splits2
    float* part;               // parts of the sums of tiles that are cut
};

// Bytes of partial sums that a launch needs.
size_t proj_partial_bytes(const ProjArgs& a, ProjKind kind, bool bf16);
// a_red, b_red: the operands are reduction-major.  The kinds other than linear take a
// reduction-major A.
hipError_t launch_proj(ProjArgs a, ProjKind kind, bool bf16, bool a_red, bool b_red, hipStream_t st);

// Products of few rows, x W^T (linear and gated): operands of any alignment, red_rows elements of
// the reduction, no partial sums.
bool proj_small(int M, int N);
hipError_t launch_proj_small(const ProjArgs& a, ProjKind kind, bool bf16, hipStream_t st);

// Each dst[rows][ldd] = src[rows][lds] of `width` elements, zeros behind them.
struct PackArgs {
    struct One {
        const void* src;
        long long lds;
        void* dst;
        long long ldd;
        size_t rows;
        int width;
    } one[5];
    int n;
};
hipError_t launch_proj_pack(const PackArgs& a, bool bf16, hipStream_t st);

// gz = gy * slope(pre) (act none: not written) and the column sums of it.
struct SlopeArgs {
    const void* gy;            // [rows][N]
    const void* pre;           // [rows][N], may be null (slope one)
    int act;
    void* gz;                  // [rows][ldz], zeros behind column N; may be null
    long long ldz;
    size_t rows;
    int N;
    float* part;               // partial sums, null: no sums
    void* sums;                // [N]
    bool sums_f32, bf16;
};
size_t slope_partial_bytes(size_t rows, int N);
hipError_t launch_slope(const SlopeArgs& a, hipStream_t st);

// Head norms with rotary positions.
struct HeadsView {
    const void* x;             // [B, H, N, d] by strides
    const void* gy;            // backward
    void* out;                 // forward: the rotated rows; backward: the gradient of x
    long long x_b, x_h, x_n, g_b, g_h, g_n, o_b, o_h, o_n;
    int H;
    float scale;
    const void* w;             // [d], may be null (ones)
    void* gw;                  // backward, may be null
};
struct HeadsArgs {
    HeadsView q, k;
    const float* table;
    long long table_len;
    const long long* pos;
    bool pos_batched;
    long long first;
    int B, N, d, rot;
    float eps;
    bool interleaved, backward, bf16, w_bf16;
    float* part;               // backward: partial sums of the weights' gradients
};
size_t heads_partial_bytes(int d);
hipError_t launch_heads(const HeadsArgs& a, hipStream_t st);

}  // namespace retn
