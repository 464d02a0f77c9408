// Arguments and launchers of the operators that stand around the retention in a block:
// layer normalisation, rotary positions, the short causal convolution and the selective
// scan.  Every argument has been validated (block_api.cpp) before a launcher sees it.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace retn {

// out0[d * K + j] = sum_p in[p][j][d] for j < K, then out1[d], out2[d] from rows K and K+1
// (each may be null): the second step of a gradient that sums over rows or tokens.
struct ColReduceArgs {
    const float* in;           // [P][rows][D]
    int P, rows, K, D;
    void* out0;
    void* out1;
    void* out2;
    bool out_bf16;
};
hipError_t launch_col_reduce(const ColReduceArgs& a, hipStream_t stream);

// Layer normalisation (norm.hip).
struct NormArgs {
    const void* x;
    const void* w;             // may be null (ones)
    const void* b;             // forward only, may be null (zeros)
    void* y;                   // forward: the output; backward: the gradient of x
    float* mean;               // forward: written if given; backward: read
    float* rstd;
    const void* gy;            // backward
    void* gw;                  // backward, may be null
    void* gb;                  // backward, may be null
    size_t rows;
    int D;
    float eps;
    bool bf16, w_bf16;
    bool stream;               // set by the launchers: the output is too large for the caches
    float* workspace;
};
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t stream);
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t stream);
size_t norm_bwd_workspace(size_t rows, int D);

// Rotary positions (rotary.hip).
struct RotaryView {
    const void* in;
    void* out;
    long long in_b, in_h, in_n, out_b, out_h, out_n;   // strides in elements
    int H;
    float scale;
};
struct RotaryArgs {
    RotaryView q, k;           // k.H = 0: none
    const float* table;        // [table_len][rot/2][2]
    long long table_len;
    const long long* pos;      // may be null (first + n)
    bool pos_batched;          // pos is [B, N] instead of [N]
    long long first;
    int B, N, d, rot;
    bool interleaved, transpose, bf16;
};
hipError_t launch_rotary(const RotaryArgs& a, hipStream_t stream);
hipError_t launch_rotary_table(float* table, const double* freq, int pairs, long long first, long long count,
                               float magnitude, hipStream_t stream);

// Short causal convolution (conv.hip).
struct ConvArgs {
    const void* x;             // [B, N, D] rows of stride ldx
    long long ldx;
    const void* w;             // [D, K]
    const void* b;             // [D], may be null
    const int* lengths;        // [B], may be null
    const void* state_in;      // [B, K-1, D], may be null
    void* state_out;           // forward: may be null; step: the state, updated in place
    void* y;                   // forward and step: the output; backward: the gradient of x
    const void* gy;            // backward
    const void* gstate_out;    // backward, may be null
    void* gstate_in;           // backward, may be null
    void* gw;                  // backward, may be null
    void* gb;                  // backward, may be null
    int B, N, D, K;
    bool silu, bf16, w_bf16;
    bool zero_behind;          // forward: the rows of y behind a length are zeros, else left as they were
    bool stream;               // set by the launchers
    float* workspace;
};
hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t stream);
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t stream);
hipError_t launch_conv_step(const ConvArgs& a, hipStream_t stream);
size_t conv_bwd_workspace(int B, int N, int D, int K);

// Selective scan (scan.hip, scan_bwd.hip).
struct ScanArgs {
    const void *x, *dt, *z, *Bm, *Cm;              // z may be null
    long long ldx, lddt, ldz, ldb, ldc;            // token strides; a batch is N of them apart
    const float *A, *Dskip, *bias;                 // Dskip, bias may be null
    const int* lengths;                            // [B], may be null
    const float* state_in;                         // may be null
    float* state_out;                              // may be null; step: the state, in place
    void* y;                                       // forward, step
    // backward
    const void* gy;
    const float* gstate_out;                       // may be null
    void *gx, *gdt, *gz, *gB, *gC;
    float *gA, *gD, *gbias, *gstate_in;            // gD, gbias, gstate_in may be null
    int B, N, D, G, S;
    bool softplus, bf16;
    bool zero_behind;                              // forward, as ConvArgs'
    bool stream;                                   // set by the launchers
    float* workspace;
};
struct ScanPlan {
    int nblk;                  // channel blocks (of a wave or a workgroup) over all groups
    int nseg, seg;             // segments per sequence, tokens per segment
    // workspace, in floats
    size_t off_end, off_dt;    // segment end states, then entry states; sums of dt
    size_t off_rev, off_ckpt, off_cum, off_bc, off_par;   // backward only
    size_t total;
};
ScanPlan scan_fwd_plan(int B, int N, int D, int G, int S);
ScanPlan scan_bwd_plan(int B, int N, int D, int G, int S);
hipError_t launch_scan_fwd(const ScanArgs& a, const ScanPlan& p, hipStream_t stream);
hipError_t launch_scan_bwd(const ScanArgs& a, const ScanPlan& p, hipStream_t stream);
hipError_t launch_scan_step(const ScanArgs& a, hipStream_t stream);

}  // namespace retn
