// C ABI of the operators around the retention (layer normalisation, rotary positions, the
// short causal convolution, the selective scan): argument validation and dispatch.  As in
// api.cpp, every argument is checked before anything is enqueued.

#include "../../include/retention.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <utility>

#include "block.h"
#include "launch.h"
#include "validate.h"

namespace {

constexpr int kMaxD = 1 << 20;
constexpr int kMaxStates = 64;
constexpr int kMaxHead = 256;
constexpr unsigned long long kMaxElements = 1ull << 34;   // of a [B, N, D] tensor
constexpr unsigned long long kMaxGroups = 1ull << 23;     // workgroups of a launch (2^32 threads at most)
constexpr unsigned long long kMaxLaunch = (1ull << 32) - 256;   // elements of a launch of one a thread, in whole workgroups
constexpr long long kMaxRow = 1ll << 26;                  // elements from one token to the next
constexpr long long kMaxSpan = 1ll << 40;                 // elements that one axis of a view spans
constexpr size_t kMaxTokens = (1ull << 31) - (1 << 16);   // token numbers and steps ahead of them are ints

size_t sz(long long x) { return static_cast<size_t>(x); }
size_t f32(size_t n) { return n * sizeof(float); }

// Bytes that rows of `width` elements, `ld` apart, span.
size_t rows_bytes(size_t rows, long long ld, size_t width, size_t es) {
    return rows == 0 ? 0 : ((rows - 1) * sz(ld) + width) * es;
}

// No output overlaps an input or another output.
template <size_t I, size_t O>
bool clash(const Range (&in)[I], const Range (&out)[O]) {
    for (size_t i = 0; i < O; ++i) {
        for (const Range& r : in)
            if (overlaps(out[i], r)) return true;
        for (size_t j = i + 1; j < O; ++j)
            if (overlaps(out[i], out[j])) return true;
    }
    return false;
}

Range opt(const void* p, size_t bytes) { return span(p, p != nullptr ? bytes : 0); }

// Activations of type dt and weights of type wt: fp32, or the activations' type.
bool valid_types(retn_dtype dt, retn_dtype wt) {
    return valid_dtype(dt) && valid_dtype(wt) && (wt == RETN_F32 || wt == dt);
}

retn_status done(hipError_t e) { return e == hipSuccess ? RETN_OK : RETN_ERR_HIP; }

retn_status norm_sizes(long long rows, int D) {
    if (rows < 0 || D < 1) return RETN_ERR_SHAPE;
    if (D > kMaxD || static_cast<unsigned long long>(rows) > kMaxElements ||
        static_cast<unsigned long long>(rows) * D > kMaxElements)
        return RETN_ERR_UNSUPPORTED;
    return RETN_OK;
}

// Sizes of a [B, N, D] operator.
retn_status seq_sizes(int B, int N, int D) {
    if (B < 0 || N < 0 || D < 1) return RETN_ERR_SHAPE;
    if (D > kMaxD || sz(B) * N > kMaxTokens || sz(B) * D > sz(INT32_MAX) || sz(B) * N * D >= kMaxElements)
        return RETN_ERR_UNSUPPORTED;
    return RETN_OK;
}

retn_status conv_sizes(int B, int N, int D, int K) {
    const retn_status st = seq_sizes(B, N, D);
    if (st != RETN_OK) return st;
    if (K < 1) return RETN_ERR_SHAPE;
    return K < 2 || K > 4 ? RETN_ERR_UNSUPPORTED : RETN_OK;
}

retn_status scan_sizes(int B, int N, int D, int G, int S) {
    if (G < 1 || S < 1) return RETN_ERR_SHAPE;
    const retn_status st = seq_sizes(B, N, D);
    if (st != RETN_OK) return st;
    if (D % G != 0) return RETN_ERR_SHAPE;
    // one workgroup a (sequence, block of 16 channels or more); the gradients of B and C one element a
    // thread.  (What is cut into segments has fewer than 2048 waves uncut, fewer than 6144 cut.)
    if (S > kMaxStates || sz(B) * (sz(D) / 16 + G) >= kMaxGroups || 2 * sz(B) * N * G * S > kMaxLaunch)
        return RETN_ERR_UNSUPPORTED;
    return RETN_OK;
}

bool far_rows(long long ldx, long long lddt, long long ldz, long long ldb, long long ldc) {
    return std::max({ldx, lddt, ldz, ldb, ldc}) >= kMaxRow;
}

bool bad_workspace(const void* p, size_t have, size_t need) {
    return need > 0 && (p == nullptr || have < need || !aligned16(p));
}

// A [H, N, d] tensor's place in memory by its strides; sizes of one take any stride.
struct View {
    long long sb, sh, sn;
};
size_t view_bytes(const View& v, int B, int H, int N, int d, size_t es) {
    if (B == 0 || H == 0 || N == 0) return 0;
    return ((sz(B) - 1) * sz(v.sb) + (sz(H) - 1) * sz(v.sh) + (sz(N) - 1) * sz(v.sn) + d) * es;
}
bool valid_view(const View& v, int B, int H, int N) {
    const long long st[3] = {v.sb, v.sh, v.sn};
    const int n[3] = {B, H, N};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (st[i] < 0 || st[i] > kMaxSpan / n[i])) return false;
    return true;
}
// Every element of an output has a place of its own: sorted by stride, each axis steps
// over all that the smaller ones span.
bool own_places(const View& v, int B, int H, int N, int d) {
    long long st[3] = {v.sb, v.sh, v.sn};
    int n[3] = {B, H, N};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (st[j] > st[j + 1]) {
                std::swap(st[j], st[j + 1]);
                std::swap(n[j], n[j + 1]);
            }
    long long reach = d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (st[i] < reach) return false;
        reach += st[i] * (n[i] - 1);
    }
    return true;
}
// Two tensors that lie beside each other inside rows of one stride (q and k of one joint
// projection): their spans overlap, their elements do not.
bool side_by_side(uintptr_t pa, const View& a, int Ha, uintptr_t pb, const View& b, int Hb, int B, int N, int d, size_t es) {
    if (pa > pb) return side_by_side(pb, b, Hb, pa, a, Ha, B, N, d, es);
    const bool many = N > 1, batches = B > 1;
    if ((many && a.sn != b.sn) || (batches && a.sb != b.sb)) return false;
    const long long row = many ? a.sn : batches ? a.sb : 0;
    if (row <= 0 || (many && batches && a.sb < a.sn * N)) return false;
    const size_t gap = pb - pa;
    if (gap % es != 0) return false;
    const long long off = static_cast<long long>(gap / es);
    const long long wa = (Ha > 1 ? a.sh * (Ha - 1) : 0) + d, wb = (Hb > 1 ? b.sh * (Hb - 1) : 0) + d;
    return off >= wa && off + wb <= row;
}

retn_status rotary_common(const void* q, const void* k, void* out_q, void* out_k, const long long* strides,
                          const float* table, long long table_len, const long long* positions, int per_batch,
                          long long first, int B, int Hq, int Hk, int N, int d, int rot, int interleaved, float q_scale,
                          float k_scale, retn_dtype dtype, void* stream, bool transpose) {
    if (!valid_dtype(dtype)) return RETN_ERR_DTYPE;
    if (B < 0 || Hq < 0 || Hk < 0 || N < 0 || d < 1 || rot < 2 || rot > d || rot % 2 != 0 || table_len < 0)
        return RETN_ERR_SHAPE;
    if (d > kMaxHead || sz(B) * N > kMaxTokens || sz(B) * N * d >= (1ull << 32) || sz(Hq) + Hk > 65535 ||
        table_len > kMaxSpan)
        return RETN_ERR_UNSUPPORTED;
    if (B == 0 || N == 0 || Hq + Hk == 0) return RETN_OK;
    if ((Hq > 0 && (q == nullptr || out_q == nullptr)) || (Hk > 0 && (k == nullptr || out_k == nullptr)) ||
        strides == nullptr || table == nullptr)
        return RETN_ERR_NULL;
    // (the kernel reads row 0 for a position outside of the table)
    if (positions == nullptr ? first < 0 || first > table_len - N : table_len < 1) return RETN_ERR_SHAPE;
    const View v[4] = {{strides[0], strides[1], strides[2]}, {strides[3], strides[4], strides[5]},
                       {strides[6], strides[7], strides[8]}, {strides[9], strides[10], strides[11]}};
    const int H[4] = {Hq, Hq, Hk, Hk};
    const void* const ptr[4] = {q, out_q, k, out_k};
    const size_t es = elem_bytes(dtype);
    Range r[4];
    for (int i = 0; i < 4; ++i) {
        if (H[i] > 0 && !valid_view(v[i], B, H[i], N)) return RETN_ERR_SHAPE;
        if (H[i] > 0 && (i & 1) && !own_places(v[i], B, H[i], N, d)) return RETN_ERR_ALIAS;
        r[i] = H[i] > 0 ? span(ptr[i], view_bytes(v[i], B, H[i], N, d, es)) : Range{0, 0};
    }
    const Range rt = span(table, f32(sz(table_len) * rot));
    const Range rp = opt(positions, sizeof(long long) * sz(N) * (per_batch ? B : 1));
    for (int o = 1; o < 4; o += 2) {
        if (overlaps(r[o], rt) || overlaps(r[o], rp)) return RETN_ERR_ALIAS;
        for (int i = 0; i < 4; ++i) {
            if (i == o || !overlaps(r[o], r[i])) continue;
            const bool in_place = i == o - 1 && ptr[i] == ptr[o] && (B <= 1 || v[i].sb == v[o].sb) &&
                                  (H[o] <= 1 || v[i].sh == v[o].sh) && (N <= 1 || v[i].sn == v[o].sn);
            if (!in_place && !side_by_side(r[o].lo, v[o], H[o], r[i].lo, v[i], H[i], B, N, d, es)) return RETN_ERR_ALIAS;
        }
    }
    retn::RotaryArgs a{};
    a.q = retn::RotaryView{q, out_q, v[0].sb, v[0].sh, v[0].sn, v[1].sb, v[1].sh, v[1].sn, Hq, q_scale};
    a.k = retn::RotaryView{k, out_k, v[2].sb, v[2].sh, v[2].sn, v[3].sb, v[3].sh, v[3].sn, Hk, k_scale};
    a.table = table;
    a.table_len = table_len;
    a.pos = positions;
    a.pos_batched = per_batch != 0;
    a.first = first;
    a.B = B;
    a.N = N;
    a.d = d;
    a.rot = rot;
    a.interleaved = interleaved != 0;
    a.transpose = transpose;
    a.bf16 = dtype == RETN_BF16;
    return done(retn::launch_rotary(a, static_cast<hipStream_t>(stream)));
}

// The forward of the convolution and the scan; zero_behind: the rows of y behind a length are written as zeros.
retn_status conv_forward(const void* x, long long ldx, const void* weight, const void* bias, void* y,
                         const void* state_in, void* state_out, const int* lengths, int B, int N, int D, int K, int silu,
                         retn_dtype dtype, retn_dtype wdtype, void* stream, bool zero_behind) {
    if (!valid_types(dtype, wdtype)) return RETN_ERR_DTYPE;
    const retn_status st = conv_sizes(B, N, D, K);
    if (st != RETN_OK) return st;
    if (ldx < D) return RETN_ERR_SHAPE;
    if (ldx >= kMaxRow) return RETN_ERR_UNSUPPORTED;
    const size_t tokens = sz(B) * N, es = elem_bytes(dtype), we = elem_bytes(wdtype), sb = sz(B) * (K - 1) * D * es;
    if (B == 0) return RETN_OK;
    if ((N > 0 && (x == nullptr || y == nullptr)) || weight == nullptr) return RETN_ERR_NULL;
    const Range in[] = {opt(x, rows_bytes(tokens, ldx, D, es)), span(weight, sz(D) * K * we), opt(bias, D * we),
                        opt(state_in, sb), opt(lengths, sizeof(int) * sz(B))};
    const Range out[] = {opt(y, tokens * D * es), opt(state_out, sb)};
    if (clash(in, out)) return RETN_ERR_ALIAS;
    if (N == 0 && state_out == nullptr) return RETN_OK;
    retn::ConvArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.w = weight;
    a.b = bias;
    a.lengths = lengths;
    a.state_in = state_in;
    a.state_out = state_out;
    a.y = y;
    a.B = B;
    a.N = N;
    a.D = D;
    a.K = K;
    a.silu = silu != 0;
    a.zero_behind = zero_behind && lengths != nullptr;
    a.bf16 = dtype == RETN_BF16;
    a.w_bf16 = wdtype == RETN_BF16;
    return done(retn::launch_conv_fwd(a, static_cast<hipStream_t>(stream)));
}

retn_status scan_forward(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                         const float* Dskip, const void* z, const float* dt_bias, void* y, const float* state_in,
                         float* state_out, const int* lengths, long long ldx, long long lddt, long long ldz,
                         long long ldb, long long ldc, int B, int N, int D, int G, int S, int softplus,
                         retn_dtype dtype, void* workspace, size_t workspace_bytes, void* stream, bool zero_behind) {
    if (!valid_dtype(dtype)) return RETN_ERR_DTYPE;
    const retn_status st = scan_sizes(B, N, D, G, S);
    if (st != RETN_OK) return st;
    const long long gs = static_cast<long long>(G) * S;
    if (ldx < D || lddt < D || (z != nullptr && ldz < D) || ldb < gs || ldc < gs) return RETN_ERR_SHAPE;
    if (far_rows(ldx, lddt, z != nullptr ? ldz : 0, ldb, ldc)) return RETN_ERR_UNSUPPORTED;
    if (B == 0) return RETN_OK;
    const size_t tokens = sz(B) * N, es = elem_bytes(dtype), ss = f32(sz(B) * D * S);
    if (N > 0 && (x == nullptr || dt == nullptr || A == nullptr || Bm == nullptr || Cm == nullptr || y == nullptr))
        return RETN_ERR_NULL;
    const size_t need = selective_scan_workspace_bytes(B, N, D, G, S);
    const bool in_place = state_out != nullptr && state_out == state_in;
    const Range in[] = {opt(x, rows_bytes(tokens, ldx, D, es)), opt(dt, rows_bytes(tokens, lddt, D, es)),
                        opt(A, f32(sz(D) * S)), opt(Bm, rows_bytes(tokens, ldb, gs, es)),
                        opt(Cm, rows_bytes(tokens, ldc, gs, es)), opt(Dskip, f32(D)), opt(dt_bias, f32(D)),
                        opt(z, rows_bytes(tokens, ldz, D, es)), opt(in_place ? nullptr : state_in, ss),
                        opt(lengths, sizeof(int) * sz(B))};
    const Range out[] = {opt(y, tokens * D * es), opt(state_out, ss), opt(workspace, need)};
    if (clash(in, out)) return RETN_ERR_ALIAS;
    if (bad_workspace(workspace, workspace_bytes, need)) return RETN_ERR_WORKSPACE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (N == 0) return done(retn::launch_copy_state(state_in, state_out, sz(B) * D * S, s));
    retn::ScanArgs a{};
    a.x = x;
    a.dt = dt;
    a.z = z;
    a.Bm = Bm;
    a.Cm = Cm;
    a.ldx = ldx;
    a.lddt = lddt;
    a.ldz = ldz;
    a.ldb = ldb;
    a.ldc = ldc;
    a.A = A;
    a.Dskip = Dskip;
    a.bias = dt_bias;
    a.lengths = lengths;
    a.state_in = state_in;
    a.state_out = state_out;
    a.y = y;
    a.B = B;
    a.N = N;
    a.D = D;
    a.G = G;
    a.S = S;
    a.softplus = softplus != 0;
    a.zero_behind = zero_behind && lengths != nullptr;
    a.bf16 = dtype == RETN_BF16;
    a.workspace = static_cast<float*>(workspace);
    return done(retn::launch_scan_fwd(a, retn::scan_fwd_plan(B, N, D, G, S), s));
}

}  // namespace

extern "C" {

retn_status layer_norm_fwd(const void* x, const void* weight, const void* bias, void* y, float* mean, float* rstd,
                           long long rows, int D, float eps, retn_dtype dtype, retn_dtype wdtype, void* stream) {
    if (!valid_types(dtype, wdtype)) return RETN_ERR_DTYPE;
    const retn_status st = norm_sizes(rows, D);
    if (st != RETN_OK) return st;
    if (!(eps >= 0.f)) return RETN_ERR_SHAPE;
    if (rows == 0) return RETN_OK;
    if (x == nullptr || y == nullptr) return RETN_ERR_NULL;
    const size_t n = sz(rows) * D * elem_bytes(dtype), we = D * elem_bytes(wdtype);
    const Range in[] = {span(x, n), opt(weight, we), opt(bias, we)};
    const Range out[] = {span(y, n), opt(mean, f32(rows)), opt(rstd, f32(rows))};
    if (clash(in, out)) return RETN_ERR_ALIAS;
    retn::NormArgs a{};
    a.x = x;
    a.w = weight;
    a.b = bias;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    a.rows = sz(rows);
    a.D = D;
    a.eps = eps;
    a.bf16 = dtype == RETN_BF16;
    a.w_bf16 = wdtype == RETN_BF16;
    return done(retn::launch_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t layer_norm_bwd_workspace_bytes(long long rows, int D, retn_dtype dtype) {
    if (!valid_dtype(dtype) || norm_sizes(rows, D) != RETN_OK) return 0;
    return retn::norm_bwd_workspace(sz(rows), D);
}

retn_status layer_norm_bwd(const void* x, const void* weight, const float* mean, const float* rstd, const void* grad_y,
                           void* grad_x, void* grad_weight, void* grad_bias, long long rows, int D, retn_dtype dtype,
                           retn_dtype wdtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (!valid_types(dtype, wdtype)) return RETN_ERR_DTYPE;
    const retn_status st = norm_sizes(rows, D);
    if (st != RETN_OK) return st;
    if (rows > 0 && (x == nullptr || mean == nullptr || rstd == nullptr || grad_y == nullptr || grad_x == nullptr))
        return RETN_ERR_NULL;
    const size_t n = sz(rows) * D * elem_bytes(dtype), we = D * elem_bytes(wdtype);
    const bool sums = grad_weight != nullptr || grad_bias != nullptr;
    const size_t need = sums ? layer_norm_bwd_workspace_bytes(rows, D, dtype) : 0;
    const Range in[] = {opt(x, n), opt(weight, we), opt(mean, f32(rows)), opt(rstd, f32(rows)), opt(grad_y, n)};
    const Range out[] = {opt(grad_x, n), opt(grad_weight, we), opt(grad_bias, we), sums ? opt(workspace, need) : Range{0, 0}};
    if (clash(in, out)) return RETN_ERR_ALIAS;
    if (bad_workspace(workspace, workspace_bytes, need)) return RETN_ERR_WORKSPACE;
    if (rows == 0 && !sums) return RETN_OK;
    retn::NormArgs a{};
    a.x = x;
    a.w = weight;
    a.y = grad_x;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.gy = grad_y;
    a.gw = grad_weight;
    a.gb = grad_bias;
    a.rows = sz(rows);
    a.D = D;
    a.bf16 = dtype == RETN_BF16;
    a.w_bf16 = wdtype == RETN_BF16;
    a.workspace = sums ? static_cast<float*>(workspace) : nullptr;
    return done(retn::launch_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

retn_status rotary_table(float* table, const double* freq, int pairs, long long first, long long count, float magnitude,
                         void* stream) {
    if (pairs < 1 || count < 0 || first < 0) return RETN_ERR_SHAPE;
    if (pairs > kMaxHead / 2 || count > (1ll << 31) || sz(count) * pairs > kMaxLaunch || first > (1ll << 40))
        return RETN_ERR_UNSUPPORTED;
    if (count == 0) return RETN_OK;
    if (table == nullptr || freq == nullptr) return RETN_ERR_NULL;
    if (overlaps(span(table, f32(sz(count) * pairs * 2)), span(freq, sz(pairs) * sizeof(double)))) return RETN_ERR_ALIAS;
    return done(retn::launch_rotary_table(table, freq, pairs, first, count, magnitude, static_cast<hipStream_t>(stream)));
}

retn_status rotary_fwd(const void* q, const void* k, void* out_q, void* out_k, const long long* strides,
                       const float* table, long long table_len, const long long* positions, int positions_per_batch,
                       long long first, int B, int Hq, int Hk, int N, int d, int rot, int interleaved, float q_scale,
                       float k_scale, retn_dtype dtype, void* stream) {
    return rotary_common(q, k, out_q, out_k, strides, table, table_len, positions, positions_per_batch, first, B, Hq, Hk, N,
                         d, rot, interleaved, q_scale, k_scale, dtype, stream, false);
}

retn_status rotary_bwd(const void* grad_q, const void* grad_k, void* out_q, void* out_k, const long long* strides,
                       const float* table, long long table_len, const long long* positions, int positions_per_batch,
                       long long first, int B, int Hq, int Hk, int N, int d, int rot, int interleaved, float q_scale,
                       float k_scale, retn_dtype dtype, void* stream) {
    return rotary_common(grad_q, grad_k, out_q, out_k, strides, table, table_len, positions, positions_per_batch, first, B,
                         Hq, Hk, N, d, rot, interleaved, q_scale, k_scale, dtype, stream, true);
}

retn_status causal_conv_fwd(const void* x, long long ldx, const void* weight, const void* bias,
                            void* y, const void* state_in, void* state_out, const int* lengths, int B, int N, int D, int K,
                            int silu, retn_dtype dtype, retn_dtype wdtype, void* stream) {
    return conv_forward(x, ldx, weight, bias, y, state_in, state_out, lengths, B, N, D, K, silu, dtype, wdtype, stream, false);
}

retn_status causal_conv_fwd_padded(const void* x, long long ldx, const void* weight, const void* bias,
                                   void* y, const void* state_in, void* state_out, const int* lengths, int B, int N, int D,
                                   int K, int silu, retn_dtype dtype, retn_dtype wdtype, void* stream) {
    return conv_forward(x, ldx, weight, bias, y, state_in, state_out, lengths, B, N, D, K, silu, dtype, wdtype, stream, true);
}

size_t causal_conv_bwd_workspace_bytes(int B, int N, int D, int K, retn_dtype dtype) {
    if (!valid_dtype(dtype) || conv_sizes(B, N, D, K) != RETN_OK) return 0;
    return retn::conv_bwd_workspace(B, N, D, K);
}

retn_status causal_conv_bwd(const void* x, long long ldx, const void* weight, const void* bias, const void* state_in,
                            const void* grad_y, const void* grad_state_out, const int* lengths, void* grad_x,
                            void* grad_weight, void* grad_bias, void* grad_state_in, int B, int N, int D, int K, int silu,
                            retn_dtype dtype, retn_dtype wdtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (!valid_types(dtype, wdtype)) return RETN_ERR_DTYPE;
    const retn_status st = conv_sizes(B, N, D, K);
    if (st != RETN_OK) return st;
    if (ldx < D) return RETN_ERR_SHAPE;
    if (ldx >= kMaxRow) return RETN_ERR_UNSUPPORTED;
    const size_t tokens = sz(B) * N, es = elem_bytes(dtype), we = elem_bytes(wdtype), sb = sz(B) * (K - 1) * D * es;
    // workgroups: a block of 32 channels or more of each sequence's tiles, whose sums the workspace holds
    if (retn::conv_bwd_workspace(B, N, D, K) / (f32(D) * (K + 1)) * (sz(D) / 32 + 1) >= kMaxGroups)
        return RETN_ERR_UNSUPPORTED;
    if ((tokens > 0 && (x == nullptr || grad_y == nullptr || grad_x == nullptr)) || weight == nullptr) return RETN_ERR_NULL;
    const bool sums = grad_weight != nullptr || grad_bias != nullptr;
    const size_t need = sums ? causal_conv_bwd_workspace_bytes(B, N, D, K, dtype) : 0;
    const Range in[] = {opt(x, rows_bytes(tokens, ldx, D, es)), span(weight, sz(D) * K * we), opt(bias, D * we),
                        opt(state_in, sb), opt(grad_y, tokens * D * es), opt(grad_state_out, sb),
                        opt(lengths, sizeof(int) * sz(B))};
    const Range out[] = {opt(grad_x, tokens * D * es), opt(grad_weight, sz(D) * K * we), opt(grad_bias, D * we),
                         opt(grad_state_in, sb), sums ? opt(workspace, need) : Range{0, 0}};
    if (clash(in, out)) return RETN_ERR_ALIAS;
    if (bad_workspace(workspace, workspace_bytes, need)) return RETN_ERR_WORKSPACE;
    if (tokens == 0 && !sums && grad_state_in == nullptr) return RETN_OK;
    retn::ConvArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.w = weight;
    a.b = bias;
    a.lengths = lengths;
    a.state_in = state_in;
    a.y = grad_x;
    a.gy = grad_y;
    a.gstate_out = grad_state_out;
    a.gstate_in = grad_state_in;
    a.gw = grad_weight;
    a.gb = grad_bias;
    a.B = B;
    a.N = N;
    a.D = D;
    a.K = K;
    a.silu = silu != 0;
    a.bf16 = dtype == RETN_BF16;
    a.w_bf16 = wdtype == RETN_BF16;
    a.workspace = sums ? static_cast<float*>(workspace) : nullptr;
    return done(retn::launch_conv_bwd(a, static_cast<hipStream_t>(stream)));
}

retn_status causal_conv_step(const void* x, long long ldx, const void* weight, const void* bias, void* state, void* y,
                             int B, int D, int K, int silu, retn_dtype dtype, retn_dtype wdtype, void* stream) {
    if (!valid_types(dtype, wdtype)) return RETN_ERR_DTYPE;
    const retn_status st = conv_sizes(B, 1, D, K);
    if (st != RETN_OK) return st;
    if (ldx < D) return RETN_ERR_SHAPE;
    if (ldx >= kMaxRow) return RETN_ERR_UNSUPPORTED;
    if (B == 0) return RETN_OK;
    if (x == nullptr || weight == nullptr || state == nullptr || y == nullptr) return RETN_ERR_NULL;
    const size_t es = elem_bytes(dtype), we = elem_bytes(wdtype);
    const Range in[] = {span(x, rows_bytes(B, ldx, D, es)), span(weight, sz(D) * K * we), opt(bias, D * we)};
    const Range out[] = {span(state, sz(B) * (K - 1) * D * es), span(y, sz(B) * D * es)};
    if (clash(in, out)) return RETN_ERR_ALIAS;
    retn::ConvArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.w = weight;
    a.b = bias;
    a.state_out = state;
    a.y = y;
    a.B = B;
    a.N = 1;
    a.D = D;
    a.K = K;
    a.silu = silu != 0;
    a.bf16 = dtype == RETN_BF16;
    a.w_bf16 = wdtype == RETN_BF16;
    return done(retn::launch_conv_step(a, static_cast<hipStream_t>(stream)));
}

size_t selective_scan_workspace_bytes(int B, int N, int D, int G, int S) {
    if (scan_sizes(B, N, D, G, S) != RETN_OK || B == 0 || N == 0) return 0;
    return f32(retn::scan_fwd_plan(B, N, D, G, S).total);
}

retn_status selective_scan_fwd(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                               const float* Dskip, const void* z, const float* dt_bias, void* y, const float* state_in,
                               float* state_out, const int* lengths, long long ldx, long long lddt, long long ldz,
                               long long ldb, long long ldc, int B, int N, int D, int G, int S, int softplus,
                               retn_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
    return scan_forward(x, dt, A, Bm, Cm, Dskip, z, dt_bias, y, state_in, state_out, lengths, ldx, lddt, ldz, ldb, ldc, B, N,
                        D, G, S, softplus, dtype, workspace, workspace_bytes, stream, false);
}

retn_status selective_scan_fwd_padded(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                                      const float* Dskip, const void* z, const float* dt_bias, void* y, const float* state_in,
                                      float* state_out, const int* lengths, long long ldx, long long lddt, long long ldz,
                                      long long ldb, long long ldc, int B, int N, int D, int G, int S, int softplus,
                                      retn_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
    return scan_forward(x, dt, A, Bm, Cm, Dskip, z, dt_bias, y, state_in, state_out, lengths, ldx, lddt, ldz, ldb, ldc, B, N,
                        D, G, S, softplus, dtype, workspace, workspace_bytes, stream, true);
}

size_t selective_scan_bwd_workspace_bytes(int B, int N, int D, int G, int S) {
    if (scan_sizes(B, N, D, G, S) != RETN_OK) return 0;
    return f32(retn::scan_bwd_plan(B, N, D, G, S).total);
}

retn_status selective_scan_bwd(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                               const float* Dskip, const void* z, const float* dt_bias, const float* state_in,
                               const void* grad_y, const float* grad_state_out, const int* lengths, void* grad_x,
                               void* grad_dt, float* grad_A, void* grad_B, void* grad_C, float* grad_D, void* grad_z,
                               float* grad_dt_bias, float* grad_state_in, long long ldx, long long lddt, long long ldz,
                               long long ldb, long long ldc, int B, int N, int D, int G, int S, int softplus,
                               retn_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (!valid_dtype(dtype)) return RETN_ERR_DTYPE;
    const retn_status st = scan_sizes(B, N, D, G, S);
    if (st != RETN_OK) return st;
    const long long gs = static_cast<long long>(G) * S;
    if (ldx < D || lddt < D || (z != nullptr && ldz < D) || ldb < gs || ldc < gs) return RETN_ERR_SHAPE;
    if (far_rows(ldx, lddt, z != nullptr ? ldz : 0, ldb, ldc)) return RETN_ERR_UNSUPPORTED;
    const size_t tokens = sz(B) * N, es = elem_bytes(dtype), ss = f32(sz(B) * D * S);
    if (tokens > 0 && (x == nullptr || dt == nullptr || A == nullptr || Bm == nullptr || Cm == nullptr || grad_y == nullptr ||
                       grad_x == nullptr || grad_dt == nullptr || grad_B == nullptr || grad_C == nullptr ||
                       (z != nullptr && grad_z == nullptr)))
        return RETN_ERR_NULL;
    if (grad_A == nullptr || (B > 0 && A == nullptr)) return RETN_ERR_NULL;
    const size_t need = selective_scan_bwd_workspace_bytes(B, N, D, G, S);
    const size_t bc = tokens * gs * es;
    const Range in[] = {opt(x, rows_bytes(tokens, ldx, D, es)), opt(dt, rows_bytes(tokens, lddt, D, es)),
                        opt(A, f32(sz(D) * S)), opt(Bm, rows_bytes(tokens, ldb, gs, es)),
                        opt(Cm, rows_bytes(tokens, ldc, gs, es)), opt(Dskip, f32(D)), opt(dt_bias, f32(D)),
                        opt(z, rows_bytes(tokens, ldz, D, es)), opt(state_in, ss), opt(grad_y, tokens * D * es),
                        opt(grad_state_out, ss), opt(lengths, sizeof(int) * sz(B))};
    const Range out[] = {opt(grad_x, tokens * D * es), opt(grad_dt, tokens * D * es), opt(grad_A, f32(sz(D) * S)),
                         opt(grad_B, bc), opt(grad_C, bc), opt(grad_D, f32(D)),
                         opt(z != nullptr ? grad_z : nullptr, tokens * D * es), opt(grad_dt_bias, f32(D)),
                         opt(grad_state_in, ss), opt(workspace, need)};
    if (clash(in, out)) return RETN_ERR_ALIAS;
    if (bad_workspace(workspace, workspace_bytes, need)) return RETN_ERR_WORKSPACE;
    retn::ScanArgs a{};
    a.x = x;
    a.dt = dt;
    a.z = z;
    a.Bm = Bm;
    a.Cm = Cm;
    a.ldx = ldx;
    a.lddt = lddt;
    a.ldz = ldz;
    a.ldb = ldb;
    a.ldc = ldc;
    a.A = A;
    a.Dskip = Dskip;
    a.bias = dt_bias;
    a.lengths = lengths;
    a.state_in = state_in;
    a.gy = grad_y;
    a.gstate_out = grad_state_out;
    a.gx = grad_x;
    a.gdt = grad_dt;
    a.gz = z != nullptr ? grad_z : nullptr;
    a.gB = grad_B;
    a.gC = grad_C;
    a.gA = grad_A;
    a.gD = grad_D;
    a.gbias = grad_dt_bias;
    a.gstate_in = grad_state_in;
    a.B = B;
    a.N = N;
    a.D = D;
    a.G = G;
    a.S = S;
    a.softplus = softplus != 0;
    a.bf16 = dtype == RETN_BF16;
    a.workspace = static_cast<float*>(workspace);
    return done(retn::launch_scan_bwd(a, retn::scan_bwd_plan(B, N, D, G, S), static_cast<hipStream_t>(stream)));
}

retn_status selective_scan_step(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                                const float* Dskip, const void* z, const float* dt_bias, float* state, void* y,
                                long long ldx, long long lddt, long long ldz, long long ldb, long long ldc, int B, int D,
                                int G, int S, int softplus, retn_dtype dtype, void* stream) {
    if (!valid_dtype(dtype)) return RETN_ERR_DTYPE;
    const retn_status st = scan_sizes(B, 1, D, G, S);
    if (st != RETN_OK) return st;
    const long long gs = static_cast<long long>(G) * S;
    if (ldx < D || lddt < D || (z != nullptr && ldz < D) || ldb < gs || ldc < gs) return RETN_ERR_SHAPE;
    if (far_rows(ldx, lddt, z != nullptr ? ldz : 0, ldb, ldc)) return RETN_ERR_UNSUPPORTED;
    if (B == 0) return RETN_OK;
    if (x == nullptr || dt == nullptr || A == nullptr || Bm == nullptr || Cm == nullptr || state == nullptr || y == nullptr)
        return RETN_ERR_NULL;
    const size_t es = elem_bytes(dtype);
    const Range in[] = {span(x, rows_bytes(B, ldx, D, es)), span(dt, rows_bytes(B, lddt, D, es)), span(A, f32(sz(D) * S)),
                        span(Bm, rows_bytes(B, ldb, gs, es)), span(Cm, rows_bytes(B, ldc, gs, es)), opt(Dskip, f32(D)),
                        opt(dt_bias, f32(D)), opt(z, rows_bytes(B, ldz, D, es))};
    const Range out[] = {span(state, f32(sz(B) * D * S)), span(y, sz(B) * D * es)};
    if (clash(in, out)) return RETN_ERR_ALIAS;
    retn::ScanArgs a{};
    a.x = x;
    a.dt = dt;
    a.z = z;
    a.Bm = Bm;
    a.Cm = Cm;
    a.ldx = ldx;
    a.lddt = lddt;
    a.ldz = ldz;
    a.ldb = ldb;
    a.ldc = ldc;
    a.A = A;
    a.Dskip = Dskip;
    a.bias = dt_bias;
    a.state_out = state;
    a.y = y;
    a.B = B;
    a.N = 1;
    a.D = D;
    a.G = G;
    a.S = S;
    a.softplus = softplus != 0;
    a.bf16 = dtype == RETN_BF16;
    return done(retn::launch_scan_step(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
