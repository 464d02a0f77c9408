// C ABI of the projections (the matrix product with its epilogue, the gated feed-forward
// block) and of the head norms with rotary positions: argument validation, workspaces and
// the order of launches.  As in api.cpp, every argument is checked before anything is
// enqueued.

#include "../../include/retention.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "launch.h"
#include "proj.h"
#include "views.h"

namespace {

using retn::ProjArgs;
using retn::ProjGroup;

constexpr int kMaxWidth = 1 << 20;
constexpr long long kMaxRows = 1ll << 28;             // tiles of 128 rows in a launch of 2^32 threads
constexpr unsigned long long kMaxElems = 1ull << 34;

bool valid_act(retn_activation a) { return a >= RETN_ACT_NONE && a <= RETN_ACT_SILU; }

retn_status proj_sizes(long long rows, int N, int K, long long ldx) {
    if (rows < 0 || N < 1 || K < 1 || ldx < K) return RETN_ERR_SHAPE;
    if (N > kMaxWidth || K > kMaxWidth || ldx > kMaxWidth || rows >= kMaxRows || sz(rows) * sz(std::max(N, K)) >= kMaxElems ||
        sz(N) * sz(K) >= kMaxElems)
        return RETN_ERR_UNSUPPORTED;
    return RETN_OK;
}

// Elements of 16 bytes, and a width in whole ones.
int unit(bool bf16) { return bf16 ? 8 : 4; }
int padded(int n, bool bf16) { return (n + unit(bf16) - 1) / unit(bf16) * unit(bf16); }
bool whole(long long n, bool bf16) { return n % unit(bf16) == 0; }

// Workspace laid out piece by piece, on 256-byte boundaries.
struct Layout {
    size_t total = 0;
    size_t take(size_t bytes) {
        const size_t at = total;
        total += (bytes + 255) & ~static_cast<size_t>(255);
        return at;
    }
};

// An operand: where it is read, and its row stride.
struct Rows {
    const void* p;
    long long ld;
};

struct Call {
    bool bf16;
    size_t es;
    char* ws;
    hipStream_t st;
    hipError_t err = hipSuccess;

    retn::PackArgs packs{};

    // The rows as they lie, or where the next `lay` puts them, with padded widths.
    Rows rows(const void* p, long long ld, size_t n, int width, size_t at) {
        if (aligned16(p) && whole(ld, bf16) && whole(width, bf16)) return Rows{p, ld};
        const int w = padded(width, bf16);
        packs.one[packs.n++] = retn::PackArgs::One{p, ld, ws + at, w, n, width};
        return Rows{ws + at, w};
    }
    void lay() {
        if (err == hipSuccess && packs.n > 0) err = retn::launch_proj_pack(packs, bf16, st);
        packs.n = 0;
    }
    // x W^T of few rows, read as they lie
    void small(const ProjArgs& a, retn::ProjKind kind) {
        if (err == hipSuccess) err = retn::launch_proj_small(a, kind, bf16, st);
    }
    void product(const ProjArgs& a, retn::ProjKind kind, bool a_red, bool b_red) {
        lay();
        if (err == hipSuccess) err = retn::launch_proj(a, kind, bf16, a_red, b_red, st);
    }
};

ProjGroup group(Rows a, Rows b, void* c, long long ldc, int M, int N, int bn) {
    ProjGroup g{};
    g.a = a.p;
    g.lda = static_cast<int>(a.ld);
    g.b = b.p;
    g.ldb = static_cast<int>(b.ld);
    g.c = c;
    g.ldc = ldc;
    g.M = M;
    g.N = N;
    g.bn = bn;
    return g;
}
ProjArgs product_of(int red, int red_rows) {
    ProjArgs a{};
    a.ngroups = 1;
    a.red = red;
    a.red_rows = red_rows;
    a.phases = 1;
    return a;
}
// Partial sums of a product of these sizes (they decide how it is cut).
size_t partial(int M, int N, int red, bool bf16, retn::ProjKind kind = retn::kProjLinear, int phases = 1) {
    ProjArgs a = product_of(red, red);
    a.phases = phases;
    a.g[0].M = M;
    a.g[0].N = N;
    return retn::proj_partial_bytes(a, kind, bf16);
}

struct LinearPlan {
    size_t x, w, part, total;
};
LinearPlan linear_plan(int M, int N, int K, bool bf16, bool aligned) {
    const size_t es = bf16 ? 2 : 4;
    LinearPlan p{};
    if (retn::proj_small(M, N)) return p;
    Layout l;
    p.x = l.take(aligned ? 0 : sz(M) * padded(K, bf16) * es);
    p.w = l.take(aligned ? 0 : sz(N) * padded(K, bf16) * es);
    p.part = l.take(partial(M, N, padded(K, bf16), bf16));
    p.total = l.total;
    return p;
}

struct LinearBwdPlan {
    size_t x, w, gz, part, sums, total;
};
LinearBwdPlan linear_bwd_plan(int M, int N, int K, bool act, bool bf16, bool aligned) {
    const size_t es = bf16 ? 2 : 4;
    LinearBwdPlan p{};
    Layout l;
    p.x = l.take(aligned ? 0 : sz(M) * padded(K, bf16) * es);
    p.w = l.take(aligned ? 0 : sz(N) * padded(K, bf16) * es);
    p.gz = l.take(aligned && !act ? 0 : sz(M) * padded(N, bf16) * es);
    p.part = l.take(std::max(partial(M, K, padded(N, bf16), bf16), partial(N, K, M, bf16)));
    p.sums = l.take(retn::slope_partial_bytes(sz(M), N));
    p.total = l.total;
    return p;
}

struct FfnPlan {
    size_t x, wg, wu, wd, h, part, total;
};
FfnPlan ffn_plan(int M, int D, int F, bool bf16, bool aligned) {
    const size_t es = bf16 ? 2 : 4;
    FfnPlan p{};
    Layout l;
    if (retn::proj_small(M, std::max(D, F))) {
        p.h = l.take(sz(M) * padded(F, bf16) * es);
        p.total = l.total;
        return p;
    }
    p.x = l.take(aligned ? 0 : sz(M) * padded(D, bf16) * es);
    p.wg = l.take(aligned ? 0 : sz(F) * padded(D, bf16) * es);
    p.wu = l.take(aligned ? 0 : sz(F) * padded(D, bf16) * es);
    p.wd = l.take(aligned ? 0 : sz(D) * padded(F, bf16) * es);
    p.h = l.take(sz(M) * padded(F, bf16) * es);
    p.part = l.take(std::max(partial(M, padded(F, bf16), padded(D, bf16), bf16, retn::kProjGated),
                             partial(M, D, padded(F, bf16), bf16)));
    p.total = l.total;
    return p;
}

struct FfnBwdPlan {
    size_t x, wg, wu, wd, gy, gg, gu, h, part, total;
};
// The three weights' gradients, one launch.
ProjArgs weight_grads(Rows x, Rows gy, Rows gg, Rows gu, Rows h, void* gwg, void* gwu, void* gwd, int M, int D, int F) {
    ProjArgs a = product_of(M, M);
    a.ngroups = 3;
    a.g[0] = group(gg, x, gwg, D, F, D, D);
    a.g[1] = group(gu, x, gwu, D, F, D, D);
    a.g[2] = group(gy, h, gwd, F, D, F, F);
    return a;
}
FfnBwdPlan ffn_bwd_plan(int M, int D, int F, bool bf16, bool aligned) {
    const size_t es = bf16 ? 2 : 4, hidden = sz(M) * padded(F, bf16) * es;
    FfnBwdPlan p{};
    Layout l;
    p.x = l.take(aligned ? 0 : sz(M) * padded(D, bf16) * es);
    p.wg = l.take(aligned ? 0 : sz(F) * padded(D, bf16) * es);
    p.wu = l.take(aligned ? 0 : sz(F) * padded(D, bf16) * es);
    p.wd = l.take(aligned ? 0 : sz(D) * padded(F, bf16) * es);
    p.gy = l.take(aligned ? 0 : sz(M) * padded(D, bf16) * es);
    p.gg = l.take(hidden);
    p.gu = l.take(hidden);
    p.h = l.take(hidden);
    const Rows none{nullptr, 0};
    size_t part = partial(M, padded(F, bf16), padded(D, bf16), bf16, retn::kProjGatedBwd);
    part = std::max(part, partial(M, D, padded(F, bf16), bf16, retn::kProjLinear, 2));
    part = std::max(part, retn::proj_partial_bytes(
                              weight_grads(none, none, none, none, none, nullptr, nullptr, nullptr, M, D, F),
                              retn::kProjLinear, bf16));
    p.part = l.take(part);
    p.total = l.total;
    return p;
}

// Head norms with rotary positions: queries [0] and keys [1].
struct HeadsCall {
    const void *x[2], *gy[2], *w[2];
    void *out[2], *gw[2];
};
retn_status heads_common(const HeadsCall& h, const long long* strides, const float* table, long long table_len,
                         const long long* positions, int per_batch, long long first, int B, int Hq, int Hk, int N, int d,
                         int rot, int interleaved, float eps, float q_scale, float k_scale, retn_dtype dtype,
                         retn_dtype wdtype, void* workspace, size_t workspace_bytes, void* stream, bool backward) {
    if (!valid_types(dtype, wdtype)) return RETN_ERR_DTYPE;
    if (B < 0 || Hq < 0 || Hk < 0 || N < 0 || d < 1 || rot < 2 || rot > d || rot % 2 != 0 || table_len < 0 || !(eps >= 0.f))
        return RETN_ERR_SHAPE;
    if (d > kMaxHead || sz(B) * N > kMaxTokens || sz(B) * N * d >= (1ull << 32) || sz(Hq) + Hk > 65535 ||
        table_len > kMaxSpan)
        return RETN_ERR_UNSUPPORTED;
    const bool none = B == 0 || N == 0 || Hq + Hk == 0, sums = h.gw[0] != nullptr || h.gw[1] != nullptr;
    if (none && !sums) return RETN_OK;
    const int H[2] = {Hq, Hk}, each = backward ? 3 : 2;   // tensors of a side: x, (its gradient,) output
    const size_t es = elem_bytes(dtype), we = d * elem_bytes(wdtype), need = sums ? retn::heads_partial_bytes(d) : 0;
    View v[2][3]{};
    Range r[2][3]{};
    if (!none) {
        for (int o = 0; o < 2; ++o)
            if (H[o] > 0 && (h.x[o] == nullptr || h.out[o] == nullptr || (backward && h.gy[o] == nullptr))) return RETN_ERR_NULL;
        if (strides == nullptr || table == nullptr) return RETN_ERR_NULL;
        // (the kernel reads row 0 for a position outside of the table)
        if (positions == nullptr ? first < 0 || first > table_len - N : table_len < 1) return RETN_ERR_SHAPE;
        for (int o = 0; o < 2; ++o) {
            if (H[o] == 0) continue;
            const void* const ptr[3] = {h.x[o], backward ? h.gy[o] : h.out[o], h.out[o]};
            for (int i = 0; i < each; ++i) {
                const long long* s = strides + 3 * (each * o + i);
                v[o][i] = View{s[0], s[1], s[2]};
                if (!valid_view(v[o][i], B, H[o], N)) return RETN_ERR_SHAPE;
                r[o][i] = span(ptr[i], view_bytes(v[o][i], B, H[o], N, d, es));
            }
            if (!own_places(v[o][each - 1], B, H[o], N, d)) return RETN_ERR_ALIAS;
        }
    }
    const Range rt = none ? Range{0, 0} : span(table, f32(sz(table_len) * rot));
    const Range rp = none ? Range{0, 0} : opt(positions, sizeof(long long) * sz(N) * (per_batch ? B : 1));
    const Range small_out[] = {opt(h.gw[0], we), opt(h.gw[1], we), sums ? opt(workspace, need) : Range{0, 0}};
    const Range small_in[] = {rt, rp, opt(h.w[0], we), opt(h.w[1], we)};
    if (clash(small_in, small_out)) return RETN_ERR_ALIAS;
    for (int o = 0; o < 2; ++o) {
        const int out = each - 1;
        for (const Range& s : small_in)
            if (overlaps(r[o][out], s)) return RETN_ERR_ALIAS;
        for (const Range& s : small_out)
            for (int i = 0; i < each; ++i)
                if (overlaps(r[o][i], s)) return RETN_ERR_ALIAS;
        for (int o2 = 0; o2 < 2; ++o2)
            for (int i = 0; i < each; ++i) {
                if ((o2 == o && i == out) || !overlaps(r[o][out], r[o2][i])) continue;
                const View &a = v[o][out], &b = v[o2][i];
                const void* const from = backward ? h.gy[o] : h.x[o];
                const bool in_place = o2 == o && i == out - 1 && from == h.out[o] && (B <= 1 || a.sb == b.sb) &&
                                      (H[o] <= 1 || a.sh == b.sh) && (N <= 1 || a.sn == b.sn);
                if (!in_place && !side_by_side(r[o][out].lo, a, H[o], r[o2][i].lo, b, H[o2], B, N, d, es)) return RETN_ERR_ALIAS;
            }
    }
    if (bad_workspace(workspace, workspace_bytes, need)) return RETN_ERR_WORKSPACE;
    retn::HeadsArgs a{};
    retn::HeadsView* const views[2] = {&a.q, &a.k};
    const float scale[2] = {q_scale, k_scale};
    for (int o = 0; o < 2; ++o) {
        const View &x = v[o][0], &g = v[o][1], &out = v[o][each - 1];
        *views[o] = retn::HeadsView{h.x[o], h.gy[o], h.out[o], x.sb, x.sh, x.sn, g.sb, g.sh, g.sn, out.sb, out.sh, out.sn,
                                    none ? 0 : H[o], scale[o], h.w[o], h.gw[o]};
    }
    a.table = table;
    a.table_len = table_len;
    a.pos = positions;
    a.pos_batched = per_batch != 0;
    a.first = first;
    a.B = B;
    a.N = N;
    a.d = d;
    a.rot = rot;
    a.eps = eps;
    a.interleaved = interleaved != 0;
    a.backward = backward;
    a.bf16 = dtype == RETN_BF16;
    a.w_bf16 = wdtype == RETN_BF16;
    a.part = sums ? static_cast<float*>(workspace) : nullptr;
    return done(retn::launch_heads(a, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t linear_workspace_bytes(long long rows, int N, int K, retn_dtype dtype, int aligned) {
    if (!valid_dtype(dtype) || proj_sizes(rows, N, K, K) != RETN_OK || rows == 0) return 0;
    return linear_plan(static_cast<int>(rows), N, K, dtype == RETN_BF16, aligned != 0).total;
}

retn_status linear_fwd(const void* x, long long ldx, const void* weight, const void* bias, const void* residual, void* y,
                       void* pre, long long rows, int N, int K, retn_activation activation, retn_dtype dtype,
                       retn_dtype bdtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (!valid_types(dtype, bdtype)) return RETN_ERR_DTYPE;
    const retn_status st = proj_sizes(rows, N, K, ldx);
    if (st != RETN_OK) return st;
    if (!valid_act(activation)) return RETN_ERR_SHAPE;
    if (rows == 0) return RETN_OK;
    if (x == nullptr || weight == nullptr || y == nullptr) return RETN_ERR_NULL;
    const bool bf16 = dtype == RETN_BF16;
    const int M = static_cast<int>(rows);
    const size_t es = elem_bytes(dtype), out = sz(M) * N * es;
    const bool aligned = aligned16(x) && aligned16(weight) && whole(ldx, bf16) && whole(K, bf16) && whole(N, bf16);
    const LinearPlan p = linear_plan(M, N, K, bf16, aligned);
    const Range in[] = {span(x, rows_bytes(sz(M), ldx, K, es)), span(weight, sz(N) * K * es), opt(bias, N * elem_bytes(bdtype)),
                        opt(residual == y ? nullptr : residual, out)};
    const Range outs[] = {span(y, out), opt(pre, out), opt(workspace, p.total)};
    if (clash(in, outs)) return RETN_ERR_ALIAS;
    if (bad_workspace(workspace, workspace_bytes, p.total)) return RETN_ERR_WORKSPACE;
    Call c{bf16, es, static_cast<char*>(workspace), static_cast<hipStream_t>(stream)};
    const bool small = retn::proj_small(M, N);
    const Rows rx = small ? Rows{x, ldx} : c.rows(x, ldx, sz(M), K, p.x);
    const Rows rw = small ? Rows{weight, K} : c.rows(weight, K, sz(N), K, p.w);
    const int red = small ? K : padded(K, bf16);
    ProjArgs a = product_of(red, red);
    a.g[0] = group(rx, rw, y, N, M, N, N);
    a.e.bias = bias;
    a.e.bias_f32 = bdtype == RETN_F32;
    a.e.act = activation;
    a.e.res = residual;
    a.e.pre = pre;
    a.part = reinterpret_cast<float*>(c.ws + p.part);
    if (small)
        c.small(a, retn::kProjLinear);
    else
        c.product(a, retn::kProjLinear, true, true);
    return done(c.err);
}

size_t linear_bwd_workspace_bytes(long long rows, int N, int K, retn_activation activation, retn_dtype dtype, int aligned) {
    if (!valid_dtype(dtype) || proj_sizes(rows, N, K, K) != RETN_OK || !valid_act(activation)) return 0;
    return linear_bwd_plan(static_cast<int>(rows), N, K, activation != RETN_ACT_NONE, dtype == RETN_BF16, aligned != 0).total;
}

retn_status linear_bwd(const void* x, long long ldx, const void* weight, const void* pre, const void* grad_y, void* grad_x,
                       void* grad_weight, void* grad_bias, long long rows, int N, int K, retn_activation activation,
                       retn_dtype dtype, retn_dtype bdtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (!valid_types(dtype, bdtype)) return RETN_ERR_DTYPE;
    const retn_status st = proj_sizes(rows, N, K, ldx);
    if (st != RETN_OK) return st;
    if (!valid_act(activation)) return RETN_ERR_SHAPE;
    const bool bf16 = dtype == RETN_BF16, act = activation != RETN_ACT_NONE;
    const int M = static_cast<int>(rows);
    if (M > 0 && ((grad_weight != nullptr && x == nullptr) || (grad_x != nullptr && weight == nullptr) ||
                  grad_y == nullptr || (act && pre == nullptr)))
        return RETN_ERR_NULL;
    if (grad_x == nullptr && grad_weight == nullptr && grad_bias == nullptr) return RETN_OK;
    const size_t es = elem_bytes(dtype), out = sz(M) * N * es, we = sz(N) * K * es;
    const bool aligned = aligned16(x) && aligned16(weight) && aligned16(grad_y) && whole(ldx, bf16) && whole(K, bf16) &&
                         whole(N, bf16);
    const LinearBwdPlan p = linear_bwd_plan(M, N, K, act, bf16, aligned);
    const Range in[] = {opt(x, rows_bytes(sz(M), ldx, K, es)), opt(weight, we), opt(act ? pre : nullptr, out), opt(grad_y, out)};
    const Range outs[] = {opt(grad_x, sz(M) * K * es), opt(grad_weight, we), opt(grad_bias, N * elem_bytes(bdtype)),
                          opt(workspace, p.total)};
    if (clash(in, outs)) return RETN_ERR_ALIAS;
    if (bad_workspace(workspace, workspace_bytes, p.total)) return RETN_ERR_WORKSPACE;
    Call c{bf16, es, static_cast<char*>(workspace), static_cast<hipStream_t>(stream)};
    const bool products = grad_x != nullptr || grad_weight != nullptr;
    const bool in_place = !act && aligned16(grad_y) && whole(N, bf16);
    Rows gz{grad_y, N};
    if ((products && !in_place) || grad_bias != nullptr) {
        retn::SlopeArgs s{};
        s.gy = grad_y;
        s.pre = act ? pre : nullptr;
        s.act = activation;
        s.rows = sz(M);
        s.N = N;
        s.bf16 = bf16;
        if (products && !in_place) {
            gz = Rows{c.ws + p.gz, padded(N, bf16)};
            s.gz = c.ws + p.gz;
            s.ldz = padded(N, bf16);
        }
        if (grad_bias != nullptr) {
            s.part = reinterpret_cast<float*>(c.ws + p.sums);
            s.sums = grad_bias;
            s.sums_f32 = bdtype == RETN_F32;
        }
        c.err = retn::launch_slope(s, c.st);
    }
    float* const part = reinterpret_cast<float*>(c.ws + p.part);
    Rows rw{nullptr, 8}, rx{nullptr, 8};
    if (grad_x != nullptr && M > 0) rw = c.rows(weight, K, sz(N), K, p.w);
    if (grad_weight != nullptr && M > 0) rx = c.rows(x, ldx, sz(M), K, p.x);
    if (grad_x != nullptr && M > 0) {
        ProjArgs a = product_of(padded(N, bf16), N);
        a.g[0] = group(gz, rw, grad_x, K, M, K, K);
        a.part = part;
        c.product(a, retn::kProjLinear, true, false);
    }
    if (grad_weight != nullptr) {
        ProjArgs a = product_of(M, M);
        a.g[0] = group(gz, rx, grad_weight, K, N, K, K);
        a.part = part;
        c.product(a, retn::kProjLinear, false, false);
    }
    return done(c.err);
}

size_t gated_ffn_workspace_bytes(long long rows, int D, int F, retn_dtype dtype, int aligned) {
    if (!valid_dtype(dtype) || proj_sizes(rows, F, D, D) != RETN_OK || rows == 0) return 0;
    return ffn_plan(static_cast<int>(rows), D, F, dtype == RETN_BF16, aligned != 0).total;
}

retn_status gated_ffn_fwd(const void* x, long long ldx, const void* w_gate, const void* w_up, const void* w_down,
                          const void* residual, void* y, void* gate, void* up, long long rows, int D, int F,
                          retn_activation activation, retn_dtype dtype, void* workspace, size_t workspace_bytes,
                          void* stream) {
    if (!valid_dtype(dtype)) return RETN_ERR_DTYPE;
    const retn_status st = proj_sizes(rows, F, D, ldx);
    if (st != RETN_OK) return st;
    if (!valid_act(activation)) return RETN_ERR_SHAPE;
    if (rows == 0) return RETN_OK;
    if (x == nullptr || w_gate == nullptr || w_up == nullptr || w_down == nullptr || y == nullptr ||
        (gate == nullptr) != (up == nullptr))
        return RETN_ERR_NULL;
    const bool bf16 = dtype == RETN_BF16;
    const int M = static_cast<int>(rows);
    const size_t es = elem_bytes(dtype), we = sz(D) * F * es, out = sz(M) * D * es, hidden = sz(M) * F * es;
    const bool aligned = aligned16(x) && aligned16(w_gate) && aligned16(w_up) && aligned16(w_down) && whole(ldx, bf16) &&
                         whole(D, bf16) && whole(F, bf16);
    const FfnPlan p = ffn_plan(M, D, F, bf16, aligned);
    const Range in[] = {span(x, rows_bytes(sz(M), ldx, D, es)), span(w_gate, we), span(w_up, we), span(w_down, we),
                        opt(residual == y ? nullptr : residual, out)};
    const Range outs[] = {span(y, out), opt(gate, hidden), opt(up, hidden), opt(workspace, p.total)};
    if (clash(in, outs)) return RETN_ERR_ALIAS;
    if (bad_workspace(workspace, workspace_bytes, p.total)) return RETN_ERR_WORKSPACE;
    Call c{bf16, es, static_cast<char*>(workspace), static_cast<hipStream_t>(stream)};
    const bool small = retn::proj_small(M, std::max(D, F));
    const Rows rx = small ? Rows{x, ldx} : c.rows(x, ldx, sz(M), D, p.x);
    const Rows rg = small ? Rows{w_gate, D} : c.rows(w_gate, D, sz(F), D, p.wg);
    const Rows ru = small ? Rows{w_up, D} : c.rows(w_up, D, sz(F), D, p.wu);
    const Rows rd_w = small ? Rows{w_down, F} : c.rows(w_down, F, sz(D), F, p.wd);
    const int rd = small ? D : padded(D, bf16), rf = padded(F, bf16);
    const Rows h{c.ws + p.h, rf};
    float* const part = reinterpret_cast<float*>(c.ws + p.part);
    ProjArgs a = product_of(rd, rd);
    a.g[0] = group(rx, rg, c.ws + p.h, rf, M, rf, F);
    a.g[0].b2 = ru.p;      // (one stride: a copy's is the padded width, which a width that needs none equals)
    a.e.act = activation;
    a.e.gate = gate;
    a.e.up = up;
    a.e.gate_ld = F;
    a.e.gate_n = F;
    a.part = part;
    if (small)
        c.small(a, retn::kProjGated);
    else
        c.product(a, retn::kProjGated, true, true);
    const int rr = small ? F : rf;
    ProjArgs b = product_of(rr, rr);
    b.g[0] = group(h, rd_w, y, D, M, D, D);
    b.e.res = residual;
    b.part = part;
    if (small)
        c.small(b, retn::kProjLinear);
    else
        c.product(b, retn::kProjLinear, true, true);
    return done(c.err);
}

size_t gated_ffn_bwd_workspace_bytes(long long rows, int D, int F, retn_dtype dtype, int aligned) {
    if (!valid_dtype(dtype) || proj_sizes(rows, F, D, D) != RETN_OK) return 0;
    return ffn_bwd_plan(static_cast<int>(rows), D, F, dtype == RETN_BF16, aligned != 0).total;
}

retn_status gated_ffn_bwd(const void* x, long long ldx, const void* w_gate, const void* w_up, const void* w_down,
                          const void* gate, const void* up, const void* grad_y, void* grad_x, void* grad_w_gate,
                          void* grad_w_up, void* grad_w_down, long long rows, int D, int F, retn_activation activation,
                          retn_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (!valid_dtype(dtype)) return RETN_ERR_DTYPE;
    const retn_status st = proj_sizes(rows, F, D, ldx);
    if (st != RETN_OK) return st;
    if (!valid_act(activation)) return RETN_ERR_SHAPE;
    const bool weights = grad_w_gate != nullptr;
    if (weights != (grad_w_up != nullptr) || weights != (grad_w_down != nullptr)) return RETN_ERR_NULL;
    if (rows > 0 && (x == nullptr || w_gate == nullptr || w_up == nullptr || w_down == nullptr || gate == nullptr ||
                     up == nullptr || grad_y == nullptr))
        return RETN_ERR_NULL;
    if ((grad_x == nullptr || rows == 0) && !weights) return RETN_OK;
    const bool bf16 = dtype == RETN_BF16;
    const int M = static_cast<int>(rows);
    const size_t es = elem_bytes(dtype), we = sz(D) * F * es, out = sz(M) * D * es, hidden = sz(M) * F * es;
    const bool aligned = aligned16(x) && aligned16(w_gate) && aligned16(w_up) && aligned16(w_down) && aligned16(grad_y) &&
                         whole(ldx, bf16) && whole(D, bf16) && whole(F, bf16);
    const FfnBwdPlan p = ffn_bwd_plan(M, D, F, bf16, aligned);
    const Range in[] = {opt(x, rows_bytes(sz(M), ldx, D, es)), opt(w_gate, we), opt(w_up, we), opt(w_down, we),
                        opt(gate, hidden), opt(up, hidden), opt(grad_y, out)};
    const Range outs[] = {opt(grad_x, out), opt(grad_w_gate, we), opt(grad_w_up, we), opt(grad_w_down, we),
                          opt(workspace, p.total)};
    if (clash(in, outs)) return RETN_ERR_ALIAS;
    if (bad_workspace(workspace, workspace_bytes, p.total)) return RETN_ERR_WORKSPACE;
    Call c{bf16, es, static_cast<char*>(workspace), static_cast<hipStream_t>(stream)};
    float* const part = reinterpret_cast<float*>(c.ws + p.part);
    const int pd = padded(D, bf16), pf = padded(F, bf16);
    const Rows gg{c.ws + p.gg, pf}, gu{c.ws + p.gu, pf}, h{c.ws + p.h, pf};
    Rows gy{grad_y, D}, rx{nullptr, pd}, rg{w_gate, D}, ru{w_up, D};
    if (M > 0) {
        gy = c.rows(grad_y, D, sz(M), D, p.gy);
        const Rows rw = c.rows(w_down, F, sz(D), F, p.wd);
        if (grad_x != nullptr) {
            rg = c.rows(w_gate, D, sz(F), D, p.wg);
            ru = c.rows(w_up, D, sz(F), D, p.wu);
        }
        if (weights) rx = c.rows(x, ldx, sz(M), D, p.x);
        ProjArgs a = product_of(pd, D);
        a.g[0] = group(gy, rw, nullptr, pf, M, pf, F);
        a.e.act = activation;
        a.e.gate = const_cast<void*>(gate);
        a.e.up = const_cast<void*>(up);
        a.e.gate_ld = F;
        a.e.gate_n = F;
        a.e.ggate = c.ws + p.gg;
        a.e.gup = c.ws + p.gu;
        a.e.prod = weights ? c.ws + p.h : nullptr;
        a.part = part;
        c.product(a, retn::kProjGatedBwd, true, false);
    }
    if (grad_x != nullptr && M > 0) {
        ProjArgs a = product_of(pf, F);
        a.phases = 2;
        a.g[0] = group(gg, rg, grad_x, D, M, D, D);
        a.g[0].a2 = gu.p;
        a.g[0].b2 = ru.p;
        a.part = part;
        c.product(a, retn::kProjLinear, true, false);
    }
    if (weights) {
        ProjArgs a = weight_grads(rx, gy, gg, gu, h, grad_w_gate, grad_w_up, grad_w_down, M, D, F);
        a.part = part;
        c.product(a, retn::kProjLinear, false, false);
    }
    return done(c.err);
}

size_t head_norm_rotary_bwd_workspace_bytes(int d) {
    return d < 1 || d > kMaxHead ? 0 : retn::heads_partial_bytes(d);
}

retn_status head_norm_rotary_fwd(const void* q, const void* k, void* out_q, void* out_k, const long long* strides,
                                 const void* q_weight, const void* k_weight, const float* table, long long table_len,
                                 const long long* positions, int positions_per_batch, long long first, int B, int Hq,
                                 int Hk, int N, int d, int rot, int interleaved, float eps, float q_scale, float k_scale,
                                 retn_dtype dtype, retn_dtype wdtype, void* stream) {
    HeadsCall h{};
    h.x[0] = q;
    h.x[1] = k;
    h.out[0] = out_q;
    h.out[1] = out_k;
    h.w[0] = q_weight;
    h.w[1] = k_weight;
    return heads_common(h, strides, table, table_len, positions, positions_per_batch, first, B, Hq, Hk, N, d, rot,
                        interleaved, eps, q_scale, k_scale, dtype, wdtype, nullptr, 0, stream, false);
}

retn_status head_norm_rotary_bwd(const void* q, const void* k, const void* grad_q, const void* grad_k, void* out_q,
                                 void* out_k, const long long* strides, const void* q_weight, const void* k_weight,
                                 void* grad_q_weight, void* grad_k_weight, const float* table, long long table_len,
                                 const long long* positions, int positions_per_batch, long long first, int B, int Hq,
                                 int Hk, int N, int d, int rot, int interleaved, float eps, float q_scale, float k_scale,
                                 retn_dtype dtype, retn_dtype wdtype, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    HeadsCall h{};
    h.x[0] = q;
    h.x[1] = k;
    h.gy[0] = grad_q;
    h.gy[1] = grad_k;
    h.out[0] = out_q;
    h.out[1] = out_k;
    h.w[0] = q_weight;
    h.w[1] = k_weight;
    h.gw[0] = grad_q_weight;
    h.gw[1] = grad_k_weight;
    return heads_common(h, strides, table, table_len, positions, positions_per_batch, first, B, Hq, Hk, N, d, rot,
                        interleaved, eps, q_scale, k_scale, dtype, wdtype, workspace, workspace_bytes, stream, true);
}

}  // extern "C"
