// Argument checks shared by the C ABI of the operators around the retention: overlapping
// buffers, workspaces, strided views of heads.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "validate.h"

namespace {

constexpr int kMaxHead = 256;
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

}  // namespace
