// Matrix products of a block's projections: C = A B with fp32 accumulation on the matrix
// cores and what follows a projection (bias, activation, residual, the gated product and its
// gradients) applied to the sums before they are stored.
//
// A workgroup owns a BM x BN tile of C and walks the reduction in steps of 128 bytes a row
// (64 bf16 or 32 fp32 elements).  Two to four steps of both operands lie in LDS, each as two halves
// of its rows (A: upper and lower, B: left and right), filled by asynchronous copies from memory
// whose instructions go out one at a time between the matrix instructions.  A wave owns 16-row
// blocks in both halves of either operand, so its tile falls into four quarters, and a step
// goes through them: upper left, upper right, lower right, lower left.  While a quarter's
// products run, the half that the next quarter brings in is read into registers; half of the
// step's halves are free again after each pair of quarters, where the workgroup meets, and are
// then filled for the step after the next.  So a copy has one to one and a half steps to
// arrive, and the matrix cores may run dry only at two barriers a step.
//
// Operands come in either order: reduction-major rows give 16-byte fragments as they lie;
// output-major rows (a transposed operand: a weight in the gradient of x, both operands in
// the gradient of a weight) are read by the transposing LDS loads (bf16), or by single words
// (fp32, whose matrix instructions are slow enough to hide them), so no operand is ever
// transposed in memory.
//
// Bound by the matrix cores in the main loop: 8192^3 bf16 runs at 1.32 to 1.41 PFLOP/s in any order of
// the operands (811, 785 and 791 us; the matrix cores busy 72 to 74% of the cycles), the rest goes to the
// barriers, where the older wave of a SIMD waits for the younger.  Short reductions are bound by the
// tails, in which a CU's one workgroup stores (8192 x 4096 x 1024: 70 us, 89 with gelu and two outputs).

#include "cdna4.h"
#include "common.h"
#include "launch.h"
#include "proj.h"
#include "proj_epi.h"
#include "vec_io.h"

#include <algorithm>
#include <mutex>
#include <type_traits>

namespace retn {
namespace {

constexpr uint32_t kOutside = 0x80000000u;   // a byte offset past every buffer resource here

// Half of an operand's tile in LDS: R rows of the output.
//   RED:  [R][128 bytes of the reduction]; the 16-byte unit u of row r sits at u ^ swz(r), so
//         the 16 rows of a fragment read cover all banks.
//   else: [elements of the step][R elements]; unit u of row r sits at u ^ swz(r).  A transposing
//         read of 32 lanes takes 32 bytes each from rows {0..3, 8..11} (plus 4, or 16): these
//         are spread over the 256 bytes of all banks; fp32 words come as 64 bytes from every fourth row.
template <typename T, bool RED, int R, int NW>
struct Half {
    static constexpr int kEs = sizeof(T), kStep = 128 / kEs;
    static constexpr int kRow = RED ? 128 : R * kEs;  // bytes of a row
    static constexpr int kBytes = R * 128;
    static constexpr int kCopies = R / 8 / NW;        // copies of 1 KB a wave makes for a step
    static constexpr int kBlocks = 4;                 // 16-row blocks that a wave may own
    static_assert(kCopies * 8 * NW == R && (RED || kRow >= 128), "whole copies");

    __device__ __forceinline__ static int swz(int r) {
        if (RED) return (r >> 1) & 7;
        if (kEs == 4) return ((r >> 2) & 3) << 2;
        return kRow == 128 ? 2 * (((r >> 1) & 1) | (((r >> 3) & 1) << 1)) : 2 * ((r & 3) | (((r >> 3) & 1) << 2));
    }

    uint32_t off[kCopies];      // lane's byte offset of each copy, from the half's start
    uint32_t fr[RED ? 2 : kBlocks];   // lane's LDS offset of fragments
    int unit;                   // RED: the unit that a lane copies (the same in every copy)

    // t0: the wave's first 16-row block of the half.
    __device__ __forceinline__ void init(int wave, int lane, int t0, int ld) {
        const int l16 = lane & 15, g4 = lane >> 4;
        unit = 0;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int o = (wave + NW * i) * 1024 + lane * 16, r = o / kRow, u = ((o % kRow) >> 4) ^ swz(r);
            off[i] = static_cast<uint32_t>(r) * ld * kEs + u * 16;
            static_assert(NW % 2 == 0, "the rows of a wave's copies are alike in their swizzle");
            if (RED) unit = u;
        }
        if constexpr (RED) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) fr[ks] = (t0 * 16 + l16) * 128 + (((ks * 4 + g4) ^ swz(l16)) << 4);
        } else if constexpr (kEs == 2) {
            const int r = 8 * g4 + (l16 >> 2);
#pragma unroll
            for (int t = 0; t < kBlocks; ++t)
                fr[t] = r * kRow + (((2 * (t0 + t) + ((l16 & 3) >> 1)) ^ swz(r)) << 4) + (l16 & 1) * 8;
        } else {
#pragma unroll
            for (int t = 0; t < kBlocks; ++t)
                fr[t] = 4 * g4 * kRow + (((4 * (t0 + t) + (l16 >> 2)) ^ (g4 << 2)) << 4) + (l16 & 3) * 4;
        }
    }
    // Fragment of the wave's row block t, half ks of the step, from the half at LDS address `at`.
    __device__ __forceinline__ u16x8_t read(uint32_t at, int t, int ks) const {
        if constexpr (RED) {
            return lds16a(at + fr[ks] + t * 16 * 128);
        } else if constexpr (kEs == 2) {
            const uint32_t p = at + fr[t] + ks * 32 * kRow;
            return cat(lds_tra(p), lds_tra(p + 4 * kRow));
        } else {
            typedef __attribute__((address_space(3))) const float lds_f32_t;
            const uint32_t p = at + fr[t] + ks * 16 * kRow;
            f32x4_t v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = *(lds_f32_t*)(static_cast<size_t>(p + j * kRow));
            return __builtin_bit_cast(u16x8_t, v);
        }
    }
};

// A value that the compiler keeps in scalar registers instead of loading it again.
template <typename V>
__device__ __forceinline__ V held(V v) {
    asm volatile("" : "+s"(v));
    return v;
}
// Where the copies of an operand's two halves come from, step after step: a resource each (empty
// where there is nothing: zeros arrive), the scalar offset, and (RED) how many of a row's units
// from here on hold elements of the reduction.
template <typename T, bool RED, int R>
struct Operand {
    static constexpr int kEs = sizeof(T), kStep = 128 / kEs, kEpu = 16 / kEs;
    uint64_t first, second, half;   // address of the tile in both phases, way to the second half
    int ld;
    uint32_t size[2];               // RED: bytes of a half; else: of its last row
    u32x4_t rs[2];
    uint32_t soff;
    int units;

    __device__ __forceinline__ void init(const void* a, const void* b, int ld_, int at, int count, int red) {
        ld = held(ld_);
        const uint64_t o = static_cast<uint64_t>(at) * (RED ? ld : 1) * kEs;
        first = held(reinterpret_cast<uint64_t>(a) + o);
        second = held(reinterpret_cast<uint64_t>(b) + o);
        half = held(static_cast<uint64_t>(R) * (RED ? ld : 1) * kEs);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int left = count - at - h * R;
            uint32_t n = 0;
            if (left > 0) n = static_cast<uint32_t>(RED ? (min(R, left) - 1) * static_cast<long long>(ld) + red : (left + kEpu - 1) / kEpu * kEpu) * kEs;
            size[h] = held(n);
        }
    }
    // To step kt of the phase that `two` names; any: there is such a step.
    __device__ __forceinline__ void go(int kt, bool two, int red, int red_rows, bool any) {
        soff = RED ? kt * 128 : 0;
        units = RED ? (red - kt * kStep + kEpu - 1) / kEpu : 8;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint64_t p = (two ? second : first) + (h ? half : 0);
            uint32_t n = size[h];
            if constexpr (!RED) {
                p += static_cast<uint64_t>(kt) * (static_cast<uint64_t>(kStep * kEs) * ld);
                if (n != 0) n += (min(kStep, red_rows - kt * kStep) - 1) * ld * kEs;
            }
            rs[h] = u32x4_t{static_cast<uint32_t>(p), static_cast<uint32_t>(p >> 32) & 0xFFFFu, any ? n : 0, 0x00020000u};
        }
    }
    // To the next step, where both are whole steps of one phase.
    __device__ __forceinline__ void next() {
        if constexpr (RED) {
            soff += 128;
            units -= 8;
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint64_t p = (static_cast<uint64_t>(rs[h][1]) << 32 | rs[h][0]) + static_cast<uint64_t>(kStep * kEs) * ld;
                rs[h][0] = static_cast<uint32_t>(p);
                rs[h][1] = static_cast<uint32_t>(p >> 32);
            }
        }
    }
};

// ---- the sums ------------------------------------------------------------------------------------
// A wave's tile: TI x TJ blocks of 16 x 16 in each half of rows and of columns, and how its sums
// become rows.  Lane (l16, g4) holds row l16 of a block and four columns; 16 rows at a time go
// through LDS (turn: 16 rows of 64 floats, unit u of row r at u ^ r), so that a lane holds eight
// adjacent columns of a row: the wave's columns of the left half, then of the right (pairs: the
// two projections).
template <typename T, int BM, int BN, int WM, int WN, int KIND>
struct Rows {
    static constexpr int TI = BM / 2 / WM / 16, TJ = BN / 2 / WN / 16, kWide = TJ * 16;
    static constexpr bool PAIRS = KIND == kProjGated;
    static constexpr int kTurn = 16 * 64 * 4;                        // bytes a wave
    static constexpr int kUnits = (PAIRS ? 1 : 2) * kWide / 8, kRows = 64 / kUnits, kPass = 16 / kRows;
    static constexpr int kCols = PAIRS ? BN / 2 : BN;                // columns of C of a tile
    static_assert(TJ == 2, "64 columns a wave");

    Columns<T, KIND> cols;
    int n, lane, wm;
    float* turn;

    __device__ __forceinline__ void init(const ProjEpi& e, const ProjGroup& g, int n0, int wave, int lane_, char* smem) {
        lane = lane_;
        wm = wave / WN;
        turn = reinterpret_cast<float*>(smem + wave * kTurn);
        const int u = lane % kUnits;
        n = n0 + u / (kWide / 8) * (BN / 2) + wave % WN * kWide + u % (kWide / 8) * 8;
        cols.load(e, n, g.N - n);
    }
    // A row block's sums to the turning place.
    __device__ __forceinline__ void write(const f32x4_t (&acc)[2][TJ]) const {
        const int l16 = lane & 15, g4 = lane >> 4;
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int j = 0; j < TJ; ++j)
                *reinterpret_cast<f32x4_t*>(turn + l16 * 64 + ((8 * y + 4 * j + g4) ^ l16) * 4) = acc[y][j];
    }
    // The lane's rows of block i of half x.
    __device__ __forceinline__ void rows(int m0, int x, int i, int (&m)[kPass]) const {
#pragma unroll
        for (int q = 0; q < kPass; ++q) m[q] = m0 + x * (BM / 2) + (wm * TI + i) * 16 + q * kRows + lane / kUnits;
    }
    // What follows for the written block i of half x.
    __device__ __forceinline__ void put(const ProjEpi& e, const ProjGroup& g, int m0, int x, int i,
                                        const Reads<T, KIND, kPass>& reads) const {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        float v[kPass][8], w[kPass][8];
        int m[kPass];
        rows(m0, x, i, m);
#pragma unroll
        for (int q = 0; q < kPass; ++q) {
            const int row = q * kRows + lane / kUnits, u = lane % kUnits * 2;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const f32x4_t a = *reinterpret_cast<const f32x4_t*>(turn + row * 64 + ((u + k) ^ row) * 4);
                f32x4_t b{};
                if (PAIRS) b = *reinterpret_cast<const f32x4_t*>(turn + row * 64 + ((u + k + 8) ^ row) * 4);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    v[q][4 * k + r] = a[r];
                    w[q][4 * k + r] = b[r];
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        if (n < g.N) finish<T, KIND, kPass>(e, g, cols, reads, m, n, v, w);
    }
};

// ---- the product ----------------------------------------------------------------------------------
// A launch's work: tiles, those of the last, partial round cut more finely along the reduction than
// the others.  Workgroups (items) are numbered tile by tile within a part of the reduction, so that
// those that run together walk the same columns of the operands.
struct Item {
    int tile, split, s0, s1;       // steps [s0, s1) of a tile
    bool whole;
};
__device__ __forceinline__ Item item_of(const ProjArgs& p, int id) {
    // XCD-aware order: launch ids rotate over the 8 XCDs; each XCD gets a contiguous range of a
    // region's items, whose tiles are walked in bands of rows so that those in flight share both
    // operands in its L2
    const int first = p.tiles1 * p.splits1;
    const bool late = id >= first;
    const int base = late ? first : 0, tiles = late ? p.tiles - p.tiles1 : p.tiles1, splits = late ? p.splits2 : p.splits1;
    const int total = tiles * splits;
    int k = id - base;
    const int x = k & 7, q = total >> 3, r = total & 7;
    k = x * q + min(x, r) + (k >> 3);
    Item it;
    it.split = k / tiles;
    it.tile = k % tiles + (late ? p.tiles1 : 0);
    it.s0 = p.steps * it.split / splits;         // (2^24 steps, 32 splits at most)
    it.s1 = p.steps * (it.split + 1) / splits;
    it.whole = splits == 1;
    return it;
}
// Where the part of a tile's sums is kept that split j leaves.
__device__ __forceinline__ size_t part_of(const ProjArgs& p, int tile, int j) {
    if (tile < p.tiles1) return static_cast<size_t>(j) * p.tiles1 + tile;
    return static_cast<size_t>(p.splits1 > 1 ? p.splits1 : 0) * p.tiles1 + static_cast<size_t>(j) * (p.tiles - p.tiles1) + (tile - p.tiles1);
}
// A tile's place: its product, first row and column.
struct Place {
    int gi, m0, n0;
};
template <int BM, int COLS>
__device__ __forceinline__ Place place_of(const ProjArgs& p, int t) {
    Place at;
    at.gi = 0;
    if (p.ngroups > 1 && t >= p.g[0].end) at.gi = p.ngroups > 2 && t >= p.g[1].end ? 2 : 1;
    const ProjGroup& g = p.g[at.gi];
    if (at.gi > 0) t -= p.g[at.gi - 1].end;
    const int tiles_m = (g.M + BM - 1) / BM, per = p.band * g.tiles_n, b = t / per, rem = t % per;
    const int rows = min(p.band, tiles_m - b * p.band);
    at.m0 = (b * p.band + rem % rows) * BM;
    at.n0 = rem / rows * COLS;
    return at;
}

template <typename T, bool AR, bool BR, int BM, int BN, int WM, int WN, int STAGES, int KIND>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2, 2))) void proj_kernel(const ProjArgs p) {
    typedef Rows<T, BM, BN, WM, WN, KIND> Out;
    constexpr int NW = WM * WN, TI = Out::TI, TJ = Out::TJ;       // blocks of a wave in a half
    static_assert(TI == 2 || TI == 4, "a wave's tile is up to 128 x 64");
    constexpr bool PAIRS = Out::PAIRS;               // B's halves: the two projections
    typedef Half<T, AR, BM / 2, NW> A;
    typedef Half<T, BR, BN / 2, NW> B;
    // LDS of a stage: A's upper and lower, B's left and right half
    constexpr int kStage = 2 * (A::kBytes + B::kBytes), kAb = A::kBytes, kBl = 2 * A::kBytes, kBr = kBl + B::kBytes;
    constexpr int kEs = sizeof(T), kStep = 128 / kEs;
    constexpr int kCA = A::kCopies, kCB = B::kCopies, kPair = kCA + kCB;
    constexpr int kWait = (2 * STAGES - 2) * kPair;  // copies younger than those that a barrier waits for
    static_assert(kWait < 64, "the counter's range");
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;

    const Item it = item_of(p, blockIdx.x);
    const Place at = place_of<BM, Out::kCols>(p, it.tile);
    const ProjGroup& g = p.g[at.gi];
    const int s0 = it.s0, s1 = it.s1;
    const int red = held(p.red), red_rows = held(p.red_rows), nk1 = (red + kStep - 1) / kStep;
    const uint32_t lds0 = lds_addr_of(smem);

    A sa;
    B sb;
    Operand<T, AR, BM / 2> oa;
    Operand<T, BR, BN / 2> ob;       // pairs: the halves are the two projections, at the same columns
    // Sources of step kt.  Steps follow each other by `next` except at the ends of a phase and of
    // the tile's steps: `turn_at` is the next such step.
    int turn_at = 0;
    auto source = [&](int kt) {
        if (kt != turn_at) {
            oa.next();
            ob.next();
            return;
        }
        const bool two = kt >= nk1;
        const int k = two ? kt - nk1 : kt;
        oa.go(k, two, red, red_rows, kt < s1);
        ob.go(k, two && !PAIRS, red, red_rows, kt < s1);
        turn_at = kt >= s1 ? kt + 1 : min(s1, k >= nk1 - 1 ? kt + 1 : kt + (nk1 - 1 - k));
    };
    auto copy = [&](const auto& side, const auto& from, bool by_red, int h, int i, uint32_t at) {
        const uint32_t o = by_red && side.unit >= from.units ? kOutside : side.off[i];
        buf2lds16(from.rs[h], o, from.soff, at + (wave + NW * i) * 1024);
    };
    // copy i of half h of A, of B, into the stage at `st`
    auto copy_a = [&](int h, int i, uint32_t st) { copy(sa, oa, AR, h, i, st + h * kAb); };
    auto copy_b = [&](int h, int i, uint32_t st) { copy(sb, ob, BR, h, i, st + (h ? kBr : kBl)); };
    sa.init(wave, lane, wm * TI, g.lda);
    sb.init(wave, lane, wn * TJ, g.ldb);
    oa.init(g.a, p.phases > 1 ? g.a2 : g.a, g.lda, at.m0, g.M, red);
    ob.init(g.b, PAIRS || p.phases > 1 ? g.b2 : g.b, g.ldb, at.n0, g.bn, red);
    if (PAIRS) {
        ob.half = held(ob.second - ob.first);
        ob.size[1] = ob.size[0];
    }

    f32x4_t acc[2][TI][2][TJ];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int j = 0; j < TJ; ++j) acc[x][i][y][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    {
        turn_at = s0;
#pragma unroll
        for (int k = 0; k < STAGES; ++k) {
            source(s0 + k);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < kCA; ++i) copy_a(h, i, lds0 + k * kStage);
#pragma unroll
                for (int i = 0; i < kCB; ++i) copy_b(h, i, lds0 + k * kStage);
            }
        }
        source(s0 + STAGES);
        wait_vmcnt<kWait>();
        lds_barrier();
        u16x8_t fa[2][TI][2], fb[2][TJ][2];          // A: upper, lower; B: by turns left and right
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
            for (int i = 0; i < TI; ++i) fa[0][i][ks] = sa.read(lds0, i, ks);
#pragma unroll
            for (int j = 0; j < TJ; ++j) fb[0][j][ks] = sb.read(lds0 + kBl, j, ks);
        }
        lds_barrier();
        uint32_t cur = lds0, oth = lds0 + kStage;
        // A quarter: its products, between them the reads of the half that comes in (from `in`:
        // A's lower (1) or upper (0) half, or B's right (1) or left (0)) and copies.
        auto quarter = [&](auto x, auto y, auto bx, auto read_a, auto half_in, uint32_t in, auto&& copies) {
            constexpr int X = x(), Y = y(), BX = bx(), RA = read_a(), H = half_in();
            constexpr int kReads = RA ? 2 * TI : 2 * TJ;
            // Two row blocks at a time: a sum's next product comes four instructions after its last.
            // One read or copy goes out behind each product, while the matrix cores work on it.
            // The copies are spread over the rest of the quarter, as the memory pipe takes 64 bytes a clock.
            constexpr int kMul = 2 * TI * TJ, kApart = (kMul - kReads) / (kCA > kCB ? kCA : kCB);
#pragma unroll
            for (int n = 0; n < kMul; ++n) {
                const int j = n % TJ, e = n / TJ % 2, ks = n / (2 * TJ) % 2, i = n / (4 * TJ) * 2 + e;
                acc[X][i][Y][j] = frag_mul<T>(fb[BX][j][ks], fa[X][i][ks], acc[X][i][Y][j]);
                if (n < kReads) {
                    if constexpr (RA)
                        fa[H][n >> 1][n & 1] = sa.read(in, n >> 1, n & 1);
                    else
                        fb[H][n >> 1][n & 1] = sb.read(in, n >> 1, n & 1);
                } else if ((n - kReads) % kApart == 0) {
                    copies((n - kReads) / kApart);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        constexpr std::integral_constant<int, 0> c0{};
        constexpr std::integral_constant<int, 1> c1{};
        // A step whose left half of B is in fb[P]; the next step's comes into the other.
        auto step = [&](int kt, auto par) {
            constexpr int P = par();
            constexpr std::integral_constant<int, P> l{};
            constexpr std::integral_constant<int, P ^ 1> r{};
            quarter(c0, c0, l, c0, r, cur + kBr, [&](int i) {
                if (i < kCA) copy_a(0, i, cur);
            });
            quarter(c0, c1, r, c1, c1, cur + kAb, [&](int i) {
                if (i < kCB) copy_b(0, i, cur);
            });
            wait_vmcnt<kWait>();   // the next step's upper and left halves have landed for this wave,
            lds_barrier();             // and for all; all have read this step's lower and right ones
            quarter(c1, c1, r, c1, c0, oth, [&](int i) {
                if (i < kCA) copy_a(1, i, cur);
            });
            quarter(c1, c0, l, c0, r, oth + kBl, [&](int i) {
                if (i < kCB) copy_b(1, i, cur);
            });
            source(kt + STAGES + 1);
            wait_vmcnt<kWait>();   // likewise, the other halves
            lds_barrier();
            cur = oth;
            oth = oth + kStage == lds0 + STAGES * kStage ? lds0 : oth + kStage;
        };
        int kt = s0;
        for (; kt + 1 < s1; kt += 2) {
            step(kt, c0);
            step(kt + 1, c1);
        }
        if (kt < s1) step(kt, c0);
        wait_vmcnt<0>();               // (the empty copies past the end,
        lds_barrier();                 // for all waves, before their places are filled again)

    }
    if (it.whole) {
        Out out;
        out.init(p.e, g, at.n0, wave, lane, smem);
        // (a loop, as what follows the sums is long: eight copies of it are more than the
        // instruction cache holds: 120 us instead of 95 at 8192 x 4096 x 1024 with gelu)
        // All that the blocks read besides the sums is loaded in front of the first store (gate and up in
        // fp32 are too much to hold, and are loaded block by block).
        typedef Reads<T, KIND, Out::kPass> In;
        constexpr bool kAhead = In::N > 0 && In::N * 4 * TI * Out::kPass * static_cast<int>(sizeof(T)) <= 64;   // registers
        In all[kAhead ? 2 * TI : 1], reads;
        if constexpr (kAhead) {
#pragma unroll
            for (int k = 0; k < 2 * TI; ++k) {
                int m[Out::kPass];
                out.rows(at.m0, k / TI, k % TI, m);
                all[k].load(p.e, g, m, out.n);
            }
#pragma unroll
            for (int k = 0; k < 2 * TI; ++k) all[k].wait(p.e);
        }
#pragma unroll 1
        for (int b = 0; b < 2 * TI; ++b) {
            const int now = held(b);
            if constexpr (kAhead) {
#pragma unroll
                for (int k = 0; k < 2 * TI; ++k)
                    if (now == k) reads = all[k];
            } else {
                int m[Out::kPass];
                out.rows(at.m0, now / TI, now % TI, m);
                reads.load(p.e, g, m, out.n);
            }
#pragma unroll
            for (int k = 0; k < 2 * TI; ++k)
                if (now == k) out.write(acc[k / TI][k % TI]);
            out.put(p.e, g, at.m0, now / TI, now % TI, reads);
        }
    } else {
        // a part of a tile's sums, as the lanes hold them
        f32x4_t* o = reinterpret_cast<f32x4_t*>(p.part) + (part_of(p, it.tile, it.split) * NW + wave) * (4 * TI * TJ) * 64 + lane;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int i = 0; i < TI; ++i)
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int j = 0; j < TJ; ++j) o[(((x * TI + i) * 2 + y) * TJ + j) * 64] = acc[x][i][y][j];
    }
}

// The sums of tiles whose reduction is cut, added in the order of the cuts.  A workgroup per tile
// and 16-row block of its waves.
template <typename T, int BM, int BN, int WM, int WN, int KIND>
__global__ __launch_bounds__(64 * WM * WN) void proj_join_kernel(const ProjArgs p) {
    typedef Rows<T, BM, BN, WM, WN, KIND> Out;
    constexpr int NW = WM * WN, TI = Out::TI, TJ = Out::TJ;
    __shared__ __attribute__((aligned(1024))) char smem[NW * Out::kTurn];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = blockIdx.x + (p.splits1 > 1 ? 0 : p.tiles1), xi = blockIdx.y;
    const int splits = t < p.tiles1 ? p.splits1 : p.splits2;
    if (splits == 1) return;
    const Place at = place_of<BM, Out::kCols>(p, t);
    const ProjGroup& g = p.g[at.gi];
    Out out;
    out.init(p.e, g, at.n0, wave, lane, smem);
    Reads<T, KIND, Out::kPass> reads;
    int m[Out::kPass];
    out.rows(at.m0, xi / TI, xi % TI, m);
    reads.load(p.e, g, m, out.n);
    f32x4_t acc[2][TJ];
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[y][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int j = 0; j < splits; ++j) {
        const f32x4_t* o = reinterpret_cast<const f32x4_t*>(p.part) + (part_of(p, t, j) * NW + wave) * (4 * TI * TJ) * 64 + lane;
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int k = 0; k < TJ; ++k) acc[y][k] += o[((xi * 2 + y) * TJ + k) * 64];
    }
    out.write(acc);
    out.put(p.e, g, at.m0, xi / TI, xi % TI, reads);
}

// Products over nothing (no rows in a gradient of weights): zeros.
template <typename T>
__global__ __launch_bounds__(256) void proj_zero_kernel(const ProjArgs p) {
    const ProjGroup& g = p.g[blockIdx.y];
    const size_t total = static_cast<size_t>(g.M) * g.N;
    for (size_t e = blockIdx.x * static_cast<size_t>(256) + threadIdx.x; e < total; e += static_cast<size_t>(gridDim.x) * 256)
        static_cast<T*>(g.c)[e / g.N * g.ldc + e % g.N] = T(0);
}

// ---- plan ---------------------------------------------------------------------------------------
// Tiles, by the rate of the main loop: 256 x 256 reach 1.35 PFLOP/s, 256 x 128 1.08, 128 x 128 1.15
// with two workgroups a CU and 0.8 with one; fp32 a tenth of that for any.  The last is for few
// workgroups with few steps, whose time is the copies' way from memory: four stages, one workgroup a CU.
struct Tile {
    int bm, bn, slots;     // workgroups of the chip at a time
    double rate;           // PFLOP/s of the main loop
    double tail;           // microseconds of a workgroup that do not overlap with others: first copies, last stores
    double least;          // microseconds of a step at least: a copy's way through the stages
};
constexpr Tile kTiles[4] = {{256, 256, 256, 1.35, 9.0, 1.2}, {256, 128, 256, 1.08, 6.0, 0.7}, {128, 128, 512, 1.15, 5.0, 0.9},
                            {128, 128, 256, 0.8, 5.0, 0.5}};
constexpr double kRateF32 = 0.135;

// A tile's number and how tiles are cut: all into splits1 parts of the reduction; the whole rounds of
// workgroups that this makes (tiles1 tiles) are taken as they are, the rest of the tiles are cut into
// splits2 parts, as many as fill the chip once.
struct Cut {
    int tile, tiles1, splits1, splits2;
};
Cut best_cut(const ProjArgs& a, ProjKind kind, bool bf16) {
    const int step = bf16 ? 64 : 32;
    Cut best{2, 0, 1, 1};
    double best_t = 1e30;
    for (int c = 0; c < 4; ++c) {
        // (fp32, and gate and up of a gradient, take more registers than the largest tile leaves)
        if (c == 0 && (!bf16 || kind == kProjGatedBwd)) continue;
        const Tile& t = kTiles[c];
        const int cols = kind == kProjGated ? t.bn / 2 : t.bn;
        long long tiles = 0;
        for (int i = 0; i < a.ngroups; ++i)
            tiles += static_cast<long long>((a.g[i].M + t.bm - 1) / t.bm) * ((a.g[i].N + cols - 1) / cols);
        // microseconds of so many steps with so many workgroups, of which a CU may hold two
        auto time = [&](long long groups, int steps) {
            const long long here = (std::min<long long>(groups, t.slots) + 255) / 256;   // workgroups of a CU
            const double rate = !bf16 ? kRateF32 : t.slots > 256 && here == 1 ? 0.8 : t.rate;
            return steps * std::max(t.least, 2.0 * t.bm * t.bn * step * 256 * here / (rate * 1e9)) + t.tail;
        };
        for (int s1 = 1; s1 <= 32 && s1 <= std::max(a.steps, 1); ++s1) {
            const long long items = tiles * s1;
            if (s1 > 1 && items > 4 * t.slots) break;
            const int per1 = (a.steps + s1 - 1) / s1;
            for (int cut = 0; cut < 2; ++cut) {
                // the last round: as it comes, or cut
                long long t1 = tiles, t2 = 0;
                int s2 = 1;
                double us = static_cast<double>((items + t.slots - 1) / t.slots) * time(items, per1);
                if (cut) {
                    t1 = items / t.slots * t.slots / s1;
                    t2 = tiles - t1;
                    if (t2 == 0) continue;
                    s2 = static_cast<int>(std::min<long long>(std::min(a.steps, 32), t.slots / t2));
                    if (s2 <= s1) continue;
                    us = static_cast<double>(items / t.slots) * time(items, per1) + time(t2 * s2, (a.steps + s2 - 1) / s2);
                }
                const double parts = (s1 > 1 ? static_cast<double>(t1) * s1 : 0) + (s2 > 1 ? static_cast<double>(t2) * s2 : 0);
                if (parts > 0) us += 4.0 + parts * t.bm * t.bn * 8 / 6e6;   // stored and read again, mostly from the caches
                if (us < best_t) {
                    best_t = us;
                    best = Cut{c, static_cast<int>(t1), s1, s2};
                }
            }
        }
    }
    return best;
}

// Sets tiles and cuts; returns the tile's number.  The choice is a function of the sizes alone and takes
// several microseconds, so a thread keeps those of the sizes that it used last.
int plan(ProjArgs& a, ProjKind kind, bool bf16) {
    a.steps = (a.red + (bf16 ? 64 : 32) - 1) / (bf16 ? 64 : 32) * a.phases;
    struct Entry {
        int key[9];
        Cut cut;
    };
    static thread_local Entry kept[64];
    int key[9] = {1 + kind + 4 * (bf16 ? 1 : 0) + 8 * a.ngroups, a.steps};
    unsigned at = 0;
    for (int i = 0; i < a.ngroups; ++i) {
        key[2 + 2 * i] = a.g[i].M;
        key[3 + 2 * i] = a.g[i].N;
    }
    for (int k : key) at = at * 31u + static_cast<unsigned>(k);
    Entry& e = kept[(at ^ (at >> 15)) % 64];
    if (!std::equal(key, key + 9, e.key)) {
        e.cut = best_cut(a, kind, bf16);
        std::copy(key, key + 9, e.key);
    }
    a.tiles1 = e.cut.tiles1;
    a.splits1 = e.cut.splits1;
    a.splits2 = e.cut.splits2;
    const Tile& t = kTiles[e.cut.tile];
    a.band = 8;
    int tiles = 0;
    for (int i = 0; i < a.ngroups; ++i) {
        ProjGroup& g = a.g[i];
        const int cols = kind == kProjGated ? t.bn / 2 : t.bn;
        g.tiles_n = (g.N + cols - 1) / cols;
        tiles += (g.M + t.bm - 1) / t.bm * g.tiles_n;
        g.end = tiles;
    }
    a.tiles = tiles;
    return e.cut.tile;
}
// Parts of sums that cut tiles leave.
size_t parts_of(const ProjArgs& a) {
    const size_t t1 = a.tiles1, t2 = a.tiles - a.tiles1;
    return (a.splits1 > 1 ? t1 * a.splits1 : 0) + (a.splits2 > 1 ? t2 * a.splits2 : 0);
}

template <typename T, bool AR, bool BR, int BM, int BN, int WM, int WN, int STAGES, int KIND>
hipError_t launch_tile(const ProjArgs& a, hipStream_t st) {
    constexpr int lds = STAGES * (BM + BN) * 128;
    static_assert(lds >= WM * WN * Rows<T, BM, BN, WM, WN, KIND>::kTurn, "turning places");
    const int items = a.tiles1 * a.splits1 + (a.tiles - a.tiles1) * a.splits2;
    // the LDS limit belongs to a device's function: set once on each, whichever thread comes first
    constexpr int kDevices = 64;
    static std::once_flag attr_once[kDevices];
    int dev = 0;
    hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess) return err;
    if (dev < 0 || dev >= kDevices) return hipErrorInvalidDevice;
    std::call_once(attr_once[dev], [] {
        (void)hipFuncSetAttribute(reinterpret_cast<const void*>(&proj_kernel<T, AR, BR, BM, BN, WM, WN, STAGES, KIND>),
                                  hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    });
    {
        ProfScope prof(kProfProj, st);
        hipLaunchKernelGGL((proj_kernel<T, AR, BR, BM, BN, WM, WN, STAGES, KIND>), dim3(items), dim3(64 * WM * WN), lds, st, a);
    }
    err = hipGetLastError();
    if (err != hipSuccess || parts_of(a) == 0) return err;
    ProfScope prof(kProfProjJoin, st);
    hipLaunchKernelGGL((proj_join_kernel<T, BM, BN, WM, WN, KIND>), dim3(a.splits1 > 1 ? a.tiles : a.tiles - a.tiles1, BM / WM / 16),
                       dim3(64 * WM * WN), 0, st, a);
    return hipGetLastError();
}

template <typename T, bool AR, bool BR, int KIND>
hipError_t launch_sized(const ProjArgs& a, int tile, hipStream_t st) {
    if constexpr (sizeof(T) == 2 && KIND != kProjGatedBwd) {
        if (tile == 0) return launch_tile<T, AR, BR, 256, 256, 2, 4, 2, KIND>(a, st);
    }
    if (tile == 1) return launch_tile<T, AR, BR, 256, 128, 4, 2, 3, KIND>(a, st);
    if (tile == 2) return launch_tile<T, AR, BR, 128, 128, 2, 2, 2, KIND>(a, st);
    return launch_tile<T, AR, BR, 128, 128, 2, 2, 4, KIND>(a, st);
}

template <typename T>
hipError_t launch_typed(const ProjArgs& a, int tile, ProjKind kind, bool a_red, bool b_red, hipStream_t st) {
    if (a.steps == 0) {
        size_t most = 0;
        for (int i = 0; i < a.ngroups; ++i) most = std::max(most, static_cast<size_t>(a.g[i].M) * a.g[i].N);
        ProfScope prof(kProfProjPass, st);
        const unsigned blocks = static_cast<unsigned>(std::min<size_t>((most + 255) / 256, 1u << 14));
        hipLaunchKernelGGL((proj_zero_kernel<T>), dim3(blocks, a.ngroups), dim3(256), 0, st, a);
        return hipGetLastError();
    }
    if (kind == kProjGated) return launch_sized<T, true, true, kProjGated>(a, tile, st);
    if (kind == kProjGatedBwd) return launch_sized<T, true, false, kProjGatedBwd>(a, tile, st);
    if (a_red) return b_red ? launch_sized<T, true, true, kProjLinear>(a, tile, st) : launch_sized<T, true, false, kProjLinear>(a, tile, st);
    return launch_sized<T, false, false, kProjLinear>(a, tile, st);
}

// ---- packing and slopes ------------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(256) void pack_kernel(PackArgs a) {
    constexpr int V = kPack<T>;
    const PackArgs::One& o = a.one[blockIdx.y];
    const int units = static_cast<int>(o.ldd / V);
    const size_t total = o.rows * units;
    for (size_t e = blockIdx.x * static_cast<size_t>(256) + threadIdx.x; e < total; e += static_cast<size_t>(gridDim.x) * 256) {
        const size_t r = e / units;
        const int n = static_cast<int>(e % units) * V;
        raw_store<T, V>(static_cast<T*>(o.dst) + r * o.ldd + n, raw_load_n<T, V>(static_cast<const T*>(o.src) + r * o.lds + n, o.width - n));
    }
}

// Lanes of a wave lie over units of eight columns, lpr of them a row; a workgroup takes a
// strip of 8 lpr columns and a chunk of rows, and leaves one row of partial sums.  In bf16 gz is rounded to bf16, which
// is what the products take (gradients behind an activation: 2.3e-3 off instead of 1.7e-3, relative to 64 bits); the
// column sums are of the values before that.
struct SlopePlan {
    int lpr, strips, chunks;
    size_t per;
};
SlopePlan slope_plan(size_t rows, int N) {
    SlopePlan s;
    s.lpr = 1;
    while (s.lpr < 64 && s.lpr * 8 < N) s.lpr *= 2;
    s.strips = (N + 8 * s.lpr - 1) / (8 * s.lpr);
    const size_t at_once = 4 * (64 / s.lpr);                         // rows of a workgroup's trip
    const size_t trips = (rows + at_once - 1) / at_once;
    // about 2048 workgroups, eight trips at least each
    size_t want = 2048 / s.strips;
    if (want < 1) want = 1;
    if (want > 512) want = 512;
    size_t per = (trips + want - 1) / want;
    if (per < 8) per = 8;
    s.per = per * at_once;
    s.chunks = static_cast<int>((rows + s.per - 1) / s.per);
    if (s.chunks < 1) s.chunks = 1;
    return s;
}

template <typename T>
__global__ __launch_bounds__(256) void slope_kernel(SlopeArgs a, int lpr, size_t per) {
    __shared__ float sums[256][9];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, rpw = 64 / lpr;
    const int n = (blockIdx.x * lpr + lane % lpr) * 8, left = a.N - n;
    const size_t r0 = blockIdx.y * per, r1 = min(r0 + per, a.rows);
    float s[8] = {};
    const bool pad = a.gz != nullptr && n < a.ldz;                   // columns of gz, zeros among them
    if (left > 0 || pad) {
        for (size_t r = r0 + wave * rpw + lane / lpr; r < r1; r += 4 * rpw) {
            float g[8] = {};
            if (left > 0) load8<T>(static_cast<const T*>(a.gy) + r * a.N + n, left, g);
            if (a.pre != nullptr) {
                float z[8] = {};
                if (left > 0) load8<T>(static_cast<const T*>(a.pre) + r * a.N + n, left, z);
                float v[8];
                act_slopes(z, v, a.act);
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = i < left ? g[i] * z[i] : 0.f;
            }
            if (pad) store8<T>(static_cast<T*>(a.gz) + r * a.ldz + n, g, static_cast<int>(a.ldz) - n);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] += g[i];
        }
    }
    if (a.part == nullptr) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[threadIdx.x][i] = s[i];
    __syncthreads();
    if (threadIdx.x >= lpr) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float t = 0.f;
        for (int k = threadIdx.x; k < 256; k += lpr) t += sums[k][i];
        if (i < left) a.part[static_cast<size_t>(blockIdx.y) * a.N + n + i] = t;
    }
}

}  // namespace

size_t proj_partial_bytes(const ProjArgs& args, ProjKind kind, bool bf16) {
    ProjArgs a = args;
    const Tile& t = kTiles[plan(a, kind, bf16)];
    return a.steps == 0 ? 0 : parts_of(a) * t.bm * t.bn * sizeof(float);
}

hipError_t launch_proj(ProjArgs a, ProjKind kind, bool bf16, bool a_red, bool b_red, hipStream_t st) {
    const int tile = plan(a, kind, bf16);
    if (a.tiles == 0) return hipSuccess;
    return bf16 ? launch_typed<bf16_t>(a, tile, kind, a_red, b_red, st) : launch_typed<float>(a, tile, kind, a_red, b_red, st);
}

hipError_t launch_proj_pack(const PackArgs& a, bool bf16, hipStream_t st) {
    size_t most = 0;
    for (int i = 0; i < a.n; ++i) most = std::max(most, a.one[i].rows * static_cast<size_t>(a.one[i].ldd / (bf16 ? 8 : 4)));
    if (most == 0) return hipSuccess;
    const dim3 grid(static_cast<unsigned>(std::min<size_t>((most + 255) / 256, 1u << 14)), a.n);
    ProfScope prof(kProfProjPass, st);
    if (bf16)
        hipLaunchKernelGGL((pack_kernel<bf16_t>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((pack_kernel<float>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

size_t slope_partial_bytes(size_t rows, int N) {
    return static_cast<size_t>(slope_plan(rows, N).chunks) * N * sizeof(float);
}

hipError_t launch_slope(const SlopeArgs& a, hipStream_t st) {
    const SlopePlan s = slope_plan(a.rows, a.N);
    {
        ProfScope prof(kProfProjPass, st);
        const dim3 grid(s.strips, s.chunks);
        if (a.bf16)
            hipLaunchKernelGGL((slope_kernel<bf16_t>), grid, dim3(256), 0, st, a, s.lpr, s.per);
        else
            hipLaunchKernelGGL((slope_kernel<float>), grid, dim3(256), 0, st, a, s.lpr, s.per);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || a.part == nullptr) return e;
    }
    ColReduceArgs c{};
    c.in = a.part;
    c.P = s.chunks;
    c.rows = 1;
    c.K = 1;
    c.D = a.N;
    c.out0 = a.sums;
    c.out_bf16 = a.bf16 && !a.sums_f32;
    return launch_col_reduce(c, st);
}

}  // namespace retn
