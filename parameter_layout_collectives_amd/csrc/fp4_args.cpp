// Host side of the 4-bit block operators: argument checks and the choice of a
// product's kernel.  Makes no HIP call.
#include <algorithm>

#include "checks.h"
#include "fp4.h"

namespace tide {
namespace {

uint32_t known_flags(Fp4Op op) {
    return TIDE_F_OUT_BF16 |
           (op == kFp4Linear ? TIDE_F_QUANT_X | TIDE_F_GRAD_F16 | TIDE_F_GRAD_F32 : 0u);
}

constexpr int64_t kRound = 255;
int64_t rounded(int64_t n) { return (n + kRound) & ~kRound; }

// Flags and sizes; as in the 8-bit products, a launch counts its lanes in 32 bits.
tide_status check_product(const char *name, Fp4Op op, int64_t M, int64_t N, int64_t K,
                          uint32_t flags) {
    tide_status st = check_flags(name, flags, known_flags(op));
    if (st != TIDE_OK) return st;
    if ((flags & (TIDE_F_GRAD_F16 | TIDE_F_GRAD_F32)) && !(flags & TIDE_F_QUANT_X))
        return bad(name, "an x in fp16 or fp32 without TIDE_F_QUANT_X");
    for (int64_t rows : {M, N})
        for (int64_t cols : {N, K})
            if ((st = check_dims(name, rows, cols)) != TIDE_OK) return st;
    if (N > kMaxLine || K > kMaxLine)
        return fail(TIDE_E_UNSUPPORTED, std::string(name) + ": n or k above 2^22");
    const int64_t cols = op == kFp4Dx ? K : N;
    for (bool aligned : {false, true}) {
        const Fp4Choice c = fp4_choose(op, M, N, K, flags, aligned, INT64_MAX);
        if (c.kernel != kFp4Tiles && c.kernel != kFp4Wide) continue;
        const int64_t T = c.mm.tile, tiles = ((M + T - 1) / T) * ((cols + T - 1) / T);
        const int64_t cut = (tiles - c.mm.direct) * c.mm.splits;
        if (c.mm.direct + cut > 0xffffffffll / (T == 256 ? 512 : 256) ||
            (tiles - c.mm.direct) * (T * T / 1024) > 0xffffffffll / 256 ||
            ((flags & TIDE_F_QUANT_X) && M * block_count(K) > 0xffffffffll / 4 - 64))
            return fail(TIDE_E_UNSUPPORTED, std::string(name) + ": more than 2^32 lanes");
    }
    return TIDE_OK;
}

// The skinny kernel's workgroups, one for 16 rows of W, each read all of x; the
// strips' share it among 128 and cost a second launch, in which the sum's pieces meet.
// So the skinny kernel takes up to 16 rows, of few multiplications or where a compute
// unit has one workgroup and x is small (rows x N x K, us, skinny against strips):
// 1 x 14336 x 4096 10.8 : 13.5, 2 12.6 : 13.5, 4 15.7 : 13.5, 16 21.9 : 13.9;
// 3 x 8192 x 8192 16.1 : 14.8; 1 x 28672 x 8192 34 : 33; 16 x 4096 x 4096 7.9 : 11.1,
// 8 x 4096 x 14336 14.4 : 15.4, 16 19.5 : 15.6.
constexpr int64_t kFewRows = 16;
constexpr int64_t kFewSum = int64_t(1) << 27;
constexpr int64_t kFewX = int64_t(1) << 17;
// The strips take matrices from a size on (x N x K, us, strips against tiles of 64:
// 17 x 256 x 8192 8.3 : 9.1, 64 x 300 x 2000 11.7 : 7.7, 20 x 1000 x 1000 10.2 : 6.9),
// and rows, of bf16 x up to 64 (64 x 4096 x 4096 13.8 : 16.2, 64 x 8192 x 8192 19.7 :
// 28); against the 4-bit tiles, whose operand x lies ready, larger matrices and up to 32
// (32 x 4096 x 4096 13.1 : 12.2, 17 x 14336 x 4096 16.8 : 19.3, 64 x 4096 x 4096 16 : 13.4).
constexpr int64_t kStripMost = 64, kStripMost4 = 32;
constexpr int64_t kStripLeast = int64_t(1) << 21, kStripLeast4 = int64_t(1) << 25;
// Workgroups that fill the card, one per compute unit (with two, 64 x 28672 x 8192
// takes 52 us for 48, 32 x 8192 x 28672 41 for 40.7), and least units of 128 columns in a
// piece of a sum (40 x 1024 x 4096 8.7 us, with 8 units 11.1).
constexpr int64_t kStripGroups = kCus;
constexpr int64_t kStripUnits = 4;
// Least steps in a piece of a large tile.
constexpr int64_t kDeepSteps = 16;
// Least steps that a cut has to save.
constexpr int64_t kCutSaves = 24;
// An operand is turned if the other has so many rows and both so many columns; an x
// that is quantised here is made so from fewer rows on, as it costs nothing more
// (M x N x K, us, turned / as it lies).  x: 128 x 8192 x 8192 25.8 / 31.7, 512 41 / 50,
// 8192 322 / 386, over 512 columns 10.5 / 10.5; given in blocks 512 x 8192 x 8192 38.7 /
// 44.3, 512 x 4096 x 8192 32.3 / 31.6.  w: 2048 x 8192 x 8192 90.2 / 89.6, 4096 166 /
// 170, 8192 306 / 322.
constexpr int64_t kTurnRows = 4096;
constexpr int64_t kTurnSum = 1024;
constexpr int64_t kTurnMade = 128;
// x is prepared inside the product for so many bytes of bf16 rows.
constexpr int64_t kInOneBytesFp4 = 57344 + 16;

}  // namespace

bool fp4_whole(const void *x, int64_t K) {
    return K % kBlockCols == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
}

Fp4Choice fp4_choose(Fp4Op op, int64_t M, int64_t N, int64_t K, uint32_t flags, bool aligned,
                     int64_t workspace_bytes) {
    Fp4Choice c = {};
    const int64_t cols = op == kFp4Dx ? K : N, sum = op == kFp4Dx ? N : K;
    const bool quant = op == kFp4Linear && (flags & TIDE_F_QUANT_X);
    const int64_t padded = M * block_cols(K) * 2;       // x as bf16 rows of whole units
    const bool few = M <= kFewRows && (M * N * K <= kFewSum || (N <= 16 * kCus && M * K <= kFewX));
    const bool strips = M <= (op == kFp4Mm || quant ? kStripMost4 : kStripMost) &&
                        N * K >= (op == kFp4Mm ? kStripLeast4 : kStripLeast);
    const bool room = op != kFp4Dx && workspace_bytes >= rounded(padded);
    if (op == kFp4Linear && M <= kFewRows && M * (block_cols(K) * 2 + 16) <= kInOneBytesFp4 &&
        (few || !strips || !room)) {
        c.kernel = kFp4SkinnyInOne;
        return c;
    }
    if (room && (few || strips)) {
        c.kernel = few ? kFp4Skinny : kFp4Strips;
        c.x = rounded(padded);
        if (few) return c;
        const int64_t units = std::max<int64_t>(1, block_count(K));
        const int64_t groups = std::max<int64_t>(1, (N + kStripRows - 1) / kStripRows);
        const int64_t pieces = std::max<int64_t>(1, std::min(kStripGroups / groups, units / kStripUnits));
        c.mm.splits = 1;
        c.mm.chunk = units;
        const int64_t chunk = (units + pieces * 4 - 1) / (pieces * 4) * 4, n = (units + chunk - 1) / chunk;
        if (n > 1 && c.x + n * M * N * 4 <= workspace_bytes) {
            c.mm.splits = static_cast<int>(n);
            c.mm.chunk = chunk;
            c.mm.workspace = n * M * N * 4;
        }
        return c;
    }
    c.kernel = op == kFp4Mm || quant ? kFp4Tiles : kFp4Wide;
    if (quant) {
        c.x_scales = rounded(M * kFours.code_bytes(K));
        c.x = rounded(c.x_scales + M * kFours.scale_bytes(K));
    }
    // Operands are turned where a step's loads bound the tiles; an x that is quantised
    // here is made so at once, in place of its blocks.
    c.x_turned = c.w_turned = -1;
    auto turn = [&](int64_t rows, int64_t from, int64_t *at) {
        const int64_t bytes = rounded(rows * block_count(K) * 68);
        if (bytes >= int64_t(1) << 31 || from + bytes > workspace_bytes) return;
        *at = from;
        c.x = from + bytes;
    };
    if (c.kernel == kFp4Tiles && K >= kTurnSum) {
        if (quant ? M >= kTurnMade : N >= kTurnRows) turn(M, quant ? 0 : c.x, &c.x_turned);
        if (M >= kTurnRows) turn(N, c.x, &c.w_turned);
    }
    auto tiles = [&](int64_t t) { return ((M + t - 1) / t) * ((cols + t - 1) / t); };
    const bool four = c.kernel == kFp4Tiles;
    // The 4-bit tiles' step is 128 columns, and two of them cost what cut_sums takes for
    // one.  A cut that leaves no whole set has to save more than its second launch costs,
    // kCutSaves steps, and of the 4-bit tiles, whose steps are short, also its traffic
    // (M x N x K, us, cut / whole): bf16 x 300 x 2048 x 1024 12.5 / 7.8, 500 x 2048 x 2048
    // 18.6 / 13.9, 500 x 2048 x 4096 26.4 / 34, 100 x 512 x 2048 8.1 / 11.4, 200 x 1024 x 2048
    // 12.5 / 11.6, 200 x 1024 x 4096 15.1 / 20.3; 4 bits 200 x 1024 x 4096 15.0 / 12.5, over
    // 8192 20.3 / 19.0, over 16384 23.2 / 29.7, 100 x 512 x 8192 15.2 / 21.5, 500 x 2048 x 16384
    // 40 / 33.
    const int64_t step = four ? 256 : 64, per = four ? 2 : 1;
    auto tiled = [&](int T) {
        MmChoice m = {};
        m.tile = T;
        m.direct = tiles(T);
        m.splits = 1;
        m.chunk = (sum + step - 1) / step;
        MmChoice cut = m;
        cut_sums(cut, m.direct, m.chunk);
        const int64_t least = std::max(kCutSaves, four ? m.direct * 3 / 4 : 0);
        if (cut.direct == 0 && m.chunk - cut.chunk < least) cut = m;
        if (c.x + cut.workspace > workspace_bytes) cut = m;
        cut.chunk *= per;
        return cut;
    };
    // In bf16, large tiles also where they have to be cut to fill the card, if most of
    // each is used and the pieces are long (dX, M x N x K, us, large / middle tiles):
    // 256 x 8192 x 8192 55 / 62, 1024 122 / 154, 2048 x 14336 x 4096 190 / 253, 1024 x 4096 x
    // 4096 50 / 50; pieces of 8 steps, 2048 x 1024 x 4096 33 / 25.  Uncut they leave most of
    // it idle.
    const int64_t large = tiles(256), pieces = std::min(kCus / std::max<int64_t>(large, 1), kMaxSplits);
    if (aligned && !four && pieces >= 2 && large >= kCus / 8 && tiles(128) >= 3 * large &&
        sum >= pieces * kDeepSteps * 64) {
        c.mm = tiled(256);
        if (c.mm.splits > 1) return c;
    }
    c.mm = tiled(aligned && large >= kCus * 3 / 4 ? 256 : tiles(128) < kCus / 2 ? 64 : 128);
    return c;
}

tide_status check_fp4(Fp4Op op, const char *name, const Fp4Args &a) {
    tide_status st = check_product(name, op, a.M, a.N, a.K, a.flags);
    if (st != TIDE_OK) return st;
    if (a.workspace_bytes < 0) return bad(name, "workspace_bytes < 0");
    if (a.workspace_bytes > 0 && !a.workspace) return bad(name, "workspace is NULL");
    if (misaligned(a.workspace, 16)) return bad(name, "workspace is not 16-byte aligned");
    const int64_t ocols = op == kFp4Dx ? a.K : a.N, sum = op == kFp4Dx ? a.N : a.K;
    if (a.M == 0 || ocols == 0) return TIDE_OK;
    const int os = elem_size(out_type(a.flags));
    if (!a.out) return bad(name, "out is NULL");
    if (misaligned(a.out, os)) return bad(name, "out is not aligned to its element size");
    const Bytes out = bytes_of(a.out, a.M * ocols * os);
    const Bytes wsp = bytes_of(a.workspace, a.workspace ? a.workspace_bytes : 0);
    if (overlap(out, wsp)) return bad(name, "out overlaps the workspace");
    if (sum == 0) return TIDE_OK;
    Bytes in[4];
    int n = 0;
    if (op == kFp4Mm) {
        st = check_blocks(name, "x's", a.a, a.a_scales);
        if (st != TIDE_OK) return st;
        in[n++] = bytes_of(a.a, a.M * kFours.code_bytes(a.K));
        in[n++] = bytes_of(a.a_scales, a.M * kFours.scale_bytes(a.K));
    } else {
        const char *what = op == kFp4Dx ? "dy" : "x";
        const int es = elem_size(in_type(a.flags));
        if (!a.a) return bad(name, (std::string(what) + " is NULL").c_str());
        if (misaligned(a.a, es))
            return bad(name, (std::string(what) + " is not aligned to its element size").c_str());
        in[n++] = bytes_of(a.a, a.M * (op == kFp4Dx ? a.N : a.K) * es);
    }
    st = check_blocks(name, "w's", a.b, a.b_scales);
    if (st != TIDE_OK) return st;
    in[n++] = bytes_of(a.b, a.N * kFours.code_bytes(a.K));
    in[n++] = bytes_of(a.b_scales, a.N * kFours.scale_bytes(a.K));
    for (int k = 0; k < n; k++) {
        if (overlap(out, in[k])) return bad(name, "out overlaps an operand");
        if (overlap(wsp, in[k])) return bad(name, "the workspace overlaps an operand");
    }
    return TIDE_OK;
}

}  // namespace tide

using tide::bad;

extern "C" {

int64_t tide_mx_cols(int64_t cols) {
    return cols < 0 || cols >= tide::kMaxDim ? -1 : tide::block_cols(cols);
}

tide_status tide_plan_create_mx(const tide_plan *plan, int32_t n, const int32_t *select,
                                 tide_plan **out_plan) {
    return tide::create_plan("tide_plan_create_mx", tide::kFours, plan, n, select, out_plan);
}

int64_t tide_mx_workspace(int32_t op, int64_t m, int64_t n, int64_t k, uint32_t flags) {
    const char *name = "tide_mx_workspace";
    if (op < 0 || op > 2) {
        bad(name, "op outside [0, 2]");
        return -1;
    }
    const tide::Fp4Op o = static_cast<tide::Fp4Op>(op);
    if (tide::check_product(name, o, m, n, k, flags) != TIDE_OK) return -1;
    if (m == 0 || (o == tide::kFp4Dx ? k : n) == 0 || (o == tide::kFp4Dx ? n : k) == 0) return 0;
    int64_t most = 0;                    // whichever way dY or x is aligned
    for (bool aligned : {false, true}) {
        const tide::Fp4Choice c = tide::fp4_choose(o, m, n, k, flags, aligned, INT64_MAX);
        most = std::max(most, c.x + c.mm.workspace);
    }
    return most;
}

}  // extern "C"
