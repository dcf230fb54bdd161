// Matrices in microscaled 4-bit blocks: the products' choice of kernels
// (fp4_args.cpp, host only) and their launches (fp4_cast.hip, fp4_mm.hip).
//
// A matrix [R, C] is held as codes [R, Cp / 2] (two e2m1 numbers a byte, the even
// column in the low half, Cp = C rounded up to 128) and scales [R, Cp / 32] (e8m0
// bytes): element (r, c) is e2m1(code) * 2^(scales[r, c / 32] - 127).
#pragma once

#include "block.h"

namespace tide {

// out[i, j] = sum over c of I(i, c) * J(c, j), with J = W in 4-bit blocks:
//   kFp4Mm      I = X in 4-bit blocks
//   kFp4Dx      I = dY (bf16), c = row of W
//   kFp4Linear  I = x (bf16, or rounded to 4-bit blocks on the way)
enum Fp4Op { kFp4Mm = 0, kFp4Dx = 1, kFp4Linear = 2 };

struct Fp4Args {
    const void *a, *a_scales;    // X's codes and scales; dY or x
    const void *b, *b_scales;    // W
    int64_t M, N, K;
    void *out;
    void *workspace;
    int64_t workspace_bytes;
    uint32_t flags;
};

constexpr int64_t kStripWaves = 4, kStripRows = kStripWaves * 32;   // rows of W in a strip
enum Fp4Kernel {
    kFp4Tiles,        // 4-bit instruction, both operands in 4-bit blocks
    kFp4Wide,         // bf16 instruction, W widened on its way into LDS
    kFp4Strips,       // bf16 instruction, W widened in registers, x through LDS; some rows
    kFp4Skinny,       // bf16 instruction, W widened in registers; few rows
    kFp4SkinnyInOne,  // the same, x (rounded) in LDS in the same launch
};
// How a product runs.  `x` bytes at the start of the workspace hold x as the
// kernel reads it (blocks, their scales from `x_scales` on, or padded bf16 rows) and
// turned operands (codes, then scales) from `x_turned` and `w_turned` on, or -1; the
// pieces' sums of a cut product follow.
struct Fp4Choice {
    Fp4Kernel kernel;
    MmChoice mm;
    int64_t x_scales, x;
    int64_t x_turned, w_turned;
};
Fp4Choice fp4_choose(Fp4Op op, int64_t M, int64_t N, int64_t K, uint32_t flags, bool aligned,
                     int64_t workspace_bytes);
// x's rows can be read as they lie: whole units of 128 columns, 16-byte aligned.
bool fp4_whole(const void *x, int64_t K);
tide_status check_fp4(Fp4Op op, const char *name, const Fp4Args &a);

}  // namespace tide
