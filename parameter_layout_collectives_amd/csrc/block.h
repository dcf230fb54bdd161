// Matrices in 8-bit blocks: the format, the checks of its entry points
// (block_args.cpp, host only) and the launches (block_cast.hip, block_mm.hip).
//
// A matrix [R, C] is held as codes [R, Cp] (e4m3 bytes, Cp = C rounded up to
// 128) and scales [R, Sp] (e8m0 bytes, one per 128 columns, rounded up to 4):
// element (r, c) is e4m3(codes[r, c]) * 2^(scales[r, c / 128] - 127).  Blocks
// lie inside one row, so a dim-0 shard boundary never cuts one.
#pragma once

#include "internal.h"

namespace tide {

constexpr int64_t kBlockCols = 128;
inline int64_t block_cols(int64_t c) { return (c + kBlockCols - 1) / kBlockCols * kBlockCols; }
inline int64_t block_count(int64_t c) { return (c + kBlockCols - 1) / kBlockCols; }
inline int64_t block_scale_cols(int64_t c) { return (block_count(c) + 3) / 4 * 4; }

// Element types that become 8-bit blocks or come back from them.
enum ElemType { kElemBf16 = 0, kElemF16 = 1, kElemF32 = 2 };
inline ElemType in_type(uint32_t flags) {
    return (flags & TIDE_F_GRAD_F32) ? kElemF32 : (flags & TIDE_F_GRAD_F16) ? kElemF16 : kElemBf16;
}
inline ElemType out_type(uint32_t flags) {
    return (flags & TIDE_F_OUT_BF16) ? kElemBf16 : (flags & TIDE_F_OUT_F16) ? kElemF16 : kElemF32;
}
inline int elem_size(ElemType t) { return t == kElemF32 ? 4 : 2; }

// The three products.  Each is out[i, j] = sum over c of I(i, c) * J(c, j),
// with J always in 8-bit blocks:
//   kMm    i = token, j = row of W, c = column: I = X (blocks), J = W
//   kMmDx  i = token, j = column of W, c = row of W: I = dY (bf16), J = W
//   kMmDw  i = row of W, j = column, c = token: I = dY transposed, J = X
enum MmOp { kMm = 0, kMmDx = 1, kMmDw = 2 };

// MI355X's compute units: a product's tiles are counted against them.  Fewer of
// them (a partition of the card) would change the choice's speed, not its results.
constexpr int64_t kCus = 256;
// The skinny kernel takes up to 24 rows (16 against the 8-bit instruction's
// tiles), and up to 64 if W is small: there the second launch of a cut sum costs
// more than the tiles gain.  Skinny against tiles with fp32 sums and join, us, W
// from memory (and from the last-level cache, where tiles gain more):
//   n = 8192, k = 28672:  17 rows 73 / 88 (64 / 61), 24: 83 / 90 (74 / 63),
//                         28: 88 / 92 (80 / 64), 32: 95 / 94 (85 / 70)
//   n = 14336, k = 4096:  17 rows 23 / 27 (22 / 21), 24: 25 / 27 (23 / 22),
//                         28: 27 / 28 (26 / 22), 32: 29 / 28 (27 / 22)
//   n = k = 5120:         17 rows 13 / 14, 20: 14 / 14, 24: 15 / 14, 32: 17 / 15
//   n = k = 4096:         32 rows 9.4 / 12.0, 48: 11.7 / 12.9, 64: 13.2 / 14.0
//   n = k = 2048:         40 rows 6.2 / 8.7, 64: 7.3 / 9.5
// and against the 8-bit instruction's, n = 8192, k = 28672, 32 rows: 95 / 61.
constexpr int64_t kSkinnyRows = 24;
constexpr int64_t kSkinnyShort = 16;
constexpr int64_t kSkinnyMost = 64;
constexpr int64_t kSkinnyWeights = int64_t(1) << 24;
// x's blocks are made inside the product for one row of at most 28 KB of codes,
// or more rows of at most 8 KB together: every workgroup repeats that work.
// In one launch against two, us:
//   one row, n = 8192:    k = 24576 41 / 47, 28672 49 / 55, 32768 66 / 62
//   n = 14336, k = 4096:  1 row 15.6 / 18.8, 2: 17.6 / 20.2, 3: 19.3 / 20.4,
//                         4: 21.2 / 20.8, 8: 28.2 / 22.1
//   16 rows, n = 4096:    k = 512 3.5 / 6.2, 1024 7.2 / 8.2
constexpr int64_t kInOneRows = 16;
constexpr int64_t kInOneRow = 28672;     // 56 KB of LDS
constexpr int64_t kInOneBytes = 8192;
// The least steps (64 or 128 values) in a piece of a cut sum, and the most pieces.
// 4 steps against 8, us: 512 x 512 over 512 6.6 / 5.2, over 2048 11.7 / 9.2;
// 512 x 1024 over 1024 11 / 10; 64 x 64 over 512 5.7 / 4.7, over 1024 5.9 / 6.7;
// 128 x 512 over 1024 6.4 / 7.0.  16 pieces against 8 and 32, over 16384: 64 x 64
// (dW) 11.0 / 14.8 / 10.3, 128 x 512 12.8 / 15.6 / 15.3.
constexpr int64_t kMinSplitSteps = 4;
constexpr int64_t kMaxSplits = 16;

// How a product runs: the kernel, its tile, and which tiles' sums are cut.
enum MmKernel { kMmEight, kMmWide, kMmSkinny };
struct MmChoice {
    MmKernel kernel;
    int tile;            // 256, 128 or 64 rows and columns of the output per workgroup
    int64_t direct;      // tiles that one workgroup computes; the others are cut
    int splits;          // into so many pieces each,
    int64_t chunk;       // of so many steps
    int64_t workspace;   // bytes for the pieces' sums
};
// dY's rows can be loaded in 16-byte pieces (X's and W's codes always can).
inline bool mm_aligned(MmOp op, const void *dy, int64_t N) {
    return op == kMm || (reinterpret_cast<uintptr_t>(dy) % 16 == 0 && N % 8 == 0);
}
MmChoice mm_choose(MmOp op, int64_t M, int64_t N, int64_t K, uint32_t flags, bool aligned,
                   bool may_split);

tide_status check_block_quant(const void *x, int64_t rows, int64_t cols, const void *codes,
                              const void *scales, uint32_t flags);
tide_status check_block_dequant(const void *codes, const void *scales, int64_t rows, int64_t cols,
                                const void *out, uint32_t flags);
tide_status check_block_shard(const tide_plan *bp, int32_t rank, const void *master,
                              const void *block, uint32_t flags);
tide_status check_block_unshard(const tide_plan *bp, const void *gathered, void *const *params,
                                uint32_t flags);

// Operands of a product as its entry point got them: `a` is X's codes or dY.
struct MmArgs {
    const void *a, *a_scales;
    const void *b, *b_scales;
    int64_t M, N, K;
    void *out;
    void *workspace;
    int64_t workspace_bytes;
    uint32_t flags;
};
tide_status check_mm(MmOp op, const char *name, const MmArgs &g);

// A product whose x is not in blocks yet.
struct LinearArgs {
    const void *x;
    const void *b, *b_scales;
    int64_t M, N, K;
    void *out;
    void *workspace;
    int64_t workspace_bytes;
    uint32_t flags;
};
// in_one: the kernel makes x's blocks in LDS.  Else they lie at the start of the
// workspace, the scales from `scales` on, `blocks` bytes in all.
struct LinearChoice {
    bool in_one;
    int64_t scales, blocks;
};
LinearChoice linear_choose(int64_t M, int64_t K);
tide_status check_linear(const LinearArgs &a);

}  // namespace tide
