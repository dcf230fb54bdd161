// Kernels that write and read matrices in 8-bit blocks, and their entry
// points: tide_block_quant / tide_block_dequant (the activation checkpoint)
// and tide_block_shard / tide_block_unshard (the 8-bit gather of sharded
// weights).
//
// For a block x[0..127] of one row, with a = max|x| over its finite values:
//   e = the smallest integer with a <= 448 * 2^e, kept in [-117, 119], 0 if a = 0
//   code = the e4m3 number nearest to x * 2^-e, ties to even; |x * 2^-e| is cut
//          at 448 (only a > 448 * 2^119 gets there); inf and NaN become NaN
// A power of two as scale makes both directions exact but for the one rounding
// to e4m3: the scaling moves the exponent alone, and code * 2^e is a bf16
// number, since e4m3 has 4 significant bits and the bounds on e keep it normal.
// (Within 2^e of 448 itself, a quarter of an octave of e4m3 is left unused for
// some blocks, against a fp32 scale; its relative rounding error is the same.)
//
// All four move bytes with little arithmetic, so HBM bounds them: 16 lanes
// share a block, 8 elements each (two 16-byte loads of fp32, one of bf16), and
// each 16-lane group has kUnroll blocks in flight.  Measured: quantising 8192 x
// 8192 bf16 39.4 us (5.2 TB/s), reading it back 32 to 36 us (5.6 to 6.3 TB/s); one
// of 8 ranks of an 8B layer's matrices 26.7 us (5.1 TB/s), placing the whole layer
// in bf16 94.7 us (6.9 TB/s, part of it from the last-level cache).  Rows of any
// width and start are read and written in vectors aligned as one element is, all
// but the last elements of a row: 8191 x 8189 bf16 44.0 and 39.0 us, where 8
// accesses per lane took 77.5 and 94.5.
#include "cast_device.h"

using namespace tide;

extern "C" tide_status tide_block_quant(const void *x, int64_t rows, int64_t cols, void *codes,
                                        void *scales, uint32_t flags, void *stream) {
    const tide_status st = check_block_quant(x, rows, cols, codes, scales, flags);
    if (st != TIDE_OK) return st;
    return run_quant<Eights>("tide_block_quant", x, rows, cols, codes, scales, flags, stream);
}

extern "C" tide_status tide_block_dequant(const void *codes, const void *scales, int64_t rows,
                                          int64_t cols, void *out, uint32_t flags, void *stream) {
    const tide_status st = check_block_dequant(codes, scales, rows, cols, out, flags);
    if (st != TIDE_OK) return st;
    return run_dequant<Eights>("tide_block_dequant", codes, scales, rows, cols, out, flags, stream);
}

extern "C" tide_status tide_block_shard(const tide_plan *plan, int32_t rank, const float *master,
                                        void *block, uint32_t flags, void *stream) {
    const tide_status st = check_block_shard(plan, rank, master, block, flags);
    if (st != TIDE_OK) return st;
    return run_shard<Eights>("tide_block_shard", plan, rank, master, block, stream);
}

extern "C" tide_status tide_block_unshard(const tide_plan *plan, const void *gathered,
                                          void *const *params, uint32_t flags, void *stream) {
    const tide_status st = check_block_unshard(plan, gathered, params, flags);
    if (st != TIDE_OK) return st;
    return run_unshard<Eights>("tide_block_unshard", plan, gathered, params, flags, stream);
}
