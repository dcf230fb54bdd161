// Entry points that write and read matrices in 4-bit blocks: tide_mx_quant,
// tide_mx_dequant, and the 4-bit gather of sharded weights, tide_mx_shard and
// tide_mx_unshard.
//
// For a block x[0..31] of one row, with a = max|x|:
//   e = the smallest integer with a <= 6 * 2^e, kept in [-125, 125], 0 if a = 0
//   code = the e2m1 number (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) nearest
//          to x * 2^-e, ties to the even code; |x| above 6 * 2^125 is cut there
// and a block that holds an infinity or a NaN is NaN as a whole (scale byte 255).
// Scaling by a power of two moves the exponent alone, so the only rounding is the
// one to e2m1, and every value is a bf16 number.  The smallest e without a cut, not
// the one with the finest steps (which cuts up to a quarter off the largest value):
// a weight's largest entries carry most of what a product sums.
//
// As for 8-bit blocks, HBM bounds all of them: 16 lanes share 128 columns, 8
// elements each (4 lanes a block), four such units in flight.  A rank's eighth of an 8B
// layer from fp32 shards 24.4 us, 5.1 TB/s; the gathered layer to bf16 78 us, 7.1 TB/s
// (what was just written comes from the last-level cache); 14336 x 4096 fp32 into blocks
// 54 us, 4.9 TB/s (a copy reaches 4.8 to 5.3).
#include "cast_device.h"
#include "fp4.h"

using namespace tide;

extern "C" tide_status tide_mx_quant(const void *x, int64_t rows, int64_t cols, void *codes,
                                      void *scales, uint32_t flags, void *stream) {
    const char *name = "tide_mx_quant";
    const tide_status st = check_quant(name, kFours, x, rows, cols, codes, scales, flags);
    if (st != TIDE_OK) return st;
    return run_quant<Fours>(name, x, rows, cols, codes, scales, flags, stream);
}

extern "C" tide_status tide_mx_dequant(const void *codes, const void *scales, int64_t rows,
                                        int64_t cols, void *out, uint32_t flags, void *stream) {
    const char *name = "tide_mx_dequant";
    const tide_status st = check_dequant(name, kFours, codes, scales, rows, cols, out, flags);
    if (st != TIDE_OK) return st;
    return run_dequant<Fours>(name, codes, scales, rows, cols, out, flags, stream);
}

extern "C" tide_status tide_mx_shard(const tide_plan *plan, int32_t rank, const float *master,
                                      void *block, uint32_t flags, void *stream) {
    const char *name = "tide_mx_shard";
    const tide_status st = check_shard(name, kFours, plan, rank, master, block, flags);
    if (st != TIDE_OK) return st;
    return run_shard<Fours>(name, plan, rank, master, block, stream);
}

extern "C" tide_status tide_mx_unshard(const tide_plan *plan, const void *gathered,
                                        void *const *params, uint32_t flags, void *stream) {
    const char *name = "tide_mx_unshard";
    const tide_status st = check_unshard(name, kFours, plan, gathered, params, flags);
    if (st != TIDE_OK) return st;
    return run_unshard<Fours>(name, plan, gathered, params, flags, stream);
}
