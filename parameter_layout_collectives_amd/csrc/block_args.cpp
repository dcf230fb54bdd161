// Host side of the 8-bit block operators: block plans, argument checks and
// the choice of a product's kernel.  Makes no HIP call.
#include <algorithm>
#include <new>

#include "block.h"
#include "checks.h"

namespace tide {
namespace {

// Flags and sizes of a product; `known`: the flags it takes.  A launch counts its
// lanes in 32 bits: that too is checked here, before anything is enqueued.
tide_status check_product(const char *name, MmOp op, int64_t M, int64_t N, int64_t K,
                          uint32_t flags, uint32_t known, bool aligned) {
    tide_status st = check_flags(name, flags, known);
    if (st != TIDE_OK) return st;
    for (int64_t rows : {M, N})
        for (int64_t cols : {N, K})
            if ((st = check_dims(name, rows, cols)) != TIDE_OK) return st;
    if (N > kMaxLine || K > kMaxLine)
        return fail(TIDE_E_UNSUPPORTED, std::string(name) + ": n or k above 2^22");
    const int64_t rows = op == kMmDw ? N : M, cols = op == kMm ? N : K;
    const MmChoice c = mm_choose(op, M, N, K, flags, aligned, true);
    const int64_t tiles = ((rows + c.tile - 1) / c.tile) * ((cols + c.tile - 1) / c.tile);
    const int64_t cut = (tiles - c.direct) * c.splits;
    if (tiles + cut > 0xffffffffll / 512 || cut * (c.tile * c.tile / 1024) > 0xffffffffll / 256)
        return fail(TIDE_E_UNSUPPORTED, std::string(name) + ": more than 2^32 lanes");
    return TIDE_OK;
}

uint32_t known_flags(MmOp op) {
    return TIDE_F_OUT_BF16 | (op == kMmDw ? TIDE_F_ACCUMULATE : 0u) |
           (op == kMm ? TIDE_F_SHORT_SUMS : 0u);
}
constexpr uint32_t kLinearFlags =
    TIDE_F_GRAD_F16 | TIDE_F_GRAD_F32 | TIDE_F_OUT_BF16 | TIDE_F_SHORT_SUMS;

tide_status check_plan(const char *name, Format f, const tide_plan *bp) {
    if (!bp) return bad(name, "plan is NULL");
    if (!bp->nblk || bp->blk_bits != f.bits)
        return bad(name, f.bits == 4 ? "not a plan of tide_plan_create_mx"
                                     : "not a plan of tide_plan_create_blocks");
    return TIDE_OK;
}

}  // namespace

tide_status check_quant(const char *name, Format f, const void *x, int64_t rows, int64_t cols,
                        const void *codes, const void *scales, uint32_t flags) {
    tide_status st = check_flags(name, flags, TIDE_F_GRAD_F16 | TIDE_F_GRAD_F32);
    if (st == TIDE_OK) st = check_dims(name, rows, cols);
    if (st != TIDE_OK || rows == 0 || cols == 0) return st;
    const int es = elem_size(in_type(flags));
    if (!x) return bad(name, "x is NULL");
    if (misaligned(x, es)) return bad(name, "x is not aligned to its element size");
    st = check_blocks(name, "the output's", codes, scales);
    if (st != TIDE_OK) return st;
    const Bytes in = bytes_of(x, rows * cols * es), c = bytes_of(codes, rows * f.code_bytes(cols)),
                s = bytes_of(scales, rows * f.scale_bytes(cols));
    if (overlap(in, c) || overlap(in, s) || overlap(c, s))
        return bad(name, "an output overlaps the input or the other output");
    return TIDE_OK;
}

tide_status check_dequant(const char *name, Format f, const void *codes, const void *scales,
                          int64_t rows, int64_t cols, const void *out, uint32_t flags) {
    tide_status st = check_flags(name, flags, TIDE_F_OUT_BF16 | TIDE_F_OUT_F16);
    if (st == TIDE_OK) st = check_dims(name, rows, cols);
    if (st != TIDE_OK || rows == 0 || cols == 0) return st;
    st = check_blocks(name, "the input's", codes, scales);
    if (st != TIDE_OK) return st;
    const int es = elem_size(out_type(flags));
    if (!out) return bad(name, "out is NULL");
    if (misaligned(out, es)) return bad(name, "out is not aligned to its element size");
    const Bytes o = bytes_of(out, rows * cols * es);
    if (overlap(o, bytes_of(codes, rows * f.code_bytes(cols))) ||
        overlap(o, bytes_of(scales, rows * f.scale_bytes(cols))))
        return bad(name, "out overlaps the input");
    return TIDE_OK;
}

tide_status check_shard(const char *name, Format f, const tide_plan *bp, int32_t rank,
                        const void *master, const void *block, uint32_t flags) {
    tide_status st = check_plan(name, f, bp);
    if (st != TIDE_OK) return st;
    if (rank < 0 || rank >= bp->N)
        return fail(TIDE_E_INVALID, std::string(name) + ": rank " + std::to_string(rank) +
                                        " outside [0, " + std::to_string(bp->N) + ")");
    st = check_flags(name, flags, 0);
    if (st != TIDE_OK || bp->S == 0) return st;
    if (!master) return bad(name, "master is NULL");
    if (misaligned(master, 4)) return bad(name, "master is not aligned to its element size");
    if (!block) return bad(name, "block is NULL");
    if (misaligned(block, 16)) return bad(name, "block is not 16-byte aligned");
    if (overlap(bytes_of(master, bp->blk_S * 4), bytes_of(block, bp->S * 4)))
        return bad(name, "block overlaps master");
    return TIDE_OK;
}

tide_status check_unshard(const char *name, Format f, const tide_plan *bp, const void *gathered,
                          void *const *params, uint32_t flags) {
    tide_status st = check_plan(name, f, bp);
    if (st != TIDE_OK) return st;
    st = check_flags(name, flags, TIDE_F_OUT_BF16 | TIDE_F_OUT_F16);
    if (st != TIDE_OK || bp->psi == 0) return st;
    if (!gathered) return bad(name, "gathered is NULL");
    if (misaligned(gathered, 16)) return bad(name, "gathered is not 16-byte aligned");
    if (!params) return bad(name, "params array is NULL");
    const int es = elem_size(out_type(flags));
    const Bytes src = bytes_of(gathered, bp->S * 4 * bp->N);
    std::vector<Bytes> dst;
    try {
        dst.reserve(bp->nblk);
    } catch (const std::bad_alloc &) {
        return fail(TIDE_E_NOMEM, std::string(name) + ": out of host memory");
    }
    for (int32_t j = 0; j < bp->nblk; j++) {
        const int64_t n = bp->d0[j] * bp->blk_inner[j];
        if (n == 0) continue;
        const std::string which = "params[" + std::to_string(j) + "]";
        if (!params[j]) return bad(name, (which + " is NULL").c_str());
        if (misaligned(params[j], es))
            return bad(name, (which + " is not aligned to its element size").c_str());
        dst.push_back(bytes_of(params[j], n * es));
        if (overlap(dst.back(), src))
            return bad(name, (which + " overlaps the gathered buffer").c_str());
    }
    std::sort(dst.begin(), dst.end(), [](const Bytes &a, const Bytes &b) { return a.lo < b.lo; });
    for (size_t k = 1; k < dst.size(); k++)
        if (overlap(dst[k - 1], dst[k])) return bad(name, "a destination overlaps another");
    return TIDE_OK;
}

tide_status create_plan(const char *name, Format f, const tide_plan *plan, int32_t n,
                        const int32_t *select, tide_plan **out_plan) {
    if (!out_plan) return bad(name, "out_plan is NULL");
    *out_plan = nullptr;
    if (!plan) return bad(name, "plan is NULL");
    if (plan->nblk) return bad(name, "plan is a block plan itself");
    if (n < 1 || n > plan->P) return bad(name, "n outside [1, nparams]");
    if (!select) return bad(name, "select is NULL");
    try {
        std::vector<int64_t> d0(2 * static_cast<size_t>(n)), words(d0.size()), off(n), inner(n);
        std::vector<char> seen(plan->P, 0);
        for (int32_t j = 0; j < n; j++) {
            const int32_t i = select[j];
            if (i < 0 || i >= plan->P) return bad(name, "select holds an index out of range");
            if (seen[i]) return bad(name, "select holds an index twice");
            seen[i] = 1;
            const tide_status st = check_dims(name, plan->d0[i], plan->inner[i]);
            if (st != TIDE_OK) return st;
            d0[j] = d0[n + j] = plan->d0[i];
            words[j] = f.code_bytes(plan->inner[i]) / 4;
            words[n + j] = f.scale_bytes(plan->inner[i]) / 4;
            off[j] = plan->off[i];
            inner[j] = plan->inner[i];
        }
        // offsets at multiples of 4 words: every segment starts 16-byte aligned
        tide_plan *p = nullptr;
        const tide_status st =
            tide_plan_create(plan->N, 2 * n, d0.data(), words.data(), 4, &p);
        if (st != TIDE_OK) return st;
        if (p->S / 4 > 0xffffffffll) {
            tide_plan_destroy(p);
            return bad(name, "a rank block of more than 2^36 bytes");
        }
        p->nblk = n;
        p->blk_bits = f.bits;
        p->blk_S = plan->S;
        p->blk_off.swap(off);
        p->blk_inner.swap(inner);
        *out_plan = p;
    } catch (const std::bad_alloc &) {
        return fail(TIDE_E_NOMEM, std::string(name) + ": out of host memory");
    }
    return TIDE_OK;
}

tide_status check_mm(MmOp op, const char *name, const MmArgs &g) {
    tide_status st = check_product(name, op, g.M, g.N, g.K, g.flags, known_flags(op),
                                   mm_aligned(op, g.a, g.N));
    if (st != TIDE_OK) return st;
    if (g.workspace_bytes < 0) return bad(name, "workspace_bytes < 0");
    if (g.workspace_bytes > 0 && !g.workspace) return bad(name, "workspace is NULL");
    if (g.workspace && misaligned(g.workspace, 16))
        return bad(name, "workspace is not 16-byte aligned");
    const int64_t orows = op == kMmDw ? g.N : g.M, ocols = op == kMm ? g.N : g.K;
    const int64_t sum = op == kMm ? g.K : op == kMmDx ? g.N : g.M;
    if (orows == 0 || ocols == 0) return TIDE_OK;
    const int es = elem_size(out_type(g.flags));
    if (!g.out) return bad(name, "out is NULL");
    if (misaligned(g.out, es)) return bad(name, "out is not aligned to its element size");
    const Bytes out = bytes_of(g.out, orows * ocols * es);
    const Bytes wsp = bytes_of(g.workspace, g.workspace ? g.workspace_bytes : 0);
    if (overlap(out, wsp)) return bad(name, "out overlaps the workspace");
    if (sum == 0) return TIDE_OK;
    // a: X in blocks [M, K] (kMm) or dY [M, N]; b: W [N, K] or X [M, K] in blocks
    Bytes in[4];
    int n = 0;
    if (op == kMm) {
        st = check_blocks(name, "x's", g.a, g.a_scales);
        in[n++] = bytes_of(g.a, g.M * block_cols(g.K));
        in[n++] = bytes_of(g.a_scales, g.M * block_scale_cols(g.K));
    } else {
        if (!g.a) return bad(name, "dy is NULL");
        if (misaligned(g.a, 2)) return bad(name, "dy is not aligned to its element size");
        in[n++] = bytes_of(g.a, g.M * g.N * 2);
    }
    if (st == TIDE_OK) st = check_blocks(name, op == kMmDw ? "x's" : "w's", g.b, g.b_scales);
    if (st != TIDE_OK) return st;
    const int64_t brows = op == kMmDw ? g.M : g.N;
    in[n++] = bytes_of(g.b, brows * block_cols(g.K));
    in[n++] = bytes_of(g.b_scales, brows * block_scale_cols(g.K));
    for (int k = 0; k < n; k++) {
        if (overlap(out, in[k])) return bad(name, "out overlaps an operand");
        if (overlap(wsp, in[k])) return bad(name, "the workspace overlaps an operand");
    }
    return TIDE_OK;
}

LinearChoice linear_choose(int64_t M, int64_t K) {
    const int64_t bytes = M * block_cols(K);
    LinearChoice c = {M <= kInOneRows && bytes <= (M == 1 ? kInOneRow : kInOneBytes), 0, 0};
    if (c.in_one) return c;
    const int64_t round = 255;
    c.scales = (M * block_cols(K) + round) & ~round;
    c.blocks = (c.scales + M * block_scale_cols(K) + round) & ~round;
    return c;
}

tide_status check_linear(const LinearArgs &a) {
    const char *name = "tide_block_linear";
    tide_status st = check_product(name, kMm, a.M, a.N, a.K, a.flags, kLinearFlags, true);
    if (st != TIDE_OK) return st;
    if (a.workspace_bytes < 0) return bad(name, "workspace_bytes < 0");
    if (a.workspace_bytes > 0 && !a.workspace) return bad(name, "workspace is NULL");
    if (misaligned(a.workspace, 16)) return bad(name, "workspace is not 16-byte aligned");
    if (a.M == 0 || a.N == 0) return TIDE_OK;
    const int es = elem_size(in_type(a.flags)), os = elem_size(out_type(a.flags));
    if (!a.out) return bad(name, "out is NULL");
    if (misaligned(a.out, os)) return bad(name, "out is not aligned to its element size");
    const Bytes out = bytes_of(a.out, a.M * a.N * os);
    const Bytes wsp = bytes_of(a.workspace, a.workspace ? a.workspace_bytes : 0);
    if (overlap(out, wsp)) return bad(name, "out overlaps the workspace");
    if (a.K == 0) return TIDE_OK;
    if (!a.x) return bad(name, "x is NULL");
    if (misaligned(a.x, es)) return bad(name, "x is not aligned to its element size");
    st = check_blocks(name, "w's", a.b, a.b_scales);
    if (st != TIDE_OK) return st;
    for (const Bytes &in : {bytes_of(a.x, a.M * a.K * es), bytes_of(a.b, a.N * block_cols(a.K)),
                            bytes_of(a.b_scales, a.N * block_scale_cols(a.K))}) {
        if (overlap(out, in)) return bad(name, "out overlaps an operand");
        if (overlap(wsp, in)) return bad(name, "the workspace overlaps an operand");
    }
    return TIDE_OK;
}

void cut_sums(MmChoice &c, int64_t tiles, int64_t steps) {
    // The tiles that run at one time; what is left after whole sets of them is
    // cut if that leaves at least half of the card idle (more tiles could not be
    // cut in two: 256 + 128 large tiles, 4096 x 6144, over 8192: cut 330 us, else
    // 384).  The pieces' sums go through memory, so a piece has at least
    // kMinSplitSteps steps, and behind whole sets (where one is long) at least four
    // times that (256 + 16 large tiles, 4352 x 4096, over 2048: pieces of 16 steps
    // 90 us, of 8 82, not cut 105; over 8192 243, 242, cut in fewer 257).
    const int64_t full = kCus * (c.tile == 256 ? 1 : 2);
    const int64_t left = tiles % full, least = tiles < full ? kMinSplitSteps : 4 * kMinSplitSteps;
    if (left == 0 || left * 2 > full || steps < 2 * least) return;
    const int64_t s = std::min({full / left, steps / least, kMaxSplits});
    const int64_t chunk = ((steps + s - 1) / s + 3) / 4 * 4;   // scale bytes are read in fours
    const int64_t pieces = (steps + chunk - 1) / chunk;
    if (pieces < 2) return;
    c.chunk = chunk;
    c.splits = static_cast<int>(pieces);
    c.direct = tiles - left;
    c.workspace = left * pieces * c.tile * c.tile * 4;
}

MmChoice mm_choose(MmOp op, int64_t M, int64_t N, int64_t K, uint32_t flags, bool aligned,
                   bool may_split) {
    MmChoice c;
    const int64_t rows = op == kMmDw ? N : M, cols = op == kMm ? N : K;
    const int64_t sum = op == kMm ? K : op == kMmDx ? N : M;
    const bool eight = op == kMm && (flags & TIDE_F_SHORT_SUMS);
    const bool skinny = M <= (eight ? kSkinnyShort : kSkinnyRows) ||
                        (M <= kSkinnyMost && N * K <= kSkinnyWeights);
    c.kernel = op == kMm && skinny ? kMmSkinny : eight ? kMmEight : kMmWide;
    const int64_t step = eight ? 128 : 64;
    const int64_t steps = (sum + step - 1) / step;
    auto tiles = [&](int64_t t) { return ((rows + t - 1) / t) * ((cols + t - 1) / t); };
    // Large tiles once they fill three quarters of the card, small ones (not in
    // the 8-bit kernel) while middle ones would leave half of it idle.  x w^T, us:
    //   256 / 128 wide over 1024 and 8192:
    //     2560 x 3328 (130 large tiles)  34 / 36, 186 / 156
    //     2816 x 4096 (176)              33 / 35, 187 / 227
    //     3584 x 3584 (196)              35 / 43, 187 / 279
    //   128 / 64 wide over 512, 2048 and 8192:
    //     1024 x 1152 (72 middle tiles)  14 / 7, 27 / 18, 39 / 61
    //     1280 x 1280 (100)              17 / 7, 26 / 18, 46 / 63
    //     1408 x 1536 (132)              22 / 8, 27 / 21, 62 / 67
    //     1920 x 1920 (225)              24 / 11, 32 / 29, 83 / 105
    // So the borders lie where sums of about 8192 (large tiles) and 4096 (small
    // ones) change sides; shorter and longer ones would have theirs elsewhere.
    c.tile = aligned && tiles(256) >= kCus * 3 / 4 ? 256
             : !eight && tiles(128) < kCus / 2     ? 64
                                                   : 128;
    const int64_t t = tiles(c.tile);
    c.direct = t;
    c.splits = 1;
    c.chunk = steps;
    c.workspace = 0;
    if (c.kernel == kMmSkinny || !may_split) return c;
    cut_sums(c, t, steps);
    return c;
}

}  // namespace tide

using tide::bad;
using tide::fail;

extern "C" {

int64_t tide_block_cols(int64_t cols) {
    return cols < 0 || cols >= tide::kMaxDim ? -1 : tide::block_cols(cols);
}

int64_t tide_block_scale_cols(int64_t cols) {
    return cols < 0 || cols >= tide::kMaxDim ? -1 : tide::block_scale_cols(cols);
}

tide_status tide_plan_create_blocks(const tide_plan *plan, int32_t n, const int32_t *select,
                                    tide_plan **out_plan) {
    return tide::create_plan("tide_plan_create_blocks", tide::kEights, plan, n, select, out_plan);
}

int64_t tide_block_workspace(int32_t op, int64_t m, int64_t n, int64_t k, uint32_t flags) {
    const char *name = "tide_block_workspace";
    if (op < 0 || op > 3) {
        bad(name, "op outside [0, 3]");
        return -1;
    }
    const tide::MmOp mm = op == 3 ? tide::kMm : static_cast<tide::MmOp>(op);
    const uint32_t known = op == 3 ? tide::kLinearFlags : tide::known_flags(mm);
    if (tide::check_product(name, mm, m, n, k, flags, known, tide::mm_aligned(mm, nullptr, n)) !=
        TIDE_OK)
        return -1;
    if (op == 3) {               // tide_block_linear: x's blocks, then the product's
        const tide::LinearChoice c = tide::linear_choose(m, k);
        if (c.in_one || n == 0) return 0;
        return c.blocks +
               tide_block_workspace(0, m, n, k, flags & (TIDE_F_OUT_BF16 | TIDE_F_SHORT_SUMS));
    }
    // whichever way dY is aligned
    int64_t most = 0;
    for (bool aligned : {false, true})
        most = std::max(most, tide::mm_choose(static_cast<tide::MmOp>(op), m, n, k, flags, aligned,
                                              true).workspace);
    return most;
}

}  // extern "C"
