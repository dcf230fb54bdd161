// Orthogonalised updates: the workspace's layout and the argument checks
// (ortho_args.cpp, host only), and the launches (ortho.hip).
#pragma once

#include <vector>

#include "block.h"

namespace tide {

// P X takes X's lo as well up to this many rows (the smaller side), and for any where the
// steps raise what is near zero by more than kOrthoRaisedHi; up to kOrthoSmall rows the
// steps run on X X^T alone, in 64 bits, until they have raised it by kOrthoRaised: see
// ortho.hip.
constexpr uint32_t kOrthoBoth = 256, kOrthoSmall = 32;
constexpr double kOrthoRaisedHi = 512.0;
constexpr int64_t kOrthoSmallCols = 128;       // columns of a small matrix in LDS
constexpr double kOrthoRaised = 32768.0;

// Equal matrices [nr, nc] of one call, as the kernels see them.  r is the smaller
// side; the padded sizes are multiples of 64, zeros in between.
struct OrthoGroup {
    uint32_t nr, nc;             // rows and columns
    uint32_t nrp, ncp;           // padded
    uint32_t first, count;       // its matrices' numbers
    uint32_t parts;              // pieces of a matrix's sum of squares
    uint32_t wg0;                // first workgroup of a launch that works on them
    int64_t base, stride;        // bytes of the first matrix in the workspace, and from one to the next

    __host__ __device__ bool tall() const { return nr > nc; }
    __host__ __device__ uint32_t r() const { return tall() ? nc : nr; }
    __host__ __device__ uint32_t rp() const { return tall() ? ncp : nrp; }
    // fp16 matrices [R, C] lie in panels of 32 columns, [C / 32, R, 32]: the bytes that a
    // workgroup loads for one step of a sum, along the rows or across them, are runs of
    // 1 KB or more.  X is held twice (a step reads one and writes the other), each time
    // as a matrix hi and behind it lo.
    __host__ __device__ int64_t x_bytes() const { return 4 * static_cast<int64_t>(nrp) * ncp; }
    __host__ __device__ int64_t lo() const { return static_cast<int64_t>(nrp) * ncp; }
    // Whether lo enters P X, too, by the rows alone.
    __host__ __device__ bool both() const { return r() <= kOrthoBoth; }
    // Then A = X X^T and P [rp, rp] without their diagonals, and these in fp32 [rp].
    __host__ __device__ int64_t a_at() const { return 2 * x_bytes(); }
    __host__ __device__ int64_t p_at() const {
        return a_at() + 2 * static_cast<int64_t>(rp()) * rp();
    }
    __host__ __device__ int64_t a_diag() const { return p_at() + 2 * static_cast<int64_t>(rp()) * rp(); }
    __host__ __device__ int64_t p_diag() const { return a_diag() + 4 * rp(); }
    // A small matrix: G in fp32, a later X in fp64, `parts` sums of X X^T, and the matrix
    // that X is multiplied by, followed by the exponent of 2 that it is divided by (fp64).
    __host__ __device__ bool small() const { return r() <= kOrthoSmall; }
    __host__ __device__ int64_t later_at() const { return (4 * static_cast<int64_t>(nr) * nc + 15) / 16 * 16; }
    __host__ __device__ int64_t gram_at() const { return later_at() + 8 * static_cast<int64_t>(nr) * nc; }
    __host__ __device__ int64_t map_at() const { return gram_at() + 8 * static_cast<int64_t>(parts) * r() * r(); }
    __host__ __device__ int64_t bytes() const {
        return small() ? map_at() + 8 * (static_cast<int64_t>(r()) * r() + 1) : p_diag() + 4 * rp();
    }
};

constexpr uint32_t kOrthoParts = 256;          // most pieces of a sum of squares
constexpr int64_t kOrthoPiece = 16384;         // elements of a piece, if that is not too many
constexpr int kOrthoGroups = 48;               // groups per launch, as kernel arguments

struct OrthoArgs {
    int32_t n;
    const void *const *src;
    void *const *out;
    const int64_t *rows, *cols;
    int32_t steps;
    const float *coefficients;
    uint32_t flags;
    void *workspace;
    int64_t workspace_bytes;
};
// The call's groups, its matrices in their order, and the workspace:
// {src, out} pointers, one pair a matrix, from 0 on; sums of squares, kOrthoParts
// doubles a matrix, from `sums` on; {scale, its square} of a matrix's first
// step from `scales` on; the groups' matrices.
struct OrthoPlan {
    std::vector<OrthoGroup> groups;
    std::vector<int32_t> order;
    int64_t sums = 0, scales = 0, bytes = 0;
};
tide_status ortho_plan(const char *name, int32_t n, const int64_t *rows, const int64_t *cols,
                       OrthoPlan *plan);
tide_status check_ortho(const OrthoArgs &a, OrthoPlan *plan);

}  // namespace tide
