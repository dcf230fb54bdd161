// Argument checks that the blocked matrices' entry points share (block_args.cpp,
// fp4_args.cpp, ortho_args.cpp).  Host only, no HIP call.
#pragma once

#include <string>

#include "block.h"

namespace tide {

constexpr int64_t kMaxDim = int64_t(1) << 31;   // rows and columns of a block matrix
constexpr int64_t kMaxLine = int64_t(1) << 22;  // n and k of a product: its kernels address the
                                                // rows of a tile, 2 * 2^22 bytes each, in 32 bits

struct Bytes {
    uintptr_t lo, hi;
};
inline Bytes bytes_of(const void *p, int64_t n) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + static_cast<uintptr_t>(n)};
}
inline bool overlap(const Bytes &a, const Bytes &b) { return a.lo < b.hi && b.lo < a.hi; }
inline bool misaligned(const void *p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

inline tide_status bad(const char *name, const char *what) {
    return fail(TIDE_E_INVALID, std::string(name) + ": " + what);
}

inline tide_status check_flags(const char *name, uint32_t flags, uint32_t known) {
    if (flags & ~known) return fail(TIDE_E_UNSUPPORTED, std::string(name) + ": unknown flag bits");
    if ((flags & TIDE_F_GRAD_F16) && (flags & TIDE_F_GRAD_F32))
        return bad(name, "TIDE_F_GRAD_F16 and TIDE_F_GRAD_F32 both set");
    if ((flags & TIDE_F_OUT_BF16) && (flags & TIDE_F_OUT_F16))
        return bad(name, "TIDE_F_OUT_BF16 and TIDE_F_OUT_F16 both set");
    if ((flags & TIDE_F_SHORT_SUMS) && !(flags & TIDE_F_OUT_BF16))
        return bad(name, "TIDE_F_SHORT_SUMS without TIDE_F_OUT_BF16");
    return TIDE_OK;
}

inline tide_status check_dims(const char *name, int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return bad(name, "negative size");
    if (rows >= kMaxDim || cols >= kMaxDim) return bad(name, "a size of 2^31 or more");
    // the products' byte offsets then fit int64 with room to spare
    if (rows && block_cols(cols) > (int64_t(1) << 60) / rows) return bad(name, "sizes overflow");
    return TIDE_OK;
}

// A matrix in 8-bit or 4-bit blocks: both pointers present and aligned for the widest
// loads the kernels make of them.
inline tide_status check_blocks(const char *name, const char *which, const void *codes,
                         const void *scales) {
    if (!codes) return bad(name, (std::string(which) + " codes are NULL").c_str());
    if (!scales) return bad(name, (std::string(which) + " scales are NULL").c_str());
    if (misaligned(codes, 16))
        return bad(name, (std::string(which) + " codes are not 16-byte aligned").c_str());
    if (misaligned(scales, 4))
        return bad(name, (std::string(which) + " scales are not 4-byte aligned").c_str());
    return TIDE_OK;
}

}  // namespace tide
