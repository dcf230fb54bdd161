// The workspace that tide_mx_workspace names is the one with which a product runs as it
// does with any larger one: over random sizes, operand alignments and flags, built with
// g++ from csrc/plan.cpp, block_args.cpp, fp4_args.cpp and this file only.  No GPU.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>
#include <random>

#include "../../parameter_layout_collectives_amd/csrc/fp4.h"

namespace tide {
void release_device_states(const tide_plan *) {}
}  // namespace tide

namespace {

bool same(const tide::Fp4Choice &a, const tide::Fp4Choice &b) {
    return a.kernel == b.kernel && a.x_scales == b.x_scales && a.x == b.x &&
           a.x_turned == b.x_turned && a.w_turned == b.w_turned && a.mm.tile == b.mm.tile &&
           a.mm.direct == b.mm.direct && a.mm.splits == b.mm.splits && a.mm.chunk == b.mm.chunk &&
           a.mm.workspace == b.mm.workspace;
}

constexpr int64_t kAll = std::numeric_limits<int64_t>::max();

int check(tide::Fp4Op op, int64_t M, int64_t N, int64_t K, uint32_t flags) {
    const int64_t asked = tide_mx_workspace(op, M, N, K, flags);
    int wrong = asked < 0;
    for (bool aligned : {false, true}) {
        const tide::Fp4Choice most = tide::fp4_choose(op, M, N, K, flags, aligned, kAll);
        for (int64_t bytes : {asked, asked + 1, 2 * asked + (int64_t(1) << 20), asked + (int64_t(1) << 40)})
            if (!same(tide::fp4_choose(op, M, N, K, flags, aligned, bytes), most)) wrong++;
    }
    if (wrong)
        std::fprintf(stderr, "FAILED: op %d, %lld x %lld x %lld, flags %x, asked %lld\n", op, (long long)M,
                     (long long)N, (long long)K, flags, (long long)asked);
    return wrong;
}

}  // namespace

int main() {
    constexpr uint32_t bf16 = TIDE_F_OUT_BF16;
    int wrong = check(tide::kFp4Dx, 832, 8320, 1920, bf16) + check(tide::kFp4Dx, 479, 3148, 11218, bf16) +
                check(tide::kFp4Dx, 1024, 8192, 8192, bf16) + check(tide::kFp4Linear, 256, 8192, 8192, bf16);
    std::mt19937_64 g(5);
    auto size = [&](int64_t lo, int64_t hi) {
        return int64_t(std::exp(std::uniform_real_distribution<double>(std::log(double(lo)), std::log(double(hi)))(g)));
    };
    for (int t = 0; t < 400000 && wrong < 20; t++) {
        const tide::Fp4Op op = static_cast<tide::Fp4Op>(g() % 3);
        uint32_t flags = g() % 2 ? bf16 : 0u;
        if (op == tide::kFp4Linear && g() % 2) flags |= TIDE_F_QUANT_X | (g() % 2 ? TIDE_F_GRAD_F32 : 0u);
        // half of them where large tiles may be cut
        const bool cut = g() % 2;
        const int64_t M = cut ? size(200, 5000) : size(1, 20000), N = cut ? size(1000, 30000) : size(1, 1 << 20),
                      K = cut ? size(1000, 30000) : size(1, 1 << 20);
        wrong += check(op, M, N, K, flags);
    }
    if (wrong) return 1;
    std::puts("fp4 choice checks passed");
    return 0;
}
