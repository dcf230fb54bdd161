// The host code of the 8-bit blocks (sizes, argument checks, block plans and the
// choice of a product's kernel) under AddressSanitizer and
// UndefinedBehaviorSanitizer.  Built with g++ from csrc/plan.cpp,
// csrc/block_args.cpp and this file only: no HIP call, no GPU.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>
#include <random>
#include <vector>

#include "../../parameter_layout_collectives_amd/csrc/block.h"

namespace tide {
void release_device_states(const tide_plan *) {}
}  // namespace tide

namespace {

int failures = 0;

void expect(bool ok, const char *what, int line) {
    if (!ok) {
        std::fprintf(stderr, "FAILED at line %d: %s (last error: %s)\n", line, what,
                     tide_last_error());
        failures++;
    }
}
#define EXPECT(c) expect((c), #c, __LINE__)

constexpr uint32_t kBf16 = TIDE_F_OUT_BF16, kShort = TIDE_F_OUT_BF16 | TIDE_F_SHORT_SUMS;

void workspace_refusals() {
    const int64_t most = std::numeric_limits<int64_t>::max();
    for (int32_t op = 0; op <= 3; op++) {
        for (int64_t big : {int64_t(1) << 31, int64_t(1) << 40, int64_t(1) << 62, most}) {
            EXPECT(tide_block_workspace(op, big, 64, 64, kBf16) == -1);
            EXPECT(tide_block_workspace(op, 64, big, 64, kBf16) == -1);
            EXPECT(tide_block_workspace(op, 64, 64, big, kBf16) == -1);
            EXPECT(tide_block_workspace(op, big, big, big, kBf16) == -1);
        }
        EXPECT(tide_block_workspace(op, 64, (1 << 22) + 1, 64, kBf16) == -1);
        EXPECT(tide_block_workspace(op, 64, 64, 1 << 23, kBf16) == -1);
        EXPECT(tide_block_workspace(op, int64_t(3) << 29, 8, 1, kBf16) >= 0);
        EXPECT((tide_block_workspace(op, 1, 1 << 22, 1 << 22, kBf16) == -1) == (op == 2));
        // more lanes than a launch counts
        EXPECT(tide_block_workspace(op, (int64_t(1) << 31) - 1, 1 << 22, 1 << 22, kBf16) == -1);
        EXPECT(tide_block_workspace(op, 64, -1, 64, kBf16) == -1);
        EXPECT(tide_block_workspace(op, 64, 64, 64, 0x80000000u) == -1);
        EXPECT((tide_block_workspace(op, 64, 64, 64, kBf16 | TIDE_F_ACCUMULATE) == -1) == (op != 2));
        EXPECT((tide_block_workspace(op, 64, 64, 64, kShort) == -1) == (op == 1 || op == 2));
        EXPECT((tide_block_workspace(op, 64, 64, 64, TIDE_F_GRAD_F32) == -1) == (op != 3));
    }
    EXPECT(tide_block_workspace(-1, 1, 1, 1, 0) == -1 && tide_block_workspace(4, 1, 1, 1, 0) == -1);
    for (int64_t c : {int64_t(-1), int64_t(1) << 31, most})
        EXPECT(tide_block_cols(c) == -1 && tide_block_scale_cols(c) == -1);
    EXPECT(tide_block_cols((int64_t(1) << 31) - 1) == int64_t(1) << 31);
}

// A cut product's pieces cover its sum once, and the workspace holds them.
void choice(int op, int64_t M, int64_t N, int64_t K, uint32_t flags) {
    const int64_t asked = tide_block_workspace(op, M, N, K, flags);
    EXPECT(asked >= 0);
    for (bool aligned : {false, true})
        for (bool split : {false, true}) {
            const tide::MmChoice c =
                tide::mm_choose(static_cast<tide::MmOp>(op), M, N, K, flags, aligned, split);
            const int64_t rows = op == 2 ? N : M, cols = op == 0 ? N : K;
            const int64_t sum = op == 0 ? K : op == 1 ? N : M;
            const int64_t step = c.kernel == tide::kMmEight ? 128 : 64;
            const int64_t steps = (sum + step - 1) / step;
            const int64_t tiles = ((rows + c.tile - 1) / c.tile) * ((cols + c.tile - 1) / c.tile);
            EXPECT(c.tile == 64 || c.tile == 128 || (c.tile == 256 && aligned));
            EXPECT(c.kernel != tide::kMmEight || (op == 0 && c.tile != 64 && flags == kShort));
            EXPECT(c.kernel != tide::kMmSkinny || (op == 0 && M <= 64 && c.workspace == 0));
            EXPECT(c.direct >= 0 && c.direct <= tiles && c.splits >= 1);
            EXPECT(c.workspace <= asked);
            if (c.kernel == tide::kMmSkinny) continue;
            if (c.workspace == 0) {
                EXPECT(c.direct == tiles && c.splits == 1 && c.chunk >= steps);
                continue;
            }
            EXPECT(split && c.splits >= 2 && c.splits <= tide::kMaxSplits && c.chunk % 4 == 0);
            EXPECT((c.splits - 1) * c.chunk < steps && steps <= c.splits * c.chunk);
            EXPECT(c.workspace == (tiles - c.direct) * c.splits * c.tile * c.tile * 4);
        }
}

void choices(std::mt19937_64 &g) {
    auto size = [&](int bits) {
        const int64_t top = int64_t(1) << (g() % (bits + 1));
        return static_cast<int64_t>(g() % (top + 1));
    };
    for (int t = 0; t < 20000; t++) {
        const int64_t M = size(t % 3 ? 15 : 30), N = size(t % 3 ? 15 : 22), K = size(t % 3 ? 15 : 22);
        // twice as many lanes as a launch counts and more, or an eighth as many and less
        const double most = std::max({1.0 * M * N, 1.0 * M * K, 1.0 * N * K});
        if (most > std::ldexp(1.0, 36)) {
            if (1.0 * M * N > std::ldexp(1.0, 40)) {
                EXPECT(tide_block_workspace(0, M, N, K, kBf16) == -1);
                EXPECT(tide_block_workspace(3, M, N, K, kBf16) == -1);
            }
            continue;
        }
        for (int op = 0; op < 3; op++) choice(op, M, N, K, g() % 2 ? kBf16 : 0);
        choice(0, M, N, K, kShort);
        for (uint32_t f : {uint32_t(0), kBf16, kShort, kBf16 | TIDE_F_GRAD_F16}) {
            const tide::LinearChoice c = tide::linear_choose(M, K);
            const int64_t asked = tide_block_workspace(3, M, N, K, f);
            if (c.in_one || N == 0) {
                EXPECT(asked == 0);
                continue;
            }
            EXPECT(c.scales % 256 == 0 && c.scales >= M * tide::block_cols(K));
            EXPECT(c.blocks % 256 == 0 && c.blocks - c.scales >= M * tide::block_scale_cols(K));
            EXPECT(asked == c.blocks + tide_block_workspace(0, M, N, K, f & kShort));
        }
    }
}

// The kernel variants that the GPU tests' shapes are there for.
void variants() {
    struct Row {
        int op;
        int64_t M, N, K;
        uint32_t flags;
        bool aligned;
        tide::MmKernel kernel;
        int tile;
        bool cut;
    };
    const Row rows[] = {
        {0, 16, 200, 700, kBf16, true, tide::kMmSkinny, 64, false},
        {0, 24, 8192, 4099, kBf16, true, tide::kMmSkinny, 128, false},
        {0, 25, 8192, 4099, kBf16, true, tide::kMmWide, 64, true},
        {0, 64, 300, 520, kBf16, true, tide::kMmSkinny, 64, false},
        {0, 65, 72, 2048, kBf16, true, tide::kMmWide, 64, true},
        {0, 1500, 1510, 2060, kBf16, true, tide::kMmWide, 128, true},
        {0, 1500, 1510, 460, 0, true, tide::kMmWide, 128, true},
        {0, 1500, 1510, 440, 0, true, tide::kMmWide, 128, false},
        {0, 4000, 4104, 1100, kBf16, true, tide::kMmWide, 256, false},
        {0, 4400, 4200, 4250, kBf16, true, tide::kMmWide, 256, true},
        {0, 40, 5000, 4099, kShort, true, tide::kMmEight, 128, true},
        {0, 4000, 4104, 1100, kShort, true, tide::kMmEight, 256, false},
        {1, 130, 200, 392, kBf16, true, tide::kMmWide, 64, false},
        {1, 131, 201, 392, kBf16, false, tide::kMmWide, 64, false},
        {1, 2050, 2049, 2060, kBf16, false, tide::kMmWide, 128, false},
        {1, 2050, 2056, 2060, kBf16, true, tide::kMmWide, 128, false},
        {1, 4100, 1101, 4000, kBf16, false, tide::kMmWide, 128, false},
        {1, 4100, 1104, 4000, kBf16, true, tide::kMmWide, 256, false},
        {1, 4200, 2200, 4400, kBf16, true, tide::kMmWide, 256, true},
        {2, 2050, 2049, 2060, kBf16, false, tide::kMmWide, 128, false},
        {2, 2050, 2056, 2060, kBf16, true, tide::kMmWide, 128, false},
        {2, 1101, 4100, 4000, kBf16, true, tide::kMmWide, 256, false},
        {2, 2200, 4200, 4400, kBf16, true, tide::kMmWide, 256, true},
    };
    for (const Row &r : rows) {
        const tide::MmChoice c = tide::mm_choose(static_cast<tide::MmOp>(r.op), r.M, r.N, r.K,
                                                 r.flags, r.aligned, true);
        const bool ok = c.kernel == r.kernel && (c.kernel == tide::kMmSkinny || c.tile == r.tile) &&
                        (c.workspace > 0) == r.cut;
        if (!ok)
            std::fprintf(stderr, "op %d m %lld n %lld k %lld: kernel %d tile %d splits %d\n", r.op,
                         static_cast<long long>(r.M), static_cast<long long>(r.N),
                         static_cast<long long>(r.K), c.kernel, c.tile, c.splits);
        EXPECT(ok);
    }
}

void block_plans(std::mt19937_64 &g) {
    for (int t = 0; t < 500; t++) {
        const int32_t N = 1 + static_cast<int32_t>(g() % 40), P = 1 + static_cast<int32_t>(g() % 10);
        std::vector<int64_t> d0(P), in(P);
        for (int32_t i = 0; i < P; i++) {
            d0[i] = g() % 9 == 0 ? 0 : static_cast<int64_t>(g() % 200);
            in[i] = g() % 9 == 0 ? 0 : static_cast<int64_t>(g() % 1500);
        }
        tide_plan *p = nullptr, *b = nullptr;
        EXPECT(tide_plan_create(N, P, d0.data(), in.data(), 1, &p) == TIDE_OK);
        if (!p) continue;
        std::vector<int32_t> pick;
        for (int32_t i = 0; i < P; i++)
            if (g() % 2) pick.push_back(i);
        if (pick.empty()) pick.push_back(0);
        const int32_t n = static_cast<int32_t>(pick.size());
        EXPECT(tide_plan_create_blocks(p, n, pick.data(), &b) == TIDE_OK);
        if (b) {
            const void *far = reinterpret_cast<const void *>(uintptr_t(0x7f0000000000ull));
            const int64_t words = tide_plan_shard_numel(b);
            EXPECT(words % 4 == 0 && tide_plan_nparams(b) == 2 * n);
            const tide_status s = tide::check_block_shard(
                b, 0, far, reinterpret_cast<const void *>(uintptr_t(0x7f1000000000ull)), 0);
            EXPECT(s == TIDE_OK);
            EXPECT(tide::check_block_shard(b, N, far, far, 0) == TIDE_E_INVALID);
            std::vector<void *> out(n);
            for (int32_t j = 0; j < n; j++)
                out[j] = reinterpret_cast<void *>(uintptr_t(0x7f2000000000ull) + (uintptr_t(j) << 24));
            EXPECT(tide::check_block_unshard(b, far, out.data(), kBf16) == TIDE_OK);
        }
        tide_plan_destroy(p);                       // the block plan does not refer to it
        if (b) EXPECT(tide_plan_world(b) == N);
        tide_plan_destroy(b);
    }
}

}  // namespace

int main() {
    std::mt19937_64 g(7);
    workspace_refusals();
    choices(g);
    variants();
    block_plans(g);
    if (failures) return 1;
    std::puts("block checks passed");
    return 0;
}
