// The host code of the 4-bit blocks and of the orthogonalised updates (argument
// checks, the choice of a product's kernel, a workspace's layout) under
// AddressSanitizer and UndefinedBehaviorSanitizer.  Built with g++ from csrc/plan.cpp,
// block_args.cpp, fp4_args.cpp, ortho_args.cpp and this file only: no HIP call, no GPU.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>
#include <random>
#include <vector>

#include "../../parameter_layout_collectives_amd/csrc/fp4.h"
#include "../../parameter_layout_collectives_amd/csrc/ortho.h"

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

constexpr uint32_t kBf16 = TIDE_F_OUT_BF16, kQuant = TIDE_F_OUT_BF16 | TIDE_F_QUANT_X;

void workspace_refusals() {
    const int64_t most = std::numeric_limits<int64_t>::max();
    for (int32_t op = 0; op <= 2; op++) {
        for (int64_t big : {int64_t(1) << 31, int64_t(1) << 40, int64_t(1) << 62, most}) {
            EXPECT(tide_mx_workspace(op, big, 64, 64, kBf16) == -1);
            EXPECT(tide_mx_workspace(op, 64, big, 64, kBf16) == -1);
            EXPECT(tide_mx_workspace(op, 64, 64, big, kBf16) == -1);
            EXPECT(tide_mx_workspace(op, big, big, big, kBf16) == -1);
        }
        EXPECT(tide_mx_workspace(op, 64, (1 << 22) + 1, 64, kBf16) == -1);
        EXPECT(tide_mx_workspace(op, (int64_t(1) << 31) - 1, 1 << 22, 1 << 22, kBf16) == -1);
        EXPECT(tide_mx_workspace(op, 1, 1 << 22, 1 << 22, kBf16) >= 0);
        EXPECT(tide_mx_workspace(op, 64, 64, 64, 0x80000000u) == -1);
    }
    EXPECT(tide_mx_workspace(2, 1000, 64, 1 << 22, kQuant) >= (int64_t(1000) << 21));
}

// Whatever the sizes, a choice's pieces cover the sum once, its tiles the output,
// and what it needs of the workspace is what it was given.
void choices(std::mt19937_64 &g) {
    for (int t = 0; t < 200000; t++) {
        auto size = [&](int64_t hi) {
            return int64_t(std::exp(std::uniform_real_distribution<double>(0, std::log(double(hi)))(g)));
        };
        const tide::Fp4Op op = static_cast<tide::Fp4Op>(g() % 3);
        const int64_t M = size(20000), N = size(1 << 22), K = size(1 << 22);
        const uint32_t flags = op == tide::kFp4Linear && g() % 2 ? kQuant : kBf16;
        const int64_t all = tide_mx_workspace(op, M, N, K, flags);
        EXPECT(all >= 0);
        const int64_t given = g() % 3 == 0 ? 0 : g() % 2 ? all : std::max<int64_t>(0, size(1 << 30) - 1);
        const tide::Fp4Choice c = tide::fp4_choose(op, M, N, K, flags, g() % 2 == 0, given);
        if (c.kernel == tide::kFp4SkinnyInOne) {
            EXPECT(M <= 16 && M * (tide::block_cols(K) * 2 + 16) <= 57360 && c.x == 0);
            continue;
        }
        if (c.kernel == tide::kFp4Skinny) {
            EXPECT(c.x <= given && c.x >= M * tide::block_cols(K) * 2);
            continue;
        }
        if (c.kernel == tide::kFp4Strips) {
            EXPECT(M <= 64 && c.x <= given && c.x >= M * tide::block_cols(K) * 2);
            const int64_t units = tide::block_count(K);
            EXPECT(c.mm.chunk * c.mm.splits >= units && c.mm.chunk * (c.mm.splits - 1) < units);
            EXPECT(c.mm.workspace == (c.mm.splits > 1 ? c.mm.splits * M * N * 4 : 0));
            EXPECT(c.x + c.mm.workspace <= given);
            continue;
        }
        const int64_t sum = op == tide::kFp4Dx ? N : K, cols = op == tide::kFp4Dx ? K : N;
        const int64_t step = c.kernel == tide::kFp4Tiles ? 128 : 64, steps = (sum + step - 1) / step;
        const int64_t T = c.mm.tile, tiles = ((M + T - 1) / T) * ((cols + T - 1) / T);
        EXPECT(c.mm.direct >= 0 && c.mm.direct <= tiles && c.mm.splits >= 1);
        EXPECT(c.mm.chunk * c.mm.splits >= steps && c.mm.chunk * (c.mm.splits - 1) < steps);
        EXPECT((c.mm.splits == 1) == (c.mm.direct == tiles));
        EXPECT(c.mm.workspace == 0 || c.x + c.mm.workspace <= given);
        EXPECT(c.mm.workspace >= (tiles - c.mm.direct) * (c.mm.splits > 1 ? c.mm.splits : 0) * T * T * 4);
    }
}

// Matrices lie apart in the workspace, in groups of equal ones that name each once.
void ortho_layouts(std::mt19937_64 &g) {
    for (int t = 0; t < 3000; t++) {
        const int32_t n = static_cast<int32_t>(g() % 40);
        std::vector<int64_t> rows(n), cols(n);
        for (int32_t i = 0; i < n; i++) {
            rows[i] = static_cast<int64_t>(g() % (g() % 2 ? 5 : 3000));
            cols[i] = static_cast<int64_t>(g() % (g() % 2 ? 5 : 3000));
        }
        tide::OrthoPlan p;
        EXPECT(tide::ortho_plan("t", n, rows.data(), cols.data(), &p) == TIDE_OK);
        std::vector<int> seen(n, 0);
        for (int32_t i : p.order) seen[i]++;
        for (int32_t i = 0; i < n; i++) EXPECT(seen[i] == (rows[i] && cols[i] ? 1 : 0));
        int64_t end = p.scales + static_cast<int64_t>(p.order.size()) * 8;
        EXPECT(p.sums >= static_cast<int64_t>(p.order.size()) * 16);
        EXPECT(p.scales >= p.sums + static_cast<int64_t>(p.order.size()) * tide::kOrthoParts * 8);
        uint32_t at = 0;
        for (const tide::OrthoGroup &q : p.groups) {
            EXPECT(q.first == at && q.count > 0 && q.parts >= 1 && q.parts <= tide::kOrthoParts);
            EXPECT(q.base >= end && q.base % 256 == 0 && q.stride >= q.bytes());
            EXPECT(q.nrp % 64 == 0 && q.nrp >= q.nr && q.ncp % 64 == 0 && q.ncp >= q.nc);
            EXPECT(q.p_at() % 16 == 0 && q.a_diag() % 16 == 0 && q.p_diag() % 16 == 0);
            for (uint32_t k = 0; k < q.count; k++) {
                EXPECT(rows[p.order[at + k]] == q.nr && cols[p.order[at + k]] == q.nc);
            }
            at += q.count;
            end = q.base + q.count * q.stride;
        }
        EXPECT(at == p.order.size() && (p.order.empty() || end == p.bytes));
    }
    const int64_t most = std::numeric_limits<int64_t>::max(), one = 1;
    EXPECT(tide_ortho_workspace(1, &most, &one) == -1 && tide_ortho_workspace(1, &one, &most) == -1);
    EXPECT(tide_ortho_workspace(-1, &one, &one) == -1 && tide_ortho_workspace(1, nullptr, &one) == -1);
    std::vector<int64_t> big(1 << 14, 1 << 15);          // 2^14 matrices of 2^30 elements
    EXPECT(tide_ortho_workspace(1 << 14, big.data(), big.data()) == -1);
}

}  // namespace

int main() {
    std::mt19937_64 g(11);
    workspace_refusals();
    choices(g);
    ortho_layouts(g);
    if (failures) return 1;
    std::puts("fp4 checks passed");
    return 0;
}
