// Host side of tide_ortho: argument checks and the workspace's layout.  Makes no
// HIP call.
#include <algorithm>
#include <cmath>
#include <new>

#include "checks.h"
#include "ortho.h"

namespace tide {
namespace {

constexpr int64_t kMaxSide = int64_t(1) << 15;   // of the smaller side
constexpr int64_t kMaxNumel = int64_t(1) << 33;  // 2^22 workgroups of the first pass

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

}  // namespace

tide_status ortho_plan(const char *name, int32_t n, const int64_t *rows, const int64_t *cols,
                       OrthoPlan *plan) {
    if (n < 0) return bad(name, "n < 0");
    if (n > 1 << 20) return fail(TIDE_E_UNSUPPORTED, std::string(name) + ": more than 2^20 matrices");
    if (n > 0 && (!rows || !cols)) return bad(name, "rows or cols is NULL");
    for (int32_t i = 0; i < n; i++) {
        const tide_status st = check_dims(name, rows[i], cols[i]);
        if (st != TIDE_OK) return st;
        if (std::max(rows[i], cols[i]) > kMaxLine || std::min(rows[i], cols[i]) > kMaxSide)
            return fail(TIDE_E_UNSUPPORTED,
                        std::string(name) + ": a side above 2^22, or both above 2^15");
        if (rows[i] * cols[i] > kMaxNumel)
            return fail(TIDE_E_UNSUPPORTED, std::string(name) + ": more than 2^33 elements");
    }
    try {
        plan->order.reserve(n);
        for (int32_t i = 0; i < n; i++)
            if (rows[i] && cols[i]) plan->order.push_back(i);
        std::stable_sort(plan->order.begin(), plan->order.end(), [&](int32_t a, int32_t b) {
            return rows[a] != rows[b] ? rows[a] < rows[b] : cols[a] < cols[b];
        });
        const int64_t live = static_cast<int64_t>(plan->order.size());
        plan->sums = up(live * 16, 256);
        plan->scales = up(plan->sums + live * kOrthoParts * 8, 256);
        plan->bytes = up(plan->scales + live * 8, 256);
        for (int64_t i = 0; i < live; i++) {
            const uint32_t nr = static_cast<uint32_t>(rows[plan->order[i]]);
            const uint32_t nc = static_cast<uint32_t>(cols[plan->order[i]]);
            if (plan->groups.empty() || plan->groups.back().nr != nr || plan->groups.back().nc != nc) {
                OrthoGroup g = {};
                g.nr = nr;
                g.nc = nc;
                g.nrp = static_cast<uint32_t>(up(nr, 64));
                g.ncp = static_cast<uint32_t>(up(nc, 64));
                g.first = static_cast<uint32_t>(i);
                const int64_t pieces = g.small() ? up(std::max(nr, nc), kOrthoSmallCols) / kOrthoSmallCols
                                                 : up(static_cast<int64_t>(nr) * nc, kOrthoPiece) / kOrthoPiece;
                g.parts = static_cast<uint32_t>(std::min<int64_t>(pieces, kOrthoParts));
                g.base = plan->bytes;
                g.stride = up(g.bytes(), 256);
                plan->groups.push_back(g);
            }
            OrthoGroup &g = plan->groups.back();
            g.count++;
            plan->bytes += g.stride;
            if (plan->bytes > int64_t(1) << 46) return bad(name, "sizes overflow");
        }
    } catch (const std::bad_alloc &) {
        return fail(TIDE_E_NOMEM, std::string(name) + ": out of host memory");
    }
    return TIDE_OK;
}

tide_status check_ortho(const OrthoArgs &a, OrthoPlan *plan) {
    const char *name = "tide_ortho";
    tide_status st = check_flags(name, a.flags, TIDE_F_GRAD_F16 | TIDE_F_GRAD_F32);
    if (st == TIDE_OK) st = ortho_plan(name, a.n, a.rows, a.cols, plan);
    if (st != TIDE_OK) return st;
    if (a.steps < 1 || a.steps > 64) return bad(name, "steps outside [1, 64]");
    if (!a.coefficients) return bad(name, "coefficients is NULL");
    for (int32_t i = 0; i < 3 * a.steps; i++)
        if (!std::isfinite(a.coefficients[i])) return bad(name, "a coefficient is not finite");
    if (plan->order.empty()) return TIDE_OK;
    if (!a.src) return bad(name, "src is NULL");
    if (!a.out) return bad(name, "out is NULL");
    if (!a.workspace) return bad(name, "workspace is NULL");
    if (misaligned(a.workspace, 256)) return bad(name, "workspace is not 256-byte aligned");
    if (a.workspace_bytes < plan->bytes)
        return fail(TIDE_E_INVALID, std::string(name) + ": the workspace holds " +
                                        std::to_string(a.workspace_bytes) + " bytes of " +
                                        std::to_string(plan->bytes));
    const int es = elem_size(in_type(a.flags));
    const Bytes wsp = bytes_of(a.workspace, plan->bytes);
    std::vector<Bytes> dst;
    try {
        dst.reserve(plan->order.size());
        for (const int32_t i : plan->order) {
            const std::string s = "src[" + std::to_string(i) + "]", o = "out[" + std::to_string(i) + "]";
            const int64_t numel = a.rows[i] * a.cols[i];
            if (!a.src[i]) return bad(name, (s + " is NULL").c_str());
            if (!a.out[i]) return bad(name, (o + " is NULL").c_str());
            if (misaligned(a.src[i], es))
                return bad(name, (s + " is not aligned to its element size").c_str());
            if (misaligned(a.out[i], 2))
                return bad(name, (o + " is not aligned to its element size").c_str());
            if (overlap(bytes_of(a.src[i], numel * es), wsp))
                return bad(name, (s + " overlaps the workspace").c_str());
            dst.push_back(bytes_of(a.out[i], numel * 2));
            if (overlap(dst.back(), wsp)) return bad(name, (o + " overlaps the workspace").c_str());
        }
    } catch (const std::bad_alloc &) {
        return fail(TIDE_E_NOMEM, std::string(name) + ": out of host memory");
    }
    std::sort(dst.begin(), dst.end(), [](const Bytes &x, const Bytes &y) { return x.lo < y.lo; });
    for (size_t k = 1; k < dst.size(); k++)
        if (overlap(dst[k - 1], dst[k])) return bad(name, "an out overlaps another");
    return TIDE_OK;
}

}  // namespace tide

extern "C" int64_t tide_ortho_workspace(int32_t n, const int64_t *rows, const int64_t *cols) {
    tide::OrthoPlan plan;
    if (tide::ortho_plan("tide_ortho_workspace", n, rows, cols, &plan) != TIDE_OK) return -1;
    return plan.order.empty() ? 0 : plan.bytes;
}
