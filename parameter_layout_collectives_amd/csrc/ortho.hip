// tide_ortho: gradient matrices orthogonalised by Newton-Schulz products.
//
// From X = G / ||G||_F, with r the smaller side and X written as [r, c] (a tall
// matrix is its transpose throughout; nothing is transposed in memory):
//   A = X X^T,  P = a I + b A + c A^2,  X <- P X
// A step is three products.  A and P are symmetric: tiles on and below their
// diagonals are computed and stored to both sides, so a step takes
// r^2 c + r^3 + 2 r^2 c multiplications and additions.
//
// Precision.  The matrix instruction takes fp16 factors and adds in fp32.  Held in
// one fp16 (or bf16) number, X would lose what a few heavy directions leave of the
// light ones, which the steps then raise by up to 3.4^5: with few singular values
// far above the others the result is off by 3e-3 to 2e-2 of its norm (bf16: 2e-2 to
// 2e-1).  What raises a light direction is P's diagonal, though (A is small there),
// so A and P are split into diagonal and rest, A = D + O, P = Q + R:
//   R_ij = b O_ij + c ((d_i + d_j) O_ij + (O^2)_ij),  i != j
//   q_i  = a + b d_i + c (d_i^2 + (O^2)_ii)
//   X    <- R X + Q X
// D, Q and all of these sums are fp32, X is two fp16 numbers hi + lo (22 bits) in
// Q X, and only O, R and, in X X^T and R X, hi are rounded to fp16.  So the products
// run at fp16's full rate and the result is off by 3e-4 to 1e-3 of its norm before
// it is rounded to bf16 (1.7e-3), by up to 1.6e-3 for matrices whose rank is an
// eighth of r (an emulation in 64 bits).  With fewer rows R outweighs Q there (37 of
// rank 4: 4e-3), so up to kOrthoBoth of them R X takes lo as well, as one sum of
// twice the length.
// Powers of two keep the numbers in fp16's range: X by 2^ex, about sqrt(r c), O by
// 2^12, R by 2^10.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "block.h"
#include "block_device.h"
#include "mm_device.h"
#include "ortho.h"

namespace tide {
namespace {

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float kScaleA = 4096.0f, kScaleP = 1024.0f;

struct Groups {
    OrthoGroup g[kOrthoGroups];
    int n;
};
static_assert(sizeof(OrthoGroup) == 48 && sizeof(Groups) <= 2400, "groups exceed the kernel arguments");

// The group that workgroup `wg` works on: the last one with wg0 <= wg.
__device__ __forceinline__ OrthoGroup group_of(const Groups &a, uint32_t wg) {
    int k = 0;
    for (int i = 1; i < a.n; i++)
        if (a.g[i].wg0 <= wg) k = i;
    return a.g[k];
}

struct Pointers {
    uint64_t src, out;
};
constexpr int kPointersPerLaunch = 200;
struct PointerArgs {
    Pointers p[kPointersPerLaunch];
};
__global__ __launch_bounds__(256) void pointers_kernel(PointerArgs a, int n, Pointers *__restrict__ to) {
    if (static_cast<int>(threadIdx.x) < n) to[threadIdx.x] = a.p[threadIdx.x];
}

// The workspace's parts.
struct Space {
    char *base;
    const Pointers *pointers;
    double *sums;
    float2 *scales;
};

// ------------------------------------------------------- ||G||_F and X's first pair

// The sum of v over a workgroup of 256, in every lane: a fixed order.
__device__ __forceinline__ double sum256(double v, double *part) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = v;
    __syncthreads();
    return (part[0] + part[1]) + (part[2] + part[3]);
}

// Squares are added in fp64, where those of all fp32 numbers lie in range.
template <int ET>
__global__ __launch_bounds__(256) void squares_kernel(Groups a, Space s) {
    constexpr int ES = ET == kElemF32 ? 4 : 2;
    __shared__ double part[4];
    const OrthoGroup g = group_of(a, blockIdx.x);
    const uint32_t in = blockIdx.x - g.wg0, m = in / g.parts, q = in % g.parts;
    const char *src = reinterpret_cast<const char *>(s.pointers[g.first + m].src);
    const int64_t numel = static_cast<int64_t>(g.nr) * g.nc;
    const int64_t chunk = ((numel + g.parts - 1) / g.parts + 7) / 8 * 8;
    const int64_t lo = q * chunk, hi = min(lo + chunk, numel);
    double v = 0;
    for (int64_t i = lo + threadIdx.x * 8; i < hi; i += 2048) {
        float x[8];
        load8<ET>(src + i * ES, static_cast<int>(min(hi - i, static_cast<int64_t>(8))), false, x);
#pragma unroll
        for (int k = 0; k < 8; k++) v += static_cast<double>(x[k]) * x[k];
    }
    v = sum256(v, part);
    if (threadIdx.x == 0) s.sums[static_cast<int64_t>(g.first + m) * kOrthoParts + q] = v;
}

// 2^ex: X's scale.  About sqrt(r c), which brings the first X's elements near 1.
__host__ __device__ inline int x_exponent(uint32_t nr, uint32_t nc) {
    int e = 0;
    for (uint64_t n = static_cast<uint64_t>(nr) * nc; n >= 4; n >>= 2) e++;
    return min(e, 14);
}

// With ||G||_F = m 2^k, 0.5 <= m < 1: X = (G 2^-k) / m.  The power of two is exact
// and applied here; 1 / m multiplies the first step's products.  16 rows x 128
// columns of the padded matrix per workgroup, 8 elements per lane.
template <int ET>
__global__ __launch_bounds__(256) void first_kernel(Groups a, Space s) {
    constexpr int ES = ET == kElemF32 ? 4 : 2;
    __shared__ double part[4];
    const OrthoGroup g = group_of(a, blockIdx.x);
    const uint32_t tc = (g.ncp + 127) / 128, per = tc * (g.nrp / 16);
    const uint32_t in = blockIdx.x - g.wg0, m = in / per, at = in % per;
    const uint32_t row = at / tc * 16 + threadIdx.x / 16, col = at % tc * 128 + threadIdx.x % 16 * 8;
    const uint32_t id = g.first + m;
    const char *src = reinterpret_cast<const char *>(s.pointers[id].src);
    float x[8];
    const int n = row < g.nr && col < g.nc ? static_cast<int>(min(g.nc - col, 8u)) : 0;
    load8<ET>(src + (static_cast<int64_t>(row) * g.nc + col) * ES, n, false, x);
    const double norm = sqrt(sum256(threadIdx.x < g.parts ? s.sums[static_cast<int64_t>(id) * kOrthoParts + threadIdx.x] : 0.0, part));
    const int ex = x_exponent(g.nr, g.nc);
    int k = 0;
    double frac = 1.0;
    if (norm > 0 && norm < __builtin_inf()) frac = frexp(norm, &k);
    // an infinity or a NaN in G makes all of X NaN
    const float bad = norm < __builtin_inf() ? 0.0f : __builtin_nanf("");
    if (at == 0 && threadIdx.x == 0) {
        const float t = static_cast<float>(1.0 / frac);
        s.scales[id] = make_float2(t, static_cast<float>(1.0 / (frac * frac)));
    }
    if (col >= g.ncp) return;
    f16x8 h, l;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float v = ldexpf(x[i], ex - k) + bad;
        h[i] = static_cast<_Float16>(v);
        l[i] = static_cast<_Float16>(v - static_cast<float>(h[i]));
    }
    _Float16 *X = reinterpret_cast<_Float16 *>(s.base + g.base + m * g.stride) + row * g.pitch() + col;
    *reinterpret_cast<f16x8 *>(X) = h;
    *reinterpret_cast<f16x8 *>(X + g.lo()) = l;
}

// ------------------------------------------------------- the products

// out[i, j] = sum over c of I(i, c) J(c, j) for fp16 factors that lie in memory
// padded and aligned, so that both go straight into LDS; the layouts and
// fragments of the bf16 products' stages (which move bits).  Two buffers: the step
// after next is asked for once the barrier has freed a buffer, so its loads have a
// whole step to arrive; the next step's first fragments are read under this step's
// last multiplications.
template <Mode MI, Mode MJ, int T, int WI, int WJ>
struct Half {
    static constexpr int NT = WI * WJ * 64;
    static constexpr int FI = T / WI / 16, FJ = T / WJ / 16;
    static constexpr int LINES = 2 * FI, RING = FI >= 4 ? 4 : 2, D = RING - 1;
    static constexpr int TILE = T * 128;
    typedef Stage<MI, T, NT, true> SI;
    typedef Stage<MJ, T, NT, true> SJ;
    static_assert(SI::DIRECT && SJ::DIRECT, "factors go straight into LDS");
    static_assert(LINES % RING == 0 && D <= FI,
                  "a step starts at ring entry 0, and its first half is over when the next "
                  "step's J fragments replace it");

    SI si;
    SJ sj;
    int lane, wave, wi, wj;
    f32x4 acc[FI][FJ];

    __device__ __forceinline__ void fetch(LDS_AS char *ti, LDS_AS char *tj) {
        si.fetch(ti, wave);
        sj.fetch(tj, wave);
    }
    __device__ __forceinline__ f16x8 line(const LDS_AS char *b, int n) const {
        return __builtin_bit_cast(f16x8, SI::frag(b, wi * (T / WI) + n % FI * 16, n / FI, lane));
    }
    __device__ __forceinline__ void rows(f16x8 *r, const LDS_AS char *b, int kk) const {
#pragma unroll
        for (int y = 0; y < FJ; y++)
            r[y] = __builtin_bit_cast(f16x8, SJ::frag(b, wj * (T / WJ) + y * 16, kk, lane));
    }
    template <bool LAST>
    __device__ __forceinline__ void step(f16x8 *l, f16x8 (*r)[FJ], LDS_AS char *here_i,
                                         LDS_AS char *here_j, LDS_AS char *there_i,
                                         LDS_AS char *there_j) {
        rows(r[1], here_j, 1);
#pragma unroll
        for (int n = 0; n < LINES; n++) {
            if (n + D < LINES) l[(n + D) % RING] = line(here_i, n + D);
            if (!LAST && n + D == LINES) {
                landed();
                fetch(here_i, here_j);
                rows(r[0], there_j, 0);
            }
            if (!LAST && n + D >= LINES) l[(n + D) % RING] = line(there_i, n + D - LINES);
#pragma unroll
            for (int y = 0; y < FJ; y++)
                acc[n % FI][y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    r[n / FI][y], l[n % RING], acc[n % FI][y], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    __device__ __forceinline__ void run(LDS_AS char *__restrict__ i0, LDS_AS char *__restrict__ i1,
                                        LDS_AS char *__restrict__ j0, LDS_AS char *__restrict__ j1,
                                        uint32_t steps) {
        fetch(i0, j0);
        fetch(i1, j1);
        landed();
        f16x8 l[RING], r[2][FJ];
        rows(r[0], j0, 0);
#pragma unroll
        for (int n = 0; n < D; n++) l[n] = line(i0, n);
        // Past the last step zeros are fetched, or values that nothing uses,
        // which keeps branches out of the loop.
        for (; steps > 1; steps -= 2) {
            step<false>(l, r, i0, j0, i1, j1);
            step<false>(l, r, i1, j1, i0, j0);
        }
        if (steps) step<true>(l, r, i0, j0, i1, j1);
        landed();                // no load may still be on its way to LDS at the end
    }
};

// What one product's launch computes.
enum Stage3 { kGram, kPoly, kApply };
struct ProductArgs {
    Groups a;
    Space s;
    float ca, cb, cc;            // the step's coefficients (kPoly)
    int from;                    // which of the two X is read
    int first, last;             // of the steps
    uint32_t total;              // workgroups
};

// Tiles of a matrix's A or P: on and below the diagonal; of its X: all.
__host__ __device__ inline uint32_t tiles_of(const OrthoGroup &g, int stage, uint32_t T) {
    if (stage == kApply) return (g.nrp + T - 1) / T * ((g.ncp + T - 1) / T);
    const uint32_t n = (g.rp() + T - 1) / T;
    return n * (n + 1) / 2;
}

__device__ __forceinline__ f16x4 to_half(f32x4 v) {
    return f16x4{static_cast<_Float16>(v[0]), static_cast<_Float16>(v[1]), static_cast<_Float16>(v[2]),
                 static_cast<_Float16>(v[3])};
}

template <int STAGE, Mode MI, Mode MJ, int T, int WI, int WJ>
__device__ __forceinline__ void product_tile(const ProductArgs &p, const OrthoGroup &g, uint32_t m,
                                             uint32_t ti, uint32_t tj, LDS_AS char *lds) {
    typedef Half<MI, MJ, T, WI, WJ> K;
    const int t = threadIdx.x, lane = t & 63;
    char *const base = p.s.base + g.base + static_cast<int64_t>(m) * g.stride;
    char *const x = base + p.from * g.x_bytes();
    const int64_t rp = g.rp(), xp = g.pitch() * 2;
    const int64_t i0 = static_cast<int64_t>(ti) * T, j0 = static_cast<int64_t>(tj) * T;
    K k;
    k.wave = __builtin_amdgcn_readfirstlane(t >> 6);
    k.lane = lane;
    k.wi = k.wave / WJ;
    k.wj = k.wave % WJ;
    int64_t sum;
    if (STAGE == kGram) {
        sum = g.tall() ? g.nrp : g.ncp;
        k.si.init(x, nullptr, xp, 0, i0, rp, sum, 0, t);
        k.sj.init(x, nullptr, xp, 0, j0, rp, sum, 0, t);
    } else if (STAGE == kPoly) {
        sum = rp;
        k.si.init(base + g.a_at(), nullptr, rp * 2, 0, i0, rp, sum, 0, t);
        k.sj.init(base + g.a_at(), nullptr, rp * 2, 0, j0, rp, sum, 0, t);
    } else {
        sum = g.p_pitch();
        if (g.tall()) {
            k.si.init(x, nullptr, xp, 0, i0, g.nrp, sum, 0, t);
            k.sj.init(base + g.p_at(), nullptr, sum * 2, 0, j0, rp, sum, 0, t);
        } else {
            k.si.init(base + g.p_at(), nullptr, sum * 2, 0, i0, rp, sum, 0, t);
            k.sj.init(x, nullptr, xp, 0, j0, g.ncp, sum, 0, t);
        }
    }
#pragma unroll
    for (int a = 0; a < K::FI; a++)
#pragma unroll
        for (int b = 0; b < K::FJ; b++) k.acc[a][b] = f32x4{0, 0, 0, 0};
    k.run(lds, lds + K::TILE, lds + 2 * K::TILE, lds + 3 * K::TILE, uniform((sum + 63) / 64));

    const float2 t1 = p.first ? p.s.scales[g.first + m] : make_float2(1.0f, 1.0f);
    const int ex = x_exponent(g.nr, g.nc);
    const uint32_t li = static_cast<uint32_t>(i0) + k.wi * (T / WI) + (lane & 15);
    const uint32_t lj = static_cast<uint32_t>(j0) + k.wj * (T / WJ) + (lane >> 4) * 4;
    float *const ad = reinterpret_cast<float *>(base + g.a_diag());
    float *const pd = reinterpret_cast<float *>(base + g.p_diag());
    if (STAGE == kGram) {
        const float f = ldexpf(t1.y, -2 * ex);
        _Float16 *const o = reinterpret_cast<_Float16 *>(base + g.a_at());
#pragma unroll
        for (int a = 0; a < K::FI; a++)
#pragma unroll
            for (int b = 0; b < K::FJ; b++) {
                const uint32_t i = li + a * 16, j = lj + b * 16;
                if (i >= rp || j >= rp) continue;      // X's padding makes A's zeros
                f32x4 v = k.acc[a][b] * f;
#pragma unroll
                for (int n = 0; n < 4; n++)
                    if (i == j + n) {
                        ad[i] = v[n];
                        v[n] = 0.0f;
                    }
                const f16x4 h = to_half(v * kScaleA);
                *reinterpret_cast<f16x4 *>(o + i * rp + j) = h;
                if (ti != tj)
#pragma unroll
                    for (int n = 0; n < 4; n++) o[(j + n) * rp + i] = h[n];
            }
        return;
    }
    if (STAGE == kPoly) {
        const _Float16 *const o = reinterpret_cast<const _Float16 *>(base + g.a_at());
        _Float16 *const q = reinterpret_cast<_Float16 *>(base + g.p_at());
        const int64_t qp = g.p_pitch();
        const uint32_t r = g.r();
#pragma unroll
        for (int b = 0; b < K::FJ; b++) {
            const uint32_t j = lj + b * 16;
            if (j >= rp) continue;
            const f32x4 dj = *reinterpret_cast<const f32x4 *>(ad + j);
#pragma unroll
            for (int a = 0; a < K::FI; a++) {
                const uint32_t i = li + a * 16;
                if (i >= rp) continue;
                const float di = ad[i];
                const f16x4 old = *reinterpret_cast<const f16x4 *>(o + i * rp + j);
                f32x4 v = k.acc[a][b] * (1.0f / (kScaleA * kScaleA));
#pragma unroll
                for (int n = 0; n < 4; n++) {
                    const float oij = static_cast<float>(old[n]) / kScaleA;
                    if (i == j + n) {
                        pd[i] = i < r ? p.ca + p.cb * di + p.cc * (di * di + v[n]) : 0.0f;
                        v[n] = 0.0f;
                    } else {
                        v[n] = p.cb * oij + p.cc * ((di + dj[n]) * oij + v[n]);
                    }
                }
                const f16x4 h = to_half(v * kScaleP);
                for (int64_t c = 0; c < qp; c += rp) {
                    *reinterpret_cast<f16x4 *>(q + i * qp + c + j) = h;
                    if (ti != tj)
#pragma unroll
                        for (int n = 0; n < 4; n++) q[(j + n) * qp + c + i] = h[n];
                }
            }
        }
        return;
    }
    // R X / 2^10 + Q X, as X is held; times the first step's factor
    const _Float16 *const from = reinterpret_cast<const _Float16 *>(x);
    _Float16 *const to = reinterpret_cast<_Float16 *>(base + (1 - p.from) * g.x_bytes());
    const float f = p.last ? ldexpf(t1.x, -ex) : t1.x;
    MmLaunch out = {};
    out.out = reinterpret_cast<char *>(p.s.pointers[g.first + m].out);
    out.rows = g.nr;
    out.cols = g.nc;
    out.out_bf16 = 1;
#pragma unroll
    for (int b = 0; b < K::FJ; b++) {
        const uint32_t j = lj + b * 16;
        if (j >= g.ncp) continue;
        f32x4 qj = {0, 0, 0, 0};
        if (g.tall()) qj = *reinterpret_cast<const f32x4 *>(pd + j);
#pragma unroll
        for (int a = 0; a < K::FI; a++) {
            const uint32_t i = li + a * 16;
            if (i >= g.nrp) continue;
            const int64_t at = i * g.pitch() + j;
            const f16x4 h = *reinterpret_cast<const f16x4 *>(from + at);
            const f16x4 l = *reinterpret_cast<const f16x4 *>(from + at + g.lo());
            if (!g.tall()) {
                const float qi = pd[i];
                qj = f32x4{qi, qi, qi, qi};
            }
            f32x4 v;
#pragma unroll
            for (int n = 0; n < 4; n++)
                v[n] = (k.acc[a][b][n] * (1.0f / kScaleP) +
                        qj[n] * (static_cast<float>(h[n]) + static_cast<float>(l[n]))) * f;
            if (p.last) {
                store4(out, i, j, v);
                continue;
            }
            const f16x4 nh = to_half(v);
            f32x4 rest;
#pragma unroll
            for (int n = 0; n < 4; n++) rest[n] = v[n] - static_cast<float>(nh[n]);
            *reinterpret_cast<f16x4 *>(to + at) = nh;
            *reinterpret_cast<f16x4 *>(to + at + g.lo()) = to_half(rest);
        }
    }
}

template <int STAGE, int T, int WI, int WJ>
__global__ __launch_bounds__(WI * WJ * 64, 1) void product_kernel(ProductArgs p) {
    __shared__ __attribute__((aligned(1024))) char lds[4 * T * 128];
    LDS_AS char *const b = (LDS_AS char *)lds;
    // Workgroup IDs go to the 8 XCDs in turn and each XCD has its own L2, so every
    // XCD takes one contiguous run of tiles.
    const uint32_t q = p.total / 8, rm = p.total % 8, xcd = blockIdx.x % 8;
    const uint32_t v = xcd * q + min(xcd, rm) + blockIdx.x / 8;
    const OrthoGroup g = group_of(p.a, v);
    const uint32_t per = tiles_of(g, STAGE, T), in = v - g.wg0;
    const uint32_t m = uniform(in / per), at = uniform(in % per);
    if (STAGE == kApply) {
        // 8 tile rows advance together, as in the blocked products
        const uint32_t tr = (g.nrp + T - 1) / T, tc = (g.ncp + T - 1) / T;
        const uint32_t pg = 8 * tc, gr = at / pg, l = at - gr * pg, h = min(8u, tr - 8 * gr);
        const uint32_t ti = uniform(8 * gr + l % h), tj = uniform(l / h);
        if (g.tall())
            product_tile<STAGE, kBf16Along, kBf16Along, T, WI, WJ>(p, g, m, ti, tj, b);
        else
            product_tile<STAGE, kBf16Along, kBf16Across, T, WI, WJ>(p, g, m, ti, tj, b);
        return;
    }
    // at = ti (ti + 1) / 2 + tj, tj <= ti
    uint32_t ti = static_cast<uint32_t>((sqrtf(8.0f * at + 1.0f) - 1.0f) * 0.5f);
    while ((ti + 1) * (ti + 2) / 2 <= at) ti++;
    while (ti * (ti + 1) / 2 > at) ti--;
    ti = uniform(ti);
    const uint32_t tj = uniform(at - ti * (ti + 1) / 2);
    if (STAGE == kGram && g.tall())
        product_tile<STAGE, kBf16Across, kBf16Across, T, WI, WJ>(p, g, m, ti, tj, b);
    else
        product_tile<STAGE, kBf16Along, kBf16Along, T, WI, WJ>(p, g, m, ti, tj, b);
}

constexpr int64_t kMaxWgs = 0xffffffffll / 512;

// Calls launch(groups, workgroups) over the plan's groups, as many at a time as
// kernel arguments hold and a launch can count; wgs(g): workgroups of one matrix of
// g, which are fewer than that (ortho_plan).
template <class Wgs, class Launch>
tide_status over_groups(const OrthoPlan &plan, Wgs wgs, Launch launch) {
    size_t at = 0;
    uint32_t done = 0;           // matrices of group `at` launched before
    while (at < plan.groups.size()) {
        Groups a;
        a.n = 0;
        int64_t total = 0;
        while (at < plan.groups.size() && a.n < kOrthoGroups) {
            OrthoGroup g = plan.groups[at];
            const int64_t per = wgs(g);
            const int64_t n = std::min<int64_t>(g.count - done, (kMaxWgs - total) / per);
            if (n == 0) break;
            g.first += done;
            g.base += done * g.stride;
            g.wg0 = static_cast<uint32_t>(total);
            a.g[a.n++] = g;
            total += n * per;
            done += static_cast<uint32_t>(n);
            if (done < g.count) break;
            done = 0;
            at++;
        }
        launch(a, static_cast<uint32_t>(total));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return hip_fail("tide_ortho: kernel launch", e);
    }
    return TIDE_OK;
}

// Large tiles once they fill three quarters of the card, small ones while middle
// ones would leave half of it idle (the blocked products' rule).
int tile_for(const OrthoPlan &plan, int stage) {
    auto tiles = [&](uint32_t T) {
        int64_t n = 0;
        for (const OrthoGroup &g : plan.groups)
            n += static_cast<int64_t>(g.count) * tiles_of(g, stage, T);
        return n;
    };
    return tiles(256) >= kCus * 3 / 4 ? 256 : tiles(128) < kCus / 2 ? 64 : 128;
}

template <int STAGE>
tide_status run_product(const OrthoPlan &plan, ProductArgs p, hipStream_t s) {
    const int T = tile_for(plan, STAGE);
    return over_groups(
        plan, [&](const OrthoGroup &g) { return tiles_of(g, STAGE, static_cast<uint32_t>(T)); },
        [&](const Groups &a, uint32_t total) {
            p.a = a;
            p.total = total;
            if (T == 256)
                product_kernel<STAGE, 256, 2, 4><<<dim3(total), dim3(512), 0, s>>>(p);
            else if (T == 128)
                product_kernel<STAGE, 128, 2, 2><<<dim3(total), dim3(256), 0, s>>>(p);
            else
                product_kernel<STAGE, 64, 2, 2><<<dim3(total), dim3(256), 0, s>>>(p);
        });
}

template <int ET>
tide_status run_first(const OrthoPlan &plan, const Space &sp, hipStream_t s) {
    tide_status st = over_groups(
        plan, [](const OrthoGroup &g) { return g.parts; },
        [&](const Groups &a, uint32_t total) {
            squares_kernel<ET><<<dim3(total), dim3(256), 0, s>>>(a, sp);
        });
    if (st != TIDE_OK) return st;
    return over_groups(
        plan, [](const OrthoGroup &g) { return g.nrp / 16 * ((g.ncp + 127) / 128); },
        [&](const Groups &a, uint32_t total) {
            first_kernel<ET><<<dim3(total), dim3(256), 0, s>>>(a, sp);
        });
}

tide_status run_ortho(const OrthoArgs &a, void *stream) {
    OrthoPlan plan;
    tide_status st = check_ortho(a, &plan);
    if (st != TIDE_OK) return st;
    if (plan.order.empty()) {
        clear_error();
        return TIDE_OK;
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    Space sp;
    sp.base = static_cast<char *>(a.workspace);
    sp.pointers = reinterpret_cast<const Pointers *>(sp.base);
    sp.sums = reinterpret_cast<double *>(sp.base + plan.sums);
    sp.scales = reinterpret_cast<float2 *>(sp.base + plan.scales);
    const int n = static_cast<int>(plan.order.size());
    for (int at = 0; at < n; at += kPointersPerLaunch) {
        PointerArgs args;
        const int m = std::min(kPointersPerLaunch, n - at);
        for (int i = 0; i < m; i++) {
            const int32_t k = plan.order[at + i];
            args.p[i] = Pointers{reinterpret_cast<uintptr_t>(a.src[k]), reinterpret_cast<uintptr_t>(a.out[k])};
        }
        pointers_kernel<<<dim3(1), dim3(256), 0, s>>>(args, m, reinterpret_cast<Pointers *>(sp.base) + at);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return hip_fail("tide_ortho: kernel launch", e);
    }
    switch (in_type(a.flags)) {
        case kElemBf16: st = run_first<kElemBf16>(plan, sp, s); break;
        case kElemF16: st = run_first<kElemF16>(plan, sp, s); break;
        case kElemF32: st = run_first<kElemF32>(plan, sp, s); break;
    }
    for (int i = 0; i < a.steps && st == TIDE_OK; i++) {
        ProductArgs p;
        p.s = sp;
        p.ca = a.coefficients[3 * i];
        p.cb = a.coefficients[3 * i + 1];
        p.cc = a.coefficients[3 * i + 2];
        p.from = i % 2;
        p.first = i == 0;
        p.last = i == a.steps - 1;
        st = run_product<kGram>(plan, p, s);
        if (st == TIDE_OK) st = run_product<kPoly>(plan, p, s);
        if (st == TIDE_OK) st = run_product<kApply>(plan, p, s);
    }
    if (st == TIDE_OK) clear_error();
    return st;
}

}  // namespace
}  // namespace tide

using namespace tide;

extern "C" tide_status tide_ortho(int32_t n, const void *const *src, void *const *out,
                                  const int64_t *rows, const int64_t *cols, int32_t steps,
                                  const float *coefficients, uint32_t flags, void *workspace,
                                  int64_t workspace_bytes, void *stream) {
    return run_ortho(OrthoArgs{n, src, out, rows, cols, steps, coefficients, flags, workspace,
                               workspace_bytes},
                     stream);
}
