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
// eighth of r (an emulation in 64 bits).  Only where a matrix of rank one has entries of
// one magnitude are all rounded alike: there the result is off by up to 1e-2.
// With fewer rows R outweighs Q in matrices of a low rank (37 rows of rank 4: 4e-3), so up
// to kOrthoBoth of them R X takes lo as well, as one sum of twice the length.  What hi alone
// loses in directions where X has little is raised by a in every later step: with 5 of the
// usual ones (3.4445^5 = 485) [300, 420] of rank 37 is 1.5e-3 off, with 6 4e-3, with 8
// 5e-2; with lo 7e-4, 7e-4, 9e-4.  So above kOrthoRaisedHi lo enters for any number of
// rows, in all steps (the first alone, or all but the last five, would leave 4e-3 to 2e-2;
// [4096, 4096] 425 us a step for 270).
// Few rows average none of these roundings out (2 x 2: up to 8e-3), and cost next to
// nothing: up to kOrthoSmall of them the steps run in fp64 on A alone, since P and A
// commute: A <- P A P and M <- P M from M = I, and the result is M X, one pass over G.
// A's rounding, 1e-16 of its norm, makes eigenvalues at zero negative, which X X^T never
// is, and P A P raises them by a^2 a step until the polynomial, unbounded below zero, runs
// away with them (16 x 64 of rank 4: 1.4e-3 off at 14 steps, NaN at 30).  So before steps
// have raised them by kOrthoRaised^2 = 2^30, that is to 1e-7, where P is still a to 1e-6, X
// <- M X is formed in fp64 and A from it anew: 8 of the usual steps.
// Powers of two keep the numbers in fp16's range: X by 2^ex, about sqrt(r c), O by
// 2^12, R by 2^10.
//
// The products bound it, and where the sums are short X's traffic: P X reads X (hi for
// the product, hi and lo for its join) and writes it, 8 bytes an element and step.  Five
// steps of [4096, 4096] take 1.51 to 1.61 ms, 0.9 PFLOP/s of the multiplications above,
// of an 8B layer's seven matrices 14.1 ms, 1.05 PFLOP/s (fp16's library product 1.58),
// of 48 x [768, 2048] 1.7 ms: X X^T 85 us, P 40, P X 203 a step, at 3.7 TB/s.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <type_traits>
#include <vector>

#include "block.h"
#include "block_device.h"
#include "mm_device.h"
#include "ortho.h"

namespace tide {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

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
    int lo;                      // X's lo enters P X whatever the rows
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
    int64_t i = lo + threadIdx.x * 8;
    // four loads in flight: [4096, 4096] 11 us, one at a time 17 to 22
    for (; i + 3 * 2048 + 8 <= hi; i += 4 * 2048) {
        float x[4][8];
#pragma unroll
        for (int u = 0; u < 4; u++) load8<ET>(src + (i + u * 2048) * ES, 8, false, x[u]);
#pragma unroll
        for (int u = 0; u < 4; u++)
#pragma unroll
            for (int k = 0; k < 8; k++) v += static_cast<double>(x[u][k]) * x[u][k];
    }
    for (; i < hi; i += 2048) {
        float x[8];
        load8<ET>(src + i * ES, static_cast<int>(min(hi - i, static_cast<int64_t>(8))), false, x);
#pragma unroll
        for (int k = 0; k < 8; k++) v += static_cast<double>(x[k]) * x[k];
    }
    v = sum256(v, part);
    if (threadIdx.x == 0) s.sums[static_cast<int64_t>(g.first + m) * kOrthoParts + q] = v;
}

// Where (row, col) of a matrix of `rows` rows in panels lies, in elements.
__device__ __forceinline__ int64_t panel_at(uint32_t rows, uint32_t row, uint32_t col) {
    return ((static_cast<int64_t>(col >> 5) * rows + row) << 5) + (col & 31);
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
    const double *const sums = s.sums + static_cast<int64_t>(id) * kOrthoParts;
    const double norm = sqrt(sum256(threadIdx.x < g.parts ? sums[threadIdx.x] : 0.0, part));
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
    _Float16 *X = reinterpret_cast<_Float16 *>(s.base + g.base + m * g.stride) + panel_at(g.nrp, row, col);
    *reinterpret_cast<f16x8 *>(X) = h;
    if (ET == kElemF32 || g.both() || s.lo) *reinterpret_cast<f16x8 *>(X + g.lo()) = l;
}

// ------------------------------------------------------- few rows
//
// Latency bounds these: three launches for all steps, where the products take three a
// step (after every 8 of them three more).  A chunk of kOrthoSmallCols columns is in LDS,
// a row after the other; G is read once, as an out may be another matrix's src.
constexpr int kSmallPitch = kOrthoSmallCols + 1;
constexpr int kLater = -1;       // in place of an element type: X in the workspace, fp64

template <int ET>
using small_t = std::conditional_t<ET == kLater, double, float>;

template <int ET>
__device__ __forceinline__ small_t<ET> load1(const char *p, int64_t i) {
    if constexpr (ET == kLater) return reinterpret_cast<const double *>(p)[i];
    if (ET == kElemF32) return reinterpret_cast<const float *>(p)[i];
    if (ET == kElemF16) return static_cast<float>(reinterpret_cast<const _Float16 *>(p)[i]);
    return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[i]) << 16);
}

// Columns [c0, c0 + n) of a small matrix, its elements in the order of memory: load(offset
// in the matrix) of eight a thread, then store(offset, place in the chunk, value) of them.
template <class T, class Load, class Store>
__device__ __forceinline__ void over_chunk(const OrthoGroup &g, int64_t c0, int n, Load load, Store store) {
    const int r = g.r(), all = r * n, d = g.tall() ? r : n;
    const float inverse = 1.0f / d;
    auto row_of = [&](int e) {                             // e / d: e < 2^13, d <= 2^8
        return static_cast<int>((e + 0.5f) * inverse);
    };
    for (int e0 = threadIdx.x; e0 < all; e0 += 2048) {
        T v[8];
        int64_t off[8];
        int at[8];
#pragma unroll
        for (int u = 0; u < 8; u++) {
            const int e = min(e0 + u * 256, all - 1), q = row_of(e), rest = e - q * d;
            off[u] = g.tall() ? c0 * r + e : static_cast<int64_t>(q) * g.nc + c0 + rest;
            at[u] = g.tall() ? rest * kSmallPitch + q : q * kSmallPitch + rest;
            v[u] = load(off[u], at[u]);
        }
#pragma unroll
        for (int u = 0; u < 8; u++)
            if (e0 + u * 256 < all) store(off[u], at[u], v[u]);
    }
}

// X X^T (at first of X = G) of a piece of the columns: a thread sums a 2 x 2 block (r = 1:
// 1 x 1) over some of them.
template <int ET>
__global__ __launch_bounds__(256) void small_gram_kernel(Groups a, Space s) {
    typedef small_t<ET> T;
    __shared__ T x[kOrthoSmall * kSmallPitch];
    __shared__ double part[256][4];
    const OrthoGroup g = group_of(a, blockIdx.x);
    const uint32_t in = blockIdx.x - g.wg0, m = in / g.parts, q = in % g.parts;
    char *const base = s.base + g.base + m * g.stride;
    const char *const src = ET == kLater ? base + g.later_at()
                                         : reinterpret_cast<const char *>(s.pointers[g.first + m].src);
    const int r = g.r(), t = threadIdx.x;
    const int64_t c = g.tall() ? g.nr : g.nc;
    const int64_t chunks = (c + kOrthoSmallCols - 1) / kOrthoSmallCols, per = (chunks + g.parts - 1) / g.parts;
    const int64_t c0 = q * per * kOrthoSmallCols, c1 = min(c0 + per * kOrthoSmallCols, c);
    int side = 1;                                          // threads along a row of blocks
    while (side * 2 < r) side *= 2;
    const int B = r > 1 ? 2 : 1, per_set = side * side, sets = 256 / per_set;
    const int pt = t % per_set, pi = pt / side * B, pj = pt % side * B;
    const int pi1 = min(pi + B - 1, r - 1), pj1 = min(pj + B - 1, r - 1);
    double v00 = 0, v01 = 0, v10 = 0, v11 = 0;
    for (int64_t at = c0; at < c1; at += kOrthoSmallCols) {
        const int n = static_cast<int>(min(kOrthoSmallCols, c1 - at));
        __syncthreads();
        over_chunk<T>(
            g, at, n, [&](int64_t off, int) { return load1<ET>(src, off); },
            [&](int64_t off, int place, T v) {
                if constexpr (ET != kLater) reinterpret_cast<float *>(base)[off] = v;
                x[place] = v;
            });
        __syncthreads();
        if (pi < r && pj < r)
#pragma unroll 4
            for (int col = t / per_set; col < n; col += sets) {
                const double i0 = x[pi * kSmallPitch + col], i1 = x[pi1 * kSmallPitch + col];
                const double j0 = x[pj * kSmallPitch + col], j1 = x[pj1 * kSmallPitch + col];
                v00 += i0 * j0;
                v01 += i0 * j1;
                v10 += i1 * j0;
                v11 += i1 * j1;
            }
    }
    part[t][0] = v00;
    part[t][1] = v01;
    part[t][2] = v10;
    part[t][3] = v11;
    __syncthreads();
    double *const to = reinterpret_cast<double *>(base + g.gram_at()) + static_cast<int64_t>(q) * r * r;
    for (int e = t; e < r * r; e += 256) {
        const int i = e / r, j = e % r, p = i / B * side + j / B, k = i % B * 2 + j % B;
        double v = 0;
        for (int u = 0; u < sets; u++) v += part[u * per_set + p][k];
        to[e] = v;
    }
}

struct SmallArgs {
    Groups a;
    Space s;
    float coefficients[192];
    int steps;
    int later;                   // not the first steps
};

// The steps on A, one workgroup a matrix; what X 2^-k is multiplied by, and k.  At first
// X = G, whose norm is divided by; later k = 0.
__global__ __launch_bounds__(256) void small_steps_kernel(SmallArgs p) {
    constexpr int R = kOrthoSmall, W = R + 2;              // zeros past r
    __shared__ __attribute__((aligned(16))) double A[R * W], P[R * W], M[R * W], T[R * W], U[R * W];
    const OrthoGroup g = group_of(p.a, blockIdx.x);
    char *const base = p.s.base + g.base + (blockIdx.x - g.wg0) * g.stride;
    const double *const gram = reinterpret_cast<const double *>(base + g.gram_at());
    const int r = g.r(), n = r * r, t = threadIdx.x;
    // a thread's 2 x 2 block of every matrix
    const int bi = t / 16 * 2, bj = t % 16 * 2;
    int at[4], from[4];
    double v[4] = {0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < 4; u++) {
        const int i = bi + u / 2, j = bj + u % 2;
        at[u] = i * W + j;
        from[u] = min(i, r - 1) * r + min(j, r - 1);
    }
#pragma unroll 4
    for (uint32_t q = 0; q < g.parts; q++)
#pragma unroll
        for (int u = 0; u < 4; u++) v[u] += gram[static_cast<int64_t>(q) * n + from[u]];
#pragma unroll
    for (int u = 0; u < 4; u++) {
        const int i = bi + u / 2, j = bj + u % 2;
        A[at[u]] = i < r && j < r ? v[u] : 0.0;
        M[at[u]] = i == j && i < r;
    }
    __syncthreads();
    double sum = 0;
    for (int i = 0; i < r; i++) sum += A[i * W + i];
    __syncthreads();
    const double norm = p.later ? 1.0 : sqrt(sum);
    const bool finite = norm < __builtin_inf();
    if (!p.later)
#pragma unroll
        for (int u = 0; u < 4; u++) A[at[u]] = norm > 0 ? A[at[u]] / sum : 0.0;
    int k = 0;
    const double frac = !p.later && finite && norm > 0 ? frexp(norm, &k) : 1.0;
    __syncthreads();
    auto times = [&](double *out, const double *x, const double *y) {
        double o[4] = {0, 0, 0, 0};
#pragma unroll 8
        for (int j = 0; j < r; j++) {
            const double a = x[bi * W + j], b = x[bi * W + W + j], c = y[j * W + bj], d = y[j * W + bj + 1];
            o[0] += a * c;
            o[1] += a * d;
            o[2] += b * c;
            o[3] += b * d;
        }
#pragma unroll
        for (int u = 0; u < 4; u++) out[at[u]] = o[u];
    };
    for (int q = 0; q < p.steps; q++) {
        const double ca = p.coefficients[3 * q], cb = p.coefficients[3 * q + 1], cc = p.coefficients[3 * q + 2];
        times(T, A, A);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const int i = bi + u / 2, j = bj + u % 2;
            P[at[u]] = (i == j && i < r ? ca : 0.0) + cb * A[at[u]] + cc * T[at[u]];
        }
        __syncthreads();
        times(T, P, M);
        times(U, P, A);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 4; u++) M[at[u]] = T[at[u]];
        times(A, U, P);
        __syncthreads();
    }
    double *const map = reinterpret_cast<double *>(base + g.map_at());
    for (int e = t; e < n; e += 256) {
        const double o = M[e / r * W + e % r];
        map[e] = !finite ? __builtin_nan("") : norm > 0 ? o / frac : 0.0;
    }
    if (t == 0) map[n] = k;
}

// M (X 2^-k), a chunk a workgroup: X = G or (FROM) a later one; to out or (TO) to the later
// X, in its place.
template <bool FROM, bool TO>
__global__ __launch_bounds__(256) void small_apply_kernel(Groups a, Space s) {
    constexpr int R = kOrthoSmall;
    typedef std::conditional_t<FROM || TO, double, float> T;
    __shared__ T x[R * kSmallPitch];
    __shared__ __attribute__((aligned(16))) double M[R * R];
    const OrthoGroup g = group_of(a, blockIdx.x);
    const int64_t c = g.tall() ? g.nr : g.nc;
    const uint32_t per = static_cast<uint32_t>((c + kOrthoSmallCols - 1) / kOrthoSmallCols);
    const uint32_t in = blockIdx.x - g.wg0, m = in / per;
    char *const base = s.base + g.base + m * g.stride;
    double *const later = reinterpret_cast<double *>(base + g.later_at());
    const double *const map = reinterpret_cast<const double *>(base + g.map_at());
    const int r = g.r(), k = -static_cast<int>(map[r * r]), t = threadIdx.x;
    const int64_t c0 = static_cast<int64_t>(in % per) * kOrthoSmallCols;
    const int n = static_cast<int>(min(kOrthoSmallCols, c - c0));
    for (int e = t; e < R * R; e += 256) M[e] = e / R < r && e % R < r ? map[e / R * r + e % R] : 0.0;
    for (int e = t; e < (R - r) * kSmallPitch; e += 256) x[r * kSmallPitch + e] = 0;
    over_chunk<T>(
        g, c0, n,
        [&](int64_t off, int) -> T {
            if constexpr (FROM) return later[off];
            return ldexpf(reinterpret_cast<const float *>(base)[off], k);
        },
        [&](int64_t, int place, T v) { x[place] = v; });
    __syncthreads();
    // a column's rows by 2 threads
    constexpr int COLS = static_cast<int>(kOrthoSmallCols), SHARE = 256 / COLS;
    const int col = t % COLS;
    T v[R];
#pragma unroll
    for (int j = 0; j < R; j++) v[j] = x[j * kSmallPitch + col];
    __syncthreads();
    if (col < n)
        for (int i = t / COLS; i < r; i += SHARE) {
            double even = 0, odd = 0;
#pragma unroll
            for (int j8 = 0; j8 < R; j8 += 8) {
                if (j8 >= r) break;
#pragma unroll
                for (int j = j8; j < j8 + 8; j += 2) {
                    even += M[i * R + j] * v[j];
                    odd += M[i * R + j + 1] * v[j + 1];
                }
            }
            x[i * kSmallPitch + col] = static_cast<T>(even + odd);
        }
    __syncthreads();
    __bf16 *const out = reinterpret_cast<__bf16 *>(s.pointers[g.first + m].out);
    over_chunk<T>(
        g, c0, n, [&](int64_t, int place) { return x[place]; },
        [&](int64_t off, int, T v) {
            if constexpr (TO)
                later[off] = v;
            else
                out[off] = static_cast<__bf16>(static_cast<float>(v));
        });
}

// ------------------------------------------------------- the products

// out[i, j] = sum over c of I(i, c) J(c, j) for fp16 factors in panels, so that both
// go straight into LDS, in runs of at least 1 KB: rows of 64 bytes each from a
// row-major matrix are half lines of the cache (an 8B layer 17.9 ms, in panels, with
// larger fragments and more steps in LDS, 15.4).  A T x T tile of
// the output per workgroup of 4 waves, 2 x 2; one step of the sum is 32 values, 64 T
// bytes of a factor:
//   along   (the sum runs along the rows): T rows of one panel
//   across  (the sum runs over the rows): 32 rows of T / 32 panels, read with the
//           transposing read, which hands each lane 4 values along the sum
// In both, chunk h (16 bytes) of a panel's row r lies at h ^ key(r) in LDS: the rows
// that a read of either kind takes at a time fall into different banks.
constexpr int kThreads = 256;
constexpr int kStep = 32;
// Steps in LDS: 160 KB of it for one workgroup a unit, 80 KB for two.
__host__ __device__ constexpr int buffers(int T) { return T == 64 ? 10 : 5; }

__device__ __forceinline__ int key(int r) { return r >> 3 & 3; }

template <bool ACROSS, int T>
struct Feed {
    static constexpr int SLOTS = T * 4 / kThreads;         // 16-byte loads per thread and step
    static constexpr int BYTES = T * 64;

    const char *base;            // of the next step
    int64_t left;                // bytes from base to the end of what may be read
    uint32_t advance;            // bytes from one step to the next
    uint32_t panel;              // bytes of a panel
    int live;                    // steps that are left: after them nothing may be read
    int turn;                    // steps until the sum goes on elsewhere,
    int64_t jump, again;         // so many bytes from there, with so many left
    uint32_t off;                // this thread's first slot

    // Lines [first, first + T) of a matrix [rows, cols] in panels, for `steps` steps;
    // after `half` of them the sum goes on `to` bytes from the matrix's start (a
    // multiple of its size).
    __device__ __forceinline__ void init(const char *p, uint32_t rows, uint32_t cols, uint32_t first,
                                         uint32_t steps, uint32_t half, int64_t to, int t) {
        live = uniform(steps);
        panel = uniform(static_cast<int64_t>(rows) * 64);
        const int64_t bytes = static_cast<int64_t>(panel) * (cols / 32);
        turn = uniform(half);
        int64_t at;
        if (ACROSS) {
            at = static_cast<int64_t>(first / 32) * panel;
            left = bytes - at;
            advance = kStep * 64;
        } else {
            at = static_cast<int64_t>(first) * 64;
            left = min(static_cast<int64_t>(rows - first), static_cast<int64_t>(T)) * 64;
            advance = panel;
        }
        base = scalar(p + at);
        jump = to - static_cast<int64_t>(half) * advance;
        left = again = uniform64(left);
        jump = uniform64(jump);
        const int row = t / 4;                              // of 64, in a panel
        const int at16 = (row & 31) * 64 + ((t & 3) ^ key(row)) * 16;
        off = at16 + (row >> 5) * (ACROSS ? panel : 32 * 64);
    }
    static __device__ __forceinline__ int64_t uniform64(int64_t v) {
        return static_cast<int64_t>(reinterpret_cast<uint64_t>(scalar(reinterpret_cast<const char *>(v))));
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer() const {
        const int64_t most = 0xffffffc0ll;
        return buffer_of(base, live > 0 ? static_cast<uint32_t>(left < most ? left : most) : 0);
    }
    // Asks for slot q of the next step: 64 rows further (along), 2 panels (across).
    // What lies outside, and past the last step everything, comes as zeros.
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, LDS_AS char *lds, int wave, int q) const {
        direct_load(r, lds + (wave + q * 4) * 1024, off, q * (ACROSS ? 2 * panel : 64 * 64));
    }
    __device__ __forceinline__ void next() {
        live--;
        base += advance;
        if (ACROSS) left -= advance;
        if (--turn == 0) {
            base += jump;
            if (ACROSS) left = again;
        }
    }
    // A fragment is 32 lines x 16 values: lane (r32, g) holds values 8 g + 0..7 of line
    // r32.  This lane's part of its address.
    static __device__ __forceinline__ int lane_at(int lane) {
        if (!ACROSS) {
            const int r = lane & 31, g = lane >> 5;
            return r * 64 + ((g ^ key(r)) << 4);
        }
        // rows 8 g + q, and 4 further on; columns 16 h + 4 p .. + 3 (chunks 2 h + p / 2)
        const int q = lane >> 2 & 3, p = lane & 3, h = lane >> 4 & 1, row = (lane >> 5) * 8 + q;
        return row * 64 + (((2 * h + (p >> 1)) ^ key(row)) << 4) + (p & 1) * 8;
    }
    // The fragment of lines [32 f, 32 f + 32), values [16 k, 16 k + 16) of the step.
    static __device__ __forceinline__ f16x8 frag(const LDS_AS char *lds, int lane, int f, int k) {
        if (!ACROSS)             // chunks 2 k and 2 k + 1
            return *reinterpret_cast<const LDS_AS f16x8 *>(lds + f * 2048 + (lane ^ k * 32));
        union {
            i16x4 h[2];
            f16x8 v;
        } u;
        // rows 16 k on: key() differs in its second bit
        const LDS_AS char *p = lds + f * 2048 + k * 1024 + (lane ^ k * 32);
        u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4 *)p);
        u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4 *)(p + 256));
        return u.v;
    }
};

// BUFFERS steps are in LDS.  While one is multiplied, the fragments of the next are
// read, a J and an I fragment per line (all multiplications of one I fragment), and
// the loads of the last one that fits set out into the buffer that the barrier has just
// freed; so (of 5) a step's loads have two to three steps to arrive, and reads and loads
// come evenly.
template <bool AI, bool AJ, int T>
struct Half {
    static constexpr int F = T / 2 / 32;                   // 32 x 32 fragments of a wave, each way
    static constexpr int LINES = 2 * F;                    // of a step: 2 x 16 values
    static constexpr int D = LINES >= 8 ? 3 : 1, RING = D + 1;   // I fragments read ahead
    typedef Feed<AI, T> FI;
    typedef Feed<AJ, T> FJ;
    static constexpr int LOADS = FI::SLOTS + FJ::SLOTS;
    static constexpr int PER_LINE = LOADS / LINES;         // loads issued with a line
    static constexpr int BUFFERS = buffers(T);
    // Loads return in order, so the first steps would wait for any that set out before
    // them; under the last steps, two workgroups a unit, 48 x [768, 2048] take 1706 us
    // for 1784.  The large tiles, alone on their unit and in long sums, are as fast with
    // them at the start (8B layer 14.2 ms for 14.35), behind the first steps' loads.
    static constexpr uint32_t LATE = T == 256 ? 1u << 30 : 32;
    static constexpr int TILE = FI::BYTES, BUFFER = 2 * TILE, LDS = BUFFERS * BUFFER;
    static_assert(LINES % RING == 0 && LOADS % LINES == 0, "a step starts at ring entry 0");

    FI fi;
    FJ fj;
    int lane, wave, wi, wj, ai, aj;
    f32x16 acc[F][F];

    // All but this wave's newest N loads have arrived, and every wave is here.  The
    // fragments read before have all been multiplied but for those of the current
    // step, whose buffer stays: reads need not be waited for.  Loads return in order,
    // and any that the compiler might add only make the wait longer.
    template <int N>
    static __device__ __forceinline__ void wait() {
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" : : "n"(N) : "memory");
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t ri, __amdgpu_buffer_rsrc_t rj,
                                         LDS_AS char *b, int q) const {
        if (q < FI::SLOTS)
            fi.load(ri, b, wave, q);
        else
            fj.load(rj, b + TILE, wave, q - FI::SLOTS);
    }
    __device__ __forceinline__ f16x8 line(const LDS_AS char *b, int n) const {
        return FI::frag(b + wi * (TILE / 2), ai, n % F, n / F);
    }
    __device__ __forceinline__ f16x8 row(const LDS_AS char *b, int n) const {
        return FJ::frag(b + TILE + wj * (TILE / 2), aj, n % F, n / F);
    }
    // One step from `here`; `there` is the next one, `to` receives the one that comes
    // BUFFERS - 1 after it.
    __device__ __forceinline__ void step(f16x8 *l, const f16x8 *r, f16x8 *next, const LDS_AS char *here,
                                         const LDS_AS char *there, LDS_AS char *to) {
        const __amdgpu_buffer_rsrc_t ri = fi.buffer(), rj = fj.buffer();
        // the next step has arrived; newer are the loads of those behind it
        wait<(BUFFERS - 3) * LOADS>();
#pragma unroll
        for (int n = 0; n < LINES; n++) {
            l[(n + D) % RING] = n + D < LINES ? line(here, n + D) : line(there, n + D - LINES);
            next[n] = row(there, n);
#pragma unroll
            for (int y = 0; y < F; y++) {
                acc[n % F][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(r[n / F * F + y], l[n % RING],
                                                                       acc[n % F][y], 0, 0, 0);
                if (y == 0) {
#pragma unroll
                    for (int q = 0; q < PER_LINE; q++) load(ri, rj, to, n * PER_LINE + q);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        fi.next();
        fj.next();
    }
    // ask(c), c < ASKS: loads of the caller's own, which set out when LATE (c = 0) and
    // LATE / 2 (c = 1) steps are left.
    template <int ASKS, class Ask>
    __device__ __forceinline__ void run(LDS_AS char *lds, uint32_t steps, Ask ask) {
        ai = FI::lane_at(lane);
        aj = FJ::lane_at(lane);
#pragma unroll
        for (int b = 0; b < BUFFERS - 1; b++) {
            const __amdgpu_buffer_rsrc_t ri = fi.buffer(), rj = fj.buffer();
#pragma unroll
            for (int q = 0; q < LOADS; q++) load(ri, rj, lds + b * BUFFER, q);
            fi.next();
            fj.next();
        }
        wait<(BUFFERS - 2) * LOADS>();
        f16x8 l[RING], r0[LINES], r1[LINES];
#pragma unroll
        for (int n = 0; n < LINES; n++) r0[n] = row(lds, n);
#pragma unroll
        for (int n = 0; n < D; n++) l[n] = line(lds, n);
        uint32_t here = 0, to = (BUFFERS - 1) * BUFFER;
        auto after = [](uint32_t b) { return b == (BUFFERS - 1) * BUFFER ? 0 : b + BUFFER; };
        // sums are of 64 values or a multiple: steps come in pairs
        auto until = [&](uint32_t left) {
            for (; steps > left; steps -= 2) {
                const uint32_t there = after(here), to2 = after(to);
                step(l, r0, r1, lds + here, lds + there, lds + to);
                here = after(there);
                step(l, r1, r0, lds + there, lds + here, lds + to2);
                to = after(to2);
            }
        };
        if (ASKS > 0) {
            until(LATE);
            ask(0);
        }
        if (ASKS > 1) {
            until(LATE / 2);
            ask(1);
        }
        until(0);
        arrived();               // no load may still be on its way to LDS at the end,
        __syncthreads();         // nor a read of what the sums will overwrite
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
    int short_g;                 // G is in 16 bits
};

// A sum rounded to fp32 and then to fp16.  Left to itself the compiler takes an
// instruction that adds and rounds once, to fp16, for some of a row's entries.
__device__ __forceinline__ _Float16 rounded_twice(float v) {
    asm("" : "+v"(v));
    return static_cast<_Float16>(v);
}

// Tiles of a matrix's A or P: on and below the diagonal; of its X: all.
__host__ __device__ inline uint32_t tiles_of(const OrthoGroup &g, int stage, uint32_t T) {
    if (stage == kApply) return (g.nrp + T - 1) / T * ((g.ncp + T - 1) / T);
    const uint32_t n = (g.rp() + T - 1) / T;
    return n * (n + 1) / 2;
}

// A wave's sums go through its own part of LDS, 32 rows at a time, so that a lane gets
// 8 neighbours of a row, 16 bytes of a panel, and a wave's accesses are runs of 1 KB
// (16 rows of a panel).
template <int T>
struct Turn {
    static constexpr int W = T / 2, PITCH = W * 4 + 16;    // a wave's tile is W x W
    static constexpr int PASSES = 32 * W / 512;

    LDS_AS char *lds;
    int lane;
    int per;                     // lanes of a row: 4 (a panel's row), or W / 8

    template <int F>
    __device__ __forceinline__ void put(const f32x16 (&acc)[F][F], int c) const {
        // a lane holds columns 8 q + 4 g + 0..3 of its row, q = 0..3
#pragma unroll
        for (int y = 0; y < F; y++)
#pragma unroll
            for (int q = 0; q < 4; q++)
                *reinterpret_cast<LDS_AS f32x4 *>(lds + (lane & 31) * PITCH + y * 128 + q * 32 +
                                                  (lane >> 5) * 16) =
                    f32x4{acc[c][y][4 * q], acc[c][y][4 * q + 1], acc[c][y][4 * q + 2], acc[c][y][4 * q + 3]};
    }
    // This lane's row and first column in pass q.
    __device__ __forceinline__ int row(int q) const {
        return per == 4 ? q % 2 * 16 + lane / 4 : q * (64 / (W / 8)) + lane / (W / 8);
    }
    __device__ __forceinline__ int col(int q) const {
        return per == 4 ? q / 2 * 32 + lane % 4 * 8 : lane % (W / 8) * 8;
    }
    __device__ __forceinline__ LDS_AS char *at(int q) const { return lds + row(q) * PITCH + col(q) * 4; }
    __device__ __forceinline__ void get(float *v, int q) const {
        const f32x4 a = *reinterpret_cast<const LDS_AS f32x4 *>(at(q));
        const f32x4 b = *reinterpret_cast<const LDS_AS f32x4 *>(at(q) + 16);
#pragma unroll
        for (int n = 0; n < 4; n++) v[n] = a[n], v[4 + n] = b[n];
    }
    // The 32 rows once more, as fp16 numbers, behind the sums, to be read down the
    // columns: rows 8 g .. 8 g + 7 of column 16 q + r16 for lane (r16, g), a run of 1 KB in
    // the matrix's other half.
    static constexpr int HALF = 32 * PITCH, HALF_PITCH = W * 2 + 16;
    static_assert(HALF + 32 * HALF_PITCH <= buffers(T) * 2 * T * 64 / 4, "a wave's part of LDS");
    __device__ __forceinline__ void set(int q, const f16x8 &h) const {
        *reinterpret_cast<LDS_AS f16x8 *>(lds + HALF + row(q) * HALF_PITCH + col(q) * 2) = h;
    }
    __device__ __forceinline__ f16x8 column(int q) const {
        union {
            i16x4 h[2];
            f16x8 v;
        } u;
        const LDS_AS char *p = lds + HALF + ((lane >> 4) * 8 + (lane >> 2 & 3)) * HALF_PITCH + q * 32 + (lane & 3) * 8;
        u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4 *)p);
        u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4 *)(p + 4 * HALF_PITCH));
        return u.v;
    }
};

template <int STAGE, bool AI, bool AJ, int T>
__device__ __forceinline__ void product_tile(const ProductArgs &p, const OrthoGroup &g, uint32_t m,
                                             uint32_t ti, uint32_t tj, LDS_AS char *lds) {
    typedef Half<AI, AJ, T> K;
    const int t = threadIdx.x, lane = t & 63;
    char *const base = p.s.base + g.base + static_cast<int64_t>(m) * g.stride;
    char *const x = base + p.from * g.x_bytes();
    const uint32_t rp = g.rp(), i0 = ti * T, j0 = tj * T;
    K k;
    k.wave = __builtin_amdgcn_readfirstlane(t >> 6);
    k.lane = lane;
    k.wi = k.wave / 2;
    k.wj = k.wave % 2;
    // with both, hi's sum goes on with lo, and P's from its start again
    const uint32_t once = (STAGE == kGram ? max(g.nrp, g.ncp) : rp) / kStep;
    const bool both = g.both() || p.s.lo, twice = STAGE == kApply && both;
    const uint32_t steps = twice ? 2 * once : once, half = twice ? once : ~0u;
    const int64_t lo = twice ? 2 * g.lo() : 0;
    if (STAGE == kGram) {
        k.fi.init(x, g.nrp, g.ncp, i0, steps, half, 0, t);
        k.fj.init(x, g.nrp, g.ncp, j0, steps, half, 0, t);
    } else if (STAGE == kPoly) {
        k.fi.init(base + g.a_at(), rp, rp, i0, steps, half, 0, t);
        k.fj.init(base + g.a_at(), rp, rp, j0, steps, half, 0, t);
    } else if (g.tall()) {
        k.fi.init(x, g.nrp, g.ncp, i0, steps, half, lo, t);
        k.fj.init(base + g.p_at(), rp, rp, j0, steps, half, 0, t);
    } else {
        k.fi.init(base + g.p_at(), rp, rp, i0, steps, half, 0, t);
        k.fj.init(x, g.nrp, g.ncp, j0, steps, half, lo, t);
    }
#pragma unroll
    for (int a = 0; a < K::F; a++)
#pragma unroll
        for (int b = 0; b < K::F; b++)
#pragma unroll
            for (int n = 0; n < 16; n++) k.acc[a][b][n] = 0.0f;
    typedef Turn<T> U;
    // the last step's output is row-major
    const U turn = {lds + k.wave * (K::LDS / 4), lane, STAGE == kApply && p.last ? U::W / 8 : 4};
    const uint32_t li = i0 + k.wi * U::W, lj = j0 + k.wj * U::W;       // the wave's first row and column
    // What the sums are joined with, 32 rows of the wave's tile at a time: asked for
    // ahead, the first KEEP times under the products, so that its latency and (all
    // workgroups come here together) its traffic lie under them; see LATE.
    const char *const __restrict__ old = STAGE == kPoly ? base + g.a_at() : x;
    const uint32_t orows = STAGE == kPoly ? rp : g.nrp, ocols = STAGE == kPoly ? rp : g.ncp;
    constexpr int PARTS = STAGE == kGram ? 0 : STAGE == kPoly ? 1 : 2;
    constexpr int KEEP = K::F < 2 ? 1 : 2;
    f16x8 held[KEEP][U::PASSES][PARTS ? PARTS : 1];
    // A G in 16 bits is hi alone in the first step (down to 2^-25 of X's elements'
    // mean).  Without lo in the last one, a matrix of low rank would be off by more than
    // its rounding to bf16.
    const bool lows = both || !p.first || !p.short_g;
    if (PARTS == 2)
#pragma unroll
        for (int c = 0; c < KEEP; c++)
#pragma unroll
            for (int q = 0; q < U::PASSES; q++) held[c][q][1] = f16x8{0, 0, 0, 0, 0, 0, 0, 0};
    auto ask = [&](int c) {
#pragma unroll
        for (int q = 0; q < U::PASSES; q++) {
            // Past the matrix its last row or columns, whose values nothing uses.  Not a
            // branch by lanes: here, between the loops, the compiler (ROCm 7.2) has
            // placed a register's copy before the lanes are joined again.
            const uint32_t i = min(li + c * 32 + turn.row(q), orows - 1);
            const uint32_t j = min(lj + turn.col(q), ocols - 8);
            const char *from = old + panel_at(orows, i, j) * 2;
#pragma unroll
            for (int h = 0; h < PARTS; h++)
                if (h == 0 || lows)
                    held[c % KEEP][q][h] = *reinterpret_cast<const f16x8 *>(from + h * 2 * g.lo());
        }
    };
    k.template run<PARTS ? KEEP : 0>(lds, uniform(steps), ask);

    const float2 t1 = p.first ? p.s.scales[g.first + m] : make_float2(1.0f, 1.0f);
    const int ex = x_exponent(g.nr, g.nc);
    float *const ad = reinterpret_cast<float *>(base + g.a_diag());
    float *const pd = reinterpret_cast<float *>(base + g.p_diag());
    const float f = STAGE == kGram    ? ldexpf(t1.y, -2 * ex)
                    : STAGE == kPoly  ? 1.0f / (kScaleA * kScaleA)
                    : p.last          ? ldexpf(t1.x, -ex)
                                      : t1.x;
    if (STAGE != kApply) {
        _Float16 *const __restrict__ to =
            reinterpret_cast<_Float16 *>(base + (STAGE == kGram ? g.a_at() : g.p_at()));
        const uint32_t r = g.r();
        const bool diagonal = ti == tj;
#pragma unroll
        for (int c = 0; c < K::F; c++) {
            turn.put(k.acc, c);
#pragma unroll
            for (int q = 0; q < U::PASSES; q++) {
                const uint32_t i = li + c * 32 + turn.row(q), j = lj + turn.col(q);
                float v[8];
                turn.get(v, q);
                f16x8 h = {0, 0, 0, 0, 0, 0, 0, 0};
                if (i < rp && j < rp) {                  // X's padding makes zeros of A's and P's
                    if (STAGE == kGram) {
#pragma unroll
                        for (int n = 0; n < 8; n++) h[n] = rounded_twice(v[n] * (f * kScaleA));
                        if (diagonal)
#pragma unroll
                            for (int n = 0; n < 8; n++)
                                if (i == j + n) {
                                    ad[i] = v[n] * f;
                                    h[n] = 0;
                                }
                    } else {
                        // O_ij (b + c (d_i + d_j)) + c (O^2)_ij, in the scales of O and R:
                        // rounded alike for (i, j) and (j, i), as it depends on the tiles'
                        // size whether an entry is mirrored or computed on both sides
                        const float cs = p.cc * (kScaleP / kScaleA), co = p.cc * f * kScaleP;
                        const float di = ad[i], bs = p.cb * (kScaleP / kScaleA);
                        const f32x4 dl = *reinterpret_cast<const f32x4 *>(ad + j);
                        const f32x4 dh = *reinterpret_cast<const f32x4 *>(ad + j + 4);
                        const f16x8 o = held[c % KEEP][q][0];
#pragma unroll
                        for (int n = 0; n < 8; n++)
                            h[n] = rounded_twice(
                                __builtin_fmaf(static_cast<float>(o[n]),
                                               __builtin_fmaf(cs, di + (n < 4 ? dl[n] : dh[n - 4]), bs),
                                               v[n] * co));
                        if (diagonal)
#pragma unroll
                            for (int n = 0; n < 8; n++)
                                if (i == j + n) {
                                    pd[i] = i < r ? p.ca + p.cb * di + p.cc * (di * di + v[n] * f) : 0.0f;
                                    h[n] = 0;
                                }
                    }
                    *reinterpret_cast<f16x8 *>(to + panel_at(rp, i, j)) = h;
                }
                if (!diagonal) turn.set(q, h);
            }
            if (PARTS && c + KEEP < K::F) ask(c + KEEP);
            if (!diagonal) {                             // the other side
#pragma unroll
                for (int q = 0; q < U::W / 16; q++) {
                    const uint32_t i = li + c * 32 + (lane >> 4) * 8, j = lj + q * 16 + (lane & 15);
                    const f16x8 h = turn.column(q);
                    if (i < rp && j < rp) *reinterpret_cast<f16x8 *>(to + panel_at(rp, j, i)) = h;
                }
            }
        }
        return;
    }
    // R X / 2^10 + Q X, as X is held; times the first step's factor
    _Float16 *const __restrict__ to = reinterpret_cast<_Float16 *>(base + (1 - p.from) * g.x_bytes());
    __bf16 *const __restrict__ out =
        p.last ? reinterpret_cast<__bf16 *>(p.s.pointers[g.first + m].out) : nullptr;
    const bool tall = g.tall();
#pragma unroll
    for (int c = 0; c < K::F; c++) {
        turn.put(k.acc, c);
#pragma unroll
        for (int q = 0; q < U::PASSES; q++) {
            const uint32_t i = li + c * 32 + turn.row(q), j = lj + turn.col(q);
            float v[8];
            turn.get(v, q);
            if (i >= g.nrp || j >= g.ncp) continue;
            const f16x8 h = held[c % KEEP][q][0], l = held[c % KEEP][q][PARTS - 1];
            f32x4 ql, qh;
            if (tall) {
                ql = *reinterpret_cast<const f32x4 *>(pd + j) * f;
                qh = *reinterpret_cast<const f32x4 *>(pd + j + 4) * f;
            } else {
                const float qi = pd[i] * f;
                ql = qh = f32x4{qi, qi, qi, qi};
            }
            // in instructions that take fp16 factors as they are: 5 or 6 an element,
            // where the conversions apart would be 12, and this is what a short sum's
            // tile spends as much time on as on its products
#pragma unroll
            for (int n = 0; n < 8; n++) {
                const float qn = n < 4 ? ql[n] : qh[n - 4];
                v[n] = __builtin_fmaf(static_cast<float>(h[n]), qn, v[n] * (f / kScaleP));
                v[n] = __builtin_fmaf(static_cast<float>(l[n]), qn, v[n]);
            }
            if (!p.last) {
                const int64_t at = panel_at(g.nrp, i, j);
                f16x8 nh, nl;
#pragma unroll
                for (int n = 0; n < 8; n++) {
                    nh[n] = static_cast<_Float16>(v[n]);
                    nl[n] = static_cast<_Float16>(__builtin_fmaf(static_cast<float>(nh[n]), -1.0f, v[n]));
                }
                *reinterpret_cast<f16x8 *>(to + at) = nh;
                *reinterpret_cast<f16x8 *>(to + at + g.lo()) = nl;
                continue;
            }
            if (i >= g.nr || j >= g.nc) continue;
            __bf16 *o = out + static_cast<int64_t>(i) * g.nc + j;
            if (g.nc - j >= 8) {
                *reinterpret_cast<half_u32x4 *>(o) =
                    half_u32x4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
            } else {
#pragma unroll
                for (int n = 0; n < 8; n++)
                    if (j + n < g.nc) o[n] = static_cast<__bf16>(v[n]);
            }
        }
        if (c + KEEP < K::F) ask(c + KEEP);
    }
}

template <int STAGE, int T>
__global__ __launch_bounds__(kThreads, T == 256 ? 1 : 2) void product_kernel(ProductArgs p) {
    __shared__ __attribute__((aligned(1024))) char lds[Half<false, false, T>::LDS];
    LDS_AS char *const b = (LDS_AS char *)lds;
    // Workgroup IDs go to the 8 XCDs in turn and each XCD has its own L2, so every
    // XCD takes one contiguous run of each group's tiles (all of one length).
    const OrthoGroup g = group_of(p.a, blockIdx.x);
    const uint32_t per = tiles_of(g, STAGE, T), n = per * g.count;
    const uint32_t id = blockIdx.x - g.wg0, xcd = id % 8;
    const uint32_t in = xcd * (n / 8) + min(xcd, n % 8) + id / 8;
    const uint32_t m = uniform(in / per), at = uniform(in % per);
    if (STAGE == kApply) {
        // 8 tile rows advance together, as in the blocked products
        const uint32_t tr = (g.nrp + T - 1) / T, tc = (g.ncp + T - 1) / T;
        const uint32_t pg = 8 * tc, gr = at / pg, l = at - gr * pg, h = min(8u, tr - 8 * gr);
        const uint32_t ti = uniform(8 * gr + l % h), tj = uniform(l / h);
        if (g.tall())
            product_tile<STAGE, false, false, T>(p, g, m, ti, tj, b);
        else
            product_tile<STAGE, false, true, T>(p, g, m, ti, tj, b);
        return;
    }
    // at = ti (ti + 1) / 2 + tj, tj <= ti
    uint32_t ti = static_cast<uint32_t>((sqrtf(8.0f * at + 1.0f) - 1.0f) * 0.5f);
    while ((ti + 1) * (ti + 2) / 2 <= at) ti++;
    while (ti * (ti + 1) / 2 > at) ti--;
    ti = uniform(ti);
    const uint32_t tj = uniform(at - ti * (ti + 1) / 2);
    if (STAGE == kGram && g.tall())
        product_tile<STAGE, true, true, T>(p, g, m, ti, tj, b);
    else
        product_tile<STAGE, false, false, T>(p, g, m, ti, tj, b);
}

constexpr int64_t kMaxWgs = 0xffffffffll / 512;

// Calls launch(groups, workgroups) over the groups in their order, as many at a time as
// kernel arguments hold and a launch can count; wgs(g): workgroups of one matrix of
// g, which are fewer than that (ortho_plan).
template <class Wgs, class Launch>
tide_status over_groups(const std::vector<OrthoGroup> &groups, Wgs wgs, Launch launch) {
    size_t at = 0;
    uint32_t done = 0;           // matrices of group `at` launched before
    while (at < groups.size()) {
        Groups a;
        a.n = 0;
        int64_t total = 0;
        while (at < groups.size() && a.n < kOrthoGroups) {
            OrthoGroup g = groups[at];
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

// Small tiles while middle ones would leave half of the card idle.  Else by whole
// rounds of the card, 256 large tiles or 512 middle ones (half the work, 0.55 of the
// time).  48 x [768, 2048]: X X^T and P, 2 rounds of each, 120 and 74 us with large
// tiles, 91 and 46 with middle ones; P X, 5 rounds against 9, 220 against 200.  [4096,
// 4096]: X X^T and P, 1 round against 2, 94 and 100 against 91 and 96, but P X, 1
// against 2, 135 against 149, and all steps 1555 against 1650.
int tile_for(const std::vector<OrthoGroup> &groups, int stage) {
    auto tiles = [&](uint32_t T) {
        int64_t n = 0;
        for (const OrthoGroup &g : groups)
            n += static_cast<int64_t>(g.count) * tiles_of(g, stage, T);
        return n;
    };
    const int64_t middle = tiles(128);
    if (middle < kCus / 2) return 64;
    const int64_t large = (tiles(256) + kCus - 1) / kCus, half = (middle + 2 * kCus - 1) / (2 * kCus);
    return large * 20 <= half * 11 ? 256 : 128;
}

// For X X^T the groups with the longest sums first: else their tiles leave most of
// the card idle at the launch's end (the 8B layer, sums of 14336 and 4096, 910 us, so
// 830).  The other products' sums are up to r, and their order gains nothing (P X of
// the same layer 1680 to 1700 us as they come, 1740 the longest first).
std::vector<OrthoGroup> longest_first(const std::vector<OrthoGroup> &groups) {
    std::vector<OrthoGroup> v = groups;
    std::stable_sort(v.begin(), v.end(), [](const OrthoGroup &a, const OrthoGroup &b) {
        return std::max(a.nrp, a.ncp) > std::max(b.nrp, b.ncp);
    });
    return v;
}

template <int STAGE>
tide_status run_product(const std::vector<OrthoGroup> &groups, ProductArgs p, hipStream_t s) {
    const int T = tile_for(groups, STAGE);
    return over_groups(
        groups, [&](const OrthoGroup &g) { return tiles_of(g, STAGE, static_cast<uint32_t>(T)); },
        [&](const Groups &a, uint32_t total) {
            p.a = a;
            if (T == 256)
                product_kernel<STAGE, 256><<<dim3(total), dim3(kThreads), 0, s>>>(p);
            else if (T == 128)
                product_kernel<STAGE, 128><<<dim3(total), dim3(kThreads), 0, s>>>(p);
            else
                product_kernel<STAGE, 64><<<dim3(total), dim3(kThreads), 0, s>>>(p);
        });
}

// What reads the matrices: of the large ones, and of the small ones.
template <int ET>
tide_status run_first(const std::vector<OrthoGroup> &groups, const std::vector<OrthoGroup> &small,
                      const Space &sp, hipStream_t s) {
    tide_status st = over_groups(
        groups, [](const OrthoGroup &g) { return g.parts; },
        [&](const Groups &a, uint32_t total) {
            squares_kernel<ET><<<dim3(total), dim3(256), 0, s>>>(a, sp);
        });
    if (st == TIDE_OK)
        st = over_groups(
            small, [](const OrthoGroup &g) { return g.parts; },
            [&](const Groups &a, uint32_t total) {
                small_gram_kernel<ET><<<dim3(total), dim3(256), 0, s>>>(a, sp);
            });
    if (st != TIDE_OK) return st;
    return over_groups(
        groups, [](const OrthoGroup &g) { return g.nrp / 16 * ((g.ncp + 127) / 128); },
        [&](const Groups &a, uint32_t total) {
            first_kernel<ET><<<dim3(total), dim3(256), 0, s>>>(a, sp);
        });
}

// By how much step i raises what is near zero.
double raises(const OrthoArgs &a, int i) {
    return std::max(1.0, std::fabs(static_cast<double>(a.coefficients[3 * i])));
}

// The steps of small matrices whose G G^T is known.
tide_status run_small(const std::vector<OrthoGroup> &small, const OrthoArgs &a, const Space &sp,
                      hipStream_t s) {
    SmallArgs p;
    p.s = sp;
    for (int from = 0, to = 0; from < a.steps; from = to) {
        // as many steps as raise by less than kOrthoRaised, one at least
        double raised = raises(a, to++);
        for (; to < a.steps && raised * raises(a, to) <= kOrthoRaised; to++) raised *= raises(a, to);
        p.later = from > 0;
        p.steps = to - from;
        std::copy(a.coefficients + 3 * from, a.coefficients + 3 * to, p.coefficients);
        tide_status st = TIDE_OK;
        if (p.later)
            st = over_groups(
                small, [](const OrthoGroup &g) { return g.parts; },
                [&](const Groups &g, uint32_t total) {
                    small_gram_kernel<kLater><<<dim3(total), dim3(256), 0, s>>>(g, sp);
                });
        if (st == TIDE_OK)
            st = over_groups(
                small, [](const OrthoGroup &) { return 1; },
                [&](const Groups &g, uint32_t total) {
                    p.a = g;
                    small_steps_kernel<<<dim3(total), dim3(256), 0, s>>>(p);
                });
        if (st == TIDE_OK)
            st = over_groups(
                small,
                [](const OrthoGroup &g) {
                    return (std::max(g.nr, g.nc) + kOrthoSmallCols - 1) / kOrthoSmallCols;
                },
                [&](const Groups &g, uint32_t total) {
                    const dim3 n(total), b(256);
                    if (from == 0 && to == a.steps)
                        small_apply_kernel<false, false><<<n, b, 0, s>>>(g, sp);
                    else if (from == 0)
                        small_apply_kernel<false, true><<<n, b, 0, s>>>(g, sp);
                    else if (to < a.steps)
                        small_apply_kernel<true, true><<<n, b, 0, s>>>(g, sp);
                    else
                        small_apply_kernel<true, false><<<n, b, 0, s>>>(g, sp);
                });
        if (st != TIDE_OK) return st;
    }
    return TIDE_OK;
}

tide_status run_ortho(const OrthoArgs &a, void *stream) {
    OrthoPlan plan;
    tide_status st = check_ortho(a, &plan);
    if (st != TIDE_OK) return st;
    if (plan.order.empty()) {
        clear_error();
        return TIDE_OK;
    }
    std::vector<OrthoGroup> groups, small, by_length;
    try {
        for (const OrthoGroup &g : plan.groups) (g.small() ? small : groups).push_back(g);
        by_length = longest_first(groups);
    } catch (const std::bad_alloc &) {
        return fail(TIDE_E_NOMEM, "tide_ortho: out of host memory");
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    Space sp;
    sp.base = static_cast<char *>(a.workspace);
    sp.pointers = reinterpret_cast<const Pointers *>(sp.base);
    sp.sums = reinterpret_cast<double *>(sp.base + plan.sums);
    sp.scales = reinterpret_cast<float2 *>(sp.base + plan.scales);
    double raised = 1.0;
    for (int i = 0; i < a.steps; i++) raised *= raises(a, i);
    sp.lo = raised > kOrthoRaisedHi;
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
        case kElemBf16: st = run_first<kElemBf16>(groups, small, sp, s); break;
        case kElemF16: st = run_first<kElemF16>(groups, small, sp, s); break;
        case kElemF32: st = run_first<kElemF32>(groups, small, sp, s); break;
    }
    if (st == TIDE_OK && !small.empty()) st = run_small(small, a, sp, s);
    for (int i = 0; i < a.steps && st == TIDE_OK && !groups.empty(); i++) {
        ProductArgs p;
        p.s = sp;
        p.ca = a.coefficients[3 * i];
        p.cb = a.coefficients[3 * i + 1];
        p.cc = a.coefficients[3 * i + 2];
        p.from = i % 2;
        p.first = i == 0;
        p.last = i == a.steps - 1;
        p.short_g = in_type(a.flags) != kElemF32;
        st = run_product<kGram>(by_length, p, s);
        if (st == TIDE_OK) st = run_product<kPoly>(groups, p, s);
        if (st == TIDE_OK) st = run_product<kApply>(groups, p, s);
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
