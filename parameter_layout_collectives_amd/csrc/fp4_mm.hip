// Matrix products over microscaled 4-bit blocks, and their entry points:
//   tide_mx_mm      Y[m, n]  = sum over k of X[m, k] W[n, k]    X, W in 4-bit blocks
//   tide_mx_linear  Y[m, n]  = sum over k of x[m, k] W[n, k]    x in bf16, or rounded to
//                                                                4-bit blocks on the way
//   tide_mx_mm_dx   dX[m, k] = sum over n of dY[m, n] W[n, k]   dY in bf16
//
// As in the 8-bit products, W takes the matrix instruction's row side, so that a
// lane's 4 results are neighbours in memory, and sums are held in fp32.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "block.h"
#include "block_device.h"
#include "fp4.h"
#include "mm_device.h"

namespace tide {
namespace {

// ---------------------------------------------------------------------------
// Y = X W^T with the 4-bit matrix instruction
// ---------------------------------------------------------------------------
//
// The scaled instruction (16 x 16 x 128) takes a scale byte per lane, which is one
// per 32 values of a row: exactly a 4-bit block's, so scales cost no arithmetic.
// Unlike its 8-bit form it holds sums in fp32: products of e2m1 numbers are
// multiples of 1/4 up to 36, so those under one pair of scales add without any
// loss, and between blocks the instruction keeps 24 bits.  Measured against exact
// sums, over random codes and scales 2^-20..2^20 apart: off by at most 2^-23.8 of the
// sum of the magnitudes, and 36 * 2^35 - 36 * 2^35 + 1 in three blocks is 1.
//
// A T x T tile of the output per workgroup of 4 waves, 2 x 2, in fragments of 32 x 32
// x 64: of the instruction's shapes the one that leaves most time between two issues
// of a wave, which stands alone on its SIMD at T = 256.  One step of the sum is 128
// columns: 64 bytes of a row, 4 chunks of 16, one block each.  Chunk h of row r lies at
// h ^ (r >> 3 & 3) in LDS, so that the rows that a read takes at a time fall into
// different banks.  Codes and scales go straight into LDS, BUFFERS steps deep: a load
// that misses the L2 takes longer than two steps.
// 8192 x 28672 x 8192: 0.86 to 0.91 ms, 4.2 to 4.5 PFLOP/s (bf16's library product reaches
// 1.58), matrix units busy 56% of the cycles at a clock of 1.8 GHz; with x's and W's
// turning 0.94 ms.  In steps of 256 columns, two of them in LDS, it took 2.3 ms; with 8
// waves in fragments of 16 x 16, 1.1.
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTileThreads = 256;

// Where a step finds an operand's codes (64 bytes of a row) or scales (4 bytes): the
// next row's `row` bytes further, the next step's `step` bytes.  As they lie in the
// operand row is its pitch; turned into [steps, rows, 64] and [steps, rows, 4], row is
// 64 and 4 and a load's lines of the cache are whole.
struct Way {
    const char *at;
    uint32_t row, step;
    int turned;
};
struct TilesLaunch : MmLaunch {
    Way ci, cj, si, sj;
};

template <int T>
struct Tiles {
    static constexpr int F = T / 2 / 32;                   // 32 x 32 fragments of a wave, each way
    static constexpr int LINES = 2 * F;                    // of a step: 2 x 64 columns
    static constexpr int D = LINES >= 8 ? 3 : 1, RING = D + 1;   // I fragments read ahead
    static constexpr int SLOTS = T * 4 / kTileThreads;     // 16-byte loads per thread and operand
    static constexpr int TILE = T * 64;                    // bytes of an operand's codes
    static constexpr int SLOADS = (2 * T / 64 + 3) / 4;    // loads of 64 rows' scales per wave
    static constexpr int BUFFER = 2 * TILE + SLOADS * 4 * 256;
    static constexpr int BUFFERS = T == 64 ? 8 : 4, LDS = BUFFERS * BUFFER;
    static constexpr int LOADS = 2 * SLOTS + SLOADS;       // spread over a step's lines
    static_assert(LINES % RING == 0, "a step starts at ring entry 0");

    struct From {                // a Way, for this thread
        __amdgpu_buffer_rsrc_t r;
        uint32_t v, rows, step;  // first slot; 64 rows, and a step, further
    };
    From ci, cj, si, sj;
    int lane, wave, wi, wj, fa;  // fa: a fragment's lane's part of its address
    int shift;                   // of this lane's byte in a word of scales
    f32x16 acc[F][F];

    // Load q of step s: scales first (64-row groups 0 .. T/64-1 are the tile's rows of
    // I, the others those of J), then codes of I and J.
    __device__ __forceinline__ void load(LDS_AS char *b, uint32_t s, int q) const {
        if (q < SLOADS) {
            const int w = wave + q * 4;                    // past the operands: unused
            const bool i = w < T / 64;
            const uint32_t k = i ? w : w - T / 64;
            direct_word(i ? si.r : sj.r, b + 2 * TILE + w * 256, i ? si.v : sj.v,
                        i ? k * si.rows + s * si.step : k * sj.rows + s * sj.step);
        } else if (q < LOADS) {
            const int c = q - SLOADS, k = c % SLOTS;
            const From &f = c < SLOTS ? ci : cj;
            direct_load(f.r, b + (c < SLOTS ? 0 : TILE) + (wave + k * 4) * 1024, f.v,
                        k * f.rows + s * f.step);
        }
    }
    // As direct_load, 4 bytes per lane.
    static __device__ __forceinline__ void direct_word(__amdgpu_buffer_rsrc_t r, LDS_AS char *to,
                                                       uint32_t at, uint32_t off) {
        const uint32_t lds = __builtin_amdgcn_readfirstlane(
            static_cast<uint32_t>(reinterpret_cast<uintptr_t>(to)));
        asm volatile(
            "s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
            :
            : "s"(lds), "v"(at), "s"(r), "s"(__builtin_amdgcn_readfirstlane(off))
            : "memory", "m0");
    }
    // All but this wave's newest N loads have landed, and every wave is here.
    template <int N>
    static __device__ __forceinline__ void wait() {
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" : : "n"(N) : "memory");
    }
    // The fragment of rows [32 f, 32 f + 32) of the wave's, columns [64 k, 64 k + 64) of
    // the step, n = k F + f: lane (r32, g) holds block 2 k + g of row r32.
    __device__ __forceinline__ u32x4 frag(const LDS_AS char *codes, int half, int n) const {
        return *reinterpret_cast<const LDS_AS u32x4 *>(codes + half * (TILE / 2) + n % F * 2048 +
                                                       (fa ^ n / F * 32));
    }
    // The scales of rows [row, row + 32): shifted, this lane's blocks g and 2 + g are in
    // bytes 0 and 2.
    __device__ __forceinline__ uint32_t scale(const LDS_AS char *words, int row) const {
        return *reinterpret_cast<const LDS_AS uint32_t *>(words + (row + (lane & 31)) * 4);
    }
    static __device__ __forceinline__ i32x8 wide(u32x4 v) {
        return i32x8{static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]),
                     static_cast<int>(v[3]), 0, 0, 0, 0};
    }
    struct Step {                // what is read ahead for a step
        u32x4 j[LINES];
        uint32_t sj[F], si[F];
    };
    __device__ __forceinline__ void scales(Step &r, const LDS_AS char *b, int n) const {
        r.si[n] = scale(b + 2 * TILE, wi * (T / 2) + n * 32);
        r.sj[n] = scale(b + 2 * TILE, T + wj * (T / 2) + n * 32);
    }
    // One step from `here`; `there` is the next one, s + BUFFERS - 1 goes to `to`, which
    // the barrier has just freed (its reads have all been multiplied).
    __device__ __forceinline__ void step(u32x4 *l, const Step &r, Step &next, const LDS_AS char *here,
                                         const LDS_AS char *there, LDS_AS char *to, uint32_t s) {
        // the next step has landed; newer are the loads of those behind it
        wait<(BUFFERS - 3) * LOADS>();
        // not where they are read, which would wait for them
        int sj[F], si[F];
#pragma unroll
        for (int y = 0; y < F; y++) {
            sj[y] = static_cast<int>(r.sj[y] >> shift);
            si[y] = static_cast<int>(r.si[y] >> shift);
        }
#pragma unroll
        for (int n = 0; n < LINES; n++) {
            l[(n + D) % RING] = n + D < LINES ? frag(here, wi, n + D) : frag(there, wi, n + D - LINES);
            next.j[n] = frag(there + TILE, wj, n);
            if (n < F) scales(next, there, n);
            const int x = n % F, k = n / F;
#pragma unroll
            for (int y = 0; y < F; y++) {
                if (k == 0)
                    acc[x][y] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        wide(r.j[y]), wide(l[n % RING]), acc[x][y], 4, 4, 0, sj[y], 0, si[x]);
                else
                    acc[x][y] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        wide(r.j[F + y]), wide(l[n % RING]), acc[x][y], 4, 4, 2, sj[y], 2, si[x]);
                if (y == 0) {
#pragma unroll
                    for (int q = n * LOADS / LINES; q < (n + 1) * LOADS / LINES; q++)
                        load(to, s + BUFFERS - 1, q);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    __device__ __forceinline__ void run(LDS_AS char *lds, uint32_t s0, uint32_t s1) {
#pragma unroll
        for (int b = 0; b < BUFFERS - 1; b++)
#pragma unroll
            for (int q = 0; q < LOADS; q++) load(lds + b * BUFFER, s0 + b, q);
        wait<(BUFFERS - 2) * LOADS>();
        u32x4 l[RING];
        Step r0, r1;
#pragma unroll
        for (int n = 0; n < LINES; n++) r0.j[n] = frag(lds + TILE, wj, n);
#pragma unroll
        for (int n = 0; n < F; n++) scales(r0, lds, n);
#pragma unroll
        for (int n = 0; n < D; n++) l[n] = frag(lds, wi, n);
        // What lies past the last step is fetched and read as well (in bounds by the
        // descriptors, used by nothing), which keeps branches out of the loop.
        uint32_t here = 0, to = (BUFFERS - 1) * BUFFER, s = s0;
        auto after = [](uint32_t b) { return b == (BUFFERS - 1) * BUFFER ? 0 : b + BUFFER; };
        for (; s + 1 < s1; s += 2) {
            const uint32_t there = after(here), to2 = after(to);
            step(l, r0, r1, lds + here, lds + there, lds + to, s);
            here = after(there);
            step(l, r1, r0, lds + there, lds + here, lds + to2, s + 1);
            to = after(to2);
        }
        if (s < s1) step(l, r0, r1, lds + here, lds + after(here), lds + to, s);
        arrived();               // no load may still be on its way to LDS at the end,
        __syncthreads();         // nor a read of what the sums will overwrite
    }
};

// An operand's codes [rows, steps, 64 bytes] -> [steps, rows, 64 bytes] and scales
// [rows, steps, 4] -> [steps, rows, 4]: a workgroup takes 64 rows of 4 steps, a lane 16
// bytes of codes in each.
__global__ __launch_bounds__(256) void turn_kernel(const char *__restrict__ codes,
                                                   const char *__restrict__ scales, int64_t rows,
                                                   uint32_t steps, char *__restrict__ to,
                                                   char *__restrict__ sto) {
    const uint32_t fours = (steps + 3) / 4;
    const int64_t row = static_cast<int64_t>(blockIdx.x / fours) * 64 + (threadIdx.x >> 2);
    const int c = threadIdx.x & 3;
    const uint32_t s0 = blockIdx.x % fours * 4;
    if (row >= rows) return;
    const u32x4 *in = reinterpret_cast<const u32x4 *>(codes + row * steps * 64) + c;
    u32x4 v[4];
#pragma unroll
    for (int k = 0; k < 4; k++)
        if (s0 + k < steps) v[k] = in[(s0 + k) * 4];
    if (s0 + c < steps)
        *reinterpret_cast<uint32_t *>(sto + ((s0 + c) * rows + row) * 4) =
            *reinterpret_cast<const uint32_t *>(scales + (row * steps + s0 + c) * 4);
#pragma unroll
    for (int k = 0; k < 4; k++)
        if (s0 + k < steps) *(reinterpret_cast<u32x4 *>(to + ((s0 + k) * rows + row) * 64) + c) = v[k];
}

// x [rows, cols] -> turned 4-bit blocks, as tide_mx_quant and turn_kernel make them.  16
// lanes a unit of 128 columns, 8 values each; a workgroup takes 16 rows of 4 units, the
// next one the next units: 8192 x 8192 bf16 36 us, 4.7 TB/s (down the rows first 48).
template <int ET>
__global__ __launch_bounds__(256) void quant_turned_kernel(const char *__restrict__ x, int64_t rows,
                                                           int64_t cols, char *__restrict__ to,
                                                           char *__restrict__ sto, int vec) {
    constexpr int ES = ET == kElemF32 ? 4 : 2;
    const int64_t units = (cols + 127) / 128;
    const uint32_t fours = static_cast<uint32_t>((units + 3) / 4);
    const int64_t row = static_cast<int64_t>(blockIdx.x / fours) * 16 + (threadIdx.x >> 4);
    const int lane = threadIdx.x & 15;
    const int64_t unit0 = static_cast<int64_t>(blockIdx.x % fours) * 4;
    float v[4][8];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const int64_t c = (unit0 + k) * 128 + lane * 8;
        const int64_t left = max(min(cols - c, static_cast<int64_t>(8)), static_cast<int64_t>(0));
        const int n = row < rows ? static_cast<int>(left) : 0;
        load8<ET>(x + (row * cols + c) * ES, n, vec != 0, v[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; k++) {
        uint32_t scale;
        const uint32_t c = encode4(v[k], &scale);
        if (row >= rows || unit0 + k >= units) continue;
        const int64_t at = (unit0 + k) * rows + row;
        *reinterpret_cast<uint32_t *>(to + at * 64 + lane * 4) = c;
        if (lane % 4 == 0) sto[at * 4 + lane / 4] = static_cast<char>(scale);
    }
}

// The sums of a wave go through its part of LDS, 32 rows at a time: a lane holds 4
// neighbours of a row at a distance of 8, and leaves with 8.
template <int T>
__device__ __forceinline__ void store_sums(const MmLaunch &p, const Work &w, const Tiles<T> &e,
                                           LDS_AS char *lds) {
    constexpr int W = T / 2, PITCH = W * 4 + 16, F = Tiles<T>::F, PER = W / 8;
    static_assert(32 * PITCH <= Tiles<T>::LDS / 4, "a wave's part of LDS");
    lds += e.wave * (Tiles<T>::LDS / 4);
#pragma unroll
    for (int c = 0; c < F; c++) {
#pragma unroll
        for (int y = 0; y < F; y++)
#pragma unroll
            for (int q = 0; q < 4; q++)
                *reinterpret_cast<LDS_AS f32x4 *>(lds + (e.lane & 31) * PITCH + y * 128 + q * 32 +
                                                  (e.lane >> 5) * 16) =
                    f32x4{e.acc[c][y][4 * q], e.acc[c][y][4 * q + 1], e.acc[c][y][4 * q + 2],
                          e.acc[c][y][4 * q + 3]};
#pragma unroll
        for (int q = 0; q < 32 * PER / 64; q++) {
            const int row = q * (64 / PER) + e.lane / PER, col = e.lane % PER * 8;
            const LDS_AS f32x4 *v = reinterpret_cast<const LDS_AS f32x4 *>(lds + row * PITCH + col * 4);
            const f32x4 a = v[0], b = v[1];
            const int li = e.wi * W + c * 32 + row, lj = e.wj * W + col;
            const int64_t i = static_cast<int64_t>(w.r) * T + li, j = static_cast<int64_t>(w.c) * T + lj;
            if (w.part) {
                if (i < p.rows && j < p.cols) {
                    f32x4 *o = reinterpret_cast<f32x4 *>(w.part + li * T + lj);
                    o[0] = a;
                    o[1] = b;
                }
            } else if (p.out_bf16 && i < p.rows && p.cols - j >= 8) {
                *reinterpret_cast<half_u32x4 *>(p.out + (i * p.cols + j) * 2) =
                    half_u32x4{pack2(a[0], a[1]), pack2(a[2], a[3]), pack2(b[0], b[1]), pack2(b[2], b[3])};
            } else {
                store4(p, i, j, a);
                store4(p, i, j + 4, b);
            }
        }
    }
}

template <int T>
__global__ __launch_bounds__(kTileThreads, T == 256 ? 1 : 2) void tiles_kernel(TilesLaunch p) {
    typedef Tiles<T> E;
    __shared__ __attribute__((aligned(1024))) char lds[E::LDS];
    const int t = threadIdx.x, lane = t & 63;
    const int64_t steps = (p.sum + 127) / 128;
    const Work work = work_of<T>(p, steps);
    const int64_t i0 = static_cast<int64_t>(work.r) * T, j0 = static_cast<int64_t>(work.c) * T;

    // A buffer from the tile's first row on: as it lies to the tile's last row, turned
    // (below 2^31 bytes) to the last step's, with rows that are not the tile's own,
    // whose products nothing stores.
    const auto from = [&](const Way &w, int64_t first, int64_t all, uint32_t bytes, uint32_t v) {
        const int64_t n = w.turned ? (steps * all - first) * bytes
                                   : min(all - first, static_cast<int64_t>(T)) * w.row;
        return typename E::From{buffer_of(scalar(w.at + first * w.row), uniform(n)), v, 64 * w.row, w.step};
    };
    // A wave's load of codes fills 16 rows of 4 chunks: LDS chunk c of row r is chunk
    // c ^ (r >> 3 & 3) of memory.
    const uint32_t chunk = ((t & 3) ^ (t >> 5 & 3)) * 16;
    E e;
    e.lane = lane;
    e.wave = __builtin_amdgcn_readfirstlane(t >> 6);
    e.wi = e.wave / 2;
    e.wj = e.wave % 2;
    e.ci = from(p.ci, i0, p.rows, 64, (t >> 2) * p.ci.row + chunk);
    e.cj = from(p.cj, j0, p.cols, 64, (t >> 2) * p.cj.row + chunk);
    e.si = from(p.si, i0, p.rows, 4, lane * p.si.row);
    e.sj = from(p.sj, j0, p.cols, 4, lane * p.sj.row);
    const int r = lane & 31, g = lane >> 5;
    e.fa = r * 64 + ((g ^ (r >> 3 & 3)) << 4);
    e.shift = 8 * g;
#pragma unroll
    for (int x = 0; x < E::F; x++)
#pragma unroll
        for (int y = 0; y < E::F; y++)
#pragma unroll
            for (int n = 0; n < 16; n++) e.acc[x][y][n] = 0.0f;
    e.run((LDS_AS char *)lds, uniform(work.s0), uniform(work.s1));
    store_sums<T>(p, work, e, (LDS_AS char *)lds);
}

// ---------------------------------------------------------------------------
// Y = x W^T for few rows of x
// ---------------------------------------------------------------------------
//
// W's bytes bound it (1 x 14336 x 4096: 9.5 us, 31 MB at 3.3 TB/s, of which 2 us are the
// launch's start and 1 the join).  Each workgroup takes 16 rows of W and all of x's, up
// to 16; its waves cut the sum into groups of GB units of 128 columns and join through
// LDS in wave order.  Codes go from memory to registers as 16-byte loads, one block
// each, become bf16 there (exactly) and enter the bf16 instruction; the k-order inside a
// load is the same on both sides.
//
// SRC: where x comes from.  kPadded: bf16 rows of whole units in memory.  Else an
// element type: every workgroup reads x itself and holds it in LDS as bf16, rounded
// to 4-bit blocks with QUANT, while its first codes of W are on their way.
constexpr int kFewWaves = 8;
constexpr int kPadded = -1;

// 8 values of a block shared by 4 lanes, rounded to it, as bf16.
__device__ __forceinline__ bf16x8 rounded8(const float *v) {
    uint32_t scale;
    const uint32_t c = encode4(v, &scale);
    return widen4(c, __uint_as_float(scale << 23));
}
__device__ __forceinline__ bf16x8 plain8(const float *v) {
    bf16x8 r;
#pragma unroll
    for (int i = 0; i < 8; i++) r[i] = static_cast<__bf16>(v[i]);
    return r;
}

typedef u32x4 word_u32x4 __attribute__((aligned(4)));

template <int SRC, bool QUANT>
__global__ __launch_bounds__(kFewWaves * 64) void few_kernel(MmLaunch p) {
    constexpr bool MADE = SRC != kPadded;
    constexpr int GB = 4;                            // units in a group
    extern __shared__ __attribute__((aligned(16))) char made[];
    __shared__ __attribute__((aligned(16))) f32x4 part[kFewWaves][64];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int r16 = lane & 15, g = lane >> 4;
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * 16;
    const int nb = static_cast<int>((p.sum + 127) / 128);
    const int64_t wrow = min(j0 + r16, p.cols - 1);
    const char *w = p.b + wrow * p.b_pitch + g * 16;
    const char *ws = p.bs + wrow * p.bs_pitch;
    u32x4 wv[GB], wsc;
    // A whole group's scales in one load: each takes a line of the cache per row.
    auto load_w = [&](int b, int n) {
        if (n == GB) {
            wsc = *reinterpret_cast<const word_u32x4 *>(ws + b * 4);
        } else {
#pragma unroll
            for (int q = 0; q < GB; q++)
                if (q < n) wsc[q] = *reinterpret_cast<const uint32_t *>(ws + (b + q) * 4);
        }
#pragma unroll
        for (int q = 0; q < GB; q++)
            if (q < n) wv[q] = *reinterpret_cast<const u32x4 *>(w + (b + q) * 64);
    };
    int b = wave * GB;
    if (b < nb) load_w(b, min(nb - b, GB));

    const char *x;
    if (!MADE) {
        x = p.a + min(static_cast<int64_t>(r16), p.rows - 1) * p.a_pitch + g * 64;
    } else {
        // a pitch of 16 bytes more than a row, so that 16 rows' pieces lie in
        // different banks
        constexpr int ES = SRC == kElemF32 ? 4 : 2;
        const int rows = static_cast<int>(p.rows), units = rows * nb, pitch = nb * 256 + 16;
        for (int u0 = 0; u0 < units; u0 += kFewWaves * 4) {
            const int u = u0 + (t >> 4), row = u / nb, unit = u % nb, c = unit * 128 + (t & 15) * 8;
            const int left = u < units ? static_cast<int>(min(p.sum - c, static_cast<int64_t>(8))) : 0;
            float v[8];
            load8<MADE ? SRC : kElemBf16>(p.a + (static_cast<int64_t>(row) * p.sum + c) * ES, left,
                                          p.aligned != 0, v);
            const bf16x8 h = QUANT ? rounded8(v) : plain8(v);
            if (u < units) *reinterpret_cast<bf16x8 *>(made + row * pitch + c * 2) = h;
        }
        __syncthreads();
        x = made + min(r16, rows - 1) * pitch + g * 64;
    }

    f32x4 acc = {0, 0, 0, 0};
    // Units b .. b + n - 1, n = GB with FULL.
    auto group = [&](auto full, int n) {
        constexpr bool FULL = decltype(full)::value;
#pragma unroll
        for (int q = 0; q < GB; q++) {
            if (!FULL && q >= n) break;
            const float s = __uint_as_float((wsc[q] >> (8 * g) & 0xffu) << 23);
#pragma unroll
            for (int e = 0; e < 4; e++)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    widen4(wv[q][e], s),
                    *reinterpret_cast<const bf16x8 *>(x + (b + q) * 256 + e * 16), acc, 0, 0, 0);
        }
    };
    for (; b < nb; b += kFewWaves * GB) {
        const int n = min(nb - b, GB);
        if (n == GB)
            group(std::true_type{}, GB);
        else
            group(std::false_type{}, n);
        const int next = b + kFewWaves * GB;
        if (next < nb) load_w(next, min(nb - next, GB));
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave > 0) return;
    f32x4 sum = part[0][lane];
#pragma unroll
    for (int q = 1; q < kFewWaves; q++) sum += part[q][lane];
    store4(p, r16, j0 + g * 4, sum);
}

// ---------------------------------------------------------------------------
// Y = x W^T for some rows of x
// ---------------------------------------------------------------------------
//
// W's bytes should still bound it, but x, which every row of W meets, is too large to
// be read again for each 16 of them.  A workgroup takes 32 rows of W per wave and a
// piece of the sum.  x's rows (16 MT) go through registers into LDS, GU units of 128
// columns (16 KB, a group) at a time, and every wave multiplies by them; W's codes go
// from memory to registers, become bf16 there and are multiplied at once.  Both are
// asked for two groups ahead (four ahead, or two workgroups on a compute unit, are no
// faster).  The pieces' sums meet in the workspace.  32 x 8192 x 28672: 34.3 us, of which
// the second launch takes 4 to 5; W's 125 MB come at 4.1 TB/s (a copy of 128 MiB: 5.3), and
// x's 1.8 MB once for each 128 rows of W, 117 MB, through the L2.  Alone, without x,
// products and scales, the loads of W take 24 to 27.
//
// LDS: a row's unit is 16 chunks of 16 bytes, chunk c of row r at c ^ strip_key(r), so
// that the lanes that a read takes at a time fall into different banks.
struct StripLaunch : MmLaunch {
    int64_t units;               // of 128 columns
    uint32_t groups;             // workgroups along W's rows
};

__device__ __forceinline__ int strip_key(int r) { return (r & 3) | ((r & 8) ? 12 : 0); }

template <int MT>
__global__ __launch_bounds__(kStripWaves * 64, 2) void strip_kernel(StripLaunch p) {
    constexpr int GU = 4 / MT, BUFFER = 16384;
    constexpr int SLOTS = BUFFER / (kStripWaves * 1024);   // of 16 bytes of x, per thread
    struct Rows {                // of x, in one group
        u32x4 v[SLOTS];
    };
    constexpr int AHEAD = 2;     // groups of W
    constexpr int PITCH = 80;    // of a row's scales in LDS
    struct Codes {               // a wave's 2 x 16 rows of W in one group
        u32x4 v[GU][2];
    };
    __shared__ __attribute__((aligned(1024))) char mem[2 * BUFFER + kStripRows * PITCH];
    LDS_AS char *const lds = (LDS_AS char *)mem;
    const int t = threadIdx.x, lane = t & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const uint32_t group = uniform(blockIdx.x % p.groups), piece = uniform(blockIdx.x / p.groups);
    const int64_t j0 = static_cast<int64_t>(uniform(group * kStripWaves + wave)) * 32;
    const int u0 = static_cast<int>(uniform(piece * p.chunk));
    const int u1 = static_cast<int>(uniform(min((piece + 1) * p.chunk, p.units)));

    // x: a wave's slot is 4 rows of one unit; rows and columns past the end are zeros
    const __amdgpu_buffer_rsrc_t rx = buffer_of(scalar(p.a), uniform(p.rows * p.a_pitch));
    auto ask_x = [&](Rows &x, int it) {
#pragma unroll
        for (int q = 0; q < SLOTS; q++) {
            const int k = q * static_cast<int>(kStripWaves) + wave;
            const int u = u0 + it * GU + k / (4 * MT), row = k % (4 * MT) * 4 + g;
            const int c = u * 128 + (r16 ^ strip_key(row)) * 8;
            const uint32_t at = static_cast<uint32_t>(row * p.a_pitch) + c * 2;
            x.v[q] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                   rx, u < u1 && row < p.rows ? at : 0x80000000u, 0, 0));
        }
    };
    auto put_x = [&](const Rows &x, int buffer) {
#pragma unroll
        for (int q = 0; q < SLOTS; q++)
            *reinterpret_cast<LDS_AS u32x4 *>(lds + buffer * BUFFER + (q * kStripWaves + wave) * 1024 +
                                              lane * 16) = x.v[q];
    };
    // W: rows past the last one are zeros; units past the row's end are the next
    // row's, which nothing multiplies
    const int64_t there = max(min(p.cols - j0, static_cast<int64_t>(32)), static_cast<int64_t>(0));
    const __amdgpu_buffer_rsrc_t rw = buffer_of(scalar(p.b + j0 * p.b_pitch), uniform(there * p.b_pitch));
    const __amdgpu_buffer_rsrc_t rs = buffer_of(scalar(p.bs + j0 * p.bs_pitch), uniform(there * p.bs_pitch));
    uint32_t wat[2], sat[2];
#pragma unroll
    for (int f = 0; f < 2; f++) {
        wat[f] = (f * 16 + r16) * static_cast<uint32_t>(p.b_pitch) + g * 16;
        sat[f] = (f * 16 + r16) * static_cast<uint32_t>(p.bs_pitch) + g * 16;
    }
    auto ask_w = [&](Codes &c, int it) {
        const uint32_t u = u0 + it * GU;
#pragma unroll
        for (int f = 0; f < 2; f++)
#pragma unroll
            for (int q = 0; q < GU; q++)
                c.v[q][f] = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, wat[f], (u + q) * 64, 0));
    };
    // Scales of 16 units at a time, which a row's 4 lanes share out and each wave reads
    // back by bytes from its own part of LDS: a load per group would take a line of the
    // cache for each row and 4 or 8 bytes.
    u32x4 sc[2];
    LDS_AS char *const sto = lds + 2 * BUFFER + (wave * 32 + r16) * PITCH;
    auto ask_scales = [&](int u) {
#pragma unroll
        for (int f = 0; f < 2; f++)
            sc[f] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, sat[f], (u0 + u) * 4, 0));
    };
    auto put_scales = [&] {
#pragma unroll
        for (int f = 0; f < 2; f++)
            *reinterpret_cast<LDS_AS u32x4 *>(sto + f * 16 * PITCH + g * 16) = sc[f];
    };
    f32x4 acc[2][MT];
#pragma unroll
    for (int f = 0; f < 2; f++)
#pragma unroll
        for (int m = 0; m < MT; m++) acc[f][m] = f32x4{0, 0, 0, 0};
    const int key = strip_key(r16);
    auto multiply = [&](auto full, const Codes &c, int it, int buffer) {
        const LDS_AS char *const x = lds + buffer * BUFFER + r16 * 256;
#pragma unroll
        for (int q = 0; q < GU; q++) {
            if (!decltype(full)::value && u0 + it * GU + q >= u1) break;
            float s[2];
#pragma unroll
            for (int f = 0; f < 2; f++)
                s[f] = __uint_as_float(
                    static_cast<uint32_t>(*reinterpret_cast<const LDS_AS uint8_t *>(
                        sto + f * 16 * PITCH + (it * GU + q) % 16 * 4 + g)) << 23);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                bf16x8 xf[MT];
#pragma unroll
                for (int m = 0; m < MT; m++)
                    xf[m] = *reinterpret_cast<const LDS_AS bf16x8 *>(x + (q * MT + m) * 4096 +
                                                                     (((g * 4 + e) ^ key) << 4));
#pragma unroll
                for (int f = 0; f < 2; f++) {
                    const bf16x8 wf = widen4(c.v[q][f][e], s[f]);
#pragma unroll
                    for (int m = 0; m < MT; m++)
                        acc[f][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[m], acc[f][m], 0, 0, 0);
                }
            }
        }
    };
    Rows x[2];
    Codes c[AHEAD];
    ask_x(x[0], 0);
    ask_scales(0);
    ask_w(c[0], 0);
    ask_x(x[1], 1);
#pragma unroll
    for (int k = 1; k < AHEAD; k++) ask_w(c[k], k);
    put_x(x[0], 0);
    ask_x(x[0], 2);
    // Group `it` of x is in LDS, and every wave has read the buffer that is filled next.
    auto turns = [&](auto full, int it) {
#pragma unroll
        for (int k = 0; k < AHEAD; k++) {
            __syncthreads();
            if (k == 0 && it * GU % 16 == 0) {
                put_scales();
                ask_scales(it * GU + 16);
            }
            put_x(x[(k + 1) % 2], (k + 1) % 2);
            ask_x(x[(k + 1) % 2], it + k + 3);
            __builtin_amdgcn_sched_barrier(0);
            multiply(full, c[k], it + k, k % 2);
            ask_w(c[k], it + k + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    int it = 0;
    for (; u0 + (it + AHEAD) * GU <= u1; it += AHEAD) turns(std::true_type{}, it);
    if (u0 + it * GU < u1) turns(std::false_type{}, it);

    float *const part = p.splits > 1 ? p.partial + piece * p.rows * p.cols : nullptr;
#pragma unroll
    for (int f = 0; f < 2; f++)
#pragma unroll
        for (int m = 0; m < MT; m++) {
            const int64_t row = m * 16 + r16, col = j0 + f * 16 + g * 4;
            if (!part) {
                store4(p, row, col, acc[f][m]);
            } else if (row < p.rows) {
                float *o = part + row * p.cols + col;
                if (p.cols - col >= 4)
                    *reinterpret_cast<row_f32x4 *>(o) = acc[f][m];
                else
                    for (int k = 0; k < 4; k++)
                        if (col + k < p.cols) o[k] = acc[f][m][k];
            }
        }
}

// Adds the pieces' sums [splits, rows, cols] in their order.
__global__ __launch_bounds__(256) void strip_join_kernel(MmLaunch p) {
    const int64_t all = p.rows * p.cols;
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
    if (at >= all) return;
    f32x4 sum = {0, 0, 0, 0};
    if (all - at >= 4) {
#pragma unroll 8
        for (int q = 0; q < p.splits; q++)
            sum += *reinterpret_cast<const row_f32x4 *>(p.partial + q * all + at);
    } else {
        for (int q = 0; q < p.splits; q++)
            for (int k = 0; k < all - at; k++) sum[k] += p.partial[q * all + at + k];
    }
    p.rows = 1;                  // the output as one row
    p.cols = all;
    store4(p, 0, at, sum);
}

// x [rows, cols] -> bf16 rows of whole units of 128 columns, zeros past the last
// column, rounded to 4-bit blocks with QUANT.  16 lanes a unit.
template <int ET, bool QUANT>
__global__ __launch_bounds__(256) void pad_kernel(const char *__restrict__ x, int64_t rows,
                                                  int64_t cols, char *__restrict__ out, int vec) {
    constexpr int ES = ET == kElemF32 ? 4 : 2;
    const int64_t nb = (cols + 127) / 128, u = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
    const int64_t row = u / nb, c = u % nb * 128 + (threadIdx.x & 15) * 8;
    const bool there = row < rows;
    float v[8];
    load8<ET>(x + (row * cols + c) * ES,
              there ? static_cast<int>(min(cols - c, static_cast<int64_t>(8))) : 0, vec != 0, v);
    const bf16x8 h = QUANT ? rounded8(v) : plain8(v);
    if (there) *reinterpret_cast<bf16x8 *>(out + (row * nb * 128 + c) * 2) = h;
}

// The values of 4-bit blocks as bf16 rows of whole units.
__global__ __launch_bounds__(256) void widen_kernel(const char *__restrict__ codes,
                                                    const char *__restrict__ scales, int64_t blocks,
                                                    char *__restrict__ out) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;   // 8 values each
    if (i >= blocks * 4) return;
    const uint32_t s = static_cast<uint8_t>(scales[i / 4]);
    *reinterpret_cast<bf16x8 *>(out + i * 16) =
        widen4(*reinterpret_cast<const uint32_t *>(codes + i * 4), __uint_as_float(s << 23));
}

template <Mode MI, Mode MJ>
void launch_wide(const MmLaunch &p, int tile, dim3 grid, hipStream_t s) {
    if (tile == 256)
        wide_kernel<MI, MJ, 256, 2, 4, true><<<grid, dim3(512), 0, s>>>(p);
    else if (tile == 128 && p.aligned)
        wide_kernel<MI, MJ, 128, 2, 2, true><<<grid, dim3(256), 0, s>>>(p);
    else if (tile == 128)
        wide_kernel<MI, MJ, 128, 2, 2, false><<<grid, dim3(256), 0, s>>>(p);
    else if (p.aligned)
        wide_kernel<MI, MJ, 64, 2, 2, true><<<grid, dim3(256), 0, s>>>(p);
    else
        wide_kernel<MI, MJ, 64, 2, 2, false><<<grid, dim3(256), 0, s>>>(p);
}

// x in bf16 rows of whole units.
void launch_strips(const MmLaunch &mm, const MmChoice &c, char *partial, hipStream_t s) {
    StripLaunch p = {mm, block_count(mm.sum), static_cast<uint32_t>((mm.cols + kStripRows - 1) / kStripRows)};
    p.sum = p.units * 128;
    p.chunk = c.chunk;
    p.splits = c.splits;
    p.partial = reinterpret_cast<float *>(partial);
    const dim3 g(p.groups * c.splits), b(kStripWaves * 64);
    if (p.rows <= 16)
        strip_kernel<1><<<g, b, 0, s>>>(p);
    else if (p.rows <= 32)
        strip_kernel<2><<<g, b, 0, s>>>(p);
    else
        strip_kernel<4><<<g, b, 0, s>>>(p);
    if (c.splits > 1)
        strip_join_kernel<<<dim3(static_cast<unsigned>((p.rows * p.cols + 1023) / 1024)), dim3(256),
                            0, s>>>(p);
}

template <int ET>
void launch_pad(const char *x, int64_t M, int64_t K, char *out, bool quant, hipStream_t s) {
    const dim3 g(static_cast<unsigned>((M * block_count(K) + 15) / 16)), b(256);
    if (quant)
        pad_kernel<ET, true><<<g, b, 0, s>>>(x, M, K, out, K % 8 == 0);
    else
        pad_kernel<ET, false><<<g, b, 0, s>>>(x, M, K, out, K % 8 == 0);
}

template <int ET>
void launch_in_one(const MmLaunch &p, bool quant, hipStream_t s) {
    const dim3 g(static_cast<unsigned>((p.cols + 15) / 16)), b(kFewWaves * 64);
    const unsigned lds = static_cast<unsigned>(p.rows * (2 * block_cols(p.sum) + 16));
    if (quant)
        few_kernel<ET, true><<<g, b, lds, s>>>(p);
    else
        few_kernel<ET, false><<<g, b, lds, s>>>(p);
}

tide_status run_fp4(Fp4Op op, const char *name, const Fp4Args &a, void *stream) {
    tide_status st = check_fp4(op, name, a);
    if (st != TIDE_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    MmLaunch p = {};
    p.rows = a.M;
    p.cols = op == kFp4Dx ? a.K : a.N;
    p.sum = op == kFp4Dx ? a.N : a.K;
    if (p.rows == 0 || p.cols == 0) {
        clear_error();
        return TIDE_OK;
    }
    p.out = static_cast<char *>(a.out);
    p.out_bf16 = (a.flags & TIDE_F_OUT_BF16) != 0;
    if (p.sum == 0) {
        const int64_t n = p.rows * p.cols;
        const unsigned flat = static_cast<unsigned>(std::min<int64_t>((n + 1023) / 1024, kCus * 8));
        zero_kernel<<<dim3(flat), dim3(256), 0, s>>>(p.out, n, p.out_bf16 ? 2 : 4);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return hip_fail((std::string(name) + ": zeros").c_str(), e);
        clear_error();
        return TIDE_OK;
    }
    const bool quant = (a.flags & TIDE_F_QUANT_X) != 0;
    const ElemType in = in_type(a.flags);
    const bool aligned = op == kFp4Mm || quant ||
                         (reinterpret_cast<uintptr_t>(a.a) % 16 == 0 && (op == kFp4Dx ? a.N : a.K) % 8 == 0);
    const Fp4Choice c = fp4_choose(op, a.M, a.N, a.K, a.flags, aligned, a.workspace_bytes);
    p.a = static_cast<const char *>(a.a);
    p.as = static_cast<const char *>(a.a_scales);
    p.a_pitch = op == kFp4Mm || quant ? kFours.code_bytes(a.K) : 2 * (op == kFp4Dx ? a.N : a.K);
    p.as_pitch = kFours.scale_bytes(a.K);
    p.b = static_cast<const char *>(a.b);
    p.bs = static_cast<const char *>(a.b_scales);
    p.b_pitch = kFours.code_bytes(a.K);
    p.bs_pitch = kFours.scale_bytes(a.K);
    p.aligned = aligned;
    char *const ws = static_cast<char *>(a.workspace);
    const char *const x = p.a;
    if (c.kernel == kFp4SkinnyInOne) {
        p.aligned = a.K % 8 == 0;      // x is read in whole vectors
        switch (in) {
            case kElemBf16: launch_in_one<kElemBf16>(p, quant, s); break;
            case kElemF16: launch_in_one<kElemF16>(p, quant, s); break;
            case kElemF32: launch_in_one<kElemF32>(p, quant, s); break;
        }
    } else if (c.kernel == kFp4Skinny || c.kernel == kFp4Strips) {
        p.a_pitch = block_cols(a.K) * 2;
        if (op == kFp4Mm) {
            const int64_t blocks = a.M * block_cols(a.K) / 32;
            widen_kernel<<<dim3(static_cast<unsigned>((blocks * 4 + 255) / 256)), dim3(256), 0, s>>>(
                x, p.as, blocks, ws);
            p.a = ws;
        } else if (quant || !fp4_whole(x, a.K)) {
            switch (in) {
                case kElemBf16: launch_pad<kElemBf16>(x, a.M, a.K, ws, quant, s); break;
                case kElemF16: launch_pad<kElemF16>(x, a.M, a.K, ws, quant, s); break;
                case kElemF32: launch_pad<kElemF32>(x, a.M, a.K, ws, quant, s); break;
            }
            p.a = ws;
        }
        if (c.kernel == kFp4Skinny)
            few_kernel<kPadded, false><<<dim3(static_cast<unsigned>((p.cols + 15) / 16)),
                                         dim3(kFewWaves * 64), 0, s>>>(p);
        else
            launch_strips(p, c.mm, ws + c.x, s);
    } else {
        if (quant && c.x_turned < 0) {
            if (a.workspace_bytes < c.x)
                return fail(TIDE_E_INVALID, std::string(name) + ": the workspace holds " +
                                                std::to_string(a.workspace_bytes) +
                                                " bytes, x's blocks need " + std::to_string(c.x));
            st = tide_mx_quant(x, a.M, a.K, ws, ws + c.x_scales,
                                a.flags & (TIDE_F_GRAD_F16 | TIDE_F_GRAD_F32), stream);
            if (st != TIDE_OK) return st;
            p.a = ws;
            p.as = ws + c.x_scales;
        }
        TilesLaunch q = {};
        if (c.kernel == kFp4Tiles) {
            // as they lie, or turned
            const int64_t steps = block_count(a.K);
            const unsigned fours = static_cast<unsigned>((steps + 3) / 4);
            auto ways = [&](const char *codes, const char *scales, int64_t rows, int64_t at, Way &cw, Way &sw) {
                cw = Way{codes, static_cast<uint32_t>(p.b_pitch), 64, 0};
                sw = Way{scales, static_cast<uint32_t>(p.bs_pitch), 4, 0};
                if (at < 0) return;
                char *const to = ws + at, *const sto = to + steps * rows * 64;
                if (quant && at == c.x_turned) {
                    const dim3 g(static_cast<unsigned>((rows + 15) / 16) * fours), b(256);
                    const int vec = a.K % 8 == 0;
                    switch (in) {
                        case kElemBf16: quant_turned_kernel<kElemBf16><<<g, b, 0, s>>>(x, rows, a.K, to, sto, vec); break;
                        case kElemF16: quant_turned_kernel<kElemF16><<<g, b, 0, s>>>(x, rows, a.K, to, sto, vec); break;
                        case kElemF32: quant_turned_kernel<kElemF32><<<g, b, 0, s>>>(x, rows, a.K, to, sto, vec); break;
                    }
                } else {
                    turn_kernel<<<dim3(static_cast<unsigned>((rows + 63) / 64) * fours), dim3(256), 0, s>>>(
                        codes, scales, rows, static_cast<uint32_t>(steps), to, sto);
                }
                cw = Way{to, 64, static_cast<uint32_t>(rows * 64), 1};
                sw = Way{sto, 4, static_cast<uint32_t>(rows * 4), 1};
            };
            ways(p.a, p.as, a.M, c.x_turned, q.ci, q.si);
            ways(p.b, p.bs, a.N, c.w_turned, q.cj, q.sj);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return hip_fail((std::string(name) + ": kernel launch").c_str(), e);
        }
        const int T = c.mm.tile;
        const int64_t tr = (p.rows + T - 1) / T, tc = (p.cols + T - 1) / T;
        const int64_t cut = (tr * tc - c.mm.direct) * c.mm.splits;
        p.chunk = c.mm.chunk;
        p.splits = c.mm.splits;
        p.direct = static_cast<uint32_t>(c.mm.direct);
        p.partial = reinterpret_cast<float *>(ws + c.x);
        p.tr = static_cast<uint32_t>(tr);
        p.tc = static_cast<uint32_t>(tc);
        const dim3 grid(static_cast<unsigned>(c.mm.direct + cut));
        static_cast<MmLaunch &>(q) = p;
        if (c.kernel == kFp4Tiles && T == 256)
            tiles_kernel<256><<<grid, dim3(kTileThreads), 0, s>>>(q);
        else if (c.kernel == kFp4Tiles && T == 128)
            tiles_kernel<128><<<grid, dim3(kTileThreads), 0, s>>>(q);
        else if (c.kernel == kFp4Tiles)
            tiles_kernel<64><<<grid, dim3(kTileThreads), 0, s>>>(q);
        else if (op == kFp4Dx)
            launch_wide<kBf16Along, kFoursAcross>(p, T, grid, s);
        else
            launch_wide<kBf16Along, kFoursAlong>(p, T, grid, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return hip_fail((std::string(name) + ": kernel launch").c_str(), e);
        if (cut) {
            const dim3 g(static_cast<unsigned>((tr * tc - c.mm.direct) * (T * T / 1024))), b(256);
            if (T == 256)
                join_kernel<256><<<g, b, 0, s>>>(p);
            else if (T == 128)
                join_kernel<128><<<g, b, 0, s>>>(p);
            else
                join_kernel<64><<<g, b, 0, s>>>(p);
        }
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return hip_fail((std::string(name) + ": kernel launch").c_str(), e);
    clear_error();
    return TIDE_OK;
}

}  // namespace
}  // namespace tide

using namespace tide;

extern "C" tide_status tide_mx_mm(const void *x_codes, const void *x_scales, int64_t m,
                                   const void *w_codes, const void *w_scales, int64_t n, int64_t k,
                                   void *out, uint32_t flags, void *workspace,
                                   int64_t workspace_bytes, void *stream) {
    return run_fp4(kFp4Mm, "tide_mx_mm",
                   Fp4Args{x_codes, x_scales, w_codes, w_scales, m, n, k, out, workspace,
                           workspace_bytes, flags},
                   stream);
}

extern "C" tide_status tide_mx_linear(const void *x, int64_t m, int64_t k, const void *w_codes,
                                       const void *w_scales, int64_t n, void *out, uint32_t flags,
                                       void *workspace, int64_t workspace_bytes, void *stream) {
    return run_fp4(kFp4Linear, "tide_mx_linear",
                   Fp4Args{x, nullptr, w_codes, w_scales, m, n, k, out, workspace, workspace_bytes,
                           flags},
                   stream);
}

extern "C" tide_status tide_mx_mm_dx(const void *dy, int64_t m, int64_t n, const void *w_codes,
                                      const void *w_scales, int64_t k, void *dx, uint32_t flags,
                                      void *workspace, int64_t workspace_bytes, void *stream) {
    return run_fp4(kFp4Dx, "tide_mx_mm_dx",
                   Fp4Args{dy, nullptr, w_codes, w_scales, m, n, k, dx, workspace, workspace_bytes,
                           flags},
                   stream);
}
