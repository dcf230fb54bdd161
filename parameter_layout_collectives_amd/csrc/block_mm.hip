// Matrix products over 8-bit blocks, and their entry points:
//   tide_block_mm      Y[m, n]  = sum over k of X[m, k] W[n, k]
//   tide_block_mm_dx   dX[m, k] = sum over n of dY[m, n] W[n, k]
//   tide_block_mm_dw   dW[n, k] = sum over m of dY[m, n] X[m, k]
// with X and W the values of their 8-bit blocks and dY in bf16.
//
// All three are out[i, j] = sum over c of I(i, c) J(c, j).  J is the 8-bit
// operand whose index runs along the output's rows in memory; it takes the
// matrix instruction's row side, so that a lane's 4 results are neighbours in
// memory.  Sums are held in fp32.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "block.h"
#include "block_device.h"

namespace tide {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
// Four values of an output row of any width: aligned as one value is.
typedef uint32_t row_u32x2 __attribute__((ext_vector_type(2), aligned(2)));
typedef __bf16 row_bf16x4 __attribute__((ext_vector_type(4), aligned(2)));

#define LDS_AS __attribute__((address_space(3)))

struct MmLaunch {
    const char *a, *as;          // I: X's codes and scales, or dY
    const char *b, *bs;          // J: codes and scales
    char *out;
    float *partial;              // pieces' sums, T x T each
    int64_t rows, cols, sum;     // of the output, and the length of the sum
    int64_t a_pitch, as_pitch;   // bytes between rows
    int64_t b_pitch, bs_pitch;
    int64_t chunk;               // steps of the sum in one piece of a cut tile
    int splits;                  // pieces of a cut tile
    uint32_t direct;             // tiles that are not cut: the first ones
    uint32_t tr, tc;             // tiles along rows and columns
    int out_bf16, accumulate, aligned;
};

// A value that is the same in all lanes, in a scalar register: 64-bit minima
// and divisions run in vector registers and would drag what follows there.
__device__ __forceinline__ uint32_t uniform(int64_t v) {
    return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
}

// What a workgroup computes: a tile of the output and a piece of its sum.
struct Work {
    uint32_t r, c;               // tile
    int64_t s0, s1;              // steps of the sum
    float *part;                 // where a piece's T x T sums go, or null for a whole tile
};

// Tiles are numbered so that 8 tile rows advance together.  The first `direct`
// are whole; workgroup IDs go to the 8 XCDs in turn and each XCD has its own L2,
// so every XCD takes one contiguous run of them, and the tiles it works on at
// one time share their operands' rows.  The others' pieces follow.
template <int T>
__device__ __forceinline__ Work work_of(const MmLaunch &p, int64_t steps) {
    const uint32_t id = blockIdx.x;
    Work w;
    uint32_t v;
    if (id < p.direct) {
        const uint32_t q = p.direct / 8, rm = p.direct % 8, x = id % 8;
        v = x * q + min(x, rm) + id / 8;
        w.s0 = 0;
        w.s1 = steps;
        w.part = nullptr;
    } else {
        const uint32_t k = id - p.direct, piece = uniform(k % p.splits);
        v = p.direct + k / p.splits;
        w.s0 = piece * p.chunk;
        w.s1 = min(w.s0 + p.chunk, steps);
        w.part = p.partial + static_cast<int64_t>(k) * T * T;
    }
    const uint32_t per = 8 * p.tc, g = v / per, in = v - g * per, h = min(8u, p.tr - 8 * g);
    w.r = uniform(8 * g + in % h);
    w.c = uniform(in / h);
    return w;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
}

// Stores 4 neighbouring results of one output row, as many as exist.
__device__ __forceinline__ void store4(const MmLaunch &p, int64_t row, int64_t col, f32x4 v) {
    const int64_t left = p.cols - col;
    if (row >= p.rows || left <= 0) return;
    const int64_t at = row * p.cols + col;
    if (p.out_bf16) {
        __bf16 *o = reinterpret_cast<__bf16 *>(p.out) + at;
        if (left >= 4) {
            if (p.accumulate) {
                const bf16x4 old = *reinterpret_cast<const row_bf16x4 *>(o);
                for (int i = 0; i < 4; i++) v[i] += static_cast<float>(old[i]);
            }
            *reinterpret_cast<row_u32x2 *>(o) = u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
        } else {
            for (int i = 0; i < 4; i++)
                if (i < left)
                    o[i] = static_cast<__bf16>(p.accumulate ? static_cast<float>(o[i]) + v[i] : v[i]);
        }
        return;
    }
    float *o = reinterpret_cast<float *>(p.out) + at;
    if (left >= 4) {
        if (p.accumulate) v += *reinterpret_cast<const row_f32x4 *>(o);
        *reinterpret_cast<row_f32x4 *>(o) = v;
    } else {
        for (int i = 0; i < 4; i++)
            if (i < left) o[i] = p.accumulate ? o[i] + v[i] : v[i];
    }
}

// A wave's 16 x 16 fragments of a tile: this lane's line of the first at (i, j).
template <int T, int FI, int FJ>
__device__ __forceinline__ void store_tile(const MmLaunch &p, const Work &w, int i, int j,
                                           const f32x4 (&acc)[FI][FJ]) {
#pragma unroll
    for (int x = 0; x < FI; x++)
#pragma unroll
        for (int y = 0; y < FJ; y++) {
            const int li = i + x * 16, lj = j + y * 16;
            const int64_t row = static_cast<int64_t>(w.r) * T + li;
            const int64_t col = static_cast<int64_t>(w.c) * T + lj;
            if (!w.part)
                store4(p, row, col, acc[x][y]);
            else if (row < p.rows && col < p.cols)
                *reinterpret_cast<f32x4 *>(w.part + li * T + lj) = acc[x][y];
        }
}

// The cut tiles: adds the pieces' sums in their order.  A workgroup takes 1024
// values of a tile.
template <int T>
__global__ __launch_bounds__(256) void join_kernel(MmLaunch p) {
    const uint32_t per_tile = T * T / 1024;
    const uint32_t k = blockIdx.x / per_tile;
    const uint32_t at = blockIdx.x % per_tile * 1024 + threadIdx.x * 4;
    const uint32_t v = p.direct + k;
    const uint32_t per = 8 * p.tc, g = v / per, in = v - g * per, h = min(8u, p.tr - 8 * g);
    const int64_t row = static_cast<int64_t>(8 * g + in % h) * T + at / T;
    const int64_t col = static_cast<int64_t>(in / h) * T + at % T;
    if (row >= p.rows || col >= p.cols) return;
    const float *s = p.partial + static_cast<int64_t>(k) * p.splits * T * T + at;
    f32x4 sum = *reinterpret_cast<const f32x4 *>(s);
#pragma unroll 4
    for (int q = 1; q < p.splits; q++)
        sum += *reinterpret_cast<const f32x4 *>(s + static_cast<int64_t>(q) * T * T);
    store4(p, row, col, sum);
}

// An empty sum: zeros.
__global__ __launch_bounds__(256) void zero_kernel(char *out, int64_t n, int es) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        if (es == 4)
            reinterpret_cast<float *>(out)[i] = 0.0f;
        else
            reinterpret_cast<uint16_t *>(out)[i] = 0;
    }
}

// ---------------------------------------------------------------------------
// Y = X W^T with the 8-bit matrix instruction (TIDE_F_SHORT_SUMS)
// ---------------------------------------------------------------------------
//
// One step of the sum is one block of 128 columns: the scaled instruction
// (16 x 16 x 128) takes both operands' e8m0 scales, so a block's scale costs no
// arithmetic.  But its sums keep fewer bits than fp32: 8 neighbouring products are
// lined up with the one under the largest exponent and cut 13 bits below it.  On
// normal data that loses 1.6e-5 of the result's norm, 100 times less than the
// bf16 output's own rounding; where large products cancel it can exceed the result
// (pairs of 448 * 448 that cancel among 392 products: off by 92 in about 200).  So
// this kernel runs only where the caller asks for it; without the flag sums are
// held in fp32 by the kernel below.
//
// A T x T tile of the output per workgroup, WI x WJ waves.  A row's 128 codes
// are 8 chunks of 16 bytes; chunk h of row r lies at h ^ (r & 7) in LDS, so the
// 16 lanes that read one chunk of 16 rows touch all banks.  Operand k-order
// inside a step is free as long as both sides agree: a lane reads chunks g and
// g + 4 (g = lane / 16).  Two buffers: the next step's codes travel straight into
// the other one while this one is multiplied.
//
// 256 x 256 tiles, 8192 x 8192 x 8192: 0.43 to 0.48 ms, 2.3 to 2.5 PFLOP/s (torch's
// product of the same 8-bit numbers without block scales: 3.2); 8192 x 28672 x
// 8192: 1.7 ms.  Counters there: matrix units busy 53 to 62% of the cycles, LDS 25
// to 30%, no bank conflicts, waits in 35 to 43% of the wave cycles, clock 1.8 to 2.1
// GHz.  Leaving out three quarters of the loads makes it 15%
// faster, leaving out most LDS reads nothing.  Slower here: 32 x 32 x 64
// fragments (6%), a burst of all loads behind the barrier (2%), a raised wave
// priority around the multiplications (3%).

// Buffer descriptor of `bytes` bytes at p (the same in all lanes): loads past
// its end give zeros.  The end is compared with the lane's offset plus the scalar
// one and does not wrap: checked on the card for every form of load used here,
// with sums past 2^32 too, as is that only the words past the end become zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const char *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(p), 0, static_cast<int>(bytes),
                                             0x00020000);
}

// This wave's loads have arrived, those into LDS among them.
__device__ __forceinline__ void arrived() {
    __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0); the other counters as they are
}

// Every wave's loads into LDS have landed, and every wave's reads of LDS are done.
// __syncthreads() alone need not wait for loads into LDS: the compiler counts
// them for reads that may alias, which the buffers' __restrict__ denies.
__device__ __forceinline__ void landed() {
    arrived();
    __syncthreads();
}

template <int T, int WI, int WJ>
struct Eight {
    static constexpr int NT = WI * WJ * 64, NW = WI * WJ;
    static constexpr int FI = T / WI / 16, FJ = T / WJ / 16;   // 16 x 16 fragments per wave
    static constexpr int SLOTS = T * 8 / NT;                   // 16-byte loads per thread and operand
    static constexpr int TILE = T * 128;                       // bytes of an operand's codes
    static constexpr int WORDS = 2 * T * 4;                    // and of both operands' scale words
    static constexpr int LDS = 4 * TILE + 2 * WORDS;
    static constexpr int SLOADS = 2 * T / NT;                  // scale words per thread
    // I's fragments (lines) go through a ring of registers, D ahead of the
    // multiplications.
    static constexpr int RING = 2, D = RING - 1;
    static_assert(FI % RING == 0 && SLOTS <= FI, "a step starts at ring entry 0");

    __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
    uint32_t vc, vs;             // this thread's first code slot, and its scale words' row
    uint32_t pitch, spitch;
    int wave, fa, fb, sa, sb;    // fragments and their scale words, in a buffer
    f32x4 acc[FI][FJ];

    // Part q of step s's codes (and with the last one the scale words) -> a
    // buffer (I's codes, J's, words).
    __device__ __forceinline__ void fetch(LDS_AS char *ta, LDS_AS char *tb, LDS_AS char *tw,
                                          uint32_t s, int q) const {
        const int at = (wave + q * NW) * 1024;
        const uint32_t off = q * (NT / 8) * pitch + s * 128;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (LDS_AS void *)(ta + at), 16, vc, off, 0, 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (LDS_AS void *)(tb + at), 16, vc, off, 0, 0);
        if (q < SLOTS - 1) return;
        // words 0 .. T-1 are the tile's rows of I, T .. 2T-1 those of J
#pragma unroll
        for (int k = 0; k < SLOADS; k++) {
            const int w = wave + k * NW, half = T / 64;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                w < half ? rsa : rsb, (LDS_AS void *)(tw + w * 256), 4, vs,
                (w < half ? w : w - half) * 64 * spitch + (s & ~3u), 0, 0);
        }
    }
    static __device__ __forceinline__ i32x8 frag(const LDS_AS char *at, int lo_at) {
        // chunk g + 4 of a row lies 64 bytes from chunk g, up or down
        const u32x4 lo = *reinterpret_cast<const LDS_AS u32x4 *>(at + lo_at);
        const u32x4 hi = *reinterpret_cast<const LDS_AS u32x4 *>(at + (lo_at ^ 64));
        return i32x8{static_cast<int>(lo[0]), static_cast<int>(lo[1]), static_cast<int>(lo[2]),
                     static_cast<int>(lo[3]), static_cast<int>(hi[0]), static_cast<int>(hi[1]),
                     static_cast<int>(hi[2]), static_cast<int>(hi[3])};
    }
    struct Rows {                // the J side of one step
        i32x8 v[FJ];
        int scale[FJ];
    };
    struct Line {                // one fragment of the I side
        i32x8 v;
        int scale;
    };
    __device__ __forceinline__ void rows(Rows &r, const LDS_AS char *b, const LDS_AS char *w,
                                         uint32_t s) const {
#pragma unroll
        for (int y = 0; y < FJ; y++) {
            r.v[y] = frag(b + y * 2048, fb);
            r.scale[y] = *reinterpret_cast<const LDS_AS uint8_t *>(w + sb + y * 64 + (s & 3));
        }
    }
    __device__ __forceinline__ void line(Line &l, const LDS_AS char *a, const LDS_AS char *w, int x,
                                         uint32_t s) const {
        l.v = frag(a + x * 2048, fa);
        l.scale = *reinterpret_cast<const LDS_AS uint8_t *>(w + sa + x * 64 + (s & 3));
    }
    __device__ __forceinline__ void multiply(int x, const Line &l, const Rows &r) {
#pragma unroll
        for (int y = 0; y < FJ; y++)
            acc[x][y] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                r.v[y], l.v, acc[x][y], 0, 0, 0, r.scale[y], 0, l.scale);
    }
    // Step s, whose first D lines and J rows are in registers: reads the rest from
    // its buffer (h*); once nothing of it is left to read, the first reads of step
    // s + 1 from the other (t*) begin under the multiplications that remain, and
    // step s + 2 starts travelling to h*.  Loads go out a part at a time: a burst
    // of them would hold up the reads behind it (issued in order, 16 cycles of the
    // address path each, 64 a step and workgroup).
    template <bool LAST>
    __device__ __forceinline__ void step(Line *l, const Rows &r, Rows &next, LDS_AS char *ha,
                                         LDS_AS char *hb, LDS_AS char *hw, LDS_AS char *ta,
                                         LDS_AS char *tb, LDS_AS char *tw, uint32_t s) {
#pragma unroll
        for (int x = 0; x < FI; x++) {
            if (x + D < FI) line(l[(x + D) % RING], ha, hw, x + D, s);
            if (!LAST && x + D == FI) {
                landed();
                rows(next, tb, tw, s + 1);
            }
            if (!LAST && x + D >= FI) line(l[(x + D) % RING], ta, tw, x + D - FI, s + 1);
            if (!LAST && x < SLOTS - 1) fetch(ta, tb, tw, s + 1, x + 1);
            multiply(x, l[x % RING], r);
            if (!LAST && x == FI - 1) fetch(ha, hb, hw, s + 2, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    __device__ __forceinline__ void run(LDS_AS char *__restrict__ a0, LDS_AS char *__restrict__ a1,
                                        LDS_AS char *__restrict__ b0, LDS_AS char *__restrict__ b1,
                                        LDS_AS char *__restrict__ w0, LDS_AS char *__restrict__ w1,
                                        uint32_t s0, uint32_t s1) {
#pragma unroll
        for (int q = 0; q < SLOTS; q++) fetch(a0, b0, w0, s0, q);
        fetch(a1, b1, w1, s0 + 1, 0);
        landed();
        Line l[RING];
        Rows r0, r1;
        rows(r0, b0, w0, s0);
#pragma unroll
        for (int x = 0; x < D; x++) line(l[x], a0, w0, x, s0);
        uint32_t s = s0;
        // What lies past the last step is fetched and read as well (in bounds by
        // the descriptors, used by nothing), which keeps branches out of the loop.
        for (; s + 1 < s1; s += 2) {
            step<false>(l, r0, r1, a0, b0, w0, a1, b1, w1, s);
            step<false>(l, r1, r0, a1, b1, w1, a0, b0, w0, s + 1);
        }
        if (s < s1) step<true>(l, r0, r1, a0, b0, w0, a1, b1, w1, s);
        landed();                // no load may still be on its way to LDS at the end
    }
};

template <int T, int WI, int WJ>
__global__ __launch_bounds__(WI * WJ * 64, 1) void eight_kernel(MmLaunch p) {
    typedef Eight<T, WI, WJ> E;
    __shared__ __attribute__((aligned(1024))) char lds[E::LDS];
    const int t = threadIdx.x, lane = t & 63;
    const int r16 = lane & 15, g = lane >> 4;
    const Work work = work_of<T>(p, (p.sum + 127) / 128);
    const int64_t i0 = static_cast<int64_t>(work.r) * T, j0 = static_cast<int64_t>(work.c) * T;
    const uint32_t s0 = uniform(work.s0), s1 = uniform(work.s1);
    const uint32_t ni = uniform(min(p.rows - i0, static_cast<int64_t>(T)));
    const uint32_t nj = uniform(min(p.cols - j0, static_cast<int64_t>(T)));

    E e;
    e.pitch = static_cast<uint32_t>(p.a_pitch);
    e.spitch = static_cast<uint32_t>(p.as_pitch);
    e.wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wi = e.wave / WJ, wj = e.wave % WJ;
    e.ra = buffer_of(p.a + i0 * e.pitch, ni * e.pitch);
    e.rb = buffer_of(p.b + j0 * e.pitch, nj * e.pitch);
    e.rsa = buffer_of(p.as + i0 * e.spitch, ni * e.spitch);
    e.rsb = buffer_of(p.bs + j0 * e.spitch, nj * e.spitch);
    // A wave's load fills 8 rows of 8 chunks: LDS chunk c of row r is chunk
    // c ^ (r & 7) of memory.
    e.vc = (t >> 3) * e.pitch + ((t & 7) ^ (t >> 3 & 7)) * 16;
    e.vs = lane * e.spitch;
    e.fa = (wi * (T / WI) + r16) * 128 + ((g ^ (r16 & 7)) << 4);
    e.fb = (wj * (T / WJ) + r16) * 128 + ((g ^ (r16 & 7)) << 4);
    e.sa = (wi * (T / WI) + r16) * 4;
    e.sb = (T + wj * (T / WJ) + r16) * 4;
#pragma unroll
    for (int x = 0; x < E::FI; x++)
#pragma unroll
        for (int y = 0; y < E::FJ; y++) e.acc[x][y] = f32x4{0, 0, 0, 0};
    // An operand's two buffers lie side by side: one address and constant offsets
    // (below 64 KB) reach both.
    LDS_AS char *const b = (LDS_AS char *)lds, *const w = b + 4 * E::TILE;
    e.run(b, b + E::TILE, b + 2 * E::TILE, b + 3 * E::TILE, w, w + E::WORDS, s0, s1);
    store_tile<T>(p, work, wi * (T / WI) + r16, wj * (T / WJ) + g * 4, e.acc);
}

// ---------------------------------------------------------------------------
// Products with bf16 factors
// ---------------------------------------------------------------------------
//
// 8-bit operands become bf16 on their way into LDS (exactly: code * 2^e is a
// bf16 number), so every product of the bf16 instruction is exact and only the
// fp32 sums round.  This is the kernel where a scale cannot go into the matrix
// instruction, because it changes along the sum (dX and dW: one scale per row
// of W or X and 128 columns, summed over rows), and for Y = X W^T, whose sums the
// 8-bit instruction would cut.
//
// 8192 x 8192 x 8192: dX 0.72 to 0.84 ms, dW 0.75 to 0.87 ms (torch's bf16 product
// on the same cards 0.67 to 0.73 ms, 0.90 to 0.98 ms with its left operand
// transposed), Y 0.81 to 0.90 ms; matrix units busy 62% of the cycles,
// clock 1.7 to 2.0 GHz.
//
// A step of the sum is 64 values.  LDS layouts of an operand's tile:
//   along   (sum index contiguous in memory): T rows of 64 bf16, 8 chunks of 16
//           bytes, chunk h of row r at h ^ (r & 7)
//   across  (sum index is the memory row): 64 rows of T bf16; a wave's 16 lanes
//           read 4 rows x 32 bytes with the transposing read, which hands each
//           lane 4 values along the sum.  The 32-byte piece h of row c lies at
//           h ^ ((c & 3) | (c >> 1 & 4)), or h ^ (c & 3) for T = 64, so the rows of
//           a read fall into different banks.
enum Mode { kBf16Along, kBf16Across, kCodesAlong, kCodesAcross };

__host__ __device__ constexpr bool is_across(Mode m) {
    return m == kBf16Across || m == kCodesAcross;
}
__host__ __device__ constexpr bool is_codes(Mode m) {
    return m == kCodesAlong || m == kCodesAcross;
}

template <int T>
__device__ __forceinline__ int swz_across(int c) {
    return T == 64 ? c & 3 : (c & 3) | ((c >> 1) & 4);
}

// 16 bytes per lane from r + at + off straight into LDS, from `to` on.  The
// builtin for it would make the compiler wait for the load before the next
// transposing read of LDS, of whatever buffer: it cannot tell that they do not
// meet.  An asm statement is not counted, which is safe: its only output is
// LDS, for which arrived() waits, and loads return in order, so a wait for a
// counted load is at worst longer than needed.
__device__ __forceinline__ void direct_load(__amdgpu_buffer_rsrc_t r, LDS_AS char *to, uint32_t at,
                                            uint32_t off) {
    const uint32_t lds = __builtin_amdgcn_readfirstlane(
        static_cast<uint32_t>(reinterpret_cast<uintptr_t>(to)));
    asm volatile(
        "s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
        :
        : "s"(lds), "v"(at), "s"(r), "s"(off)
        : "memory", "m0");
}

// One operand's way from memory to LDS, for a T-wide tile and NT threads, 16
// bytes at a time: fetch() asks for a step's bytes, put() stores one slot of
// them.  What lies outside the operand (rows or columns past its end) comes as
// zeros, by the buffer's bounds or by an offset beyond them, so nothing from
// there enters a sum.
template <Mode M, int T, int NT, bool ALIGNED>
struct Stage {
    static constexpr int EL = is_codes(M) ? 16 : 8;        // values in 16 bytes
    static constexpr int ES = is_codes(M) ? 1 : 2;
    static constexpr int SLOTS = T * 64 / EL / NT;         // slots per thread
    static constexpr int PER = is_across(M) ? T / EL : 64 / EL;   // slots in a memory row
    static constexpr int ROWS = NT / PER;                  // memory rows from one slot to the next
    static constexpr uint32_t OUTSIDE = 0x80000000u;       // past every buffer's end
    // bf16 whose 16-byte pieces are aligned goes straight into LDS: there a
    // wave's lanes fill consecutive pieces, so the swizzle picks the source.
    static constexpr bool DIRECT = !is_codes(M) && ALIGNED;

    const char *base, *sbase;    // along: the tile's first row; across: the operand
    uint32_t pitch, spitch;
    uint32_t lines;              // along: the tile's memory rows; across: those left of the sum
    int end;                     // along: values left of the sum from the slot's next one on
    uint32_t at0, sat0;          // across: bytes before the tile in a row
    uint32_t next;               // first value of the sum not yet asked for
    uint32_t off, soff;          // this thread's first slot
    int have;                    // across: values of the slot's row from its first one on
    int first;                   // first value of the slot
    int put_at;
    u32x4 v[SLOTS];
    uint32_t scale[is_codes(M) ? SLOTS : 1];

    // The tile's lines [at, at + T) of `count`, from step s0 on.  Sums are
    // below 2^31 and rows at most 2^23 bytes long, so the bytes of T rows fit
    // 32 bits.
    __device__ __forceinline__ void init(const char *p, const char *sp, int64_t pitch_,
                                         int64_t spitch_, int64_t at, int64_t count, int64_t sum_,
                                         uint32_t s0, int t) {
        pitch = static_cast<uint32_t>(pitch_);
        spitch = static_cast<uint32_t>(spitch_);
        const int row = t / PER;
        first = t % PER * EL;
        // the swizzles are their own inverses
        if (DIRECT) first = lds_at(row, t % PER) / 16 % PER * 8;
        off = row * pitch + first * ES;
        soff = row * spitch;
        put_at = lds_at(row, first / 8);
        next = s0 * 64;
        end = static_cast<int>(sum_) - static_cast<int>(next) - first;
        base = p;
        sbase = sp;
        if (is_across(M)) {
            at0 = static_cast<uint32_t>(at * ES);
            sat0 = static_cast<uint32_t>(at / kBlockCols);
            lines = static_cast<uint32_t>(sum_) - next;
            have = static_cast<int>(min(count - at - first, static_cast<int64_t>(EL)));
            if (have <= 0) off = OUTSIDE;
            soff += first / kBlockCols;
        } else {
            base += at * pitch_;
            sbase += at * spitch_;
            lines = uniform(min(count - at, static_cast<int64_t>(T)));
        }
    }

    // Asks for the next step, into registers or straight into `lds`.  Past the
    // last one: for nothing, by the bounds.
    __device__ __forceinline__ void fetch(LDS_AS char *lds, int wave) {
        // across: 64 memory rows from row `next`, from column byte at0 on;
        // along: all of the tile's rows, from value `next` on
        const char *p = base, *sp = sbase;
        uint32_t n = lines, skip = 0, sskip = 0;
        uint32_t at = off;
        int there = have;
        if (is_across(M)) {
            p += static_cast<uint64_t>(next) * pitch;
            sp += static_cast<uint64_t>(next) * spitch;
            n = min(lines, 64u);
            lines -= n;
            skip = at0;
            sskip = sat0;
        } else {
            skip = next * ES;
            sskip = next / kBlockCols;
            there = end;
            if (there <= 0) at = OUTSIDE;
            end -= 64;
        }
        next += 64;
        const __amdgpu_buffer_rsrc_t r = buffer_of(p, n * pitch);
#pragma unroll
        for (int q = 0; q < SLOTS; q++) {
            if (DIRECT) {
                direct_load(r, lds + (wave + q * (NT / 64)) * 1024, at, q * ROWS * pitch + skip);
            } else if (is_codes(M)) {
                v[q] = __builtin_amdgcn_raw_buffer_load_b128(r, at, q * ROWS * pitch + skip, 0);
            } else {
                v[q] = u32x4{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const uint32_t h = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(
                        r, i < there ? at + 2 * i : OUTSIDE, q * ROWS * pitch + skip, 0));
                    v[q][i / 2] |= h << (16 * (i & 1));
                }
            }
        }
        if (is_codes(M)) {
            const __amdgpu_buffer_rsrc_t rs = buffer_of(sp, n * spitch);
#pragma unroll
            for (int q = 0; q < SLOTS; q++)
                scale[q] = static_cast<uint8_t>(
                    __builtin_amdgcn_raw_buffer_load_b8(rs, soff, q * ROWS * spitch + sskip, 0));
        }
    }

    static __device__ __forceinline__ int lds_at(int r, int chunk) {   // 16-byte chunk of row r
        if (is_across(M))
            return r * T * 2 + ((((chunk >> 1) ^ swz_across<T>(r)) << 1 | (chunk & 1)) << 4);
        return r * 128 + ((chunk ^ (r & 7)) << 4);
    }

    __device__ __forceinline__ void put(LDS_AS char *lds, int q) const {
        // Slot q lies ROWS rows further: a multiple of 16, which leaves the
        // swizzles as they are (along, rows step by more than 8).
        static_assert(ROWS % 16 == 0, "slots keep their swizzle");
        LDS_AS char *to = lds + put_at + q * ROWS * (is_across(M) ? T * 2 : 128);
        if (!is_codes(M)) {
            *reinterpret_cast<LDS_AS u32x4 *>(to) = v[q];
            return;
        }
        const float s = __uint_as_float(scale[q] << 23);
        // the slot's first chunk is an even one: its other half is 16 bytes away,
        // up or (along, where the swizzle moves single chunks) down
        const int half = is_across(M) ? 16 : (put_at ^ 16) - put_at;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const uint32_t c = v[q][2 * h + i];
                w[2 * i] = __builtin_bit_cast(
                    uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, false));
                w[2 * i + 1] = __builtin_bit_cast(
                    uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, true));
            }
            *reinterpret_cast<LDS_AS u32x4 *>(h == 0 ? to : to + half) = w;
        }
    }

    // The 16 x 32 fragment of tile rows (or columns) [at, at + 16), sum values
    // [32 kk, 32 kk + 32): lane (r16, g) holds values 8 g + 0..7 of line r16.
    static __device__ __forceinline__ bf16x8 frag(const LDS_AS char *lds, int at, int kk, int lane) {
        const int r16 = lane & 15, g = lane >> 4;
        if (!is_across(M))
            return *reinterpret_cast<const LDS_AS bf16x8 *>(
                lds + (at + r16) * 128 + (((g ^ (r16 & 7)) << 4) ^ (kk << 6)));
        union {
            i16x4 h[2];
            bf16x8 v;
        } u;
        const int c = g * 8 + (r16 >> 2);        // the swizzle is the same for all kk and h
        const LDS_AS char *p = lds + lds_at(c, at / 8 + ((r16 & 3) >> 1)) + (r16 & 1) * 8;
#pragma unroll
        for (int h = 0; h < 2; h++)
            u.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (LDS_AS i16x4 *)(p + (kk * 32 + h * 4) * T * 2));
        return u.v;
    }
};

// As in the 8-bit kernel, the next step's first fragments are read under this
// step's last multiplications.  A step is two halves of 32 values; its 2 FI
// lines (a fragment of I each) run through the J fragments of their half.
// While step s is multiplied from one buffer, step s + 1 goes from registers
// to the other (or is on its way there directly); step s + 2 is asked for once
// the barrier has freed registers and buffer.
template <Mode MI, Mode MJ, int T, int WI, int WJ, bool ALIGNED>
struct Wide {
    static constexpr int NT = WI * WJ * 64;
    static constexpr int FI = T / WI / 16, FJ = T / WJ / 16;
    static constexpr int LINES = 2 * FI, RING = FI >= 4 ? 4 : 2, D = RING - 1;
    static constexpr int TILE = T * 128;                   // bytes of one operand's tile
    typedef Stage<MI, T, NT, ALIGNED> SI;
    typedef Stage<MJ, T, NT, true> SJ;
    static constexpr int IPUTS = SI::DIRECT ? 0 : SI::SLOTS, PUTS = IPUTS + SJ::SLOTS;
    static_assert(LINES % RING == 0 && D <= FI,
                  "a step starts at ring entry 0, and its first half is over when the next "
                  "step's J fragments replace it");

    SI si;
    SJ sj;
    int lane, wave, wi, wj;
    f32x4 acc[FI][FJ];

    // A buffer: I's tile and J's.  All four tiles are separate objects to the
    // compiler (run()'s __restrict__), so that reads and stores of one do not
    // wait for loads that travel to another.
    __device__ __forceinline__ void fetch(LDS_AS char *ti, LDS_AS char *tj) {
        sj.fetch(tj, wave);      // first: its registers are waited for first
        si.fetch(ti, wave);
    }
    __device__ __forceinline__ void put(LDS_AS char *ti, LDS_AS char *tj, int q) const {
        if (q < IPUTS)
            si.put(ti, q);
        else
            sj.put(tj, q - IPUTS);
    }
    __device__ __forceinline__ bf16x8 line(const LDS_AS char *b, int n) const {
        return SI::frag(b, wi * (T / WI) + n % FI * 16, n / FI, lane);
    }
    __device__ __forceinline__ void rows(bf16x8 *r, const LDS_AS char *b, int kk) const {
#pragma unroll
        for (int y = 0; y < FJ; y++) r[y] = SJ::frag(b, wj * (T / WJ) + y * 16, kk, lane);
    }
    // LAST: nothing is left to ask for.
    template <bool LAST>
    __device__ __forceinline__ void step(bf16x8 *l, bf16x8 (*r)[FJ], LDS_AS char *here_i,
                                         LDS_AS char *here_j, LDS_AS char *there_i,
                                         LDS_AS char *there_j) {
        rows(r[1], here_j, 1);
#pragma unroll
        for (int n = 0; n < LINES; n++) {
            if (n + D < LINES) l[(n + D) % RING] = line(here_i, n + D);
            // the stores, spread over the second half's lines before the barrier:
            // their loads had half a step to arrive
            constexpr int FROM = LINES / 2 - 1, TO = LINES - D - 1;
#pragma unroll
            for (int q = 0; q < PUTS; q++)
                if (!LAST && n == FROM + q * (TO - FROM) / PUTS) put(there_i, there_j, q);
            // The loads straight into LDS were asked for a step ago.  They are waited
            // for before others set out: a wait for all but a number of later loads
            // would hold only as long as the compiler keeps that number.
            if (SI::DIRECT && !LAST && n == TO) arrived();
            if (!LAST && n == TO) sj.fetch(here_j, wave);
            if (!LAST && n == TO && !SI::DIRECT) si.fetch(here_i, wave);
            if (!LAST && n + D == LINES) {
                __syncthreads();
                if (SI::DIRECT) si.fetch(here_i, wave);
                rows(r[0], there_j, 0);
            }
            if (!LAST && n + D >= LINES) l[(n + D) % RING] = line(there_i, n + D - LINES);
#pragma unroll
            for (int y = 0; y < FJ; y++)
                acc[n % FI][y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    r[n / FI][y], l[n % RING], acc[n % FI][y], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    __device__ __forceinline__ void run(LDS_AS char *__restrict__ i0, LDS_AS char *__restrict__ i1,
                                        LDS_AS char *__restrict__ j0, LDS_AS char *__restrict__ j1,
                                        uint32_t steps) {
        fetch(i0, j0);
#pragma unroll
        for (int q = 0; q < PUTS; q++) put(i0, j0, q);
        fetch(i1, j1);
        landed();
        bf16x8 l[RING], r[2][FJ];
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

template <Mode MI, Mode MJ, int T, int WI, int WJ, bool ALIGNED>
__global__ __launch_bounds__(WI * WJ * 64, 1) void wide_kernel(MmLaunch p) {
    typedef Wide<MI, MJ, T, WI, WJ, ALIGNED> K;
    __shared__ __attribute__((aligned(1024))) char lds[4 * K::TILE];
    const int t = threadIdx.x, lane = t & 63;
    const Work work = work_of<T>(p, (p.sum + 63) / 64);
    const int64_t i0 = static_cast<int64_t>(work.r) * T, j0 = static_cast<int64_t>(work.c) * T;
    const uint32_t s0 = uniform(work.s0), s1 = uniform(work.s1);
    // Codes exist up to the end of their last block.
    const int64_t whole = static_cast<int64_t>(127);
    const int64_t cols = MJ == kCodesAcross ? (p.cols + whole) & ~whole : p.cols;
    const int64_t isum = MI == kCodesAlong ? (p.sum + whole) & ~whole : p.sum;
    const int64_t jsum = MJ == kCodesAlong ? (p.sum + whole) & ~whole : p.sum;

    K k;
    k.wave = __builtin_amdgcn_readfirstlane(t >> 6);
    k.lane = lane;
    k.wi = k.wave / WJ;
    k.wj = k.wave % WJ;
    k.si.init(p.a, p.as, p.a_pitch, p.as_pitch, i0, p.rows, isum, s0, t);
    k.sj.init(p.b, p.bs, p.b_pitch, p.bs_pitch, j0, cols, jsum, s0, t);
#pragma unroll
    for (int x = 0; x < K::FI; x++)
#pragma unroll
        for (int y = 0; y < K::FJ; y++) k.acc[x][y] = f32x4{0, 0, 0, 0};
    // I's two buffers, then J's: one address and constant offsets (below 64 KB)
    // reach both buffers of an operand.
    LDS_AS char *const b = (LDS_AS char *)lds;
    k.run(b, b + K::TILE, b + 2 * K::TILE, b + 3 * K::TILE, s1 - s0);
    const int r16 = lane & 15, g = lane >> 4;
    store_tile<T>(p, work, k.wi * (T / WI) + r16, k.wj * (T / WJ) + g * 4, k.acc);
}

// ---------------------------------------------------------------------------
// Y = X W^T for few rows of X
// ---------------------------------------------------------------------------
//
// W's bytes bound it: each workgroup takes 16 rows of W and all rows of X (MT
// groups of 16), its waves cut the sum into groups of 4 blocks (one load of
// scales each) and join through LDS in wave order.  Codes go from memory to
// registers as 16-byte loads, become bf16 there (exactly) and enter the bf16
// instruction; the k-order inside a load is the same on both sides.  Reading W
// this way alone takes 12.5 us for 14336 x 4096 and 41.5 us (5.7 TB/s) for
// 8192 x 28672.
//
// SRC: where X comes from.  kFromCodes: 8-bit blocks in memory.  Else an element
// type: every workgroup makes the blocks itself, and their bf16 values, in LDS,
// while its first codes of W are on their way; for the few values this is for
// that costs less than a launch of its own.
constexpr int kSkinnyWaves = 8;
constexpr int kFromCodes = -1;

// 8 codes times 2^e (as a float) in bf16.
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi, float s) {
    union {
        bf16x2 p[4];
        bf16x8 v;
    } u;
    u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false);
    u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true);
    u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false);
    u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true);
    return u.v;
}

template <int MT, int SRC>
__global__ __launch_bounds__(kSkinnyWaves * 64) void skinny_kernel(MmLaunch p) {
    constexpr bool CODES = SRC == kFromCodes;
    constexpr int GB = 4;                            // blocks in a group
    constexpr int XQ = CODES && MT <= 2 ? GB : 1;    // blocks of X in flight
    extern __shared__ __attribute__((aligned(16))) char made[];
    __shared__ __attribute__((aligned(16))) f32x4 part[kSkinnyWaves][MT][64];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int r16 = lane & 15, g = lane >> 4;
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * 16;
    const int nb = static_cast<int>((p.sum + 127) / 128);
    const int64_t wrow = min(j0 + r16, p.cols - 1);
    const char *w = p.b + wrow * p.b_pitch + g * 16;
    const char *ws = p.bs + wrow * p.bs_pitch;
    u32x4 wv[GB][2];
    uint32_t wsc = 0;
    auto load_w = [&](int b, int n) {
        wsc = *reinterpret_cast<const uint32_t *>(ws + b);
#pragma unroll
        for (int q = 0; q < GB; q++)
            if (q < n) {
#pragma unroll
                for (int h = 0; h < 2; h++)
                    wv[q][h] = *reinterpret_cast<const u32x4 *>(w + (b + q) * 128 + h * 64);
            }
    };
    int b = wave * GB;
    if (b < nb) load_w(b, min(nb - b, GB));

    // Codes: X's pieces in memory.  Else its values in LDS, with a pitch of 16
    // bytes more than a row, so that 16 rows' pieces lie in different banks.
    const char *x[MT], *xs[MT];
    if (CODES) {
#pragma unroll
        for (int m = 0; m < MT; m++) {
            const int64_t row = min(static_cast<int64_t>(m * 16 + r16), p.rows - 1);
            x[m] = p.a + row * p.a_pitch + g * 16;
            xs[m] = p.as + row * p.as_pitch;
        }
    } else {
        constexpr int ES = SRC == kElemF32 ? 4 : 2;
        const int rows = static_cast<int>(p.rows), units = rows * nb, pitch = nb * 256 + 16;
        for (int u0 = 0; u0 < units; u0 += kSkinnyWaves * 4) {
            const int u = u0 + (t >> 4), row = u / nb, blk = u % nb, c = blk * 128 + (t & 15) * 8;
            const int left = u < units ? static_cast<int>(min(p.sum - c, static_cast<int64_t>(8))) : 0;
            float v[8];
            load8<CODES ? kElemBf16 : SRC>(p.a + (static_cast<int64_t>(row) * p.sum + c) * ES, left,
                                           p.aligned != 0, v);
            uint32_t scale;
            const u32x2 codes = encode8(v, &scale);
            if (u < units)
                *reinterpret_cast<bf16x8 *>(made + row * pitch + c * 2) =
                    widen8(codes.x, codes.y, __uint_as_float(scale << 23));
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; m++)
            x[m] = made + min(m * 16 + r16, rows - 1) * pitch + g * 32;
    }

    f32x4 acc[MT];
#pragma unroll
    for (int m = 0; m < MT; m++) acc[m] = f32x4{0, 0, 0, 0};
    // Blocks b .. b + n - 1, n = GB with FULL.
    auto group = [&](auto full, int n) {
        constexpr bool FULL = decltype(full)::value;
        uint32_t xsc[MT];
        u32x4 xv[XQ][2][MT];             // codes
        auto load_x = [&](int q) {
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int m = 0; m < MT; m++)
                    xv[q % XQ][h][m] =
                        *reinterpret_cast<const u32x4 *>(x[m] + (b + q) * 128 + h * 64);
        };
        if (CODES) {
#pragma unroll
            for (int m = 0; m < MT; m++) xsc[m] = *reinterpret_cast<const uint32_t *>(xs[m] + b);
        }
        if (XQ == GB) {
#pragma unroll
            for (int q = 0; q < GB; q++)
                if (FULL || q < n) load_x(q);
        }
#pragma unroll
        for (int q = 0; q < GB; q++) {
            if (!FULL && q >= n) break;
            if (CODES && XQ < GB) load_x(q);
            const float sw = __uint_as_float((wsc >> (8 * q) & 0xffu) << 23);
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const bf16x8 wf = widen8(wv[q][h][2 * e], wv[q][h][2 * e + 1], sw);
#pragma unroll
                    for (int m = 0; m < MT; m++) {
                        bf16x8 xf;
                        if (CODES)
                            xf = widen8(xv[q % XQ][h][m][2 * e], xv[q % XQ][h][m][2 * e + 1],
                                        __uint_as_float((xsc[m] >> (8 * q) & 0xffu) << 23));
                        else
                            xf = *reinterpret_cast<const bf16x8 *>(x[m] + (b + q) * 256 + h * 128 +
                                                                   e * 16);
                        acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf, acc[m], 0, 0, 0);
                    }
                }
        }
    };
    for (; b < nb; b += kSkinnyWaves * GB) {
        const int n = min(nb - b, GB);
        if (n == GB)
            group(std::true_type{}, GB);
        else
            group(std::false_type{}, n);
        const int next = b + kSkinnyWaves * GB;
        if (next < nb) load_w(next, min(nb - next, GB));
    }
#pragma unroll
    for (int m = 0; m < MT; m++) part[wave][m][lane] = acc[m];
    __syncthreads();
    for (int i = t; i < MT * 64; i += kSkinnyWaves * 64) {
        const int m = i / 64, l = i % 64;
        f32x4 s = part[0][m][l];
#pragma unroll
        for (int q = 1; q < kSkinnyWaves; q++) s += part[q][m][l];
        store4(p, m * 16 + (l & 15), j0 + (l >> 4) * 4, s);
    }
}

template <Mode MI, Mode MJ>
void launch_wide(const MmLaunch &p, int tile, dim3 grid, hipStream_t s) {
    constexpr bool any = is_codes(MI);       // no bf16 operand to be aligned
    if (tile == 256)
        wide_kernel<MI, MJ, 256, 2, 4, true><<<grid, dim3(512), 0, s>>>(p);
    else if (tile == 128 && (any || p.aligned))
        wide_kernel<MI, MJ, 128, 2, 2, true><<<grid, dim3(256), 0, s>>>(p);
    else if (tile == 128)
        wide_kernel<MI, MJ, 128, 2, 2, any><<<grid, dim3(256), 0, s>>>(p);
    else if (any || p.aligned)
        wide_kernel<MI, MJ, 64, 2, 2, true><<<grid, dim3(256), 0, s>>>(p);
    else
        wide_kernel<MI, MJ, 64, 2, 2, any><<<grid, dim3(256), 0, s>>>(p);
}

tide_status run_mm(MmOp op, const char *name, const MmArgs &a, void *stream) {
    tide_status st = check_mm(op, name, a);
    if (st != TIDE_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    MmLaunch p = {};
    p.rows = op == kMmDw ? a.N : a.M;
    p.cols = op == kMm ? a.N : a.K;
    p.sum = op == kMm ? a.K : op == kMmDx ? a.N : a.M;
    if (p.rows == 0 || p.cols == 0) {
        clear_error();
        return TIDE_OK;
    }
    const int64_t n = p.rows * p.cols;
    p.out = static_cast<char *>(a.out);
    p.out_bf16 = (a.flags & TIDE_F_OUT_BF16) != 0;
    p.accumulate = (a.flags & TIDE_F_ACCUMULATE) != 0;
    const unsigned flat = static_cast<unsigned>(std::min<int64_t>((n + 1023) / 1024, kCus * 8));
    if (p.sum == 0) {
        if (!p.accumulate) {
            zero_kernel<<<dim3(flat), dim3(256), 0, s>>>(p.out, n, p.out_bf16 ? 2 : 4);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return hip_fail("tide_block_mm: zeros", e);
        }
        clear_error();
        return TIDE_OK;
    }
    p.aligned = mm_aligned(op, a.a, a.N);
    MmChoice c = mm_choose(op, a.M, a.N, a.K, a.flags, p.aligned, true);
    if (c.workspace > a.workspace_bytes)
        c = mm_choose(op, a.M, a.N, a.K, a.flags, p.aligned, false);
    p.a = static_cast<const char *>(a.a);
    p.as = static_cast<const char *>(a.a_scales);
    p.b = static_cast<const char *>(a.b);
    p.bs = static_cast<const char *>(a.b_scales);
    p.a_pitch = op == kMm ? block_cols(a.K) : a.N * 2;
    p.as_pitch = block_scale_cols(a.K);
    p.b_pitch = block_cols(a.K);
    p.bs_pitch = block_scale_cols(a.K);
    p.chunk = c.chunk;
    p.splits = c.splits;
    p.direct = static_cast<uint32_t>(c.direct);
    p.partial = static_cast<float *>(a.workspace);
    const int64_t tr = (p.rows + c.tile - 1) / c.tile, tc = (p.cols + c.tile - 1) / c.tile;
    const int64_t cut = (tr * tc - c.direct) * c.splits;
    p.tr = static_cast<uint32_t>(tr);
    p.tc = static_cast<uint32_t>(tc);
    const dim3 grid(static_cast<unsigned>(c.direct + cut));
    if (c.kernel == kMmSkinny) {
        const dim3 g(static_cast<unsigned>((p.cols + 15) / 16)), b(kSkinnyWaves * 64);
        if (p.rows <= 16)
            skinny_kernel<1, kFromCodes><<<g, b, 0, s>>>(p);
        else if (p.rows <= 32)
            skinny_kernel<2, kFromCodes><<<g, b, 0, s>>>(p);
        else
            skinny_kernel<4, kFromCodes><<<g, b, 0, s>>>(p);
    } else if (c.kernel == kMmEight) {
        if (c.tile == 256)
            eight_kernel<256, 2, 4><<<grid, dim3(512), 0, s>>>(p);
        else
            eight_kernel<128, 2, 2><<<grid, dim3(256), 0, s>>>(p);
    } else if (op == kMm) {
        launch_wide<kCodesAlong, kCodesAlong>(p, c.tile, grid, s);
    } else if (op == kMmDx) {
        launch_wide<kBf16Along, kCodesAcross>(p, c.tile, grid, s);
    } else {
        launch_wide<kBf16Across, kCodesAcross>(p, c.tile, grid, s);
    }
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && cut && c.kernel != kMmSkinny) {
        const dim3 g(static_cast<unsigned>((tr * tc - c.direct) * (c.tile * c.tile / 1024))), b(256);
        if (c.tile == 256)
            join_kernel<256><<<g, b, 0, s>>>(p);
        else if (c.tile == 128)
            join_kernel<128><<<g, b, 0, s>>>(p);
        else
            join_kernel<64><<<g, b, 0, s>>>(p);
        e = hipGetLastError();
    }
    if (e != hipSuccess) return hip_fail((std::string(name) + ": kernel launch").c_str(), e);
    clear_error();
    return TIDE_OK;
}

// x w^T for an x that is not in blocks yet: in one launch for few rows, else
// through blocks in the workspace.
tide_status run_linear(const LinearArgs &a, void *stream) {
    const char *name = "tide_block_linear";
    tide_status st = check_linear(a);
    if (st != TIDE_OK) return st;
    const ElemType in = in_type(a.flags);
    const uint32_t oflags = a.flags & (TIDE_F_OUT_BF16 | TIDE_F_SHORT_SUMS);
    const LinearChoice c = linear_choose(a.M, a.K);
    char *const ws = static_cast<char *>(a.workspace);
    if (!c.in_one || a.N == 0 || a.M == 0 || a.K == 0) {
        if (a.M && a.N && a.K) {
            if (a.workspace_bytes < c.blocks)
                return fail(TIDE_E_INVALID, std::string(name) + ": the workspace holds " +
                                                std::to_string(a.workspace_bytes) + " bytes, x's " +
                                                "blocks need " + std::to_string(c.blocks));
            st = tide_block_quant(a.x, a.M, a.K, ws, ws + c.scales, a.flags & ~oflags, stream);
            if (st != TIDE_OK) return st;
        }
        const int64_t left = std::max<int64_t>(a.workspace_bytes - c.blocks, 0);
        return run_mm(kMm, name,
                      MmArgs{ws, ws ? ws + c.scales : nullptr, a.b, a.b_scales, a.M, a.N, a.K, a.out,
                             left ? ws + c.blocks : nullptr, left, oflags},
                      stream);
    }
    MmLaunch p = {};
    p.rows = a.M;
    p.cols = a.N;
    p.sum = a.K;
    p.a = static_cast<const char *>(a.x);
    p.b = static_cast<const char *>(a.b);
    p.bs = static_cast<const char *>(a.b_scales);
    p.b_pitch = block_cols(a.K);
    p.bs_pitch = block_scale_cols(a.K);
    p.out = static_cast<char *>(a.out);
    p.out_bf16 = (oflags & TIDE_F_OUT_BF16) != 0;
    p.aligned = a.K % 8 == 0;          // x is read in whole vectors
    const dim3 g(static_cast<unsigned>((a.N + 15) / 16)), b(kSkinnyWaves * 64);
    const unsigned lds = static_cast<unsigned>(a.M * (2 * block_cols(a.K) + 16));
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (in) {
        case kElemBf16: skinny_kernel<1, kElemBf16><<<g, b, lds, s>>>(p); break;
        case kElemF16: skinny_kernel<1, kElemF16><<<g, b, lds, s>>>(p); break;
        case kElemF32: skinny_kernel<1, kElemF32><<<g, b, lds, s>>>(p); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return hip_fail("tide_block_linear: kernel launch", e);
    clear_error();
    return TIDE_OK;
}

}  // namespace
}  // namespace tide

using namespace tide;

extern "C" tide_status tide_block_mm(const void *x_codes, const void *x_scales, int64_t m,
                                     const void *w_codes, const void *w_scales, int64_t n,
                                     int64_t k, void *out, uint32_t flags, void *workspace,
                                     int64_t workspace_bytes, void *stream) {
    return run_mm(kMm, "tide_block_mm",
                  MmArgs{x_codes, x_scales, w_codes, w_scales, m, n, k, out, workspace,
                         workspace_bytes, flags},
                  stream);
}

extern "C" tide_status tide_block_mm_dx(const void *dy, int64_t m, int64_t n, const void *w_codes,
                                        const void *w_scales, int64_t k, void *dx, uint32_t flags,
                                        void *workspace, int64_t workspace_bytes, void *stream) {
    return run_mm(kMmDx, "tide_block_mm_dx",
                  MmArgs{dy, nullptr, w_codes, w_scales, m, n, k, dx, workspace, workspace_bytes,
                         flags},
                  stream);
}

extern "C" tide_status tide_block_mm_dw(const void *dy, int64_t m, int64_t n, const void *x_codes,
                                        const void *x_scales, int64_t k, void *dw, uint32_t flags,
                                        void *workspace, int64_t workspace_bytes, void *stream) {
    return run_mm(kMmDw, "tide_block_mm_dw",
                  MmArgs{dy, nullptr, x_codes, x_scales, m, n, k, dw, workspace, workspace_bytes,
                         flags},
                  stream);
}

extern "C" tide_status tide_block_linear(const void *x, int64_t m, int64_t k, const void *w_codes,
                                         const void *w_scales, int64_t n, void *out,
                                         uint32_t flags, void *workspace, int64_t workspace_bytes,
                                         void *stream) {
    return run_linear(
        LinearArgs{x, w_codes, w_scales, m, n, k, out, workspace, workspace_bytes, flags}, stream);
}
