// Device code that the products over blocked matrices share (block_mm.hip,
// fp4_mm.hip): a launch's tiles and pieces, the stores of their sums, and the
// kernel whose factors are bf16 numbers.
#pragma once

#include <hip/hip_runtime.h>

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

// A pointer that is the same in all lanes, in scalar registers.
__device__ __forceinline__ const char *scalar(const char *p) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32));
    return reinterpret_cast<const char *>(static_cast<uint64_t>(hi) << 32 | lo);
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

// ---------------------------------------------------------------------------
// Products with bf16 factors
// ---------------------------------------------------------------------------
//
// 8-bit and 4-bit operands become bf16 on their way into LDS (exactly: code * 2^e
// is a bf16 number), so every product of the bf16 instruction is exact and only the
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
enum Mode { kBf16Along, kBf16Across, kCodesAlong, kCodesAcross, kFoursAlong, kFoursAcross };

__host__ __device__ constexpr bool is_across(Mode m) {
    return m == kBf16Across || m == kCodesAcross || m == kFoursAcross;
}
__host__ __device__ constexpr bool is_codes(Mode m) {
    return m == kCodesAlong || m == kCodesAcross || m == kFoursAlong || m == kFoursAcross;
}
__host__ __device__ constexpr bool is_fours(Mode m) {
    return m == kFoursAlong || m == kFoursAcross;
}

// 8 e2m1 codes times 2^e (as a float) in bf16; an infinite "2^e" (scale byte 255)
// gives NaNs.
__device__ __forceinline__ bf16x8 widen4(uint32_t c, float s) {
    union {
        bf16x2 p[4];
        bf16x8 v;
    } u;
    u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0);
    u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1);
    u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2);
    u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3);
    return u.v;
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
// bytes at a time (4-bit codes: 8 bytes): fetch() asks for a step's bytes, put()
// stores one slot of them.  What lies outside the operand (rows or columns past its end) comes as
// zeros, by the buffer's bounds or by an offset beyond them, so nothing from
// there enters a sum.
template <Mode M, int T, int NT, bool ALIGNED>
struct Stage {
    static constexpr int EL = is_codes(M) ? 16 : 8;        // values in a slot
    // bytes of n values, and columns that share a scale
    static constexpr uint32_t bytes(uint32_t n) {
        return is_fours(M) ? n / 2 : is_codes(M) ? n : 2 * n;
    }
    static constexpr int BLOCK = is_fours(M) ? 32 : static_cast<int>(kBlockCols);
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
        off = row * pitch + bytes(first);
        soff = row * spitch;
        put_at = lds_at(row, first / 8);
        next = s0 * 64;
        end = static_cast<int>(sum_) - static_cast<int>(next) - first;
        base = p;
        sbase = sp;
        if (is_across(M)) {
            at0 = bytes(static_cast<uint32_t>(at));
            sat0 = static_cast<uint32_t>(at / BLOCK);
            lines = static_cast<uint32_t>(sum_) - next;
            have = static_cast<int>(min(count - at - first, static_cast<int64_t>(EL)));
            if (have <= 0) off = OUTSIDE;
            soff += first / BLOCK;
        } else {
            if (is_fours(M)) soff += first / BLOCK;    // a step holds two blocks of 32
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
            skip = bytes(next);
            sskip = next / BLOCK;
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
            } else if (is_fours(M)) {
                const u32x2 c =
                    __builtin_amdgcn_raw_buffer_load_b64(r, at, q * ROWS * pitch + skip, 0);
                v[q] = u32x4{c.x, c.y, 0, 0};
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
            if (is_fours(M)) {
                *reinterpret_cast<LDS_AS bf16x8 *>(h == 0 ? to : to + half) = widen4(v[q][h], s);
                continue;
            }
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
    const int64_t cols = is_codes(MJ) && is_across(MJ) ? (p.cols + whole) & ~whole : p.cols;
    const int64_t isum = is_codes(MI) && !is_across(MI) ? (p.sum + whole) & ~whole : p.sum;
    const int64_t jsum = is_codes(MJ) && !is_across(MJ) ? (p.sum + whole) & ~whole : p.sum;

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

}  // namespace
}  // namespace tide
