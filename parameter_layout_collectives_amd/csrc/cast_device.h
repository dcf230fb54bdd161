// Kernels and launches that write and read matrices in 8-bit or 4-bit blocks,
// whole or as shards of a unit (block_cast.hip, fp4_cast.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "block.h"
#include "block_device.h"

namespace tide {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kLanes = 256;                        // lanes of a workgroup
constexpr int kGroup = 16;                         // lanes that share a block
constexpr int kGroups = kLanes / kGroup;           // blocks a workgroup handles at a time
constexpr int kUnroll = 4;                         // blocks in flight per group
constexpr int kChunk = kGroups * kUnroll;          // blocks a workgroup handles in all

// The formats.  16 lanes make or read 128 columns of a row at a time (a unit):
// one 8-bit block, or four 4-bit ones.  cp and sp: bytes of a row's codes and
// scales, for nb units.
struct Eights {
    static constexpr int kCodeBytes = 8;               // of a lane's 8 values
    static __host__ __device__ int64_t cp(uint32_t nb) { return static_cast<int64_t>(nb) * 128; }
    static __host__ __device__ int64_t sp(uint32_t nb) { return (nb + 3) / 4 * 4; }
};
struct Fours {
    static constexpr int kCodeBytes = 4;
    static __host__ __device__ int64_t cp(uint32_t nb) { return static_cast<int64_t>(nb) * 64; }
    static __host__ __device__ int64_t sp(uint32_t nb) { return static_cast<int64_t>(nb) * 4; }
};

// A matrix of a unit, for the kernels below.
struct alignas(16) Rows {
    int64_t src;           // first element of its rows in the source (or the destination's address)
    uint32_t codes;        // where its codes and its scales start in a rank block, in 16 bytes
    uint32_t scales;
    uint32_t rows, real;   // rows to write, and of them rows that exist in the source
    uint32_t cols;
    uint32_t wg0;          // first workgroup that works on it
    __host__ __device__ uint32_t nb() const { return (cols + kBlockCols - 1) / kBlockCols; }
};

// Reads blocks [first, first + kChunk) of `d` (row-major), encodes and stores
// them.  The last block of a row also fills the row's spare scale bytes.
template <class F, int ET>
__device__ __forceinline__ void encode_chunk(const Rows &d, int64_t first, const char *src,
                                             char *codes, char *scales, bool vec) {
    constexpr int ES = ET == kElemF32 ? 4 : 2;
    const int group = threadIdx.x / kGroup, lane = threadIdx.x % kGroup;
    const uint32_t nb = d.nb();
    const int64_t units = static_cast<int64_t>(d.rows) * nb;
    const int64_t row0 = first / nb;                        // uniform
    const uint32_t b0 = static_cast<uint32_t>(first - row0 * nb);
    const int64_t cp = F::cp(nb), sp = F::sp(nb);
    float v[kUnroll][8];
    int64_t row[kUnroll];
    uint32_t blk[kUnroll];
#pragma unroll
    for (int q = 0; q < kUnroll; q++) {
        const uint32_t i = b0 + q * kGroups + group;        // < nb + kChunk
        row[q] = row0 + i / nb;
        blk[q] = i % nb;
        const int64_t c = static_cast<int64_t>(blk[q]) * kBlockCols + lane * 8;
        const bool there = first + q * kGroups + group < units && row[q] < d.real;
        const int64_t left = static_cast<int64_t>(d.cols) - c;
        load8<ET>(src + (row[q] * d.cols + c) * ES,
                  there ? static_cast<int>(left < 8 ? left : 8) : 0, vec, v[q]);
    }
#pragma unroll
    for (int q = 0; q < kUnroll; q++) {
        uint32_t scale;
        if constexpr (std::is_same<F, Fours>::value) {
            const uint32_t c = encode4(v[q], &scale);
            if (first + q * kGroups + group >= units) continue;
            *reinterpret_cast<uint32_t *>(codes + row[q] * cp + static_cast<int64_t>(blk[q]) * 64 +
                                          lane * 4) = c;
            if (lane % 4 == 0)
                scales[row[q] * sp + static_cast<int64_t>(blk[q]) * 4 + lane / 4] =
                    static_cast<char>(scale);
            continue;
        }
        const u32x2 c = encode8(v[q], &scale);
        if (first + q * kGroups + group >= units) continue;
        *reinterpret_cast<u32x2 *>(codes + row[q] * cp + static_cast<int64_t>(blk[q]) * kBlockCols +
                                   lane * 8) = c;
        char *s = scales + row[q] * sp + blk[q];
        if (lane == 0) *s = static_cast<char>(scale);
        if (blk[q] == nb - 1 && lane > 0 && blk[q] + lane < sp) s[lane] = 127;
    }
}

template <class F, int ET>
__global__ __launch_bounds__(kLanes) void quant_kernel(const char *__restrict__ x, int64_t rows,
                                                       int64_t cols, char *__restrict__ codes,
                                                       char *__restrict__ scales, int vec) {
    const Rows d{0, 0, 0, static_cast<uint32_t>(rows), static_cast<uint32_t>(rows),
                 static_cast<uint32_t>(cols), 0};
    encode_chunk<F, ET>(d, static_cast<int64_t>(blockIdx.x) * kChunk, x, codes, scales, vec != 0);
}

// 8 codes of one block -> the output type, stored at p.
template <class F, int ET>
__device__ __forceinline__ void decode8(u32x2 c, uint32_t scale, char *p, int n, bool vec) {
    // 8-bit scale bytes are 10..246; a 4-bit block's may be 255, which gives NaNs
    const float s = __uint_as_float(scale << 23);
    bf16x2 h[4];
    if constexpr (std::is_same<F, Fours>::value) {
        h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.x, s, 0);
        h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.x, s, 1);
        h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.x, s, 2);
        h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.x, s, 3);
    } else {
        h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, s, false);
        h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, s, true);
        h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, s, false);
        h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, s, true);
    }
    if (ET == kElemF32) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = static_cast<float>(h[i / 2][i & 1]);
        if (vec || n >= 8) {
            row_f32x4 *o = reinterpret_cast<row_f32x4 *>(p);
            __builtin_nontemporal_store(row_f32x4{v[0], v[1], v[2], v[3]}, o);
            __builtin_nontemporal_store(row_f32x4{v[4], v[5], v[6], v[7]}, o + 1);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (i < n) reinterpret_cast<float *>(p)[i] = v[i];
        }
        return;
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (ET == kElemBf16) {
            w[i] = __builtin_bit_cast(uint32_t, h[i]);
        } else {   // fp16: bf16 -> fp32 is exact, then one rounding (to inf past 65504)
            const f16x2 f = {static_cast<_Float16>(static_cast<float>(h[i][0])),
                             static_cast<_Float16>(static_cast<float>(h[i][1]))};
            w[i] = __builtin_bit_cast(uint32_t, f);
        }
    }
    if (vec || n >= 8) {
        __builtin_nontemporal_store(half_u32x4{w[0], w[1], w[2], w[3]},
                                    reinterpret_cast<half_u32x4 *>(p));
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < n)
                reinterpret_cast<uint16_t *>(p)[i] =
                    static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
    }
}

// Blocks [first, first + kChunk) of a matrix of `rows` rows; row r's codes and
// scales are found by at(r, &codes, &scales).
template <class F, int ET, class At>
__device__ __forceinline__ void decode_chunk(int64_t rows, int64_t cols, uint32_t nb, int64_t first,
                                             At at, char *out, bool vec) {
    constexpr int ES = ET == kElemF32 ? 4 : 2;
    const int group = threadIdx.x / kGroup, lane = threadIdx.x % kGroup;
    const int64_t units = rows * nb;
    const int64_t row0 = first / nb;
    const uint32_t b0 = static_cast<uint32_t>(first - row0 * nb);
    u32x2 c[kUnroll];
    uint32_t scale[kUnroll];
    char *o[kUnroll];
    int n[kUnroll];
#pragma unroll
    for (int q = 0; q < kUnroll; q++) {
        const uint32_t i = b0 + q * kGroups + group;
        const int64_t row = row0 + i / nb;
        const uint32_t blk = i % nb;
        const int64_t col = static_cast<int64_t>(blk) * kBlockCols + lane * 8;
        const int64_t left = cols - col;
        n[q] = first + q * kGroups + group < units ? static_cast<int>(left < 8 ? left : 8) : 0;
        o[q] = out + (row * cols + col) * ES;
        if (n[q] > 0) {
            const char *codes, *scales;
            at(row, &codes, &scales);
            if constexpr (std::is_same<F, Fours>::value) {
                c[q].x = __builtin_nontemporal_load(
                    reinterpret_cast<const uint32_t *>(codes + col / 2));
                scale[q] = static_cast<uint8_t>(scales[col / 32]);
            } else {
                c[q] = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(codes + col));
                scale[q] = static_cast<uint8_t>(scales[blk]);
            }
        }
    }
#pragma unroll
    for (int q = 0; q < kUnroll; q++)
        if (n[q] > 0) decode8<F, ET>(c[q], scale[q], o[q], n[q], vec);
}

template <class F, int ET>
__global__ __launch_bounds__(kLanes) void dequant_kernel(const char *__restrict__ codes,
                                                         const char *__restrict__ scales,
                                                         int64_t rows, int64_t cols,
                                                         char *__restrict__ out, int vec) {
    const uint32_t nb = static_cast<uint32_t>((cols + kBlockCols - 1) / kBlockCols);
    const int64_t cp = F::cp(nb), sp = F::sp(nb);
    decode_chunk<F, ET>(rows, cols, nb, static_cast<int64_t>(blockIdx.x) * kChunk,
                     [=](int64_t r, const char **c, const char **s) {
                         *c = codes + r * cp;
                         *s = scales + r * sp;
                     },
                     out, vec != 0);
}

// A unit's matrices travel as kernel arguments (no table in device memory, so
// nothing to allocate, upload or keep for a captured launch): as many slots per
// launch as fit 4 KB.  A matrix takes one slot; matrices that repeat at a fixed
// distance (an MoE layer's experts) take two for all of them, the first one's
// Rows and a Step.
constexpr int kPerLaunch = 112;
constexpr uint32_t kIsStep = 0xffffffffu;   // past every workgroup's number
struct alignas(16) Step {
    int64_t src;           // from one matrix to the next, as in Rows
    uint32_t codes, scales;
    uint32_t wgs;          // workgroups per matrix
    uint32_t unused[2];
    uint32_t mark;         // kIsStep, where Rows holds wg0
};
union Slot {
    Rows m;
    Step step;
    u32x4 v[2];
};
template <int N>
struct Slots {
    Slot m[N];
    int n;
};
// What a wave reads of the slots and a launch copies should follow what the unit
// fills: with 16 slots an 8B layer's 9 casts and placement (7 matrices) take 318
// us, with 112 325; an MoE layer's 17 launches (14 slots) 964 and 1001.
constexpr int kFew = 16;
static_assert(sizeof(Slot) == 32 && sizeof(Slot) * kPerLaunch <= 3600, "matrix descriptors exceed the kernel arguments");
static_assert(offsetof(Rows, wg0) == 28 && offsetof(Step, mark) == 28, "wg0 and mark share a word");

// The matrix that workgroup `wg` works on: the last one with wg0 <= wg.  Kernel
// arguments may lie in host memory, so they are read once, all of them by every
// wave (two slots per lane), and the one that is wanted comes from its lane: one
// latency, where a search would have eight in a row.
template <int N>
__device__ __forceinline__ Rows matrix_of(const Slots<N> &a, uint32_t wg) {
    static_assert(N <= 128, "two slots per lane");
    const int lane = threadIdx.x & 63;
    Slot one, two;
    const int i = min(lane, N - 1), j = min(lane + 64, N - 1);
#pragma unroll
    for (int h = 0; h < 2; h++) {
        one.v[h] = a.m[i].v[h];
        two.v[h] = N > 64 ? a.m[j].v[h] : one.v[h];
    }
    const auto slot = [&](int k) {
        Slot w;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const uint32_t x = N <= 64 || k < 64 ? one.v[e / 4][e & 3] : two.v[e / 4][e & 3];
            w.v[e / 4][e & 3] = __builtin_amdgcn_readlane(x, k & 63);
        }
        return w;
    };
    // slot 0 is always a matrix with wg0 = 0, so a bit of `first` is set
    const uint64_t first = __ballot(lane < a.n && one.m.wg0 <= wg);
    const uint64_t second = N > 64 ? __ballot(lane + 64 < a.n && two.m.wg0 <= wg) : 0;
    const int k = __builtin_amdgcn_readfirstlane(second ? 127 - __clzll(second) : 63 - __clzll(first));
    Rows d = slot(k).m;
    if (k + 1 < a.n) {
        const Step s = slot(k + 1).step;
        if (s.mark == kIsStep) {
            const uint32_t q = (wg - d.wg0) / s.wgs;
            d.src += static_cast<int64_t>(q) * s.src;
            d.codes += q * s.codes;
            d.scales += q * s.scales;
            d.wg0 += q * s.wgs;
        }
    }
    return d;
}

template <class F, int N>
__global__ __launch_bounds__(kLanes) void shard_kernel(Slots<N> a, const char *__restrict__ master,
                                                       char *__restrict__ block) {
    const Rows d = matrix_of(a, blockIdx.x);
    const bool vec = d.cols % 8 == 0;
    encode_chunk<F, kElemF32>(d, static_cast<int64_t>(blockIdx.x - d.wg0) * kChunk,
                           master + d.src * 4, block + static_cast<int64_t>(d.codes) * 16,
                           block + static_cast<int64_t>(d.scales) * 16, vec);
}

// `src` of a matrix holds its destination's address here, `rows` its rows and
// `real` the c rows of a rank; row r lies in rank block r / c at row r % c.
template <class F, int ET, int N>
__global__ __launch_bounds__(kLanes) void unshard_kernel(Slots<N> a,
                                                         const char *__restrict__ gathered,
                                                         int64_t rank_bytes) {
    const Rows d = matrix_of(a, blockIdx.x);
    char *out = reinterpret_cast<char *>(d.src);
    const bool vec = d.cols % 8 == 0;
    const uint32_t nb = d.nb();
    const int64_t cp = F::cp(nb), sp = F::sp(nb);
    const int64_t at_codes = static_cast<int64_t>(d.codes) * 16;
    const int64_t at_scales = static_cast<int64_t>(d.scales) * 16;
    const uint32_t c = d.real;
    decode_chunk<F, ET>(d.rows, d.cols, nb, static_cast<int64_t>(blockIdx.x - d.wg0) * kChunk,
                     [=](int64_t r, const char **codes, const char **scales) {
                         const uint32_t row = static_cast<uint32_t>(r), rank = row / c;
                         const int64_t in = row - rank * c;
                         const char *b = gathered + rank * rank_bytes;
                         *codes = b + at_codes + in * cp;
                         *scales = b + at_scales + in * sp;
                     },
                     out, vec);
}

// A launch counts its lanes in 32 bits.
constexpr int64_t kMaxGrid = 0xffffffffll / kLanes;

int64_t chunks(int64_t units) { return (units + kChunk - 1) / kChunk; }

tide_status too_many(const char *name) {
    return fail(TIDE_E_UNSUPPORTED, std::string(name) + ": more than 2^32 lanes");
}

int64_t chunks_of(const Rows &r) { return chunks(static_cast<int64_t>(r.rows) * r.nb()); }

// The smallest group of matrices from `j` on whose shapes come three times in a
// row, or 0.
int32_t period(const tide_plan *bp, int32_t j) {
    constexpr int32_t kMost = 8;
    for (int32_t p = 1; p <= kMost && p <= (bp->nblk - j) / 3; p++) {
        int32_t i = j;
        while (i < j + 2 * p && bp->d0[i] == bp->d0[i + p] && bp->blk_inner[i] == bp->blk_inner[i + p])
            i++;
        if (i == j + 2 * p) return p;
    }
    return 0;
}

// How many groups of `p` matrices from `j` on have one group's shapes and lie at
// one distance, `step`.
template <class Fill>
int32_t repeats(const tide_plan *bp, Fill fill, int32_t j, int32_t p, Step *step) {
    Rows a, b;
    fill(j, &a);
    fill(j + p, &b);
    const uint64_t src = static_cast<uint64_t>(b.src) - static_cast<uint64_t>(a.src);
    *step = Step{static_cast<int64_t>(src), b.codes - a.codes, b.scales - a.scales, 0, {}, kIsStep};
    for (uint32_t q = 1; ; q++)
        for (int32_t t = 0; t < p; t++) {
            const int64_t i = j + t + static_cast<int64_t>(q) * p;
            if (i >= bp->nblk) return static_cast<int32_t>(q);
            fill(j + t, &a);
            fill(static_cast<int32_t>(i), &b);
            if (chunks_of(a) == 0 || b.rows != a.rows || b.real != a.real || b.cols != a.cols ||
                static_cast<uint64_t>(b.src) != static_cast<uint64_t>(a.src) + q * src ||
                b.codes != a.codes + q * step->codes || b.scales != a.scales + q * step->scales)
                return static_cast<int32_t>(q);
        }
}

// Launches `launch(args, grid)` over the plan's matrices, as many at a time as
// the slots hold; `fill(j, &rows)` describes matrix j, with rows.rows = 0 for
// nothing to do.  In a unit of more matrices than one launch has slots, groups
// that come three times or more (experts, each of them with its gate, up and
// down projection, say) share theirs; twice would take as many, and a smaller
// unit has its one launch without the search.  The MoE layer's 389 matrices take
// one launch instead of four, its 16 casts 632 us instead of 784.
template <class Fill, class Launch>
tide_status over_matrices(const char *name, const tide_plan *bp, Fill fill, Launch launch) {
    for (int32_t i = 0; i < bp->nblk; i++) {     // before anything is enqueued
        Rows r;
        fill(i, &r);
        if (chunks_of(r) > kMaxGrid) return too_many(name);
    }
    int32_t j = 0;
    while (j < bp->nblk) {
        Slots<kPerLaunch> a;
        a.n = 0;
        int64_t grid = 0;
        while (j < bp->nblk) {
            Rows r;
            fill(j, &r);
            if (chunks_of(r) == 0) {
                j++;
                continue;
            }
            Step step;
            int32_t p = bp->nblk > kPerLaunch ? period(bp, j) : 0;
            int64_t n = p ? repeats(bp, fill, j, p, &step) : 1;
            if (n < 3) p = n = 1;
            int64_t wgs = 0;
            for (int32_t t = 0; t < p; t++) {
                fill(j + t, &r);
                wgs += chunks_of(r);
            }
            if (n > 1 && wgs * n > kMaxGrid) {       // one by one, over several launches
                p = n = 1;
                fill(j, &r);
                wgs = chunks_of(r);
            }
            if (grid + wgs * n > kMaxGrid || a.n + (n > 1 ? 2 * p : 1) > kPerLaunch) break;
            for (int32_t t = 0; t < p; t++) {
                fill(j + t, &r);
                r.wg0 = static_cast<uint32_t>(grid);
                a.m[a.n++].m = r;
                grid += chunks_of(r) * n;
                if (n > 1) {
                    step.wgs = static_cast<uint32_t>(chunks_of(r));
                    a.m[a.n++].step = step;
                }
            }
            j += p * static_cast<int32_t>(n);
        }
        if (a.n == 0) break;
        if (a.n <= kFew) {
            Slots<kFew> few;
            few.n = a.n;
            std::copy(a.m, a.m + a.n, few.m);
            launch(few, static_cast<unsigned>(grid));
        } else {
            launch(a, static_cast<unsigned>(grid));
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return hip_fail((std::string(name) + ": kernel launch").c_str(), e);
    }
    return TIDE_OK;
}

// An offset in 4-byte words (a multiple of 4) in 16 bytes.
uint32_t in16(int64_t words) { return static_cast<uint32_t>(words / 4); }


// The entry points' launches, behind their checks.
template <class F>
tide_status run_quant(const char *name, const void *x, int64_t rows, int64_t cols, void *codes,
                      void *scales, uint32_t flags, void *stream) {
    if (rows && cols) {
        const int64_t grid = chunks(rows * block_count(cols));
        if (grid > kMaxGrid) return too_many(name);
        const int vec = cols % 8 == 0;
        const dim3 g(static_cast<unsigned>(grid)), b(kLanes);
        hipStream_t s = static_cast<hipStream_t>(stream);
        const char *in = static_cast<const char *>(x);
        char *c = static_cast<char *>(codes), *sc = static_cast<char *>(scales);
        switch (in_type(flags)) {
            case kElemBf16: quant_kernel<F, kElemBf16><<<g, b, 0, s>>>(in, rows, cols, c, sc, vec); break;
            case kElemF16: quant_kernel<F, kElemF16><<<g, b, 0, s>>>(in, rows, cols, c, sc, vec); break;
            case kElemF32: quant_kernel<F, kElemF32><<<g, b, 0, s>>>(in, rows, cols, c, sc, vec); break;
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return hip_fail((std::string(name) + ": kernel launch").c_str(), e);
    }
    clear_error();
    return TIDE_OK;
}

template <class F>
tide_status run_dequant(const char *name, const void *codes, const void *scales, int64_t rows,
                        int64_t cols, void *out, uint32_t flags, void *stream) {
    if (rows && cols) {
        const int64_t grid = chunks(rows * block_count(cols));
        if (grid > kMaxGrid) return too_many(name);
        const int vec = cols % 8 == 0;
        const dim3 g(static_cast<unsigned>(grid)), b(kLanes);
        hipStream_t s = static_cast<hipStream_t>(stream);
        const char *c = static_cast<const char *>(codes), *sc = static_cast<const char *>(scales);
        char *o = static_cast<char *>(out);
        switch (out_type(flags)) {
            case kElemBf16: dequant_kernel<F, kElemBf16><<<g, b, 0, s>>>(c, sc, rows, cols, o, vec); break;
            case kElemF16: dequant_kernel<F, kElemF16><<<g, b, 0, s>>>(c, sc, rows, cols, o, vec); break;
            case kElemF32: dequant_kernel<F, kElemF32><<<g, b, 0, s>>>(c, sc, rows, cols, o, vec); break;
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return hip_fail((std::string(name) + ": kernel launch").c_str(), e);
    }
    clear_error();
    return TIDE_OK;
}

template <class F>
tide_status run_shard(const char *name, const tide_plan *plan, int32_t rank, const float *master,
                      void *block, void *stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    const tide_status st = over_matrices(
        name, plan,
        [&](int32_t j, Rows *r) {
            const int64_t c = plan->c[j], d0 = plan->d0[j];
            *r = Rows{plan->blk_off[j], in16(plan->off[j]), in16(plan->off[plan->nblk + j]),
                      static_cast<uint32_t>(c),
                      static_cast<uint32_t>(std::min(c, std::max<int64_t>(0, d0 - rank * c))),
                      static_cast<uint32_t>(plan->blk_inner[j]), 0};
        },
        [&](const auto &a, unsigned grid) {
            shard_kernel<F><<<dim3(grid), dim3(kLanes), 0, s>>>(
                a, reinterpret_cast<const char *>(master), static_cast<char *>(block));
        });
    if (st == TIDE_OK) clear_error();
    return st;
}

template <class F>
tide_status run_unshard(const char *name, const tide_plan *plan, const void *gathered,
                        void *const *params, uint32_t flags, void *stream) {
    if (plan->psi == 0) {
        clear_error();
        return TIDE_OK;
    }
    const ElemType t = out_type(flags);
    const int64_t rank_bytes = plan->S * 4;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const char *g = static_cast<const char *>(gathered);
    const tide_status st = over_matrices(
        name, plan,
        [&](int32_t j, Rows *r) {
            *r = Rows{static_cast<int64_t>(reinterpret_cast<uintptr_t>(params[j])),
                      in16(plan->off[j]), in16(plan->off[plan->nblk + j]),
                      static_cast<uint32_t>(plan->d0[j]), static_cast<uint32_t>(plan->c[j]),
                      static_cast<uint32_t>(plan->blk_inner[j]), 0};
        },
        [&](const auto &a, unsigned grid) {
            const dim3 gr(grid), b(kLanes);
            switch (t) {
                case kElemBf16: unshard_kernel<F, kElemBf16><<<gr, b, 0, s>>>(a, g, rank_bytes); break;
                case kElemF16: unshard_kernel<F, kElemF16><<<gr, b, 0, s>>>(a, g, rank_bytes); break;
                case kElemF32: unshard_kernel<F, kElemF32><<<gr, b, 0, s>>>(a, g, rank_bytes); break;
            }
        });
    if (st == TIDE_OK) clear_error();
    return st;
}

}  // namespace
}  // namespace tide
