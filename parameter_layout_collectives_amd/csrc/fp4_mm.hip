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
// A T x T tile of the output per workgroup, WI x WJ waves.  One step of the sum is
// 256 columns: 128 bytes of a row, 8 chunks of 16, one block each; chunk h of row r
// lies at h ^ (r & 7) in LDS, so the 16 lanes that read one chunk of 16 rows touch
// all banks.  Lane (r16, g) multiplies blocks g and g + 4 of its rows.  Two buffers:
// the next step's codes travel straight into the other one while this one is
// multiplied.
template <int T, int WI, int WJ>
struct Tiles {
    static constexpr int NT = WI * WJ * 64, NW = WI * WJ;
    static constexpr int FI = T / WI / 16, FJ = T / WJ / 16;   // 16 x 16 fragments per wave
    static constexpr int SLOTS = T * 8 / NT;                   // 16-byte loads per thread and operand
    static constexpr int TILE = T * 128;                       // bytes of an operand's codes
    static constexpr int SCALES = 2 * T * 8;                   // and of both operands' scales
    static constexpr int LDS = 4 * TILE + 2 * SCALES;
    static constexpr int SLOADS = 2 * T / 32 / NW;             // loads of 32 rows' scales per wave
    // I's fragments (lines) go through a ring of registers, D ahead of the
    // multiplications.
    static constexpr int RING = 2, D = RING - 1;
    static constexpr uint32_t OUTSIDE = 0x80000000u;           // past every buffer's end
    static_assert(FI % RING == 0 && SLOTS <= FI, "a step starts at ring entry 0");

    __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
    uint32_t vc, vc_half;        // this thread's first code slot; in a step of 128 columns
    uint32_t vs, vs_half;        // its scale words' row, likewise
    uint32_t half_step;          // the step that has only 128 columns, if any
    uint32_t pitch, spitch;
    int wave, fa, fb, sa, sb;    // fragments and their scales, in a buffer
    int shift;                   // of this lane's byte in a word of scales
    f32x4 acc[FI][FJ];

    // Part q of step s's codes (and with the last one the scales) -> a buffer (I's
    // codes, J's, scales).
    __device__ __forceinline__ void fetch(LDS_AS char *ta, LDS_AS char *tb, LDS_AS char *tw,
                                          uint32_t s, int q) const {
        const int at = (wave + q * NW) * 1024;
        const uint32_t off = q * (NT / 8) * pitch + s * 128;
        const uint32_t v = s == half_step ? vc_half : vc;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (LDS_AS void *)(ta + at), 16, v, off, 0, 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (LDS_AS void *)(tb + at), 16, v, off, 0, 0);
        if (q < SLOTS - 1) return;
        const uint32_t vw = s == half_step ? vs_half : vs;
        // 32-row groups 0 .. T/32-1 are the tile's rows of I, the others those of J
#pragma unroll
        for (int k = 0; k < SLOADS; k++) {
            const int w = wave + k * NW, half = T / 32;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                w < half ? rsa : rsb, (LDS_AS void *)(tw + w * 256), 4, vw,
                (w < half ? w : w - half) * 32 * spitch + s * 8, 0, 0);
        }
    }
    struct Frag {                // 16 rows of one step
        u32x4 v[2];              // blocks g and g + 4
        uint32_t scale[2];       // this lane's in the low byte
    };
    __device__ __forceinline__ Frag frag(const LDS_AS char *codes, int at, const LDS_AS char *sc) const {
        Frag f;
        f.v[0] = *reinterpret_cast<const LDS_AS u32x4 *>(codes + at);
        f.v[1] = *reinterpret_cast<const LDS_AS u32x4 *>(codes + (at ^ 64));
        const u32x2 w = *reinterpret_cast<const LDS_AS u32x2 *>(sc);
        f.scale[0] = w.x >> shift;
        f.scale[1] = w.y >> shift;
        return f;
    }
    __device__ __forceinline__ void rows(Frag *r, const LDS_AS char *b, const LDS_AS char *w) const {
#pragma unroll
        for (int y = 0; y < FJ; y++) r[y] = frag(b + y * 2048, fb, w + sb + y * 128);
    }
    __device__ __forceinline__ Frag line(const LDS_AS char *a, const LDS_AS char *w, int x) const {
        return frag(a + x * 2048, fa, w + sa + x * 128);
    }
    static __device__ __forceinline__ i32x8 wide(u32x4 v) {
        return i32x8{static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]),
                     static_cast<int>(v[3]), 0, 0, 0, 0};
    }
    __device__ __forceinline__ void multiply(int x, const Frag &l, const Frag *r) {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int y = 0; y < FJ; y++)
                acc[x][y] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    wide(r[y].v[h]), wide(l.v[h]), acc[x][y], 4, 4, 0,
                    static_cast<int>(r[y].scale[h]), 0, static_cast<int>(l.scale[h]));
    }
    // Step s, whose first D lines and J rows are in registers: reads the rest from
    // its buffer (h*); once nothing of it is left to read, the first reads of step
    // s + 1 from the other (t*) begin under the multiplications that remain, and
    // step s + 2 starts travelling to h*.
    template <bool LAST>
    __device__ __forceinline__ void step(Frag *l, const Frag *r, Frag *next, LDS_AS char *ha,
                                         LDS_AS char *hb, LDS_AS char *hw, LDS_AS char *ta,
                                         LDS_AS char *tb, LDS_AS char *tw, uint32_t s) {
#pragma unroll
        for (int x = 0; x < FI; x++) {
            if (x + D < FI) l[(x + D) % RING] = line(ha, hw, x + D);
            if (!LAST && x + D == FI) {
                landed();
                rows(next, tb, tw);
            }
            if (!LAST && x + D >= FI) l[(x + D) % RING] = line(ta, tw, x + D - FI);
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
        Frag l[RING], r0[FJ], r1[FJ];
        rows(r0, b0, w0);
#pragma unroll
        for (int x = 0; x < D; x++) l[x] = line(a0, w0, x);
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
__global__ __launch_bounds__(WI * WJ * 64, 1) void tiles_kernel(MmLaunch p) {
    typedef Tiles<T, WI, WJ> E;
    __shared__ __attribute__((aligned(1024))) char lds[E::LDS];
    const int t = threadIdx.x, lane = t & 63;
    const int r16 = lane & 15, g = lane >> 4;
    const Work work = work_of<T>(p, (p.sum + 255) / 256);
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
    // c ^ (r & 7) of memory.  A row ends inside a step if its 128-column units are
    // odd in number: the step's second half is then fetched as zeros.
    const int chunk = (t & 7) ^ (t >> 3 & 7);
    e.vc = (t >> 3) * e.pitch + chunk * 16;
    e.vc_half = chunk < 4 ? e.vc : E::OUTSIDE;
    e.vs = (lane >> 1) * e.spitch + (lane & 1) * 4;
    e.vs_half = (lane & 1) ? E::OUTSIDE : e.vs;
    e.half_step = e.pitch % 128 ? e.pitch / 128 : 0xffffffffu;
    e.fa = (wi * (T / WI) + r16) * 128 + ((g ^ (r16 & 7)) << 4);
    e.fb = (wj * (T / WJ) + r16) * 128 + ((g ^ (r16 & 7)) << 4);
    e.sa = (wi * (T / WI) + r16) * 8;
    e.sb = (T + wj * (T / WJ) + r16) * 8;
    e.shift = 8 * g;
#pragma unroll
    for (int x = 0; x < E::FI; x++)
#pragma unroll
        for (int y = 0; y < E::FJ; y++) e.acc[x][y] = f32x4{0, 0, 0, 0};
    LDS_AS char *const b = (LDS_AS char *)lds, *const w = b + 4 * E::TILE;
    e.run(b, b + E::TILE, b + 2 * E::TILE, b + 3 * E::TILE, w, w + E::SCALES, s0, s1);
    store_tile<T>(p, work, wi * (T / WI) + r16, wj * (T / WJ) + g * 4, e.acc);
}

// ---------------------------------------------------------------------------
// Y = x W^T for few rows of x
// ---------------------------------------------------------------------------
//
// W's bytes bound it.  Each workgroup takes 16 rows of W and all rows of x (MT
// groups of 16); its waves cut the sum into groups of GB units of 128 columns and
// join through LDS in wave order.  Codes go from memory to registers as 16-byte
// loads, one block each, become bf16 there (exactly) and enter the bf16 instruction;
// the k-order inside a load is the same on both sides.
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

template <int MT, int SRC, bool QUANT>
__global__ __launch_bounds__(kFewWaves * 64) void few_kernel(MmLaunch p) {
    constexpr bool MADE = SRC != kPadded;
    constexpr int GB = 4;                            // units in a group
    extern __shared__ __attribute__((aligned(16))) char made[];
    __shared__ __attribute__((aligned(16))) f32x4 part[kFewWaves][MT][64];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int r16 = lane & 15, g = lane >> 4;
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * 16;
    const int nb = static_cast<int>((p.sum + 127) / 128);
    const int64_t wrow = min(j0 + r16, p.cols - 1);
    const char *w = p.b + wrow * p.b_pitch + g * 16;
    const char *ws = p.bs + wrow * p.bs_pitch;
    u32x4 wv[GB];
    uint32_t wsc[GB];
    auto load_w = [&](int b, int n) {
#pragma unroll
        for (int q = 0; q < GB; q++)
            if (q < n) {
                wsc[q] = *reinterpret_cast<const uint32_t *>(ws + (b + q) * 4);
                wv[q] = *reinterpret_cast<const u32x4 *>(w + (b + q) * 64);
            }
    };
    int b = wave * GB;
    if (b < nb) load_w(b, min(nb - b, GB));

    const char *x[MT];
    if (!MADE) {
#pragma unroll
        for (int m = 0; m < MT; m++) {
            const int64_t row = min(static_cast<int64_t>(m * 16 + r16), p.rows - 1);
            x[m] = p.a + row * p.a_pitch + g * 64;
        }
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
#pragma unroll
        for (int m = 0; m < MT; m++)
            x[m] = made + min(m * 16 + r16, rows - 1) * pitch + g * 64;
    }

    f32x4 acc[MT];
#pragma unroll
    for (int m = 0; m < MT; m++) acc[m] = f32x4{0, 0, 0, 0};
    // Units b .. b + n - 1, n = GB with FULL.
    auto group = [&](auto full, int n) {
        constexpr bool FULL = decltype(full)::value;
#pragma unroll
        for (int q = 0; q < GB; q++) {
            if (!FULL && q >= n) break;
            const float s = __uint_as_float((wsc[q] >> (8 * g) & 0xffu) << 23);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const bf16x8 wf = widen4(wv[q][e], s);
#pragma unroll
                for (int m = 0; m < MT; m++)
                    acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        wf, *reinterpret_cast<const bf16x8 *>(x[m] + (b + q) * 256 + e * 16), acc[m],
                        0, 0, 0);
            }
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
#pragma unroll
    for (int m = 0; m < MT; m++) part[wave][m][lane] = acc[m];
    __syncthreads();
    for (int i = t; i < MT * 64; i += kFewWaves * 64) {
        const int m = i / 64, l = i % 64;
        f32x4 s = part[0][m][l];
#pragma unroll
        for (int q = 1; q < kFewWaves; q++) s += part[q][m][l];
        store4(p, m * 16 + (l & 15), j0 + (l >> 4) * 4, s);
    }
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

template <int MT>
void launch_few(const MmLaunch &p, hipStream_t s) {
    const dim3 g(static_cast<unsigned>((p.cols + 15) / 16)), b(kFewWaves * 64);
    few_kernel<MT, kPadded, false><<<g, b, 0, s>>>(p);
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
        few_kernel<1, ET, true><<<g, b, lds, s>>>(p);
    else
        few_kernel<1, ET, false><<<g, b, lds, s>>>(p);
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
    } else if (c.kernel == kFp4Skinny) {
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
        if (a.M <= 16)
            launch_few<1>(p, s);
        else if (a.M <= 32)
            launch_few<2>(p, s);
        else
            launch_few<4>(p, s);
    } else {
        if (quant) {
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
        if (c.kernel == kFp4Tiles && T == 256)
            tiles_kernel<256, 2, 4><<<grid, dim3(512), 0, s>>>(p);
        else if (c.kernel == kFp4Tiles)
            tiles_kernel<128, 2, 2><<<grid, dim3(256), 0, s>>>(p);
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
