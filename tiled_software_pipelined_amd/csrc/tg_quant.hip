// Quantisation of a matrix to 8-bit floating point with a power-of-two scale
// for each 128 elements of a row, or for each 128 x 128 block, and the same
// of its transpose, in one pass over the matrix.
//
// For a block with largest finite magnitude a, and FMAX the type's largest
// value: e = the least integer with a <= FMAX 2^e (0 for a block of zeros,
// never below -127), q = x 2^-e rounded to the nearest 8-bit value, ties to
// even.  x 2^-e is exact (where it does not fall below every 8-bit value), so
// q is the only rounding.  With a = m 2^E, 1 <= m < 2, and FMAX = 1.75 2^T:
// e = E - T, one more if m > 1.75; both come from the bits of a.  Scales are
// stored as the byte e + 127, block by block: S[block][row].  NaN stays NaN;
// an infinity, which does not enter a, becomes the type's infinity (e5m2) or
// NaN (e4m3).
//
// A workgroup of 256 threads takes one 128 x 128 block: thread (rg, cg)
// holds rows 8 rg .. 8 rg + 7 of columns 8 cg .. 8 cg + 7, loaded once.  A
// row's 16 threads are one 16-lane DPP row, so its maximum takes four
// register rotations; a column's maximum goes through LDS.  The transposed
// image is written from LDS, each thread having put 8 rows of a column
// there as one 8-byte word.
//
// Bound by memory, every element read once and each image written once, as
// long as the vector work stays small: maxima are taken over the integer
// patterns, two 16-bit elements to an instruction, and the conversion
// instructions divide by 2^e themselves, two values at a time (widening every
// element, with comparisons and products in float, took 31 us a call for bfloat16
// 8192x4096 with both images; now 27.4, of which the kernel 24.7, 5.5 TB/s; a plain
// copy of as many bytes takes 26).
#include <hip/hip_runtime.h>

#include <climits>
#include <type_traits>

#include "tg_device.hpp"
#include "tg_fp8.hpp"
#include "tg_host.hpp"
#include "tgemm.h"

namespace tg {

struct QuantArgs {
    const void* X;
    uint8_t* Q;
    uint8_t* S;
    uint8_t* Qt;
    uint8_t* St;
    int64_t ldx, ldq, lds, ldqt, ldst;
    int32_t rows, cols, blocks_c;
    int32_t by_xcd;  // 1: neighbouring blocks run on one XCD
};

template <int FMT>
__device__ __forceinline__ int scale_exponent(float amax) {
    constexpr int top = FMT == FMT_E4M3 ? 8 : 15;
    const uint32_t b = __builtin_bit_cast(uint32_t, amax);
    const int e = (int)(b >> 23) - 127 - top + ((b & 0x7fffff) > 0x600000);
    return b == 0 ? 0 : max(e, -127);
}

// What the conversions divide by: they take 2^e from the exponent's bits alone
// (0 for e = -127).
__device__ __forceinline__ float scale_of(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

typedef int16_t s16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Eight elements of a row are WORDS registers.  order(w): magnitudes so biased
// that unsigned comparison orders the finite ones above every infinity and
// NaN, which wrap around to the bottom; bigger: the larger of each; top: the
// largest in a word; magnitude: back to a float, 0 where nothing was finite.
// pair / column: two neighbours of a row / of a column to 8 bits, divided by
// the scale and rounded to nearest even, into half HI of a word.
struct InF32 {
    typedef float T;
    static constexpr int WORDS = 8;
    static constexpr uint32_t BIAS = 0x80800000u;
    __device__ static __forceinline__ uint32_t order(uint32_t w) { return (w & 0x7fffffffu) + BIAS; }
    __device__ static __forceinline__ uint32_t bigger(uint32_t a, uint32_t b) { return max(a, b); }
    __device__ static __forceinline__ uint32_t top(uint32_t w) { return w; }
    __device__ static __forceinline__ float magnitude(uint32_t m) {
        return __builtin_bit_cast(float, m >= BIAS ? m - BIAS : 0u);
    }
    template <int FMT, bool HI>
    __device__ static __forceinline__ s16x2 convert(float x, float y, s16x2 old, float scale) {
        if constexpr (FMT == FMT_E4M3) return __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(old, x, y, scale, HI);
        else return __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(old, x, y, scale, HI);
    }
    template <int FMT, bool HI>
    __device__ static __forceinline__ s16x2 pair(const uint32_t* w, int j, s16x2 old, float scale) {
        return convert<FMT, HI>(__builtin_bit_cast(float, w[j]), __builtin_bit_cast(float, w[j + 1]), old, scale);
    }
    template <int FMT, bool HI>
    __device__ static __forceinline__ s16x2 column(const uint32_t* r, const uint32_t* next, int j, s16x2 old, float scale) {
        return convert<FMT, HI>(__builtin_bit_cast(float, r[j]), __builtin_bit_cast(float, next[j]), old, scale);
    }
};
template <bool BF>
struct In16 {
    typedef uint16_t T;
    static constexpr int WORDS = 4;
    static constexpr uint16_t BIAS = BF ? 0x8080 : 0x8400;  // largest finite + BIAS = 0xffff
    __device__ static __forceinline__ uint32_t order(uint32_t w) {
        const u16x2 m = __builtin_bit_cast(u16x2, w & 0x7fff7fffu) + u16x2{BIAS, BIAS};
        return __builtin_bit_cast(uint32_t, m);
    }
    __device__ static __forceinline__ uint32_t bigger(uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                      __builtin_bit_cast(u16x2, b)));
    }
    __device__ static __forceinline__ uint32_t top(uint32_t w) { return max(w & 0xffffu, w >> 16); }
    __device__ static __forceinline__ float magnitude(uint32_t m) {
        const uint16_t b = m >= BIAS ? (uint16_t)(m - BIAS) : 0;
        if constexpr (BF) return __builtin_bit_cast(float, (uint32_t)b << 16);
        else return (float)__builtin_bit_cast(_Float16, b);
    }
    template <int FMT, bool HI>
    __device__ static __forceinline__ s16x2 convert(uint32_t w, s16x2 old, float scale) {
        if constexpr (BF) {
            const bf16x2 v = __builtin_bit_cast(bf16x2, w);
            if constexpr (FMT == FMT_E4M3) return __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(old, v, scale, HI);
            else return __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(old, v, scale, HI);
        } else {
            const f16x2 v = __builtin_bit_cast(f16x2, w);
            if constexpr (FMT == FMT_E4M3) return __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(old, v, scale, HI);
            else return __builtin_amdgcn_cvt_scalef32_pk_bf8_f16(old, v, scale, HI);
        }
    }
    template <int FMT, bool HI>
    __device__ static __forceinline__ s16x2 pair(const uint32_t* w, int j, s16x2 old, float scale) {
        return convert<FMT, HI>(w[j / 2], old, scale);
    }
    template <int FMT, bool HI>
    __device__ static __forceinline__ s16x2 column(const uint32_t* r, const uint32_t* next, int j, s16x2 old, float scale) {
        return convert<FMT, HI>(__builtin_amdgcn_perm(next[j / 2], r[j / 2], j % 2 ? 0x07060302u : 0x05040100u), old, scale);
    }
};
typedef In16<true> InBF16;
typedef In16<false> InF16;

// Maximum over the 16 lanes of a DPP row, in all of them.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
    auto turn = [](uint32_t x, auto ctrl) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, 0xf, 0xf, false);
    };
    v = max(v, turn(v, std::integral_constant<int, 0x128>{}));  // row_ror:8, 4, 2, 1
    v = max(v, turn(v, std::integral_constant<int, 0x124>{}));
    v = max(v, turn(v, std::integral_constant<int, 0x122>{}));
    v = max(v, turn(v, std::integral_constant<int, 0x121>{}));
    return v;
}

template <class In, int FMT, bool SQUARE, bool TRANS>
__global__ __launch_bounds__(256) void quantize_kernel(QuantArgs g) {
    typedef typename In::T T;
    constexpr int WORDS = In::WORDS, PW = 8 / WORDS;  // PW columns in a word
    __shared__ __attribute__((aligned(16))) char image[TRANS ? 128 * 128 : 16];
    __shared__ __attribute__((aligned(16))) uint32_t most[4][16 * WORDS];
    __shared__ uint8_t row_scale[128];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int cg = tid & 15, rg = tid >> 4;
    const int rank = g.by_xcd ? xcd_rank(blockIdx.x, gridDim.x) : blockIdx.x;
    const int bc = rank % g.blocks_c, br = rank / g.blocks_c;
    const int r0 = br * 128, c0 = bc * 128;
    const int col = c0 + 8 * cg;

    uint32_t x[8][WORDS];
    {
        const bool whole = col + 8 <= g.cols;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            // rows past the last are read from it and dropped
            const T* src = static_cast<const T*>(g.X) + (int64_t)min(r0 + 8 * rg + p, g.rows - 1) * g.ldx;
            union { T t[8]; i32x4 v[WORDS / 4]; } u;
            if (whole) {
#pragma unroll
                for (int h = 0; h < WORDS / 4; ++h) u.v[h] = load16(src + col + 4 * PW * h);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) u.t[j] = load_or_zero(src + col + j, col + j < g.cols);
            }
#pragma unroll
            for (int w = 0; w < WORDS; ++w) x[p][w] = (uint32_t)u.v[w / 4][w % 4];
        }
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const bool in = r0 + 8 * rg + p < g.rows;
#pragma unroll
            for (int w = 0; w < WORDS; ++w) x[p][w] = in ? x[p][w] : 0u;
        }
    }

    // the scales of the rows
    float scale[8];
    int block_e = 0;
    {
        uint32_t m[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            m[p] = In::order(x[p][0]);
#pragma unroll
            for (int w = 1; w < WORDS; ++w) m[p] = In::bigger(m[p], In::order(x[p][w]));
        }
        if constexpr (SQUARE) {
#pragma unroll
            for (int p = 1; p < 8; ++p) m[0] = In::bigger(m[0], m[p]);
            const uint32_t top = row16_max(In::top(m[0]));
            if ((lane & 15) == 0) most[wave][lane >> 4] = top;
            __syncthreads();
            uint32_t all = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int q = 0; q < 4; ++q) all = max(all, most[w][q]);
            block_e = scale_exponent<FMT>(In::magnitude(all));
#pragma unroll
            for (int p = 0; p < 8; ++p) scale[p] = scale_of(block_e);
        } else {
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const int e = scale_exponent<FMT>(In::magnitude(row16_max(In::top(m[p]))));
                scale[p] = scale_of(e);
                if (cg == 0) row_scale[8 * rg + p] = (uint8_t)(e + 127);
            }
        }
    }

    // the image of the rows
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        s16x2 w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[h] = In::template pair<FMT, false>(x[p], 4 * h, s16x2{0, 0}, scale[p]);
            w[h] = In::template pair<FMT, true>(x[p], 4 * h + 2, w[h], scale[p]);
        }
        const int r = r0 + 8 * rg + p;
        if (r < g.rows) {
            uint8_t* dst = g.Q + (int64_t)r * g.ldq + col;
            if (col + 8 <= g.cols) {
                __builtin_memcpy(dst, w, 8);
            } else {
                uint8_t b[8];
                __builtin_memcpy(b, w, 8);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + j < g.cols) dst[j] = b[j];
            }
        }
    }

    // the transposed image, into LDS: column c's 128 rows at 128 c, its
    // 8-byte word of row group rg at word rg ^ (c / 8)
    if constexpr (TRANS) {
        float col_scale[8];
        if constexpr (SQUARE) {
#pragma unroll
            for (int j = 0; j < 8; ++j) col_scale[j] = scale[0];
        } else {
#pragma unroll
            for (int w = 0; w < WORDS; ++w) {
                uint32_t m = In::order(x[0][w]);
#pragma unroll
                for (int p = 1; p < 8; ++p) m = In::bigger(m, In::order(x[p][w]));
                m = In::bigger(m, (uint32_t)__shfl_xor((int)m, 16, 64));
                m = In::bigger(m, (uint32_t)__shfl_xor((int)m, 32, 64));
                if (lane < 16) most[wave][WORDS * cg + w] = m;
            }
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WORDS; ++w) {
                const int c = WORDS * cg + w;
                const uint32_t m = In::bigger(In::bigger(most[0][c], most[1][c]), In::bigger(most[2][c], most[3][c]));
#pragma unroll
                for (int k = 0; k < PW; ++k) {
                    const int j = PW * w + k;
                    const int e = scale_exponent<FMT>(In::magnitude(PW == 1 ? m : k ? m >> 16 : m & 0xffffu));
                    col_scale[j] = scale_of(e);
                    if (rg == 0 && col + j < g.cols) g.St[(int64_t)br * g.ldst + col + j] = (uint8_t)(e + 127);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s16x2 w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w[h] = In::template column<FMT, false>(x[4 * h], x[4 * h + 1], j, s16x2{0, 0}, col_scale[j]);
                w[h] = In::template column<FMT, true>(x[4 * h + 2], x[4 * h + 3], j, w[h], col_scale[j]);
            }
            __builtin_memcpy(image + (8 * cg + j) * 128 + 8 * (rg ^ cg), w, 8);
        }
    }
    __syncthreads();  // row_scale and image are whole

    if constexpr (SQUARE) {
        if (tid < 128) {
            if (r0 + tid < g.rows) g.S[(int64_t)bc * g.lds + r0 + tid] = (uint8_t)(block_e + 127);
        } else if (TRANS && c0 + tid - 128 < g.cols) {
            g.St[(int64_t)br * g.ldst + c0 + tid - 128] = (uint8_t)(block_e + 127);
        }
    } else {
        if (tid < 128 && r0 + tid < g.rows) g.S[(int64_t)bc * g.lds + r0 + tid] = row_scale[tid];
    }
    if constexpr (TRANS) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = 32 * q + (tid >> 3), v = tid & 7;  // 16 rows: words 2 v, 2 v + 1
            const int x16 = (2 * v) ^ ((c >> 3) & 14);
            i32x4 w = *reinterpret_cast<const i32x4*>(image + c * 128 + 8 * x16);
            if ((c >> 3) & 1) w = i32x4{w.z, w.w, w.x, w.y};
            const int r = r0 + 16 * v;
            if (c0 + c < g.cols && r < g.rows) {
                uint8_t* dst = g.Qt + (int64_t)(c0 + c) * g.ldqt + r;
                if (r + 16 <= g.rows) {
                    __builtin_memcpy(dst, &w, 16);
                } else {
                    union { i32x4 w; uint8_t b[16]; } u;
                    u.w = w;
#pragma unroll
                    for (int t = 0; t < 16; ++t)
                        if (r + t < g.rows) dst[t] = u.b[t];
                }
            }
        }
    }
}

typedef void (*QuantFn)(QuantArgs);

template <class In, int FMT>
static QuantFn quant_fn(bool square, bool trans) {
    if (square) return trans ? quantize_kernel<In, FMT, true, true> : quantize_kernel<In, FMT, true, false>;
    return trans ? quantize_kernel<In, FMT, false, true> : quantize_kernel<In, FMT, false, false>;
}
template <class In>
static QuantFn quant_fn(int fmt, bool square, bool trans) {
    return fmt == FMT_E4M3 ? quant_fn<In, FMT_E4M3>(square, trans) : quant_fn<In, FMT_E5M2>(square, trans);
}

}  // namespace tg

extern "C" int tgemm_fp8_quantize(int64_t rows, int64_t cols, int32_t dtype, const void* X, int64_t ldx, int32_t fmt,
                                  int32_t block, void* Q, int64_t ldq, void* S, int64_t lds, void* Qt, int64_t ldqt,
                                  void* St, int64_t ldst, void* stream) {
    using namespace tg;
    const bool trans = Qt != nullptr || St != nullptr;
    if (rows < 0 || cols < 0 || rows > INT_MAX - 256 || cols > INT_MAX - 256) {
        set_error("rows=%lld cols=%lld out of range", (long long)rows, (long long)cols);
        return TGEMM_E_ARG;
    }
    if (dtype != TGEMM_F32 && dtype != TGEMM_BF16 && dtype != TGEMM_F16) {
        set_error("dtype %d: float32, bfloat16 or float16 is quantised", dtype);
        return TGEMM_E_ARG;
    }
    if ((fmt != TGEMM_E4M3 && fmt != TGEMM_E5M2) || (block != TGEMM_BLOCK_ROW && block != TGEMM_BLOCK_SQUARE)) {
        set_error("unknown format %d or block %d", fmt, block);
        return TGEMM_E_ARG;
    }
    if (ldx < cols || ldq < cols || lds < rows || (trans && (ldqt < rows || ldst < cols))) {
        set_error("a leading dimension is shorter than its row");
        return TGEMM_E_ARG;
    }
    if (ldx > MOST_STRIDE || ldq > MOST_STRIDE || lds > MOST_STRIDE || (trans && (ldqt > MOST_STRIDE || ldst > MOST_STRIDE))) {
        set_error("a leading dimension is out of range");
        return TGEMM_E_ARG;
    }
    if (rows == 0 || cols == 0) {
        clear_error();
        return TGEMM_OK;
    }
    if (!X || !Q || !S || (trans && (!Qt || !St))) {
        set_error("NULL matrix or scale pointer");
        return TGEMM_E_NULL;
    }
    if ((uintptr_t)X % (dtype == TGEMM_F32 ? 4 : 2)) {
        set_error("X not aligned to its element size");
        return TGEMM_E_ALIGN;
    }
    const int64_t blocks_c = (cols + 127) / 128, blocks = blocks_c * ((rows + 127) / 128);
    if (blocks > INT_MAX || !grid_fits((double)blocks, 256)) {
        set_error("%lld x %lld has too many blocks", (long long)rows, (long long)cols);
        return TGEMM_E_ARG;
    }
    const int rc = current_device_ok();
    if (rc != TGEMM_OK) return rc;
    QuantArgs g{X, (uint8_t*)Q, (uint8_t*)S, (uint8_t*)Qt, (uint8_t*)St, ldx, ldq, lds, ldqt, ldst,
                (int32_t)rows, (int32_t)cols, (int32_t)blocks_c, 0};
    // Images whose rows are not whole cache lines: blocks that share lines run
    // on one XCD, whose L2 joins their writes (float 4095x4104, both images:
    // 31 -> 26 us).  Whole lines go faster dealt over all XCDs (bfloat16
    // 8192x4096, both images: 30 us against 36).
    g.by_xcd = ldq % 128 != 0 || (trans && ldqt % 128 != 0);
    const bool square = block == TGEMM_BLOCK_SQUARE;
    const QuantFn fn = dtype == TGEMM_F32 ? quant_fn<InF32>(fmt, square, trans)
                       : dtype == TGEMM_BF16 ? quant_fn<InBF16>(fmt, square, trans)
                                             : quant_fn<InF16>(fmt, square, trans);
    void* args[] = {&g};
    const hipError_t err = hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)blocks), dim3(256), args, 0,
                                           static_cast<hipStream_t>(stream));
    if (err != hipSuccess) {
        set_error("launch of the quantiser failed: %s", hipGetErrorString(err));
        return TGEMM_E_HIP;
    }
    clear_error();
    return TGEMM_OK;
}
