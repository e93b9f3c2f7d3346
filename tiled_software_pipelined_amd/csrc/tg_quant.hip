// Quantisation of a matrix to 8-bit floating point with a power-of-two scale
// for each 128 elements of a row, or for each 128 x 128 block, and the same
// of its transpose, in one pass over the matrix.
//
// For a block with largest finite magnitude a, and FMAX the type's largest
// value: e = the least integer with a <= FMAX 2^e (0 for a block of zeros,
// never below -127), q = x 2^-e rounded to the nearest 8-bit value, ties to
// even.  2^-e is a normal float and the product with it is exact (where it
// does not fall below every 8-bit value), so q is the only rounding.  With
// a = m 2^E, 1 <= m < 2, and FMAX = 1.75 2^T: e = E - T, one more if m > 1.75;
// both come from the bits of a.  Scales are stored as the byte e + 127, block
// by block: S[block][row].  NaN stays NaN; an infinity, which does not enter
// a, becomes the type's infinity (e5m2) or NaN (e4m3).
//
// A workgroup of 256 threads takes one 128 x 128 block: thread (rg, cg)
// holds rows 8 rg .. 8 rg + 7 of columns 8 cg .. 8 cg + 7, loaded once.  A
// row's 16 threads are one 16-lane DPP row, so its maximum takes four
// register rotations; a column's maximum goes through LDS.  The transposed
// image is written from LDS, each thread having put 8 rows of a column
// there as one 8-byte word.  Bound by memory: every element is read once and
// each image written once.
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
};

template <int FMT>
__device__ __forceinline__ int scale_exponent(float amax) {
    constexpr int top = FMT == FMT_E4M3 ? 8 : 15;
    const uint32_t b = __builtin_bit_cast(uint32_t, amax);
    const int e = (int)(b >> 23) - 127 - top + ((b & 0x7fffff) > 0x600000);
    return b == 0 ? 0 : max(e, -127);
}

// 2^-e, -127 <= e <= 120
__device__ __forceinline__ float inverse_scale(int e) { return __builtin_bit_cast(float, (uint32_t)(127 - e) << 23); }

__device__ __forceinline__ float finite_abs(float x) {
    const float a = __builtin_fabsf(x);
    return a < __builtin_inff() ? a : 0.0f;  // false for NaN too
}

// Two 8-bit values into half `HI` of a word.
template <int FMT, bool HI>
__device__ __forceinline__ int pack2(float x, float y, int old) {
    if constexpr (FMT == FMT_E4M3) return __builtin_amdgcn_cvt_pk_fp8_f32(x, y, old, HI);
    else return __builtin_amdgcn_cvt_pk_bf8_f32(x, y, old, HI);
}
template <int FMT>
__device__ __forceinline__ i32x2 pack8(const float (&y)[8]) {
    i32x2 w;
    w.x = pack2<FMT, true>(y[2], y[3], pack2<FMT, false>(y[0], y[1], 0));
    w.y = pack2<FMT, true>(y[6], y[7], pack2<FMT, false>(y[4], y[5], 0));
    return w;
}

// Maximum over the 16 lanes of a DPP row, in all of them.
__device__ __forceinline__ float row16_max(float v) {
    auto turn = [](float x, auto ctrl) {
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value,
                                                                     0xf, 0xf, false));
    };
    v = fmaxf(v, turn(v, std::integral_constant<int, 0x128>{}));  // row_ror:8, 4, 2, 1
    v = fmaxf(v, turn(v, std::integral_constant<int, 0x124>{}));
    v = fmaxf(v, turn(v, std::integral_constant<int, 0x122>{}));
    v = fmaxf(v, turn(v, std::integral_constant<int, 0x121>{}));
    return v;
}

struct InF32 {
    typedef float T;
    __device__ static __forceinline__ float up(float x) { return x; }
};
struct InBF16 {
    typedef uint16_t T;
    __device__ static __forceinline__ float up(uint16_t x) { return __builtin_bit_cast(float, (uint32_t)x << 16); }
};
struct InF16 {
    typedef uint16_t T;
    __device__ static __forceinline__ float up(uint16_t x) { return (float)__builtin_bit_cast(_Float16, x); }
};

template <class In, int FMT, bool SQUARE, bool TRANS>
__global__ __launch_bounds__(256) void quantize_kernel(QuantArgs g) {
    typedef typename In::T T;
    __shared__ __attribute__((aligned(16))) char image[TRANS ? 128 * 128 : 16];
    __shared__ __attribute__((aligned(16))) float most[4][128];
    __shared__ uint8_t row_scale[128];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int cg = tid & 15, rg = tid >> 4;
    const int bc = blockIdx.x % g.blocks_c, br = blockIdx.x / g.blocks_c;
    const int r0 = br * 128, c0 = bc * 128;
    const int col = c0 + 8 * cg;

    float x[8][8];
    {
        const bool whole = col + 8 <= g.cols;
        union { T t[8]; i32x4 v[sizeof(T) / 2]; } u[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            // rows past the last are read from it and dropped
            const T* src = static_cast<const T*>(g.X) + (int64_t)min(r0 + 8 * rg + p, g.rows - 1) * g.ldx;
            if (whole) {
#pragma unroll
                for (int h = 0; h < (int)sizeof(T) / 2; ++h) u[p].v[h] = load16(src + col + 8 * h * 2 / (int)sizeof(T));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) u[p].t[j] = load_or_zero(src + col + j, col + j < g.cols);
            }
        }
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const bool in = r0 + 8 * rg + p < g.rows;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[p][j] = in ? In::up(u[p].t[j]) : 0.0f;
        }
    }

    float inv[8];  // of the rows (SQUARE: all the same)
    int block_e = 0;
    if constexpr (SQUARE) {
        float a = 0.0f;
#pragma unroll
        for (int p = 0; p < 8; ++p)
#pragma unroll
            for (int j = 0; j < 8; ++j) a = fmaxf(a, finite_abs(x[p][j]));
        a = row16_max(a);
        if ((lane & 15) == 0) most[wave][lane >> 4] = a;
        __syncthreads();
        a = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int q = 0; q < 4; ++q) a = fmaxf(a, most[w][q]);
        block_e = scale_exponent<FMT>(a);
#pragma unroll
        for (int p = 0; p < 8; ++p) inv[p] = inverse_scale(block_e);
    } else {
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            float a = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) a = fmaxf(a, finite_abs(x[p][j]));
            const int e = scale_exponent<FMT>(row16_max(a));
            inv[p] = inverse_scale(e);
            if (cg == 0) row_scale[8 * rg + p] = (uint8_t)(e + 127);
        }
    }

    // the image of the rows
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[p][j] * inv[p];
        const i32x2 w = pack8<FMT>(y);
        const int r = r0 + 8 * rg + p;
        if (r < g.rows) {
            uint8_t* dst = g.Q + (int64_t)r * g.ldq + col;
            if (col + 8 <= g.cols) {
                __builtin_memcpy(dst, &w, 8);
            } else {
                union { i32x2 w; uint8_t b[8]; } u;
                u.w = w;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + j < g.cols) dst[j] = u.b[j];
            }
        }
    }

    // the transposed image, into LDS: column c's 128 rows at 128 c, its
    // 8-byte word of row group rg at word rg ^ (c / 8)
    float col_inv[8];
    if constexpr (TRANS && !SQUARE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float a = 0.0f;
#pragma unroll
            for (int p = 0; p < 8; ++p) a = fmaxf(a, finite_abs(x[p][j]));
            a = fmaxf(a, __shfl_xor(a, 16, 64));
            a = fmaxf(a, __shfl_xor(a, 32, 64));
            if (lane < 16) most[wave][8 * cg + j] = a;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = 8 * cg + j;
            const float a = fmaxf(fmaxf(most[0][c], most[1][c]), fmaxf(most[2][c], most[3][c]));
            const int e = scale_exponent<FMT>(a);
            col_inv[j] = inverse_scale(e);
            if (rg == 0 && col + j < g.cols) g.St[(int64_t)br * g.ldst + col + j] = (uint8_t)(e + 127);
        }
    }
    if constexpr (TRANS) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float y[8];
#pragma unroll
            for (int p = 0; p < 8; ++p) y[p] = x[p][j] * (SQUARE ? inv[0] : col_inv[j]);
            *reinterpret_cast<i32x2*>(image + (8 * cg + j) * 128 + 8 * (rg ^ cg)) = pack8<FMT>(y);
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
    if (blocks > INT_MAX) {
        set_error("%lld x %lld has too many blocks", (long long)rows, (long long)cols);
        return TGEMM_E_ARG;
    }
    const int rc = current_device_ok();
    if (rc != TGEMM_OK) return rc;
    QuantArgs g{X, (uint8_t*)Q, (uint8_t*)S, (uint8_t*)Qt, (uint8_t*)St, ldx, ldq, lds, ldqt, ldst,
                (int32_t)rows, (int32_t)cols, (int32_t)blocks_c};
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
