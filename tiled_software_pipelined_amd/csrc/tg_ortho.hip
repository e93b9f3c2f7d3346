// Orthogonalised update: Newton-Schulz products that bring the singular
// values of a matrix near one (the update of the Muon optimiser).
//
// X_0 = G / (|G|_F + eps), taken with its rows along the shorter side (m x n,
// m <= n); then for each step, with its coefficients a, b, c:
//
//   A = X X^T,   B = b A + c A^2,   X <- a X + B X.
//
// Where the precision is spent.  Small singular values grow by |a| a step, so
// a rounding of X is amplified with them, by hundreds over five steps, where
// a rounding inside B X is not (it lies along large singular values).  So X
// is held as two half precision numbers, hi + lo (22 bits), and a X is taken
// from both; products use hi alone.  The diagonals of A and B are far larger
// than their other elements and would leave only rounding noise of their own
// size: they are held apart in float (d), so with A = D + A' (A' zero on the
// diagonal) the elements are
//
//   B'_ij = b A'_ij + c ((d_i + d_j) A'_ij + (A'^2)_ij)     (i != j)
//   e_i   = b d_i + c (d_i^2 + (A'^2)_ii)
//   X_i  <- (a + e_i) X_i + (B' X)_i.
//
// Matrices are stored times 2^12: half precision then holds magnitudes from
// 2^-36 to 15 to full precision, and the host refuses coefficients that could
// leave that range.  Against 64 bits the result is off by 0.5 - 1e-3 of its
// norm before its one rounding to bfloat16 (itself 1.7e-3); by up to 4e-3
// where a few equal singular values hold all of the norm, from the rounding
// of X in B X (taking lo into that product would cost half of the update's
// time again).
//
// All products have both operands K-contiguous: X X^T; A' A' (symmetric); and
// B' X with X's transpose, which the update writes beside X, as its second
// operand.  A and B' are symmetric: tiles on and below the diagonal are
// computed and written twice.  The workspace's matrices are padded to whole
// tiles with zeros, which every product keeps zero, so only the first and the
// last kernel meet edges.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>

#include "tg_host.hpp"
#include "tg_nt.hpp"
#include "tgemm.h"

namespace tg {

constexpr float ONE = 4096.0f;  // 2^12, what stands for 1 in the workspace

struct OrthoArgs {
    // matrix z of a batch: the pointers plus z times the strides (elements)
    const _Float16* hi;    // mp x np: X
    const _Float16* lo;
    _Float16* hi_out;      // may be hi, lo: a tile is read and written by its own workgroup
    _Float16* lo_out;
    const _Float16* xt;    // np x mp: X transposed
    _Float16* xt_out;
    _Float16* a;           // mp x mp: A'
    _Float16* b;           // mp x mp: B'
    float* d;              // mp: diagonal of A
    float* e;              // mp: diagonal of B
    uint16_t* out;         // bfloat16 result
    int64_t ldo, stride_o;
    int32_t mp, np, m, n, tall;
    int32_t tiles;         // tiles of one matrix
    int32_t tiles_m, tiles_n;
    float ca, cb, cc;
};

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

template <int N>
struct Halves {
    _Float16 v[N];
};

// The 4 FM values of one column that lane `lane` holds in registers 4 q .. 4 q
// + 3 of fragments 0 .. FM - 1, in row order: rows 4 FM (2 q + lane / 32) + ..
template <int FM>
__device__ __forceinline__ int quad_row(int q, int lane) { return 4 * FM * (2 * q + (lane >> 5)); }

template <class G>
struct OrthoTile {
    int z, tm, tn, m0, n0, wm0, wn0, lane, wave;
    __device__ __forceinline__ OrthoTile(const OrthoArgs& g, bool symmetric) {
        lane = lane_id();
        wave = wave_id();
        const int r = xcd_rank(blockIdx.x, gridDim.x);
        z = r / g.tiles;
        const int t = r - z * g.tiles;
        if (symmetric) {
            // tile t of the lower triangle, row by row
            tm = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
            while (tm * (tm + 1) / 2 > t) --tm;
            while ((tm + 1) * (tm + 2) / 2 <= t) ++tm;
            tn = t - tm * (tm + 1) / 2;
        } else {
            grouped_tile(t, g.tiles_m, g.tiles_n, 4, tm, tn);
        }
        constexpr int WAVES_N = G::BN / G::WTN;
        m0 = tm * G::BM;
        n0 = tn * G::BN;
        wm0 = (wave / WAVES_N) * G::WTM;
        wn0 = (wave % WAVES_N) * G::WTN;
    }
};

__device__ __forceinline__ NtOperands ortho_operands(const _Float16* a, const _Float16* b, int rows_a, int rows_b, int k) {
    return NtOperands{reinterpret_cast<const char*>(a), reinterpret_cast<const char*>(b), nullptr, nullptr,
                      rows_a, rows_b, 2 * k, 2 * (int64_t)k, 2 * (int64_t)k, 0, 0};
}

// Write the wave's block of a symmetric matrix, and its mirror image where the
// tile lies below the diagonal.  value(i, j, r): element of register r.
template <class G, class F>
__device__ __forceinline__ void store_symmetric(_Float16* S, int ld, const OrthoTile<G>& t, F value) {
    const int mb = t.m0 + t.wm0, nb = t.n0 + t.wn0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        Halves<4 * G::FM> col[G::FN];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < G::FM; ++i) {
                Halves<G::FN> row;
#pragma unroll
                for (int j = 0; j < G::FN; ++j) {
                    row.v[j] = (_Float16)value(i, j, 4 * q + e);
                    col[j].v[G::FM * e + i] = row.v[j];
                }
                __builtin_memcpy(S + (int64_t)(mb + G::row_of(i, 4 * q + e, t.lane)) * ld + nb + G::col_of(0, t.lane),
                                 &row, sizeof row);
            }
        if (t.tm != t.tn) {
#pragma unroll
            for (int j = 0; j < G::FN; ++j)
                __builtin_memcpy(S + (int64_t)(nb + G::col_of(j, t.lane)) * ld + mb + quad_row<G::FM>(q, t.lane),
                                 &col[j], sizeof col[j]);
        }
    }
}

// A = X X^T: A' (diagonal zero) and d.
template <class G>
__global__ __launch_bounds__(G::NT) void ortho_gram_kernel(OrthoArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[G::LDS_BYTES];
    const OrthoTile<G> t(g, true);
    const int64_t x = (int64_t)t.z * g.mp * g.np, s = (int64_t)t.z * g.mp * g.mp;
    typename G::Acc acc[G::FM][G::FN];
    G::product(ortho_operands(g.hi + x, g.hi + x, g.mp, g.mp, g.np), t.m0, t.n0, (TG_LDS char*)smem_raw, acc, t.wm0,
               t.wn0, t.lane, t.wave);
    float* d = g.d + (int64_t)t.z * g.mp;
    store_symmetric<G>(g.a + s, g.mp, t, [&](int i, int j, int r) {
        const int row = t.m0 + t.wm0 + G::row_of(i, r, t.lane), col = t.n0 + t.wn0 + G::col_of(j, t.lane);
        const float v = acc[i][j][r] * (1.0f / (ONE * ONE));
        if (row == col) d[row] = v;
        return row == col ? 0.0f : v * ONE;
    });
}

// B = b A + c A^2: B' (diagonal zero) and e.
template <class G>
__global__ __launch_bounds__(G::NT) void ortho_poly_kernel(OrthoArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[G::LDS_BYTES];
    const OrthoTile<G> t(g, true);
    const int64_t s = (int64_t)t.z * g.mp * g.mp;
    const _Float16* A = g.a + s;
    typename G::Acc acc[G::FM][G::FN];
    G::product(ortho_operands(A, A, g.mp, g.mp, g.mp), t.m0, t.n0, (TG_LDS char*)smem_raw, acc, t.wm0, t.wn0, t.lane,
               t.wave);
    const float* d = g.d + (int64_t)t.z * g.mp;
    float* e = g.e + (int64_t)t.z * g.mp;
    float dn[G::FN];
#pragma unroll
    for (int j = 0; j < G::FN; ++j) dn[j] = d[t.n0 + t.wn0 + G::col_of(j, t.lane)];
    store_symmetric<G>(g.b + s, g.mp, t, [&](int i, int j, int r) {
        const int row = t.m0 + t.wm0 + G::row_of(i, r, t.lane), col = t.n0 + t.wn0 + G::col_of(j, t.lane);
        const float dm = d[row], sq = acc[i][j][r] * (1.0f / (ONE * ONE));
        const float av = (float)A[(int64_t)row * g.mp + col] * (1.0f / ONE);
        if (row == col) e[row] = g.cb * dm + g.cc * (dm * dm + sq);
        return row == col ? 0.0f : (g.cb * av + g.cc * ((dm + dn[j]) * av + sq)) * ONE;
    });
}

// X <- (a + e) X + B' X; LAST writes the result instead.
template <class G, bool LAST>
__global__ __launch_bounds__(G::NT) void ortho_update_kernel(OrthoArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[G::LDS_BYTES];
    const OrthoTile<G> t(g, false);
    const int64_t x = (int64_t)t.z * g.mp * g.np, s = (int64_t)t.z * g.mp * g.mp;
    typename G::Acc acc[G::FM][G::FN];
    G::product(ortho_operands(g.b + s, g.xt + x, g.mp, g.np, g.mp), t.m0, t.n0, (TG_LDS char*)smem_raw, acc, t.wm0,
               t.wn0, t.lane, t.wave);
    const float* e = g.e + (int64_t)t.z * g.mp;
    const int mb = t.m0 + t.wm0, nb = t.n0 + t.wn0, n = nb + G::col_of(0, t.lane);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        Halves<4 * G::FM> col[G::FN];
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int i = 0; i < G::FM; ++i) {
                const int m = mb + G::row_of(i, 4 * q + p, t.lane);
                const int64_t at = x + (int64_t)m * g.np + n;
                Halves<G::FN> h, l;
                __builtin_memcpy(&h, g.hi + at, sizeof h);
                __builtin_memcpy(&l, g.lo + at, sizeof l);
                const float k = g.ca + e[m];
                uint16_t o[G::FN];
#pragma unroll
                for (int j = 0; j < G::FN; ++j) {
                    const float y = k * ((float)h.v[j] + (float)l.v[j]) + acc[i][j][4 * q + p] * (1.0f / ONE);
                    if constexpr (LAST) {
                        o[j] = __builtin_bit_cast(uint16_t, (__bf16)(y * (1.0f / ONE)));
                        col[j].v[G::FM * p + i] = __builtin_bit_cast(_Float16, o[j]);
                    } else {
                        h.v[j] = (_Float16)y;
                        l.v[j] = (_Float16)(y - (float)h.v[j]);
                        col[j].v[G::FM * p + i] = h.v[j];
                    }
                }
                if constexpr (LAST) {
                    if (!g.tall && m < g.m) {
                        uint16_t* dst = g.out + (int64_t)t.z * g.stride_o + (int64_t)m * g.ldo + n;
                        if (n + G::FN <= g.n) __builtin_memcpy(dst, o, sizeof o);
                        else
#pragma unroll
                            for (int j = 0; j < G::FN; ++j)
                                if (n + j < g.n) dst[j] = o[j];
                    }
                } else {
                    __builtin_memcpy(g.hi_out + at, &h, sizeof h);
                    __builtin_memcpy(g.lo_out + at, &l, sizeof l);
                }
            }
        const int m = mb + quad_row<G::FM>(q, t.lane);
#pragma unroll
        for (int j = 0; j < G::FN; ++j) {
            if constexpr (LAST) {
                if (g.tall && n + j < g.n) {
                    uint16_t* dst = g.out + (int64_t)t.z * g.stride_o + (int64_t)(n + j) * g.ldo + m;
                    if (m + 4 * G::FM <= g.m) __builtin_memcpy(dst, &col[j], sizeof col[j]);
                    else
#pragma unroll
                        for (int k = 0; k < 4 * G::FM; ++k)
                            if (m + k < g.m) dst[k] = __builtin_bit_cast(uint16_t, col[j].v[k]);
                }
            } else {
                __builtin_memcpy(g.xt_out + x + (int64_t)(n + j) * g.mp + m, &col[j], sizeof col[j]);
            }
        }
    }
}

// ---- the first step's X ------------------------------------------------------

struct OrthoInArgs {
    const void* G;
    int64_t ldg, stride_g;
    int32_t dtype, rows, cols;  // of G
    double* part;               // PARTS sums of squares for each matrix
    _Float16 *hi, *lo, *xt;
    int32_t mp, np, tall;
    double eps;
};

constexpr int PARTS = 64;

__device__ __forceinline__ float element(const void* G, int32_t dtype, int64_t at) {
    if (dtype == TGEMM_F32) return static_cast<const float*>(G)[at];
    const uint16_t v = static_cast<const uint16_t*>(G)[at];
    return dtype == TGEMM_BF16 ? __builtin_bit_cast(float, (uint32_t)v << 16)
                               : (float)__builtin_bit_cast(_Float16, v);
}

// Workgroup (p, z): part p of matrix z's sum of squares, in double (squares
// of any float fit), in a fixed order.
__global__ __launch_bounds__(256) void ortho_norm_kernel(OrthoInArgs g) {
    __shared__ double sums[256];
    const int p = blockIdx.x % PARTS, z = blockIdx.x / PARTS;
    double s = 0.0;
    for (int r = p; r < g.rows; r += PARTS) {
        const int64_t row = (int64_t)z * g.stride_g + (int64_t)r * g.ldg;
        for (int c = threadIdx.x; c < g.cols; c += 256) {
            const double v = element(g.G, g.dtype, row + c);
            s += v * v;
        }
    }
    sums[threadIdx.x] = s;
    for (int w = 128; w > 0; w >>= 1) {
        __syncthreads();
        if (threadIdx.x < w) sums[threadIdx.x] += sums[threadIdx.x + w];
    }
    if (threadIdx.x == 0) g.part[(int64_t)z * PARTS + p] = sums[0];
}

// A workgroup takes a 64 x 64 block of X (padded): X = G / (|G| + eps) times
// 2^12 as hi + lo, and its transpose.
__global__ __launch_bounds__(256) void ortho_load_kernel(OrthoInArgs g) {
    __shared__ float tile[64][65];
    __shared__ double factor;
    const int tn = g.np / 64, per = tn * (g.mp / 64);
    const int z = blockIdx.x / per, b = blockIdx.x - z * per;
    const int m0 = b / tn * 64, n0 = b % tn * 64;
    if (threadIdx.x < 64) {
        double s = g.part[(int64_t)z * PARTS + threadIdx.x];
        for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
        if (threadIdx.x == 0) factor = (double)ONE / (sqrt(s) + g.eps);
    }
    __syncthreads();
    const double f = factor;  // in double: 1 / |G| may leave float's range
    // rows and columns of G: those of X, or the other way round
    const int r0 = g.tall ? n0 : m0, c0 = g.tall ? m0 : n0;
    for (int i = threadIdx.x; i < 64 * 64; i += 256) {
        const int r = i >> 6, c = i & 63;
        float v = 0.0f;
        if (r0 + r < g.rows && c0 + c < g.cols)
            v = (float)(element(g.G, g.dtype, (int64_t)z * g.stride_g + (int64_t)(r0 + r) * g.ldg + c0 + c) * f);
        tile[r][c] = v;
    }
    __syncthreads();
    const int64_t x = (int64_t)z * g.mp * g.np;
    for (int i = threadIdx.x; i < 64 * 64; i += 256) {
        const int r = i >> 6, c = i & 63;
        const float v = g.tall ? tile[c][r] : tile[r][c];
        const _Float16 h = (_Float16)v;
        g.hi[x + (int64_t)(m0 + r) * g.np + n0 + c] = h;
        g.lo[x + (int64_t)(m0 + r) * g.np + n0 + c] = (_Float16)(v - (float)h);
        const float w = g.tall ? tile[r][c] : tile[c][r];
        g.xt[x + (int64_t)(n0 + r) * g.mp + m0 + c] = (_Float16)w;
    }
}

// ---- host ------------------------------------------------------------------------

typedef void (*OrthoFn)(OrthoArgs);
struct OrthoKernels {
    int tile, threads;
    OrthoFn gram, poly, update, last;
};

template <class G>
static OrthoKernels ortho_kernels() {
    return OrthoKernels{G::BM, G::NT, ortho_gram_kernel<G>, ortho_poly_kernel<G>, ortho_update_kernel<G, false>,
                        ortho_update_kernel<G, true>};
}

static const OrthoKernels* ortho_table() {
    static const OrthoKernels t[3] = {
        ortho_kernels<NtGemm<NtF16, 256, 256, 2, 2, 2, false>>(),
        ortho_kernels<NtGemm<NtF16, 128, 128, 2, 2, 4, true>>(),
        ortho_kernels<NtGemm<NtF16, 64, 64, 2, 2, 8, true>>(),
    };
    return t;
}

struct OrthoPlan {
    int64_t m, n, mp, np;
    const OrthoKernels *sym, *upd;
    int64_t off_hi, off_lo, off_t0, off_t1, off_a, off_b, off_d, off_e, off_part, bytes;
};

static int64_t up_to(int64_t v, int64_t step) { return (v + step - 1) / step * step; }

// Tiles, and where things stand in the workspace.
static OrthoPlan ortho_plan(int64_t batch, int64_t rows, int64_t cols) {
    OrthoPlan p{};
    p.m = rows < cols ? rows : cols;
    p.n = rows < cols ? cols : rows;
    const OrthoKernels* t = ortho_table();
    auto tiles = [&](int64_t v, int e) { return (v + t[e].tile - 1) / t[e].tile; };
    auto grid = [&](int e) { return batch * tiles(p.m, e) * tiles(p.n, e); };
    auto tri = [&](int e) { return batch * tiles(p.m, e) * (tiles(p.m, e) + 1) / 2; };
    p.upd = grid(0) >= 192 ? &t[0] : grid(1) >= 128 ? &t[1] : &t[2];
    p.sym = tri(0) >= 192 ? &t[0] : tri(1) >= 128 ? &t[1] : &t[2];
    const int64_t tile = p.upd->tile > p.sym->tile ? p.upd->tile : p.sym->tile;
    p.mp = up_to(p.m, tile);
    p.np = up_to(p.n, tile);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t o = at;
        at += up_to(bytes, 256);
        return o;
    };
    const int64_t x = 2 * batch * p.mp * p.np, s = 2 * batch * p.mp * p.mp;
    p.off_hi = take(x);
    p.off_lo = take(x);
    p.off_t0 = take(x);
    p.off_t1 = take(x);
    p.off_a = take(s);
    p.off_b = take(s);
    p.off_d = take(4 * batch * p.mp);
    p.off_e = take(4 * batch * p.mp);
    p.off_part = take(8 * batch * PARTS);
    p.bytes = at;
    return p;
}

static bool ortho_sizes_ok(int64_t batch, int64_t rows, int64_t cols) {
    // products of padded sizes stay far inside 64 bits, grids inside 32
    return batch >= 0 && rows >= 0 && cols >= 0 && rows <= (1 << 20) && cols <= (1 << 20) && batch <= (1 << 16);
}

// The largest singular value the steps before the last can reach from [0, 1],
// and the largest |b s^2 + c s^4|: NaN or large where the coefficients make
// the iteration leave the range that the workspace holds.
static void ortho_reach(int steps, const double* coef, double* x, double* poly) {
    double top = 1.0, most = 1.0, p = 0.0;
    for (int k = 0; k < steps; ++k) {
        const double a = coef[3 * k], b = coef[3 * k + 1], c = coef[3 * k + 2];
        double next = 0.0;
        for (int i = 0; i <= 4096; ++i) {
            const double s = top * i / 4096.0, q = b * s * s + c * s * s * s * s, y = fabs((a + q) * s);
            if (!(y <= next)) next = y;
            if (!(fabs(q) <= p)) p = fabs(q);
        }
        top = next;
        if (k + 1 < steps && !(top <= most)) most = top;
    }
    *x = most;
    *poly = p;
}

}  // namespace tg

extern "C" {

int64_t tgemm_orthogonalize_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
    using namespace tg;
    if (!ortho_sizes_ok(batch, rows, cols)) return -1;
    if (batch == 0 || rows == 0 || cols == 0) return 0;
    return ortho_plan(batch, rows, cols).bytes;
}

int tgemm_orthogonalize(int64_t batch, int64_t rows, int64_t cols, int32_t dtype, const void* G, int64_t ldg,
                        int64_t stride_g, void* O, int64_t ldo, int64_t stride_o, int32_t steps,
                        const double* coefficients, double eps, void* workspace, int64_t workspace_bytes,
                        void* stream) {
    using namespace tg;
    if (!ortho_sizes_ok(batch, rows, cols)) {
        set_error("batch=%lld rows=%lld cols=%lld out of range", (long long)batch, (long long)rows, (long long)cols);
        return TGEMM_E_ARG;
    }
    if (dtype != TGEMM_F32 && dtype != TGEMM_BF16 && dtype != TGEMM_F16) {
        set_error("dtype %d: float32, bfloat16 or float16 is orthogonalised", dtype);
        return TGEMM_E_ARG;
    }
    if (ldg < cols || ldo < cols) {
        set_error("a leading dimension is shorter than its row");
        return TGEMM_E_ARG;
    }
    if (batch > 1 && ((rows - 1) * ldg + cols > stride_g || (rows - 1) * ldo + cols > stride_o)) {
        set_error("matrices of the batch overlap");
        return TGEMM_E_ARG;
    }
    if (steps < 1 || steps > 64 || !(eps >= 0.0) || !(eps <= 1e30)) {
        set_error("steps=%d (1 .. 64) or eps=%g out of range", steps, eps);
        return TGEMM_E_ARG;
    }
    if (!coefficients) {
        set_error("NULL coefficients");
        return TGEMM_E_NULL;
    }
    for (int i = 0; i < 3 * steps; ++i)
        if (!std::isfinite(coefficients[i])) {
            set_error("coefficient %d is not finite", i);
            return TGEMM_E_ARG;
        }
    double reach, poly;
    ortho_reach(steps, coefficients, &reach, &poly);
    if (!(reach <= 3.5) || !(poly <= 14.0)) {
        set_error("these coefficients let singular values reach %g (3.5) or b s^2 + c s^4 reach %g (14)", reach, poly);
        return TGEMM_E_ARG;
    }
    if (batch == 0 || rows == 0 || cols == 0) {
        clear_error();
        return TGEMM_OK;
    }
    if (!G || !O || !workspace) {
        set_error("NULL matrix or workspace pointer");
        return TGEMM_E_NULL;
    }
    if ((uintptr_t)G % (dtype == TGEMM_F32 ? 4 : 2) || (uintptr_t)O % 2 || (uintptr_t)workspace % 256) {
        set_error("pointer not aligned to its element size, or workspace not 256-byte aligned");
        return TGEMM_E_ALIGN;
    }
    const OrthoPlan p = ortho_plan(batch, rows, cols);
    if (workspace_bytes < p.bytes) {
        set_error("workspace of %lld bytes, %lld needed", (long long)workspace_bytes, (long long)p.bytes);
        return TGEMM_E_ARG;
    }
    const int64_t ut = p.upd->tile, st = p.sym->tile;
    const int64_t tri = (p.mp / st) * (p.mp / st + 1) / 2, upd = (p.mp / ut) * (p.np / ut);
    const int64_t load = (p.mp / 64) * (p.np / 64);
    if (batch * tri > INT_MAX || batch * upd > INT_MAX || batch * load > INT_MAX ||
        (p.upd->tile - 1) * 2 * (p.np > p.mp ? p.np : p.mp) + 128 > INT64_C(0xffffffff)) {
        set_error("too many tiles");
        return TGEMM_E_ARG;
    }
    const int rc = current_device_ok();
    if (rc != TGEMM_OK) return rc;
    char* ws = static_cast<char*>(workspace);
    const hipStream_t s = static_cast<hipStream_t>(stream);

    OrthoInArgs in{};
    in.G = G;
    in.ldg = ldg;
    in.stride_g = stride_g;
    in.dtype = dtype;
    in.rows = (int32_t)rows;
    in.cols = (int32_t)cols;
    in.part = (double*)(ws + p.off_part);
    in.hi = (_Float16*)(ws + p.off_hi);
    in.lo = (_Float16*)(ws + p.off_lo);
    in.xt = (_Float16*)(ws + p.off_t0);
    in.mp = (int32_t)p.mp;
    in.np = (int32_t)p.np;
    in.tall = rows > cols;
    in.eps = eps;
    hipLaunchKernelGGL(ortho_norm_kernel, dim3((unsigned)(PARTS * batch)), dim3(256), 0, s, in);
    hipLaunchKernelGGL(ortho_load_kernel, dim3((unsigned)(batch * load)), dim3(256), 0, s, in);
    hipError_t err = hipGetLastError();

    OrthoArgs g{};
    g.hi = g.hi_out = in.hi;
    g.lo = g.lo_out = in.lo;
    g.a = (_Float16*)(ws + p.off_a);
    g.b = (_Float16*)(ws + p.off_b);
    g.d = (float*)(ws + p.off_d);
    g.e = (float*)(ws + p.off_e);
    g.out = (uint16_t*)O;
    g.ldo = ldo;
    g.stride_o = stride_o;
    g.mp = in.mp;
    g.np = in.np;
    g.m = (int32_t)p.m;
    g.n = (int32_t)p.n;
    g.tall = in.tall;
    auto launch = [&](OrthoFn fn, const OrthoKernels& k, int64_t tiles) {
        if (err != hipSuccess) return;
        g.tiles = (int32_t)tiles;
        g.tiles_m = (int32_t)(p.mp / k.tile);
        g.tiles_n = (int32_t)(p.np / k.tile);
        void* args[] = {&g};
        err = hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)(batch * tiles)), dim3(k.threads), args, 0,
                              s);
    };
    for (int k = 0; k < steps; ++k) {
        g.ca = (float)coefficients[3 * k];
        g.cb = (float)coefficients[3 * k + 1];
        g.cc = (float)coefficients[3 * k + 2];
        g.xt = (const _Float16*)(ws + (k % 2 ? p.off_t1 : p.off_t0));
        g.xt_out = (_Float16*)(ws + (k % 2 ? p.off_t0 : p.off_t1));
        launch(p.sym->gram, *p.sym, tri);
        launch(p.sym->poly, *p.sym, tri);
        launch(k + 1 < steps ? p.upd->update : p.upd->last, *p.upd, upd);
    }
    if (err != hipSuccess) {
        set_error("launch failed: %s", hipGetErrorString(err));
        return TGEMM_E_HIP;
    }
    clear_error();
    return TGEMM_OK;
}

}  // extern "C"
