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
// is held as two half precision numbers, hi + lo, and a X is taken from both;
// products use hi alone (with up to 64 rows lo too, see below).  The diagonals of
// A and B are far larger than their other elements and would leave only rounding
// noise of their own size: they are held apart in float (d), so with A = D + A'
// (A' zero on the diagonal) the elements are
//
//   B'_ij = b A'_ij + c ((d_i + d_j) A'_ij + (A'^2)_ij)     (i != j)
//   e_i   = b d_i + c (d_i^2 + (A'^2)_ii)
//   X_i  <- (a + e_i) X_i + (B' X)_i.
//
// e_i X_i takes lo, and B' X only hi: what is left out is B' lo.  Of matrices of
// low rank B lo is next to nothing, but e_i lo_i alone is noise of full rank, of
// which the part outside X's few singular vectors grows by |a| a step.  e_i is
// about the sum of B's eigenvalues over m, so this shows where rows are few (rank
// one: 4e-2 of the result's norm at 3 x 21, 6e-3 at 64 x 65).  Up to 64 rows,
// where a product is bound by its launch and copies, lo is taken into X X^T and B
// X: rank one then comes to 1e-3 (a call of 64 x 256 49 -> 52 us, of 64 x 4096 73
// -> 81, of 300 of 40 x 70 93 -> 106).  More rows: a row i whose A' is large beside
// d_i, |A'_i|^2 > d_i^2 (for a projection: less than half of the row's unit vector
// lies in it), takes e_i from hi as well, so that what is left out is B lo;
// others take it from hi + lo, where B' lo is the smaller (random elements, 300 x
// 301: 6e-4 against 1.3e-3).  Rank one, 65 x 70: 6e-3 -> 1e-3.
//
// hi, A' and B' are rounded up or down by thresholds of an element's place, not
// to nearest (see Dither below).
//
// Matrices are stored times 2^12: half precision then holds magnitudes from
// 2^-26 to 15 to full precision, and smaller ones in steps of 2^-36; the host
// refuses coefficients that could leave that range.  hi + lo is off by up to
// 2^-21 of an element, or by 2^-37 where that is more.  Against 64 bits the result is off by
// 0.5 - 1.3e-3 of its norm before its one rounding to bfloat16 (itself 1.7e-3)
// for random matrices, and by at most 5.5e-3 in 6000 of low rank or with repeated
// elements (emulated; the tests hold the kernels to the emulation).
//
// All products have both operands K-contiguous: X X^T; A' A' (symmetric); and
// B' X with X's transpose, which the update writes beside X, as its second
// operand.  A and B' are symmetric: tiles on and below the diagonal are
// computed and written twice.  The workspace's X is padded to whole update
// tiles with zeros, which every product keeps zero, so only the first and the
// last kernel meet the edges of G and O.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <type_traits>

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
    _Float16* a;           // ms x ms: A'
    _Float16* b;           // ms x ms: B'
    float* d;              // ms: diagonal of A
    float* e;              // ms: diagonal of B
    float* part;           // split gram: parts x 4096 floats for each tile
    int32_t* arrived;      // split gram: one counter a tile, zero between launches
    uint16_t* out;         // bfloat16 result
    int64_t ldo, stride_o;
    int32_t mp, np, ms, m, n, tall;
    int32_t tiles;             // tiles of one matrix
    int32_t tiles_m, tiles_n;  // of the update
    int32_t parts, run;        // split gram: workgroups a tile, columns of X for each
    float ca, cb, cc;
};

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

// e_i's last bit says which of the two its row takes (see above).
__device__ __forceinline__ float with_choice(float e, bool high_only) {
    return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, e) & ~1u) | (uint32_t)high_only);
}
__device__ __forceinline__ bool high_only(float e) { return __builtin_bit_cast(uint32_t, e) & 1u; }

template <int N>
struct Halves {
    _Float16 v[N];
};

// Rounding to half precision, up or down by a threshold of the element's place,
// so that equal elements are not all off the same way: rounded to nearest, equal
// elements of X, A' and B' move a singular value together (4 blocks of 50 x 125
// ones on the diagonal: result off by 1.5e-2 of its norm, now 1e-3; one
// rounding's error at random places grows by a half).  The thresholds of matrix S
// are the fractions of (m n C + m R + n D) / 2^32.  C / 2^32 is far from simple
// fractions, so they are spread evenly along every row and column, like the phases
// of a chirp, and rows do not resemble each other; for A and B, R = D keeps them
// symmetric.  A NaN may change in A' or B'; X keeps it.
//
// Elements are visited one after the other, down a column or along a row: an
// addition makes the next threshold (a call of 256 x 256: a product for each
// 74.6 us, so 72.5, rounding to nearest 70.5).
// The 13 bits that a float has beyond half precision are carried into by the
// threshold's, and cut off by the conversion.
enum Rounded { ROUND_X = 0, ROUND_A, ROUND_B };
template <Rounded S>
struct Dither {
    static constexpr uint32_t C = S == ROUND_X ? 0xd1b54a33u : S == ROUND_A ? 0x9e3779b1u : 0xb5297a4du;
    static constexpr uint32_t R = S == ROUND_X ? 0x8cb92ba7u : S == ROUND_A ? 0x68e31da4u : 0x1b56c4e9u;
    static constexpr uint32_t D = S == ROUND_X ? 0xabc98389u : R;
    uint32_t at, step;
    // from element (m, n): the next is (m + 1, n) or (m, n + 1)
    __device__ __forceinline__ static Dither down(int m, int n) {
        const uint32_t step = (uint32_t)n * C + R;
        return Dither{(uint32_t)m * step + (uint32_t)n * D, step};
    }
    __device__ __forceinline__ static Dither along(int m, int n) {
        const uint32_t step = (uint32_t)m * C + D;
        return Dither{(uint32_t)n * step + (uint32_t)m * R, step};
    }
    __device__ __forceinline__ _Float16 round(float x) {
        const uint32_t b = __builtin_bit_cast(uint32_t, x) + (at >> 19);
        at += step;
        const auto h = __builtin_amdgcn_cvt_pkrtz(__builtin_bit_cast(float, b), 0.0f);
        return (_Float16)h[0];
    }
};

// The 4 FM values of one column that lane `lane` holds in registers 4 q .. 4 q
// + 3 of fragments 0 .. FM - 1, in row order: rows 4 FM (2 q + lane / 32) + ..
template <int FM>
__device__ __forceinline__ int quad_row(int q, int lane) { return 4 * FM * (2 * q + (lane >> 5)); }

// The diagonal's entries of those 4 FM rows.
template <int FM>
struct QuadDiagonal {
    float v[4 * FM];
    __device__ __forceinline__ void load(const float* d, int m) { __builtin_memcpy(v, d + m, sizeof v); }
};

// Tile t of the lower triangle (tn <= tm): bands of BAND tile rows, each
// walked column by column, so that the tiles that run on one XCD at a time
// share operand panels.
constexpr int BAND = 6;
__device__ __forceinline__ void lower_tile(int t, int tile_rows, int& tm, int& tn) {
    int row = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);  // if walked row by row
    while (row * (row + 1) / 2 > t) --row;
    while ((row + 1) * (row + 2) / 2 <= t) ++row;
    const int first = row / BAND * BAND;
    int u = t - first * (first + 1) / 2;
    // columns 0 .. first hold BAND tiles of the band each (fewer in a last,
    // partial band), later ones one less each
    const int rows = min(BAND, tile_rows - first);
    if (u < (first + 1) * rows) {
        tn = u / rows;
        tm = first + u - tn * rows;
        return;
    }
    u -= (first + 1) * rows;
    tn = first + 1;
    while (u >= first + rows - tn) u -= first + rows - tn++;
    tm = tn + u;
}

template <class G>
struct OrthoTile {
    int z, tm, tn, m0, n0, wm0, wn0, lane, wave;
    __device__ __forceinline__ OrthoTile(const OrthoArgs& g, bool symmetric)
        : OrthoTile(g, symmetric, xcd_rank(blockIdx.x, gridDim.x)) {}
    // tile r of the batch's
    __device__ __forceinline__ OrthoTile(const OrthoArgs& g, bool symmetric, int r) {
        lane = lane_id();
        wave = wave_id();
        z = r / g.tiles;
        const int t = r - z * g.tiles;
        if (symmetric) {
            lower_tile(t, g.ms / G::BM, tm, tn);
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

__device__ __forceinline__ NtOperands ortho_operands(const _Float16* a, int rows_a, int lda, const _Float16* b,
                                                     int rows_b, int ldb, int k) {
    return NtOperands{reinterpret_cast<const char*>(a), reinterpret_cast<const char*>(b), nullptr, nullptr,
                      rows_a, rows_b, 2 * k, 2 * (int64_t)lda, 2 * (int64_t)ldb, 0, 0};
}

// Write the wave's block of a symmetric matrix (leading dimension ld), and its
// mirror image where the tile lies below the diagonal.  value(i, r, row, out):
// the FN values of register r in fragments (i, ..), row by row; request(q) is
// called before registers 4 q .. are stored.
template <class G, class R, class F>
__device__ __forceinline__ void store_symmetric(_Float16* S, int ld, const OrthoTile<G>& t, R request, F value) {
    const int mb = t.m0 + t.wm0, nb = t.n0 + t.wn0, n = nb + G::col_of(0, t.lane);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        request(q);
        Halves<4 * G::FM> col[G::FN];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < G::FM; ++i) {
                const int m = mb + G::row_of(i, 4 * q + e, t.lane);
                Halves<G::FN> row;
                value(i, 4 * q + e, m, row);
#pragma unroll
                for (int j = 0; j < G::FN; ++j) col[j].v[G::FM * e + i] = row.v[j];
                __builtin_memcpy(S + (int64_t)m * ld + n, &row, sizeof row);
            }
        if (t.tm != t.tn) {
#pragma unroll
            for (int j = 0; j < G::FN; ++j)
                __builtin_memcpy(S + (int64_t)(n + j) * ld + mb + quad_row<G::FM>(q, t.lane), &col[j], sizeof col[j]);
        }
    }
}

// A' (diagonal zero) and d from the sums of a tile of X X^T.
template <class G>
__device__ __forceinline__ void store_gram(const OrthoArgs& g, const OrthoTile<G>& t, const typename G::Acc (&acc)[G::FM][G::FN]) {
    float* d = g.d + (int64_t)t.z * g.ms;
    const int mb = t.m0 + t.wm0, n = t.n0 + t.wn0 + G::col_of(0, t.lane);
    Dither<ROUND_A> dither[G::FN];
    auto request = [&](int q) {
#pragma unroll
        for (int j = 0; j < G::FN; ++j) dither[j] = Dither<ROUND_A>::down(mb + quad_row<G::FM>(q, t.lane), n + j);
    };
    store_symmetric<G>(g.a + (int64_t)t.z * g.ms * g.ms, g.ms, t, request, [&](int i, int r, int m, Halves<G::FN>& out) {
#pragma unroll
        for (int j = 0; j < G::FN; ++j) {
            const float v = acc[i][j][r] * (1.0f / (ONE * ONE));
            const bool diagonal = m == n + j;
            if (diagonal) d[m] = v;
            out.v[j] = dither[j].round(diagonal ? 0.0f : v * ONE);
        }
    });
}

// A = X X^T.
template <class G>
__global__ __launch_bounds__(G::NT) void ortho_gram_kernel(OrthoArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[G::LDS_BYTES];
    const OrthoTile<G> t(g, true);
    const _Float16* X = g.hi + (int64_t)t.z * g.mp * g.np;
    typename G::Acc acc[G::FM][G::FN];
    G::product(ortho_operands(X, g.mp, g.np, X, g.mp, g.np, g.np), t.m0, t.n0, (TG_LDS char*)smem_raw, acc, t.wm0, t.wn0,
               t.lane, t.wave);
    store_gram<G>(g, t, acc);
}

// X X^T of a matrix of one tile (up to 64 rows), with hi and lo: hi hi^T + (hi
// lo^T + lo hi^T), what is left out is below 2^-20 of it.  The copies bring hi as rows
// of A and lo as rows of B, no more bytes than hi twice; both are read for the
// wave's rows and for its columns.  The sums are kept apart until the end, which
// leaves X X^T symmetric bit for bit.  Fragments are read a slice ahead,
// as in the tiled product.
template <class G>
__device__ __forceinline__ void gram_of_one_tile(const NtOperands& o, TG_LDS char* smem, typename G::Acc& acc, int wm0,
                                                 int wn0, int lane, int wave) {
    typename G::Offsets off;
    G::offsets(off, o, 0, 0, wave, lane);
    const int slices = o.k / G::ROW;
    auto slot = [&](int t) { return smem + (t % G::SLOTS) * G::SLOT; };
    auto copy = [&](int t) { G::copy_slice(slot(t), off, G::source(o, 0, 0, t, wave), wave); };
    typename G::Acc high, low;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = high[r] = low[r] = 0.0f;
    typename G::Frag f[G::KSUB][4];
    auto read = [&](int s, int t) {
        const TG_LDS char* hi = slot(t);
        const TG_LDS char* lo = hi + G::A_BYTES;
        f[s][0].v[0] = G::read_chunk(hi, wm0, s, 0, lane);
        f[s][1].v[0] = G::read_chunk(hi, wn0, s, 0, lane);
        f[s][2].v[0] = G::read_chunk(lo, wm0, s, 0, lane);
        f[s][3].v[0] = G::read_chunk(lo, wn0, s, 0, lane);
    };
#pragma unroll
    for (int t = 0; t < G::SLOTS - 1; ++t)
        if (t < slices) copy(t);
    G::wait_slice(min(G::SLOTS - 2, slices - 1));
    if (G::SLOTS - 1 < slices) copy(G::SLOTS - 1);
#pragma unroll
    for (int s = 0; s < G::KSUB; ++s) read(s, 0);
    auto slice = [&](int t, auto next) {
#pragma unroll
        for (int s = 0; s < G::KSUB; ++s) {
            acc = NtF16::mma<0, 0>(f[s][0], f[s][1], acc, 0, 0);
            high = NtF16::mma<0, 0>(f[s][0], f[s][3], high, 0, 0);
            low = NtF16::mma<0, 0>(f[s][2], f[s][1], low, 0, 0);
            if constexpr (decltype(next)::value) {
                if (s == 0) {
                    // slice t + 1 has landed, and every wave has read slice t
                    G::wait_slice(min(G::SLOTS - 2, slices - 2 - t));
                    if (t + G::SLOTS < slices) copy(t + G::SLOTS);
                }
                read(s, t + 1);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    for (int t = 0; t + 1 < slices; ++t) slice(t, std::true_type{});
    slice(slices - 1, std::false_type{});
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] += high[r] + low[r];
}

// B' and e of a matrix of one tile from the sums of X X^T: A' goes to LDS as the
// one slice that A' A' walks, d beside it.
template <class G>
__device__ __forceinline__ void poly_of_one_tile(const OrthoArgs& g, const OrthoTile<G>& t, typename G::Acc& acc,
                                                 TG_LDS char* slot, float* d) {
    static_assert(G::FM == 1 && G::FN == 1 && G::BM == 64 && G::BN == 64, "64 half precision columns are one slice");
    const int n = t.wn0 + (t.lane & 31);
    __syncthreads();  // the product's slices are read
    _Float16 a[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int m = t.wm0 + quad_row<1>(q, t.lane);
        auto dither = Dither<ROUND_A>::down(m, n);
        Halves<4> four;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float v = acc[4 * q + k] * (1.0f / (ONE * ONE));
            if (m + k == n) d[n] = v;
            a[4 * q + k] = four.v[k] = dither.round(m + k == n ? 0.0f : v * ONE);
        }
        // A' is symmetric: rows m .. m + 3 of column n are columns of row n
        __builtin_memcpy(slot + n * G::ROW + G::chunk_of(n, m / 8) * 16 + m % 8 * 2, &four, sizeof four);
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
#pragma unroll
    for (int s = 0; s < G::KSUB; ++s) {
        typename G::Frag x, y;
        x.v[0] = G::read_chunk(slot, t.wm0, s, 0, t.lane);
        y.v[0] = G::read_chunk(slot, t.wn0, s, 0, t.lane);
        acc = NtF16::mma<0, 0>(x, y, acc, 0, 0);
    }
    _Float16* B = g.b + (int64_t)t.z * g.ms * g.ms;
    const float dn = d[n];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int m0 = t.wm0 + quad_row<1>(q, t.lane);
        auto dither = Dither<ROUND_B>::down(m0, n);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int m = m0 + k, r = 4 * q + k;
            const float di = d[m], sq = acc[r] * (1.0f / (ONE * ONE)), av = (float)a[r] * (1.0f / ONE);
            if (m == n) g.e[(int64_t)t.z * g.ms + m] = g.cb * di + g.cc * (di * di + sq);
            B[(int64_t)m * g.ms + n] = dither.round(m == n ? 0.0f : (g.cb * av + g.cc * ((di + dn) * av + sq)) * ONE);
        }
    }
}

// The same with each tile's long axis split over g.parts workgroups, for few
// tiles: what bounds a workgroup there is the rate at which one compute unit's
// copies arrive (kernel times, one workgroup a tile and split: 64 x 4096 12.4, 8.0
// us, 64 x 16384 40, 11.2, 128 x 4096 13.1, 8.4, 512 x 4096 13.8, 10.2).
// Each leaves its sums in the workspace and counts itself; the one that counts
// last adds all of them, in their order, so the result does not depend on which
// that is.  No workgroup waits for another.  Sums and counters are atomics of
// device scope, which go past the caches that XCDs do not share.  Every wave
// waits for its sums' stores before the barrier ahead of the count, whose
// release and acquire order them between workgroups: one a workgroup, since
// each flushes its XCD's cache (128 x 4096 in 8 parts: 8.9 us, with a device
// fence in every wave 10.7).
//
// POLY: the matrix is this one tile (up to 64 rows), and its workgroup goes on
// to B' and e: a launch less each step (64 x 1024: a call's kernels 80 us,
// now 62).
template <class G, bool POLY>
__global__ __launch_bounds__(G::NT) void ortho_gram_split_kernel(OrthoArgs g) {
    static_assert(G::FM == 1 && G::FN == 1, "16 sums a lane");
    __shared__ __attribute__((aligned(1024))) char smem_raw[G::LDS_BYTES];
    __shared__ int last;
    const int tile = blockIdx.x / g.parts, part = blockIdx.x - tile * g.parts;
    const OrthoTile<G> t(g, true, tile);
    const int from = part * g.run, k = min(g.run, g.np - from);  // from: below np for every part
    const int64_t x = (int64_t)t.z * g.mp * g.np + from;
    typename G::Acc acc[1][1];
    if constexpr (POLY)
        gram_of_one_tile<G>(ortho_operands(g.hi + x, g.mp, g.np, g.lo + x, g.mp, g.np, k), (TG_LDS char*)smem_raw, acc[0][0],
                            t.wm0, t.wn0, t.lane, t.wave);
    else
        G::product(ortho_operands(g.hi + x, g.mp, g.np, g.hi + x, g.mp, g.np, k), t.m0, t.n0, (TG_LDS char*)smem_raw, acc,
                   t.wm0, t.wn0, t.lane, t.wave);

    if (g.parts > 1) {
        constexpr int TILE = G::BM * G::BN;
        float* sums = g.part + (int64_t)tile * g.parts * TILE + 1024 * t.wave + t.lane;
#pragma unroll
        for (int r = 0; r < 16; ++r)
            __hip_atomic_store(sums + (int64_t)part * TILE + 64 * r, acc[0][0][r], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0)
            last = __hip_atomic_fetch_add(g.arrived + tile, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == g.parts - 1;
        __syncthreads();
        if (!last) return;
        if (threadIdx.x == 0) g.arrived[tile] = 0;  // for the next step's launch
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[0][0][r] = 0.0f;
        // four parts' sums in flight at a time
        for (int p = 0; p < g.parts; p += 4) {
            float v[4][16];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    v[u][r] = __hip_atomic_load(sums + (int64_t)min(p + u, g.parts - 1) * TILE + 64 * r, __ATOMIC_RELAXED,
                                                __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[0][0][r] += p + u < g.parts ? v[u][r] : 0.0f;
        }
    }
    if constexpr (POLY) {
        __shared__ float d[G::BM];
        poly_of_one_tile<G>(g, t, acc[0][0], (TG_LDS char*)smem_raw, d);
    } else {
        store_gram<G>(g, t, acc);
    }
}

// B = b A + c A^2: B' (diagonal zero) and e.
template <class G>
__global__ __launch_bounds__(G::NT) void ortho_poly_kernel(OrthoArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[G::LDS_BYTES];
    const OrthoTile<G> t(g, true);
    const int64_t s = (int64_t)t.z * g.ms * g.ms;
    const _Float16* A = g.a + s;
    const float* d = g.d + (int64_t)t.z * g.ms;
    float* e = g.e + (int64_t)t.z * g.ms;
    // A' and d of one register quad.  Large tiles request them a quad ahead of
    // their use: the compiler may not move a load over a store, and a load's
    // latency for each row would add up (4096 x 4096
    // on 256 x 256 tiles: 110 us against 99).
    // Small ones have the registers to request all before the product.
    const int mb = t.m0 + t.wm0, n = t.n0 + t.wn0 + G::col_of(0, t.lane);
    struct Quad {
        Halves<G::FN> a[G::FM][4];
        QuadDiagonal<G::FM> d;
    };
    constexpr int HELD = G::EARLY ? 4 : 2;
    Quad ahead[HELD];
    auto load = [&](Quad& x, int q) {
        x.d.load(d, mb + quad_row<G::FM>(q, t.lane));
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int i = 0; i < G::FM; ++i)
                __builtin_memcpy(&x.a[i][p], A + (int64_t)(mb + G::row_of(i, 4 * q + p, t.lane)) * g.ms + n,
                                 sizeof x.a[0][0]);
    };
    float dn[G::FN];
#pragma unroll
    for (int j = 0; j < G::FN; ++j) dn[j] = d[n + j];
    if constexpr (G::EARLY) {
#pragma unroll
        for (int q = 0; q < 4; ++q) load(ahead[q], q);
    }
    typename G::Acc acc[G::FM][G::FN];
    G::product(ortho_operands(A, g.mp, g.ms, A, g.mp, g.ms, g.mp), t.m0, t.n0, (TG_LDS char*)smem_raw, acc, t.wm0, t.wn0, t.lane,
               t.wave);
    if constexpr (!G::EARLY) load(ahead[0], 0);
    Dither<ROUND_B> dither[G::FN];
    store_symmetric<G>(
        g.b + s, g.ms, t,
        [&](int q) {
            if (!G::EARLY && q < 3) load(ahead[(q + 1) % HELD], q + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < G::FN; ++j) dither[j] = Dither<ROUND_B>::down(mb + quad_row<G::FM>(q, t.lane), n + j);
        },
        [&](int i, int r, int m, Halves<G::FN>& out) {
            const Quad& x = ahead[(r >> 2) % HELD];
            const float di = x.d.v[G::FM * (r & 3) + i];
#pragma unroll
            for (int j = 0; j < G::FN; ++j) {
                const float sq = acc[i][j][r] * (1.0f / (ONE * ONE)), av = (float)x.a[i][r & 3].v[j] * (1.0f / ONE);
                const bool diagonal = m == n + j;
                if (diagonal) e[m] = with_choice(g.cb * di + g.cc * (di * di + sq), sq > di * di);
                out.v[j] = dither[j].round(diagonal ? 0.0f : (g.cb * av + g.cc * ((di + dn[j]) * av + sq)) * ONE);
            }
        });
}

// B' lo for X of one tile of rows, added to a tile's B' hi: the tile's own block
// of lo is all of B' lo's second operand there, so it goes from the registers of
// the epilogue to the ring's second slot (the product took one slice), transposed.
// B' is still in the first.
template <class G, class Q>
__device__ __forceinline__ void add_low(typename G::Acc& acc, TG_LDS char* smem, const Q (&x)[4], const OrthoTile<G>& t) {
    static_assert(G::BM == 64 && G::BN == 64 && G::FM == 1 && G::FN == 1 && G::SLOTS > 1, "one slice of 64 rows");
    TG_LDS char* lo = smem + G::SLOT;
    const int n = t.wn0 + (t.lane & 31);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int m = t.wm0 + quad_row<1>(q, t.lane);
        Halves<4> four;
#pragma unroll
        for (int p = 0; p < 4; ++p) four.v[p] = x[q].l[0][p].v[0];
        __builtin_memcpy(lo + n * G::ROW + G::chunk_of(n, m / 8) * 16 + m % 8 * 2, &four, sizeof four);
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < G::KSUB; ++s) {
        typename G::Frag a, b;
        a.v[0] = G::read_chunk(smem, t.wm0, s, 0, t.lane);
        b.v[0] = G::read_chunk(lo, t.wn0, s, 0, t.lane);
        acc = NtF16::mma<0, 0>(a, b, acc, 0, 0);
    }
}

// X <- (a + e) X + B' X; LAST writes the result instead.  LOW: X has up to 64
// rows, and B' lo is taken too.
template <class G, bool LAST, bool LOW>
__global__ __launch_bounds__(G::NT) void ortho_update_kernel(OrthoArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[G::LDS_BYTES];
    const OrthoTile<G> t(g, false);
    const int64_t x = (int64_t)t.z * g.mp * g.np, s = (int64_t)t.z * g.ms * g.ms;
    const float* e = g.e + (int64_t)t.z * g.ms;
    const int mb = t.m0 + t.wm0, nb = t.n0 + t.wn0, n = nb + G::col_of(0, t.lane);
    // X and e of one register quad, requested as in the kernel above
    struct Quad {
        Halves<G::FN> h[G::FM][4], l[G::FM][4];
        QuadDiagonal<G::FM> e;
    };
    auto load = [&](Quad& x4, int q) {
        x4.e.load(e, mb + quad_row<G::FM>(q, t.lane));
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int i = 0; i < G::FM; ++i) {
                const int64_t at = x + (int64_t)(mb + G::row_of(i, 4 * q + p, t.lane)) * g.np + n;
                __builtin_memcpy(&x4.h[i][p], g.hi + at, sizeof x4.h[0][0]);
                __builtin_memcpy(&x4.l[i][p], g.lo + at, sizeof x4.l[0][0]);
            }
    };
    constexpr int HELD = G::EARLY ? 4 : 2;
    Quad ahead[HELD];
    if constexpr (G::EARLY) {
#pragma unroll
        for (int q = 0; q < 4; ++q) load(ahead[q], q);
    }
    typename G::Acc acc[G::FM][G::FN];
    G::product(ortho_operands(g.b + s, g.mp, g.ms, g.xt + x, g.np, g.mp, g.mp), t.m0, t.n0, (TG_LDS char*)smem_raw, acc, t.wm0,
               t.wn0, t.lane, t.wave);
    if constexpr (LOW) add_low<G>(acc[0][0], (TG_LDS char*)smem_raw, ahead, t);
    if constexpr (!G::EARLY) load(ahead[0], 0);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (!G::EARLY && q < 3) load(ahead[(q + 1) % HELD], q + 1);
        __builtin_amdgcn_sched_barrier(0);
        Quad& x4 = ahead[q % HELD];
        Dither<ROUND_X> dither[G::FN];
#pragma unroll
        for (int j = 0; j < G::FN; ++j) dither[j] = Dither<ROUND_X>::down(mb + quad_row<G::FM>(q, t.lane), n + j);
        Halves<4 * G::FM> col[G::FN];
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int i = 0; i < G::FM; ++i) {
                const int m = mb + G::row_of(i, 4 * q + p, t.lane);
                const int64_t at = x + (int64_t)m * g.np + n;
                Halves<G::FN>&h = x4.h[i][p], &l = x4.l[i][p];
                const float ei = x4.e.v[G::FM * p + i], k = g.ca + ei, kl = !LOW && high_only(ei) ? g.ca : k;
                uint16_t o[G::FN];
#pragma unroll
                for (int j = 0; j < G::FN; ++j) {
                    const float y = fmaf(k, (float)h.v[j], fmaf(kl, (float)l.v[j], acc[i][j][4 * q + p] * (1.0f / ONE)));
                    if constexpr (LAST) {
                        o[j] = __builtin_bit_cast(uint16_t, (__bf16)(y * (1.0f / ONE)));
                        col[j].v[G::FM * p + i] = __builtin_bit_cast(_Float16, o[j]);
                    } else {
                        h.v[j] = dither[j].round(y);
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
    int32_t rows, cols;  // of G
    double* part;        // room for PARTS sums of squares for each matrix
    int32_t parts;       // of which are used
    _Float16 *hi, *lo, *xt;
    int32_t mp, np, tall;
    int32_t lane_bits;   // the norm's: 2^lane_bits threads take one row together
    int32_t* arrived;    // counters to clear
    int32_t counters;    // at most 256
    double eps;
};

constexpr int PARTS = 256;

struct EF32 {
    typedef float T;
    __device__ static __forceinline__ float up(float x) { return x; }
};
struct EBF16 {
    typedef uint16_t T;
    __device__ static __forceinline__ float up(uint16_t x) { return __builtin_bit_cast(float, (uint32_t)x << 16); }
};
struct EF16 {
    typedef uint16_t T;
    __device__ static __forceinline__ float up(uint16_t x) { return (float)__builtin_bit_cast(_Float16, x); }
};

// Elements c .. c + 7 of a row as floats, zero from `end` on.  Whole groups
// are loaded without a branch (from a block of zeros where there is none), so
// that several calls' loads are in flight together.
template <class E>
__device__ __forceinline__ void load8(float (&v)[8], const typename E::T* row, int c, int end) {
    typedef typename E::T T;
    union { T t[8]; i32x4 w[sizeof(T) / 2]; } u;
    const bool whole = c + 8 <= end;
#pragma unroll
    for (int h = 0; h < (int)sizeof(T) / 2; ++h)
        u.w[h] = load16(whole ? static_cast<const void*>(row + c + 16 / (int)sizeof(T) * h) : g_zeros);
    if (!whole && c < end) {
#pragma unroll
        for (int k = 0; k < 8; ++k) u.t[k] = load_or_zero(row + c + k, c + k < end);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = E::up(u.t[k]);
}

// Workgroup (p, z): pieces p, p + parts .. of matrix z, a piece 2048 elements
// of a row, or as many rows together as 256 threads reach where rows are
// short; its sum of squares in double (squares of any float fit), always in
// the same order.  Four pieces are requested at a time (one: 4096x4096 25 us;
// now 16).
template <class E>
__global__ __launch_bounds__(256) void ortho_norm_kernel(OrthoInArgs g) {
    __shared__ double sums[4];
    constexpr int AT_ONCE = 4;
    const int p = blockIdx.x % g.parts, z = blockIdx.x / g.parts;
    const int tid = threadIdx.x, lanes = 1 << g.lane_bits, rows = 256 >> g.lane_bits;
    const int per = (g.cols + 8 * lanes - 1) / (8 * lanes);
    const int64_t pieces = (int64_t)((g.rows + rows - 1) / rows) * per;
    double s = 0.0;
    for (int64_t i = p; i < pieces; i += AT_ONCE * g.parts) {
        float v[AT_ONCE][8];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            const int64_t k = min(i + u * g.parts, pieces - 1);
            const int r = (int)(k / per) * rows + (tid >> g.lane_bits);
            const int c = (int)(k % per) * 8 * lanes + 8 * (tid & (lanes - 1));
            // a piece, rows or columns past the last: zeros
            const int end = i + u * g.parts < pieces && r < g.rows ? g.cols : 0;
            load8<E>(v[u], static_cast<const typename E::T*>(g.G) + (int64_t)z * g.stride_g +
                               (int64_t)min(r, g.rows - 1) * g.ldg, c, end);
        }
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u)
#pragma unroll
            for (int k = 0; k < 8; ++k) s += (double)v[u][k] * (double)v[u][k];
    }
    for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) g.part[(int64_t)z * PARTS + p] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// A workgroup takes a 64 x 64 block of X (padded): X = G / (|G| + eps) times
// 2^12 as hi + lo, and its transpose.  A thread loads 8 elements of two rows
// of G, and writes 8 of each image.
template <class E>
__global__ __launch_bounds__(256) void ortho_load_kernel(OrthoInArgs g) {
    __shared__ float tile[64][65];
    __shared__ double sums[4];
    const int tid = threadIdx.x;
    const int tn = g.np / 64, per = tn * (g.mp / 64);
    const int z = blockIdx.x / per, b = blockIdx.x - z * per;
    const int m0 = b / tn * 64, n0 = b % tn * 64;
    // rows and columns of G: those of X, or the other way round
    const int r0 = g.tall ? n0 : m0, c0 = g.tall ? m0 : n0;
    float v[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = r0 + 32 * h + (tid >> 3);
        load8<E>(v[h], static_cast<const typename E::T*>(g.G) + (int64_t)z * g.stride_g + (int64_t)min(r, g.rows - 1) * g.ldg,
                 c0 + 8 * (tid & 7), r < g.rows ? g.cols : 0);
    }
    if (blockIdx.x == 0 && tid < g.counters) g.arrived[tid] = 0;
    double s = tid < g.parts ? g.part[(int64_t)z * PARTS + tid] : 0.0;
    static_assert(PARTS == 256, "a part for each thread");
    for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
    if ((tid & 63) == 0) sums[tid >> 6] = s;
    __syncthreads();
    // in double: 1 / |G| may leave float's range
    const double f = (double)ONE / (sqrt((sums[0] + sums[1]) + (sums[2] + sums[3])) + g.eps);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 8; ++k) tile[32 * h + (tid >> 3)][8 * (tid & 7) + k] = (float)(v[h][k] * f);
    __syncthreads();
    const int64_t x = (int64_t)z * g.mp * g.np;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = 32 * h + (tid >> 3), c = 8 * (tid & 7);
        Halves<8> hi, lo, xt;
        auto row = Dither<ROUND_X>::along(m0 + r, n0 + c), column = Dither<ROUND_X>::down(m0 + c, n0 + r);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float y = g.tall ? tile[c + k][r] : tile[r][c + k];
            hi.v[k] = row.round(y);
            lo.v[k] = (_Float16)(y - (float)hi.v[k]);
            xt.v[k] = column.round(g.tall ? tile[r][c + k] : tile[c + k][r]);
        }
        __builtin_memcpy(g.hi + x + (int64_t)(m0 + r) * g.np + n0 + c, &hi, 16);
        __builtin_memcpy(g.lo + x + (int64_t)(m0 + r) * g.np + n0 + c, &lo, 16);
        __builtin_memcpy(g.xt + x + (int64_t)(n0 + r) * g.mp + m0 + c, &xt, 16);
    }
}

// ---- host ------------------------------------------------------------------------

typedef void (*OrthoFn)(OrthoArgs);
typedef void (*OrthoInFn)(OrthoInArgs);

// Kernels of the symmetric products (gram, poly) and of the update (middle
// steps, last), by tile, with a model of their time in microseconds fitted to
// runs of all of them at K = 64 .. 4096 and 1 .. 2080 tiles: start + rounds
// (fixed + per_k K), K the product's inner size.  Tiles of which two share a
// compute unit (`shared`) overlap their rounds; the others run whole rounds of
// 256.  Medians of kernel times, when all roundings were to nearest (the choice
// at 4096^2 takes 80 and 140 us now):
//   gram, us          64     128    192    256
//   K =  256 (256^2)    4.3    5.9   10.1   10.6
//   K = 1024 (1024^2)   7.6   11.2   18.5   26.4
//   K = 2048 (2048^2)  22.3   18.2   28.6   43.6
//   K = 4096 (4096^2) 117     97     76     93
//   update, us        64     128    256
//   K = 1024 (1024^2)   9.8   14.4   32.7
//   K = 1024 (x 4096)  22.9   19.6   35.4
//   K = 2048 (2048^2)  34.8   26.3   52.7
//   K = 4096 (4096^2) 207    155    133
struct OrthoKernels {
    int tile, threads;
    OrthoFn first, second;
    bool shared;
    double start, fixed, per_k;
};

template <class G>
static OrthoKernels symmetric_kernels(bool shared, double start, double fixed, double per_k) {
    return OrthoKernels{G::BM, G::NT, ortho_gram_kernel<G>, ortho_poly_kernel<G>, shared, start, fixed, per_k};
}
template <class G>
static OrthoKernels update_kernels(bool shared, double start, double fixed, double per_k) {
    return OrthoKernels{G::BM, G::NT, ortho_update_kernel<G, false, false>, ortho_update_kernel<G, true, false>, shared,
                        start, fixed, per_k};
}

// 64: four slots, so that two workgroups fit a compute unit (eight slots and
// one: 10 % slower alone, 1.5 times as long where there are several rounds).
// 128: eight waves of 64 x 32 (four of 64 x 64: 11.2 -> 12.8 us at 1024^2).
// 192: twelve waves of 96 x 32 (four of 96 x 96: gram 80 -> 88 us, poly 84 -> 95
// at 4096^2).
typedef NtGemm<NtF16, 256, 256, 2, 4, 2, false> Ortho256;
typedef NtGemm<NtF16, 192, 192, 2, 6, 3, true> Ortho192;
typedef NtGemm<NtF16, 128, 128, 2, 4, 4, true> Ortho128;
typedef NtGemm<NtF16, 64, 64, 2, 2, 4, true> Ortho64;

static const OrthoKernels* symmetric_table(int* count) {
    static const OrthoKernels t[4] = {symmetric_kernels<Ortho256>(false, 0.0, 9.0, 0.0205),
                                      symmetric_kernels<Ortho192>(false, 0.0, 5.0, 0.0165),
                                      symmetric_kernels<Ortho128>(false, 0.0, 4.3, 0.0060),
                                      symmetric_kernels<Ortho64>(true, 0.0, 3.3, 0.0028)};
    *count = 4;
    return t;
}
static const OrthoKernels* update_table(int* count) {
    static const OrthoKernels t[3] = {update_kernels<Ortho256>(false, 0.0, 28.0, 0.0255),
                                      update_kernels<Ortho128>(false, 0.0, 10.0, 0.0075),
                                      update_kernels<Ortho64>(true, 3.5, 2.9, 0.0026)};
    *count = 3;
    return t;
}

struct OrthoPlan {
    int64_t m, n, mp, np, ms;
    const OrthoKernels *sym, *upd;
    int64_t tri;  // symmetric tiles of one matrix
    // workgroups a tile of the gram product (more than 1: the split kernel), and
    // the columns of X that each takes, the last perhaps fewer
    int parts;
    int64_t run;
    int64_t upd_tiles, load_tiles;  // workgroups of one matrix: update, load
    // the norm's: 2^lane_bits threads take one row together; workgroups a matrix
    int lane_bits, norm_parts;
    bool fits;  // every launch fits a grid
    int64_t off_hi, off_lo, off_t0, off_t1, off_a, off_b, off_d, off_e, off_part, off_sums, off_arrived, bytes;
};

static int64_t up_to(int64_t v, int64_t step) { return (v + step - 1) / step * step; }

// The cheapest kernel of a table for tiles(size) workgroups and inner size k.
template <class F>
static const OrthoKernels* cheapest(const OrthoKernels* t, int count, int64_t k, F tiles) {
    const OrthoKernels* best = t;
    double least = 0.0;
    for (int i = 0; i < count; ++i) {
        const int64_t n = tiles(t[i].tile);
        const double rounds = !t[i].shared ? (double)((n + 255) / 256) : n > 256 ? n / 256.0 : 1.0;
        const double c = t[i].start + rounds * (t[i].fixed + t[i].per_k * (double)k);
        if (i == 0 || c < least) {
            least = c;
            best = t + i;
        }
    }
    return best;
}

// Tiles, and where things stand in the workspace.  X is padded to whole
// update tiles, with zeros that every product keeps.  A and B have room for
// whole symmetric tiles; what lies past X's rows there is read by no product.
static OrthoPlan ortho_plan(int64_t batch, int64_t rows, int64_t cols) {
    OrthoPlan p{};
    p.m = rows < cols ? rows : cols;
    p.n = rows < cols ? cols : rows;
    auto tiles = [](int64_t v, int64_t tile) { return (v + tile - 1) / tile; };
    int count;
    const OrthoKernels* t = update_table(&count);
    // up to 64 rows the kernels for one tile of rows (64 x 64, the cheapest there by
    // the model too)
    p.upd = p.m <= 64 ? t + count - 1 : cheapest(t, count, p.m, [&](int64_t tile) { return batch * tiles(p.m, tile) * tiles(p.n, tile); });
    p.mp = up_to(p.m, p.upd->tile);
    p.np = up_to(p.n, p.upd->tile);
    auto tri = [&](int64_t tile) { return tiles(p.mp, tile) * (tiles(p.mp, tile) + 1) / 2; };
    t = symmetric_table(&count);
    p.sym = p.m <= 64 ? t + count - 1 : cheapest(t, count, (p.np + p.mp) / 2, [&](int64_t tile) { return batch * tri(tile); });  // gram: np, poly: mp
    p.tri = tri(p.sym->tile);
    p.ms = up_to(p.mp, p.sym->tile);
    // Split the gram product of few 64 x 64 tiles, at least 4 slices a part and
    // 256 workgroups at most.  A part's columns take 2.6 us for each 1024 of
    // them; joining takes about 1 us (1.8 here, to split only where it gains), 0.24
    // for each part to add and 0.025 for each workgroup (fitted to 4 .. 32 parts of 1 .. 36
    // tiles; us, 8, 16, 32 parts: 64 x 4096 7.6, 8.8,
    // 64 x 16384 11.2, 10.7, 12.8, 64 x 100000 36.3, 23.3, 19.0, 256 x 4096 9.1,
    // 12.3).
    p.parts = 1;
    p.run = p.np;
    if (p.sym->tile == 64) {
        const int64_t groups = batch * p.tri, slices = p.np / 64;
        const double columns = 0.0026 * (double)p.np;
        double least = columns;
        for (int64_t n = 2; n <= slices / 4 && n * groups <= 256; ++n) {
            const double t = 1.8 + columns / (double)n + (double)n * (0.24 + 0.025 * (double)groups);
            if (t >= least) continue;
            least = t;
            p.run = 64 * tiles(slices, n);
            p.parts = (int)tiles(p.np, p.run);
        }
    }
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t o = at;
        at += up_to(bytes, 256);
        return o;
    };
    const int64_t x = 2 * batch * p.mp * p.np, s = 2 * batch * p.ms * p.ms;
    p.off_hi = take(x);
    p.off_lo = take(x);
    p.off_t0 = take(x);
    p.off_t1 = take(x);
    p.off_a = take(s);
    p.off_b = take(s);
    p.off_d = take(4 * batch * p.ms);
    p.off_e = take(4 * batch * p.ms);
    p.off_part = take(8 * batch * PARTS);
    p.off_sums = take(p.parts > 1 ? 4 * batch * p.tri * p.parts * 4096 : 0);
    p.off_arrived = take(p.parts > 1 ? 4 * batch * p.tri : 0);
    p.bytes = at;
    p.upd_tiles = (p.mp / p.upd->tile) * (p.np / p.upd->tile);
    p.load_tiles = (p.mp / 64) * (p.np / 64);
    while (p.lane_bits < 8 && (INT64_C(8) << p.lane_bits) < cols) ++p.lane_bits;
    // a workgroup for each piece, up to PARTS (PARTS for every matrix: 300 of
    // 40 x 70 61 us, now 5.5)
    const int64_t pieces = tiles(rows, 256 >> p.lane_bits) * tiles(cols, 2048);
    p.norm_parts = (int)(pieces < PARTS ? pieces : PARTS);
    p.fits = grid_fits((double)(batch * p.tri), p.sym->threads) && grid_fits((double)(batch * p.upd_tiles), p.upd->threads) &&
             grid_fits((double)(batch * p.load_tiles), 256) && grid_fits((double)(batch * p.norm_parts), 256);
    return p;
}

// Products of padded sizes stay far inside 64 bits, and a tile's copies reach
// its rows by 32-bit offsets.
constexpr int64_t MOST_SIDE = 1 << 20, MOST_BATCH = 1 << 16;
static_assert(255 * 2 * (MOST_SIDE + 256) + 128 <= INT64_C(0xffffffff), "offsets of a tile's copies");
static bool ortho_sizes_ok(int64_t batch, int64_t rows, int64_t cols) {
    return batch >= 0 && rows >= 0 && cols >= 0 && rows <= MOST_SIDE && cols <= MOST_SIDE && batch <= MOST_BATCH;
}

// The largest singular value the steps before the last can reach from [0, 1],
// and the largest |b s^2 + c s^4| in any, up to the first step that passes what
// the workspace holds.  Both polynomials are largest at an end of the range or
// where their derivative is zero.
constexpr double MOST_X = 3.5, MOST_POLY = 14.0;
static void ortho_reach(int steps, const double* coef, double* x, double* poly) {
    double top = 1.0, most = 1.0, p = 0.0;
    for (int k = 0; k < steps; ++k) {
        const double a = coef[3 * k], b = coef[3 * k + 1], c = coef[3 * k + 2];
        double next = 0.0;
        auto look = [&](double t) {  // t = s^2
            if (!(t >= 0.0 && t <= top * top)) return;
            const double q = (b + c * t) * t, y = fabs((a + q) * sqrt(t));
            if (!(y <= next)) next = y;
            if (!(fabs(q) <= p)) p = fabs(q);
        };
        look(top * top);
        if (c != 0.0) look(-b / (2.0 * c));
        // a + 3 b t + 5 c t^2 = 0, by the quotients that lose no digits
        const double r = 9.0 * b * b - 20.0 * a * c;
        if (r >= 0.0) {
            const double u = -0.5 * (3.0 * b + copysign(sqrt(r), b));
            if (c != 0.0) look(u / (5.0 * c));
            if (u != 0.0) look(a / u);
        }
        top = next;
        if (k + 1 < steps && !(top <= most)) most = top;
        if (!(most <= MOST_X) || !(p <= MOST_POLY)) break;
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
    const OrthoPlan p = ortho_plan(batch, rows, cols);
    return p.fits ? p.bytes : -1;
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
    if (ldg > MOST_STRIDE || ldo > MOST_STRIDE || (batch > 1 && (stride_g > MOST_STRIDE || stride_o > MOST_STRIDE))) {
        set_error("a stride is out of range");
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
        if (!(fabs(coefficients[i]) <= 1e15)) {  // the kernels take them as float, their squares are taken here
            set_error("coefficient %d is not finite or above 1e15", i);
            return TGEMM_E_ARG;
        }
    double reach, poly;
    ortho_reach(steps, coefficients, &reach, &poly);
    if (!(reach <= MOST_X) || !(poly <= MOST_POLY)) {
        set_error("these coefficients let singular values reach %g (%g) or b s^2 + c s^4 reach %g (%g)", reach, MOST_X, poly,
                  MOST_POLY);
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
    if (!p.fits) {
        set_error("batch=%lld rows=%lld cols=%lld: too many tiles", (long long)batch, (long long)rows, (long long)cols);
        return TGEMM_E_ARG;
    }
    if (workspace_bytes < p.bytes) {
        set_error("workspace of %lld bytes, %lld needed", (long long)workspace_bytes, (long long)p.bytes);
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
    in.rows = (int32_t)rows;
    in.cols = (int32_t)cols;
    in.part = (double*)(ws + p.off_part);
    in.hi = (_Float16*)(ws + p.off_hi);
    in.lo = (_Float16*)(ws + p.off_lo);
    in.xt = (_Float16*)(ws + p.off_t0);
    in.mp = (int32_t)p.mp;
    in.np = (int32_t)p.np;
    in.tall = rows > cols;
    in.lane_bits = p.lane_bits;
    in.parts = p.norm_parts;
    in.eps = eps;
    in.arrived = (int32_t*)(ws + p.off_arrived);
    in.counters = p.parts > 1 ? (int32_t)(batch * p.tri) : 0;
    const OrthoInFn norm_fn = dtype == TGEMM_F32 ? ortho_norm_kernel<EF32>
                              : dtype == TGEMM_BF16 ? ortho_norm_kernel<EBF16> : ortho_norm_kernel<EF16>;
    const OrthoInFn load_fn = dtype == TGEMM_F32 ? ortho_load_kernel<EF32>
                              : dtype == TGEMM_BF16 ? ortho_load_kernel<EBF16> : ortho_load_kernel<EF16>;
    void* in_args[] = {&in};
    hipError_t err = hipLaunchKernel(reinterpret_cast<const void*>(norm_fn), dim3((unsigned)(in.parts * batch)), dim3(256),
                                     in_args, 0, s);
    if (err == hipSuccess)
        err = hipLaunchKernel(reinterpret_cast<const void*>(load_fn), dim3((unsigned)(batch * p.load_tiles)), dim3(256), in_args, 0,
                              s);

    OrthoArgs g{};
    g.hi = g.hi_out = in.hi;
    g.lo = g.lo_out = in.lo;
    g.a = (_Float16*)(ws + p.off_a);
    g.b = (_Float16*)(ws + p.off_b);
    g.d = (float*)(ws + p.off_d);
    g.e = (float*)(ws + p.off_e);
    g.part = (float*)(ws + p.off_sums);
    g.arrived = in.arrived;
    g.parts = p.parts;
    g.run = (int32_t)p.run;
    g.out = (uint16_t*)O;
    g.ldo = ldo;
    g.stride_o = stride_o;
    g.mp = in.mp;
    g.np = in.np;
    g.ms = (int32_t)p.ms;
    g.m = (int32_t)p.m;
    g.n = (int32_t)p.n;
    g.tall = in.tall;
    g.tiles_m = (int32_t)(p.mp / p.upd->tile);
    g.tiles_n = (int32_t)(p.np / p.upd->tile);
    auto launch = [&](OrthoFn fn, const OrthoKernels& k, int64_t tiles, int64_t parts) {
        if (err != hipSuccess) return;
        g.tiles = (int32_t)tiles;
        void* args[] = {&g};
        err = hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)(batch * tiles * parts)), dim3(k.threads),
                              args, 0, s);
    };
    // up to 64 rows: one symmetric tile, tiles of 64 rows, and products that take lo
    const bool small = p.mp == 64;
    const OrthoFn update = small ? ortho_update_kernel<Ortho64, false, true> : p.upd->first;
    const OrthoFn last = small ? ortho_update_kernel<Ortho64, true, true> : p.upd->second;
    for (int k = 0; k < steps; ++k) {
        g.ca = (float)coefficients[3 * k];
        g.cb = (float)coefficients[3 * k + 1];
        g.cc = (float)coefficients[3 * k + 2];
        g.xt = (const _Float16*)(ws + (k % 2 ? p.off_t1 : p.off_t0));
        g.xt_out = (_Float16*)(ws + (k % 2 ? p.off_t0 : p.off_t1));
        if (small) {
            launch(ortho_gram_split_kernel<Ortho64, true>, *p.sym, p.tri, p.parts);
        } else {
            launch(p.parts > 1 ? ortho_gram_split_kernel<Ortho64, false> : p.sym->first, *p.sym, p.tri, p.parts);
            launch(p.sym->second, *p.sym, p.tri, 1);
        }
        launch(k + 1 < steps ? update : last, *p.upd, p.upd_tiles, 1);
    }
    if (err != hipSuccess) {
        set_error("launch failed: %s", hipGetErrorString(err));
        return TGEMM_E_HIP;
    }
    clear_error();
    return TGEMM_OK;
}

}  // extern "C"
