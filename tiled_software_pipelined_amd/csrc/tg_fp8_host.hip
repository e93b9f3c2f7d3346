// Host side of the block-scaled 8-bit product: argument checks, choice of
// kernel, launch.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>

#include "tg_fp8.hpp"
#include "tg_host.hpp"
#include "tgemm.h"

namespace tg {

static const Fp8Kernel* kernels_of(int fa, int fb) {
    if (fa == TGEMM_E4M3) return fb == TGEMM_E4M3 ? fp8_kernels_e4m3_e4m3() : fp8_kernels_e4m3_e5m2();
    return fb == TGEMM_E4M3 ? fp8_kernels_e5m2_e4m3() : fp8_kernels_e5m2_e5m2();
}

// A lane of a tiled kernel's copies reaches up to BM - 1 rows past the tile's
// first by a 32-bit offset; longer rows run on the kernels for few rows,
// whose addresses are 64-bit.
static bool offsets_fit(const Fp8Kernel& k, int64_t lda, int64_t ldb) {
    return (k.bm - 1) * lda + 128 <= INT64_C(0xffffffff) && (k.bn - 1) * ldb + 128 <= INT64_C(0xffffffff);
}

// Model of a kernel's time in microseconds, fitted to runs of every kernel at
// 23 shapes (1 .. 8192 rows and columns, K = 512 .. 16384; graph replays, a
// different B each time).  A round is 256 workgroups, one a compute unit; a
// further round of the kernels for few rows has a least time, however short K
// (509x3712x114 on rows32: 32 us).
//   us               256    128  128 pair   64   rows16  32
//   1x1024x1024                             4.4    2.9   3.1
//   1x4096x4096                             9.5    6.0   6.2
//   1x8192x8192                            19.6   14.0  16.9
//   32x4096x4096             16.1          10.0   10.2   8.4
//   64x1024x1024              7.1   8.9     4.7    3.3   3.8
//   64x4096x4096             16.4   20.9    9.8   17.5  15.0
//   512x4096x4096    39.4    18.5   26.4   16.5
//   1024x1024x1024   16.5     7.9    8.9    5.5
//   2048x2048x2048   24.9    14.2   16.5   18.2
//   2048x4096x4096   42.3    41.9   34.5   57.6
//   4096x4096x4096   52.5    81.8   67.4  107
// Few rows and many columns are bound by one read of B, which each kernel takes
// at a rate of its own (tiles: `read`, megabytes of A and B over TB/s), and the
// kernels for few rows by the rows that they do hold as well (184 shapes of 1 ..
// 128 rows, 1024 .. 128256 columns and K = 1024 .. 8192, B cold: the choice is
// within 4 % of the best kernel at each, 0.07 % in the mean).
//   1x11008x4096             18.9   34.4   13.2   11.9
//   1x50257x4096             51.6   50.8   47.7   41.8
//   1x128256x4096           119    124     95.8   94.3
//   16x128256x4096          120    125    102    126    188
//   64x128256x4096  137     129    129    118    490    450
//   100x28672x4096   48.6    31.5   40.6   38.9         179
static double time_of(Fp8Pick p, const Fp8Kernel& k, int64_t M, int64_t N, int64_t K) {
    const double tiles_m = (double)((M + k.bm - 1) / k.bm), n = tiles_m * (double)((N + k.bn - 1) / k.bn);
    const double k1 = (double)K / 1024.0, more = n > 256.0 ? n / 256.0 : 1.0;
    const double read = ((double)M + (double)N) * (double)K * 1e-6;
    const double held = (double)M / (tiles_m * k.bm);  // share of a tile's rows that are A's
    switch (p) {
        case PICK_256: {
            // a partial round leaves clock and bandwidth to the busy units
            const double whole = floor(n / 256.0), rest = n / 256.0 - whole;
            return fmax((whole + (rest > 0.0 ? 0.72 + 0.28 * rest : 0.0)) * (9.5 + 11.0 * k1), 2.0 + read / 3.8);
        }
        case PICK_128: return fmax(2.5 + ceil(n / 256.0) * (3.5 + 4.1 * k1), 2.5 + read / 4.4);
        case PICK_128_PAIR:
            return fmax(2.0 + (n > 410.0 ? more : n > 256.0 ? 1.6 : 2.0) * (2.3 + 3.67 * k1), 2.5 + read / 4.2);
        case PICK_64: return fmax(2.9 + more * (0.95 + 2.05 * k1), 3.0 + read / 5.2);
        case PICK_ROWS16: return 2.6 + 1.0 * k1 + (more - 1.0) * fmax((0.7 + 0.3 * held) * k1, 1.2 + 0.4 * held);
        default: return 2.4 + 1.5 * k1 + (more - 1.0) * fmax((1.2 + 0.6 * held) * k1, 2.2);
    }
}

// One launch: a kernel on a part of C.  swap: A and B change places (few
// columns instead of few rows).
struct Piece {
    Fp8Pick pick;
    bool swap;
    int64_t m0, n0, M, N;
    double time;
};

static Piece best_piece(const Fp8Kernel* t, int64_t m0, int64_t n0, int64_t M, int64_t N, int64_t K, int64_t lda,
                        int64_t ldb) {
    Piece best{PICK_COUNT, false, m0, n0, M, N, 0.0};
    for (int i = 0; i < PICK_COUNT; ++i) {
        const Fp8Pick p = (Fp8Pick)i;
        if (p <= PICK_64 && !offsets_fit(t[i], lda, ldb)) continue;
        const bool swap = p >= PICK_ROWS16 && N < M;
        const int64_t few = swap ? N : M, many = swap ? M : N;
        const int64_t n = ((few + t[i].bm - 1) / t[i].bm) * ((many + t[i].bn - 1) / t[i].bn);
        if (n > INT_MAX || !grid_fits((double)n, t[i].threads)) continue;
        const double c = time_of(p, t[i], few, many, K);
        if (best.pick == PICK_COUNT || c < best.time) best = Piece{p, swap, m0, n0, M, N, c};
    }
    return best;  // PICK_COUNT: no kernel's grid holds it
}

// The launches of a product: one, or a part of whole 256 x 256 tiles and the
// last columns (or rows) on the kernels for few, where that is quicker: 17
// tile columns for 4097 take two rounds (4095x4097x4096: 86 us in one launch,
// split 59).
static int pieces_of(const Fp8Kernel* t, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, Piece (&out)[2]) {
    out[0] = best_piece(t, 0, 0, M, N, K, lda, ldb);
    int count = 1;
    if (out[0].pick == PICK_COUNT) return 0;
    const int64_t rn = N % 256, rm = M % 256;
    double least = out[0].time;
    for (int d = 0; d < 2; ++d) {
        const int64_t r = d ? rm : rn;
        if (r == 0 || r > 64 || (d ? M : N) < 256) continue;
        const Piece a = d ? best_piece(t, 0, 0, M - r, N, K, lda, ldb) : best_piece(t, 0, 0, M, N - r, K, lda, ldb);
        const Piece b = d ? best_piece(t, M - r, 0, r, N, K, lda, ldb) : best_piece(t, 0, N - r, M, r, K, lda, ldb);
        if (a.pick == PICK_COUNT || b.pick == PICK_COUNT || a.time + b.time >= least) continue;
        least = a.time + b.time;
        out[0] = a;
        out[1] = b;
        count = 2;
    }
    return count;
}

static bool sizes_ok(int64_t M, int64_t N, int64_t K) {
    const int64_t most = INT_MAX - 256;
    return M >= 0 && N >= 0 && K >= 0 && M <= most && N <= most && K <= most;
}

}  // namespace tg

extern "C" {

const char* tgemm_fp8_gemm_kernel(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int32_t piece) {
    using namespace tg;
    if (!sizes_ok(M, N, K) || M == 0 || N == 0 || lda > MOST_STRIDE || ldb > MOST_STRIDE) return "";
    const Fp8Kernel* t = fp8_kernels_e4m3_e4m3();
    Piece p[2];
    return piece >= 0 && piece < pieces_of(t, M, N, K, lda, ldb, p) ? t[p[piece].pick].name : "";
}

int tgemm_fp8_gemm(int64_t M, int64_t N, int64_t K, int32_t fmt_a, const void* A, int64_t lda, const void* SA,
                   int64_t ldsa, int32_t fmt_b, const void* B, int64_t ldb, const void* SB, int64_t ldsb, void* C,
                   int64_t ldc, void* stream) {
    using namespace tg;
    if (!sizes_ok(M, N, K)) {
        set_error("M=%lld N=%lld K=%lld out of range", (long long)M, (long long)N, (long long)K);
        return TGEMM_E_ARG;
    }
    if ((fmt_a != TGEMM_E4M3 && fmt_a != TGEMM_E5M2) || (fmt_b != TGEMM_E4M3 && fmt_b != TGEMM_E5M2)) {
        set_error("unknown format %d or %d", fmt_a, fmt_b);
        return TGEMM_E_ARG;
    }
    if (lda < K || ldb < K || ldsa < M || ldsb < N || ldc < N) {
        set_error("a leading dimension is shorter than its row");
        return TGEMM_E_ARG;
    }
    if (lda > MOST_STRIDE || ldb > MOST_STRIDE || ldsa > MOST_STRIDE || ldsb > MOST_STRIDE || ldc > MOST_STRIDE) {
        set_error("a leading dimension is out of range");
        return TGEMM_E_ARG;
    }
    if (M == 0 || N == 0) {
        clear_error();
        return TGEMM_OK;
    }
    if (!C || (K > 0 && (!A || !B || !SA || !SB))) {
        set_error("NULL matrix or scale pointer");
        return TGEMM_E_NULL;
    }
    if ((uintptr_t)C % 2) {
        set_error("C not aligned to its element size");
        return TGEMM_E_ALIGN;
    }
    if (K > 0 && (ldsa % 4 || ldsb % 4 || (uintptr_t)SA % 4 || (uintptr_t)SB % 4)) {
        set_error("scale tables need 4-byte aligned rows (ldsa=%lld, ldsb=%lld)", (long long)ldsa, (long long)ldsb);
        return TGEMM_E_ALIGN;
    }
    Piece p[2];
    const int count = pieces_of(kernels_of(fmt_a, fmt_b), M, N, K, lda, ldb, p);
    if (count == 0) {
        set_error("too many tiles");
        return TGEMM_E_ARG;
    }
    const int rc = current_device_ok();
    if (rc != TGEMM_OK) return rc;
    const bool bytes = (((uintptr_t)A | (uintptr_t)B) % 4) || lda % 4 || ldb % 4;
    for (int i = 0; i < count; ++i) {
        const NtOperands a{(const char*)A + p[i].m0 * lda, (const char*)B + p[i].n0 * ldb, (const uint8_t*)SA + p[i].m0,
                           (const uint8_t*)SB + p[i].n0, (int32_t)p[i].M, (int32_t)p[i].N, (int32_t)K, lda, ldb, ldsa, ldsb};
        const bool swap = p[i].swap;
        const Fp8Kernel& k = kernels_of(swap ? fmt_b : fmt_a, swap ? fmt_a : fmt_b)[p[i].pick];
        Fp8Args g{};
        g.op = swap ? NtOperands{a.b, a.a, a.sb, a.sa, a.N, a.M, a.k, ldb, lda, ldsb, ldsa} : a;
        g.C = (uint16_t*)C + p[i].m0 * ldc + p[i].n0;
        g.row = swap ? 1 : ldc;
        g.col = swap ? ldc : 1;
        g.tiles_m = (g.op.M + k.bm - 1) / k.bm;
        g.tiles_n = (g.op.N + k.bn - 1) / k.bn;
        g.stream = (uintptr_t)g.C % 128 == 0 && ldc % 64 == 0;
        void* args[] = {&g};
        const hipError_t err = hipLaunchKernel(reinterpret_cast<const void*>(bytes ? k.bytes : k.fn), dim3((unsigned)(g.tiles_m * g.tiles_n)),
                                               dim3(k.threads), args, 0, static_cast<hipStream_t>(stream));
        if (err != hipSuccess) {
            set_error("launch of %s failed: %s", k.name, hipGetErrorString(err));
            return TGEMM_E_HIP;
        }
    }
    clear_error();
    return TGEMM_OK;
}

}  // extern "C"
