// Host side of the block-scaled 8-bit product: argument checks, choice of
// kernel, launch.
#include <hip/hip_runtime.h>

#include <climits>

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

static Fp8Pick pick(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, const Fp8Kernel* t) {
    auto grid = [&](int e) { return ((M + t[e].bm - 1) / t[e].bm) * ((N + t[e].bn - 1) / t[e].bn); };
    Fp8Pick p = PICK_64;
    if (M <= 16) p = PICK_ROWS16;
    else if (M <= 32) p = PICK_ROWS32;
    else if (M <= 64) p = PICK_ROWS64;
    else if (grid(PICK_256) >= 192) p = PICK_256;
    else if (grid(PICK_128) >= 128) p = PICK_128;
    if (p <= PICK_64 && !offsets_fit(t[p], lda, ldb)) p = PICK_ROWS64;
    (void)K;
    return p;
}

static bool sizes_ok(int64_t M, int64_t N, int64_t K) {
    const int64_t most = INT_MAX - 256;
    return M >= 0 && N >= 0 && K >= 0 && M <= most && N <= most && K <= most;
}

}  // namespace tg

extern "C" {

const char* tgemm_fp8_gemm_kernel(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb) {
    using namespace tg;
    if (!sizes_ok(M, N, K) || M == 0 || N == 0) return "";
    const Fp8Kernel* t = fp8_kernels_e4m3_e4m3();
    return t[pick(M, N, K, lda, ldb, t)].name;
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
    const Fp8Kernel* t = kernels_of(fmt_a, fmt_b);
    const Fp8Kernel& k = t[pick(M, N, K, lda, ldb, t)];
    const int64_t tiles_m = (M + k.bm - 1) / k.bm, tiles_n = (N + k.bn - 1) / k.bn;
    if (tiles_m * tiles_n > INT_MAX) {
        set_error("too many tiles");
        return TGEMM_E_ARG;
    }
    const int rc = current_device_ok();
    if (rc != TGEMM_OK) return rc;
    Fp8Args g{};
    g.op = NtOperands{(const char*)A, (const char*)B, (const uint8_t*)SA, (const uint8_t*)SB,
                      (int32_t)M, (int32_t)N, (int32_t)K, lda, ldb, ldsa, ldsb};
    g.C = (uint16_t*)C;
    g.ldc = ldc;
    g.tiles_m = (int32_t)tiles_m;
    g.tiles_n = (int32_t)tiles_n;
    g.stream = (uintptr_t)C % 128 == 0 && ldc % 64 == 0;
    void* args[] = {&g};
    const hipError_t err = hipLaunchKernel(reinterpret_cast<const void*>(k.fn), dim3((unsigned)(tiles_m * tiles_n)),
                                           dim3(k.threads), args, 0, static_cast<hipStream_t>(stream));
    if (err != hipSuccess) {
        set_error("launch of %s failed: %s", k.name, hipGetErrorString(err));
        return TGEMM_E_HIP;
    }
    clear_error();
    return TGEMM_OK;
}

}  // extern "C"
