// The gated feed-forward block, y = (act(x Wg^T) * (x Wu^T)) Wd^T, and its
// gradients: what stands where in the caller's buffers, and the launches.
//
// Forward: gate and up projections in one kernel that ends with h, and for the
// backward pass keeps g and u in 24 bits each (Kept24); the down projection.
// Backward: dh = dy Wd in one that ends with dg = dh act'(g) u, du = dh act(g) and,
// for w_down's gradient, h again; dx = dg Wg + du Wu as one product; the three
// weights' gradients in one launch.
#include <climits>

#include "tg_mm_host.hpp"

namespace tg {

struct FfnLayout {
    int64_t g, u, low;       // forward: g and u, kept; -1: not there
    int64_t h;               // kept, or in scratch
    bool h_kept;             // the down projection's gradient is wanted alone
    int64_t ld;              // row stride of all of them: whole 128-byte lines
    int64_t split;           // forward's scratch: sums of the down projection's shared tiles
    int64_t x, wg, wu, wd;   // likewise: operands on lines, -1: read where they are
    int64_t dg, du, h2;      // backward's scratch; h2: h made again
    int64_t dx_split, dw_split;
    int64_t split_bytes, dx_split_bytes, dw_split_bytes;
    bool rows;               // few tokens: the kernels that read each weight once
    MmSize gate, down, dh, dx, dw;
    int64_t bytes[3];        // saved, forward's scratch, backward's scratch
};

static const int FFN_INNER = TGEMM_FFN_X | TGEMM_FFN_GATE | TGEMM_FFN_UP;

static FfnLayout ffn_layout(int64_t M, int64_t K, int64_t F, int64_t N, int keep) {
    FfnLayout l{};
    auto take = [&](int which, int64_t n) {
        const int64_t at = l.bytes[which];
        l.bytes[which] += (n + 255) / 256 * 256;
        return at;
    };
    l.rows = M <= MM_ROWS;
    l.ld = (F + 63) / 64 * 64;
    const int64_t inner = 2 * M * l.ld;
    const MmShape y{M, N}, x{M, K}, dw[3] = {{F, K}, {F, K}, {N, F}};
    // as far as a launch of a wave a row reaches
    const bool pack_k = mm_packs(K, M) && M + 2 * F <= MM_WAVE_ROWS, pack_f = mm_packs(F, M);
    l.gate = mm_size(FORM_GATE, M, F, mm_slices(K), false, pack_k ? 0 : K);
    l.down = mm_size(FORM_NT, M, N, mm_slices(F), true, pack_f ? 0 : F);
    l.x = l.wg = l.wu = l.wd = -1;
    if (pack_k) {
        l.x = take(1, 2 * M * mm_lines(K));
        l.wg = take(1, 2 * F * mm_lines(K));
        l.wu = take(1, 2 * F * mm_lines(K));
    }
    if (pack_f) l.wd = take(1, 2 * N * l.ld);
    l.g = l.u = l.low = l.dg = l.du = l.h2 = -1;
    l.h_kept = keep == TGEMM_FFN_DOWN;
    if (keep & FFN_INNER) {
        l.g = take(0, inner);
        l.u = take(0, inner);
        l.low = take(0, inner);
        if (keep & TGEMM_FFN_DOWN) l.h2 = take(2, inner);
    }
    l.h = take(l.h_kept ? 0 : 1, inner);
    if (!l.rows) l.split_bytes = mm_split_bytes(FORM_NT, l.down, &y, 1, mm_slices(F), false);
    l.split = take(1, l.split_bytes);
    if (keep & FFN_INNER) {
        l.dh = mm_size(FORM_DH, M, F, mm_slices(N), false, N);
        if (keep & (TGEMM_FFN_X | TGEMM_FFN_GATE)) l.dg = take(2, inner);
        if (keep & (TGEMM_FFN_X | TGEMM_FFN_UP)) l.du = take(2, inner);
    }
    if (keep & TGEMM_FFN_X) {
        l.dx = mm_size(FORM_NN, M, K, 2 * mm_slices(F), true, 0);
        l.dx_split_bytes = mm_split_bytes(FORM_NN, l.dx, &x, 1, 2 * mm_slices(F), false);
        l.dx_split = take(2, l.dx_split_bytes);
    }
    MmShape wanted[3];
    int n = 0;
    for (int i = 0; i < 3; ++i)
        if (keep & (TGEMM_FFN_GATE << i)) wanted[n++] = dw[i];
    if (n > 0) {
        l.dw = mm_size(FORM_TN, wanted, n, mm_slices(M), true, K % 8 ? K : N);
        l.dw_split_bytes = mm_split_bytes(FORM_TN, l.dw, wanted, n, mm_slices(M), false);
        l.dw_split = take(2, l.dw_split_bytes);
    }
    return l;
}

static float* room(char* base, int64_t at, int64_t bytes) { return bytes > 0 ? reinterpret_cast<float*>(base + at) : nullptr; }

static bool ffn_sizes_ok(int64_t M, int64_t K, int64_t F, int64_t N, int32_t keep) {
    if (M < 0 || K < 0 || F < 0 || N < 0 || M > MM_MOST_ROWS || K > MM_MOST || F > MM_MOST || N > MM_MOST || (keep & ~15)) {
        set_error("M=%lld K=%lld F=%lld N=%lld keep=%d out of range", (long long)M, (long long)K, (long long)F, (long long)N, keep);
        return false;
    }
    return true;
}

// Whether grids hold the launches of the backward pass (forward: those of both).
static int ffn_check_grids(const FfnLayout& l, int64_t M, int64_t K, int64_t F, int64_t N, int keep, bool forward) {
    int rc = TGEMM_OK;
    if (M == 0) return rc;
    if (forward && !l.rows) {
        rc = mm_check_tiles("gate and up projections", FORM_GATE, l.gate, M, F);
        if (rc == TGEMM_OK) rc = mm_check_tiles("down projection", FORM_NT, l.down, M, N);
    }
    if (rc == TGEMM_OK && (keep & FFN_INNER)) rc = mm_check_tiles("gradient of the inner values", FORM_DH, l.dh, M, F);
    if (rc == TGEMM_OK && (keep & TGEMM_FFN_X)) rc = mm_check_tiles("gradient of x", FORM_NN, l.dx, M, K);
    const MmShape dw[3] = {{F, K}, {F, K}, {N, F}};
    if (rc == TGEMM_OK && (keep & (TGEMM_FFN_GATE | TGEMM_FFN_UP | TGEMM_FFN_DOWN)))
        rc = mm_check_tiles("gradients of the weights", FORM_TN, l.dw, dw, 3);
    return rc;
}

static int ffn_common(int32_t dtype, int32_t act) {
    if (dtype != TGEMM_BF16 && dtype != TGEMM_F16) {
        set_error("dtype %d is not bfloat16 or float16", dtype);
        return TGEMM_E_ARG;
    }
    if (act < TGEMM_SILU || act > TGEMM_RELU) {
        set_error("unknown activation %d", act);
        return TGEMM_E_ARG;
    }
    return TGEMM_OK;
}

// own_a, own_b: an operand of ours, whose rows are whole 128-byte lines.
static MmOperands operands(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t M, int64_t N, int64_t K,
                           bool own_a = false, bool own_b = false) {
    return MmOperands{static_cast<const char*>(a), static_cast<const char*>(b), nullptr, 2 * lda, 2 * ldb, 0,
                      (int32_t)M, (int32_t)N, (int32_t)K, own_a, own_b};
}

template <bool PAIR>
static const void* rows_kernel(int dtype) {
    return dtype == TGEMM_BF16 ? reinterpret_cast<const void*>(mm_rows_kernel<MmBf16, PAIR>)
                               : reinterpret_cast<const void*>(mm_rows_kernel<MmF16, PAIR>);
}

}  // namespace tg

extern "C" {

int tgemm_ffn_bytes(int64_t M, int64_t K, int64_t F, int64_t N, int32_t keep, int64_t* bytes) {
    using namespace tg;
    if (!bytes) {
        set_error("NULL bytes");
        return TGEMM_E_NULL;
    }
    if (!ffn_sizes_ok(M, K, F, N, keep)) return TGEMM_E_ARG;
    const FfnLayout l = ffn_layout(M, K, F, N, keep);
    for (int i = 0; i < 3; ++i) bytes[i] = l.bytes[i];
    clear_error();
    return TGEMM_OK;
}

int tgemm_ffn_forward(int64_t M, int64_t K, int64_t F, int64_t N, int32_t dtype, int32_t act, const void* x, int64_t ldx,
                      const void* wg, int64_t ldg, const void* wu, int64_t ldu, const void* wd, int64_t ldd, void* y,
                      int64_t ldy, int32_t keep, void* saved, void* scratch, void* stream) {
    using namespace tg;
    if (!ffn_sizes_ok(M, K, F, N, keep)) return TGEMM_E_ARG;
    const FfnLayout l = ffn_layout(M, K, F, N, keep);
    int rc = ffn_common(dtype, act);
    if (rc == TGEMM_OK) rc = mm_check("x", x, M, K, ldx);
    if (rc == TGEMM_OK) rc = mm_check("w_gate", wg, F, K, ldg);
    if (rc == TGEMM_OK) rc = mm_check("w_up", wu, F, K, ldu);
    if (rc == TGEMM_OK) rc = mm_check("w_down", wd, N, F, ldd);
    if (rc == TGEMM_OK) rc = mm_check("y", y, M, N, ldy);
    if (rc == TGEMM_OK) rc = mm_check_buffer("saved", saved, l.bytes[0]);
    if (rc == TGEMM_OK) rc = mm_check_buffer("scratch", scratch, l.bytes[1]);
    if (rc == TGEMM_OK) rc = ffn_check_grids(l, M, K, F, N, keep, true);
    if (rc == TGEMM_OK && M > 0) rc = current_device_ok();
    if (rc != TGEMM_OK) return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    char* v = static_cast<char*>(saved);
    char* s = static_cast<char*>(scratch);
    char* h = (l.h_kept ? v : s) + l.h;
    if (M > 0) {
        MmPack list[3];
        int n = 0;
        auto pack = [&](const void*& p, int64_t& ld, int64_t rows, int64_t cols, int64_t at) {
            if (at < 0 || mm_aligned(p, ld)) return;
            list[n++] = MmPack{p, ld, rows, cols, s + at};
            p = s + at;
            ld = mm_lines(cols);
        };
        pack(x, ldx, M, K, l.x);
        pack(wg, ldg, F, K, l.wg);
        pack(wu, ldu, F, K, l.wu);
        rc = mm_pack(list, n, st);
        n = 0;
        pack(wd, ldd, N, F, l.wd);
        if (rc == TGEMM_OK) rc = mm_pack(list, n, st);
        if (rc != TGEMM_OK) return rc;
    }
    if (M > 0 && F > 0) {
        MmOperands o = operands(x, ldx, wg, ldg, M, F, K);
        o.b2 = static_cast<const char*>(wu);
        o.ldb2 = 2 * ldu;
        if (l.rows && !(keep & FFN_INNER)) {
            MmRowsArgs a{o, h, l.ld, act};
            rc = mm_launch(rows_kernel<true>(dtype), (F + 15) / 16, 512, &a, "gate and up projections", st);
        } else {
            const MmKernel& k = mm_kernels(dtype, FORM_GATE)[l.gate];
            auto kept = [&](int64_t at) { return at < 0 ? nullptr : v + at; };
            MmGateArgs a{o, mm_grid(k, M, F), h, kept(l.g), kept(l.u), kept(l.low), l.ld, act};
            rc = mm_launch(k.fn, (int64_t)a.grid.tiles_m * a.grid.tiles_n, k.threads, &a, "gate and up projections", st);
        }
    }
    if (rc == TGEMM_OK && M > 0 && N > 0) {
        if (l.rows) {
            MmRowsArgs a{operands(h, l.ld, wd, ldd, M, N, F), y, ldy, 0};
            rc = mm_launch(rows_kernel<false>(dtype), (N + 15) / 16, 512, &a, "down projection", st);
        } else {
            MmStoreArgs a{};
            a.jobs = 1;
            a.split = room(s, l.split, l.split_bytes);
            a.job[0] = MmJob{{operands(h, l.ld, wd, ldd, M, N, F), {}}, 1, {}, y, ldy, nullptr, 0};
            rc = mm_store(dtype, FORM_NT, l.down, a, st);
        }
    }
    if (rc == TGEMM_OK) clear_error();
    return rc;
}

int tgemm_ffn_backward(int64_t M, int64_t K, int64_t F, int64_t N, int32_t dtype, int32_t act, const void* x, int64_t ldx,
                       const void* wg, int64_t ldg, const void* wu, int64_t ldu, const void* wd, int64_t ldd, const void* dy,
                       int64_t lddy, int32_t keep, const void* saved, void* dx, int64_t lddx, void* dwg, int64_t lddwg,
                       void* dwu, int64_t lddwu, void* dwd, int64_t lddwd, void* scratch, void* stream) {
    using namespace tg;
    if (!ffn_sizes_ok(M, K, F, N, keep)) return TGEMM_E_ARG;
    const FfnLayout l = ffn_layout(M, K, F, N, keep);
    int rc = ffn_common(dtype, act);
    if (rc == TGEMM_OK) rc = mm_check("x", x, M, K, ldx);
    if (rc == TGEMM_OK) rc = mm_check("w_gate", wg, F, K, ldg);
    if (rc == TGEMM_OK) rc = mm_check("w_up", wu, F, K, ldu);
    if (rc == TGEMM_OK) rc = mm_check("w_down", wd, N, F, ldd);
    if (rc == TGEMM_OK) rc = mm_check("dy", dy, M, N, lddy);
    if (rc == TGEMM_OK && (keep & TGEMM_FFN_X)) rc = mm_check("dx", dx, M, K, lddx);
    if (rc == TGEMM_OK && (keep & TGEMM_FFN_GATE)) rc = mm_check("dw_gate", dwg, F, K, lddwg);
    if (rc == TGEMM_OK && (keep & TGEMM_FFN_UP)) rc = mm_check("dw_up", dwu, F, K, lddwu);
    if (rc == TGEMM_OK && (keep & TGEMM_FFN_DOWN)) rc = mm_check("dw_down", dwd, N, F, lddwd);
    if (rc == TGEMM_OK) rc = mm_check_buffer("saved", saved, l.bytes[0]);
    if (rc == TGEMM_OK) rc = mm_check_buffer("scratch", scratch, l.bytes[2]);
    if (rc == TGEMM_OK) rc = ffn_check_grids(l, M, K, F, N, keep, false);
    if (rc == TGEMM_OK && keep && (M > 0 || F > 0)) rc = current_device_ok();
    if (rc != TGEMM_OK) return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const char* v = static_cast<const char*>(saved);
    char* s = static_cast<char*>(scratch);
    auto in_scratch = [&](int64_t at) { return at < 0 ? nullptr : s + at; };
    char *dg = in_scratch(l.dg), *du = in_scratch(l.du);
    const char* h = l.h_kept ? v + l.h : in_scratch(l.h2);
    if ((keep & FFN_INNER) && M > 0 && F > 0) {
        const MmKernel& k = mm_kernels(dtype, FORM_DH)[l.dh];
        MmDhArgs a{operands(dy, lddy, wd, ldd, M, F, N), mm_grid(k, M, F), v + l.g, v + l.u, v + l.low, dg, du,
                   in_scratch(l.h2), l.ld, act};
        rc = mm_launch(k.fn, (int64_t)a.grid.tiles_m * a.grid.tiles_n, k.threads, &a, "gradient of the inner values", st);
    }
    if (rc == TGEMM_OK && (keep & TGEMM_FFN_X)) {
        MmStoreArgs a{};
        a.jobs = 1;
        a.split = room(s, l.dx_split, l.dx_split_bytes);
        a.job[0] = MmJob{{operands(dg, l.ld, wg, ldg, M, K, F), operands(du, l.ld, wu, ldu, M, K, F)}, 2, {}, dx, lddx, nullptr, 0};
        rc = mm_store(dtype, FORM_NN, l.dx, a, st);
    }
    if (rc == TGEMM_OK && (keep & (TGEMM_FFN_GATE | TGEMM_FFN_UP | TGEMM_FFN_DOWN))) {
        MmStoreArgs a{};
        a.split = room(s, l.dw_split, l.dw_split_bytes);
        if (keep & TGEMM_FFN_GATE) a.job[a.jobs++] = MmJob{{operands(dg, l.ld, x, ldx, F, K, M, true), {}}, 1, {}, dwg, lddwg, nullptr, 0};
        if (keep & TGEMM_FFN_UP) a.job[a.jobs++] = MmJob{{operands(du, l.ld, x, ldx, F, K, M, true), {}}, 1, {}, dwu, lddwu, nullptr, 0};
        if (keep & TGEMM_FFN_DOWN) a.job[a.jobs++] = MmJob{{operands(dy, lddy, h, l.ld, N, F, M, false, true), {}}, 1, {}, dwd, lddwd, nullptr, 0};
        rc = mm_store(dtype, FORM_TN, l.dw, a, st);
    }
    if (rc == TGEMM_OK) clear_error();
    return rc;
}

}  // extern "C"
