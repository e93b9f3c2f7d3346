// A linear layer in 8 bits as chains of the library's own entry points: where
// the images stand in the caller's buffers, and the order of the calls.
#include <climits>

#include "tg_host.hpp"
#include "tgemm.h"

namespace tg {

// An operand's image in a buffer: rows x cols values, rows padded to whole
// 128-byte lines (a product whose copies straddle lines takes 13 % longer:
// 4096x4096x4099 with rows 4104 apart 61.3 us, 4224 apart 54.2), then its scales,
// rows of the table padded to 16.
struct Image {
    int64_t q, ldq, s, lds;
};

struct LinearLayout {
    Image x, w, xt, wt;  // forward: x, w in scratch; xt, wt in saved
    Image g, gt;         // backward: scratch
    int64_t bytes[3];    // saved, forward's scratch, backward's scratch
};

static Image place(int64_t* at, int64_t rows, int64_t cols) {
    auto take = [&](int64_t n) {
        const int64_t o = *at;
        *at += (n + 255) / 256 * 256;
        return o;
    };
    Image m;
    m.ldq = (cols + 127) / 128 * 128;
    m.lds = (rows + 15) / 16 * 16;
    m.q = take(rows * m.ldq);
    m.s = take((cols + 127) / 128 * m.lds);
    return m;
}

static LinearLayout linear_layout(int64_t M, int64_t N, int64_t K, int keep) {
    LinearLayout l{};
    if (keep & TGEMM_KEEP_X) l.wt = place(&l.bytes[0], K, N);
    if (keep & TGEMM_KEEP_W) l.xt = place(&l.bytes[0], K, M);
    l.x = place(&l.bytes[1], M, K);
    l.w = place(&l.bytes[1], N, K);
    l.g = place(&l.bytes[2], M, N);
    if (keep & TGEMM_KEEP_W) l.gt = place(&l.bytes[2], N, M);
    return l;
}

static bool linear_sizes_ok(int64_t M, int64_t N, int64_t K, int32_t keep) {
    const int64_t most = INT_MAX - 256;
    const double area = 281474976710656.0;  // 2^48 elements: more than any memory, sums stay inside 64 bits
    if (M < 0 || N < 0 || K < 0 || M > most || N > most || K > most || (keep & ~3) || (double)M * N > area ||
        (double)M * K > area || (double)N * K > area) {
        set_error("M=%lld N=%lld K=%lld keep=%d out of range", (long long)M, (long long)N, (long long)K, keep);
        return false;
    }
    return true;
}

// Everything that the chain's calls would refuse, before the first of them.
static int check_operand(const char* name, int32_t dtype, const void* p, int64_t rows, int64_t cols, int64_t ld) {
    if (dtype != TGEMM_F32 && dtype != TGEMM_BF16 && dtype != TGEMM_F16) {
        set_error("%s: dtype %d is not float32, bfloat16 or float16", name, dtype);
        return TGEMM_E_ARG;
    }
    if (ld < cols || ld > MOST_STRIDE) {
        set_error("%s: leading dimension shorter than its row, or out of range", name);
        return TGEMM_E_ARG;
    }
    if (rows > 0 && cols > 0 && !p) {
        set_error("%s: NULL pointer", name);
        return TGEMM_E_NULL;
    }
    if ((uintptr_t)p % (dtype == TGEMM_F32 ? 4 : 2)) {
        set_error("%s: not aligned to its element size", name);
        return TGEMM_E_ALIGN;
    }
    return TGEMM_OK;
}
static int check_buffer(const char* name, const void* p, int64_t bytes) {
    if (bytes > 0 && !p) {
        set_error("%s: NULL pointer", name);
        return TGEMM_E_NULL;
    }
    if ((uintptr_t)p % 256) {
        set_error("%s: not 256-byte aligned", name);
        return TGEMM_E_ALIGN;
    }
    return TGEMM_OK;
}

}  // namespace tg

extern "C" {

int tgemm_fp8_linear_bytes(int64_t M, int64_t N, int64_t K, int32_t keep, int64_t* bytes) {
    using namespace tg;
    if (!bytes) {
        set_error("NULL bytes");
        return TGEMM_E_NULL;
    }
    if (!linear_sizes_ok(M, N, K, keep)) return TGEMM_E_ARG;
    const LinearLayout l = linear_layout(M, N, K, keep);
    for (int i = 0; i < 3; ++i) bytes[i] = l.bytes[i];
    clear_error();
    return TGEMM_OK;
}

int tgemm_fp8_linear_forward(int64_t M, int64_t N, int64_t K, int32_t x_dtype, const void* x, int64_t ldx,
                             int32_t w_dtype, const void* w, int64_t ldw, void* y, int64_t ldy, int32_t keep,
                             void* saved, void* scratch, void* stream) {
    using namespace tg;
    if (!linear_sizes_ok(M, N, K, keep)) return TGEMM_E_ARG;
    const LinearLayout l = linear_layout(M, N, K, keep);
    int rc = check_operand("x", x_dtype, x, M, K, ldx);
    if (rc == TGEMM_OK) rc = check_operand("w", w_dtype, w, N, K, ldw);
    if (rc == TGEMM_OK) rc = check_operand("y", TGEMM_BF16, y, M, N, ldy);
    if (rc == TGEMM_OK) rc = check_buffer("saved", saved, l.bytes[0]);
    if (rc == TGEMM_OK) rc = check_buffer("scratch", scratch, l.bytes[1]);
    if (rc == TGEMM_OK && (M > 0 || N > 0)) rc = current_device_ok();
    if (rc != TGEMM_OK) return rc;
    char* v = static_cast<char*>(saved);
    char* s = static_cast<char*>(scratch);
    const bool kx = keep & TGEMM_KEEP_X, kw = keep & TGEMM_KEEP_W;
    rc = tgemm_fp8_quantize(M, K, x_dtype, x, ldx, TGEMM_E4M3, TGEMM_BLOCK_ROW, s + l.x.q, l.x.ldq, s + l.x.s,
                            l.x.lds, kw ? v + l.xt.q : nullptr, l.xt.ldq, kw ? v + l.xt.s : nullptr, l.xt.lds, stream);
    if (rc == TGEMM_OK)
        rc = tgemm_fp8_quantize(N, K, w_dtype, w, ldw, TGEMM_E4M3, TGEMM_BLOCK_SQUARE, s + l.w.q, l.w.ldq, s + l.w.s,
                                l.w.lds, kx ? v + l.wt.q : nullptr, l.wt.ldq, kx ? v + l.wt.s : nullptr, l.wt.lds, stream);
    if (rc == TGEMM_OK)
        rc = tgemm_fp8_gemm(M, N, K, TGEMM_E4M3, s + l.x.q, l.x.ldq, s + l.x.s, l.x.lds, TGEMM_E4M3, s + l.w.q, l.w.ldq,
                            s + l.w.s, l.w.lds, y, ldy, stream);
    return rc;
}

int tgemm_fp8_linear_backward(int64_t M, int64_t N, int64_t K, int32_t g_dtype, const void* g, int64_t ldg,
                              int32_t grad_fmt, int32_t keep, const void* saved, void* dx, int64_t lddx, void* dw,
                              int64_t lddw, void* scratch, void* stream) {
    using namespace tg;
    if (!linear_sizes_ok(M, N, K, keep)) return TGEMM_E_ARG;
    if (grad_fmt != TGEMM_E4M3 && grad_fmt != TGEMM_E5M2) {
        set_error("unknown format %d", grad_fmt);
        return TGEMM_E_ARG;
    }
    const LinearLayout l = linear_layout(M, N, K, keep);
    const bool kx = keep & TGEMM_KEEP_X, kw = keep & TGEMM_KEEP_W;
    int rc = check_operand("g", g_dtype, g, M, N, ldg);
    if (rc == TGEMM_OK && kx) rc = check_operand("dx", TGEMM_BF16, dx, M, K, lddx);
    if (rc == TGEMM_OK && kw) rc = check_operand("dw", TGEMM_BF16, dw, N, K, lddw);
    if (rc == TGEMM_OK) rc = check_buffer("saved", saved, l.bytes[0]);
    if (rc == TGEMM_OK) rc = check_buffer("scratch", scratch, l.bytes[2]);
    if (rc == TGEMM_OK && (M > 0 || N > 0)) rc = current_device_ok();
    if (rc != TGEMM_OK) return rc;
    if (!kx && !kw) {
        clear_error();
        return TGEMM_OK;
    }
    const char* v = static_cast<const char*>(saved);
    char* s = static_cast<char*>(scratch);
    rc = tgemm_fp8_quantize(M, N, g_dtype, g, ldg, grad_fmt, TGEMM_BLOCK_ROW, s + l.g.q, l.g.ldq, s + l.g.s,
                            l.g.lds, kw ? s + l.gt.q : nullptr, l.gt.ldq, kw ? s + l.gt.s : nullptr, l.gt.lds, stream);
    if (rc == TGEMM_OK && kx)
        rc = tgemm_fp8_gemm(M, K, N, grad_fmt, s + l.g.q, l.g.ldq, s + l.g.s, l.g.lds, TGEMM_E4M3, v + l.wt.q, l.wt.ldq,
                            v + l.wt.s, l.wt.lds, dx, lddx, stream);
    if (rc == TGEMM_OK && kw)
        rc = tgemm_fp8_gemm(N, K, M, grad_fmt, s + l.gt.q, l.gt.ldq, s + l.gt.s, l.gt.lds, TGEMM_E4M3, v + l.xt.q, l.xt.ldq,
                            v + l.xt.s, l.xt.lds, dw, lddw, stream);
    return rc;
}

}  // extern "C"
