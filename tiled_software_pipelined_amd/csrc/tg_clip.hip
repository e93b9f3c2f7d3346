// Clipping gradients by the norm of all of them: norm = root of the sum of
// squares over every element of every tensor, then each element times min(1,
// max_norm / (norm + eps)).
//
// Three launches: sums of squares of pieces, the norm and the factor from them,
// the product.  Bound by memory: every element is read twice and written once;
// where the factor is one and the tensors stay in place, read once.  The product
// goes from the end to the beginning, so that it finds in the last-level cache
// what the squares read last.  Squares are
// added in 64 bits (float32 gradients of 1e20 would overflow a float's square;
// the conversions hide behind the loads), in an order that does not depend on
// which workgroup ends first.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdlib>

#include "tg_device.hpp"
#include "tg_host.hpp"
#include "tg_mm_host.hpp"
#include "tgemm.h"

namespace tg {

constexpr int CLIP_TENSORS = 112;  // of one launch: their table is the kernel's argument (4 KB at most)
constexpr int CLIP_THREADS = 256;

struct ClipArgs {
    const void* in[CLIP_TENSORS];
    void* out[CLIP_TENSORS];
    int64_t count[CLIP_TENSORS];
    uint32_t first[CLIP_TENSORS];  // workgroup at which a tensor starts
    uint8_t dtype[CLIP_TENSORS];
    int32_t tensors;
    int32_t piece;                 // elements a workgroup takes
    double* sums;                  // one a workgroup
    const float* factor;
};
static_assert(sizeof(ClipArgs) <= 4096, "kernel arguments");

// The tensor and the piece of it that this workgroup takes.
struct ClipPlace {
    int tensor;
    int64_t begin, end;
    __device__ __forceinline__ ClipPlace(const ClipArgs& g, uint32_t group) {
        int lo = 0, hi = g.tensors - 1;  // the last tensor that starts at or before this workgroup
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (g.first[mid] <= group) lo = mid;
            else hi = mid - 1;
        }
        tensor = lo;
        begin = (int64_t)(group - g.first[lo]) * g.piece;
        end = min(begin + g.piece, g.count[lo]);
    }
};

template <class T>
struct Packed {
    static constexpr int N = 16 / sizeof(T);
    T v[N];
};

template <class T>
__device__ __forceinline__ double piece_squares(const T* p, int64_t begin, int64_t end) {
    constexpr int N = Packed<T>::N, U = 4;
    double acc[4] = {0, 0, 0, 0};
    auto add = [&](const Packed<T>& x) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const double d = (double)(float)x.v[e];
            acc[e & 3] = __builtin_fma(d, d, acc[e & 3]);
        }
    };
    int64_t i = begin + threadIdx.x * N;
    for (; i + (U - 1) * CLIP_THREADS * N + N <= end; i += U * CLIP_THREADS * N) {
        Packed<T> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) __builtin_memcpy(&x[u], p + i + u * CLIP_THREADS * N, 16);
#pragma unroll
        for (int u = 0; u < U; ++u) add(x[u]);
    }
    for (; i < end; i += CLIP_THREADS * N) {
        Packed<T> x;
        if (i + N <= end) {
            __builtin_memcpy(&x, p + i, 16);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) x.v[e] = load_or_zero(p + i + e, i + e < end);
        }
        add(x);
    }
    return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

template <int WAVES>
__device__ __forceinline__ double clip_block_sum(double v) {
    __shared__ double held[WAVES];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) held[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) s += held[w];
    return s;
}

__global__ __launch_bounds__(CLIP_THREADS) void clip_squares_kernel(ClipArgs g) {
    const ClipPlace at(g, blockIdx.x);
    double s;
    switch (g.dtype[at.tensor]) {
        case TGEMM_F32: s = piece_squares(static_cast<const float*>(g.in[at.tensor]), at.begin, at.end); break;
        case TGEMM_BF16: s = piece_squares(static_cast<const __bf16*>(g.in[at.tensor]), at.begin, at.end); break;
        default: s = piece_squares(static_cast<const _Float16*>(g.in[at.tensor]), at.begin, at.end);
    }
    s = clip_block_sum<CLIP_THREADS / 64>(s);
    if (threadIdx.x == 0) g.sums[blockIdx.x] = s;
}

__global__ __launch_bounds__(1024) void clip_norm_kernel(const double* sums, int64_t count, double max_norm, double eps,
                                                         float* norm, float* factor) {
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < count; i += 1024) v += sums[i];
    v = clip_block_sum<16>(v);
    if (threadIdx.x == 0) {
        const double n = sqrt(v), f = max_norm / (n + eps);
        *norm = (float)n;
        *factor = f >= 1.0 ? 1.0f : (float)f;  // NaN stays NaN
    }
}

// Results go past the caches, which then keep what the squares have read (67
// million values in float16, read once more for the product: 84.5 us to 68; 1.4
// billion in bfloat16: 1584 to 1538).
template <class T>
__device__ __forceinline__ void piece_times(const T* in, T* out, int64_t begin, int64_t end, float f) {
    constexpr int N = Packed<T>::N, U = 4;
    typedef int32_t Loose __attribute__((ext_vector_type(4), aligned(2)));  // at any element
    auto times = [&](Packed<T>& x) {
#pragma unroll
        for (int e = 0; e < N; ++e) x.v[e] = (T)((float)x.v[e] * f);
    };
    int64_t i = begin + threadIdx.x * N;
    for (; i + (U - 1) * CLIP_THREADS * N + N <= end; i += U * CLIP_THREADS * N) {
        Packed<T> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) __builtin_memcpy(&x[u], in + i + u * CLIP_THREADS * N, 16);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            times(x[u]);
            Loose w;
            __builtin_memcpy(&w, &x[u], 16);
            __builtin_nontemporal_store(w, reinterpret_cast<Loose*>(out + i + u * CLIP_THREADS * N));
        }
    }
    for (; i < end; i += CLIP_THREADS * N) {
        Packed<T> x;
        if (i + N <= end) {
            __builtin_memcpy(&x, in + i, 16);
            times(x);
            __builtin_memcpy(out + i, &x, 16);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) x.v[e] = load_or_zero(in + i + e, i + e < end);
            times(x);
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (i + e < end) out[i + e] = x.v[e];
        }
    }
}

__global__ __launch_bounds__(CLIP_THREADS) void clip_times_kernel(ClipArgs g) {
    // tensors are listed from the last on; each from its end on
    ClipPlace at(g, blockIdx.x);
    const int64_t pieces = (g.count[at.tensor] + g.piece - 1) / g.piece;
    at.begin = (pieces - 1) * g.piece - at.begin;
    at.end = min(at.begin + g.piece, g.count[at.tensor]);
    const float f = *g.factor;
    const void* in = g.in[at.tensor];
    void* out = g.out[at.tensor];
    if (f == 1.0f && in == out) return;
    switch (g.dtype[at.tensor]) {
        case TGEMM_F32: piece_times(static_cast<const float*>(in), static_cast<float*>(out), at.begin, at.end, f); break;
        case TGEMM_BF16: piece_times(static_cast<const __bf16*>(in), static_cast<__bf16*>(out), at.begin, at.end, f); break;
        default: piece_times(static_cast<const _Float16*>(in), static_cast<_Float16*>(out), at.begin, at.end, f);
    }
}

// Elements a workgroup takes: at least 8192 (16 or 32 KB), and so many that there
// are about 16384 workgroups.
static int64_t clip_piece(double total) {
    double p = total / 16384.0;
    p = p < 8192.0 ? 8192.0 : p;
    return ((int64_t)p + 4095) / 4096 * 4096;
}

static bool clip_total(int64_t tensors, const int64_t* counts, double* total) {
    *total = 0.0;
    for (int64_t i = 0; i < tensors; ++i) {
        if (counts[i] < 0) return false;
        *total += (double)counts[i];
    }
    return *total <= 1099511627776.0;  // 2^40
}

// Whether a tensor that is written shares elements with another one: they would be
// scaled twice, or read half scaled.  Tensors that are only read may.
static int clip_check_overlap(int64_t tensors, const void* const* in, void* const* out, const int64_t* counts, const int32_t* dtypes) {
    struct Span {
        uintptr_t begin, end;
        bool written;
    };
    Span* spans = static_cast<Span*>(std::malloc(sizeof(Span) * 2 * (size_t)tensors + 1));
    if (!spans) {
        set_error("no host memory for the table of %lld tensors", (long long)tensors);
        return TGEMM_E_ARG;
    }
    int64_t n = 0;
    for (int64_t i = 0; i < tensors; ++i) {
        if (counts[i] == 0) continue;
        const uintptr_t bytes = (uintptr_t)counts[i] * (dtypes[i] == TGEMM_F32 ? 4 : 2), a = (uintptr_t)in[i], b = (uintptr_t)out[i];
        spans[n++] = Span{b, b + bytes, true};
        if (a != b) spans[n++] = Span{a, a + bytes, false};
    }
    std::sort(spans, spans + n, [](const Span& x, const Span& y) { return x.begin < y.begin; });
    uintptr_t any = 0, written = 0;  // where what was passed ends
    bool overlap = false;
    for (int64_t i = 0; i < n && !overlap; ++i) {
        overlap = spans[i].begin < (spans[i].written ? any : written);
        any = std::max(any, spans[i].end);
        if (spans[i].written) written = std::max(written, spans[i].end);
    }
    std::free(spans);
    if (overlap) set_error("tensors overlap");
    return overlap ? TGEMM_E_ARG : TGEMM_OK;
}

}  // namespace tg

extern "C" {

int64_t tgemm_clip_workspace_bytes(int64_t tensors, const int64_t* counts) {
    using namespace tg;
    double total;
    if (tensors < 0 || tensors > INT_MAX || (tensors > 0 && !counts) || !clip_total(tensors, counts, &total)) return -1;
    const int64_t piece = clip_piece(total);
    int64_t n = 0;
    for (int64_t i = 0; i < tensors; ++i) n += (counts[i] + piece - 1) / piece;
    return 256 + 8 * n;
}

int tgemm_clip(int64_t tensors, const void* const* in, void* const* out, const int64_t* counts, const int32_t* dtypes,
               double max_norm, double eps, float* norm, void* workspace, int64_t workspace_bytes, void* stream) {
    using namespace tg;
    const int64_t need = tgemm_clip_workspace_bytes(tensors, counts);
    if (need < 0 || !(max_norm >= 0.0) || !(eps >= 0.0)) {
        set_error("tensors=%lld, max_norm=%g, eps=%g or a tensor's size out of range", (long long)tensors, max_norm, eps);
        return TGEMM_E_ARG;
    }
    if (!norm || !workspace || (tensors > 0 && (!in || !out || !dtypes))) {
        set_error("NULL table, norm or workspace");
        return TGEMM_E_NULL;
    }
    if (workspace_bytes < need) {
        set_error("workspace of %lld bytes, %lld needed", (long long)workspace_bytes, (long long)need);
        return TGEMM_E_ARG;
    }
    if ((uintptr_t)norm % 4 || (uintptr_t)workspace % 256) {
        set_error("norm or workspace not aligned");
        return TGEMM_E_ALIGN;
    }
    double total;
    clip_total(tensors, counts, &total);
    for (int64_t i = 0; i < tensors; ++i) {
        if (dtypes[i] != TGEMM_F32 && dtypes[i] != TGEMM_BF16 && dtypes[i] != TGEMM_F16) {
            set_error("tensor %lld: dtype %d is not float32, bfloat16 or float16", (long long)i, dtypes[i]);
            return TGEMM_E_ARG;
        }
        if (counts[i] > 0 && (!in[i] || !out[i])) {
            set_error("tensor %lld: NULL pointer", (long long)i);
            return TGEMM_E_NULL;
        }
        if (((uintptr_t)in[i] | (uintptr_t)out[i]) % (dtypes[i] == TGEMM_F32 ? 4 : 2)) {
            set_error("tensor %lld: not aligned to its element size", (long long)i);
            return TGEMM_E_ALIGN;
        }
    }
    int rc = clip_check_overlap(tensors, in, out, counts, dtypes);
    if (rc == TGEMM_OK) rc = current_device_ok();
    if (rc != TGEMM_OK) return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    float* factor = static_cast<float*>(workspace);
    double* sums = reinterpret_cast<double*>(static_cast<char*>(workspace) + 256);
    const int64_t piece = clip_piece(total);
    // Up to CLIP_TENSORS tensors a launch, from the first on or from the last.
    auto launches = [&](const void* fn, bool back, int64_t* groups) {
        for (int64_t i = 0; i < tensors && rc == TGEMM_OK;) {
            ClipArgs a{};
            a.piece = (int32_t)piece;
            a.sums = sums + *groups;
            a.factor = factor;
            int64_t n = 0;
            for (; i < tensors && a.tensors < CLIP_TENSORS; ++i) {
                const int64_t t = back ? tensors - 1 - i : i;
                if (counts[t] == 0) continue;
                const int k = a.tensors++;
                a.in[k] = in[t];
                a.out[k] = out[t];
                a.count[k] = counts[t];
                a.dtype[k] = (uint8_t)dtypes[t];
                a.first[k] = (uint32_t)n;
                n += (counts[t] + piece - 1) / piece;
            }
            if (n == 0) continue;
            rc = mm_launch(fn, n, CLIP_THREADS, &a, "clipping", st);
            *groups += n;
        }
    };
    int64_t groups = 0, again = 0;
    launches(reinterpret_cast<const void*>(clip_squares_kernel), false, &groups);
    if (rc == TGEMM_OK) {
        void* args[] = {&sums, &groups, &max_norm, &eps, &norm, &factor};
        rc = mm_launch_list(reinterpret_cast<const void*>(clip_norm_kernel), 1, 1024, args, "norm", st);
    }
    launches(reinterpret_cast<const void*>(clip_times_kernel), true, &again);
    if (rc == TGEMM_OK) clear_error();
    return rc;
}

}  // extern "C"
