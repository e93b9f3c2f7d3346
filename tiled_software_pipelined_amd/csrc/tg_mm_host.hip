// Choice of kernel and launches of the 16-bit products with fused ends, and the
// kernel that joins partial sums.
#include "tg_mm_host.hpp"

#include <climits>
#include <cmath>

namespace tg {

#define TG_MM_TABLES(t)                                                                                         \
    const MmKernel *mm_nt_##t(), *mm_nn_##t(), *mm_tn_##t(), *mm_gate_##t(), *mm_dh_##t(), *mm_stats_##t(), *mm_dz_##t(); \
    static const MmKernel* mm_kernels_##t(int form) {                                                           \
        switch (form) {                                                                                         \
            case FORM_NT: return mm_nt_##t();                                                                   \
            case FORM_NN: return mm_nn_##t();                                                                   \
            case FORM_TN: return mm_tn_##t();                                                                   \
            case FORM_GATE: return mm_gate_##t();                                                               \
            case FORM_DH: return mm_dh_##t();                                                                   \
            case FORM_STATS: return mm_stats_##t();                                                             \
            default: return mm_dz_##t();                                                                        \
        }                                                                                                       \
    }
TG_MM_TABLES(bf16)
TG_MM_TABLES(f16)
#undef TG_MM_TABLES

const MmKernel* mm_kernels(int dtype, int form) {
    return dtype == TGEMM_BF16 ? mm_kernels_bf16(form) : mm_kernels_f16(form);
}

static int tile_m(int s) { return s == SIZE_256 ? 256 : s == SIZE_128 ? 128 : 64; }
static int tile_n(int form, int s) { return (s == SIZE_256 ? 256 : 128) / (form == FORM_GATE ? 2 : 1); }

// Microseconds of one launch.
static double mm_time(int form, int size, double tiles, double slices) {
    (void)form;
    const double slots = size == SIZE_256 ? 256.0 : 512.0;
    const double slice = size == SIZE_256 ? 0.43 : size == SIZE_128 ? 0.30 : 0.20;
    const double alone = size == SIZE_256 ? 0.43 : size == SIZE_128 ? 0.22 : 0.14;
    if (tiles <= 256.0) return 4.0 + alone * slices;
    return 4.0 + ceil(tiles / slots) * (1.0 + slice * slices);
}

MmPlan mm_plan(int form, const MmShape* shapes, int jobs, int64_t slices, bool may_split) {
    MmPlan best{SIZE_64, 1, (int)(slices > 0 ? slices : 1)};
    double least = -1.0, area = 0.0;
    for (int i = 0; i < jobs; ++i) area += (double)shapes[i].M * (double)shapes[i].N;
    for (int s = 0; s < SIZE_COUNT; ++s) {
        double tiles = 0.0;
        for (int i = 0; i < jobs; ++i)
            tiles += (double)((shapes[i].M + tile_m(s) - 1) / tile_m(s)) * (double)((shapes[i].N + tile_n(form, s) - 1) / tile_n(form, s));
        for (int splits = 1; splits <= 16; ++splits) {
            const int64_t per = (slices + splits - 1) / splits;
            if (splits > 1 && (!may_split || per < 8 || tiles * splits > 1024.0)) break;
            if (splits > 1 && (splits - 1) * per >= slices) continue;  // a part would be empty
            double t = mm_time(form, s, tiles * splits, (double)per);
            // sums written and read again, and another launch
            if (splits > 1) t += 3.0 + area * (8.0 * splits + 2.0) / 4e6;
            if (least < 0.0 || t < least) {
                least = t;
                best = MmPlan{(MmSize)s, splits, (int)(per > 0 ? per : 1)};
            }
        }
    }
    return best;
}

MmGrid mm_grid(const MmKernel& k, const MmPlan& p, int64_t M, int64_t N) {
    return MmGrid{(int32_t)((M + k.bm - 1) / k.bm), (int32_t)((N + k.bn - 1) / k.bn), p.splits, p.per};
}

int mm_launch(const void* fn, int64_t workgroups, int threads, void* args, const char* name, hipStream_t stream) {
    if (workgroups > INT_MAX || !grid_fits((double)workgroups, threads)) {
        set_error("%s: too many tiles", name);
        return TGEMM_E_ARG;
    }
    void* list[] = {args};
    const hipError_t err = hipLaunchKernel(fn, dim3((unsigned)workgroups), dim3(threads), list, 0, stream);
    if (err != hipSuccess) {
        set_error("launch of %s failed: %s", name, hipGetErrorString(err));
        return TGEMM_E_HIP;
    }
    return TGEMM_OK;
}

int mm_store(int dtype, int form, const MmPlan& plan, const MmStoreArgs& given, hipStream_t stream) {
    const MmKernel& k = mm_kernels(dtype, form)[plan.size];
    MmStoreArgs args{};
    args.alpha = given.alpha;
    args.rows = given.rows;
    args.rows_are_k = given.rows_are_k;
    args.map = given.map;
    int64_t n = 0;
    for (int i = 0; i < given.jobs; ++i) {
        const MmOperands& o = given.job[i].op[0];
        if (o.M == 0 || o.N == 0) continue;
        MmJob& j = args.job[args.jobs++];
        j = given.job[i];
        j.grid = mm_grid(k, plan, o.M, o.N);
        n += (int64_t)j.grid.tiles_m * j.grid.tiles_n * j.grid.splits;
    }
    return n == 0 ? TGEMM_OK : mm_launch(k.fn, n, k.threads, &args, "product", stream);
}

// ---- partial sums ------------------------------------------------------------
struct JoinArgs {
    struct {
        const float* part;
        void* C;
        int64_t ldc, M, N, stride;  // stride: floats from a split to the next
        int64_t first;              // workgroups before this job's
    } job[3];
    int32_t jobs, splits;
    const float* alpha;
    const int32_t *rows, *map;  // NULL, or as MmStoreArgs has them
};

// 4 adjacent columns a thread, splits in order (the result does not depend on
// who finished first).
template <class T>
__global__ __launch_bounds__(256) void mm_join_kernel(JoinArgs g) {
    int which = 0;
    while (which + 1 < g.jobs && (int64_t)blockIdx.x >= g.job[which + 1].first) ++which;
    const auto& j = g.job[which];
    const int64_t quads = (j.N + 3) / 4, q = ((int64_t)blockIdx.x - j.first) * 256 + threadIdx.x;
    if (q >= (g.rows ? *g.rows : j.M) * quads) return;
    const int64_t m = q / quads, n = (q - m * quads) * 4;
    const int count = (int)min(j.N - n, (int64_t)4);
    const float* p = j.part + m * j.N + n;
    float v[4] = {0, 0, 0, 0};
    for (int s = 0; s < g.splits; ++s, p += j.stride) {
        float x[4] = {0, 0, 0, 0};
        if (count == 4) {
            __builtin_memcpy(x, p, 16);
        } else {
            for (int e = 0; e < 3; ++e)
                if (e < count) x[e] = p[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += x[e];
    }
    const float alpha = g.alpha ? *g.alpha : 1.0f;
    T o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = (T)(v[e] * alpha);
    T* dst = static_cast<T*>(j.C) + (g.map ? g.map[m] : m) * j.ldc + n;
    if (count == 4) {
        __builtin_memcpy(dst, o, 8);
    } else {
        for (int e = 0; e < 3; ++e)
            if (e < count) dst[e] = o[e];
    }
}

int mm_join(int dtype, const MmPlan& plan, const MmStoreArgs& args, hipStream_t stream) {
    JoinArgs g{};
    int64_t n = 0;
    for (int i = 0; i < args.jobs; ++i) {
        const MmJob& a = args.job[i];
        const int64_t M = a.op[0].M, N = a.op[0].N;
        if (M == 0 || N == 0) continue;
        auto& j = g.job[g.jobs++];
        j.part = a.part;
        j.C = a.C;
        j.ldc = a.ldc;
        j.M = M;
        j.N = N;
        j.stride = M * N;
        j.first = n;
        n += (M * ((N + 3) / 4) + 255) / 256;
    }
    if (n == 0) return TGEMM_OK;
    g.splits = plan.splits;
    g.alpha = args.alpha;
    if (!args.rows_are_k) g.rows = args.rows;
    g.map = args.map;
    const void* fn = dtype == TGEMM_BF16 ? reinterpret_cast<const void*>(mm_join_kernel<__bf16>)
                                         : reinterpret_cast<const void*>(mm_join_kernel<_Float16>);
    return mm_launch(fn, n, 256, &g, "join", stream);
}

// ---- arguments -----------------------------------------------------------------
int mm_check(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld) {
    if (ld < cols || ld > MM_MOST) {
        set_error("%s: leading dimension %lld shorter than its row of %lld, or above 2^22", name, (long long)ld, (long long)cols);
        return TGEMM_E_ARG;
    }
    if (rows > 0 && cols > 0 && !p) {
        set_error("%s: NULL pointer", name);
        return TGEMM_E_NULL;
    }
    if ((uintptr_t)p % 2) {
        set_error("%s: not aligned to its element size", name);
        return TGEMM_E_ALIGN;
    }
    return TGEMM_OK;
}

int mm_check_buffer(const char* name, const void* p, int64_t bytes) {
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
