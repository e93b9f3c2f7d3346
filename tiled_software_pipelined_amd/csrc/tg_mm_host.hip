// Choice of kernel and launches of the 16-bit products with fused ends, and the
// kernel that joins partial sums.
#include "tg_mm_host.hpp"

#include <climits>
#include <cmath>

namespace tg {

#define TG_MM_TABLES(t)                                                                                         \
    const MmKernel *mm_nt_##t(), *mm_nn_##t(), *mm_tn_##t(), *mm_nn_sum_##t(), *mm_gate_##t(), *mm_dh_##t(), *mm_stats_##t(), *mm_dz_##t(), \
        *mm_stats_keep_##t();                                                                                   \
    static const MmKernel* mm_kernels_##t(int form) {                                                           \
        switch (form) {                                                                                         \
            case FORM_NT: return mm_nt_##t();                                                                   \
            case FORM_NN: return mm_nn_##t();                                                                   \
            case FORM_TN: return mm_tn_##t();                                                                   \
            case FORM_NN_SUM: return mm_nn_sum_##t();                                                           \
            case FORM_GATE: return mm_gate_##t();                                                               \
            case FORM_DH: return mm_dh_##t();                                                                   \
            case FORM_STATS: return mm_stats_##t();                                                             \
            case FORM_STATS_KEEP: return mm_stats_keep_##t();                                                   \
            default: return mm_dz_##t();                                                                        \
        }                                                                                                       \
    }
TG_MM_TABLES(bf16)
TG_MM_TABLES(f16)
#undef TG_MM_TABLES

const MmKernel* mm_kernels(int dtype, int form) {
    return dtype == TGEMM_BF16 ? mm_kernels_bf16(form) : mm_kernels_f16(form);
}

static double tiles_of(const MmKernel& k, const MmShape* shapes, int jobs) {
    double n = 0.0;
    for (int i = 0; i < jobs; ++i)
        n += (double)((shapes[i].M + k.bm - 1) / k.bm) * (double)((shapes[i].N + k.bn - 1) / k.bn);
    return n;
}

// Model of a launch's time in microseconds, from runs of every form and tile at
// 14 shapes (100 .. 4096 rows, 768 .. 50240 columns, K = 64 .. 50240).  A slice of 64
// k: `alone` where at most 256 workgroups run, `full` where the machine is (tiles
// that stand twice on a compute unit: of both), where the weight comes from memory for
// few rows at least `cold`.  `fixed`: the way in and out, by form.
//   us                          256    128     64  128 deep
//   nt   512x1024x2816         30.6   24.2   16.1   18.0
//   nt   1024x1024x4096        37.2   27.8   21.6   24.4
//   nt   2048x2048x5440        61.7   55.5   55.8   46.2
//   nt   4096x4096x4096         110    133    172    145
//   tn   50240x768x64          27.6   22.0   36.0   36.9
//   gate 100x11008x4096        97.0   63.3   58.4   48.6
//   gate 256x11008x4096        99.1   78.2   86.2   84.2
//   nt   256x4096x11008        59.8   51.2   51.7   44.6
//   gate 2048x5440x2048         106    109    140    124
//   dh   2048x5440x2048       66.7   63.0   73.2   64.6
//   stats 60x50240x768         24.8   20.1   18.9   21.4
//   stats 2048x5440x2048       45.3   52.5   59.4   49.5
struct MmRate {
    double alone, full, cold[2], fixed[FORM_COUNT];  // cold: up to 256 workgroups, and more
};
//                                               nt   nn   tn  sum  gate  dh  stats dz
static const MmRate MM_RATES[SIZE_COUNT] = {
    {0.99, 1.60, {1.40, 1.6}, {6.3, 6.3, 6.3, 9.0, 9.5, 20.0, 6.5, 9.7}},
    {0.60, 1.00, {0.90, 1.2}, {1.5, 1.5, 1.5, 3.0, 4.4, 4.5, 3.0, 4.0}},
    {0.30, 0.70, {0.46, 0.85}, {3.4, 3.8, 5.0, 5.0, 3.5, 4.0, 3.7, 4.5}},
    {0.35, 0.54, {0.65, 0.65}, {3.7, 4.0, 4.4, 5.0, 6.0, 5.0, 3.9, 5.0}},
};

// n workgroups of some slices each
static double mm_rounds(int form, int size, int slots, double n, double slices, bool cold) {
    const MmRate& r = MM_RATES[size];
    const double fixed = r.fixed[form], whole = floor(n / slots), rest = n - whole * slots;
    auto least = [&](double v, int i) { return cold && r.cold[i] > v ? r.cold[i] : v; };
    double t = whole * (fixed + least(r.full, 1) * slices);
    if (rest > 0.0)
        t += fixed + slices * (slots == 256 ? least(r.alone + (r.full - r.alone) * rest / 256.0, 0)
                                            : rest <= 256.0 ? least(r.alone, 0) : least(r.full, 1));
    return t;
}

static double mm_time(int form, int size, const MmKernel& k, double tiles, int64_t slices, bool may_split, bool cold) {
    if (tiles > 1e6) return mm_rounds(form, size, k.slots, tiles, (double)slices, cold);
    const MmSchedule s = mm_schedule((int)tiles, (int)slices, k.slots, k.slice, k.tile_kb, may_split);
    double t = mm_rounds(form, size, k.slots, s.full, (double)slices, cold);
    if (s.rest) t += mm_rounds(form, size, k.slots, s.rest * s.splits, s.per, cold) + 9.0 + s.rest * s.splits * k.tile_kb * 0.4e-3;
    return t;
}

// What rows off 16-byte boundaries cost: at even elements, at odd ones.
static const double MM_EVEN[SIZE_COUNT] = {1.2, 1.3, 1.45, 1.5}, MM_ODD[SIZE_COUNT] = {1.3, 2.3, 2.0, 2.0};

MmSize mm_size(int form, const MmShape* shapes, int jobs, int64_t slices, bool may_split, int64_t row) {
    MmSize best = SIZE_64;
    double least = -1.0;
    const MmKernel* table = mm_kernels(TGEMM_BF16, form);  // the types' tiles are alike
    for (int s = 0; s < SIZE_COUNT; ++s) {
        const bool cold = shapes[0].M <= 256;
        double t = mm_time(form, s, table[s], tiles_of(table[s], shapes, jobs), slices, may_split, cold);
        // across k a chunk's rows are further apart and the cost is less
        const double off = row % 8 == 0 ? 0.0 : (row % 2 ? MM_ODD[s] : MM_EVEN[s]) - 1.0;
        t *= 1.0 + off * (form == FORM_TN ? 0.5 : 1.0);
        if (least < 0.0 || t < least) {
            least = t;
            best = (MmSize)s;
        }
    }
    return best;
}

int64_t mm_split_bytes(int form, MmSize size, const MmShape* shapes, int jobs, int64_t slices, bool fewer) {
    const MmKernel& k = mm_kernels(TGEMM_BF16, form)[size];
    const double tiles = tiles_of(k, shapes, jobs);
    if (tiles > 1e6 || tiles < 1.0 || slices < MM_LEAST_SLICES) return 0;
    const int64_t tile = (int64_t)k.bm * k.bn * 4;
    // up to `slots` parts, in any number of tiles
    if (fewer) return k.slots * tile;
    const MmSchedule s = mm_schedule((int)tiles, (int)slices, k.slots, k.slice, k.tile_kb, true);
    return s.rest * s.splits * tile;
}

MmGrid mm_grid(const MmKernel& k, int64_t M, int64_t N) {
    return MmGrid{(int32_t)((M + k.bm - 1) / k.bm), (int32_t)((N + k.bn - 1) / k.bn)};
}

int mm_check_grid(const char* name, double workgroups, int threads) {
    if (workgroups > INT_MAX || !grid_fits(workgroups, threads)) {
        set_error("%s: too many tiles", name);
        return TGEMM_E_ARG;
    }
    return TGEMM_OK;
}

int mm_check_tiles(const char* name, int form, MmSize size, const MmShape* shapes, int jobs) {
    const MmKernel& k = mm_kernels(TGEMM_BF16, form)[size];
    // `slots` more: parts of tiles that a launch shares out
    return mm_check_grid(name, tiles_of(k, shapes, jobs) + k.slots, k.threads);
}

int mm_launch_list(const void* fn, int64_t workgroups, int threads, void** args, const char* name, hipStream_t stream) {
    const int rc = mm_check_grid(name, (double)workgroups, threads);
    if (rc != TGEMM_OK) return rc;
    const hipError_t err = hipLaunchKernel(fn, dim3((unsigned)workgroups), dim3(threads), args, 0, stream);
    if (err != hipSuccess) {
        set_error("launch of %s failed: %s", name, hipGetErrorString(err));
        return TGEMM_E_HIP;
    }
    return TGEMM_OK;
}

int mm_store(int dtype, int form, MmSize size, const MmStoreArgs& given, hipStream_t stream) {
    const MmKernel& k = mm_kernels(dtype, form)[size];
    MmStoreArgs args = given;
    args.jobs = 0;
    double tiles = 0.0;
    for (int i = 0; i < given.jobs; ++i) {
        const MmOperands& o = given.job[i].op[0];
        if (o.M == 0 || o.N == 0) continue;
        MmJob& j = args.job[args.jobs++];
        j = given.job[i];
        j.grid = mm_grid(k, o.M, o.N);
        j.stream = (uintptr_t)j.C % 128 == 0 && j.ldc % 64 == 0;
        tiles += (double)j.grid.tiles_m * j.grid.tiles_n;
    }
    if (args.jobs == 0) return TGEMM_OK;
    int64_t slices = 0;
    for (int p = 0; p < args.job[0].pairs; ++p) slices += mm_slices(args.job[0].op[p].K);
    if (tiles > 1e6 || slices < MM_LEAST_SLICES) args.split = nullptr;
    if (tiles > INT_MAX / 2) {
        set_error("product: too many tiles");
        return TGEMM_E_ARG;
    }
    const MmSchedule s = mm_schedule((int)tiles, (int)slices, k.slots, k.slice, k.tile_kb, args.split != nullptr);
    // fewer rows than the host knows of may be shared out in up to `slots` parts
    const bool fewer = args.rows && args.split;
    int rc = mm_launch(k.fn, fewer ? (int64_t)tiles + k.slots : s.total(), k.threads, &args, "product", stream);
    const int64_t rest = fewer ? (tiles < k.slots / 2 ? (int64_t)tiles : k.slots / 2) : s.rest;
    if (rc == TGEMM_OK && args.split && rest > 0) rc = mm_launch(k.join, rest * (k.bm * k.bn / MM_JOIN), 256, &args, "join", stream);
    return rc;
}

int mm_round(int dtype, const MmStoreArgs& args, hipStream_t stream) {
    MmStoreArgs a = args;
    const int64_t M = a.job[0].op[0].M, N = a.job[0].op[0].N;
    if (M == 0 || N == 0) return TGEMM_OK;
    const void* fn = dtype == TGEMM_BF16 ? reinterpret_cast<const void*>(mm_round_kernel<__bf16>)
                                         : reinterpret_cast<const void*>(mm_round_kernel<_Float16>);
    return mm_launch(fn, (M * ((N + 3) / 4) + 255) / 256, 256, &a, "rounding", stream);
}

// ---- rows on lines ---------------------------------------------------------------
struct MmPackArgs {
    struct {
        const uint16_t* src;
        uint16_t* dst;
        int64_t ld, rows, cols, ldto, first;  // first: workgroup at which it starts
    } job[3];
    int32_t jobs;
};

// A wave a row; what is behind the row's end up to the line's is not written.
__global__ __launch_bounds__(256) void mm_pack_kernel(MmPackArgs g) {
    int which = 0;
    while (which + 1 < g.jobs && (int64_t)blockIdx.x >= g.job[which + 1].first) ++which;
    const auto& j = g.job[which];
    const int64_t r = ((int64_t)blockIdx.x - j.first) * 4 + wave_id();
    if (r >= j.rows) return;
    const uint16_t* src = j.src + r * j.ld;
    uint16_t* dst = j.dst + r * j.ldto;
    for (int64_t k = 8 * lane_id(); k < j.cols; k += 512) {
        i32x4 v;
        if (k + 8 <= j.cols) {
            v = load16(src + k);
        } else {
            union { i32x4 v; uint16_t e[8]; } u;
#pragma unroll
            for (int e = 0; e < 8; ++e) u.e[e] = load_or_zero(src + k + e, k + e < j.cols);
            v = u.v;
        }
        *reinterpret_cast<i32x4*>(dst + k) = v;
    }
}

int mm_pack(const MmPack* list, int count, hipStream_t stream) {
    MmPackArgs a{};
    int64_t n = 0;
    for (int i = 0; i < count; ++i) {
        if (list[i].rows == 0 || list[i].cols == 0) continue;
        auto& j = a.job[a.jobs++];
        j.src = static_cast<const uint16_t*>(list[i].src);
        j.dst = static_cast<uint16_t*>(list[i].dst);
        j.ld = list[i].ld;
        j.rows = list[i].rows;
        j.cols = list[i].cols;
        j.ldto = mm_lines(list[i].cols);
        j.first = n;
        n += (list[i].rows + 3) / 4;
    }
    return n == 0 ? TGEMM_OK : mm_launch(reinterpret_cast<const void*>(mm_pack_kernel), n, 256, &a, "rows on lines", stream);
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
