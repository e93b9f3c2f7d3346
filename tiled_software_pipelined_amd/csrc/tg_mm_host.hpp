// Host side of the 16-bit products with fused ends: choice of kernel, launches.
#pragma once

#include <hip/hip_runtime.h>

#include "tg_host.hpp"
#include "tg_mm_kernels.hpp"
#include "tgemm.h"

namespace tg {

// Row strides and contracted sizes up to this (elements): a lane of a copy
// reaches 255 rows past its tile's first by a 32-bit byte offset.
constexpr int64_t MM_MOST = INT64_C(1) << 22;
constexpr int64_t MM_MOST_ROWS = INT64_C(1) << 30;

// How a product is laid out on the machine.
struct MmPlan {
    MmSize size;
    int splits, per;  // parts of k, slices of 64 k each
};

const MmKernel* mm_kernels(int dtype, int form);
// The plan of one launch's products, each M x N with this many slices of k; and
// the bytes of one product's partial sums, 0 without a split.
struct MmShape {
    int64_t M, N;
};
MmPlan mm_plan(int form, const MmShape* shapes, int jobs, int64_t slices, bool may_split);
inline int64_t mm_part_bytes(const MmPlan& p, int64_t M, int64_t N, bool add) {
    return p.splits > 1 || add ? (4 * p.splits * M * N + 255) / 256 * 256 : 0;
}
inline int64_t mm_slices(int64_t K) { return (K + 63) / 64; }
MmGrid mm_grid(const MmKernel& k, const MmPlan& p, int64_t M, int64_t N);

// Launches `jobs` products of the store forms by one plan; jobs without rows or
// columns are left out.  Partial sums (job.part set) are not joined here.
int mm_store(int dtype, int form, const MmPlan& plan, const MmStoreArgs& args, hipStream_t stream);
// C = alpha sum of the jobs' partial sums.
int mm_join(int dtype, const MmPlan& plan, const MmStoreArgs& args, hipStream_t stream);
int mm_launch(const void* fn, int64_t workgroups, int threads, void* args, const char* name, hipStream_t stream);

// A tensor argument's checks: rows x cols of `dtype`, leading dimension ld.
int mm_check(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld);
int mm_check_buffer(const char* name, const void* p, int64_t bytes);

}  // namespace tg
