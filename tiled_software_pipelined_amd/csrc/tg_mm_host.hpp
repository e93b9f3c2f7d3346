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
// Rows that a launch with a wave for each reaches (a grid holds 2^32 - 1 threads),
// with some workgroups to spare.
constexpr int64_t MM_WAVE_ROWS = (INT64_C(1) << 26) - 128;

const MmKernel* mm_kernels(int dtype, int form);
inline int64_t mm_slices(int64_t K) { return (K + 63) / 64; }

// The tile of one launch's products, each M x N with this many slices of k.
struct MmShape {
    int64_t M, N;
};
// row: elements of an operand's row as the copies read it (K along k, else the
// result's rows or columns); its last bits are its alignment.
MmSize mm_size(int form, const MmShape* shapes, int jobs, int64_t slices, bool may_split, int64_t row);
inline MmSize mm_size(int form, int64_t M, int64_t N, int64_t slices, bool may_split, int64_t row) {
    const MmShape s{M, N};
    return mm_size(form, &s, 1, slices, may_split, row);
}

// Copies of an operand's rows to whole 128-byte lines.  Rows that start at odd
// elements make the tile kernels' copies up to twice as slow (2047x2050x5461 along k:
// 128 tiles 135 us, on lines 64; 256 tiles 81), so a copy of the weights pays where
// many rows of the other operand M read them, each at least K wide.  Forward passes
// of seven blocks (K 769 .. 4097), bfloat16 and float16, time without copies over
// time with them, geometric means:
//   M                512   768  1024  1500  2047  3000  4096  6000  8192
//   odd K, odd F    0.95  0.97  0.99  0.98  0.96  1.01  1.05  1.10  1.07
// and of a training step's loss, whose backward pass reads w twice (V 32000 .. 128001):
//   K 513 .. 4097               0.93        0.99  1.02  1.02  1.04  1.04
//   K 65 .. 385                 0.96        0.94  0.97  0.95  1.02  1.00
// Of the loss's forward pass, which reads it once, 0.94 to 1.01.  Rows at other even
// elements cost a fifth at most (2048x5440x2050 gate and up 128 us, 2048 wide 107), and
// copies of theirs pay nowhere (block 0.82 to 1.05, loss 0.44 to 1.00).
inline bool mm_packs(int64_t K, int64_t M) { return K % 2 && K >= 512 && M >= 3000; }
inline int64_t mm_lines(int64_t K) { return (K + 63) / 64 * 64; }
struct MmPack {
    const void* src;
    int64_t ld, rows, cols;
    void* dst;  // row stride mm_lines(cols)
};
inline bool mm_aligned(const void* p, int64_t ld) { return ld % 8 == 0 && (uintptr_t)p % 16 == 0; }
int mm_pack(const MmPack* list, int count, hipStream_t stream);
// Bytes for the sums of tiles that a launch shares out (MmStoreArgs::split), for
// as many rows as given or, where only the device knows them (`fewer`), less.
int64_t mm_split_bytes(int form, MmSize size, const MmShape* shapes, int jobs, int64_t slices, bool fewer);

MmGrid mm_grid(const MmKernel& k, int64_t M, int64_t N);
// TGEMM_OK where a grid holds a launch: the entry points ask for all of theirs
// before the first.
int mm_check_grid(const char* name, double workgroups, int threads);
int mm_check_tiles(const char* name, int form, MmSize size, const MmShape* shapes, int jobs);
inline int mm_check_tiles(const char* name, int form, MmSize size, int64_t M, int64_t N) {
    const MmShape s{M, N};
    return mm_check_tiles(name, form, size, &s, 1);
}

// Launches products of the store forms on tiles of one size, and the join of
// what it shares out; jobs without rows or columns are left out.
int mm_store(int dtype, int form, MmSize size, const MmStoreArgs& args, hipStream_t stream);
// The first job's float sums into its C.
int mm_round(int dtype, const MmStoreArgs& args, hipStream_t stream);
int mm_launch_list(const void* fn, int64_t workgroups, int threads, void** args, const char* name, hipStream_t stream);
inline int mm_launch(const void* fn, int64_t workgroups, int threads, void* args, const char* name, hipStream_t stream) {
    void* list[] = {args};
    return mm_launch_list(fn, workgroups, threads, list, name, stream);
}

// A tensor argument's checks: rows x cols of `dtype`, leading dimension ld.
int mm_check(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld);
int mm_check_buffer(const char* name, const void* p, int64_t bytes);

}  // namespace tg
