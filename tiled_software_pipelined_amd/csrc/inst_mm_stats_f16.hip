#include "tg_mm_kernels.hpp"

namespace tg {
typedef MmTiles<MmF16, ALONG, ALONG, false> Tiles;
const MmKernel* mm_stats_f16() {
    static const MmKernel table[SIZE_COUNT] = {
        mm_entry<Tiles::T256>(reinterpret_cast<const void*>(mm_stats_kernel<Tiles::T256, false>)),
        mm_entry<Tiles::T128>(reinterpret_cast<const void*>(mm_stats_kernel<Tiles::T128, false>)),
        mm_entry<Tiles::T64>(reinterpret_cast<const void*>(mm_stats_kernel<Tiles::T64, false>)),
        mm_entry<Tiles::T128Deep>(reinterpret_cast<const void*>(mm_stats_kernel<Tiles::T128Deep, false>)),
    };
    return table;
}
}  // namespace tg
