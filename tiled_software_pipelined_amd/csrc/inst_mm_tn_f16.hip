#include "tg_mm_kernels.hpp"

namespace tg {
typedef MmTiles<MmF16, ACROSS, ACROSS, false> Tiles;
const MmKernel* mm_tn_f16() {
    static const MmKernel table[SIZE_COUNT] = {
        mm_entry<Tiles::T256>(reinterpret_cast<const void*>(mm_store_kernel<Tiles::T256, false>), reinterpret_cast<const void*>(mm_join_kernel<Tiles::T256>)),
        mm_entry<Tiles::T128>(reinterpret_cast<const void*>(mm_store_kernel<Tiles::T128, false>), reinterpret_cast<const void*>(mm_join_kernel<Tiles::T128>)),
        mm_entry<Tiles::T64>(reinterpret_cast<const void*>(mm_store_kernel<Tiles::T64, false>), reinterpret_cast<const void*>(mm_join_kernel<Tiles::T64>)),
        mm_entry<Tiles::T128Deep>(reinterpret_cast<const void*>(mm_store_kernel<Tiles::T128Deep, false>), reinterpret_cast<const void*>(mm_join_kernel<Tiles::T128Deep>)),
    };
    return table;
}
}  // namespace tg
