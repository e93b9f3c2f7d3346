#include "tg_mm_kernels.hpp"

namespace tg {
typedef MmTiles<MmF16, ALONG, ALONG, false> Tiles;
const MmKernel* mm_dz_f16() {
    static const MmKernel table[SIZE_COUNT] = {
        mm_entry<Tiles::T256>(reinterpret_cast<const void*>(mm_dz_kernel<Tiles::T256>)),
        mm_entry<Tiles::T128>(reinterpret_cast<const void*>(mm_dz_kernel<Tiles::T128>)),
        mm_entry<Tiles::T64>(reinterpret_cast<const void*>(mm_dz_kernel<Tiles::T64>)),
        mm_entry<Tiles::T128Deep>(reinterpret_cast<const void*>(mm_dz_kernel<Tiles::T128Deep>)),
    };
    return table;
}
}  // namespace tg
