#include "tg_mm_kernels.hpp"

namespace tg {
typedef MmTiles<MmBf16, ALONG, ACROSS, false> Tiles;
const MmKernel* mm_dh_bf16() {
    static const MmKernel table[SIZE_COUNT] = {
        mm_entry<Tiles::T256Loads>(reinterpret_cast<const void*>(mm_dh_kernel<Tiles::T256Loads>)),
        mm_entry<Tiles::T128>(reinterpret_cast<const void*>(mm_dh_kernel<Tiles::T128>)),
        mm_entry<Tiles::T64>(reinterpret_cast<const void*>(mm_dh_kernel<Tiles::T64>)),
        mm_entry<Tiles::T128Deep>(reinterpret_cast<const void*>(mm_dh_kernel<Tiles::T128Deep>)),
    };
    return table;
}
}  // namespace tg
