#include "tg_mm_kernels.hpp"

namespace tg {
typedef MmTiles<MmF16, ALONG, ACROSS, false> Tiles;
const MmKernel* mm_dh_f16() {
    static const MmKernel table[SIZE_COUNT] = {
        {reinterpret_cast<const void*>(mm_dh_kernel<Tiles::T256>), Tiles::T256::BM, Tiles::T256::TILE_N, Tiles::T256::NT},
        {reinterpret_cast<const void*>(mm_dh_kernel<Tiles::T128>), Tiles::T128::BM, Tiles::T128::TILE_N, Tiles::T128::NT},
        {reinterpret_cast<const void*>(mm_dh_kernel<Tiles::T64>), Tiles::T64::BM, Tiles::T64::TILE_N, Tiles::T64::NT},
    };
    return table;
}
}  // namespace tg
