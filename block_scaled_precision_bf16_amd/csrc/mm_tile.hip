// mm_tile.hip -- the tiled MXFP8 product kernel, bf16 outputs.
#include "mm_tile.h"

namespace mxk {

hipError_t launch_mm_tile(const MmArgs &a, const MmTable &t, hipStream_t stream)
{
    return a.tiled ? launch_mm_tile_mode<kMx, kMmTileM, kMmTileN, true>(a, t, stream)
                   : launch_mm_tile_mode<kMx, kMmTileM, kMmTileN, false>(a, t, stream);
}

}  // namespace mxk
