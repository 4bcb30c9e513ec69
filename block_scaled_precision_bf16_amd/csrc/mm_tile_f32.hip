// mm_tile_f32.hip -- the tiled MXFP8 product kernel, fp32 outputs.
#include "mm_tile.h"

namespace mxk {

hipError_t launch_mm_tile_f32(const MmArgs &a, const MmTable &t, hipStream_t stream)
{
    return a.tiled ? launch_mm_tile_mode<kExact, kMmTileM, kMmTileN, true>(a, t, stream)
                   : launch_mm_tile_mode<kExact, kMmTileM, kMmTileN, false>(a, t, stream);
}

}  // namespace mxk
