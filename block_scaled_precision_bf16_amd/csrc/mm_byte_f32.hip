// mm_byte_f32.hip -- the tiled MXFP8 product kernel, rows at any byte, fp32 outputs.
#include "mm_tile.h"

namespace mxk {

hipError_t launch_mm_byte_f32(const MmArgs &a, const MmTable &t, hipStream_t stream)
{
    return a.tiled ? launch_mm_tile_mode<kExact, kMmByteM, kMmByteN, true, false>(a, t, stream)
                   : launch_mm_tile_mode<kExact, kMmByteM, kMmByteN, false, false>(a, t, stream);
}

}  // namespace mxk
