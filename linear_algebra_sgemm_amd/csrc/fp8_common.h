// What the two kernel files of the block-scaled product share.
#pragma once

#include "lm_common.h"
#include "lm_launch.h"

namespace lasg {

// The tiled kernels (fp8_tile_kernels.hip): tiles 0 to 4 of fp8_tile.  Tiles 0
// to 3 copy straight into LDS, which the call has to allow (fp8_direct).
bool fp8_direct(const Fp8Call& c);
hipError_t launch_fp8_tile(const Fp8Call& c, int tile, hipStream_t s);

}  // namespace lasg
