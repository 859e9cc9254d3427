// w4_block_f32.hip - the 4-bit products' form for many rows (w4_block.h) over fp32 rows.
#include "w4_block.h"

namespace moe {

hipError_t launch_w4_block_f32(const W4Params &p, hipStream_t s) { return launch_form<float>(p, s); }

}  // namespace moe
