// w4_block_bf16.hip - the 4-bit products' form for many rows (w4_block.h) over bf16 rows.
#include "w4_block.h"

namespace moe {

hipError_t launch_w4_block_bf16(const W4Params &p, hipStream_t s) { return launch_form<uint16_t>(p, s); }

}  // namespace moe
