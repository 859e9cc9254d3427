// w4_block_round.hip - the 4-bit products' form for many rows (w4_block.h) over bf16 rows, weights rounded
// to bf16.
#include "w4_block.h"

namespace moe {

hipError_t launch_w4_block_round(const W4Params &p, hipStream_t s) { return launch_form<uint16_t, true>(p, s); }

}  // namespace moe
