// Weights in 4 bits: how a word holds the codes of eight input rows of a column (internal).
//
// Row 8j+i's code, plus 8, lies at bit 4*(i/2) + 16*(i%2) of word j: the codes of rows 2p and 2p+1 are 16 bits apart,
// so one shift and one mask bring both into the two halves of a register that a bf16 matrix operand wants.
#pragma once

#include "moonep_common.h"

namespace moonep {

__host__ __device__ __forceinline__ int code4_bit(int i) { return 4 * (i / 2) + 16 * (i % 2); }
__device__ __forceinline__ int code4(uint32_t word, int i) { return (int)((word >> code4_bit(i)) & 15u) - 8; }

}  // namespace moonep
