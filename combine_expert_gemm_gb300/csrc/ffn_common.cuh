// What the forward and the backward of the dense gated feed-forward block share.
#pragma once

#include "../../include/moe_dense.h"
#include "pair_gemm.cuh"

namespace moe {

// Tile counts and coordinates are 32-bit, offsets of elements 64-bit.
inline moe_status check_ffn(int32_t T, int32_t d, int32_t h) {
    if (T < 0 || d <= 0 || h <= 0) return MOE_ERR_INVALID_ARG;
    if (d % 8 != 0 || h % 8 != 0) return MOE_ERR_ALIGNMENT;
    if (d > 65536 || h > 65536 || (int64_t)T > (int64_t)1 << 24) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace moe
