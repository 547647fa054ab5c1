// Tensor maps of row matrices, for the kernels that load operands with them.
#pragma once
#include <cuda.h>

#include "rows.cuh"

namespace spconv {

// Copies of [outer] rows of `inner` elements, `ld` elements apart, in boxes of
// box_bytes (128 or 64) x box_outer rows, swizzled in shared memory over as
// many bytes; what lies outside reads zeros and is not written.  The rows
// satisfy tma_ok.
int make_tensor_map(CUtensorMap* map, const void* base, size_t es, int64_t inner, int64_t outer, int64_t ld, int32_t box_outer,
                    int32_t box_bytes = 128);

// The same rows in blocks of 64 bf16 columns (inner % 64 == 0), copied as
// 64 columns x 64 rows x `blocks` blocks: coordinates (0, row, block).
int make_tensor_map_blocks(CUtensorMap* map, const void* base, int64_t inner, int64_t outer, int64_t ld, int32_t blocks);

}  // namespace spconv
