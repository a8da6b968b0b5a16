// tensor_map.h - TMA tensor maps of q and of K/V rows (tensor_map.cu).
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace pkv {

// q [total_q][Hq][D] bf16 as a 3-D tensor, box {64, g, tpt}.
bool tensor_map_q(CUtensorMap *m, const void *q, uint64_t total_q, uint64_t hq, uint64_t d,
                  uint32_t g, uint32_t tpt);
// `rows` rows of `cols` bf16, boxes of box_rows rows x 64 columns.
bool tensor_map_rows(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols,
                     uint32_t box_rows);

}  // namespace pkv
