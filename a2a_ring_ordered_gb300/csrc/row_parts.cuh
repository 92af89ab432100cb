// row_parts.cuh -- the part of a rank's rows that a CTA has (RankParts).
#pragma once

#include "device_common.cuh"

namespace ccl {

struct RowPart {
  int r;             // rank
  uint32_t lo, hi;   // its rows lo .. hi - 1
};

__device__ __forceinline__ RowPart row_part(const RankParts& parts, int p, uint32_t cta) {
  int lo = 0, hi = p;  // the last rank whose first part is not behind the CTA: ranks without parts have none
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (parts.first[mid] <= cta) lo = mid;
    else hi = mid;
  }
  const uint64_t n = parts.first[lo + 1] - parts.first[lo], i = cta - parts.first[lo], rows = parts.rows[lo];
  return {lo, static_cast<uint32_t>(rows * i / n), static_cast<uint32_t>(rows * (i + 1) / n)};
}

}  // namespace ccl
