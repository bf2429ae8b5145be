// Host side of sd_attention_masked shared by its translation units.
#pragma once

#include <cuda.h>

#include "sd_internal.h"

namespace sd {
namespace masked {

struct Params;

// What the entry point settles before it picks a kernel.
struct Launch {
  const sd_attention_masked_args* args;
  int64_t group;  // query heads per key head
  cudaStream_t stream;
};

// Kernels for heads of up to 64, 128 and 160 columns, each in a translation unit of its own.
sd_status launch_dh64(const Launch& l);
sd_status launch_dh128(const Launch& l);
sd_status launch_dh160(const Launch& l);

// Tensor map of a [B, L, heads, dh] view of 16-bit values with strides {batch, token, head} in
// elements: dimensions {dh, heads, L, B}, boxes of 64 columns x `box_heads` x `box_rows`, 128-byte
// swizzle. Columns past dh and rows past L read as zero.
sd_status make_view_map(CUtensorMap* map, const void* ptr, const int64_t* stride, int64_t B, int64_t L, int64_t heads,
                        int64_t dh, int box_heads, int box_rows, bool f16);

}  // namespace masked
}  // namespace sd
