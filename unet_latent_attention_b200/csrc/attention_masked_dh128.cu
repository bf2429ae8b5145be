// sd_attention_masked for heads of 72 to 128 columns: tiles of 64 keys, so that S, P and O fit 256 columns of
// tensor memory and two CTAs an SM ([2, 8, 4096, 128]: 144 us; tiles of 128 keys with P over S 161, with one CTA
// an SM and three stages 159).
#include "attention_masked_launch.cuh"

sd_status sd::masked::launch_dh128(const Launch& l) {
  return l.args->dtype ? by_score<128, 64, 2, 2, 2, true>(l) : by_score<128, 64, 2, 2, 2, false>(l);
}
