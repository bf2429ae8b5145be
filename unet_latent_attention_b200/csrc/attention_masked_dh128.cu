// sd_attention_masked for heads of 72 to 128 columns.
#include "attention_masked_launch.cuh"

sd_status sd::masked::launch_dh128(const Launch& l) {
  return l.args->dtype ? by_score<128, 64, 2, 2, 2, true, true>(l) : by_score<128, 64, 2, 2, 2, true, false>(l);
}
