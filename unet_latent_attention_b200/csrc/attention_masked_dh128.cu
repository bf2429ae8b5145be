// sd_attention_masked for heads of 72 to 128 columns: with two query tiles P lies over S; two stages
// of 32 KB key and value tiles (three with one query tile, where P has columns of its own).
#include "attention_masked_launch.cuh"

sd_status sd::masked::launch_dh128(const Launch& l) {
  return l.args->dtype ? by_score<128, 128, 2, 2, 2, false, true, true>(l) : by_score<128, 128, 2, 2, 2, false, true, false>(l);
}
