// sd_attention_masked for heads of up to 160 columns.
#include "attention_masked_launch.cuh"

sd_status sd::masked::launch_dh160(const Launch& l) {
  return l.args->dtype ? by_score<160, 64, 3, 3, 1, true, true>(l) : by_score<160, 64, 3, 3, 1, true, false>(l);
}
