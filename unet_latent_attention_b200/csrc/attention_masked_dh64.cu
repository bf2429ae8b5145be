// sd_attention_masked for heads of up to 64 columns.
#include "attention_masked_launch.cuh"

sd_status sd::masked::launch_dh64(const Launch& l) {
  return l.args->dtype ? by_score<64, 128, 2, 2, 2, true, true>(l) : by_score<64, 128, 2, 2, 2, true, false>(l);
}
