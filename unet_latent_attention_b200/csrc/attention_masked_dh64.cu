// sd_attention_masked for heads of up to 64 columns: S, P and O of two query tiles side by side fill
// tensor memory; four stages of 16 KB key and value tiles.
#include "attention_masked_launch.cuh"

sd_status sd::masked::launch_dh64(const Launch& l) {
  return l.args->dtype ? by_score<64, 128, 2, 4, 6, true, true, true>(l) : by_score<64, 128, 2, 4, 6, true, true, false>(l);
}
