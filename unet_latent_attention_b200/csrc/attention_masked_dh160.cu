// sd_attention_masked for heads of up to 160 columns.
#include "attention_masked_launch.cuh"

#ifndef V
#define V 1, 1, 2
#define VSEP true
#endif
sd_status sd::masked::launch_dh160(const Launch& l) {
  return l.args->dtype ? by_score<160, 64, V, VSEP, true>(l) : by_score<160, 64, V, VSEP, false>(l);
}
