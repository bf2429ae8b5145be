// sd_attention_masked for heads of up to 128 columns.
#include "attention_masked_launch.cuh"

#ifndef V
#define V 1, 1, 2
#define VSEP false
#endif
sd_status sd::masked::launch_dh128(const Launch& l) {
  return l.args->dtype ? by_score<128, 128, V, VSEP, true>(l) : by_score<128, 128, V, VSEP, false>(l);
}
