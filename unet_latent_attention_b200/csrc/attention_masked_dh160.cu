// sd_attention_masked for heads of 136 to 160 columns: tiles of 64 keys, three stages of 24 KB each, one CTA an
// SM ([2, 4, 4096, 160]: 114 us, and with a fourth stage of V; two CTAs with one stage each 143).
#include "attention_masked_launch.cuh"

sd_status sd::masked::launch_dh160(const Launch& l) {
  return l.args->dtype ? by_score<160, 64, 3, 3, 1, true>(l) : by_score<160, 64, 3, 3, 1, false>(l);
}
