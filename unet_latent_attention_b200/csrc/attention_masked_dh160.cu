// sd_attention_masked for heads of 136 to 160 columns: one query tile a CTA (two tiles' S and O exceed
// tensor memory), key tiles of 64 keys, three stages of 24 KB each.
#include "attention_masked_launch.cuh"

sd_status sd::masked::launch_dh160(const Launch& l) {
  return l.args->dtype ? by_score<160, 64, 1, 3, 3, true, true, true>(l) : by_score<160, 64, 1, 3, 3, true, true, false>(l);
}
