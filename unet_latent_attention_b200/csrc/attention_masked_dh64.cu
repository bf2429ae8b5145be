// sd_attention_masked for heads of up to 64 columns: tiles of 128 keys, two stages of 16 KB each for keys and
// values, S, P and O in 256 columns of tensor memory, two CTAs an SM: 146 us for [2, 10, 4096, 64]. (Beside 152 at the
// time, tiles of 64 keys took 179, and with three and four CTAs an SM 202 and 205.)
#include "attention_masked_launch.cuh"

sd_status sd::masked::launch_dh64(const Launch& l) {
  return l.args->dtype ? by_score<64, 128, 2, 2, 2, true>(l) : by_score<64, 128, 2, 2, 2, false>(l);
}
