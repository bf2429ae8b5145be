// sd_attention_masked for heads of 72 to 128 columns: tiles of 64 keys, so that S, P and O fit 256 columns of
// tensor memory and two CTAs an SM: 141 us for [2, 8, 4096, 128]. (Beside 144 at the time, tiles of 128 keys with P
// over S took 161, and one CTA an SM with three stages 159.) V has a third stage where a bias's windows do not need
// the room: a CTA with few queries waits for memory, and 32 KB more on their way to an SM took one token of
// [16, 16 / 4 heads, 8192 ragged, 128] from 43.7 to 39.1 us (a third stage of K instead: 44.0); it is 40.0 now. Full
// tiles take the same time within 1%, and at 64 columns of a head third stages change nothing.
#include "attention_masked_launch.cuh"

sd_status sd::masked::launch_dh128(const Launch& l) {
  return l.args->dtype ? by_score<128, 64, 2, 3, 2, true, 2, 2>(l) : by_score<128, 64, 2, 3, 2, false, 2, 2>(l);
}
