// Launch of one attention_masked_sm100 configuration and the choice among those of a head size.
#pragma once

#include <algorithm>
#include <atomic>

#include "attention_masked.cuh"
#include "attention_masked.h"

namespace sd {
namespace masked {

constexpr int kMaxSplits = 8;  // CTAs of a portable cluster

template <class C>
sd_status launch(const Launch& l, int pack, int64_t tiles, int splits) {
  const sd_attention_masked_args& a = *l.args;
  const int64_t keys = std::max<int64_t>(a.Lk, 1);  // a tensor map has no empty dimension; without keys nothing is loaded
  CUtensorMap mq, mk, mv;
  sd_status st = make_view_map(&mq, a.q, a.q_stride, a.B, a.Lq, a.heads, a.dh, pack, BM / pack, C::F16);
  if (st == SD_OK) st = make_view_map(&mk, a.k, a.k_stride, a.B, keys, a.kv_heads, a.dh, 1, C::BN, C::F16);
  if (st == SD_OK) st = make_view_map(&mv, a.v, a.v_stride, a.B, keys, a.kv_heads, a.dh, 1, C::BN, C::F16);
  if (st != SD_OK) return st;
  Params p = {};
  p.out = a.o;
  p.v = static_cast<const uint16_t*>(a.v);
  p.bias = a.bias;
  p.kv_lens = a.kv_lens, p.q_starts = a.q_starts, p.prefix_lens = a.prefix_lens;
  p.q_offsets = a.q_offsets, p.k_offsets = a.k_offsets;
  p.o_batch = a.o_stride[0], p.o_token = a.o_stride[1], p.o_head = a.o_stride[2];
  p.v_batch = a.v_stride[0], p.v_token = a.v_stride[1], p.v_head = a.v_stride[2];
  p.heads = static_cast<int>(a.heads), p.group = static_cast<int>(l.group), p.pack = pack;
  while (1 << p.pack_log2 < pack) ++p.pack_log2;
  p.Lq = static_cast<int>(a.Lq), p.Lk = static_cast<int>(a.Lk), p.dh = static_cast<int>(a.dh);
  p.docs = a.q_offsets ? static_cast<int>(a.docs) : 0;
  p.radius = static_cast<int>(a.bias_radius), p.causal = a.causal;
  p.tiles = static_cast<int>(tiles);
  p.planes = static_cast<int>(a.B * (a.heads / pack));
  // Where items differ in length, as many planes are mixed as have 48 MB of keys and values, under half of
  // L2 (causal [2, 10, 4096, 64]: 74 us; beside 77 at the time 106 with one plane after the other).
  const int64_t plane_bytes = std::max<int64_t>(a.Lk * a.dh * 4 * pack / l.group, 1);
  p.plane_group = a.causal || a.q_offsets || a.kv_lens
                      ? static_cast<int>(std::min<int64_t>(std::max<int64_t>((int64_t(48) << 20) / plane_bytes, 1), p.planes))
                      : 1;
  constexpr float kLog2e = 1.4426950408889634f;
  // scale 0: a masked score must not become 0 * -infinity; a scale near fp32's end: 0 must not become 0 * infinity
  p.scale_log2 = std::min(std::max(a.scale * kLog2e, 1.17549435e-38f), 3.402823466e38f);
  p.cap_in = C::CAP ? a.scale / a.cap : 0.f;
  p.cap_out = a.cap * kLog2e;
  if (C::CAP) {
    p.cap_scale = a.scale, p.cap_inv = 1.f / a.cap;
    // The smallest coefficient of the polynomial in q.k, cap k^7 log2(e) / 23, has to keep its 24 bits.
    const float k = p.cap_in, least = std::min(1.f, k * k * k * k * k * k) * p.cap_out * k / 23.f;
    p.cap_raw = least >= 1.17549435e-38f;
  }
  p.err = sd::device_status_word();
  if (!p.err) return SD_ERR_CUDA;

  auto kern = attention_masked_sm100<C>;
  static std::atomic<uint64_t> smem_set{0};  // one bit per device: opt-in to large shared memory done
  int dev = 0;
  st = sd::cuda_check(cudaGetDevice(&dev), "cudaGetDevice");
  if (st != SD_OK) return st;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(smem_set.load(std::memory_order_acquire) & bit)) {
    st = sd::cuda_check(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM),
                        "cudaFuncSetAttribute(attention_masked smem)");
    if (st != SD_OK) return st;
    smem_set.fetch_or(bit, std::memory_order_acq_rel);
  }
  const int64_t ctas = a.B * (a.heads / pack) * tiles * splits;
  if (ctas > 0x7fffffff) return sd::fail(SD_ERR_UNSUPPORTED, "sd_attention_masked: too many query tiles");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = l.stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = sd::pdl_attr(&attr[0]);
  if (splits > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  return sd::cuda_check(cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, p), "sd_attention_masked launch");
}

template <class C>
sd_status choose(const Launch& l) {
  const sd_attention_masked_args& a = *l.args;
  // Heads that share a key head become rows of one tile while that fills tiles better: few queries.
  // (The bias of a row's head would differ within a tile.)
  int pack = 1;
  if (!C::BIAS && a.Lq <= BM / 2 && l.group > 1 && BM % l.group == 0) pack = static_cast<int>(l.group);
  const int64_t planes = a.B * (a.heads / pack), tiles = (a.Lq * pack + BM - 1) / BM;
  // Idle SMs: split the keys over a cluster, two key tiles a CTA at least, while all clusters run at once.
  // (Beyond that the clusters' starts, joins and ends cost more than they even out: B200, [32, 16, 1, 2048
  // ragged, 64] takes 52, 61, 91 and 167 us with 1, 2, 4 and 8 parts; [4, 32 / 8 heads, 1, 16384, 128] 232, 122, 68 and 49;
  // [16, 16 / 4 heads, 1, 8192 ragged, 128] 40 with 4 parts and, beside 39 at the time, 46 with 8.)
  int splits = 1;
  const int64_t key_tiles = (a.Lk + C::BN - 1) / C::BN;
  while (2 * splits <= kMaxSplits && planes * tiles * 2 * splits <= C::CTAS * sd::sm_count() && key_tiles >= 4 * splits) splits *= 2;
  return launch<C>(l, pack, tiles, splits);
}

// KS, VS: stages of K and V; BKS, BVS: beside a bias's windows.
template <int DHT, int BN, int KS, int VS, int CTAS, bool F16, int BKS = KS, int BVS = VS>
sd_status by_score(const Launch& l) {
  const bool cap = l.args->cap != 0.f, bias = l.args->bias != nullptr;
  if (cap && bias) return choose<Cfg<DHT, BN, BKS, BVS, CTAS, F16, true, true>>(l);
  if (cap) return choose<Cfg<DHT, BN, KS, VS, CTAS, F16, true, false>>(l);
  if (bias) return choose<Cfg<DHT, BN, BKS, BVS, CTAS, F16, false, true>>(l);
  return choose<Cfg<DHT, BN, KS, VS, CTAS, F16, false, false>>(l);
}

}  // namespace masked
}  // namespace sd
