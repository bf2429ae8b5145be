// sd_attention_masked: argument checks, tensor maps of strided views and the choice of the head size.
#include "attention_masked.h"

#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "attn_common.cuh"

namespace {

struct View {
  const char* name;
  const void* ptr;
  const int64_t* stride;  // batch, token, head, in elements
  int64_t n[3];           // B, L, heads
  int64_t dh;

  int64_t bytes() const {  // from the first element to the end of the last
    int64_t last = dh;
    for (int i = 0; i < 3; ++i) last += (n[i] - 1) * stride[i];
    return last * 2;
  }
};

sd_status check_view(const View& v, bool output) {
  if (!v.ptr) return sd::fail(SD_ERR_INVALID_ARG, "sd_attention_masked: %s is null", v.name);
  if (!sd::aligned16(v.ptr)) return sd::fail(SD_ERR_MISALIGNED, "sd_attention_masked: %s must be 16-byte aligned", v.name);
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 3; ++i) {
    if (v.n[i] <= 1) continue;
    if (v.stride[i] < v.dh || v.stride[i] >= (int64_t(1) << 38))
      return sd::fail(SD_ERR_UNSUPPORTED, "sd_attention_masked: a stride of %s is below dh or >= 2^38", v.name);
    if (v.stride[i] % 8)
      return sd::fail(SD_ERR_MISALIGNED, "sd_attention_masked: the strides of %s must be multiples of 8 elements", v.name);
  }
  if (!output) return SD_OK;
  std::sort(order, order + 3, [&](int i, int j) { return v.stride[i] < v.stride[j]; });
  int64_t span = v.dh;
  for (int i : order) {
    if (v.n[i] <= 1) continue;
    if (v.stride[i] < span) return sd::fail(SD_ERR_INVALID_ARG, "sd_attention_masked: the strides of %s make its heads overlap", v.name);
    span += (v.n[i] - 1) * v.stride[i];
  }
  return SD_OK;
}

}  // namespace

sd_status sd::masked::make_view_map(CUtensorMap* map, const void* ptr, const int64_t* stride, int64_t B, int64_t L,
                                    int64_t heads, int64_t dh, int box_heads, int box_rows, bool f16) {
  auto fn = sd::attn::encode_fn();
  if (!fn) return sd::fail(SD_ERR_CUDA, "sd_attention_masked: cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(dh), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(L),
                              static_cast<cuuint64_t>(B)};
  // The stride of a dimension of one element is never used, but it is checked.
  const auto bytes = [&](int64_t n, int64_t s) { return static_cast<cuuint64_t>((n > 1 ? s : dh) * 2); };
  const cuuint64_t strides[3] = {bytes(heads, stride[2]), bytes(L, stride[1]), bytes(B, stride[0])};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                        const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return sd::fail(SD_ERR_CUDA, "sd_attention_masked: cuTensorMapEncodeTiled failed (%d)", (int)r);
  return SD_OK;
}

extern "C" sd_status sd_attention_masked(const sd_attention_masked_args* args, void* stream) {
  if (!args) return sd::fail(SD_ERR_INVALID_ARG, "sd_attention_masked: null arguments");
  const sd_attention_masked_args& a = *args;
  if (a.B < 0 || a.heads < 0 || a.kv_heads < 0 || a.Lq < 0 || a.Lk < 0)
    return sd::fail(SD_ERR_INVALID_ARG, "sd_attention_masked: negative size");
  if (a.dtype != 0 && a.dtype != 1) return sd::fail(SD_ERR_INVALID_ARG, "sd_attention_masked: dtype must be 0 or 1");
  if (a.causal != 0 && a.causal != 1) return sd::fail(SD_ERR_INVALID_ARG, "sd_attention_masked: causal must be 0 or 1");
  if (a.dh < 8 || a.dh > 160 || a.dh % 8)
    return sd::fail(SD_ERR_UNSUPPORTED, "sd_attention_masked: head dim %lld is not a multiple of 8 from 8 to 160", (long long)a.dh);
  if (!std::isfinite(a.scale) || !std::isfinite(a.cap) || a.cap < 0.f)
    return sd::fail(SD_ERR_INVALID_ARG, "sd_attention_masked: scale must be finite, cap finite and >= 0");
  if (a.scale < 0.f) return sd::fail(SD_ERR_UNSUPPORTED, "sd_attention_masked: negative scale");
  if (a.cap > 0.f) {  // the cap's polynomial has coefficients up to cap * (scale / cap)^7
    const float k = a.scale / a.cap, top = 1.5f * a.cap * k * k * k * k * k * k * k;
    if (!(a.cap >= 1e-6f && a.cap <= 1e30f) || !std::isfinite(k * k * k * k * k * k) || !std::isfinite(top))
      return sd::fail(SD_ERR_UNSUPPORTED, "sd_attention_masked: cap must lie in [1e-6, 1e30], scale / cap below 1e5");
  }
  if (a.bias && (a.bias_radius < 0 || a.bias_radius >= (int64_t(1) << 29)))
    return sd::fail(SD_ERR_INVALID_ARG, "sd_attention_masked: bias_radius must lie in [0, 2^29)");
  if (a.prefix_lens && !a.causal) return sd::fail(SD_ERR_INVALID_ARG, "sd_attention_masked: prefix_lens needs causal");
  if (!a.q_offsets != !a.k_offsets) return sd::fail(SD_ERR_INVALID_ARG, "sd_attention_masked: q_offsets and k_offsets go together");
  if (a.q_offsets) {
    if (a.B != 1 || a.kv_lens)
      return sd::fail(SD_ERR_INVALID_ARG, "sd_attention_masked: packed documents take B = 1 and no kv_lens");
    if (a.docs < 1 || a.docs >= (int64_t(1) << 30))
      return sd::fail(SD_ERR_INVALID_ARG, "sd_attention_masked: docs must lie in [1, 2^30)");
  }
  if (a.B == 0 || a.heads == 0 || a.Lq == 0) return SD_OK;
  if (a.kv_heads == 0 || a.heads % a.kv_heads)
    return sd::fail(SD_ERR_INVALID_ARG, "sd_attention_masked: kv_heads must divide heads");
  if (a.Lq >= (int64_t(1) << 30) || a.Lk >= (int64_t(1) << 30) || a.heads > 65536 || a.B > 0x7fffffff / a.heads)
    return sd::fail(SD_ERR_UNSUPPORTED, "sd_attention_masked: L must be < 2^30, heads <= 65536 and B * heads < 2^31");
  const View q{"q", a.q, a.q_stride, {a.B, a.Lq, a.heads}, a.dh}, o{"o", a.o, a.o_stride, {a.B, a.Lq, a.heads}, a.dh};
  const View k{"k", a.k, a.k_stride, {a.B, a.Lk, a.kv_heads}, a.dh}, v{"v", a.v, a.v_stride, {a.B, a.Lk, a.kv_heads}, a.dh};
  sd_status st = check_view(q, false);
  if (st == SD_OK) st = check_view(o, true);
  if (st == SD_OK && a.Lk) st = check_view(k, false);
  if (st == SD_OK && a.Lk) st = check_view(v, false);
  if (st != SD_OK) return st;
  for (const int32_t* x : {a.kv_lens, a.q_starts, a.prefix_lens, a.q_offsets, a.k_offsets, reinterpret_cast<const int32_t*>(a.bias)})
    if (reinterpret_cast<uintptr_t>(x) % 4) return sd::fail(SD_ERR_MISALIGNED, "sd_attention_masked: an int32 or fp32 array is misaligned");
  for (const View& in : {q, k, v})
    if (in.n[1] && sd::overlaps(o.ptr, o.bytes(), in.ptr, in.bytes()))
      return sd::fail(SD_ERR_INVALID_ARG, "sd_attention_masked: o overlaps %s", in.name);
  sd_attention_masked_args b = a;
  if (a.Lk == 0) {  // no key: nothing is loaded, but a tensor map has no empty dimension and checks its strides
    b.k = b.v = b.q;
    for (int i = 0; i < 3; ++i) b.k_stride[i] = b.v_stride[i] = b.dh;
  }
  sd::masked::Launch l{&b, a.heads / a.kv_heads, static_cast<cudaStream_t>(stream)};
  if (a.dh <= 64) return sd::masked::launch_dh64(l);
  if (a.dh <= 128) return sd::masked::launch_dh128(l);
  return sd::masked::launch_dh160(l);
}
