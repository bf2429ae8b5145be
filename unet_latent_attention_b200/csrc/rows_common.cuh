// Pieces shared by the row kernels (rms_norm.cu, rope_axes.cu): 16-byte packs of bf16, fp16 or fp32
// values as floats, and the host's checks for tensors whose rows overlap.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

namespace sd {
namespace rows {

// Values in 16 bytes.
template <typename T>
struct PackOf {
  static constexpr int N = 16 / sizeof(T);
};

#ifdef __CUDACC__
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }

template <typename T>
__device__ __forceinline__ T from_float(float v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
  else return __float2bfloat16_rn(v);
}

// Two neighbouring 16-bit values of a 32-bit word.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (std::is_same<T, __half>::value) {
    __half2 h;
    *reinterpret_cast<uint32_t*>(&h) = w;
    return __half22float2(h);
  } else {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (std::is_same<T, __half>::value) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// N contiguous values, N * sizeof(T) = 8 or 16 bytes (aligned to that), or a multiple of 16.
template <typename T, int N>
__device__ __forceinline__ void load(const T* p, float (&v)[N]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 t = reinterpret_cast<const float4*>(p)[i];
      v[4 * i] = t.x, v[4 * i + 1] = t.y, v[4 * i + 2] = t.z, v[4 * i + 3] = t.w;
    }
  } else if constexpr (N == 4) {
    const uint2 t = *reinterpret_cast<const uint2*>(p);
    const float2 a = unpack2<T>(t.x), b = unpack2<T>(t.y);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
  } else {
    static_assert(sizeof(T) == 4 || N == 8, "16-bit packs hold 4 or 8 values");
    const uint4 t = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = unpack2<T>(w[i]);
      v[2 * i] = a.x, v[2 * i + 1] = a.y;
    }
  }
}

template <typename T, int N>
__device__ __forceinline__ void store(T* p, const float (&v)[N]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else if constexpr (N == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]),
                                              pack2<T>(v[6], v[7]));
  }
}

// Two e4m3 values (round to nearest even, magnitudes above 448 become 448, NaN stays), lo in bits 0-7.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
#endif

// `rows` rows of `bytes` bytes each, `stride` bytes apart.
struct RowSpan {
  const void* ptr;
  int64_t stride, bytes;
};

inline bool same(const RowSpan& a, const RowSpan& b) { return a.ptr == b.ptr && a.stride == b.stride; }

// True if any row of a meets any row of b. Exact for equal strides (column slices of one buffer are
// apart); else by the whole extents.
inline bool overlap(const RowSpan& a, const RowSpan& b, int64_t rows) {
  if (!a.ptr || !b.ptr) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.ptr), pb = reinterpret_cast<uintptr_t>(b.ptr);
  const uintptr_t ea = pa + static_cast<uintptr_t>(a.stride) * (rows - 1) + a.bytes;
  const uintptr_t eb = pb + static_cast<uintptr_t>(b.stride) * (rows - 1) + b.bytes;
  if (pa >= eb || pb >= ea) return false;
  if (a.stride != b.stride || a.stride <= 0) return true;
  const int64_t d = pb >= pa ? static_cast<int64_t>((pb - pa) % a.stride)
                             : (a.stride - static_cast<int64_t>((pa - pb) % a.stride)) % a.stride;
  return d < a.bytes || d > a.stride - b.bytes;
}

}  // namespace rows
}  // namespace sd
