// RMS norm of rows, with the residual's addition before it and an output of the input's type or of
// e4m3 with scales (sd_rms_norm, sd_rms_norm_fp8).
//
//   h = x + residual (fp32),  residual_out = round(h),
//   y = h * rsqrt(mean(h^2) + eps) * w           from the unrounded h, rounded once;
//   e4m3: per block of columns of a row (or the whole row) s = max(max|y| / 448, 2^-126), q = e4m3(y / s).
//
// Bound by HBM: every value is read once and written once, four operations each. So a row stays in
// registers between the statistics and the output: a pack of 16 bytes per load, up to NV packs per
// thread, all loads of a row in flight before the first is used. Narrow rows: one warp per row, whose
// reductions are shuffles and which meets no barrier. Others: one CTA per row, whose warps exchange
// one partial sum each through shared memory. Rows beyond what 512 threads hold (kMaxThreads *
// kMaxPacks packs) are read twice. B200: [32760, 2048] bf16 with residual 80.6 us, 6650 GB/s (a plain
// copy: 6560); [8192, 1280] into e4m3 with blocks of 128 15.8 us, 4670 GB/s, where the instructions of
// the conversion share the time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "rows_common.cuh"
#include "sd_internal.h"

namespace {

using sd::rows::PackOf;

constexpr float kE4m3Max = 448.0f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126: the scale of a block of zeros
constexpr int kMaxThreads = 512;              // 128 registers a thread: a row's packs stay in them
constexpr int kMaxPacks = 8;
constexpr int kWarpRows = 8;                  // rows of a CTA that takes one row per warp

struct RmsArgs {
  const void* x;
  const void* residual;  // or NULL
  const void* weight;    // or NULL (ones)
  void* y;               // T, or e4m3
  void* residual_out;    // or NULL
  float* scales;         // e4m3: [rows, ceil(cols / block)], or [rows] for block = 0
  long long x_stride, residual_stride, y_stride, residual_out_stride;  // elements between rows
  long long rows;
  int cols;
  int block;        // columns with one scale: 32, 64 or 128, or 0: the row
  int block_log2, nblocks;
  float eps, inv_cols;
  int weight_f32;
};

// max that keeps a NaN, so that a block holding one gets a NaN scale.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Over groups of `lanes` neighbouring lanes (a power of two, the same for the whole grid).
__device__ __forceinline__ float lanes_max(float v, int lanes) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    if (o < lanes) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The row's sum of squares and, where it has one scale, its largest magnitude, over all threads that
// share it: the warp, or the CTA's warps with one exchange through shared memory (and one barrier: the
// exchange is used once).
struct Totals {
  float sum, top;
};
template <bool TOP>
__device__ __forceinline__ Totals row_totals(float sum, float top, bool warp_row, float (&part)[2][kMaxThreads / 32]) {
  sum = warp_sum(sum);
  if (TOP) top = lanes_max(top, 32);
  if (warp_row) return {sum, top};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
    part[0][warp] = sum;
    if (TOP) part[1][warp] = top;
  }
  __syncthreads();
  sum = part[0][0];
  if (TOP) top = part[1][0];
  for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) {  // every thread in the same order: broadcasts
    sum += part[0][w];
    if (TOP) top = max_nan(top, part[1][w]);
  }
  return {sum, top};
}

// Column of element e of pack p. VECT: packs are contiguous (one 16-byte access). Otherwise the 32
// packs of a warp's chunk are transposed, so that each scalar access of a warp is contiguous and
// any alignment and width will do.
template <bool VECT, int PACK>
__device__ __forceinline__ int column(int p, int e) {
  if (VECT) return p * PACK + e;
  return (p >> 5) * (32 * PACK) + e * 32 + (p & 31);
}

template <typename T, bool VECT, int PACK>
__device__ __forceinline__ void load_pack(const T* row, int p, int cols, float (&v)[PACK]) {
  if constexpr (VECT) {
    if (p * PACK < cols) {
      sd::rows::load(row + p * PACK, v);
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < PACK; ++e) {
    const int c = column<VECT, PACK>(p, e);
    v[e] = (!VECT && c < cols) ? sd::rows::to_float(row[c]) : 0.f;
  }
}

template <typename T, bool VECT, int PACK>
__device__ __forceinline__ void store_pack(T* row, int p, int cols, const float (&v)[PACK]) {
  if constexpr (VECT) {
    if (p * PACK < cols) sd::rows::store(row + p * PACK, v);
  } else {
#pragma unroll
    for (int e = 0; e < PACK; ++e) {
      const int c = column<VECT, PACK>(p, e);
      if (c < cols) row[c] = sd::rows::from_float<T>(v[e]);
    }
  }
}

// Largest magnitude of the block of each element of a pack. Every lane of the warp takes part (packs
// past the row hold zeros). A block of 32, 64 or 128 columns never leaves a warp's packs.
template <bool VECT, int PACK>
__device__ __forceinline__ void block_tops(int block, const float (&v)[PACK], float (&top)[PACK]) {
  if constexpr (VECT) {  // a block: block / PACK neighbouring lanes
    float m = fabsf(v[0]);
#pragma unroll
    for (int e = 1; e < PACK; ++e) m = max_nan(m, fabsf(v[e]));
    top[0] = lanes_max(m, block / PACK);
  } else {  // a block: elements e .. e + block / 32 of all 32 lanes
    const int per = block / 32;
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < PACK; ++e) {
      m = max_nan(m, fabsf(v[e]));
      if ((e + 1) % per == 0) {
        m = lanes_max(m, 32);
#pragma unroll
        for (int f = 0; f < PACK; ++f)
          if (f <= e && f > e - per) top[f] = m;
        m = 0.f;
      }
    }
  }
}

__device__ __forceinline__ float scale_of(float top, float rstd) {
  return max_nan(top * rstd * (1.0f / kE4m3Max), kMinScale);
}

// e4m3 values of a pack of h * w, and the scales of the blocks that begin in it.
template <bool VECT, int PACK>
__device__ __forceinline__ void store_fp8(const RmsArgs& a, long long row, int p, const float (&hw)[PACK],
                                          const float (&top)[PACK], float rstd) {
  uint8_t* q = static_cast<uint8_t*>(a.y) + row * a.y_stride;
  float* out = a.scales + row * a.nblocks;
  if constexpr (VECT) {
    const float s = scale_of(top[0], rstd), inv = __fdividef(1.0f, s);
    if (p * PACK < a.cols) {
      if (a.block && (p * PACK & (a.block - 1)) == 0) out[p * PACK >> a.block_log2] = s;
      uint32_t w[PACK / 4];
#pragma unroll
      for (int i = 0; i < PACK / 4; ++i)
        w[i] = sd::rows::e4m3x2(hw[4 * i] * rstd * inv, hw[4 * i + 1] * rstd * inv) |
               (sd::rows::e4m3x2(hw[4 * i + 2] * rstd * inv, hw[4 * i + 3] * rstd * inv) << 16);
      if constexpr (PACK == 8) *reinterpret_cast<uint2*>(q + p * PACK) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(q + p * PACK) = w[0];
    }
  } else {
#pragma unroll
    for (int e = 0; e < PACK; ++e) {
      const int c = column<VECT, PACK>(p, e);
      if (c >= a.cols) continue;
      const float s = scale_of(top[e], rstd);
      if (a.block && (c & (a.block - 1)) == 0) out[c >> a.block_log2] = s;
      q[c] = static_cast<uint8_t>(sd::rows::e4m3x2(hw[e] * rstd * __fdividef(1.0f, s), 0.f));
    }
  }
}

// NV > 0: a thread keeps up to NV packs of its row in registers. NV = 0: the row is read again.
template <typename T, bool FP8, bool VECT, int NV>
__global__ void __launch_bounds__(kMaxThreads) rms_norm_kernel(const RmsArgs a, int warp_row) {
  constexpr int PACK = PackOf<T>::N;
  __shared__ float part[2][kMaxThreads / 32];
  sd::grid_dep_wait();
  sd::grid_dep_launch();
  const int row_threads = warp_row ? 32 : blockDim.x;  // threads that share a row
  const int tid = warp_row ? (threadIdx.x & 31) : threadIdx.x;
  const long long row = warp_row ? static_cast<long long>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5)
                                 : static_cast<long long>(blockIdx.x);
  if (row >= a.rows) return;  // whole warps (warp_row), never a CTA that shares a row
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.residual_stride : nullptr;
  T* ro = a.residual_out ? static_cast<T*>(a.residual_out) + row * a.residual_out_stride : nullptr;
  T* y = static_cast<T*>(a.y) + (FP8 ? 0 : row * a.y_stride);

  auto read = [&](int p, float (&h)[PACK]) {
    load_pack<T, VECT, PACK>(x, p, a.cols, h);
    if (r) {
      float t[PACK];
      load_pack<T, VECT, PACK>(r, p, a.cols, t);
#pragma unroll
      for (int e = 0; e < PACK; ++e) h[e] += t[e];
    }
  };
  auto weighted = [&](int p, float (&h)[PACK]) {  // h * w; zeros past the row stay zeros
    if (!a.weight) return;
    float w[PACK];
    if (a.weight_f32) {
      const float* f = static_cast<const float*>(a.weight);
      if constexpr (VECT) {
        if (p * PACK < a.cols) {
#pragma unroll
          for (int e = 0; e < PACK; ++e) w[e] = __ldg(f + p * PACK + e);
        } else {
#pragma unroll
          for (int e = 0; e < PACK; ++e) w[e] = 0.f;
        }
      } else {
        load_pack<float, VECT, PACK>(f, p, a.cols, w);
      }
    } else {
      load_pack<T, VECT, PACK>(static_cast<const T*>(a.weight), p, a.cols, w);
    }
#pragma unroll
    for (int e = 0; e < PACK; ++e) h[e] *= w[e];
  };
  auto rstd_of = [&](float sum) { return rsqrtf(fmaf(sum, a.inv_cols, a.eps)); };

  if constexpr (NV > 0) {
    float h[NV][PACK], top[NV][PACK];
    float ss = 0.f, row_top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) read(i * row_threads + tid, h[i]);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int p = i * row_threads + tid;
#pragma unroll
      for (int e = 0; e < PACK; ++e) ss = fmaf(h[i][e], h[i][e], ss);
      if (ro) store_pack<T, VECT, PACK>(ro, p, a.cols, h[i]);
      // y = (h w) rstd with rstd the same all over the row: the magnitudes' order is that of h w, so
      // the blocks' maxima do not wait for the row's sum.
      weighted(p, h[i]);
      if constexpr (FP8) {
        if (a.block) {
          block_tops<VECT, PACK>(a.block, h[i], top[i]);
        } else {
#pragma unroll
          for (int e = 0; e < PACK; ++e) row_top = max_nan(row_top, fabsf(h[i][e]));
        }
      }
    }
    const bool one_scale = FP8 && a.block == 0;
    const Totals t = one_scale ? row_totals<FP8>(ss, row_top, warp_row, part) : row_totals<false>(ss, 0.f, warp_row, part);
    const float rstd = rstd_of(t.sum);
    if (one_scale && tid == 0) a.scales[row] = scale_of(t.top, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int p = i * row_threads + tid;
      if constexpr (FP8) {
        if (one_scale) {
#pragma unroll
          for (int e = 0; e < PACK; ++e) top[i][e] = t.top;
        }
        store_fp8<VECT, PACK>(a, row, p, h[i], top[i], rstd);
      } else {
#pragma unroll
        for (int e = 0; e < PACK; ++e) h[i][e] *= rstd;
        store_pack<T, VECT, PACK>(y, p, a.cols, h[i]);
      }
    }
  } else {
    const int chunk = row_threads * PACK;  // columns that the row's threads take at a time
    // A thread adds up to 2^19 packs: in fp32 the roundings of equal terms would all point one way (2e-4 at 2^24
    // columns of 1.1), so the packs' sums are added in fp64.
    double packs = 0.0;
    float row_top = 0.f;
    for (int i = 0; static_cast<long long>(i) * chunk < a.cols; ++i) {
      float h[PACK], ss = 0.f;
      read(i * row_threads + tid, h);
#pragma unroll
      for (int e = 0; e < PACK; ++e) ss = fmaf(h[e], h[e], ss);
      packs += ss;
      if (FP8 && a.block == 0) {
        weighted(i * row_threads + tid, h);
#pragma unroll
        for (int e = 0; e < PACK; ++e) row_top = max_nan(row_top, fabsf(h[e]));
      }
    }
    const Totals t = row_totals<FP8>(static_cast<float>(packs), row_top, warp_row, part);
    const float rstd = rstd_of(t.sum);
    if (FP8 && a.block == 0 && tid == 0) a.scales[row] = scale_of(t.top, rstd);
    for (int i = 0; static_cast<long long>(i) * chunk < a.cols; ++i) {
      const int p = i * row_threads + tid;
      float h[PACK];
      read(p, h);
      if (ro) store_pack<T, VECT, PACK>(ro, p, a.cols, h);
      weighted(p, h);
      if constexpr (FP8) {
        float top[PACK];
        if (a.block) {
          block_tops<VECT, PACK>(a.block, h, top);
        } else {
#pragma unroll
          for (int e = 0; e < PACK; ++e) top[e] = t.top;
        }
        store_fp8<VECT, PACK>(a, row, p, h, top, rstd);
      } else {
#pragma unroll
        for (int e = 0; e < PACK; ++e) h[e] *= rstd;
        store_pack<T, VECT, PACK>(y, p, a.cols, h);
      }
    }
  }
}

template <typename T, bool FP8, bool VECT, int NV>
sd_status launch(const RmsArgs& a, int threads, bool warp_row, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const long long per = warp_row ? kWarpRows : 1;
  cfg.gridDim = dim3(static_cast<unsigned>((a.rows + per - 1) / per));
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  cfg.attrs = attr;
  cfg.numAttrs = sd::pdl_attr(&attr[0]);
  return sd::cuda_check(cudaLaunchKernelEx(&cfg, rms_norm_kernel<T, FP8, VECT, NV>, a, warp_row ? 1 : 0),
                        "sd_rms_norm launch");
}

template <typename T, bool FP8, bool VECT>
sd_status dispatch(const RmsArgs& a, cudaStream_t s) {
  constexpr int PACK = PackOf<T>::N;
  const int packs = (a.cols + 32 * PACK - 1) / (32 * PACK) * 32;  // whole warps of packs
  // Threads per row, measured in us (B200, bf16, residual; [rows, cols], e4m3 marked 8):
  //   rows all resident at once: one pack a thread  ([300, 1280] 8: 160 threads 2.5, 96 2.8, a warp 4.1);
  //   else narrow rows: a warp each                 ([8192, 320]: a warp 4.7, 64 threads 9.0; [8192, 640] 8: 7.2, 10.4);
  //   else two packs a thread                       ([32760, 2048]: 128 threads 80.6, 256 92, a warp 103;
  //                                                  [8192, 1280] 8: 96 threads 15.8, 160 18.0, a warp 16.7).
  const bool resident = a.rows * std::min(packs, kMaxThreads) <= 2048LL * sd::sm_count();
  const bool warp_row = !resident && packs <= 96;
  const int one = std::min(packs, kMaxThreads), two = std::min((packs / 2 + 31) / 32 * 32, kMaxThreads);
  const int threads = warp_row ? 32 * kWarpRows : resident ? one : two;
  const int row_threads = warp_row ? 32 : threads, nv = (packs + row_threads - 1) / row_threads;
  if (nv <= 1) return launch<T, FP8, VECT, 1>(a, threads, warp_row, s);
  if (nv <= 2) return launch<T, FP8, VECT, 2>(a, threads, warp_row, s);
  if (nv <= 3) return launch<T, FP8, VECT, 3>(a, threads, warp_row, s);
  if (nv <= kMaxPacks) return launch<T, FP8, VECT, kMaxPacks>(a, threads, warp_row, s);
  return launch<T, FP8, VECT, 0>(a, threads, warp_row, s);
}

sd_status rms_impl(const char* name, RmsArgs a, int64_t rows, int64_t cols, int dtype, int weight_f32, bool fp8,
                   void* stream) {
  if (rows < 0 || cols < 0) return sd::fail(SD_ERR_INVALID_ARG, "%s: negative size", name);
  if (dtype < 0 || dtype > 2) return sd::fail(SD_ERR_INVALID_ARG, "%s: dtype must be 0, 1 or 2", name);
  if (weight_f32 != 0 && weight_f32 != 1) return sd::fail(SD_ERR_INVALID_ARG, "%s: weight_f32 must be 0 or 1", name);
  if (!std::isfinite(a.eps) || a.eps < 0.f) return sd::fail(SD_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", name);
  if (fp8 && a.block != 0 && a.block != 32 && a.block != 64 && a.block != 128)
    return sd::fail(SD_ERR_UNSUPPORTED, "%s: block %d not in {0, 32, 64, 128}", name, a.block);
  if (rows == 0 || cols == 0) return SD_OK;
  if (rows > 0x7fffffff || cols > (int64_t(1) << 30))
    return sd::fail(SD_ERR_UNSUPPORTED, "%s: rows must be < 2^31 and cols <= 2^30", name);
  if (!a.x || !a.y || (fp8 && !a.scales)) return sd::fail(SD_ERR_INVALID_ARG, "%s: null pointer", name);
  if (a.residual_out && !a.residual) return sd::fail(SD_ERR_INVALID_ARG, "%s: residual_out without residual", name);
  const int64_t size = dtype == 2 ? 4 : 2;
  if (a.x_stride < cols || a.y_stride < cols || (a.residual && a.residual_stride < cols) ||
      (a.residual_out && a.residual_out_stride < cols))
    return sd::fail(SD_ERR_INVALID_ARG, "%s: a row stride is smaller than cols", name);
  const int64_t most = (int64_t(1) << 62) / rows / 4;  // no byte offset passes 63 bits
  if (a.x_stride > most || a.y_stride > most || (a.residual && a.residual_stride > most) ||
      (a.residual_out && a.residual_out_stride > most))
    return sd::fail(SD_ERR_UNSUPPORTED, "%s: a row stride is too large", name);
  for (const void* p : {a.x, a.residual, static_cast<const void*>(a.residual_out), fp8 ? nullptr : static_cast<const void*>(a.y)})
    if (reinterpret_cast<uintptr_t>(p) % size) return sd::fail(SD_ERR_MISALIGNED, "%s: a pointer breaks its type's alignment", name);
  if (reinterpret_cast<uintptr_t>(a.scales) % 4 || reinterpret_cast<uintptr_t>(a.weight) % (weight_f32 ? 4 : size))
    return sd::fail(SD_ERR_MISALIGNED, "%s: a pointer breaks its type's alignment", name);

  // Outputs: exactly an input (in place), or apart from every input and from one another.
  using sd::rows::RowSpan;
  const int64_t ysize = fp8 ? 1 : size;
  const RowSpan x{a.x, a.x_stride * size, cols * size}, r{a.residual, a.residual_stride * size, cols * size};
  const RowSpan y{a.y, a.y_stride * ysize, cols * ysize}, ro{a.residual_out, a.residual_out_stride * size, cols * size};
  const int64_t nblocks = a.block ? (cols + a.block - 1) / a.block : 1;
  const RowSpan sc{a.scales, nblocks * 4, nblocks * 4};
  const int64_t wbytes = cols * (weight_f32 ? 4 : size);
  const RowSpan w{a.weight, wbytes, wbytes};
  const RowSpan ins[2] = {x, r};
  for (const RowSpan& in : ins) {
    if (!in.ptr) continue;
    if (sd::rows::overlap(y, in, rows) && (fp8 || !sd::rows::same(y, in)))
      return sd::fail(SD_ERR_INVALID_ARG, "%s: y overlaps an input", name);
    if (a.residual_out && sd::rows::overlap(ro, in, rows) && !sd::rows::same(ro, in))
      return sd::fail(SD_ERR_INVALID_ARG, "%s: residual_out overlaps an input", name);
    if (fp8 && sd::rows::overlap(sc, in, rows)) return sd::fail(SD_ERR_INVALID_ARG, "%s: scales overlap an input", name);
  }
  if (a.residual_out && sd::rows::overlap(ro, y, rows))
    return sd::fail(SD_ERR_INVALID_ARG, "%s: residual_out overlaps y", name);
  if (fp8 && (sd::rows::overlap(sc, y, rows) || (a.residual_out && sd::rows::overlap(sc, ro, rows))))
    return sd::fail(SD_ERR_INVALID_ARG, "%s: scales overlap another output", name);
  if (a.weight)
    for (const RowSpan& out : {y, ro, sc})
      if (out.ptr && sd::overlaps(out.ptr, out.stride * (rows - 1) + out.bytes, a.weight, w.bytes))
        return sd::fail(SD_ERR_INVALID_ARG, "%s: an output overlaps the weight", name);

  a.rows = rows;
  a.cols = static_cast<int>(cols);
  a.weight_f32 = weight_f32;
  a.inv_cols = 1.0f / static_cast<float>(cols);
  a.block_log2 = a.block == 128 ? 7 : a.block == 64 ? 6 : 5;
  a.nblocks = static_cast<int>(nblocks);
  // 16-byte accesses want every row of every tensor to start on one, and whole packs in a row.
  const int64_t pack = 16 / size;
  auto vec = [&](const void* p, int64_t stride, int64_t align) {
    return !p || (reinterpret_cast<uintptr_t>(p) % align == 0 && (stride * (fp8 && p == a.y ? 1 : size)) % align == 0);
  };
  const bool vect = cols % pack == 0 && vec(a.x, a.x_stride, 16) && vec(a.residual, a.residual_stride, 16) &&
                    vec(a.residual_out, a.residual_out_stride, 16) && vec(a.y, a.y_stride, fp8 ? pack : 16) &&
                    (!a.weight || weight_f32 || reinterpret_cast<uintptr_t>(a.weight) % 16 == 0);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto typed = [&](auto t) {
    using T = decltype(t);
    if (fp8) return vect ? dispatch<T, true, true>(a, s) : dispatch<T, true, false>(a, s);
    return vect ? dispatch<T, false, true>(a, s) : dispatch<T, false, false>(a, s);
  };
  if (dtype == 0) return typed(__nv_bfloat16());
  if (dtype == 1) return typed(__half());
  return typed(float());
}

}  // namespace

extern "C" sd_status sd_rms_norm(const void* x, const void* residual, const void* weight, void* y, void* residual_out,
                                 int64_t rows, int64_t cols, int64_t x_stride, int64_t residual_stride,
                                 int64_t y_stride, int64_t residual_out_stride, float eps, int dtype, int weight_f32,
                                 void* stream) {
  RmsArgs a = {};
  a.x = x, a.residual = residual, a.weight = weight, a.y = y, a.residual_out = residual_out;
  a.x_stride = x_stride, a.residual_stride = residual_stride, a.y_stride = y_stride;
  a.residual_out_stride = residual_out_stride, a.eps = eps;
  return rms_impl("sd_rms_norm", a, rows, cols, dtype, weight_f32, false, stream);
}

extern "C" sd_status sd_rms_norm_fp8(const void* x, const void* residual, const void* weight, void* y, float* scales,
                                     void* residual_out, int64_t rows, int64_t cols, int64_t x_stride,
                                     int64_t residual_stride, int64_t y_stride, int64_t residual_out_stride, float eps,
                                     int dtype, int weight_f32, int block, void* stream) {
  RmsArgs a = {};
  a.x = x, a.residual = residual, a.weight = weight, a.y = y, a.residual_out = residual_out, a.scales = scales;
  a.x_stride = x_stride, a.residual_stride = residual_stride, a.y_stride = y_stride;
  a.residual_out_stride = residual_out_stride, a.eps = eps, a.block = block;
  return rms_impl("sd_rms_norm_fp8", a, rows, cols, dtype, weight_f32, true, stream);
}
