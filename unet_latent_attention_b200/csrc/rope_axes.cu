// Rotary positions with several axes for q and k, with the RMS norm of their heads before it
// (sd_rope_axes).
//
//   y = x                                     (no weight)      over the head's dh columns
//   y = x * rsqrt(mean(x^2) + eps) * w        (with a weight)
//   pair m of axis a turns by angle = 2 pi * turns,  turns = position[token, a] * freq[m] * 2^-64:
//   (u, v) -> (u cos - v sin, u sin + v cos)
//
// The frequency is a 64-bit fraction of a turn per position, and the product is taken modulo 2^64,
// that is modulo whole turns: the fraction of a turn is exact at every 32-bit position, where a
// product in fp32 is a radian off at positions of 10^7. Its upper 32 bits go to sincospi in fp32.
//
// Bound by HBM: q and k are read once and written once. A team of lanes holds one head of one token,
// eight columns (four pairs) a lane, in registers; the four sines and cosines of a lane are formed
// once per token and serve HEADS heads of q and k (at one head a thread the sine work alone would
// take longer than the transfer), whose loads are all in flight together.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "rows_common.cuh"
#include "sd_internal.h"

namespace {

constexpr int kThreads = 256;
constexpr int kMaxAxes = 4;

struct RopeTensor {
  const void* in;
  void* out;
  const float* weight;                 // or NULL: no norm
  long long in_batch, in_token, in_head;   // strides in elements
  long long out_batch, out_token, out_head;
};

struct RopeKernelArgs {
  RopeTensor q, k;
  const int32_t* positions;            // [B, L, axes], or [L, axes] (pos_batch = 0)
  const unsigned long long* freqs;     // [rot / 2]
  long long pos_batch;
  unsigned int L, teams, groups;       // groups: head groups of a token
  int heads, kv_heads, dh, rot, axes;
  int axis_end[kMaxAxes];              // pairs before the end of each axis
  float eps;
};

// LANES: lanes of a team, a power of two >= dh / 8. HEADS: heads a team takes, one after another.
template <typename T, bool HALF, int LANES, int HEADS>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeKernelArgs a) {
  sd::grid_dep_wait();
  sd::grid_dep_launch();
  const unsigned int team = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  const int u = threadIdx.x % LANES;  // this lane's eight columns
  const bool live = team < a.teams;   // every lane stays for the shuffles
  const unsigned int token = live ? team / a.groups : 0, group = live ? team % a.groups : 0;
  const unsigned int b = token / a.L, t = token % a.L;
  const int half = a.rot / 2;
  const bool holds = live && u < a.dh / 8, turns = holds && u < a.rot / 8;
  // columns of the lane's first and second four values
  const bool split = HALF && turns;
  const int c0 = split ? 4 * u : 8 * u, c1 = split ? half + 4 * u : 8 * u + 4;

  // Loads first: the angles are formed while they are on their way.
  float v[HEADS][8];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int h = static_cast<int>(group + i * a.groups);  // neighbouring teams take neighbouring heads
    const bool is_q = h < a.heads;
    if (holds && h < a.heads + a.kv_heads) {
      const RopeTensor& x = is_q ? a.q : a.k;
      const T* p = static_cast<const T*>(x.in) + b * x.in_batch + t * x.in_token + (is_q ? h : h - a.heads) * x.in_head;
      if constexpr (HALF) {
        float lo[4], hi[4];
        sd::rows::load(p + c0, lo);
        sd::rows::load(p + c1, hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] = lo[e], v[i][4 + e] = hi[e];
      } else {
        sd::rows::load(p + c0, v[i]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    }
  }

  float cs[4], sn[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) cs[e] = 1.f, sn[e] = 0.f;
  if (turns) {
    const int32_t* pos = a.positions + b * a.pos_batch + static_cast<long long>(t) * a.axes;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int m = 4 * u + e;
      int axis = 0;
#pragma unroll
      for (int i = 0; i + 1 < kMaxAxes; ++i) axis += (i + 1 < a.axes && m >= a.axis_end[i]) ? 1 : 0;
      const unsigned long long f = __ldg(a.freqs + m);
      const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(__ldg(pos + axis))) * f;
      // the upper 32 bits as a signed fraction: half turns in [-1, 1)
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f, &sn[e], &cs[e]);
    }
  }

#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int h = static_cast<int>(group + i * a.groups);
    const bool is_q = h < a.heads, there = holds && h < a.heads + a.kv_heads;
    const RopeTensor& x = is_q ? a.q : a.k;
    if (a.q.weight || a.k.weight) {  // the same for the whole grid: every lane takes part in the sum
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
#pragma unroll
      for (int o = LANES / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (there && x.weight) {
        const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.dh) + a.eps);
        const float4 w0 = *reinterpret_cast<const float4*>(x.weight + c0);
        const float4 w1 = *reinterpret_cast<const float4*>(x.weight + c1);
        v[i][0] *= rstd * w0.x, v[i][1] *= rstd * w0.y, v[i][2] *= rstd * w0.z, v[i][3] *= rstd * w0.w;
        v[i][4] *= rstd * w1.x, v[i][5] *= rstd * w1.y, v[i][6] *= rstd * w1.z, v[i][7] *= rstd * w1.w;
      }
    }
    if (!there) continue;
    float r[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p0 = split ? e : 2 * e, p1 = split ? 4 + e : 2 * e + 1;
      const float x0 = HALF ? (split ? v[i][e] : v[i][2 * e]) : v[i][2 * e];
      const float x1 = HALF ? (split ? v[i][4 + e] : v[i][2 * e + 1]) : v[i][2 * e + 1];
      const float y0 = fmaf(x0, cs[e], -x1 * sn[e]), y1 = fmaf(x0, sn[e], x1 * cs[e]);
      if (HALF) {
        if (split) r[e] = y0, r[4 + e] = y1;
        else r[2 * e] = y0, r[2 * e + 1] = y1;
      } else {
        r[p0] = y0, r[p1] = y1;
      }
    }
    if (!turns) {  // columns behind the rotated ones pass (an infinity must not meet a zero sine)
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = v[i][e];
    }
    T* p = static_cast<T*>(x.out) + b * x.out_batch + t * x.out_token + (is_q ? h : h - a.heads) * x.out_head;
    if constexpr (HALF) {
      const float lo[4] = {r[0], r[1], r[2], r[3]}, hi[4] = {r[4], r[5], r[6], r[7]};
      sd::rows::store(p + c0, lo);
      sd::rows::store(p + c1, hi);
    } else {
      sd::rows::store(p + c0, r);
    }
  }
}

template <typename T, bool HALF, int LANES, int HEADS>
sd_status launch(RopeKernelArgs a, int64_t tokens, cudaStream_t s) {
  a.groups = static_cast<unsigned>((a.heads + a.kv_heads + HEADS - 1) / HEADS);
  const int64_t teams = tokens * a.groups;
  const int64_t blocks = (teams + kThreads / LANES - 1) / (kThreads / LANES);
  if (teams > 0xffffffffLL - kThreads || blocks > 0x7fffffff)
    return sd::fail(SD_ERR_UNSUPPORTED, "sd_rope_axes: too many heads and tokens");
  a.teams = static_cast<unsigned>(teams);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  cfg.attrs = attr;
  cfg.numAttrs = sd::pdl_attr(&attr[0]);
  return sd::cuda_check(cudaLaunchKernelEx(&cfg, rope_kernel<T, HALF, LANES, HEADS>, a), "sd_rope_axes launch");
}

template <typename T, bool HALF, int LANES>
sd_status by_heads(const RopeKernelArgs& a, int64_t tokens, cudaStream_t s) {
  // Four heads a thread once that still leaves every SM its 2048 threads; below, one: the call is
  // then as long as one thread's chain of loads and stores.
  const int64_t threads = tokens * (a.heads + a.kv_heads) * LANES;
  return threads >= 4LL * 2048 * sd::sm_count() ? launch<T, HALF, LANES, 4>(a, tokens, s)
                                                : launch<T, HALF, LANES, 1>(a, tokens, s);
}

template <typename T, bool HALF>
sd_status by_lanes(const RopeKernelArgs& a, int64_t tokens, cudaStream_t s) {
  const int units = a.dh / 8;
  if (units <= 2) return by_heads<T, HALF, 2>(a, tokens, s);
  if (units <= 4) return by_heads<T, HALF, 4>(a, tokens, s);
  if (units <= 8) return by_heads<T, HALF, 8>(a, tokens, s);
  if (units <= 16) return by_heads<T, HALF, 16>(a, tokens, s);
  return by_heads<T, HALF, 32>(a, tokens, s);
}

// A [B, L, heads, dh] view: dh contiguous columns at every (batch, token, head).
struct View {
  const void* ptr;
  const int64_t* stride;  // batch, token, head, in elements
  int64_t n[3];           // B, L, heads
  int64_t dh, size;

  int64_t bytes() const {  // from the first element to the end of the last
    int64_t last = dh;
    for (int i = 0; i < 3; ++i) last += (n[i] - 1) * stride[i];
    return last * size;
  }
  // One row per token, if the tokens of all batches are equally far apart.
  bool as_rows(sd::rows::RowSpan* r) const {
    if (n[0] > 1 && stride[0] != n[1] * stride[1]) return false;
    *r = {ptr, (n[1] > 1 ? stride[1] : stride[0]) * size, ((n[2] - 1) * stride[2] + dh) * size};
    return n[0] * n[1] > 1 && r->stride >= r->bytes;
  }
  // Whether two of its heads share an element.
  bool folds() const {
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int i, int j) { return stride[i] < stride[j]; });
    int64_t span = dh;
    for (int i : order) {
      if (n[i] <= 1) continue;
      if (stride[i] < span) return true;
      span += (n[i] - 1) * stride[i];
    }
    return false;
  }
};

// Views with the rows of one buffer (a fused projection's q and k) are compared row by row, others
// by their extents.
bool meet(const View& a, const View& b) {
  sd::rows::RowSpan ra, rb;
  if (a.as_rows(&ra) && b.as_rows(&rb) && ra.stride == rb.stride) return sd::rows::overlap(ra, rb, a.n[0] * a.n[1]);
  return sd::overlaps(a.ptr, a.bytes(), b.ptr, b.bytes());
}

sd_status check_view(const char* name, const View& v, bool output) {
  if (!v.ptr) return sd::fail(SD_ERR_INVALID_ARG, "sd_rope_axes: %s is null", name);
  for (int i = 0; i < 3; ++i) {
    if (v.stride[i] < 0 || v.stride[i] >= (int64_t(1) << 40))
      return sd::fail(SD_ERR_UNSUPPORTED, "sd_rope_axes: a stride of %s is negative or >= 2^40", name);
    if (v.n[i] > 1 && v.stride[i] * v.size % 16)
      return sd::fail(SD_ERR_MISALIGNED, "sd_rope_axes: the strides of %s must be multiples of 16 bytes", name);
  }
  if (!sd::aligned16(v.ptr)) return sd::fail(SD_ERR_MISALIGNED, "sd_rope_axes: %s must be 16-byte aligned", name);
  if (output && v.folds()) return sd::fail(SD_ERR_INVALID_ARG, "sd_rope_axes: the strides of %s make its heads overlap", name);
  return SD_OK;
}

}  // namespace

extern "C" sd_status sd_rope_axes(const sd_rope_args* p, void* stream) {
  if (!p) return sd::fail(SD_ERR_INVALID_ARG, "sd_rope_axes: null arguments");
  const sd_rope_args& g = *p;
  if (g.B < 0 || g.L < 0 || g.heads < 0 || g.kv_heads < 0) return sd::fail(SD_ERR_INVALID_ARG, "sd_rope_axes: negative size");
  if (g.dtype < 0 || g.dtype > 2) return sd::fail(SD_ERR_INVALID_ARG, "sd_rope_axes: dtype must be 0, 1 or 2");
  if (g.pairs != 0 && g.pairs != 1) return sd::fail(SD_ERR_INVALID_ARG, "sd_rope_axes: pairs must be 0 or 1");
  if (g.dh < 8 || g.dh > 256 || g.dh % 8)
    return sd::fail(SD_ERR_UNSUPPORTED, "sd_rope_axes: head dim %lld is not a multiple of 8 from 8 to 256", (long long)g.dh);
  if (g.axes < 1 || g.axes > kMaxAxes) return sd::fail(SD_ERR_UNSUPPORTED, "sd_rope_axes: 1 to 4 axes");
  int64_t rot = 0;
  RopeKernelArgs a = {};
  for (int i = 0; i < g.axes; ++i) {
    if (g.axis_dims[i] < 0 || g.axis_dims[i] % 2 || g.axis_dims[i] > g.dh)
      return sd::fail(SD_ERR_INVALID_ARG, "sd_rope_axes: an axis has an odd or negative number of columns, or more than dh");
    rot += g.axis_dims[i];
    a.axis_end[i] = static_cast<int>(rot / 2);
  }
  if (rot > g.dh) return sd::fail(SD_ERR_INVALID_ARG, "sd_rope_axes: the axes have more columns than the head");
  if (rot % 8) return sd::fail(SD_ERR_UNSUPPORTED, "sd_rope_axes: the axes' columns must add up to a multiple of 8");
  if (!std::isfinite(g.eps) || g.eps < 0.f) return sd::fail(SD_ERR_INVALID_ARG, "sd_rope_axes: eps must be finite and >= 0");
  if (g.B == 0 || g.L == 0 || g.heads + g.kv_heads == 0) return SD_OK;
  if (g.B > 0x7fffffff || g.L > 0x7fffffff || g.heads > 65536 || g.kv_heads > 65536 || g.B * g.L > 0x7fffffff)
    return sd::fail(SD_ERR_UNSUPPORTED, "sd_rope_axes: B * L must be < 2^31 and heads <= 65536");
  const int64_t size = g.dtype == 2 ? 4 : 2;
  if (!g.positions || (rot && !g.freqs)) return sd::fail(SD_ERR_INVALID_ARG, "sd_rope_axes: null pointer");
  if (g.positions_batch_stride != 0 && g.positions_batch_stride < g.L * g.axes)
    return sd::fail(SD_ERR_INVALID_ARG, "sd_rope_axes: the batch stride of the positions must be 0 or at least L * axes");
  if (reinterpret_cast<uintptr_t>(g.positions) % 4 || reinterpret_cast<uintptr_t>(g.freqs) % 8 ||
      !sd::aligned16(g.q_weight) || !sd::aligned16(g.k_weight))
    return sd::fail(SD_ERR_MISALIGNED, "sd_rope_axes: positions, freqs or a weight (16 bytes) is misaligned");
  auto view = [&](const void* ptr, const int64_t* stride, int64_t heads) {
    return View{ptr, stride, {g.B, g.L, heads}, g.dh, size};
  };
  const View in[2] = {view(g.q, g.q_stride, g.heads), view(g.k, g.k_stride, g.kv_heads)};
  const View out[2] = {view(g.q_out, g.q_out_stride, g.heads), view(g.k_out, g.k_out_stride, g.kv_heads)};
  const char *const in_name[2] = {"q", "k"}, *const out_name[2] = {"q_out", "k_out"};
  bool in_place[2] = {false, false};
  for (int i = 0; i < 2; ++i) {
    if (out[i].n[2] == 0) continue;
    sd_status st = check_view(in_name[i], in[i], false);
    if (st == SD_OK) st = check_view(out_name[i], out[i], true);
    if (st != SD_OK) return st;
    in_place[i] = in[i].ptr == out[i].ptr;
    for (int d = 0; d < 3; ++d)
      if (in_place[i] && out[i].n[d] > 1 && in[i].stride[d] != out[i].stride[d])
        return sd::fail(SD_ERR_INVALID_ARG, "sd_rope_axes: %s lies on its input with other strides", out_name[i]);
  }
  // An output is its own input exactly (in place), or apart from both inputs and the other output.
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      if (out[i].n[2] && in[j].n[2] && !(i == j && in_place[i]) && meet(out[i], in[j]))
        return sd::fail(SD_ERR_INVALID_ARG, "sd_rope_axes: %s overlaps %s", out_name[i], in_name[j]);
  if (out[0].n[2] && out[1].n[2] && meet(out[0], out[1]))
    return sd::fail(SD_ERR_INVALID_ARG, "sd_rope_axes: q_out overlaps k_out");

  auto fill = [](RopeTensor& r, const void* in, void* out, const float* w, const int64_t* is, const int64_t* os) {
    r.in = in, r.out = out, r.weight = w;
    r.in_batch = is[0], r.in_token = is[1], r.in_head = is[2];
    r.out_batch = os[0], r.out_token = os[1], r.out_head = os[2];
  };
  fill(a.q, g.q, g.q_out, g.q_weight, g.q_stride, g.q_out_stride);
  fill(a.k, g.k, g.k_out, g.k_weight, g.k_stride, g.k_out_stride);
  a.positions = g.positions;
  a.freqs = reinterpret_cast<const unsigned long long*>(g.freqs);
  a.pos_batch = g.positions_batch_stride;
  a.L = static_cast<unsigned>(g.L);
  a.heads = static_cast<int>(g.heads), a.kv_heads = static_cast<int>(g.kv_heads);
  a.dh = static_cast<int>(g.dh), a.rot = static_cast<int>(rot), a.axes = g.axes;
  a.eps = g.eps;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t tokens = g.B * g.L;
  auto typed = [&](auto v) {
    using T = decltype(v);
    return g.pairs ? by_lanes<T, true>(a, tokens, s) : by_lanes<T, false>(a, tokens, s);
  };
  if (g.dtype == 0) return typed(__nv_bfloat16());
  if (g.dtype == 1) return typed(__half());
  return typed(float());
}
