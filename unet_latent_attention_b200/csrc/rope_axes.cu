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
// Bound by HBM: q and k are read once and written once. A CTA forms the sines and cosines of its
// tokens once, one pair a thread, multiplies them with the weights and leaves them in shared memory as
// four coefficients a pair; with them a pair of any head is turned in four operations. (Formed by each
// head's threads for themselves they cost more than the transfer: 187 us at one head a thread against
// 88 us for [1, 32760, 16 + 16, 128] bf16 with norm, 6130 GB/s; a plain copy reaches 6560.) A team of
// lanes holds one head of one token at a time, eight columns (four pairs) a lane, in registers; the
// loads of up to four heads are in flight together, the first of them while the sines are formed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

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
  unsigned int L, tokens, all_tokens;  // tokens of a CTA; B * L
  int teams, q_teams;                  // teams of a token; those that take q's heads
  int batches, k_batches;              // batches of heads that a team takes; of k, where it takes both
  int heads, kv_heads, dh, rot, axes;
  int axis_end[kMaxAxes];              // pairs before the end of each axis
  float eps, inv_dh;
  int norms;                           // whether q or k has a weight
};

// The 16 bytes (two times 16 for fp32) of a lane's eight columns, as they lie in memory.
template <typename T, bool HALF>
struct Raw {
  static constexpr int WORDS = sizeof(T) == 4 ? 8 : 4;
  uint32_t w[WORDS];

  __device__ __forceinline__ void load(const T* p, int c0, int c1) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p + c0);
      *reinterpret_cast<uint4*>(w + 4) = *reinterpret_cast<const uint4*>(p + c1);
    } else if constexpr (HALF) {
      *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p + c0);
      *reinterpret_cast<uint2*>(w + 2) = *reinterpret_cast<const uint2*>(p + c1);
    } else {
      *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p + c0);
    }
  }
  // First (x) and second (y) values of the pairs: x[i] holds those of pairs 2i and 2i + 1, for packed
  // arithmetic. Where the lane's columns do not turn, value i of the first (second) four is the same
  // slot of x (y).
  __device__ __forceinline__ void get(float2 (&x)[2], float2 (&y)[2]) const {
    if constexpr (sizeof(T) == 4) {
      const float f[8] = {__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3]),
                          __uint_as_float(w[4]), __uint_as_float(w[5]), __uint_as_float(w[6]), __uint_as_float(w[7])};
      if constexpr (HALF) {
        x[0] = make_float2(f[0], f[1]), x[1] = make_float2(f[2], f[3]);
        y[0] = make_float2(f[4], f[5]), y[1] = make_float2(f[6], f[7]);
      } else {
        x[0] = make_float2(f[0], f[2]), x[1] = make_float2(f[4], f[6]);
        y[0] = make_float2(f[1], f[3]), y[1] = make_float2(f[5], f[7]);
      }
    } else {
      const float2 a = sd::rows::unpack2<T>(w[0]), b = sd::rows::unpack2<T>(w[1]), c = sd::rows::unpack2<T>(w[2]),
                   d = sd::rows::unpack2<T>(w[3]);
      if constexpr (HALF) {
        x[0] = a, x[1] = b, y[0] = c, y[1] = d;
      } else {
        x[0] = make_float2(a.x, b.x), x[1] = make_float2(c.x, d.x);
        y[0] = make_float2(a.y, b.y), y[1] = make_float2(c.y, d.y);
      }
    }
  }
  __device__ __forceinline__ static void store(T* p, int c0, int c1, const float2 (&x)[2], const float2 (&y)[2]) {
    if constexpr (HALF) {
      const float lo[4] = {x[0].x, x[0].y, x[1].x, x[1].y}, hi[4] = {y[0].x, y[0].y, y[1].x, y[1].y};
      sd::rows::store(p + c0, lo);
      sd::rows::store(p + c1, hi);
    } else {
      const float v[8] = {x[0].x, y[0].x, x[0].y, y[0].y, x[1].x, y[1].x, x[1].y, y[1].y};
      sd::rows::store(p + c0, v);
    }
  }
};

// The heads of one tensor that a team turns: first, first + step, ... below heads. The lane's
// coefficients of its four pairs are c[e] = (w0 cos, w0 sin, w1 cos, -w1 sin).
template <typename T, bool HALF, int LANES, bool NORM, int kBatch>
struct Rows {
  const T* in;
  T* out;
  long long in_step, out_step;
  int left;  // heads still to come, the same for all lanes of a warp's teams or less
  bool holds, turns, norm;
  int c0, c1;
  Raw<T, HALF> raw[kBatch];

  __device__ __forceinline__ void init(const RopeTensor& x, bool there, unsigned int b, unsigned int t, int first, int step,
                                       int heads) {
    in = static_cast<const T*>(x.in) + b * x.in_batch + t * x.in_token + first * x.in_head;
    out = static_cast<T*>(x.out) + b * x.out_batch + t * x.out_token + first * x.out_head;
    in_step = step * x.in_head, out_step = step * x.out_head;
    left = there ? (heads - first + step - 1) / step : 0;
    norm = NORM && x.weight != nullptr;
  }
  __device__ __forceinline__ void load() {  // the next batch
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (holds && i < left) {
        raw[i].load(in, c0, c1);
      } else {
#pragma unroll
        for (int e = 0; e < Raw<T, HALF>::WORDS; ++e) raw[i].w[e] = 0;
      }
      in += in_step;
    }
  }
  __device__ __forceinline__ void turn(const RopeKernelArgs& a, const float4 (&c)[4]) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      float2 vx[2], vy[2];
      raw[i].get(vx, vy);
      float x[4] = {vx[0].x, vx[0].y, vx[1].x, vx[1].y}, y[4] = {vy[0].x, vy[0].y, vy[1].x, vy[1].y};
      float rstd = 1.f;
      if constexpr (NORM) {  // every lane takes part in the sum
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (norm) rstd = rsqrtf(fmaf(ss, a.inv_dh, a.eps));
      }
      if (holds && i < left) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float p, q;
          if (turns) {
            p = fmaf(x[e], c[e].x, y[e] * c[e].w);
            q = fmaf(x[e], c[e].y, y[e] * c[e].z);
          } else {  // columns behind the rotated ones (an infinity must not meet a zero sine)
            p = x[e] * c[e].x;
            q = y[e] * c[e].z;
          }
          x[e] = NORM ? p * rstd : p;
          y[e] = NORM ? q * rstd : q;
        }
        const float2 rx[2] = {{x[0], x[1]}, {x[2], x[3]}}, ry[2] = {{y[0], y[1]}, {y[2], y[3]}};
        Raw<T, HALF>::store(out, c0, c1, rx, ry);
      }
      out += out_step;
    }
    left -= kBatch;
  }
};

// LANES: lanes of a team, a power of two >= dh / 8. NORM: whether q or k has a weight. A CTA turns all
// heads of a.tokens tokens, a.teams teams to a token: each takes some of q's and some of k's (BOTH), or
// a.q_teams of them take q's heads and the others k's.
template <typename T, bool HALF, int LANES, bool NORM, int kBatch, bool BOTH>
__global__ void __launch_bounds__(kThreads, !BOTH || sizeof(T) == 4 ? 1 : HALF ? 3 : 4) rope_kernel(const __grid_constant__ RopeKernelArgs a) {
  extern __shared__ float4 coef[];  // [q, k if NORM][tokens][4][LANES]
  sd::grid_dep_wait();
  sd::grid_dep_launch();
  const int u = threadIdx.x % LANES, team = threadIdx.x / LANES;
  const int slot = team / a.teams, j = team % a.teams;  // this team's token of the CTA, and its place there
  const unsigned int token = blockIdx.x * a.tokens + slot;
  const bool there = slot < static_cast<int>(a.tokens) && token < a.all_tokens;
  const unsigned int b = there ? token / a.L : 0, t = there ? token % a.L : 0;
  Rows<T, HALF, LANES, NORM, kBatch> rows;
  rows.holds = u < a.dh / 8;
  rows.turns = u < a.rot / 8;
  // columns of the lane's first and second four values in memory
  const bool split = HALF && rows.turns;
  rows.c0 = split ? 4 * u : 8 * u, rows.c1 = split ? a.rot / 2 + 4 * u : 8 * u + 4;
  const bool on_k = !BOTH && j >= a.q_teams;
  if (on_k) rows.init(a.k, there && j - a.q_teams < a.kv_heads, b, t, j - a.q_teams, a.teams - a.q_teams, a.kv_heads);
  else rows.init(a.q, there && j < a.heads, b, t, j, a.q_teams, a.heads);
  rows.load();  // on its way while the coefficients are formed

  for (int i = threadIdx.x; i < static_cast<int>(a.tokens) * 4 * LANES; i += kThreads) {
    const int lane = i % LANES, e = i / LANES % 4, k = i / (4 * LANES);  // pair 4 * lane + e of token k
    const unsigned int tok = blockIdx.x * a.tokens + k;
    if (lane >= a.dh / 8 || tok >= a.all_tokens) continue;
    float s = 0.f, c = 1.f;
    const int m = 4 * lane + e;
    const bool pair = lane < a.rot / 8;
    if (pair) {
      int axis = 0;
#pragma unroll
      for (int n = 0; n + 1 < kMaxAxes; ++n) axis += (n + 1 < a.axes && m >= a.axis_end[n]) ? 1 : 0;
      const unsigned int tb = tok / a.L, tt = tok % a.L;
      const int p = __ldg(a.positions + tb * a.pos_batch + static_cast<long long>(tt) * a.axes + axis);
      const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(p)) * __ldg(a.freqs + m);
      // the upper 32 bits as a signed fraction: half turns in [-1, 1)
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f, &s, &c);
    }
    if constexpr (NORM) {
      // columns of the pair's two values; behind the rotated ones, of the slots of x and y (see Raw)
      const int m0 = HALF ? (pair ? m : 8 * lane + e) : 2 * m, m1 = HALF ? (pair ? m + a.rot / 2 : 8 * lane + 4 + e) : 2 * m + 1;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float* w = n ? a.k.weight : a.q.weight;
        const float w0 = w ? __ldg(w + m0) : 1.f, w1 = w ? __ldg(w + m1) : 1.f;
        coef[((n * a.tokens + k) * 4 + e) * LANES + lane] = make_float4(w0 * c, w0 * s, w1 * c, -w1 * s);
      }
    } else {
      coef[(k * 4 + e) * LANES + lane] = make_float4(c, s, c, -s);
    }
  }
  __syncthreads();

  float4 c[4];
  const float4* mine = coef + (there ? slot : 0) * 4 * LANES + u;
  const int k_coef = NORM ? a.tokens * 4 * LANES : 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] = mine[(on_k ? k_coef : 0) + e * LANES];
  for (int n = 0; n < a.batches; ++n) {  // the same number for every warp of the grid
    if (n) rows.load();
    rows.turn(a, c);
  }
  if (BOTH && a.kv_heads) {
    rows.init(a.k, there && j < a.kv_heads, b, t, j, a.teams, a.kv_heads);
    if constexpr (NORM) {
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = mine[k_coef + e * LANES];
    }
    for (int n = 0; n < a.k_batches; ++n) {
      rows.load();
      rows.turn(a, c);
    }
  }
}

template <typename T, bool HALF, int LANES, bool NORM, int BATCH, bool BOTH>
sd_status launch(RopeKernelArgs a, int64_t tokens, int per, cudaStream_t s) {
  auto batches = [](int heads, int teams) { return teams ? (heads + BATCH * teams - 1) / (BATCH * teams) : 0; };
  a.tokens = per;
  a.teams = kThreads / LANES / per;
  a.all_tokens = static_cast<unsigned>(tokens);
  const int heads = a.heads + a.kv_heads;
  a.q_teams = BOTH || a.heads ? a.teams : 0;
  if (!BOTH && a.heads && a.kv_heads && a.teams > 1)  // none has much more to do than another
    a.q_teams = std::min(std::max((a.teams * a.heads + heads / 2) / heads, 1), a.teams - 1);
  a.batches = std::max(batches(a.heads, a.q_teams), batches(a.kv_heads, a.teams - a.q_teams));
  a.k_batches = batches(a.kv_heads, a.teams);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((tokens + per - 1) / per));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(per) * 4 * LANES * sizeof(float4) * (NORM ? 2 : 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  cfg.attrs = attr;
  cfg.numAttrs = sd::pdl_attr(&attr[0]);
  return sd::cuda_check(cudaLaunchKernelEx(&cfg, rope_kernel<T, HALF, LANES, NORM, BATCH, BOTH>, a), "sd_rope_axes launch");
}

template <typename T, bool HALF, int LANES>
sd_status by_heads(const RopeKernelArgs& a, int64_t tokens, cudaStream_t s) {
  // Tokens of a CTA: as many as leave two CTAs an SM and give a team no more than 20 heads. Measured
  // (us, bf16, norm): [1, 32760, 16 + 16, 128] 4 / 8 / 16 tokens: 91.8 / 86.0 / 91.7; [2, 4173, 16 + 16,
  // 64]: 19.6 / 13.6 / 12.7; [2, 1024, 8 + 8, 40]: 5.6 / 4.2 / 4.3.
  // Teams with eight heads and more take some of q and some of k, which keeps a thread within the 64
  // registers of four CTAs an SM (80 and three where half-pairs would spill: 58.4 against 63.2 us for [1,
  // 32760, 16 + 4, 128] without norm; 87.6 and 13.1 us for the first two above, 103 and 17.9 with teams of
  // their own for q and k). With fewer heads q and k go to different teams and are loaded at the same
  // time ([2, 512, 16 + 4, 128]: 4.5 against 6.1).
  constexpr int kTeams = kThreads / LANES;
  const int heads = a.heads + a.kv_heads;
  int per = 1;
  while (2 * per <= kTeams && tokens / (2 * per) >= 2LL * sd::sm_count() && heads * 2 * per <= 20 * kTeams) per *= 2;
  const int rows = (heads * per + kTeams - 1) / kTeams;  // heads of a team
  auto pick = [&](auto norm) {
    constexpr bool N = decltype(norm)::value;
    // (a token with one team has no other for k)
    if (rows >= 8 || kTeams / per == 1) return launch<T, HALF, LANES, N, 4, true>(a, tokens, per, s);
    if (rows >= 4) return launch<T, HALF, LANES, N, 2, false>(a, tokens, per, s);
    return launch<T, HALF, LANES, N, 1, false>(a, tokens, per, s);
  };
  return a.norms ? pick(std::true_type()) : pick(std::false_type());
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

// A dimension of two views: bytes from one element to the next, and how many elements each has.
struct Step {
  int64_t bytes, na, nb;
};

// Whether a block of `block_a` bytes and one of `block_b` bytes, `d` bytes behind it, meet, each moved along the
// first `n` steps. Steps contain one another (meet), so along the largest only two places come near.
bool blocks_meet(int64_t d, const Step* step, int n, int64_t block_a, int64_t block_b) {
  if (n == 0) return d < block_a && -d < block_b;
  const Step& s = step[n - 1];
  const int64_t near = d / s.bytes + (d % s.bytes > 0);  // of the first view, counted from the second
  for (int64_t t : {near, near - 1})
    if (t < s.na && -t < s.nb && blocks_meet(d - t * s.bytes, step, n - 1, block_a, block_b)) return true;
  return false;
}

// Whether two views share an element. Dimensions in which they step alike, each step past all within it, are
// followed exactly (q and k in one buffer, in any layout); what lies within the others counts as one block.
bool meet(const View& a, const View& b) {
  if (!sd::overlaps(a.ptr, a.bytes(), b.ptr, b.bytes())) return false;
  int64_t block_a = a.dh * a.size, block_b = block_a;
  Step step[3];
  int n = 0;
  for (int i = 0; i < 3; ++i) {
    if (a.n[i] > 1 && b.n[i] > 1 && a.stride[i] != b.stride[i]) {
      block_a += (a.n[i] - 1) * a.stride[i] * a.size;
      block_b += (b.n[i] - 1) * b.stride[i] * b.size;
    } else if (a.n[i] > 1 || b.n[i] > 1) {
      step[n++] = {(a.n[i] > 1 ? a.stride[i] : b.stride[i]) * a.size, a.n[i], b.n[i]};
    }
  }
  std::sort(step, step + n, [](const Step& x, const Step& y) { return x.bytes < y.bytes; });
  int64_t span_a = block_a, span_b = block_b;
  int kept = 0;
  for (int i = 0; i < n; ++i) {
    const Step s = step[i];
    const bool past = s.bytes >= span_a && s.bytes >= span_b;
    span_a += (s.na - 1) * s.bytes;
    span_b += (s.nb - 1) * s.bytes;
    if (past) step[kept++] = s;
    else kept = 0, block_a = span_a, block_b = span_b;
  }
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.ptr) - reinterpret_cast<uintptr_t>(a.ptr));
  return blocks_meet(d, step, kept, block_a, block_b);
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
  a.eps = g.eps, a.inv_dh = 1.0f / static_cast<float>(g.dh);
  a.norms = (g.heads && g.q_weight) || (g.kv_heads && g.k_weight);
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
