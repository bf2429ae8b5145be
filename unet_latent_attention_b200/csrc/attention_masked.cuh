// Masked attention on sm_100a (sd_attention_masked): the kernel, shared by the translation units that
// instantiate it per head size.
//
//   t_ij = scale q_i . k_j  (cap * tanh(t / cap))  (+ bias[h, clamp(distance)]);  o_i = softmax_j(t_ij) v_j
//
// Every mask of the operator (length, causal, prefix, document) leaves one interval of keys [lo_i, hi_i)
// per query, and both ends grow with i. So a tile of queries needs the key tiles from lo of its first
// row to hi of its last one, and only those that reach past lo of the last or hi of the first row need
// element masks: the others run as if there were no mask.
//
// A CTA of 256 threads owns 128 query rows of one (batch, head) and streams their key tiles:
//  * warp 0: TMA producer of Q and of the rings of key and value tiles (rows past the end read as
//    zeros). The rings are apart: a key tile is free once S = Q K^T is done, a value tile only after P V.
//  * warp 1 issues the tcgen05 work: S = Q K^T into tensor memory, O += P V with P read from tensor
//    memory. P has columns of its own, so the next S runs while this one is in its softmax.
//  * warp 2: the guard. It waits for every V tile and, where the tile has masked elements, sets its
//    infinities and NaN to zero: a zero probability times them would be NaN in rows that do not see
//    them. (Rows that do see one add it in the epilogue.) With a bias it also copies the values that
//    the tile's distances can take into shared memory.
//  * warps 4-7: one row a thread, fp32 maximum and sum, exp2, P rounded to the input's type. The
//    running maximum is raised only when it grows by more than 2^8.
// Two CTAs share an SM (up to 128 columns): while one waits for S, P V or a copy, the other has the
// special-function unit, and one's start and end hide behind the other's tiles. No waiting is shared
// between them, so items of any length mix. Measured for [2, 10, 4096, 64] and [2, 8, 4096, 128]: 146 and 141
// us; two query tiles in one CTA, with turns on the special-function unit, 192 and 187; eight softmax
// warps on half rows 193 and 164 with one CTA an SM, 160 at 64 columns with two.
//
// Few query rows: the CTAs of a cluster take equal parts of the key tiles and join (m, l, O) through
// distributed shared memory in rank order, so the result does not depend on timing and no workspace
// is needed. Heads that share a key head are rows of the same tile then.
//
// What bounds it (cycles of a softmax warp per 128 keys, two CTAs an SM, 64 columns, no bias or cap): exp2
// takes 1400 of 2800, where the special-function unit needs 1024 for each CTA's tile; 440 go to waiting for
// S, the others to maxima, masks and copies. 296 query tiles run at a time, so a call of few waves also
// waits for its last one.
//
// All waits on mbarriers are bounded; see attn_common.cuh.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "attn_common.cuh"
#include "sd_internal.h"
#include "sm100_ptx.cuh"

namespace sd {
namespace masked {

using namespace sm100;
using sd::attn::BM;
using sd::attn::wait_bar;

struct Params {
  void* out;
  const uint16_t* v;
  const float* bias;  // [heads, 2 R + 1]
  const int32_t *kv_lens, *q_starts, *prefix_lens, *q_offsets, *k_offsets;
  long long o_batch, o_token, o_head;  // strides in elements
  long long v_batch, v_token, v_head;
  int heads, group;      // query heads; query heads per key head
  int pack, pack_log2;   // heads that are rows of one tile (1 or group, a power of two)
  int Lq, Lk, dh, docs, radius, causal;
  int tiles;             // query tiles of a plane (one batch's packed head)
  int planes, plane_group;  // planes; planes whose items are mixed
  float scale_log2;      // scale * log2(e)
  float cap_in, cap_out; // scale / cap, cap log2(e)
  float cap_scale, cap_inv;  // scale, 1 / cap
  int cap_raw;           // whether the cap's polynomial in q.k is within fp32
  unsigned int* err;
};

// What a query sees: keys [lo, hi); distance of key j from query i: j - i + shift.
struct Row {
  int lo, hi;
  long long shift;
  bool exists;  // in the tensor, and in a document if there are any
};

constexpr long long kStartLimit = 1LL << 30;

__device__ __forceinline__ long long clampll(long long v, long long lo, long long hi) {
  return v < lo ? lo : v > hi ? hi : v;
}

__device__ inline Row row_of(const Params& p, int b, int i) {
  Row r{0, 0, 0, false};
  if (i >= p.Lq) return r;
  long long q0 = 0, k0 = 0, nq = p.Lq, nk = p.Lk;
  int s = b;
  if (p.docs) {
    int a = 0, e = p.docs + 1;  // number of offsets <= i
    while (a < e) {
      const int m = (a + e) >> 1;
      if (p.q_offsets[m] <= i) a = m + 1;
      else e = m;
    }
    s = a - 1;
    if (s < 0 || s >= p.docs) {  // before the first or behind the last document
      r.lo = r.hi = static_cast<int>(clampll(p.k_offsets[s < 0 ? 0 : p.docs], 0, p.Lk));
      return r;
    }
    q0 = p.q_offsets[s];
    nq = p.q_offsets[s + 1] - q0;
    k0 = clampll(p.k_offsets[s], 0, p.Lk);
    nk = clampll(p.k_offsets[s + 1], k0, p.Lk) - k0;
  }
  long long start = nk - nq;  // of the whole tensors without documents
  if (p.q_starts) start = clampll(p.q_starts[s], -kStartLimit, kStartLimit);
  if (p.kv_lens) nk = clampll(p.kv_lens[b], 0, p.Lk);
  long long seen = nk;
  if (p.causal) {
    seen = start + (i - q0) + 1;
    if (p.prefix_lens && p.prefix_lens[s] > seen) seen = p.prefix_lens[s];
    seen = clampll(seen, 0, nk);
  }
  r.lo = static_cast<int>(k0);
  r.hi = static_cast<int>(k0 + seen);
  r.shift = q0 - k0 - start;
  r.exists = true;
  return r;
}

// DHT: padded head size (64-column chunks of shared memory; N of O is dh rounded up to 16). BN: keys of
// a tile. KS, VS: stages of the rings of key and value tiles. CTAS: CTAs of an SM.
template <int DHT_, int BN_, int KS_, int VS_, int CTAS_, bool F16_, bool CAP_, bool BIAS_>
struct Cfg {
  static constexpr int DHT = DHT_, BN = BN_, KS = KS_, VS = VS_, CTAS = CTAS_;
  static constexpr bool F16 = F16_, CAP = CAP_, BIAS = BIAS_;
  static constexpr int NCH = (DHT + 63) / 64;
  static constexpr int Q_TILE = NCH * BM * 128, KV_TILE = NCH * BN * 128;
  static constexpr int K_OFF = Q_TILE, V_OFF = K_OFF + KS * KV_TILE;
  static constexpr int BIAS_OFF = V_OFF + VS * KV_TILE;
  // Windows of a bias, one for each stage of V: the BM + BN - 1 values of a tile's distances, in four
  // copies shifted by 1 to 4 values, so that every row reads its own 16 bytes at a time; eight
  // neighbouring rows meet all banks once (WINDOW is 8 modulo 32).
  static constexpr int WINDOW = BM + BN + 8;
  static constexpr int BAR_OFF = BIAS_OFF + (BIAS ? VS * 4 * WINDOW * 4 : 0);
  // q_full, s_full, s_free, p_full, o_done, fin, k_full[KS], k_empty[KS], v_full[VS], v_ready[VS], v_empty[VS],
  // bias_full[VS]
  static constexpr int NBARS = 6 + 2 * KS + 4 * VS;
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;  // TMEM address, abort flag, cleaned flag, mixed flag
  static constexpr int BOUNDS_OFF = MISC_OFF + 16;      // lo of the first and last row, hi of both
  static constexpr int SMEM = BOUNDS_OFF + 16;
  static constexpr int TM_P = BN, TM_O = BN + BN / 2;  // tensor memory columns: S | P | O
  static constexpr int TM_COLS = TM_O + DHT <= 256 ? 256 : 512;
  static constexpr int THREADS = 256;
  // Units of a row's maximum: those of q.k where nothing else makes up a score, else those of the score (log2).
  static constexpr bool RAW_MAX = !CAP && !BIAS;
  // Rows whose maximum passes this (units of log2) take exp2's argument from differences; see the softmax.
  static constexpr float LARGE = 65536.f;
  static constexpr bool CHECK_LARGE = !CAP;  // a cap's scores are differences from the start
  static constexpr int REG_HELPER = 48, REG_SOFT = 208;  // two CTAs an SM: registers move to the softmax warps
  // Join of a cluster's parts: rows of DHT fp32 and (m, l), over Q and the rings.
  static constexpr int JOIN_ROW = DHT + 4;  // floats a row (+4: rows start in different banks)
  static_assert(CTAS * TM_COLS <= 512 && CTAS * (SMEM + 1024) <= 228 * 1024, "on-chip memory");
  static_assert(CTAS == 1 || (CTAS == 2 && 128 * (REG_HELPER + REG_SOFT) <= 65536 / 2), "register split");
  static_assert(!BIAS || WINDOW % 32 == 8, "copies of a window in different banks");
  static_assert(BM * JOIN_ROW * 4 <= Q_TILE + (KS + VS) * KV_TILE, "the join fits Q and the rings");
};

template <int KS, int VS>
struct Bars {
  uint32_t base;
  __device__ uint32_t q_full() const { return base; }
  __device__ uint32_t s_full() const { return base + 8; }
  __device__ uint32_t s_free() const { return base + 16; }
  __device__ uint32_t p_full() const { return base + 24; }
  __device__ uint32_t o_done() const { return base + 32; }
  __device__ uint32_t fin() const { return base + 40; }
  __device__ uint32_t k_full(int s) const { return base + 8 * (6 + s); }
  __device__ uint32_t k_empty(int s) const { return base + 8 * (6 + KS + s); }
  __device__ uint32_t v_full(int s) const { return base + 8 * (6 + 2 * KS + s); }
  __device__ uint32_t v_ready(int s) const { return base + 8 * (6 + 2 * KS + VS + s); }
  __device__ uint32_t v_empty(int s) const { return base + 8 * (6 + 2 * KS + 2 * VS + s); }
  __device__ uint32_t bias_full(int s) const { return base + 8 * (6 + 2 * KS + 3 * VS + s); }
};

// A position in a ring of N stages, and the parity of its phase.
template <int N>
struct Ring {
  int s = 0, parity = 0;
  __device__ __forceinline__ void next() {
    if (++s == N) s = 0, parity ^= 1;
  }
};

// The keys that the first and last row of a query tile see.
struct Bounds {
  int lo_first, lo_last, hi_first, hi_last;
};

// Whether the distances d0 .. d0 + n - 1 all lie beyond the table's ends: one bias for all of them.
__device__ __forceinline__ bool is_far(long long d0, int n, int radius) { return d0 >= radius || d0 + n - 1 <= -radius; }

// Whether a lane's share of n packs of 16-bit values holds no infinity and no NaN: each value times
// zero is zero, or NaN. Eight packs are in flight at a time (n is a multiple of 256).
template <bool F16>
__device__ __forceinline__ bool all_finite(const uint4* tile, int n, int lane) {
  using T2 = std::conditional_t<F16, __half2, __nv_bfloat162>;
  const uint32_t zero_bits = 0;
  const T2 zero = *reinterpret_cast<const T2*>(&zero_bits);
  T2 acc[4] = {zero, zero, zero, zero};
  for (int i = lane; i < n; i += 256) {
    uint4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = tile[i + 32 * k];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const T2* v = reinterpret_cast<const T2*>(&x[k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = __hfma2(v[e], zero, acc[e]);
    }
  }
  const T2 sum = __hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3]));
  return __heq2(sum, sum).x != static_cast<decltype(sum.x)>(0.f) && __heq2(sum, sum).y != static_cast<decltype(sum.x)>(0.f);
}

// One lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// A bias in units of log2; the lowest finite value stays finite.
__device__ __forceinline__ float bias_log2(float x) {
  const float y = x * 1.4426950408889634f;
  return isinf(y) && !isinf(x) ? copysignf(3.402823466e38f, x) : y;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap * log2(e) * tanh(u) of two scores from two results of the special-function unit each: off by 2e-7 of the cap,
// which only a score of its size can bear.
__device__ __forceinline__ float2 cap_large_scores(float u0, float u1, float cap_log2) {
  const float2 t = __fmul2_rn(make_float2(u0, u1), make_float2(2.885390081777927f, 2.885390081777927f));
  const float2 e = __fadd2_rn(make_float2(ex2_approx(t.x), ex2_approx(t.y)), make_float2(1.f, 1.f));
  return __ffma2_rn(make_float2(rcp_approx(e.x), rcp_approx(e.y)), make_float2(-2.f * cap_log2, -2.f * cap_log2),
                    make_float2(cap_log2, cap_log2));
}

// The same for |u| <= 1/2 by an odd polynomial (coefficients from unet_latent_attention_b200/fit_tanh_poly.py),
// off by 2e-7 of the score: for u = x k, a polynomial in x = q.k.
struct CapPoly {
  float2 c0, c1, c2, c3;  // twice each, for packed operations
};
__device__ __forceinline__ CapPoly cap_poly(float k, float cap_log2) {
  const float k2 = k * k, a0 = cap_log2 * k, a1 = a0 * k2, a2 = a1 * k2, a3 = a2 * k2;
  const float2 c0 = {9.999976754e-01f * a0, 9.999976754e-01f * a0}, c1 = {-3.332065642e-01f * a1, -3.332065642e-01f * a1}, c2 = {1.314514577e-01f * a2, 1.314514577e-01f * a2}, c3 = {-4.337248206e-02f * a3, -4.337248206e-02f * a3};
  return {c0, c1, c2, c3};
}

// What q.k = x becomes before the polynomial: v = x unit, u = v step; the score is v P(u^2), and |u| k <= 1/2 where
// it is small. An ordinary cap has unit = step = 1. Far from it (scale / cap below 1e-7, where k^7 leaves fp32's
// range and x^2 may pass it) v is the score without its cap, u = v / cap, k = 1.
struct CapForm {
  float unit, step, k, cap_log2;
  CapPoly poly;
};
__device__ __forceinline__ CapForm cap_form(const Params& p) {
  if (p.cap_raw) return {1.f, 1.f, p.cap_in, p.cap_out, cap_poly(p.cap_in, p.cap_out)};
  return {p.cap_scale, p.cap_inv, 1.f, p.cap_out, cap_poly(1.f, 1.4426950408889634f)};
}

// N scores, each by the form of its own size, so that it does not depend on its neighbours' or on those of
// unseen keys.
template <int N>
__device__ __forceinline__ void cap_scores(float (&x)[N], const CapForm& f) {
  float u[N];
  bool any = false;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 v = __fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(f.unit, f.unit));
    const float2 w = __fmul2_rn(v, make_float2(f.step, f.step)), z = __fmul2_rn(w, w);
    float2 p = __ffma2_rn(f.poly.c3, z, f.poly.c2);
    p = __ffma2_rn(p, z, f.poly.c1);
    p = __ffma2_rn(p, z, f.poly.c0);
    p = __fmul2_rn(p, v);
    x[i] = p.x, x[i + 1] = p.y;
    const float2 t = __fmul2_rn(w, make_float2(f.k, f.k));
    u[i] = t.x, u[i + 1] = t.y;
    any = any || fabsf(t.x) > 0.5f || fabsf(t.y) > 0.5f;
  }
  if (__any_sync(0xffffffffu, any)) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 y = cap_large_scores(u[i], u[i + 1], f.cap_log2);
      x[i] = fabsf(u[i]) > 0.5f ? y.x : x[i];
      x[i + 1] = fabsf(u[i + 1]) > 0.5f ? y.y : x[i + 1];
    }
  }
}

// N scores, if all of the warp's are small (they stay below their cap by design), with the results of
// cap_scores for an ordinary cap: 5 packed operations for two values on the FMA pipe; the softmax needs the
// special-function unit for itself ([2, 10, 4096, 64]: 216 us; 452 where every tile has a score above half the
// cap). False, with nothing done, if a score of the warp lies beyond.
template <int N>
__device__ __forceinline__ bool cap_small_scores(float (&x)[N], float k, float cap_log2) {
  float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; i += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) top[e] = max3f(top[e], fabsf(x[i + e]), fabsf(x[i + 4 + e]));
  if (__any_sync(0xffffffffu, fmaxf(max3f(top[0], top[1], top[2]), top[3]) * k > 0.5f)) return false;
  const CapPoly c = cap_poly(k, cap_log2);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 v = make_float2(x[i], x[i + 1]), z = __fmul2_rn(v, v);
    float2 p = __ffma2_rn(c.c3, z, c.c2);
    p = __ffma2_rn(p, z, c.c1);
    p = __ffma2_rn(p, z, c.c0);
    p = __fmul2_rn(p, v);
    x[i] = p.x, x[i + 1] = p.y;
  }
  return true;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 peer_load4(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::CTAS)
    attention_masked_sm100(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Params p) {
  constexpr int BN = C::BN, KS = C::KS, VS = C::VS;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's period
  const uint32_t sbase = smem_u32(smem);
  const Bars<KS, VS> bars{sbase + C::BAR_OFF};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  volatile int* cleaned = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 8);  // the guard set a value to zero
  volatile int* mixed = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 12);   // rows with different shifts
  Bounds* bounds = reinterpret_cast<Bounds*>(smem + C::BOUNDS_OFF);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  // Items in groups of planes (a plane is one batch's packed heads), within a group the late queries
  // first: with a causal mask they see the most keys, and short items at the end even out the SMs.
  const int item = blockIdx.x / splits, planes = p.planes;
  const int group0 = item / (p.plane_group * p.tiles) * p.plane_group, group_n = min(p.plane_group, planes - group0);
  const int in_group = item - group0 * p.tiles;
  const int qt = p.tiles - 1 - in_group / group_n, plane = group0 + in_group % group_n;
  const int heads_packed = p.heads / p.pack;
  const int b = plane / heads_packed, h0 = plane % heads_packed * p.pack, kvh = h0 / p.group;
  const long long rows = static_cast<long long>(p.Lq) * p.pack;    // of this (batch, packed head)
  const long long row0 = static_cast<long long>(qt) * BM;
  const int q_first = static_cast<int>(row0 >> p.pack_log2);  // the first row's query

  if (threadIdx.x == 0) {
    mbar_init(bars.q_full(), 1);
    mbar_init(bars.s_full(), 1);
    mbar_init(bars.s_free(), 128);
    mbar_init(bars.p_full(), 128);
    mbar_init(bars.o_done(), 1);
    mbar_init(bars.fin(), 1);
    for (int s = 0; s < KS; ++s) {
      mbar_init(bars.k_full(s), 1);
      mbar_init(bars.k_empty(s), 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(bars.v_full(s), 1);
      mbar_init(bars.v_ready(s), 1);
      mbar_init(bars.v_empty(s), 1);
      mbar_init(bars.bias_full(s), 1);
    }
    *abort_flag = 0;
    *cleaned = 0;
    *mixed = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::TM_COLS);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  sd::grid_dep_wait();  // global memory from here on
  sd::grid_dep_launch();

  const int r_in = (warp & 3) * 32 + lane;  // softmax threads: the row of the tile
  Row me{0, 0, 0, false};
  if (warp >= 4) {
    const long long r = row0 + r_in;
    if (r < rows) {
      me = row_of(p, b, static_cast<int>(r >> p.pack_log2));
      if (r_in == 0) bounds->lo_first = me.lo, bounds->hi_first = me.hi;
      if (r_in == BM - 1 || r == rows - 1) bounds->lo_last = me.lo, bounds->hi_last = me.hi;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  long long shift0 = 0;
  if constexpr (C::BIAS) {
    // The window of distances assumes one shift for the tile's rows; documents may differ in theirs.
    shift0 = row_of(p, b, static_cast<int>(row0 >> p.pack_log2)).shift;
    if (me.exists && me.hi > me.lo && me.shift != shift0) *mixed = 1;
    __syncthreads();
  }
  // Key tiles [j0, j1) of this CTA; those outside [whole0, whole1) need element masks.
  const Bounds tb = *bounds;
  int j0 = tb.lo_first / BN, j1 = tb.hi_last > tb.lo_first ? (tb.hi_last + BN - 1) / BN : j0;
  const int whole0 = (tb.lo_last + BN - 1) / BN, whole1 = tb.hi_first / BN;
  if (splits > 1) {
    const long long n = j1 - j0;
    const int a = j0 + static_cast<int>(n * rank / splits), e = j0 + static_cast<int>(n * (rank + 1) / splits);
    j0 = a, j1 = e;
  }

  if (warp < 4) {
    // ================================================================== helper warps
    if constexpr (C::CTAS > 1) regs_dec<C::REG_HELPER>();
    const int chunks = (p.dh + 63) / 64;
    if (warp == 0) {
      // ---------------------------------------------------------------- TMA producer
      if (lane == 0 && j1 > j0) {
        mbar_arrive_expect_tx(bars.q_full(), chunks * BM * 128);
        for (int c = 0; c < chunks; ++c)
          tma_load_4d(sbase + c * BM * 128, &tm_q, bars.q_full(), c * 64, h0, static_cast<int>(row0 >> p.pack_log2), b);
        Ring<KS> rk;
        Ring<VS> rv;
        int nk = 0, nv = 0;  // tiles issued
        for (int j = j0; j < j1; ++j) {
          if (nk >= KS && !wait_bar(bars.k_empty(rk.s), rk.parity ^ 1, abort_flag, p.err)) break;
          mbar_arrive_expect_tx(bars.k_full(rk.s), chunks * BN * 128);
          for (int c = 0; c < chunks; ++c)
            tma_load_4d(sbase + C::K_OFF + rk.s * C::KV_TILE + c * BN * 128, &tm_k, bars.k_full(rk.s), c * 64, kvh, j * BN, b);
          ++nk;
          rk.next();
          if (nv >= VS && !wait_bar(bars.v_empty(rv.s), rv.parity ^ 1, abort_flag, p.err)) break;
          mbar_arrive_expect_tx(bars.v_full(rv.s), chunks * BN * 128);
          for (int c = 0; c < chunks; ++c)
            tma_load_4d(sbase + C::V_OFF + rv.s * C::KV_TILE + c * BN * 128, &tm_v, bars.v_full(rv.s), c * 64, kvh, j * BN, b);
          ++nv;
          rv.next();
        }
        // Every copy has landed before the CTA may exit.
        wait_bar(bars.q_full(), 0, abort_flag, p.err, false);
        for (int k = max(0, nk - KS); k < nk; ++k) wait_bar(bars.k_full(k % KS), (k / KS) & 1, abort_flag, p.err, false);
        for (int k = max(0, nv - VS); k < nv; ++k) wait_bar(bars.v_full(k % VS), (k / VS) & 1, abort_flag, p.err, false);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer
      // The whole warp runs the loop and one elected lane issues: descriptors then live in uniform
      // registers (a lane of its own spent 100 to 175 cycles on every MMA).
      const int ksteps = (p.dh + 15) / 16;
      constexpr uint32_t idesc_qk = idesc_f16kind_f32(BM, BN, false, C::F16);
      const uint32_t idesc_pv = idesc_f16kind_f32(BM, 16, true, C::F16) + (static_cast<uint32_t>((ksteps * 16 - 16) >> 3) << 17);
      const uint32_t tS = tmem, tP = tmem + C::TM_P, tO = tmem + C::TM_O;
      // Descriptors count addresses in units of 16 bytes.
      const uint64_t q_desc = smem_desc(sbase, 16, 1024), k_desc = smem_desc(sbase + C::K_OFF, 16, 1024);
      const uint64_t v_desc = smem_desc(sbase + C::V_OFF, BN * 128, 1024);
      auto wait = [&](uint32_t bar, int parity) { return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, p.err)) != 0; };
      auto issue_qk = [&](int s) {
        const uint64_t kd = k_desc + static_cast<uint32_t>(s * (C::KV_TILE / 16));
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < C::DHT / 16; ++ks)
            if (ks < ksteps)
              mma_ss(tS, q_desc + (ks >> 2) * (BM * 8) + (ks & 3) * 2, kd + (ks >> 2) * (BN * 8) + (ks & 3) * 2, idesc_qk,
                     ks > 0 ? 1u : 0u);
          mma_commit(bars.s_full());
          mma_commit(bars.k_empty(s));
        }
        __syncwarp();
      };
      auto issue_pv = [&](int s, bool first) {
        const uint64_t vd = v_desc + static_cast<uint32_t>(s * (C::KV_TILE / 16));
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < BN / 16; ++ks) mma_ts(tO, tP + ks * 8, vd + ks * 128, idesc_pv, (!first || ks > 0) ? 1u : 0u);
          mma_commit(bars.o_done());
          mma_commit(bars.v_empty(s));
        }
        __syncwarp();
      };
      // S of the next tile is issued before P V of this one, as soon as S has been read.
      bool ok = j1 <= j0 || wait(bars.q_full(), 0);
      Ring<KS> rk;
      Ring<VS> rv;
      auto finish = [&](int n) {  // P V of the n-th tile
        if (!wait(bars.p_full(), n & 1) || !wait(bars.v_ready(rv.s), rv.parity)) return false;
        issue_pv(rv.s, n == 0);
        rv.next();
        return true;
      };
      int n = 0;
      for (int j = j0; ok && j < j1; ++j, ++n) {
        if (!(ok = wait(bars.k_full(rk.s), rk.parity))) break;
        if (n > 0 && !(ok = wait(bars.s_free(), (n - 1) & 1))) break;
        issue_qk(rk.s);
        rk.next();
        if (n > 0 && !(ok = finish(n - 1))) break;
      }
      if (ok && n > 0) finish(n - 1);
      if (elect_one()) mma_commit(bars.fin());
      wait_bar(bars.fin(), 0, abort_flag, p.err, false);
      __syncwarp();
    } else if (warp == 2) {
      // ---------------------------------------------------------------- guard
      Ring<VS> rv;
      constexpr int N = (BM + BN) / 32;
      float window[N];  // of the next tile: on its way while this one is looked after
      bool far = false;
      auto load_window = [&](int j) {
        const long long d0 = static_cast<long long>(j) * BN - (q_first + BM - 1) + shift0;
        const float* table = p.bias + static_cast<long long>(h0) * (2LL * p.radius + 1) + p.radius;
        far = is_far(d0, BM + BN - 1, p.radius);
        if (far) {
          window[0] = __ldg(table + (d0 >= p.radius ? p.radius : -p.radius));
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) window[i] = __ldg(table + clampll(d0 + i * 32 + lane, -p.radius, p.radius));
        }
      };
      if (C::BIAS && j1 > j0) load_window(j0);
      for (int j = j0; j < j1; ++j) {
        const int s = rv.s;
        if constexpr (C::BIAS) {
          if (j - j0 >= VS && !__all_sync(0xffffffffu, wait_bar(bars.v_empty(s), rv.parity ^ 1, abort_flag, p.err))) break;
          // Value e belongs to the distance d0 + e; the copy shifted by c holds it at place e + c.
          float* w = reinterpret_cast<float*>(smem + C::BIAS_OFF) + s * 4 * C::WINDOW;
          if (far) {
            if (lane == 0) w[0] = bias_log2(window[0]);
          } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const float y = bias_log2(window[i]);
#pragma unroll
              for (int c = 1; c <= 4; ++c) w[(c - 1) * C::WINDOW + c + i * 32 + lane] = y;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bars.bias_full(s));
          if (j + 1 < j1) load_window(j + 1);
        }
        if (!__all_sync(0xffffffffu, wait_bar(bars.v_full(s), rv.parity, abort_flag, p.err))) break;
        if (j < whole0 || j >= whole1) {
          uint4* tile = reinterpret_cast<uint4*>(smem + C::V_OFF + s * C::KV_TILE);
          if (__any_sync(0xffffffffu, !all_finite<C::F16>(tile, chunks * BN * 8, lane))) {
            for (int i = lane; i < chunks * BN * 8; i += 32) {
              uint4 x = tile[i];
              uint32_t* w = reinterpret_cast<uint32_t*>(&x);
              constexpr uint32_t kExp = C::F16 ? 0x7c00u : 0x7f80u;  // all exponent bits set: infinity or NaN
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if ((w[k] & kExp) == kExp) w[k] &= 0xffff0000u;
                if ((w[k] >> 16 & kExp) == kExp) w[k] &= 0xffffu;
              }
              tile[i] = x;
            }
            if (lane == 0) *cleaned = 1;
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        if (lane == 0) mbar_arrive(bars.v_ready(s));
        rv.next();
      }
    }
  } else {
    // ================================================================== softmax warps
    if constexpr (C::CTAS > 1) regs_inc<C::REG_SOFT>();
    const int quarter = warp & 3;
    const uint32_t tbase = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t tS = tbase, tP = tbase + C::TM_P, tO = tbase + C::TM_O;
    const bool live = row0 + (r_in & ~31) < rows;  // a warp behind the last row only keeps the barriers going
    const bool is_mixed = C::BIAS && *mixed;
    const int ochunks = (p.dh + 15) / 16;
    float m_run = -INFINITY, l_run = 0.f;
    const float m_scale = C::RAW_MAX ? p.scale_log2 : 1.f;
    bool ok = true;
    if (!live) {
      for (int j = j0; ok && j < j1; ++j) {
        const int par = (j - j0) & 1;
        ok = __all_sync(0xffffffffu, wait_bar(bars.s_full(), par, abort_flag, p.err));
        if (ok) mbar_arrive(bars.s_free());
        // as the other warps: no arrival for this P before every warp's for the one before it
        if (ok && j > j0) ok = __all_sync(0xffffffffu, wait_bar(bars.o_done(), par ^ 1, abort_flag, p.err));
        if (ok) mbar_arrive(bars.p_full());
      }
    }
    for (int j = j0; live && j < j1; ++j) {
      // warp-uniform: the tcgen05 copies below are .sync.aligned
      if (!__all_sync(0xffffffffu, wait_bar(bars.s_full(), (j - j0) & 1, abort_flag, p.err))) {
        ok = false;
        break;
      }
      if (C::BIAS && !__all_sync(0xffffffffu, wait_bar(bars.bias_full((j - j0) % VS), ((j - j0) / VS) & 1, abort_flag, p.err))) {
        ok = false;
        break;
      }
      tc_fence_after();
      float sv[BN];
      auto load_scores = [&] {
#pragma unroll
        for (int c = 0; c < BN / 32; ++c) {
          uint32_t r[32];
          tmem_ld32(tS + c * 32, r);
#pragma unroll
          for (int i = 0; i < 32; ++i) sv[c * 32 + i] = __uint_as_float(r[i]);
        }
        tmem_wait_ld();
      };
      load_scores();
      // the score is sv * scale + offset, in units of log2
      float scale = C::CAP ? 1.f : p.scale_log2, offset = 0.f;
      bool biased = false;
      if constexpr (C::CAP || C::BIAS) {
        // The rare forms work on S in tensor memory, 16 or 32 columns at a time (a loop that stays out of the
        // instruction cache's way), in units of log2: large scores under a cap, and a bias over documents
        // with different shifts, where each row has its own distances.
        bool slow = is_mixed;
        if constexpr (C::CAP) slow = slow || !p.cap_raw || !cap_small_scores(sv, p.cap_in, p.cap_out);
        if (slow) {
          const float* table = p.bias + static_cast<long long>(h0) * (2LL * p.radius + 1) + p.radius;
          const long long d = static_cast<long long>(j) * BN - (q_first + r_in) + me.shift;
          CapForm form{};
          if constexpr (C::CAP) form = cap_form(p);
          constexpr int W = C::CAP ? 32 : 16;
#pragma unroll 1
          for (int c = 0; c < BN; c += W) {
            uint32_t r[W];
            float x[W];
            if constexpr (W == 32) tmem_ld32(tS + c, r);
            else tmem_ld16(tS + c, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < W; ++i) x[i] = __uint_as_float(r[i]);
            if constexpr (C::CAP) cap_scores(x, form);
            if (C::BIAS && is_mixed) {
#pragma unroll
              for (int i = 0; i < W; ++i)
                x[i] = fmaf(x[i], C::CAP ? 1.f : p.scale_log2, bias_log2(__ldg(table + clampll(d + c + i, -p.radius, p.radius))));
            }
#pragma unroll
            for (int h = 0; h < W; h += 16) {
              uint32_t w[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(x[h + i]);
              tmem_st16(tS + c + h, w);
            }
          }
          tmem_wait_st();
          load_scores();
          biased = is_mixed;
          if (is_mixed) scale = 1.f;
        }
      }
      if constexpr (!C::CHECK_LARGE) {
        tc_fence_before();
        mbar_arrive(bars.s_free());
      }
      if (C::BIAS && !biased) {
        const long long d0 = static_cast<long long>(j) * BN - (q_first + BM - 1) + shift0;  // the window's first distance
        const float* w = reinterpret_cast<const float*>(smem + C::BIAS_OFF) + ((j - j0) % VS) * 4 * C::WINDOW;
        if (is_far(d0, BM + BN - 1, p.radius)) {
          offset = w[0] == 0.f ? -0.f : w[0];  // +0 says that the sums are formed already
          // -infinity, or a type's lowest value: it swallows the score, as in a sum. (So does a large cap's score.)
          if (!(fabsf(offset) < 1e6f) || (C::CAP && p.cap_out > C::LARGE)) {
#pragma unroll
            for (int i = 0; i < BN; i += 2) fma2(sv[i], sv[i + 1], sv[i], sv[i + 1], scale, scale, offset, offset);
            scale = 1.f;
            offset = 0.f;
          }
        } else {
          // Column i of this row: value e + i, at multiples of four in the copy shifted by c.
          const int e = BM - 1 - r_in, c = 4 - (e & 3);
          const float4* mine = reinterpret_cast<const float4*>(w + (c - 1) * C::WINDOW + c + e);
#pragma unroll
          for (int i = 0; i < BN; i += 4) {
            const float4 y = mine[i / 4];
            fma2(sv[i], sv[i + 1], sv[i], sv[i + 1], scale, scale, y.x, y.y);
            fma2(sv[i + 2], sv[i + 3], sv[i + 2], sv[i + 3], scale, scale, y.z, y.w);
          }
          scale = 1.f;
        }
      }
      if (j < whole0 || j >= whole1) {
        // Element masks, 32 columns at a time: a warp's rows mostly see all or nothing of them.
        const int lo = me.lo - j * BN, hi = me.hi - j * BN;
#pragma unroll
        for (int w = 0; w < BN / 32; ++w) {
          const int l = min(max(lo - 32 * w, 0), 32), h = min(max(hi - 32 * w, 0), 32);
          const uint32_t seen = static_cast<uint32_t>(((1ull << h) - 1) & ~((1ull << l) - 1));
          if (__any_sync(0xffffffffu, seen != 0xffffffffu)) {
#pragma unroll
            for (int i = 0; i < 32; ++i) sv[32 * w + i] = seen >> i & 1 ? sv[32 * w + i] : -INFINITY;
          }
        }
      }
      float pm[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) pm[k] = sv[k];
#pragma unroll
      for (int i = 8; i + 16 <= BN; i += 16)
#pragma unroll
        for (int k = 0; k < 8; ++k) pm[k] = max3f(pm[k], sv[i + k], sv[i + 8 + k]);
#pragma unroll
      for (int k = 0; k < 8; ++k) pm[k] = fmaxf(pm[k], sv[BN - 8 + k]);
      const float mx = max3f(max3f(pm[0], pm[1], pm[2]), max3f(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7]));
      // A row without a seen key keeps m = -infinity whatever the offset is.
      const float m_new = fmaxf(m_run, C::BIAS ? (mx == -INFINITY ? mx : fmaf(mx, scale, offset)) : mx);
      // Row by row: a row's maximum never depends on its neighbours' scores. (-infinity - -infinity: no raise)
      const bool raise = (m_new - m_run) * m_scale > 8.0f, rescale = __any_sync(0xffffffffu, raise);
      const float alpha = !raise ? 1.0f : m_run == -INFINITY ? 0.f : ex2_approx((m_run - m_new) * m_scale);
      if (raise) m_run = m_new;
      // exp2(scale sv + offset - m); a row that has seen nothing gets zeros
      const float minus_m = (m_run == -INFINITY ? 0.f : -m_run * m_scale) + (C::BIAS ? offset : 0.f);
      // minus_m is off by half a step of the row's maximum. All weights of the row share that, but a step of a
      // large maximum is more than exp2 can hold: there the row's weights are formed again below, and S stays.
      bool large = false;
      if constexpr (C::CHECK_LARGE) {
        large = (C::RAW_MAX || __float_as_uint(offset) != 0) && fabsf(m_run * m_scale) > C::LARGE && fabsf(m_run) < INFINITY;
        tc_fence_before();
        mbar_arrive_if(bars.s_free(), !large);
      }
      uint32_t pk[BN / 2];
      float ls0 = 0.f, ls1 = 0.f, ls2 = 0.f, ls3 = 0.f;
#pragma unroll
      for (int i = 0; i < BN / 2; ++i) {
        float x0, x1;
        if constexpr (C::CAP && !C::BIAS) add2(x0, x1, sv[2 * i], sv[2 * i + 1], minus_m, minus_m);
        else fma2(x0, x1, sv[2 * i], sv[2 * i + 1], scale, scale, minus_m, minus_m);
        x0 = ex2_approx(x0);
        x1 = ex2_approx(x1);
        if (i & 1) add2(ls2, ls3, ls2, ls3, x0, x1);
        else add2(ls0, ls1, ls0, ls1, x0, x1);
        pk[i] = C::F16 ? pack_f16x2(x0, x1) : pack_bf16x2(x0, x1);
      }
      const float l_before = l_run * alpha;
      l_run = fmaf(l_run, alpha, (ls0 + ls1) + (ls2 + ls3));
      if (j > j0) {
        if (!__all_sync(0xffffffffu, wait_bar(bars.o_done(), (j - j0 - 1) & 1, abort_flag, p.err))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (rescale) {
          for (int c = 0; c < ochunks; ++c) {
            uint32_t r[16];
            tmem_ld16(tO + c * 16, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
            tmem_st16(tO + c * 16, r);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < BN / 32; ++c) {
        uint32_t r[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = pk[c * 16 + i];
        tmem_st16(tP + c * 16, r);
      }
      tmem_wait_st();
      if constexpr (C::CHECK_LARGE) {
        // The rows of large maxima once more, from S in tensor memory: the difference from the maximum comes
        // first and is 0 for the largest score (of q.k, or of the sum with a bias as rounded to fp32). The check
        // costs 1 to 3% of short key tiles' time ([2, 8, 4096, 128]: 139 -> 141 us, one token of [16, 16 / 4, 8192
        // ragged, 128] 39.0 -> 40.0) and nothing of the long ones' ([2, 10, 4096, 64]: 146); done before exp2,
        // where it waits for the maximum, 2 to 7%. Rows that take it: 319 us for [2, 10, 4096, 64].
        if (__any_sync(0xffffffffu, large)) {
          const int lo = me.lo - j * BN, hi = me.hi - j * BN;
          float sum = 0.f;
#pragma unroll 1
          for (int c = 0; c < BN / 32; ++c) {
            uint32_t r[32], w[16];
            tmem_ld32(tS + c * 32, r);
            tmem_ld16(tP + c * 16, w);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float y[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float x = __uint_as_float(r[i + e]);
                const int col = c * 32 + i + e;
                y[e] = col < lo || col >= hi ? 0.f : ex2_approx(C::RAW_MAX ? (x - m_run) * scale : fmaf(x, scale, offset) - m_run);
              }
              if (large) w[i / 2] = C::F16 ? pack_f16x2(y[0], y[1]) : pack_bf16x2(y[0], y[1]);
              sum += y[0] + y[1];
            }
            tmem_st16(tP + c * 16, w);
          }
          tmem_wait_st();
          if (large) l_run = l_before + sum;
          tc_fence_before();
          if (large) mbar_arrive(bars.s_free());
        }
      }
      tc_fence_before();
      mbar_arrive(bars.p_full());
    }
    if (ok && j1 > j0) ok = __all_sync(0xffffffffu, wait_bar(bars.o_done(), (j1 - j0 - 1) & 1, abort_flag, p.err));
    tc_fence_after();
    // ------------------------------------------------------------------ epilogue: one row a thread
    const long long row = row0 + r_in;
    const int i_q = static_cast<int>(row >> p.pack_log2), h = h0 + static_cast<int>(row & (p.pack - 1));
    // Values that the guard set to zero, for rows that see them: 16 columns from c16 of the masked tiles.
    auto add_cleaned = [&](int c16, float (&o)[16]) {
      const uint16_t* v = p.v + b * p.v_batch + kvh * p.v_head + c16;
      for (int j = j0; j < j1; ++j) {
        if (j >= whole0 && j < whole1) continue;
        for (int key = max(me.lo, j * BN); key < min(me.hi, (j + 1) * BN); ++key) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (c16 + i >= p.dh) continue;
            const uint32_t w = v[key * p.v_token + i];
            if (C::F16 ? (w & 0x7c00u) == 0x7c00u : (w & 0x7f80u) == 0x7f80u) {
              const bool nan = C::F16 ? (w & 0x3ffu) != 0 : (w & 0x7fu) != 0;
              o[i] += __uint_as_float(nan ? 0x7fc00000u : 0x7f800000u | (w & 0x8000u) << 16);
            }
          }
        }
      }
    };
    const bool has_o = j1 > j0 && ok, fix = has_o && *cleaned;  // the same for the warp
    const bool join = splits > 1;
    const bool store = row < rows && (join || (me.exists && ok));
    // A part of a cluster's join goes over Q and the ring: their copies and MMAs are done with the last P V.
    float* part = reinterpret_cast<float*>(smem) + r_in * C::JOIN_ROW;
    uint16_t* out = static_cast<uint16_t*>(p.out) + b * p.o_batch + i_q * p.o_token + h * p.o_head;
    const float inv = join ? 1.f : l_run == 0.f ? 0.f : 1.0f / l_run;
    if (live) {
      for (int c = 0; c < ochunks; ++c) {
        float o[16];
        if (has_o) {  // warp-wide: every lane takes part
          uint32_t r[16];
          __syncwarp();
          tmem_ld16(tO + c * 16, r);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = l_run == 0.f ? 0.f : __uint_as_float(r[i]) * inv;
          if (fix && store && l_run != 0.f) add_cleaned(c * 16, o);  // every seen score -infinity: 0 all the same
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = 0.f;
        }
        if (!store) continue;
        if (join) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4*>(part + c * 16)[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = C::F16 ? pack_f16x2(o[2 * i], o[2 * i + 1]) : pack_bf16x2(o[2 * i], o[2 * i + 1]);
          uint4* dst = reinterpret_cast<uint4*>(out + c * 16);
          dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
          if (c * 16 + 8 < p.dh) dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
      if (join && store) {
        part[C::DHT] = m_run;
        part[C::DHT + 1] = l_run;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
  if (splits > 1) {
    // Join: the rows are dealt to the CTAs; each output value is summed over the parts in rank order.
    cluster_sync();
    const int live_rows = static_cast<int>(min(rows - row0, static_cast<long long>(BM)));
    const int groups = p.dh / 8;  // 8 columns a thread
    if (!*abort_flag)
      for (int w = rank * C::THREADS + static_cast<int>(threadIdx.x); w < live_rows * groups; w += splits * C::THREADS) {
        const int r = w / groups, c = w % groups * 8;
        const long long at = row0 + r;
        if (!row_of(p, b, static_cast<int>(at >> p.pack_log2)).exists) continue;
        float m = -INFINITY;
        for (int k = 0; k < splits; ++k) m = fmaxf(m, peer_load4(sbase + (r * C::JOIN_ROW + C::DHT) * 4, k).x);
        const float m_scale = C::RAW_MAX ? p.scale_log2 : 1.f;
        const bool large = fabsf(m * m_scale) > C::LARGE;  // else the parts' own shifts are these products
        float l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < splits; ++k) {
          const float4 ml = peer_load4(sbase + (r * C::JOIN_ROW + C::DHT) * 4, k);
          if (ml.y == 0.f) continue;  // this part has no key that the row sees
          const float a = ml.x == -INFINITY ? 1.f : ex2_approx(large ? (ml.x - m) * m_scale : __fmul_rn(ml.x, m_scale) - __fmul_rn(m, m_scale));
          const float4 x = peer_load4(sbase + (r * C::JOIN_ROW + c) * 4, k);
          const float4 y = peer_load4(sbase + (r * C::JOIN_ROW + c + 4) * 4, k);
          l = fmaf(ml.y, a, l);
          o[0] = fmaf(x.x, a, o[0]), o[1] = fmaf(x.y, a, o[1]), o[2] = fmaf(x.z, a, o[2]), o[3] = fmaf(x.w, a, o[3]);
          o[4] = fmaf(y.x, a, o[4]), o[5] = fmaf(y.y, a, o[5]), o[6] = fmaf(y.z, a, o[6]), o[7] = fmaf(y.w, a, o[7]);
        }
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          q[i] = C::F16 ? pack_f16x2(o[2 * i] * inv, o[2 * i + 1] * inv) : pack_bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
        uint16_t* out = static_cast<uint16_t*>(p.out) + b * p.o_batch + (at >> p.pack_log2) * p.o_token + (h0 + (at & (p.pack - 1))) * p.o_head;
        *reinterpret_cast<uint4*>(out + c) = make_uint4(q[0], q[1], q[2], q[3]);
      }
    cluster_sync();  // no CTA leaves while a peer reads its part
  }
}

}  // namespace masked
}  // namespace sd
