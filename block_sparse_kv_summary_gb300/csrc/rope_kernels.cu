// Norms of the query and key heads and the position rotation in one pass over
// the fused projection's output: for one token per sequence (the inputs of a
// decode step) and for many (queries out, keys and values packed into the
// cache, and the block summaries of section "무엇과 다른가" formed on the way).
//
//   y = w x / sqrt(mean(x^2) + eps)              (skipped without a weight)
//   (u, v) -> (u cos - v sin, v cos + u sin)     for each pair of the first
//                                                rot_dim coordinates
//
// A head is held by D/8 lanes, four pairs (u, v) each: both members of a pair
// stand in one lane, so nothing but the sum of squares crosses lanes.  With
// the weights folded into the angles, (w_u cos, w_v sin, w_v cos, w_u sin),
// which hold for all heads of a token, a head costs two products a value and
// its norm's factor.
//
// Queries are computed in fp32.  The fp32 value of a key that is rounded to
// bf16 is the nearest one: the summaries are those of the stored keys, and a
// key that falls on the wrong side of a rounding border moves its block's mean
// and variance by a bf16 step, some thousand times more than the fp32
// arithmetic of the summary itself loses.  Where fp32 cannot tell the side,
// keys are computed again as unevaluated sums of two floats.
#include <type_traits>

#include "compkv_launch.h"
#include "kv8.cuh"
#include "tile_summary.cuh"

namespace compkv {

namespace {

// ---------------------------------------------------------------- two floats
struct F2 {  // hi + lo, |lo| <= ulp(hi) / 2
  float hi, lo;
};

__device__ __forceinline__ F2 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ F2 two_prod(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 s = two_sum(a.hi, b.hi);
  const float lo = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo));
  const float hi = __fadd_rn(s.hi, lo);
  return {hi, __fsub_rn(lo, __fsub_rn(hi, s.hi))};
}
// x w r
__device__ __forceinline__ F2 scaled(float x, float w, F2 r) {
  const F2 t = two_prod(x, w);
  F2 y = two_prod(t.hi, r.hi);
  y.lo = __fmaf_rn(t.hi, r.lo, __fmaf_rn(t.lo, r.hi, y.lo));
  return y;
}
// a c + b s
__device__ __forceinline__ F2 turn2(F2 a, float c, F2 b, float s) {
  F2 p = two_prod(a.hi, c), q = two_prod(b.hi, s);
  p.lo = __fmaf_rn(a.lo, c, p.lo);
  q.lo = __fmaf_rn(b.lo, s, q.lo);
  return add2(p, q);
}

// ---------------------------------------------------------------- a lane's part of a head
// Four pairs: `u` their first members, `v` their second.
struct Pairs {
  float u[4], v[4];
};
__device__ __forceinline__ float2 two(const float* x, int i) { return make_float2(x[2 * i], x[2 * i + 1]); }

// Where they stand: four coordinates from `a` on and four from `b` on.  INTER:
// eight coordinates in a row, pairs (2i, 2i + 1).  Otherwise u and v are half
// a rotation apart, and the coordinates behind the rotation make pairs alike,
// half of what is left apart, that do not turn.  rot is a multiple of 16.
struct Place {
  int a, b, col;  // col: the first pair's column in the table
  bool turns;
};
template <int D, bool INTER>
__device__ __forceinline__ Place place(int l, int rot) {
  if (INTER) return {8 * l, 8 * l + 4, 4 * l, 8 * l < rot};
  const int i = 4 * l;
  if (i < rot / 2) return {i, i + rot / 2, i, true};
  return {i + rot / 2, i + D / 2, 0, false};
}

// Eight coordinates as they come.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint2 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, const Place& at, bool live) {
    a = b = make_uint2(0, 0);
    if (live) {
      a = __ldcs(reinterpret_cast<const uint2*>(p + at.a));
      b = __ldcs(reinterpret_cast<const uint2*>(p + at.b));
    }
  }
  template <bool INTER>
  __device__ __forceinline__ Pairs pairs() const {
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
    Pairs p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
      if (INTER) {
        p.u[i] = lo;
        p.v[i] = hi;
      } else {
        (i < 2 ? p.u : p.v)[2 * (i & 1)] = lo;
        (i < 2 ? p.u : p.v)[2 * (i & 1) + 1] = hi;
      }
    }
    return p;
  }
  __device__ __forceinline__ uint4 bf16() const { return make_uint4(a.x, a.y, b.x, b.y); }
};
template <bool INTER>
__device__ __forceinline__ Pairs ordered(float4 a, float4 b) {
  if (INTER) return {{a.x, a.z, b.x, b.z}, {a.y, a.w, b.y, b.w}};
  return {{a.x, a.y, a.z, a.w}, {b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ uint32_t round2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, const Place& at, bool live) {
    a = b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
      a = __ldcs(reinterpret_cast<const float4*>(p + at.a));
      b = __ldcs(reinterpret_cast<const float4*>(p + at.b));
    }
  }
  template <bool INTER>
  __device__ __forceinline__ Pairs pairs() const {
    return ordered<INTER>(a, b);
  }
  __device__ __forceinline__ uint4 bf16() const {
    return make_uint4(round2(a.x, a.y), round2(a.z, a.w), round2(b.x, b.y), round2(b.z, b.w));
  }
};
// Back in the order of the coordinates: the four from a on, then those from b on.
template <bool INTER>
__device__ __forceinline__ void coordinates(const Pairs& p, float4& a, float4& b) {
  if (INTER) {
    a = make_float4(p.u[0], p.v[0], p.u[1], p.v[1]);
    b = make_float4(p.u[2], p.v[2], p.u[3], p.v[3]);
  } else {
    a = make_float4(p.u[0], p.u[1], p.u[2], p.u[3]);
    b = make_float4(p.v[0], p.v[1], p.v[2], p.v[3]);
  }
}
template <bool INTER>
__device__ __forceinline__ uint4 rounded(const Pairs& p) {
  float4 a, b;
  coordinates<INTER>(p, a, b);
  return make_uint4(round2(a.x, a.y), round2(a.z, a.w), round2(b.x, b.y), round2(b.z, b.w));
}
// bf16 values into four coordinates from `a` on and four from `b` on.
__device__ __forceinline__ void put(__nv_bfloat16* p, const Place& at, uint4 x) {
  *reinterpret_cast<uint2*>(p + at.a) = make_uint2(x.x, x.y);
  *reinterpret_cast<uint2*>(p + at.b) = make_uint2(x.z, x.w);
}
template <bool INTER>
__device__ __forceinline__ void put_query(const RopeArgs& a, int64_t head, const Place& at, const Pairs& y) {
  if (a.q_bf16) {
    const uint4 x = rounded<INTER>(y);
    __nv_bfloat16* q = reinterpret_cast<__nv_bfloat16*>(a.q) + head;
    __stcs(reinterpret_cast<uint2*>(q + at.a), make_uint2(x.x, x.y));
    __stcs(reinterpret_cast<uint2*>(q + at.b), make_uint2(x.z, x.w));
  } else {
    float4 c, d;
    coordinates<INTER>(y, c, d);
    float* q = reinterpret_cast<float*>(a.q) + head;
    __stcs(reinterpret_cast<float4*>(q + at.a), c);
    __stcs(reinterpret_cast<float4*>(q + at.b), d);
  }
}

// ---------------------------------------------------------------- a token's angles
struct Angles {
  float c[4], s[4];
};
__device__ __forceinline__ Angles angles(const float* row, int rot, const Place& at) {
  if (!at.turns) return {{1.f, 1.f, 1.f, 1.f}, {0.f, 0.f, 0.f, 0.f}};
  const float4 c = __ldg(reinterpret_cast<const float4*>(row + at.col));
  const float4 s = __ldg(reinterpret_cast<const float4*>(row + rot / 2 + at.col));
  return {{c.x, c.y, c.z, c.w}, {s.x, s.y, s.z, s.w}};
}
template <bool INTER>
__device__ __forceinline__ Pairs weights(const float* w, const Place& at) {
  if (!w) return {{1.f, 1.f, 1.f, 1.f}, {1.f, 1.f, 1.f, 1.f}};
  return ordered<INTER>(__ldg(reinterpret_cast<const float4*>(w + at.a)), __ldg(reinterpret_cast<const float4*>(w + at.b)));
}
// y_u = (u uc + v vs) r, y_v = (v vc + u us) r
struct Factors {
  float2 uc[2], vs[2], vc[2], us[2];
};
__device__ __forceinline__ Factors factors(const Pairs& w, const Angles& t) {
  Factors f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f.uc[i] = __fmul2_rn(two(w.u, i), two(t.c, i));
    f.vs[i] = __fmul2_rn(two(w.v, i), make_float2(-t.s[2 * i], -t.s[2 * i + 1]));
    f.vc[i] = __fmul2_rn(two(w.v, i), two(t.c, i));
    f.us[i] = __fmul2_rn(two(w.u, i), two(t.s, i));
  }
  return f;
}

__device__ __forceinline__ float rsqrt_approx(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A head in fp32; returns r, the norm's factor (1 without `normed`).
template <int D>
__device__ __forceinline__ float turn_head(const Pairs& x, const Factors& f, bool normed, float eps, Pairs& y) {
  float r = 1.f;
  if (normed) {
    float2 m = __fmul2_rn(two(x.u, 0), two(x.u, 0));
    m = __ffma2_rn(two(x.u, 1), two(x.u, 1), m);
    m = __ffma2_rn(two(x.v, 0), two(x.v, 0), m);
    m = __ffma2_rn(two(x.v, 1), two(x.v, 1), m);
    float q = m.x + m.y;
#pragma unroll
    for (int k = D / 16; k > 0; k >>= 1) q += __shfl_xor_sync(0xffffffffu, q, k);
    r = rsqrt_approx(fmaf(q, 1.f / D, eps));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float2 u = __ffma2_rn(two(x.u, i), f.uc[i], __fmul2_rn(two(x.v, i), f.vs[i]));
    float2 v = __ffma2_rn(two(x.v, i), f.vc[i], __fmul2_rn(two(x.u, i), f.us[i]));
    u = __fmul2_rn(u, make_float2(r, r));
    v = __fmul2_rn(v, make_float2(r, r));
    y.u[2 * i] = u.x;
    y.u[2 * i + 1] = u.y;
    y.v[2 * i] = v.x;
    y.v[2 * i + 1] = v.y;
  }
  return r;
}

// Whether an error of 16 roundings of 2^-24 could carry y over the border halfway between two bf16 values.  The
// roundings, 13: the sum of squares 9 at most (d 128), halved by the root, its eps 1/2, the root 4 (2^-22.9), weight
// times angle 1 each, a product 1, the sum 1, the factor 1; `size` is the size of what is added up.  The border is that
// of y's own bf16 step.  Just above a power of two the one below is nearer, 2^-9 y, but an error reaches it only where
// the terms cancel to 2^-11 of their size, and then the roundings of the norm's factor, which scale with y, fall away:
// the other three stay under the 8 that it takes.
__device__ __forceinline__ bool near_border(float y, float size) {
  const float border = __uint_as_float((__float_as_uint(y) & 0xffff0000u) | 0x8000u);
  return fabsf(y - border) <= size * (16.f / 16777216.f);
}

// A key head in two floats per value, rounded to fp32 and then to bf16.  Not inlined: it is rare and long.  The
// root: one step of Newton's iteration with its residual 1 - m r^2 in two floats.
template <int D, bool INTER>
__device__ __noinline__ uint4 key_exact(Pairs x, const float* row, int rot, Place at, const float* weight, float eps) {
  const Pairs w = weights<INTER>(weight, at);
  const Angles t = angles(row, rot, at);
  F2 r = {1.f, 0.f};
  if (weight) {
    F2 s = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) s = add2(add2(s, two_prod(x.u[i], x.u[i])), two_prod(x.v[i], x.v[i]));
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1)
      s = add2(s, {__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
    s.hi *= 1.f / D;  // exact: D is a power of two
    s.lo *= 1.f / D;
    const F2 m = add2(s, {eps, 0.f});
    const float r0 = rsqrtf(m.hi);
    const F2 h = two_prod(m.hi, r0);
    const float e = __fmaf_rn(-h.hi, r0, 1.f) - (h.lo + m.lo * r0) * r0;
    r = {r0, isfinite(r0) ? 0.5f * r0 * e : 0.f};
  }
  Pairs y;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const F2 u = scaled(x.u[i], w.u[i], r), v = scaled(x.v[i], w.v[i], r);
    const F2 a = turn2(u, t.c[i], v, -t.s[i]), b = turn2(v, t.c[i], u, t.s[i]);
    y.u[i] = __fadd_rn(a.hi, a.lo);
    y.v[i] = __fadd_rn(b.hi, b.lo);
  }
  return rounded<INTER>(y);
}

template <int D, bool INTER>
__device__ __forceinline__ uint4 turn_key(const Pairs& x, const Factors& f, const float* row, const RopeArgs& a, const Place& at) {
  Pairs y;
  const float r = turn_head<D>(x, f, a.k_weight != nullptr, a.eps, y);
  bool doubt = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool odd = i & 1;
    const float uc = odd ? f.uc[i / 2].y : f.uc[i / 2].x, vs = odd ? f.vs[i / 2].y : f.vs[i / 2].x;
    const float vc = odd ? f.vc[i / 2].y : f.vc[i / 2].x, us = odd ? f.us[i / 2].y : f.us[i / 2].x;
    doubt |= near_border(y.u[i], (fabsf(x.u[i] * uc) + fabsf(x.v[i] * vs)) * r);
    doubt |= near_border(y.v[i], (fabsf(x.v[i] * vc) + fabsf(x.u[i] * us)) * r);
  }
  if (__any_sync(0xffffffffu, doubt)) return key_exact<D, INTER>(x, row, a.rot, at, a.k_weight, a.eps);
  return rounded<INTER>(y);
}

// The table row of a token's position; a position outside the table is
// reported and uses the nearest row.
__device__ __forceinline__ const float* table_row(const RopeArgs& a, int pos, int s, bool report) {
  if (pos < 0 || pos >= a.table_rows) {
    if (report) set_error(a.status, kDevInvalidArg, s, -1, 2);
    pos = pos < 0 ? 0 : a.table_rows - 1;
  }
  return a.table + (int64_t)pos * a.rot;
}

// ---------------------------------------------------------------- one token per sequence
// A group of D/8 lanes per (sequence, head); the heads of a token are its
// queries, keys and values in the projection's order.  Bound by latency: the
// position, the angles and one head's arithmetic in a row, 2.0 us; for 64
// sequences of 48 heads 2.9 us.
template <int D, typename T, bool INTER>
__global__ void __launch_bounds__(128) rope_step_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LPH = D / 8;
  const int lane = threadIdx.x & 31;
  const int heads = a.Hq + 2 * a.Hkv, items = a.B * heads;
  const int raw_item = (blockIdx.x * blockDim.x + threadIdx.x) / LPH;
  const int item = min(raw_item, items - 1);  // lanes behind the last item repeat it and store nothing
  const int s = item / heads, h = item % heads;
  const Place at = place<D, INTER>(lane & (LPH - 1), a.rot);
  Raw<T> raw;
  raw.load(reinterpret_cast<const T*>(a.qkv) + (int64_t)s * a.stride + h * D, at, true);
  const int pos = a.positions ? __ldg(a.positions + s) : __ldcg(a.seq_len + s);
  const float* row = table_row(a, pos, s, raw_item < items && h == 0 && (lane & (LPH - 1)) == 0);
  const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hkv;
  const Pairs x = raw.template pairs<INTER>();
  const Factors f = factors(weights<INTER>(is_q ? a.q_weight : a.k_weight, at), angles(row, a.rot, at));
  // every lane of the warp takes the same shuffles, whatever its head is
  Pairs y;
  uint4 z;
  if (__any_sync(0xffffffffu, is_q)) turn_head<D>(x, f, a.q_weight != nullptr, a.eps, y);
  if (__any_sync(0xffffffffu, is_k)) z = turn_key<D, INTER>(x, f, row, a, at);
  if (raw_item >= items) return;
  if (is_q) put_query<INTER>(a, ((int64_t)s * a.Hq + h) * D, at, y);
  else if (is_k) put(a.k_new + ((int64_t)s * a.Hkv + h - a.Hq) * D, at, z);
  else put(a.v_new + ((int64_t)s * a.Hkv + h - a.Hq - a.Hkv) * D, at, raw.bf16());
}

// ---------------------------------------------------------------- many tokens
// Eight coordinates of a token from a block's codes, rounded to bf16.
template <int KV>
__device__ __forceinline__ uint4 dequantised(const uint8_t* p, const Place& at, float scale) {
  const float4 x = Codes<KV>::unpack(__ldcg(reinterpret_cast<const uint32_t*>(p + at.a)));
  const float4 y = Codes<KV>::unpack(__ldcg(reinterpret_cast<const uint32_t*>(p + at.b)));
  return make_uint4(round2(x.x * scale, x.y * scale), round2(x.z * scale, x.w * scale), round2(y.x * scale, y.y * scale),
                    round2(y.z * scale, y.w * scale));
}

// One CTA per 16-token cache block that receives tokens and `hc` KV heads with
// their query heads.  A warp has 32 / (D/8) tokens and goes through the heads,
// kBatch of them in flight, so that a token's factors are formed once and stay
// in registers; the stored keys and values also go to shared memory, the
// block's earlier tokens with them, and from there the warps form the
// summaries.  Bound by DRAM and the latency in front of it: 32K tokens of 48
// heads of 128 move 0.84 GB in 166 us, 0.74 of the copy rate (1.24 GB from an fp32
// projection in 231 us, 0.79); 4096 tokens take 31 us, 0.51.  In 8 bits 0.75 GB in
// 178 us, 0.62: as many loads and stores in flight, and 14 % more instructions.
constexpr int kBatch = 4;
template <int D, typename T, bool INTER, int KV>
__global__ void __launch_bounds__(256, 3) rope_prefill_kernel(const __grid_constant__ RopePrefillArgs g, int hc, bool ahead) {
  const RopeArgs& a = g.rope;
  constexpr int LPH = D / 8, TPW = 32 / LPH, WT = kBlock / TPW, TEAMS = 8 / WT;
  extern __shared__ __align__(16) __nv_bfloat16 tiles[];  // [K, V][hc][16][D]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = 0;
  while (s + 1 < a.B && g.item0[s + 1] <= (int)blockIdx.x) ++s;
  const int b = g.starts[s] / kBlock + ((int)blockIdx.x - g.item0[s]);
  const int lo = max(g.starts[s] - b * kBlock, 0);                     // slots of this block that receive tokens:
  const int hi = min(g.starts[s] + g.counts[s] - b * kBlock, kBlock);  // [lo, hi)
  const int kv0 = blockIdx.y * hc, kvn = min(hc, a.Hkv - kv0);
  if ((int)blockIdx.x == g.item0[s] && blockIdx.y == 0 && threadIdx.x == 0) a.seq_len[s] = g.starts[s] + g.counts[s];

  const int j = warp % WT * TPW + lane / LPH, team = warp / WT;  // this lane's token; warps of a team share heads
  const bool live = j >= lo && j < hi;
  const int64_t tok = (int64_t)g.token0[s] + b * kBlock - g.starts[s] + j;
  const int pos = !live ? 0 : a.positions ? __ldg(a.positions + tok) : b * kBlock + j;
  const float* row = table_row(a, pos, s, live && blockIdx.y == 0 && team == 0 && (lane & (LPH - 1)) == 0);
  const Place at = place<D, INTER>(lane & (LPH - 1), a.rot);
  const T* src = reinterpret_cast<const T*>(a.qkv) + tok * a.stride;
  // the token's heads start on their way to L2 together; the batches below then wait for L2 alone
  if (ahead && live && (lane & (LPH - 1)) == 0 && team == 0) {
    const int G = a.Hq / a.Hkv;
    prefetch_l2(src + (a.Hq + kv0) * D, kvn * D * sizeof(T));
    prefetch_l2(src + (a.Hq + a.Hkv + kv0) * D, kvn * D * sizeof(T));
    prefetch_l2(src + kv0 * G * D, kvn * G * D * sizeof(T));
  }

  {
    const int G = a.Hq / a.Hkv, nq = kvn * G;
    const T* q = src + kv0 * G * D;
    const int64_t out = (tok * a.Hq + kv0 * G) * D;
    const Factors f = factors(weights<INTER>(a.q_weight, at), angles(row, a.rot, at));
    for (int i0 = team; i0 < nq; i0 += kBatch * TEAMS) {
      Raw<T> raw[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) raw[u].load(q + (i0 + u * TEAMS) * D, at, live && i0 + u * TEAMS < nq);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (i0 + u * TEAMS >= nq) break;
        Pairs y;
        turn_head<D>(raw[u].template pairs<INTER>(), f, a.q_weight != nullptr, a.eps, y);
        if (live) put_query<INTER>(a, out + (i0 + u * TEAMS) * D, at, y);
      }
    }
  }
  {
    const T* k = src + (a.Hq + kv0) * D;
    const T* v = k + a.Hkv * D;
    const Factors f = factors(weights<INTER>(a.k_weight, at), angles(row, a.rot, at));
    const int64_t first = (g.seq_row0[s] + (int64_t)kv0 * g.cap_blocks[s] + b) * kBlock + j, step = (int64_t)g.cap_blocks[s] * kBlock;
#pragma unroll 1
    for (int h = team; h < kvn; h += TEAMS) {
      Raw<T> rk, rv;
      rk.load(k + h * D, at, live);
      rv.load(v + h * D, at, live);
      uint4 x = make_uint4(0, 0, 0, 0), y = x;
      const int64_t slot = (first + h * step) * D;
      if constexpr (KV == kKvBf16) {
        if (j < lo) {
          const __nv_bfloat16 *kd = a.k + slot, *vd = a.v + slot;
          const uint2 xa = __ldcg(reinterpret_cast<const uint2*>(kd + at.a)), xb = __ldcg(reinterpret_cast<const uint2*>(kd + at.b));
          const uint2 ya = __ldcg(reinterpret_cast<const uint2*>(vd + at.a)), yb = __ldcg(reinterpret_cast<const uint2*>(vd + at.b));
          x = make_uint4(xa.x, xa.y, xb.x, xb.y);
          y = make_uint4(ya.x, ya.y, yb.x, yb.y);
        }
      } else if (j < lo) {
        const int unit = s * a.Hkv + kv0 + h, place = tail_place(g.kv8, unit, b, lo);
        if (place >= 0) {
          const __nv_bfloat16 *kd = tail_at<D>(g.kv8, unit, place) + j * D, *vd = kd + kBlock * D;
          const uint2 xa = __ldcg(reinterpret_cast<const uint2*>(kd + at.a)), xb = __ldcg(reinterpret_cast<const uint2*>(kd + at.b));
          const uint2 ya = __ldcg(reinterpret_cast<const uint2*>(vd + at.a)), yb = __ldcg(reinterpret_cast<const uint2*>(vd + at.b));
          x = make_uint4(xa.x, xa.y, xb.x, xb.y);
          y = make_uint4(ya.x, ya.y, yb.x, yb.y);
        } else {
          x = dequantised<KV>(g.kv8.k + slot, at, __ldcg(g.kv8.kscale + slot / (kBlock * D)));
          y = dequantised<KV>(g.kv8.v + slot, at, __ldcg(g.kv8.vscale + slot / (kBlock * D)));
        }
      }
      const uint4 z = turn_key<D, INTER>(rk.template pairs<INTER>(), f, row, a, at);
      if (live) {
        x = z;
        y = rv.bf16();
        if constexpr (KV == kKvBf16) {
          put(a.k + slot, at, x);
          put(a.v + slot, at, y);
        }
      }
      put(tiles + (h * kBlock + j) * D, at, x);
      put(tiles + ((hc + h) * kBlock + j) * D, at, y);
    }
  }
  // The tail's place for this block's tokens.  The CTA of the call's last block takes 0 -- or 2, where the CTA of its first
  // block may be reading 0, or the block already stands there -- and empties the other one if it holds a block behind the
  // first; the CTA of the first block puts it into 1 if the call begins inside it, and empties what else holds it.  A call
  // that begins inside a block and ends there keeps it in 1 or takes 2: one token after another makes its new blocks in 0,
  // and what an earlier call began inside stays in 1.
  __shared__ int keep[4];
  const int begin = g.starts[s] / kBlock, last = (g.starts[s] + g.counts[s] - 1) / kBlock;
  int* len = KV == kKvBf16 ? nullptr : g.kv8.tail_len + kTails * (s * a.Hkv + kv0 + (int)threadIdx.x);
  if (KV != kKvBf16 && threadIdx.x < kvn) {
    const bool two = begin == last ? lo > 0 || tail_in(__ldcg(len + 2), b) : tail_in(__ldcg(len), begin);
    const bool one = b == begin && lo > 0 && (begin < last || tail_in(__ldcg(len + 1), b));
    keep[threadIdx.x] = one ? 1 : b == last ? (two ? 2 : 0) : -1;
  }
  __syncthreads();
  if (KV != kKvBf16 && threadIdx.x < kvn && (b == begin || b == last)) {
    const int to = keep[threadIdx.x];
#pragma unroll
    for (int i = 0; i < kTails; ++i) {
      const int had = __ldcg(len + i);
      const bool gone = begin == last ? had > b * kBlock : b == last ? i == 2 - to && had > (begin + 1) * kBlock
                                                         : i == 1 ? had > b * kBlock : tail_in(had, b);
      if (i == to) len[i] = b * kBlock + hi;
      else if (gone) len[i] = 0;
    }
  }
#pragma unroll 1
  for (int i = warp; i < 2 * kvn; i += 8) {
    const bool is_k = i < kvn;
    const int h = is_k ? i : i - kvn;
    const int64_t r = g.seq_row0[s] + (int64_t)(kv0 + h) * g.cap_blocks[s] + b;
    const __nv_bfloat16* tile = tiles + ((is_k ? 0 : hc) + h) * kBlock * D;
    tile_summary<D, KV>(tile, hi, (is_k ? a.kbar : a.vbar) + r * D, is_k ? a.dbar + r * a.r : nullptr, a.r,
                        {(is_k ? g.kv8.k : g.kv8.v) + r * kBlock * D, (is_k ? g.kv8.kscale : g.kv8.vscale) + r}, lane);
    if (KV != kKvBf16 && keep[h] >= 0) {
      uint32_t* to = reinterpret_cast<uint32_t*>(tail_at<D>(g.kv8, s * a.Hkv + kv0 + h, keep[h]) + (is_k ? 0 : kBlock * D));
#pragma unroll 4
      for (int x = lane; x < hi * (D / 2); x += 32) to[x] = reinterpret_cast<const uint32_t*>(tile)[x];
    }
  }
}

// Calls fn with the compile-time form of (d, type of the projection, kind of pairs).
template <class F>
cudaError_t form(const RopeArgs& a, F&& fn) {
  auto pairs = [&](auto d, auto t) {
    return a.interleaved ? fn(d, t, std::true_type()) : fn(d, t, std::false_type());
  };
  auto type = [&](auto d) { return a.in_f32 ? pairs(d, float()) : pairs(d, __nv_bfloat16()); };
  return a.d == 128 ? type(std::integral_constant<int, 128>()) : type(std::integral_constant<int, 64>());
}

}  // namespace

cudaError_t launch_rope_step(const RopeArgs& a, cudaStream_t st) {
  const int64_t threads = (int64_t)a.B * (a.Hq + 2 * a.Hkv) * (a.d / 8);
  const unsigned grid = (unsigned)((threads + 127) / 128);
  return form(a, [&](auto d, auto t, auto inter) {
    rope_step_kernel<decltype(d)::value, decltype(t), decltype(inter)::value><<<grid, 128, 0, st>>>(a);
    return cudaGetLastError();
  });
}

cudaError_t launch_rope_prefill(const RopePrefillArgs& g, int sms, cudaStream_t st) {
  const RopeArgs& a = g.rope;
  const int blocks = g.item0[a.B];
  if (!blocks) return cudaSuccess;
  // KV heads of a CTA: four read a token's angles once for all of them and leave room for three CTAs on a
  // multiprocessor; fewer where that would not give every multiprocessor eight (32K tokens: 164 us with four, 205
  // with one; 2500 tokens with 80 heads: 34 with two, 29 with one)
  int hc = a.Hkv < 4 ? a.Hkv : 4;
  while (hc > 1 && (int64_t)blocks * ((a.Hkv + hc - 1) / hc) < 8 * sms) hc = (hc + 1) / 2;
  const dim3 grid(blocks, (a.Hkv + hc - 1) / hc);
  const size_t smem = (size_t)2 * hc * kBlock * a.d * 2;
  // the prefetch pays where DRAM is the limit (32K tokens 170 -> 164 us) and costs where one wave of CTAs does it
  // all (200 tokens 5.7 -> 6.3 us)
  const bool ahead = (int64_t)grid.x * grid.y > 8 * sms;
  return form(a, [&](auto d, auto t, auto inter) {
    constexpr int D = decltype(d)::value;
    constexpr bool I = decltype(inter)::value;
    using T = decltype(t);
    switch (g.kv8.type) {
      case kKvInt8: rope_prefill_kernel<D, T, I, kKvInt8><<<grid, 256, smem, st>>>(g, hc, ahead); break;
      case kKvE4m3: rope_prefill_kernel<D, T, I, kKvE4m3><<<grid, 256, smem, st>>>(g, hc, ahead); break;
      default: rope_prefill_kernel<D, T, I, kKvBf16><<<grid, 256, smem, st>>>(g, hc, ahead);
    }
    return cudaGetLastError();
  });
}

}  // namespace compkv
