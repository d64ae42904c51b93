// Norms of the query and key heads and the position rotation in one pass over
// the fused projection's output: for one token per sequence (the inputs of a
// decode step) and for many (queries out, keys and values packed into the
// cache, and the block summaries of section "무엇과 다른가" formed on the way).
//
//   y = w x / sqrt(mean(x^2) + eps)              (skipped without a weight)
//   (a, b) -> (a cos - b sin, b cos + a sin)     for each pair of the first
//                                                rot_dim coordinates
//
// A head is held by D/8 lanes, 8 coordinates each: one 16-byte load of bf16.
//
// Queries are computed in fp32.  Keys are computed as unevaluated sums of two
// floats, so that the fp32 value that is then rounded to bf16 is the nearest
// one: the summaries are those of the stored keys, and a key that falls on the
// wrong side of a rounding border moves its block's mean and variance by a
// bf16 step, some thousand times more than the fp32 arithmetic of the summary
// itself loses.
#include "compkv_launch.h"

namespace compkv {

namespace {

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

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float* x) {
  const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float* x) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

__device__ __forceinline__ uint32_t pack2(__nv_bfloat16 a, __nv_bfloat16 b) {
  return (uint32_t)__bfloat16_as_ushort(a) | ((uint32_t)__bfloat16_as_ushort(b) << 16);
}
__device__ __forceinline__ uint4 pack8(const __nv_bfloat16* y) {
  return make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
}

// Where a lane's pairs are: `l` is its place among the D/8 lanes of a head.
struct Pairing {
  bool rotated;    // its coordinates are among the first rot_dim
  bool first;      // half-split pairs: it holds the first coordinate of its pairs
  int partner;     // half-split pairs: the warp lane that holds the other coordinate
  int col;         // column of its first angle in the table's cos part
};
template <int LPH>
__device__ __forceinline__ Pairing pairing(int lane, int rot, int interleaved) {
  const int l = lane & (LPH - 1);
  Pairing p;
  p.rotated = 8 * l < rot;
  const int half = rot / 16;  // lanes of half a rotation
  p.first = l < half;
  p.partner = interleaved || !p.rotated ? lane : (p.first ? lane + half : lane - half);
  p.col = interleaved ? 4 * l : 8 * (p.first ? l : l - half);
  return p;
}

// One head's 8 coordinates of this lane, normed and rotated, in fp32.
template <int D>
__device__ __forceinline__ void head_f32(float* x, const float* w, const float* row, const RopeArgs& a, Pairing p) {
  constexpr int LPH = D / 8;
  if (w) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float r = rsqrtf(s * (1.f / D) + a.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
  }
  if (a.interleaved) {
    if (p.rotated) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float c = row[p.col + i], s = row[a.rot / 2 + p.col + i];
        const float u = x[2 * i], v = x[2 * i + 1];
        x[2 * i] = u * c - v * s;
        x[2 * i + 1] = v * c + u * s;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_sync(0xffffffffu, x[i], p.partner);
      if (p.rotated) {
        const float c = row[p.col + i], s = row[a.rot / 2 + p.col + i];
        x[i] = p.first ? x[i] * c - other * s : x[i] * c + other * s;
      }
    }
  }
}

// u c + v s' (s' = s or -s) of two-float u, v.
__device__ __forceinline__ F2 turn2(F2 u, float c, F2 v, float s) {
  F2 p = two_prod(u.hi, c), q = two_prod(v.hi, s);
  p.lo = __fmaf_rn(u.lo, c, p.lo);
  q.lo = __fmaf_rn(v.lo, s, q.lo);
  return add2(p, q);
}

// 1 / sqrt(mean(x^2) + eps) of the head whose coordinates these lanes hold, in two floats: one step of Newton's
// iteration on rsqrtf with its residual 1 - m r^2 in two floats.
template <int D>
__device__ __forceinline__ F2 inverse_norm(const float* x, float eps) {
  F2 s = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 8; ++i) s = add2(s, two_prod(x[i], x[i]));
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1)
    s = add2(s, {__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
  s.hi *= 1.f / D;  // exact: D is a power of two
  s.lo *= 1.f / D;
  const F2 m = add2(s, {eps, 0.f});
  const float r0 = rsqrtf(m.hi);
  const F2 h = two_prod(m.hi, r0);
  const float e = __fmaf_rn(-h.hi, r0, 1.f) - (h.lo + m.lo * r0) * r0;
  return {r0, isfinite(r0) ? 0.5f * r0 * e : 0.f};
}
// x w r
__device__ __forceinline__ F2 scaled(float x, float w, F2 r) {
  const F2 t = two_prod(x, w);
  F2 y = two_prod(t.hi, r.hi);
  y.lo = __fmaf_rn(t.hi, r.lo, __fmaf_rn(t.lo, r.hi, y.lo));
  return y;
}

// The same with two floats per value, rounded to fp32 and then to bf16.
template <int D>
__device__ __forceinline__ void head_bf16(const float* x, const float* w, const float* row, const RopeArgs& a,
                                          Pairing p, __nv_bfloat16* out) {
  F2 y[8];
  if (w) {
    const F2 r = inverse_norm<D>(x, a.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = scaled(x[i], w[i], r);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = {x[i], 0.f};
  }
  if (a.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (p.rotated) {
        const float c = row[p.col + i], s = row[a.rot / 2 + p.col + i];
        const F2 u = y[2 * i], v = y[2 * i + 1];
        y[2 * i] = turn2(u, c, v, -s);
        y[2 * i + 1] = turn2(v, c, u, s);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const F2 other = {__shfl_sync(0xffffffffu, y[i].hi, p.partner), __shfl_sync(0xffffffffu, y[i].lo, p.partner)};
      if (p.rotated) {
        const float c = row[p.col + i], s = row[a.rot / 2 + p.col + i];
        y[i] = turn2(y[i], c, other, p.first ? -s : s);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = __float2bfloat16_rn(__fadd_rn(y[i].hi, y[i].lo));
}

__device__ __forceinline__ void weights8(const float* w, int l, float* out) {
  if (w) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w) + 2 * l), b = __ldg(reinterpret_cast<const float4*>(w) + 2 * l + 1);
    out[0] = a.x; out[1] = a.y; out[2] = a.z; out[3] = a.w;
    out[4] = b.x; out[5] = b.y; out[6] = b.z; out[7] = b.w;
  }
}

__device__ __forceinline__ void store_q(const RopeArgs& a, int64_t at, const float* x) {
  if (a.q_bf16) {
    __nv_bfloat16 y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __float2bfloat16_rn(x[i]);
    __stcs(reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.q) + at), pack8(y));
  } else {
    float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.q) + at);
    __stcs(q, make_float4(x[0], x[1], x[2], x[3]));
    __stcs(q + 1, make_float4(x[4], x[5], x[6], x[7]));
  }
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

// One token per sequence.  A group of D/8 lanes per (sequence, head); the
// heads of a token are its queries, keys and values in the projection's order.
template <int D, typename T>
__global__ void __launch_bounds__(128) rope_step_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LPH = D / 8;
  const int lane = threadIdx.x & 31, l = lane & (LPH - 1);
  const int heads = a.Hq + 2 * a.Hkv, items = a.B * heads;
  const int raw = (blockIdx.x * blockDim.x + threadIdx.x) / LPH;
  const int item = raw < items ? raw : items - 1;  // lanes behind the last item repeat it and store nothing
  const int s = item / heads, h = item % heads;
  const Pairing p = pairing<LPH>(lane, a.rot, a.interleaved);
  const int pos = a.positions ? __ldg(a.positions + s) : __ldcg(a.seq_len + s);
  float x[8], w[8];
  load8<T>(reinterpret_cast<const T*>(a.qkv) + (int64_t)s * a.stride + h * D + 8 * l, x);
  const float* row = table_row(a, pos, s, raw < items && h == 0 && l == 0);
  // every lane of the warp takes the same shuffles, whatever its head is
  const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hkv;
  const float* wt = is_q ? a.q_weight : a.k_weight;
  weights8(wt, l, w);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[i];
  __nv_bfloat16 z[8];
  if (__any_sync(0xffffffffu, is_q)) head_f32<D>(y, a.q_weight ? w : nullptr, row, a, p);
  if (__any_sync(0xffffffffu, is_k)) head_bf16<D>(x, a.k_weight ? w : nullptr, row, a, p, z);
  if (raw >= items) return;
  if (is_q) {
    store_q(a, ((int64_t)s * a.Hq + h) * D + 8 * l, y);
  } else if (is_k) {
    *reinterpret_cast<uint4*>(a.k_new + ((int64_t)s * a.Hkv + h - a.Hq) * D + 8 * l) = pack8(z);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = __float2bfloat16_rn(x[i]);
    *reinterpret_cast<uint4*>(a.v_new + ((int64_t)s * a.Hkv + h - a.Hq - a.Hkv) * D + 8 * l) = pack8(z);
  }
}

// Many tokens: a lane's part of one token's rotation, the same for all heads.
//   y_i = x_i cos_i + o_i sin_i,  o_i the other coordinate of the pair, the sign in sin_i
template <int D>
struct Turn {
  float c[8], s[8];
  int partner;   // the lane that holds the o_i; interleaved pairs are in the lane itself
  bool inside;   // interleaved
  __device__ __forceinline__ Turn(const RopeArgs& a, const float* row, int lane) {
    const Pairing p = pairing<D / 8>(lane, a.rot, a.interleaved);
    partner = p.partner;
    inside = a.interleaved;
    if (!p.rotated) {
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
    } else if (inside) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(row + p.col));
      const float4 v = __ldg(reinterpret_cast<const float4*>(row + a.rot / 2 + p.col));
      const float cc[4] = {u.x, u.y, u.z, u.w}, ss[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[2 * i] = c[2 * i + 1] = cc[i];
        s[2 * i] = -ss[i];
        s[2 * i + 1] = ss[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(row + p.col) + i);
        const float4 v = __ldg(reinterpret_cast<const float4*>(row + a.rot / 2 + p.col) + i);
        const float sign = p.first ? -1.f : 1.f;
        c[4 * i] = u.x, c[4 * i + 1] = u.y, c[4 * i + 2] = u.z, c[4 * i + 3] = u.w;
        s[4 * i] = sign * v.x, s[4 * i + 1] = sign * v.y, s[4 * i + 2] = sign * v.z, s[4 * i + 3] = sign * v.w;
      }
    }
  }
  // Weights of this lane's coordinates and of their partners.
  __device__ __forceinline__ void weights(const float* w, int lane, float* own, float* other) const {
    weights8(w, lane & (D / 8 - 1), own);
    if (inside) {
#pragma unroll
      for (int i = 0; i < 8; ++i) other[i] = own[i ^ 1];
    } else {
      weights8(w, partner & (D / 8 - 1), other);
    }
  }
};

// 8 coordinates as they come.
template <typename T>
struct Raw {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p, bool live) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      v[i] = live ? __ldcs(reinterpret_cast<const uint4*>(p) + i) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ Raw from(int lane) const {
    Raw r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      r.v[i].x = __shfl_sync(0xffffffffu, v[i].x, lane);
      r.v[i].y = __shfl_sync(0xffffffffu, v[i].y, lane);
      r.v[i].z = __shfl_sync(0xffffffffu, v[i].z, lane);
      r.v[i].w = __shfl_sync(0xffffffffu, v[i].w, lane);
    }
    return r;
  }
  __device__ __forceinline__ void floats(float* x) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (sizeof(T) == 2) {
          x[2 * k] = __uint_as_float(w[k] << 16);
          x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        } else {
          x[4 * i + k] = __uint_as_float(w[k]);
        }
      }
    }
  }
};

// The lane's coordinates and their partners'.
template <int D, typename T>
__device__ __forceinline__ void pairs(const Raw<T>& raw, const Turn<D>& t, float* x, float* o) {
  raw.floats(x);
  if (t.inside) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = x[i ^ 1];
  } else {
    raw.from(t.partner).floats(o);  // the values as they came: half the exchanges of the normed ones
  }
}

// Summary of a block from its tokens in shared memory, by one warp: mean of
// the first n tokens and, for keys, the grouped mean of the population
// variances, both in two passes over registers and in the order of
// warp_block_summary, with the same results.
template <int D>
__device__ __forceinline__ void tile_summary(const __nv_bfloat16* tile, int n, float* bar, float* dbar, int r, int lane) {
  constexpr int V = D / 32;
  float t[kBlock][V], mean[V] = {};
#pragma unroll
  for (int j = 0; j < kBlock; ++j) {
    if (j < n) {
      if (V == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(tile + j * D + lane * V);
        t[j][0] = __uint_as_float(u.x << 16);
        t[j][1] = __uint_as_float(u.x & 0xffff0000u);
        t[j][V - 2] = __uint_as_float(u.y << 16);
        t[j][V - 1] = __uint_as_float(u.y & 0xffff0000u);
      } else {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(tile + j * D + lane * V);
        t[j][0] = __uint_as_float(u << 16);
        t[j][1] = __uint_as_float(u & 0xffff0000u);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) mean[i] += t[j][i];
    }
  }
  const float fn = (float)n;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    mean[i] = mean[i] / fn;
    bar[lane * V + i] = mean[i];
  }
  if (!dbar) return;
  float var[V] = {};
#pragma unroll
  for (int j = 0; j < kBlock; ++j)
    if (j < n) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float dlt = t[j][i] - mean[i];
        var[i] = fmaf(dlt, dlt, var[i]);
      }
    }
#pragma unroll
  for (int i = 0; i < V; ++i) var[i] = var[i] / fn;
  const int gs = D / r;
  if (gs >= V) {
    const int lpg = gs / V;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) x += var[i];
    for (int o = lpg >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if ((lane & (lpg - 1)) == 0) dbar[lane / lpg] = x / (float)gs;
  } else if (gs == 2) {
#pragma unroll
    for (int i = 0; i < V; i += 2) dbar[(lane * V + i) / 2] = (var[i] + var[i + 1]) / 2.f;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) dbar[lane * V + i] = var[i];
  }
}

// One CTA per 16-token cache block that receives tokens and `hc` KV heads with
// their query heads.  A warp has 32 / (D/8) tokens and goes through the heads,
// kBatch of them in flight, so that a token's angles are read once and stay in
// registers; the stored keys and values also go to shared memory, the block's
// earlier tokens with them, and from there the warps form the summaries.
// Bound by DRAM: 32K tokens x 48 heads of 128 move 0.84 GB.
constexpr int kBatch = 4;
template <int D, typename T>
__global__ void __launch_bounds__(256) rope_prefill_kernel(const __grid_constant__ RopePrefillArgs g, int hc) {
  const RopeArgs& a = g.rope;
  constexpr int LPH = D / 8, TPW = 32 / LPH, WT = kBlock / TPW, TEAMS = 8 / WT;
  extern __shared__ __align__(16) __nv_bfloat16 tiles[];  // [K, V][hc][16][D]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & (LPH - 1);
  int s = 0;
  while (s + 1 < a.B && g.item0[s + 1] <= (int)blockIdx.x) ++s;
  const int b = g.starts[s] / kBlock + ((int)blockIdx.x - g.item0[s]);
  const int lo = max(g.starts[s] - b * kBlock, 0);                     // slots of this block that receive tokens:
  const int hi = min(g.starts[s] + g.counts[s] - b * kBlock, kBlock);  // [lo, hi)
  const int kv0 = blockIdx.y * hc, kvn = min(hc, a.Hkv - kv0);
  if ((int)blockIdx.x == g.item0[s] && blockIdx.y == 0 && threadIdx.x == 0) a.seq_len[s] = g.starts[s] + g.counts[s];

  const int j = warp % WT * TPW + lane / LPH;  // this lane's token
  const bool live = j >= lo && j < hi;
  const int64_t tok = (int64_t)g.token0[s] + b * kBlock - g.starts[s] + j;
  const int pos = !live ? 0 : a.positions ? __ldg(a.positions + tok) : b * kBlock + j;
  const Turn<D> turn(a, table_row(a, pos, s, live && blockIdx.y == 0 && warp < WT && l == 0), lane);

  // the CTA's heads: kvn G query heads, kvn key heads, kvn value heads; a team of warps takes every TEAMS-th
  const int G = a.Hq / a.Hkv, nq = kvn * G, heads = nq + 2 * kvn, team = warp / WT;
  const T* src = reinterpret_cast<const T*>(a.qkv) + tok * a.stride + 8 * l;
  auto column = [&](int i) {
    return i < nq ? kv0 * G + i : i < nq + kvn ? a.Hq + kv0 + i - nq : a.Hq + a.Hkv + kv0 + i - nq - kvn;
  };
  Raw<T> next[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int i = team + u * TEAMS;
    next[u].load(src + column(i) * D, live && i < heads);
  }
  float w[8], wo[8];
  const float* weight = a.q_weight;
  if (weight) turn.weights(weight, lane, w, wo);
  bool keys = false;
  for (int i0 = team; i0 < heads; i0 += kBatch * TEAMS) {
    Raw<T> raw[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) raw[u] = next[u];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + (kBatch + u) * TEAMS;
      next[u].load(src + column(i) * D, live && i < heads);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * TEAMS;
      if (i >= heads) break;
      if (i < nq) {
        float x[8], o[8];
        pairs<D, T>(raw[u], turn, x, o);
        if (weight) {
          float m = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) m = fmaf(x[k], x[k], m);
#pragma unroll
          for (int k = LPH / 2; k > 0; k >>= 1) m += __shfl_xor_sync(0xffffffffu, m, k);
          const float r = rsqrtf(m * (1.f / D) + a.eps);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x[k] = x[k] * r * w[k];
            o[k] = o[k] * r * wo[k];
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = fmaf(x[k], turn.c[k], o[k] * turn.s[k]);
        if (live) store_q(a, (tok * a.Hq + kv0 * G + i) * D + 8 * l, x);
        continue;
      }
      const bool is_k = i < nq + kvn;
      const int h = i - nq - (is_k ? 0 : kvn);
      const int64_t r = g.seq_row0[s] + (int64_t)(kv0 + h) * g.cap_blocks[s] + b;
      uint4* dst = reinterpret_cast<uint4*>((is_k ? a.k : a.v) + (r * kBlock + j) * D + 8 * l);
      uint4 y = make_uint4(0, 0, 0, 0);
      if (j < lo) y = __ldcg(dst);
      if (is_k) {
        if (!keys) {
          keys = true;
          weight = a.k_weight;
          if (weight) turn.weights(weight, lane, w, wo);
        }
        float x[8], o[8];
        pairs<D, T>(raw[u], turn, x, o);
        F2 r2 = {1.f, 0.f};
        if (weight) r2 = inverse_norm<D>(x, a.eps);
        __nv_bfloat16 z[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const F2 p = weight ? scaled(x[k], w[k], r2) : F2{x[k], 0.f}, q = weight ? scaled(o[k], wo[k], r2) : F2{o[k], 0.f};
          const F2 t = turn2(p, turn.c[k], q, turn.s[k]);
          z[k] = __float2bfloat16_rn(__fadd_rn(t.hi, t.lo));
        }
        if (live) y = pack8(z);
      } else if (live) {
        if (sizeof(T) == 2) {
          y = raw[u].v[0];
        } else {
          float x[8];
          __nv_bfloat16 z[8];
          raw[u].floats(x);
#pragma unroll
          for (int k = 0; k < 8; ++k) z[k] = __float2bfloat16_rn(x[k]);
          y = pack8(z);
        }
      }
      if (live) *dst = y;
      *reinterpret_cast<uint4*>(tiles + (((is_k ? 0 : hc) + h) * kBlock + j) * D + 8 * l) = y;
    }
  }
  __syncthreads();
  for (int i = warp; i < 2 * kvn; i += 8) {
    const bool is_k = i < kvn;
    const int h = is_k ? i : i - kvn;
    const int64_t r = g.seq_row0[s] + (int64_t)(kv0 + h) * g.cap_blocks[s] + b;
    tile_summary<D>(tiles + ((is_k ? 0 : hc) + h) * kBlock * D, hi, (is_k ? a.kbar : a.vbar) + r * D,
                    is_k ? a.dbar + r * a.r : nullptr, a.r, lane);
  }
}

}  // namespace

cudaError_t launch_rope_step(const RopeArgs& a, cudaStream_t st) {
  const int lph = a.d / 8;
  const int64_t threads = (int64_t)a.B * (a.Hq + 2 * a.Hkv) * lph;
  const unsigned grid = (unsigned)((threads + 127) / 128);
  if (a.d == 128) {
    if (a.in_f32) rope_step_kernel<128, float><<<grid, 128, 0, st>>>(a);
    else rope_step_kernel<128, __nv_bfloat16><<<grid, 128, 0, st>>>(a);
  } else {
    if (a.in_f32) rope_step_kernel<64, float><<<grid, 128, 0, st>>>(a);
    else rope_step_kernel<64, __nv_bfloat16><<<grid, 128, 0, st>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_rope_prefill(const RopePrefillArgs& g, int sms, cudaStream_t st) {
  const RopeArgs& a = g.rope;
  const int blocks = g.item0[a.B];
  if (!blocks) return cudaSuccess;
  // KV heads of a CTA: four read a token's angles once for all of them and leave room for several CTAs on a
  // multiprocessor; fewer where the blocks alone would not give every multiprocessor four
  int hc = a.Hkv < 4 ? a.Hkv : 4;
  while (hc > 1 && (int64_t)blocks * ((a.Hkv + hc - 1) / hc) < 4 * sms) hc = (hc + 1) / 2;
  const dim3 grid(blocks, (a.Hkv + hc - 1) / hc);
  const size_t smem = (size_t)2 * hc * kBlock * a.d * 2;
  if (a.d == 128) {
    if (a.in_f32) rope_prefill_kernel<128, float><<<grid, 256, smem, st>>>(g, hc);
    else rope_prefill_kernel<128, __nv_bfloat16><<<grid, 256, smem, st>>>(g, hc);
  } else {
    if (a.in_f32) rope_prefill_kernel<64, float><<<grid, 256, smem, st>>>(g, hc);
    else rope_prefill_kernel<64, __nv_bfloat16><<<grid, 256, smem, st>>>(g, hc);
  }
  return cudaGetLastError();
}

}  // namespace compkv
