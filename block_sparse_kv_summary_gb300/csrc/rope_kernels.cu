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

// The same with two floats per value, rounded to fp32 and then to bf16.
template <int D>
__device__ __forceinline__ void head_bf16(const float* x, const float* w, const float* row, const RopeArgs& a,
                                          Pairing p, __nv_bfloat16* out) {
  constexpr int LPH = D / 8;
  F2 y[8];
  if (w) {
    F2 s = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i) s = add2(s, two_prod(x[i], x[i]));
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1)
      s = add2(s, {__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
    s.hi *= 1.f / D;  // exact: D is a power of two
    s.lo *= 1.f / D;
    const F2 m = add2(s, {a.eps, 0.f});
    // r = r0 + r1, one step of Newton's iteration on r0 with the residual 1 - m r0^2 in two floats
    const float r0 = rsqrtf(m.hi);
    const F2 h = two_prod(m.hi, r0);
    const float e = __fmaf_rn(-h.hi, r0, 1.f) - (h.lo + m.lo * r0) * r0;
    const float r1 = isfinite(r0) ? 0.5f * r0 * e : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const F2 t = two_prod(x[i], w[i]);
      y[i] = two_prod(t.hi, r0);
      y[i].lo = __fmaf_rn(t.hi, r1, __fmaf_rn(t.lo, r0, y[i].lo));
    }
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

// Sum over the lanes that hold the same coordinates of different tokens.
template <int LPH>
__device__ __forceinline__ float token_sum(float x) {
#pragma unroll
  for (int o = LPH; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Many tokens.  One CTA per 16-token cache block that receives tokens, one
// warp per head and turn: 32 / (D/8) tokens at a time.  Key and value warps
// also read the block's earlier tokens from the cache and form its summary
// (two passes over registers: mean, then squared deviations from it).
template <int D, typename T>
__global__ void __launch_bounds__(256) rope_prefill_kernel(const __grid_constant__ RopePrefillArgs g) {
  const RopeArgs& a = g.rope;
  constexpr int LPH = D / 8, TPW = 32 / LPH, IT = kBlock / TPW;
  const int lane = threadIdx.x & 31, l = lane & (LPH - 1), sub = lane / LPH;
  int s = 0;
  while (s + 1 < a.B && g.item0[s + 1] <= (int)blockIdx.x) ++s;
  const int b = g.starts[s] / kBlock + ((int)blockIdx.x - g.item0[s]);
  const int lo = max(g.starts[s] - b * kBlock, 0);                             // slots of this block that receive tokens:
  const int hi = min(g.starts[s] + g.counts[s] - b * kBlock, kBlock);          // [lo, hi)
  const int64_t tok0 = (int64_t)g.token0[s] + b * kBlock - g.starts[s];        // token of slot 0
  const Pairing p = pairing<LPH>(lane, a.rot, a.interleaved);
  if (blockIdx.x == g.item0[s] && threadIdx.x == 0) a.seq_len[s] = g.starts[s] + g.counts[s];

  const float* row[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int j = i * TPW + sub;
    const bool live = j >= lo && j < hi;
    const int pos = !live ? 0 : a.positions ? __ldg(a.positions + tok0 + j) : b * kBlock + j;
    row[i] = table_row(a, pos, s, live && threadIdx.x < 32 && l == 0);
  }
  const int heads = a.Hq + 2 * a.Hkv;
  for (int h = threadIdx.x >> 5; h < heads; h += blockDim.x >> 5) {
    const T* src = reinterpret_cast<const T*>(a.qkv) + tok0 * a.stride + h * D + 8 * l;
    float w[8];
    if (h < a.Hq) {
      weights8(a.q_weight, l, w);
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int j = i * TPW + sub;
        const bool live = j >= lo && j < hi;
        float x[8] = {};
        if (live) load8<T>(src + j * a.stride, x);
        head_f32<D>(x, a.q_weight ? w : nullptr, row[i], a, p);
        if (live) store_q(a, ((tok0 + j) * a.Hq + h) * D + 8 * l, x);
      }
      continue;
    }
    const bool is_k = h < a.Hq + a.Hkv;
    const int64_t r = g.seq_row0[s] + (int64_t)(is_k ? h - a.Hq : h - a.Hq - a.Hkv) * g.cap_blocks[s] + b;
    __nv_bfloat16* dst = (is_k ? a.k : a.v) + r * kBlock * D + 8 * l;
    if (is_k) weights8(a.k_weight, l, w);
    float t[IT][8], sum[8] = {};
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int j = i * TPW + sub;
      const bool live = j >= lo && j < hi;
      uint4 u = make_uint4(0, 0, 0, 0);
      if (j < lo) u = __ldcg(reinterpret_cast<const uint4*>(dst + j * D));
      float x[8] = {};
      if (live) load8<T>(src + j * a.stride, x);
      __nv_bfloat16 z[8];
      if (is_k) {
        head_bf16<D>(x, a.k_weight ? w : nullptr, row[i], a, p, z);
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) z[c] = __float2bfloat16_rn(x[c]);
      }
      if (live) {
        u = pack8(z);
        __stcs(reinterpret_cast<uint4*>(dst + j * D), u);
      }
      const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        t[i][2 * c] = __uint_as_float(v[c] << 16);
        t[i][2 * c + 1] = __uint_as_float(v[c] & 0xffff0000u);
      }
      if (j < hi) {
#pragma unroll
        for (int c = 0; c < 8; ++c) sum[c] += t[i][c];
      }
    }
    const float n = (float)hi;
#pragma unroll
    for (int c = 0; c < 8; ++c) sum[c] = token_sum<LPH>(sum[c]) / n;
    float* bar = (is_k ? a.kbar : a.vbar) + r * D + 8 * l;
    if (sub == 0) {
      reinterpret_cast<float4*>(bar)[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
      reinterpret_cast<float4*>(bar)[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
    }
    if (!is_k) continue;
    float var[8] = {};
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      if (i * TPW + sub < hi) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float dlt = t[i][c] - sum[c];
          var[c] = fmaf(dlt, dlt, var[c]);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) var[c] = token_sum<LPH>(var[c]) / n;
    const int gs = D / a.r;  // coordinates of a variance group: a power of two
    float* db = a.dbar + r * a.r;
    if (gs >= 8) {
      float sum8 = ((var[0] + var[1]) + (var[2] + var[3])) + ((var[4] + var[5]) + (var[6] + var[7]));
      for (int o = gs / 16; o > 0; o >>= 1) sum8 += __shfl_xor_sync(0xffffffffu, sum8, o);
      if (sub == 0 && l % (gs / 8) == 0) db[l / (gs / 8)] = sum8 / (float)gs;
    } else if (sub == 0) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        // partial sums in place: var[c] of the first coordinate of a group gathers the group
        if (gs >= 2 && (c & 1) == 0) var[c] += var[c + 1];
      }
#pragma unroll
      for (int c = 0; c < 8; c += 4)
        if (gs >= 4) var[c] += var[c + 2];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c % gs == 0) db[(8 * l + c) / gs] = var[c] / (float)gs;
    }
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

cudaError_t launch_rope_prefill(const RopePrefillArgs& g, cudaStream_t st) {
  const RopeArgs& a = g.rope;
  const unsigned grid = (unsigned)g.item0[a.B];
  if (!grid) return cudaSuccess;
  if (a.d == 128) {
    if (a.in_f32) rope_prefill_kernel<128, float><<<grid, 256, 0, st>>>(g);
    else rope_prefill_kernel<128, __nv_bfloat16><<<grid, 256, 0, st>>>(g);
  } else {
    if (a.in_f32) rope_prefill_kernel<64, float><<<grid, 256, 0, st>>>(g);
    else rope_prefill_kernel<64, __nv_bfloat16><<<grid, 256, 0, st>>>(g);
  }
  return cudaGetLastError();
}

}  // namespace compkv
