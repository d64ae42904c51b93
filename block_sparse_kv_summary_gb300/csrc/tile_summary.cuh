// Summary of a block whose tokens stand in shared memory, and with it, in a
// cache of 8 bits, the block's codes.
#pragma once

#include "kv8.cuh"

namespace compkv {

// Summary of a block from its tokens in shared memory, by one warp: mean of
// the first n tokens and, for keys, the grouped mean of the population
// variances, both in two passes over registers and in the order of
// warp_block_summary, with the same results.
// In 8 bits, the block's codes and scale too, from the same registers.
struct TileCodes {
  uint8_t* codes;
  float* scale;
};
template <int D, int KV>
__device__ __forceinline__ void tile_summary(const __nv_bfloat16* tile, int n, float* bar, float* dbar, int r, TileCodes out,
                                             int lane) {
  constexpr int V = D / 32;
  float2 t[kBlock][V / 2], mean[V / 2] = {};
  __nv_bfloat162 most = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < kBlock; ++j) {
    if (j >= n) break;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(tile + j * D + lane * V);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      t[j][i] = make_float2(__uint_as_float(p[i] << 16), __uint_as_float(p[i] & 0xffff0000u));
      if (KV != kKvBf16) most = __hmax2_nan(most, __habs2(*reinterpret_cast<const __nv_bfloat162*>(p + i)));
      mean[i] = __fadd2_rn(mean[i], t[j][i]);
    }
  }
  const float fn = (float)n;
  auto over = [&](float x) { return n == kBlock ? x * (1.f / kBlock) : x / fn; };  // exact alike for 16
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    mean[i] = make_float2(over(mean[i].x), over(mean[i].y));
    reinterpret_cast<float2*>(bar + lane * V)[i] = mean[i];
  }
  if constexpr (KV != kKvBf16) {
    const uint32_t m = *reinterpret_cast<const uint32_t*>(&most);  // (a NaN has the largest bits)
    const Scale s = Scale::of<KV>(__reduce_max_sync(0xffffffffu, max(m << 16, m & 0xffff0000u)));
    const bool live = !isnan(s.scale);  // (an infinity times zero is a NaN: codes of such a block are set, not computed)
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
      uint32_t c = 0;
      if (j < n && live) {
        const float2 x = t[j][0], y = t[j][V / 2 - 1];
        c = Codes<KV>::pack(make_float2(__fmul_rn(x.x, s.inv), __fmul_rn(x.y, s.inv)),
                            V == 4 ? make_float2(__fmul_rn(y.x, s.inv), __fmul_rn(y.y, s.inv)) : make_float2(0.f, 0.f));
      }
      if constexpr (V == 4) reinterpret_cast<uint32_t*>(out.codes + j * D)[lane] = c;
      else reinterpret_cast<uint16_t*>(out.codes + j * D)[lane] = (uint16_t)c;
    }
    if (lane == 0) *out.scale = s.scale;
  }
  if (!dbar) return;
  float2 v2[V / 2] = {};
#pragma unroll
  for (int j = 0; j < kBlock; ++j) {
    if (j >= n) break;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 dlt = __fadd2_rn(t[j][i], make_float2(-mean[i].x, -mean[i].y));
      v2[i] = __ffma2_rn(dlt, dlt, v2[i]);
    }
  }
  float var[V];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    var[2 * i] = over(v2[i].x);
    var[2 * i + 1] = over(v2[i].y);
  }
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

}  // namespace compkv
