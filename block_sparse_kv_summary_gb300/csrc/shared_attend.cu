// Exact attention of every sequence over a prefix that one sequence of the
// cache holds for all and over its own tokens, under one softmax:
//   out = sum_j e^(z_j) v_j / sum_j e^(z_j),   z_j = q . k_j / sqrt(d),
// j over the prefix's tokens and the sequence's own.
//
// Plain kernels: one warp per (query head, sequence, key split) with a running
// maximum and sum, then one warp per query head joins the splits.
#include "compkv_launch.h"

namespace compkv {

namespace {

constexpr int kSplits = 32;

template <int D>
__global__ void __launch_bounds__(256) shared_split_kernel(const __grid_constant__ SharedArgs a) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const int Hq = a.Hkv * a.G;
  const int item = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (item >= a.B * Hq * kSplits) return;
  const int split = item % kSplits, hq = item / kSplits % Hq, s = item / kSplits / Hq, h = hq / a.G;
  const int p = a.prefix_seq[s];
  if (p == -2) return;
  auto held = [&](int x) { return max(0, min(__ldcg(a.seq_len + x), a.cap_blocks[x] * kBlock)); };
  int np = 0;
  if (p >= 0) {
    np = min(a.prefix_len[p], held(p));
    if (np < a.prefix_len[p] && lane == 0) set_error(a.status, kDevInvalidArg, p, h, 5);
  }
  const int own0 = p == s ? np : 0, no = max(0, held(s) - own0), n = np + no;
  const int64_t q0 = ((int64_t)s * Hq + hq) * D + lane * V;
  float q[V], o[V] = {}, m = -INFINITY, l = 0.f;
  const float scale = 1.f / sqrtf((float)D);
#pragma unroll
  for (int i = 0; i < V; ++i)
    q[i] = scale * (a.q_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.q)[q0 + i])
                             : reinterpret_cast<const float*>(a.q)[q0 + i]);
  const int64_t rp = p < 0 ? 0 : (a.seq_row0[p] + (int64_t)h * a.cap_blocks[p]) * kBlock;
  const int64_t ro = (a.seq_row0[s] + (int64_t)h * a.cap_blocks[s]) * kBlock + own0;
  const int j1 = (int)((int64_t)n * (split + 1) / kSplits);
  for (int j = (int)((int64_t)n * split / kSplits); j < j1; ++j) {
    const int64_t at = ((j < np ? rp + j : ro + j - np)) * D + lane * V;
    float k[V], v[V], z = 0.f;
    load_bf16<V>(a.k + at, k);
    load_bf16<V>(a.v + at, v);
#pragma unroll
    for (int i = 0; i < V; ++i) z = fmaf(q[i], k[i], z);
    z = warp_sum(z);
    const float mn = fmaxf(m, z), f = __expf(m - mn), w = __expf(z - mn);
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = o[i] * f + w * v[i];
    m = mn;
  }
  float* part = a.ws + (int64_t)item * (D + 2);
#pragma unroll
  for (int i = 0; i < V; ++i) part[lane * V + i] = o[i];
  if (lane == 0) {
    part[D] = m;
    part[D + 1] = l;
  }
}

template <int D>
__global__ void __launch_bounds__(256) shared_join_kernel(const __grid_constant__ SharedArgs a) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const int Hq = a.Hkv * a.G;
  const int item = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (item >= a.B * Hq || a.prefix_seq[item / Hq] == -2) return;
  const float* part = a.ws + (int64_t)item * kSplits * (D + 2);
  float m = -INFINITY, l = 0.f, o[V] = {};
  for (int x = 0; x < kSplits; ++x) m = fmaxf(m, part[x * (D + 2) + D]);
  for (int x = 0; x < kSplits && m > -INFINITY; ++x) {
    const float f = __expf(part[x * (D + 2) + D] - m);
    l += f * part[x * (D + 2) + D + 1];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] += f * part[x * (D + 2) + lane * V + i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float y = l > 0.f ? o[i] / l : 0.f;
    if (a.q_bf16) reinterpret_cast<__nv_bfloat16*>(a.out)[(int64_t)item * D + lane * V + i] = __float2bfloat16_rn(y);
    else reinterpret_cast<float*>(a.out)[(int64_t)item * D + lane * V + i] = y;
  }
}

}  // namespace

size_t shared_workspace_bytes(int B, int Hkv, int G, int d) { return (size_t)B * Hkv * G * kSplits * (d + 2) * 4; }

cudaError_t launch_attend_shared(const SharedArgs& a, cudaStream_t st) {
  const int rows = a.B * a.Hkv * a.G;
  if (a.d == 128) {
    shared_split_kernel<128><<<rows * kSplits / 8, 256, 0, st>>>(a);
    shared_join_kernel<128><<<(rows + 7) / 8, 256, 0, st>>>(a);
  } else {
    shared_split_kernel<64><<<rows * kSplits / 8, 256, 0, st>>>(a);
    shared_join_kernel<64><<<(rows + 7) / 8, 256, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace compkv
