// A cache in 8 bits: one token per sequence appended, and tokens read back
// (also from a cache in bf16).  Many tokens are written by rope_kernels.cu.
#include "compkv_launch.h"
#include "kv8.cuh"
#include "tile_summary.cuh"

namespace compkv {

namespace {

// One CTA per sequence, a warp for K and one for V of eight heads at a time.
// Token L (L = seq_len) joins the tokens of its block, which the tail holds in
// bf16; the block's summary and codes are formed again from all of them, so that
// a block's contents do not depend on how its tokens arrived.  A block goes on in
// the place of the tail that it stands in, and a new one takes place 0, so that
// the block that the last call of many tokens began inside (place 1 or 2) is
// there when the sequence is cut back to that beginning.  Where it was cut back
// into another older block, the tokens in front come from their codes.  Bound by
// latency: length, tail, and the block's arithmetic in a row; 5.6
// us for 8 heads of 128 (8.2 with one warp for K and V, which read their tokens
// from global memory once more for the summary).
constexpr int kAppendHeads = 8;
constexpr int append8_smem(int d, int heads) { return heads * 2 * kBlock * d * 2; }
template <int D, int KV>
__global__ void __launch_bounds__(64 * kAppendHeads) append8_kernel(const __grid_constant__ LayerArgs a,
                                                                     const __grid_constant__ Kv8Args c) {
  constexpr int V = D / 32, W = D / 64, CH = D / 8;  // coordinates of a lane, their words; 16-byte chunks of a token
  extern __shared__ __align__(16) __nv_bfloat16 tiles[];  // [head][K, V][16][D]
  pdl_wait();     // what came before on the stream may have written the cache and the token
  pdl_trigger();  // the kernels of this step may launch (they wait for this grid before reading)
  const int s = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kv = warp & 1;
  const int L = __ldcg(a.seq_len + s);
  const bool fits = L >= 0 && L < a.cap_blocks[s] * kBlock;
  const int b = L / kBlock, slot = L % kBlock;
  __nv_bfloat16* tile = tiles + warp * kBlock * D;
  for (int h0 = 0; fits && h0 < a.Hkv; h0 += kAppendHeads) {
    const int h = h0 + (warp >> 1);
    const bool mine = h < a.Hkv;
    const int64_t row = row_of(a, s, mine ? h : 0, b);
    const int unit = s * a.Hkv + (mine ? h : 0);
    const int place = tail_place(c, unit, b, slot), last = max(place, 0);
    uint8_t* codes = (kv ? c.v : c.k) + row * kBlock * D;
    float* scale = (kv ? c.vscale : c.kscale) + row;
    __nv_bfloat16* to = tail_at<D>(c, unit, last) + kv * kBlock * D;
    if (mine) {
      const __nv_bfloat16* token = (kv ? a.v_new : a.k_new) + (int64_t)unit * D;
      if (slot == 0 || place >= 0) {
        const uint4* from = reinterpret_cast<const uint4*>(tail_at<D>(c, unit, place < 0 ? 0 : place) + kv * kBlock * D);
        uint4 x[CH / 2];
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
          const int at = i * 32 + lane, j = at / CH;  // chunk `at` of the block belongs to token j
          const uint4* p = j == slot ? reinterpret_cast<const uint4*>(token) + at % CH : from + at;
          x[i] = j > slot ? make_uint4(0, 0, 0, 0) : __ldcg(p);
        }
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
          const int at = i * 32 + lane, j = at / CH;
          reinterpret_cast<uint4*>(tile)[at] = x[i];
          if (j == slot) reinterpret_cast<uint4*>(to)[at] = x[i];
        }
      } else {
        const float old = __ldcg(scale);
#pragma unroll 1
        for (int j = 0; j < kBlock; ++j) {
          uint32_t t[W] = {};
          if (j == slot) {
#pragma unroll
            for (int i = 0; i < W; ++i) t[i] = __ldcg(reinterpret_cast<const uint32_t*>(token + lane * V) + i);
          } else if (j < slot) {
            const uint8_t* p = codes + j * D + lane * V;
            const float4 x = Codes<KV>::unpack(W == 2 ? __ldcg(reinterpret_cast<const uint32_t*>(p))
                                                      : __ldcg(reinterpret_cast<const uint16_t*>(p)));
#pragma unroll
            for (int i = 0; i < W; ++i) {
              const float2 f = i ? make_float2(x.z * old, x.w * old) : make_float2(x.x * old, x.y * old);
              const __nv_bfloat162 y = __float22bfloat162_rn(f);
              t[i] = *reinterpret_cast<const uint32_t*>(&y);
            }
          }
#pragma unroll
          for (int i = 0; i < W; ++i) {
            reinterpret_cast<uint32_t*>(tile + j * D + lane * V)[i] = t[i];
            if (j <= slot) reinterpret_cast<uint32_t*>(to + j * D + lane * V)[i] = t[i];
          }
        }
      }
    }
    __syncthreads();  // every warp has read the tail's lengths
    if (mine) {
      tile_summary<D, KV>(tile, slot + 1, (kv ? a.vbar : a.kbar) + row * D, kv ? nullptr : a.dbar + row * a.r, a.r,
                          {codes, scale}, lane);
      if (!kv && lane < kTails) {
        int* len = c.tail_len + kTails * unit + lane;
        if (lane == last) *len = L + 1;
        else if (*len > b * kBlock) *len = 0;
      }
    }
    __syncthreads();  // (and the tiles are read)
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    if (fits) a.seq_len[s] = L + 1;
    else set_error(a.status, kDevCapacity, s, -1, 1);
  }
}

// 16 values of one token from their codes, or as they stand in bf16.
struct Sixteen {
  float x[16];
};
template <int KV>
__device__ __forceinline__ void values(const uint4 (&w)[KV == kKvBf16 ? 2 : 1], float scale, Sixteen& y) {
  if constexpr (KV == kKvBf16) {
    const uint32_t v[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y.x[2 * i] = __uint_as_float(v[i] << 16);
      y.x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  } else {
    const uint32_t v[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = Codes<KV>::unpack(v[i]);
      y.x[4 * i] = f.x * scale;
      y.x[4 * i + 1] = f.y * scale;
      y.x[4 * i + 2] = f.z * scale;
      y.x[4 * i + 3] = f.w * scale;
    }
  }
}
// 32 bytes in one store: a whole sector, whatever the lanes beside write.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// A warp per block, head and one of K and V: a lane takes 16 values of a token
// at a time, its loads of the whole block in flight together.  Heads follow one
// another, then blocks, so that the rows of a token come out close in time.
// Bound by DRAM: 16 sequences of up to 16381 tokens of 8 heads of 128 from int8 to
// bf16 (0.97 GB) in 145 us, 0.99 of the copy rate; the smallest calls take 3 us.
template <int D, int KV, bool F32>
__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int CH = D / 16, N = kBlock * CH / 32, L = KV == kKvBf16 ? 2 : 1;  // chunks of a token; of a lane; their loads
  const int lane = threadIdx.x & 31;
  const int64_t item = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int per = 2 * a.Hkv;
  const int64_t at = item / per;
  if (at >= a.item0[a.B]) return;
  const int kv = (int)(item % per) / a.Hkv, h = (int)(item % per) % a.Hkv;
  int s = 0;
  while (s + 1 < a.B && a.item0[s + 1] <= at) ++s;
  const int b = a.starts[s] / kBlock + (int)(at - a.item0[s]);
  const int have = __ldcg(a.seq_len + s), end = min(a.starts[s] + a.counts[s], have);
  if (a.starts[s] + a.counts[s] > have && lane == 0 && item == (int64_t)a.item0[s] * per)
    set_error(a.status, kDevInvalidArg, s, -1, 3);
  const int64_t row = a.seq_row0[s] + (int64_t)h * a.cap_blocks[s] + b;
  uint4 w[N][L];
  float scale = 1.f;
  if constexpr (KV != kKvBf16) scale = __ldg((kv ? a.kv8.vscale : a.kv8.kscale) + row);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int x = i * 32 + lane, tok = b * kBlock + x / CH;  // chunk x of the block
    const char* p = KV == kKvBf16 ? reinterpret_cast<const char*>((kv ? a.bv : a.bk) + row * kBlock * D) + x * 32
                                  : reinterpret_cast<const char*>((kv ? a.kv8.v : a.kv8.k) + row * kBlock * D) + x * 16;
#pragma unroll
    for (int l = 0; l < L; ++l) {
      w[i][l] = make_uint4(0, 0, 0, 0);
      if (tok < end && tok >= a.starts[s]) w[i][l] = __ldcs(reinterpret_cast<const uint4*>(p) + l);
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int x = i * 32 + lane, tok = b * kBlock + x / CH;
    if (tok >= end || tok < a.starts[s]) continue;
    Sixteen y;
    values<KV>(w[i], scale, y);
    const int64_t o = (((int64_t)a.token0[s] + tok - a.starts[s]) * a.Hkv + h) * D + x % CH * 16;
    uint32_t z[8];
    if constexpr (F32) {
      float* out = reinterpret_cast<float*>(kv ? a.v : a.k) + o;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = __float_as_uint(y.x[8 * k + e]);
        store32(out + 8 * k, z);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(y.x[2 * e], y.x[2 * e + 1]);
        z[e] = *reinterpret_cast<const uint32_t*>(&v);
      }
      store32(reinterpret_cast<__nv_bfloat16*>(kv ? a.v : a.k) + o, z);
    }
  }
}

template <int D, int KV>
cudaError_t read_as(const ReadArgs& a, cudaStream_t st) {
  const int64_t warps = (int64_t)a.item0[a.B] * 2 * a.Hkv;
  const unsigned grid = (unsigned)((warps + 7) / 8);
  if (a.out_f32) read_kernel<D, KV, true><<<grid, 256, 0, st>>>(a);
  else read_kernel<D, KV, false><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

template <int D, int KV>
static cudaError_t append8_as(const LayerArgs& a, const Kv8Args& c, cudaStream_t st) {
  LayerArgs args = a;
  Kv8Args codes = c;
  void* argv[] = {&args, &codes};
  const int heads = a.Hkv < kAppendHeads ? a.Hkv : kAppendHeads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.B);
  cfg.blockDim = dim3(64 * heads);
  cfg.dynamicSmemBytes = append8_smem(D, heads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(&append8_kernel<D, KV>), argv);
}

cudaError_t launch_append8(const LayerArgs& a, const Kv8Args& c, cudaStream_t st) {
  const bool i8 = c.type == kKvInt8;
  if (a.d == 128) return i8 ? append8_as<128, kKvInt8>(a, c, st) : append8_as<128, kKvE4m3>(a, c, st);
  return i8 ? append8_as<64, kKvInt8>(a, c, st) : append8_as<64, kKvE4m3>(a, c, st);
}

template <int D>
static cudaError_t prepare_append8_d() {
  const int smem = append8_smem(D, kAppendHeads);
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(&append8_kernel<D, kKvInt8>), smem);
  return e == cudaSuccess ? raise_smem_limit(reinterpret_cast<const void*>(&append8_kernel<D, kKvE4m3>), smem) : e;
}
cudaError_t prepare_append8(int d) { return d == 128 ? prepare_append8_d<128>() : prepare_append8_d<64>(); }

cudaError_t launch_read(const ReadArgs& a, cudaStream_t st) {
  if (!a.item0[a.B]) return cudaSuccess;
  if (a.d == 128) {
    switch (a.kv8.type) {
      case kKvInt8: return read_as<128, kKvInt8>(a, st);
      case kKvE4m3: return read_as<128, kKvE4m3>(a, st);
      default: return read_as<128, kKvBf16>(a, st);
    }
  }
  switch (a.kv8.type) {
    case kKvInt8: return read_as<64, kKvInt8>(a, st);
    case kKvE4m3: return read_as<64, kKvE4m3>(a, st);
    default: return read_as<64, kKvBf16>(a, st);
  }
}

}  // namespace compkv
