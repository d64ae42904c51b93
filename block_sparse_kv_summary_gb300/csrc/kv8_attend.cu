// Exact attention of one query token per sequence over a cache in 8 bits:
//
//     out = sum_j e^(z_j) v_j / sum_j e^(z_j),    z_j = (q . c_j) scale_b / sqrt(d)
//
// over every token of the sequence, or over the tokens of the selected blocks
// with Mean compensation for the others (|b| e^(zbar_b) vbar_b and |b|
// e^(zbar_b) for every block that is not selected, section "무엇과 다른가").
//
// Work.  A unit is a (sequence, KV head).  Its blocks, or its selection's
// entries, go in stages of two.  The stages of all units stand in one row that
// is cut into equal runs, one for each CTA; a run's stages go to the eight warps
// in turn.  What a CTA has of a unit is a segment: its warps' parts are joined
// in shared memory, and where other CTAs have the rest of the unit, the segment
// is left in the workspace and the last CTA to arrive joins them in their order.
//
// A stage.  Each warp has a ring of kSlots stages filled by tensor copies that
// it starts itself, the two scales of its blocks beside them, so that 192 KB are
// on their way to a multiprocessor while another segment's queries are read or
// its parts joined.  Codes become fp16, which holds them all: for int8 the byte
// is put behind the exponent of 1024 and 1152 taken off; for e4m3 its bits are
// shifted into place and the missing factor of 2^8 joins the scale.
//
// Scores are S = Q K^T on mma.sync (m16n8k16): rows 0..7 are the query heads'
// high fp16 parts, rows 8..15 their low parts, so that one product has both;
// the sum of rows r and r + 8 is q . c to the 22 bits of the two parts.  The 16
// columns of a block share one scale.  Outputs are O^T = V^T P (rows:
// coordinates, columns: heads), with the weights in high and low parts too:
// weights are e^(z - m + 14 ln 2), which keeps their low parts normal numbers.
// A block's product starts from zero and is added to the running output with the
// block's scale in fp32: the tensor cores' accumulator truncates, and the scale
// has to be applied anyway.
//
// Which coordinate stands where inside a product is free, as long as both sides
// agree: lane (r, c) = (lane / 4, lane % 4) takes the D / 4 coordinates from
// c D / 4 on of its token's key, and the D / 8 from r D / 8 on of its four
// tokens' values, each in 16-byte (values of d 64: 8-byte) loads without bank
// conflicts.  mma.sync and not tcgen05: with at most 8 query rows a tile of 128
// would be 1/16 full, and codes would have to go back to shared memory as fp16
// between their copy and the product.
#include <cuda_fp16.h>

#include "compkv_launch.h"
#include "decode_common.cuh"
#include "kv8.cuh"

namespace compkv {

namespace {

constexpr int kWarps8 = 8;
constexpr int kThreads8 = 32 * kWarps8;
constexpr int kSlots = 3;    // stages of a warp's ring
constexpr int kPair = 2;     // blocks of a stage
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLift = 14.f;  // weights are kept below 2^14: fp16 ends at 2^16

// Shared memory, from a 1024-byte boundary on.
template <int D>
struct Smem8 {
  static constexpr int kBlockBytes = kBlock * D;
  static constexpr int kStage = 2 * kPair * kBlockBytes;  // K blocks, then V blocks
  alignas(1024) uint8_t ring[kWarps8][kSlots][kStage];
  uint4 q[D / 16][32];                // A fragments of the queries (high, low, high, low)
  float part[kWarps8][4][D];          // the warps' outputs of four heads
  float comp[kMaxG][D];               // this segment's share of the compensation sums
  float scale[kWarps8][kSlots][2 * kPair];
  float ref[kWarps8 + 1][kMaxG];      // references (log2) and sums of the parts; the last: compensation
  float sum[kWarps8 + 1][kMaxG];
  float qs[kMaxG];                    // factor of a head's scores
  uint64_t full[kWarps8][kSlots];
  int tokens[kMaxBatch];              // of each sequence
  int stages[kMaxBatch];              // stages of each of its units
  int first[kMaxBatch + 1];           // first stage of its first unit
  int streamed[kMaxBatch];            // the stream's plan (selections only)
  int soff[kMaxBatch + 1];
  int seg;
  int valid;                          // entries of the unit's selection
  int last;                           // this CTA is the last of the unit's
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// d += A B, fp16 inputs
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ void split_f16(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = as_u32(h);
  lo = as_u32(__floats2half2_rn(x - f.x, y - f.y));
}

// Four codes as two pairs of fp16 (e4m3: 2^-8 of the values).
template <int KV>
struct Wide {
  static constexpr float unit = KV == kKvE4m3 ? 256.f : 1.f;
  static __device__ __forceinline__ void pairs(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (KV == kKvInt8) {
      const uint32_t x = w ^ 0x80808080u;
      const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1024 + 128
      const uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
      lo = as_u32(__hsub2(*reinterpret_cast<const __half2*>(&a), bias));
      hi = as_u32(__hsub2(*reinterpret_cast<const __half2*>(&b), bias));
    } else {
      const uint32_t a = __byte_perm(w, 0u, 0x1404), b = __byte_perm(w, 0u, 0x3424);
      lo = (a & 0x80008000u) | (a >> 1 & 0x3f803f80u);
      hi = (b & 0x80008000u) | (b >> 1 & 0x3f803f80u);
    }
  }
};

// Where 16-byte chunk x of token t stands in a block of [16][D] bytes that a tensor copy swizzled over D bytes.
template <int D>
__device__ __forceinline__ int chunk_at(int t, int x) {
  return D == 128 ? t * 128 + ((x ^ (t & 7)) << 4) : t * 64 + ((x ^ (t >> 1 & 3)) << 4);
}
// Token of column n (< 8) of a score tile.  With rows of 64 bytes, tokens of one parity share their banks; this order
// gives the four tokens that one load of values touches both parities and different chunks.
template <int D>
__device__ __forceinline__ int token_of(int n) {
  return D == 128 ? n : n ^ (n >> 1 & 1);
}

// A warp's running state: m (log2) of head r, this lane's part of the sum, O^T at coordinates r D / 8 + 2 mt (+ 1) for
// heads 2c and 2c + 1.
template <int D>
struct State {
  float m, l;
  float acc[D / 16][4];
  __device__ __forceinline__ void reset() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  }
};

// What a block of a stage is: its tokens (0: not there), and with `comp`, its mean logits and mean value, which come off.
struct Block8 {
  int n;
  float ks, vs;
  float zb;            // zbar of head r, natural units (comp)
  const float* vbar;   // null: nothing comes off
};

template <int D, int KV, bool SPARSE>
__device__ __forceinline__ void attend_pair(State<D>& st, const uint8_t* stage, const uint4 (*qf)[32], float qs, const Block8 (&blk)[kPair],
                                            int lane) {
  constexpr int KS = D / 16, B8 = kBlock * D;
  const int r = lane >> 2, c = lane & 3;
  // ---- scores
  float s[kPair][2][4];
  uint32_t kw[kPair][2][KS];
#pragma unroll
  for (int i = 0; i < kPair; ++i)
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int x = 0; x < KS / 4; ++x) {
        const int tok = t * 8 + token_of<D>(r);
        const uint4 w = *reinterpret_cast<const uint4*>(stage + i * B8 + chunk_at<D>(tok, c * (KS / 4) + x));
        kw[i][t][4 * x] = w.x;
        kw[i][t][4 * x + 1] = w.y;
        kw[i][t][4 * x + 2] = w.z;
        kw[i][t][4 * x + 3] = w.w;
      }
      s[i][t][0] = s[i][t][1] = s[i][t][2] = s[i][t][3] = 0.f;
    }
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    const uint4 q = qf[ks][lane];
#pragma unroll
    for (int i = 0; i < kPair; ++i)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        uint32_t b0, b1;
        Wide<KV>::pairs(kw[i][t][ks], b0, b1);
        mma_f16(s[i][t], q.x, q.y, q.z, q.w, b0, b1);
      }
  }
  // ---- weights: head r at tokens token_of(2c), token_of(2c + 1) and 8 further
  float z[kPair][4], bm = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPair; ++i)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool there = 8 * t + token_of<D>(2 * c + e) < blk[i].n;
        const float x = there ? (s[i][t][e] + s[i][t][e + 2]) * qs * blk[i].ks : -INFINITY;
        z[i][2 * t + e] = x;
        bm = fmaxf(bm, x);
      }
  bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 1));
  bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 2));
  float e2[kPair];
  if constexpr (SPARSE) {
#pragma unroll
    for (int i = 0; i < kPair; ++i) {
      e2[i] = blk[i].vbar ? (ln_count(blk[i].n) + blk[i].zb) * kLog2e : -INFINITY;
      bm = fmaxf(bm, e2[i]);
    }
  }
  const float mn = fmaxf(st.m, bm), low = mn == -INFINITY ? 0.f : mn - kLift;
  if (__any_sync(0xffffffffu, mn > st.m)) {
    const float fo = st.m == -INFINITY ? 0.f : ex2(st.m - mn);
    const float foA = __shfl_sync(0xffffffffu, fo, 8 * c), foB = __shfl_sync(0xffffffffu, fo, 8 * c + 4);
    st.l *= fo;
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
      st.acc[mt][0] *= foA;
      st.acc[mt][1] *= foB;
      st.acc[mt][2] *= foA;
      st.acc[mt][3] *= foB;
    }
    st.m = mn;
  }
  uint32_t ph[kPair][2], pl[kPair][2];
#pragma unroll
  for (int i = 0; i < kPair; ++i) {
    float p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[e] = ex2(z[i][e] - low);
      st.l += p[e];
    }
    split_f16(p[0], p[1], ph[i][0], pl[i][0]);
    split_f16(p[2], p[3], ph[i][1], pl[i][1]);
  }
  // ---- outputs
  const uint8_t* vals = stage + kPair * B8;
#pragma unroll
  for (int i = 0; i < kPair; ++i) {
    uint32_t w[4][D / 32];  // values of this lane's four tokens: token_of(2c), token_of(2c + 1), and 8 further
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int tok = token_of<D>(2 * c + (j & 1)) + 8 * (j >> 1);
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(vals + i * B8 + chunk_at<D>(tok, r));
        w[j][0] = x.x;
        w[j][1] = x.y;
        w[j][2] = x.z;
        w[j][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(vals + i * B8 + chunk_at<D>(tok, r >> 1) + (r & 1) * 8);
        w[j][0] = x.x;
        w[j][1] = x.y;
      }
    }
    float fnA = 0.f, fnB = 0.f;
    if constexpr (SPARSE) {
      const float fn = blk[i].vbar ? ex2(e2[i] - low) : 0.f;
      if (c == 0) st.l -= fn;
      fnA = __shfl_sync(0xffffffffu, fn, 8 * c);
      fnB = __shfl_sync(0xffffffffu, fn, 8 * c + 4);
    }
#pragma unroll
    for (int x = 0; x < D / 32; ++x) {
      // bytes of two tokens side by side: their first two coordinates of the word, then the other two
      const uint32_t a01 = __byte_perm(w[0][x], w[1][x], 0x5140), a23 = __byte_perm(w[0][x], w[1][x], 0x7362);
      const uint32_t b01 = __byte_perm(w[2][x], w[3][x], 0x5140), b23 = __byte_perm(w[2][x], w[3][x], 0x7362);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t a0, a1, a2, a3;
        Wide<KV>::pairs(y ? a23 : a01, a0, a1);
        Wide<KV>::pairs(y ? b23 : b01, a2, a3);
        float o[4] = {0.f, 0.f, 0.f, 0.f};
        mma_f16(o, a0, a1, a2, a3, pl[i][0], pl[i][1]);
        mma_f16(o, a0, a1, a2, a3, ph[i][0], ph[i][1]);
        float(&acc)[4] = st.acc[2 * x + y];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = fmaf(o[e], blk[i].vs, acc[e]);
        if constexpr (SPARSE) {
          if (blk[i].vbar) {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(blk[i].vbar + r * (D / 8)) + 2 * x + y);
            acc[0] = fmaf(-fnA, v.x, acc[0]);
            acc[1] = fmaf(-fnB, v.x, acc[1]);
            acc[2] = fmaf(-fnA, v.y, acc[2]);
            acc[3] = fmaf(-fnB, v.y, acc[3]);
          }
        }
      }
    }
  }
}

// The unit's queries as A fragments, by one warp per head: lane l < D / 4 holds
// coordinates 4 l .. 4 l + 3, which are those of lane (r, c) = (head, l / KS)
// in step l % KS.  A head is brought to magnitudes below 2^14 by a power of two,
// so that both parts of every coordinate that counts are normal numbers.
template <int D>
__device__ __forceinline__ void stage_queries(Smem8<D>& sm, const Attend8Args& a, int64_t unit, int head, int lane, float unit_scale) {
  constexpr int KS = D / 16;
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if (head < a.G && lane < D / 4) {
    const int64_t at = (unit * a.G + head) * D + 4 * lane;
    if (a.q_bf16) {
      const uint2 w = __ldcg(reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(a.q) + at));
      x[0] = __uint_as_float(w.x << 16);
      x[1] = __uint_as_float(w.x & 0xffff0000u);
      x[2] = __uint_as_float(w.y << 16);
      x[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
      const float4 w = __ldcg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.q) + at));
      x[0] = w.x;
      x[1] = w.y;
      x[2] = w.z;
      x[3] = w.w;
    }
  }
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) bits = max(bits, __float_as_uint(x[i]) & 0x7fffffffu);
  bits = __reduce_max_sync(0xffffffffu, bits);
  // 2^e <= largest magnitude < 2^(e + 1), kept where 2^(13 - e) and 2^(e - 13) are normal numbers (an infinity or a NaN
  // makes NaN of its head's scores either way)
  const int e = max(-113, min(126, (int)(bits >> 23) - 127));
  const float up = __uint_as_float((uint32_t)(13 - e + 127) << 23);
  if (lane < D / 4) {
    uint4 f;
    split_f16(x[0] * up, x[1] * up, f.x, f.y);
    split_f16(x[2] * up, x[3] * up, f.z, f.w);
    sm.q[lane % KS][head * 4 + lane / KS] = f;
  }
  if (lane == 0) sm.qs[head] = __uint_as_float((uint32_t)(e - 13 + 127) << 23) * unit_scale;
}

// This segment's share of the unit's compensation sums: the stream's records p, p + C, ... at their common reference.
template <int D>
__device__ __forceinline__ void stage_compensation(Smem8<D>& sm, const Attend8Args& a, int i0, int nseg, int p, int C, int tid) {
#pragma unroll 1
  for (int item = tid; item < a.G * D / 4; item += kThreads8) {
    const int g = item / (D / 4), col = 4 * (item % (D / 4));
    float R = -INFINITY, W = 0.f;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = p; k0 < nseg; k0 += 4 * C) {
      float4 e[4], v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool there = k0 + j * C < nseg;
        const int64_t at = (int64_t)(i0 + k0 + j * C) * a.G + g;
        e[j] = there ? __ldcg(a.rec + at) : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
        v[j] = there ? __ldcg(reinterpret_cast<const float4*>(a.comp + at * D + col)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (e[j].z == -INFINITY) continue;
        const float mn = fmaxf(R, e[j].z);
        const float fo = R == -INFINITY ? 0.f : ex2((R - mn) * kLog2e), fn = ex2((e[j].z - mn) * kLog2e);
        A.x = A.x * fo + v[j].x * fn;
        A.y = A.y * fo + v[j].y * fn;
        A.z = A.z * fo + v[j].z * fn;
        A.w = A.w * fo + v[j].w * fn;
        W = W * fo + e[j].w * fn;
        R = mn;
      }
    }
    *reinterpret_cast<float4*>(&sm.comp[g][col]) = A;
    if (col == 0) {
      sm.ref[kWarps8][g] = R * kLog2e;
      sm.sum[kWarps8][g] = W;
    }
  }
}

template <int D>
__device__ __forceinline__ void put_out(const Attend8Args& a, int64_t unit, int g, int col, float2 acc, float l) {
  // a row without tokens is zero; a sum that is NaN goes through
  const float2 y = l == 0.f ? make_float2(0.f, 0.f) : make_float2(__fdividef(acc.x, l), __fdividef(acc.y, l));
  const int64_t at = (unit * a.G + g) * D + col;
  if (a.q_bf16) *reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<__nv_bfloat16*>(a.out) + at) = __floats2bfloat162_rn(y.x, y.y);
  else *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.out) + at) = y;
}

// The part of a part whose reference is `ref`, at reference M (a part without tokens has neither, and a sum that may be NaN).
__device__ __forceinline__ float part_factor(float ref, float M) { return ref == -INFINITY ? 0.f : ex2(ref - M); }

template <int D, int KV, bool SPARSE>
__global__ void __launch_bounds__(kThreads8, 1) attend8_kernel(const __grid_constant__ Attend8Args a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Smem8<D>& sm = *reinterpret_cast<Smem8<D>*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  constexpr int B8 = kBlock * D;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, x = blockIdx.x;
  if (tid < kWarps8 * kSlots) mbar_init(&sm.full[0][0] + tid, 1 + 2 * kPair);
  if (tid == 0) fence_mbar_init();
  pdl_wait();  // what came before on the stream may have written the cache, its lengths, the queries and the selection
  if (warp == 0) {
    // the row of stages, from the lengths
    int at = 0;
#pragma unroll
    for (int k = 0; k < kMaxBatch; k += 32) {
      const int s = k + lane;
      int n = 0, st = 0;
      if (s < a.B) {
        bool fits;
        const int L = call_tokens(__ldcg(a.seq_len + s), a.cap_blocks[s], false, &fits);
        n = ceil_blocks(L);
        sm.tokens[s] = L;
        if (SPARSE) sm.streamed[s] = streamed_blocks(L, false, a.selects, a.K, false);
        st = ((SPARSE ? min(n, a.K) : n) + kPair - 1) / kPair;
        sm.stages[s] = st;
      }
      int incl = st * a.Hkv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (s <= a.B) sm.first[s] = at + incl - st * a.Hkv;
      at += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) sm.first[a.B] = at;
    if (SPARSE) {
      __syncwarp();
      plan_warp(sm.streamed, a.B, a.Hkv, a.stream_P, stage_blocks(a.r, a.G), sm.soff, &sm.seg, lane);
    }
  }
  __syncthreads();
  const int total = sm.first[a.B];
  // a run: no shorter than a stage for each warp
  const int per = max(kWarps8, (total + (int)gridDim.x - 1) / (int)gridDim.x);
  const int lo = min(total, x * per), hi = min(total, lo + per);

  // ---- this warp's copies: stages lo + warp + 8 j of the run, ahead of their use
  int issued = lo + warp, si = 0;  // next stage to copy, its sequence
  const uint64_t pol = policy_evict_first();
  auto entry = [&](int64_t unit, int i, int n) -> int {  // block of entry i of a unit's selection (-1: none, or not a valid one)
    if (i >= min(n, a.K)) return -1;
    const int* sel = a.sel + unit * a.K;
    const int e = __ldcg(sel + i), prev = i > 0 ? __ldcg(sel + i - 1) : -1;
    return e >= 0 && e < n && (i == 0 || (prev >= 0 && prev < e)) ? e : -1;
  };
  auto issue = [&](int slot) {
    if (issued >= hi) return;
    while (issued >= sm.first[si + 1]) ++si;
    const int local = issued - sm.first[si], h = local / sm.stages[si], j = local - h * sm.stages[si];
    const int n = ceil_blocks(sm.tokens[si]);
    const int64_t row0 = a.seq_row0[si] + (int64_t)h * a.cap_blocks[si];
    uint64_t* bar = &sm.full[warp][slot];
    uint8_t* dst = sm.ring[warp][slot];
    int b[kPair];
#pragma unroll
    for (int i = 0; i < kPair; ++i) {
      if (SPARSE) b[i] = entry((int64_t)si * a.Hkv + h, kPair * j + i, n);
      else b[i] = kPair * j + i < n ? kPair * j + i : -1;
    }
    __syncwarp();  // the slot's previous contents are read
    // the scales: one lane each
    if (lane < 2 * kPair) {
      const int mine = lane % kPair ? b[1] : b[0];
      if (mine >= 0) {
        const float* src = (lane < kPair ? a.kv8.kscale : a.kv8.vscale) + row0 + mine;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&sm.scale[warp][slot][lane])), "l"(src) : "memory");
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
    }
    if (lane == 0) {
      const int64_t base = (a.layer_row0 + row0) * kBlock;
      if (SPARSE) {
        mbar_arrive_expect_tx(bar, ((b[0] >= 0) + (b[1] >= 0)) * 2 * B8);
#pragma unroll
        for (int i = 0; i < kPair; ++i) {
          if (b[i] < 0) continue;
          tma_2d(dst + i * B8, a.k16, 0, (int)(base + b[i] * kBlock), bar, pol);
          tma_2d(dst + (kPair + i) * B8, a.v16, 0, (int)(base + b[i] * kBlock), bar, pol);
        }
      } else {
        // (a pair's second block may be another unit's, or lie behind the cache, which reads as zero: it is masked)
        mbar_arrive_expect_tx(bar, Smem8<D>::kStage);
        tma_2d(dst, a.k32, 0, (int)(base + kPair * j * kBlock), bar, pol);
        tma_2d(dst + kPair * B8, a.v32, 0, (int)(base + kPair * j * kBlock), bar, pol);
      }
    }
    issued += kWarps8;
  };
#pragma unroll
  for (int k = 0; k < kSlots; ++k) issue(k);

  // ---- the run's segments
  int slot = 0, phase = 0;
  bool ok = true;
  int s = 0;
  State<D> st;
  for (int at = lo; at < hi;) {
    while (at >= sm.first[s + 1]) ++s;
    const int per_unit = sm.stages[s], h = (at - sm.first[s]) / per_unit;
    const int unit0 = sm.first[s] + h * per_unit;  // the unit's stages are [unit0, unit0 + per_unit)
    const int end = min(hi, unit0 + per_unit);
    const int64_t unit = (int64_t)s * a.Hkv + h;
    const int L = sm.tokens[s], n = ceil_blocks(L);
    const int64_t row0 = a.seq_row0[s] + (int64_t)h * a.cap_blocks[s];
    const int c0 = unit0 / per, C = (unit0 + per_unit - 1) / per - c0 + 1;  // CTAs that have a part of this unit
    // queries, and what a selection takes
    const float unit_scale = Wide<KV>::unit * kLog2e * (D == 128 ? 0.08838834764831845f : 0.125f);
    stage_queries<D>(sm, a, unit, warp, lane, unit_scale);
    bool comp = false;
    if (SPARSE) {
      int valid = 0, wrong = 0;
#pragma unroll 1
      for (int i = tid; i < a.K; i += kThreads8) {
        const int e = __ldcg(a.sel + unit * a.K + i), prev = i > 0 ? __ldcg(a.sel + unit * a.K + i - 1) : -1;
        const bool good = e >= 0 && e < n && (i == 0 || (prev >= 0 && prev < e));
        valid += good;
        wrong |= (e >= 0 && !good) || e < -1;
      }
      if (tid == 0) sm.valid = 0;
      __syncthreads();
      valid = __reduce_add_sync(0xffffffffu, valid);
      if (lane == 0 && valid) atomicAdd(&sm.valid, valid);
      if (__any_sync(0xffffffffu, wrong) && lane == 0 && x == c0) set_error(a.status, kDevBadSelection, s, h, 61);
      __syncthreads();
      comp = !a.no_comp && sm.valid < n;
      if (comp) {
        const int nseg = (sm.streamed[s] + sm.seg - 1) / sm.seg;
        stage_compensation<D>(sm, a, sm.soff[s] + h * nseg, nseg, x - c0, C, tid);
      }
    }
    __syncthreads();
    const float qs = sm.qs[lane >> 2];
    st.reset();
    for (int i = at + (warp - (at - lo) % kWarps8 + kWarps8) % kWarps8; i < end; i += kWarps8) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(&sm.full[warp][slot], phase, a.status, s, h, 71));
      if (ok) {
        Block8 blk[kPair];
        const int j = i - unit0;
#pragma unroll
        for (int k = 0; k < kPair; ++k) {
          const int b = SPARSE ? entry(unit, kPair * j + k, n) : kPair * j + k < n ? kPair * j + k : -1;
          blk[k].n = b < 0 ? 0 : min(kBlock, L - b * kBlock);
          blk[k].ks = b < 0 ? 0.f : sm.scale[warp][slot][k];
          blk[k].vs = b < 0 ? 0.f : sm.scale[warp][slot][kPair + k] * Wide<KV>::unit;
          blk[k].zb = SPARSE && comp && b >= 0 && lane >> 2 < a.G ? __ldcg(a.zs + (row0 + b) * pad_g(a.G) + (lane >> 2)) : 0.f;
          blk[k].vbar = SPARSE && comp && b >= 0 ? a.vbar + (row0 + b) * D : nullptr;
        }
        if (blk[0].n | blk[1].n) attend_pair<D, KV, SPARSE>(st, sm.ring[warp][slot], sm.q, qs, blk, lane);
        issue(slot);
      }
      if (++slot == kSlots) {
        slot = 0;
        phase ^= 1;
      }
    }
    at = end;
    // ---- the warps' parts and the compensation share, four heads at a time
    float l = st.l;
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if ((lane & 3) == 0) {
      sm.ref[warp][lane >> 2] = st.m - kLift;
      sm.sum[warp][lane >> 2] = l;
    }
    const bool whole = C == 1;
    const int place = 2 * x + (x == c0 && lo < unit0);  // of this segment in the workspace
#pragma unroll 1
    for (int g0 = 0; g0 < a.G; g0 += 4) {
      const int c = lane & 3, r = lane >> 2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int g = 2 * c + e - g0;
        if (g < 0 || g >= 4) continue;
        float2* to = reinterpret_cast<float2*>(&sm.part[warp][g][r * (D / 8)]);
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) to[mt] = make_float2(st.acc[mt][e], st.acc[mt][2 + e]);
      }
      __syncthreads();
#pragma unroll 1
      for (int item = tid; item < min(4, a.G - g0) * D / 2; item += kThreads8) {
        const int g = g0 + item / (D / 2), col = 2 * (item % (D / 2));
        const int parts = kWarps8 + (SPARSE && comp);
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps8 + SPARSE; ++w)
          if (w < parts) M = fmaxf(M, sm.ref[w][g]);
        float2 A = make_float2(0.f, 0.f);
        float S = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps8 + SPARSE; ++w) {
          if (w >= parts) continue;
          const float f = part_factor(sm.ref[w][g], M);
          const float2 v = *reinterpret_cast<const float2*>(w < kWarps8 ? &sm.part[w][g - g0][col] : &sm.comp[g][col]);
          A.x = fmaf(v.x, f, A.x);
          A.y = fmaf(v.y, f, A.y);
          S = fmaf(sm.sum[w][g], f, S);
        }
        if (whole) {
          put_out<D>(a, unit, g, col, A, S);
        } else {
          __stcg(reinterpret_cast<float2*>(a.acc + ((int64_t)place * a.G + g) * D + col), A);
          if (col == 0) __stcg(a.ml + (int64_t)place * a.G + g, make_float2(M, S));
        }
      }
      __syncthreads();
    }
    if (whole) continue;
    // ---- the last of the unit's CTAs joins the segments
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      sm.last = atomicAdd(a.arrive + unit, 1) == C - 1;
      if (sm.last) a.arrive[unit] = 0;
    }
    __syncthreads();
    if (!sm.last) continue;
    __threadfence();
#pragma unroll 1
    for (int item = tid; item < a.G * D / 2; item += kThreads8) {
      const int g = item / (D / 2), col = 2 * (item % (D / 2));
      float M = -INFINITY, S = 0.f;
      float2 A = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int k0 = 0; k0 < C; k0 += 8) {
        float2 e[8], v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int y = c0 + k0 + k;
          const bool there = k0 + k < C;
          // the first CTA may have come from another unit's stages
          const int64_t at = ((int64_t)(2 * y + (k0 + k == 0 && y * per < unit0)) * a.G + g);
          e[k] = there ? __ldcg(a.ml + at) : make_float2(-INFINITY, 0.f);
          v[k] = there ? __ldcg(reinterpret_cast<const float2*>(a.acc + at * D + col)) : make_float2(0.f, 0.f);
        }
        float mn = M;
#pragma unroll
        for (int k = 0; k < 8; ++k) mn = fmaxf(mn, e[k].x);
        const float fo = part_factor(M, mn);
        A.x *= fo;
        A.y *= fo;
        S *= fo;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float f = part_factor(e[k].x, mn);
          A.x = fmaf(v[k].x, f, A.x);
          A.y = fmaf(v[k].y, f, A.y);
          S = fmaf(e[k].y, f, S);
        }
        M = mn;
      }
      put_out<D>(a, unit, g, col, A, S);
    }
  }
  if (!ok) {  // a wait ran out: let the copies in flight land before the CTA's memory goes
#pragma unroll 1
    for (int k = 0; k < kSlots; ++k) mbar_drain_bounded(&sm.full[warp][k]);
  }
  // rows of sequences without tokens
#pragma unroll 1
  for (int u = x; u < a.B * a.Hkv; u += gridDim.x) {
    if (sm.stages[u / a.Hkv]) continue;
    for (int i = tid; i < a.G * D / 2; i += kThreads8) put_out<D>(a, u, i / (D / 2), 2 * (i % (D / 2)), make_float2(0.f, 0.f), 0.f);
  }
}

template <int D, int KV, bool SPARSE>
cudaError_t attend8_as(const Attend8Args& a, cudaStream_t st) {
  Attend8Args args = a;
  void* argv[] = {&args};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.P);
  cfg.blockDim = dim3(kThreads8);
  cfg.dynamicSmemBytes = sizeof(Smem8<D>) + 1024;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(&attend8_kernel<D, KV, SPARSE>), argv);
}
template <int D>
cudaError_t attend8_d(const Attend8Args& a, cudaStream_t st) {
  if (a.kv8.type == kKvInt8) return a.sel ? attend8_as<D, kKvInt8, true>(a, st) : attend8_as<D, kKvInt8, false>(a, st);
  return a.sel ? attend8_as<D, kKvE4m3, true>(a, st) : attend8_as<D, kKvE4m3, false>(a, st);
}
template <int D>
cudaError_t prepare_d() {
  static_assert(sizeof(Smem8<D>) + 1024 <= 232448, "shared memory of a CTA");
  cudaError_t e = cudaSuccess;
  for (const void* fn : {reinterpret_cast<const void*>(&attend8_kernel<D, kKvInt8, true>), reinterpret_cast<const void*>(&attend8_kernel<D, kKvInt8, false>),
                         reinterpret_cast<const void*>(&attend8_kernel<D, kKvE4m3, true>), reinterpret_cast<const void*>(&attend8_kernel<D, kKvE4m3, false>)})
    if (e == cudaSuccess) e = raise_smem_limit(fn, (int)sizeof(Smem8<D>) + 1024);
  return e;
}

}  // namespace

cudaError_t prepare_attend8(int d) { return d == 128 ? prepare_d<128>() : prepare_d<64>(); }
cudaError_t launch_attend8(const Attend8Args& a, cudaStream_t st) { return a.d == 128 ? attend8_d<128>(a, st) : attend8_d<64>(a, st); }

}  // namespace compkv
