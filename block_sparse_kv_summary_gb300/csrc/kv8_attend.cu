// Exact attention of one query token per sequence over a cache in 8 bits:
//
//     out = sum_j e^(z_j) v_j / sum_j e^(z_j),    z_j = (q . c_j) scale_b / sqrt(d)
//
// over every token of the sequence, or over the tokens of the selected blocks
// with Mean compensation for the others (|b| e^(zbar_b) vbar_b and |b|
// e^(zbar_b) for every block that is not selected, section "무엇과 다른가").
//
// Work.  A unit is a (sequence, KV head).  Its blocks, or its selection's
// entries, go in stages of two; the stages of all units stand in one row, which
// is cut into equal runs, one for each CTA.  A run's stages go to the CTA's
// warps in turn.  What a run has of a unit is a segment: its warps' parts are
// joined in shared memory, and where other runs have the rest of the unit, the
// segment is left in the workspace, and the CTA that leaves the last one joins
// them in their order, so that results do not depend on who came last.
//
// A stage.  Each warp has a ring of stages filled by tensor copies that it starts
// itself, the scales of its blocks beside them, so that 192 KB are on their way
// to a multiprocessor while another segment's queries are read or its parts
// joined.
//
// Products.  Codes become fp16, which holds them all.  Scores are S = Q K^T on
// mma.sync (m16n8k16): rows 0..7 are the query heads' high fp16 parts, rows
// 8..15 their low parts, so that one product has both; the sum of rows r and
// r + 8 is q . c.  (Two parts hold an fp32 number to 2^-23 of itself: what the
// high part leaves is at most 2^12 units of its last place, of which the low part
// holds 11 bits.)  The 16 columns of a block share one scale.  Outputs are O^T = V^T P (rows: coordinates, columns: heads),
// with the weights in high and low parts too: weights are e^(z - m + 14 ln 2),
// which keeps their low parts normal numbers.  A block's product is added to the
// running output with the block's scale in fp32: the tensor cores' accumulator
// truncates, and the scale has to be applied anyway.
//
// Which coordinate stands where inside a product is free, as long as both sides
// agree: lane (r, c) = (lane / 4, lane % 4) takes the D / 4 coordinates from
// c D / 4 on of its token's key, and the D / 8 from r D / 8 on of its four
// tokens' values, each in 16-byte (values of d 64: 8-byte) loads without bank
// conflicts.  mma.sync and not tcgen05: with at most 8 query rows a tile of 128
// would be 1/16 full, and codes would have to go back to shared memory as fp16
// between their copy and the product.
//
// Bound by DRAM for long rows, with the instructions that widen the codes close
// behind: 64 sequences of up to 64K tokens of 8 heads, d 128 (4.4 GB of codes), 624
// us, 7.1 TB/s; one of 128K 49 us, of which 5 pass before the first stage is there
// and 8 between the first and the last CTA's end (some multiprocessors get a tenth
// less of the memory's rate) and in the join; 1025 tokens of 2 heads 7 us.  Twelve
// warps of two stages: where these took 617 us on the 64 sequences, eight of three
// took 707, ten, which leave two of the four schedulers a warp short, 787, and
// sixteen of single blocks 706.
#include <cuda_fp16.h>

#include "compkv_launch.h"
#include "decode_common.cuh"
#include "kv8.cuh"

namespace compkv {

namespace {

constexpr int kPair = 2;     // blocks of a stage
constexpr int kHeads = 2;    // heads joined at a time
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLift = 14.f;  // weights are kept below 2^14: fp16 ends at 2^16
constexpr float kUnit = 0x1p-24f;  // of outputs until they are divided: with the lift, 2^-10 of the weighted sums, so that
                                   // values up to the end of fp32 have room for 512 tokens and more

// Shared memory, from a 1024-byte boundary on.
template <int D, bool SPARSE>
struct Smem8 {
  static constexpr int kWarps = SPARSE ? 8 : 12, kThreads = 32 * kWarps;
  static constexpr int kSlots = D == 128 ? 2 : 4;                // stages of a warp's ring
  static constexpr int kStage = 2 * kPair * kBlock * D;          // K blocks, then V blocks
  alignas(1024) uint8_t ring[kWarps][kSlots][kStage];
  float vbar[SPARSE ? kWarps : 1][kSlots][kPair][D];  // mean values of a stage's blocks (selections only)
  uint4 q[D / 16][32];                // A fragments of the queries (high, low, high, low)
  float part[kWarps][kHeads][D];      // the warps' outputs of two heads; parts of a join
  float comp[SPARSE ? kMaxG : 1][D];  // this segment's share of the compensation sums
  float scale[kWarps][kSlots][2 * kPair];
  int block[kWarps][kSlots][kPair];   // a stage's blocks (selections only)
  float ref[kWarps + 1][kMaxG];       // references (log2) and sums of the parts; the last: compensation
  float sum[kWarps + 1][kMaxG];
  float qs[kMaxG];                    // factor of a head's scores
  uint64_t full[kWarps][kSlots];
  int tokens[kMaxBatch];              // of each sequence
  int stages[kMaxBatch];              // stages of each of its units
  int pitch[kMaxBatch];               // and their distance in the row
  int first[kMaxBatch + 1];           // first stage of its first unit
  int streamed[kMaxBatch];            // the stream's plan (selections only)
  int soff[kMaxBatch + 1];
  int seg;
  int valid;                          // entries of the unit's selection
  int last;                           // this CTA has left the unit's last segment
};

// Stages of a run.  Short rows: no run shorter than a stage for each warp, nor a little longer.
__device__ __forceinline__ int run_stages(int total, int ctas, int warps) {
  const int per = (total + ctas - 1) / ctas;
  return per <= 2 * warps ? max(1, (per + warps - 1) / warps) * warps : per;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// d += A B, fp16 inputs
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = A B
__device__ __forceinline__ void mma_f16_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ void split_f16(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = as_u32(h);
  lo = as_u32(__floats2half2_rn(x - f.x, y - f.y));
}

// Four codes as two pairs of fp16, in units of kCode: coordinates 0 and 1, then 2 and 3 (e4m3), or 0 and 2, then 1 and 3
// (int8).  A byte on its own is a subnormal fp16 number, byte * 2^-24, so an int8 code is made unsigned, put in place, and
// the 128 taken off again: exactly, before the products, whose sums would otherwise carry 128 times the queries or the
// weights through every step (64 sequences of up to 64K tokens 624 us; with products that start from -128 times these sums
// 612, and errors two to four times as large, more where a block has wide channels).  e4m3 has an instruction (16 x 64K: 196
// us; its bits shifted into place, 263).
template <int KV>
struct Wide {
  static constexpr float kCode = KV == kKvInt8 ? 0x1p-24f : 1.f;
  static __device__ __forceinline__ void pairs(uint32_t w, uint32_t& a, uint32_t& b) {
    if constexpr (KV == kKvInt8) {
      const uint32_t x = w ^ 0x80808080u, most = 0x00800080u;
      const uint32_t lo = x & 0x00ff00ffu, hi = __byte_perm(x, 0u, 0x4341);
      const __half2 bias = *reinterpret_cast<const __half2*>(&most);
      a = as_u32(__hsub2(*reinterpret_cast<const __half2*>(&lo), bias));
      b = as_u32(__hsub2(*reinterpret_cast<const __half2*>(&hi), bias));
    } else {
      const __half2_raw l = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w, __NV_E4M3);
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
      a = *reinterpret_cast<const uint32_t*>(&l);
      b = *reinterpret_cast<const uint32_t*>(&h);
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
  float2 acc[D / 16][2];
  __device__ __forceinline__ void reset() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) acc[i][0] = acc[i][1] = make_float2(0.f, 0.f);
  }
};

// What a block of a stage is: its tokens (0: not there), its scales, and what comes off of the compensation sums.
struct Block8 {
  int n;
  float ks, vs;        // (vs brings a product to kUnit)
  float zb;            // zbar of head r, natural units
  const float* vbar;   // mean value; null: nothing comes off
};

// This lane's places in a block: its token's key chunks, and its four tokens' values (two rows; the other two 8 further).
template <int D>
struct Places {
  int k[D / 64], v[2];
  __device__ __forceinline__ explicit Places(int lane) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int x = 0; x < D / 64; ++x) k[x] = chunk_at<D>(token_of<D>(r), c * (D / 64) + x);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int t = token_of<D>(2 * c + j);
      v[j] = D == 128 ? chunk_at<D>(t, r) : chunk_at<D>(t, r >> 1) + (r & 1) * 8;
    }
  }
};

template <int D, int KV, bool SPARSE>
__device__ __forceinline__ void attend_pair(State<D>& st, const uint8_t* stage, const uint4 (*qf)[32], float qs,
                                            const Block8 (&blk)[kPair], const Places<D>& at, int lane) {
  constexpr int KS = D / 16, B8 = kBlock * D, HALF = 8 * D;  // steps; bytes of a block, and of eight of its tokens
  using Wd = Wide<KV>;
  const int r = lane >> 2, c = lane & 3;
  // ---- scores
  float s[kPair][2][4];
#pragma unroll
  for (int x = 0; x < KS / 4; ++x) {
    uint4 w[kPair][2];
#pragma unroll
    for (int i = 0; i < kPair; ++i)
#pragma unroll
      for (int t = 0; t < 2; ++t) w[i][t] = *reinterpret_cast<const uint4*>(stage + i * B8 + t * HALF + at.k[x]);
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const uint4 q = qf[4 * x + y][lane];
#pragma unroll
      for (int i = 0; i < kPair; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          uint32_t b0, b1;
          Wd::pairs(y == 0 ? w[i][t].x : y == 1 ? w[i][t].y : y == 2 ? w[i][t].z : w[i][t].w, b0, b1);
          if (x == 0 && y == 0) mma_f16_new(s[i][t], q.x, q.y, q.z, q.w, b0, b1);
          else mma_f16(s[i][t], q.x, q.y, q.z, q.w, b0, b1);
        }
    }
  }
  // ---- weights: head r at tokens token_of(2c), token_of(2c + 1) and 8 further
  float z[kPair][4], bm = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPair; ++i) {
    const float f = qs * blk[i].ks * (1.f / Wd::kCode);
#pragma unroll
    for (int e = 0; e < 4; ++e) z[i][e] = (s[i][e >> 1][e & 1] + s[i][e >> 1][2 + (e & 1)]) * f;
    if (blk[i].n < kBlock) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (8 * (e >> 1) + token_of<D>(2 * c + (e & 1)) >= blk[i].n) z[i][e] = -INFINITY;
    }
    bm = fmaxf(fmaxf(fmaxf(z[i][0], z[i][1]), fmaxf(z[i][2], z[i][3])), bm);
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
  if (__any_sync(0xffffffffu, bm > st.m)) {
    const float mn = fmaxf(st.m, bm);
    const float fo = st.m == -INFINITY ? 0.f : ex2(st.m - mn);
    const float2 fs = make_float2(__shfl_sync(0xffffffffu, fo, 8 * c), __shfl_sync(0xffffffffu, fo, 8 * c + 4));
    st.l *= fo;
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
      st.acc[mt][0] = __fmul2_rn(st.acc[mt][0], fs);
      st.acc[mt][1] = __fmul2_rn(st.acc[mt][1], fs);
    }
    st.m = mn;
  }
  const float low = st.m == -INFINITY ? 0.f : st.m - kLift;
  // ---- outputs
  const uint8_t* vals = stage + kPair * B8;
#pragma unroll
  for (int i = 0; i < kPair; ++i) {
    uint32_t ph[2], pl[2];
    float p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = ex2(z[i][e] - low);
    split_f16(p[0], p[1], ph[0], pl[0]);
    split_f16(p[2], p[3], ph[1], pl[1]);
    st.l += (p[0] + p[1]) + (p[2] + p[3]);  // this lane's part
    float2 off = make_float2(0.f, 0.f);
    if constexpr (SPARSE) {
      const float fn = blk[i].vbar ? ex2(e2[i] - low) : 0.f;
      if (c == 0) st.l -= fn;
      off.x = -kUnit * __shfl_sync(0xffffffffu, fn, 8 * c);
      off.y = -kUnit * __shfl_sync(0xffffffffu, fn, 8 * c + 4);
    }
    uint32_t w[4][D / 32];  // values of this lane's four tokens: token_of(2c), token_of(2c + 1), and 8 further
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint8_t* from_row = vals + i * B8 + (j >> 1) * HALF + at.v[j & 1];
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(from_row);
        w[j][0] = x.x;
        w[j][1] = x.y;
        w[j][2] = x.z;
        w[j][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(from_row);
        w[j][0] = x.x;
        w[j][1] = x.y;
      }
    }
    if (KV == kKvE4m3 && blk[i].n < kBlock) {  // behind the last token there may be codes of NaN
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (token_of<D>(2 * c + (j & 1)) + 8 * (j >> 1) >= blk[i].n) {
#pragma unroll
          for (int x = 0; x < D / 32; ++x) w[j][x] = 0u;
        }
    }
    const float2 vs = make_float2(blk[i].vs, blk[i].vs);
#pragma unroll
    for (int x = 0; x < D / 32; ++x) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        // two coordinates of two tokens each, so that each pair of fp16 has one coordinate's two tokens
        constexpr bool I8 = KV == kKvInt8;
        const uint32_t sel = y ? (I8 ? 0x7632 : 0x7362) : (I8 ? 0x5410 : 0x5140);
        uint32_t a0, a1, a2, a3;
        Wd::pairs(__byte_perm(w[0][x], w[1][x], sel), a0, a1);
        Wd::pairs(__byte_perm(w[2][x], w[3][x], sel), a2, a3);
        float o[4];
        mma_f16_new(o, a0, a1, a2, a3, ph[0], ph[1]);
        mma_f16(o, a0, a1, a2, a3, pl[0], pl[1]);
        float2(&acc)[2] = st.acc[2 * x + y];
        acc[0] = __ffma2_rn(make_float2(o[0], o[1]), vs, acc[0]);
        acc[1] = __ffma2_rn(make_float2(o[2], o[3]), vs, acc[1]);
        if constexpr (SPARSE) {
          if (blk[i].vbar) {
            const float2 v = reinterpret_cast<const float2*>(blk[i].vbar + r * (D / 8))[2 * x + y];
            acc[0] = __ffma2_rn(off, make_float2(v.x, v.x), acc[0]);
            acc[1] = __ffma2_rn(off, make_float2(v.y, v.y), acc[1]);
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
__device__ __forceinline__ float4 load_query(const Attend8Args& a, int64_t unit, int head, int lane) {
  if (head >= a.G || lane >= D / 4) return make_float4(0.f, 0.f, 0.f, 0.f);
  const int64_t at = (unit * a.G + head) * D + 4 * lane;
  if (!a.q_bf16) return __ldcg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.q) + at));
  const uint2 w = __ldcg(reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(a.q) + at));
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}
template <int D, int KV, bool SPARSE>
__device__ __forceinline__ void stage_query(Smem8<D, SPARSE>& sm, float4 x, int head, int lane) {
  constexpr int KS = D / 16;
  uint32_t bits = max(max(__float_as_uint(x.x) & 0x7fffffffu, __float_as_uint(x.y) & 0x7fffffffu),
                      max(__float_as_uint(x.z) & 0x7fffffffu, __float_as_uint(x.w) & 0x7fffffffu));
  bits = __reduce_max_sync(0xffffffffu, bits);
  // 2^e <= largest magnitude < 2^(e + 1), kept where 2^(13 - e) and 2^(e - 13) are normal numbers (an infinity or a NaN
  // makes NaN of its head's scores either way)
  const int e = max(-113, min(126, (int)(bits >> 23) - 127));
  const float up = __uint_as_float((uint32_t)(13 - e + 127) << 23);
  if (KV == kKvInt8) {  // the order in which codes come apart
    const float y = x.y;
    x.y = x.z;
    x.z = y;
  }
  uint4 f;
  split_f16(x.x * up, x.y * up, f.x, f.y);
  split_f16(x.z * up, x.w * up, f.z, f.w);
  if (lane < D / 4) sm.q[lane % KS][head * 4 + lane / KS] = f;
  const float root = D == 128 ? 0.08838834764831845f : 0.125f;
  if (lane == 0) sm.qs[head] = __uint_as_float((uint32_t)(e - 13 + 127) << 23) * (kLog2e * root);
}

// This segment's share of the unit's compensation sums: the stream's records p, p + C, ... at their common reference.
template <int D, bool SPARSE>
__device__ __forceinline__ void stage_compensation(Smem8<D, SPARSE>& sm, const Attend8Args& a, int i0, int nseg, int p, int C,
                                                   int tid) {
#pragma unroll 1
  for (int item = tid; item < a.G * D / 4; item += Smem8<D, SPARSE>::kThreads) {
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
    *reinterpret_cast<float4*>(&sm.comp[g][col]) = make_float4(A.x * kUnit, A.y * kUnit, A.z * kUnit, A.w * kUnit);
    if (col == 0) {
      sm.ref[Smem8<D, SPARSE>::kWarps][g] = R * kLog2e;
      sm.sum[Smem8<D, SPARSE>::kWarps][g] = W;
    }
  }
}

template <int D>
__device__ __forceinline__ void put_out(const Attend8Args& a, int64_t unit, int g, int col, float4 acc, float l) {
  // a row without tokens is zero; a sum that is NaN goes through
  const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
  constexpr float one = 1.f / kUnit;
  const float4 y = make_float4(acc.x * inv * one, acc.y * inv * one, acc.z * inv * one, acc.w * inv * one);
  const int64_t at = (unit * a.G + g) * D + col;
  if (a.q_bf16) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = y;
  }
}

// The factor that brings a part from its reference to M; a part without tokens has no reference, and a sum of zero or NaN.
__device__ __forceinline__ float part_factor(float ref, float M) { return ref == -INFINITY ? 0.f : ex2(ref - M); }
__device__ __forceinline__ void add_part(float4& A, float& S, float4 v, float s, float f) {
  A.x = fmaf(v.x, f, A.x);
  A.y = fmaf(v.y, f, A.y);
  A.z = fmaf(v.z, f, A.z);
  A.w = fmaf(v.w, f, A.w);
  S = fmaf(s, f, S);
}

// The unit's segments joined: those of runs c0 .. c0 + C - 1, whose first may have come from another unit's stages.
// Where the rows have fewer items than there are threads, groups of threads take a share of the segments each.
template <int D, bool SPARSE>
__device__ __forceinline__ void join_segments(Smem8<D, SPARSE>& sm, const Attend8Args& a, int64_t unit, int c0, int C, bool tail,
                                              int tid) {
  const int items = a.G * D / 4, groups = max(1, min(Smem8<D, SPARSE>::kThreads, (int)sizeof(sm.part) / 24) / items);
  float4* accs = reinterpret_cast<float4*>(sm.part);                                   // [groups][items]
  float2* refs = reinterpret_cast<float2*>(accs + groups * items);
#pragma unroll 1
  for (int x = tid; x < items * groups; x += Smem8<D, SPARSE>::kThreads) {
    const int item = x % items, group = x / items, g = item / (D / 4), col = 4 * (item % (D / 4));
    float M = -INFINITY, S = 0.f;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = group; k0 < C; k0 += 4 * groups) {
      float2 e[4];
      float4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + j * groups;
        const int64_t at = (int64_t)(2 * (c0 + k) + (k == 0 && tail)) * a.G + g;
        e[j] = k < C ? __ldcg(a.ml + at) : make_float2(-INFINITY, 0.f);
        v[j] = k < C ? __ldcg(reinterpret_cast<const float4*>(a.acc + at * D + col)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float mn = M;
#pragma unroll
      for (int j = 0; j < 4; ++j) mn = fmaxf(mn, e[j].x);
      const float fo = part_factor(M, mn);
      A = make_float4(A.x * fo, A.y * fo, A.z * fo, A.w * fo);
      S *= fo;
#pragma unroll
      for (int j = 0; j < 4; ++j) add_part(A, S, v[j], e[j].y, part_factor(e[j].x, mn));
      M = mn;
    }
    if (groups == 1) {
      put_out<D>(a, unit, g, col, A, S);
    } else {
      accs[x] = A;
      refs[x] = make_float2(M, S);
    }
  }
  if (groups == 1) return;
  __syncthreads();
  if (tid < items) {
    float M = -INFINITY, S = 0.f;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < groups; ++k) M = fmaxf(M, refs[k * items + tid].x);
    for (int k = 0; k < groups; ++k) {
      const float2 e = refs[k * items + tid];
      add_part(A, S, accs[k * items + tid], e.y, part_factor(e.x, M));
    }
    put_out<D>(a, unit, tid / (D / 4), 4 * (tid % (D / 4)), A, S);
  }
  __syncthreads();
}

template <int D, int KV, bool SPARSE>
__global__ void __launch_bounds__(Smem8<D, SPARSE>::kThreads, 1) attend8_kernel(const __grid_constant__ Attend8Args a) {
  using Smem = Smem8<D, SPARSE>;
  extern __shared__ __align__(16) uint8_t raw[];
  Smem& sm = *reinterpret_cast<Smem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  constexpr int B8 = kBlock * D, SLOTS = Smem::kSlots, W = Smem::kWarps, T = Smem::kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < W * SLOTS) mbar_init(&sm.full[0][0] + tid, 1 + 2 * kPair);
  if (tid == 0) {
    sm.valid = 0;
    fence_mbar_init();
  }
  // What came before on the stream may have written the cache, its lengths, the queries and the selection.  Behind the
  // stream of a given selection, all of these are older than the stream, which waited for them before it let this
  // kernel start: only its records have to be waited for, and copies and queries come first.
  const bool early = SPARSE && !a.selects;
  if (!early) {
    pdl_wait();
  }
  if (warp == 0) {
    // the row of stages, from the lengths; in a short row every unit begins a run of its own
    int st[kMaxBatch / 32], sum = 0, padded = 0;
#pragma unroll
    for (int k = 0; k < kMaxBatch / 32; ++k) {
      const int s = 32 * k + lane;
      st[k] = 0;
      if (s < a.B) {
        bool fits;
        const int L = call_tokens(__ldcg(a.seq_len + s), a.cap_blocks[s], false, &fits), n = ceil_blocks(L);
        sm.tokens[s] = L;
        st[k] = ((SPARSE ? min(n, a.K) : n) + kPair - 1) / kPair;
        sm.stages[s] = st[k];
      }
      sum += st[k];
      padded += (st[k] + W - 1) / W * W;
    }
    padded = __reduce_add_sync(0xffffffffu, padded) * a.Hkv;
    const bool pad = padded <= W * (int)gridDim.x;
    int at = 0;
#pragma unroll
    for (int k = 0; k < kMaxBatch / 32; ++k) {
      const int s = 32 * k + lane;
      const int pitch = pad ? (st[k] + W - 1) / W * W : st[k];
      int incl = pitch * a.Hkv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (s < a.B) {
        sm.pitch[s] = pitch;
        sm.first[s] = at + incl - pitch * a.Hkv;
      }
      at += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) sm.first[a.B] = at;
  } else if (SPARSE && warp == 1) {
    // the stream's plan
    for (int s = lane; s < a.B; s += 32) {
      bool fits;
      const int L = call_tokens(__ldcg(a.seq_len + s), a.cap_blocks[s], false, &fits);
      sm.streamed[s] = streamed_blocks(L, false, a.selects, a.K, false);
    }
    __syncwarp();
    plan_warp(sm.streamed, a.B, a.Hkv, a.stream_P, stage_blocks(a.r, a.G), sm.soff, &sm.seg, lane);
  }
  __syncthreads();
  const int total = sm.first[a.B], per = run_stages(total, (int)gridDim.x, W);
  const int lo = min(total, (int)blockIdx.x * per), hi = min(total, lo + per);

  // ---- this warp's copies: stages lo + warp, lo + warp + W, ..., ahead of their use
  int to_issue = lo + warp, flying = 0, issue_slot = 0;
  int si = 0, unit_first = 0, unit_end = 0, stages_issue = 0, n_issue = 0, y_issue = 0;  // the unit of stage to_issue
  int64_t su = 0, row_issue = 0;
  const uint64_t pol = policy_evict_first();
  // block of entry i of a unit's selection (-1: none, or not a valid one)
  auto entry = [&](int64_t unit, int i, int n) -> int {
    if (i >= min(n, a.K)) return -1;
    const int* sel = a.sel + unit * a.K;
    const int e = __ldcg(sel + i), prev = i > 0 ? __ldcg(sel + i - 1) : -1;
    return e >= 0 && e < n && (i == 0 || (prev >= 0 && prev < e)) ? e : -1;
  };
  auto fill = [&]() {
#pragma unroll 1
    while (flying < SLOTS && to_issue < hi) {
      if (to_issue >= unit_end) {
#pragma unroll 1
        while (to_issue >= sm.first[si + 1]) ++si;
        const int pitch = sm.pitch[si], h = (to_issue - sm.first[si]) / pitch;
        unit_first = sm.first[si] + h * pitch;
        unit_end = unit_first + pitch;
        stages_issue = sm.stages[si];
        n_issue = ceil_blocks(sm.tokens[si]);
        su = (int64_t)si * a.Hkv + h;
        row_issue = a.seq_row0[si] + (int64_t)h * a.cap_blocks[si];
        y_issue = (int)((a.layer_row0 + row_issue) * kBlock);
      }
      const int j = to_issue - unit_first;
      const uint32_t missing = to_issue == a.lost ? 16 : 0;  // (tests: more is announced than comes)
      to_issue += W;
      if (j >= stages_issue) continue;  // behind a unit's last stage
      uint64_t* bar = &sm.full[warp][issue_slot];
      uint8_t* dst = sm.ring[warp][issue_slot];
      int b0 = kPair * j, b1 = b0 + 1 < n_issue ? b0 + 1 : -1;
      if (SPARSE) {
        b0 = entry(su, kPair * j, n_issue);
        b1 = entry(su, kPair * j + 1, n_issue);
      }
      __syncwarp();  // the slot's previous contents are read
      // the scales: one lane each
      if (lane < 2 * kPair) {
        const int mine = lane & 1 ? b1 : b0;
        if (mine >= 0) {
          const float* src = (lane < kPair ? a.kv8.kscale : a.kv8.vscale) + row_issue + mine;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&sm.scale[warp][issue_slot][lane])), "l"(src)
                       : "memory");
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
      }
      if (lane == 0) {
        if constexpr (SPARSE) {
          mbar_arrive_expect_tx(bar, ((b0 >= 0) + (b1 >= 0)) * (2 * B8 + D * 4) + missing);
#pragma unroll
          for (int i = 0; i < kPair; ++i) {
            const int b = i ? b1 : b0;
            sm.block[warp][issue_slot][i] = b;
            if (b < 0) continue;
            tma_2d(dst + i * B8, a.k16, 0, y_issue + b * kBlock, bar, pol);
            tma_2d(dst + (kPair + i) * B8, a.v16, 0, y_issue + b * kBlock, bar, pol);
            bulk_g2s(sm.vbar[warp][issue_slot][i], a.vbar + (row_issue + b) * D, D * 4, bar);
          }
        } else {
          // (a pair's second block may be another unit's, or lie behind the cache, which reads as zero: it is masked)
          mbar_arrive_expect_tx(bar, Smem::kStage + missing);
          tma_2d(dst, a.k32, 0, y_issue + b0 * kBlock, bar, pol);
          tma_2d(dst + kPair * B8, a.v32, 0, y_issue + b0 * kBlock, bar, pol);
        }
      }
      ++flying;
      if (++issue_slot == SLOTS) issue_slot = 0;
    }
  };
  // ---- the run's segments
  const Places<D> places(lane);
  int slot = 0, phase = 0, s = 0;
  bool ok = true, waited = !early, begun = false;
  State<D> st;
  float4 q;
  for (int at = lo; at < hi;) {
    while (at >= sm.first[s + 1]) ++s;
    const int h = (at - sm.first[s]) / sm.pitch[s];
    const int unit0 = sm.first[s] + h * sm.pitch[s], unit1 = unit0 + sm.stages[s];  // the unit's stages
    if (at >= unit1) {
      at = unit0 + sm.pitch[s];
      continue;
    }
    const int end = min(hi, unit1);
    const int64_t unit = (int64_t)s * a.Hkv + h;
    const int L = sm.tokens[s], n = ceil_blocks(L);
    const int64_t row0 = a.seq_row0[s] + (int64_t)h * a.cap_blocks[s];
    const int c0 = unit0 / per, C = (unit1 - 1) / per - c0 + 1;  // runs that have a part of this unit
    const bool tail = c0 * per < unit0;                          // the first of them came from another unit's stages
    if (!begun) {  // the queries of the first segment, on their way before its copies
      q = load_query<D>(a, unit, warp, lane);
      fill();
      begun = true;
    }
    if (warp < kMaxG) stage_query<D, KV>(sm, q, warp, lane);
    if (SPARSE) {
      int valid = 0, wrong = 0;
#pragma unroll 1
      for (int i = tid; i < a.K; i += T) {
        const int e = __ldcg(a.sel + unit * a.K + i), prev = i > 0 ? __ldcg(a.sel + unit * a.K + i - 1) : -1;
        const bool good = e >= 0 && e < n && (i == 0 || (prev >= 0 && prev < e));
        valid += good;
        wrong |= (e >= 0 && !good) || e < -1;
      }
      valid = __reduce_add_sync(0xffffffffu, valid);
      if (lane == 0 && valid) atomicAdd(&sm.valid, valid);
      if (__any_sync(0xffffffffu, wrong) && lane == 0 && (int)blockIdx.x == c0)
        set_error(a.status, kDevBadSelection, s, h, 61);
      if (!waited) {
        pdl_wait();
      }
      waited = true;
      if (!a.no_comp) {
        const int nseg = (sm.streamed[s] + sm.seg - 1) / sm.seg;
        stage_compensation<D>(sm, a, sm.soff[s] + h * nseg, nseg, (int)blockIdx.x - c0, C, tid);
      }
    }
    __syncthreads();
    {
      // the next segment's queries, a segment ahead: behind the copies in flight they take as long as these
      int sq = s;
      const int there = unit0 + sm.pitch[s];
      if (there < hi) {
        while (there >= sm.first[sq + 1]) ++sq;
        const int hq = (there - sm.first[sq]) / sm.pitch[sq];
        q = load_query<D>(a, (int64_t)sq * a.Hkv + hq, warp, lane);
      }
    }
    const bool comp = SPARSE && !a.no_comp && sm.valid < n;
    const float qs = sm.qs[lane >> 2];
    st.reset();
    // (a warp whose wait ran out reads no further stage: its ring is not filled again, and the block numbers there are those
    // of other stages)
    for (int i = at + (warp - (at - lo) % W + W) % W; ok && i < end; i += W) {
      Block8 blk[kPair];
      if (SPARSE) __syncwarp();  // the slot's block numbers are there
#pragma unroll
      for (int k = 0; k < kPair; ++k) {
        const int x = kPair * (i - unit0) + k;
        const int b = SPARSE ? sm.block[warp][slot][k] : x < n ? x : -1;
        blk[k].n = b < 0 ? 0 : min(kBlock, L - b * kBlock);
        blk[k].zb = comp && b >= 0 && lane >> 2 < a.G ? __ldcg(a.zs + (row0 + b) * pad_g(a.G) + (lane >> 2)) : 0.f;
        blk[k].vbar = comp && b >= 0 ? sm.vbar[SPARSE ? warp : 0][slot][k] : nullptr;
      }
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sm.full[warp][slot], phase, a.status, s, h, 71));
      if (ok) {
#pragma unroll
        for (int k = 0; k < kPair; ++k) {
          blk[k].ks = blk[k].n ? sm.scale[warp][slot][k] : 0.f;
          blk[k].vs = blk[k].n ? sm.scale[warp][slot][kPair + k] * (kUnit / Wide<KV>::kCode) : 0.f;
        }
        if (blk[0].n | blk[1].n) attend_pair<D, KV, SPARSE>(st, sm.ring[warp][slot], sm.q, qs, blk, places, lane);
        --flying;
        fill();
      }
      if (++slot == SLOTS) {
        slot = 0;
        phase ^= 1;
      }
    }
    at = end;
    // ---- the warps' parts and the compensation share, two heads at a time
    float l = st.l;
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if ((lane & 3) == 0) {
      sm.ref[warp][lane >> 2] = st.m - kLift;
      sm.sum[warp][lane >> 2] = l;
    }
    const int place = 2 * (int)blockIdx.x + ((int)blockIdx.x == c0 && tail);  // of this segment in the workspace
#pragma unroll 1
    for (int g0 = 0; g0 < a.G; g0 += kHeads) {
      const int c = lane & 3, r = lane >> 2;
      if (2 * c == g0) {  // heads 2c and 2c + 1
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float2* to = reinterpret_cast<float2*>(&sm.part[warp][e][r * (D / 8)]);
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt) {
            const float2 u = st.acc[mt][0], v = st.acc[mt][1];
            to[mt] = e ? make_float2(u.y, v.y) : make_float2(u.x, v.x);
          }
        }
      }
      __syncthreads();
      if (SPARSE && tid == 0) sm.valid = 0;
      for (int item = tid; item < min(kHeads, a.G - g0) * D / 4; item += T) {
        const int g = g0 + item / (D / 4), col = 4 * (item % (D / 4));
        float M = comp ? sm.ref[W][g] : -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, sm.ref[w][g]);
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
        float S = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w)
          add_part(A, S, *reinterpret_cast<const float4*>(&sm.part[w][g - g0][col]), sm.sum[w][g],
                   part_factor(sm.ref[w][g], M));
        if (comp)
          add_part(A, S, *reinterpret_cast<const float4*>(&sm.comp[SPARSE ? g : 0][col]), sm.sum[W][g],
                   part_factor(sm.ref[W][g], M));
        if (C == 1) {
          put_out<D>(a, unit, g, col, A, S);
        } else {
          __stcg(reinterpret_cast<float4*>(a.acc + ((int64_t)place * a.G + g) * D + col), A);
          if (col == 0) __stcg(a.ml + (int64_t)place * a.G + g, make_float2(M, S));
        }
      }
      __syncthreads();
    }
    if (C == 1) continue;
    // ---- whoever leaves the unit's last segment joins them
    if (tid == 0) {  // (the barrier above orders the CTA's stores before this thread's fence)
      __threadfence();
      sm.last = atomicAdd(a.arrive + unit, 1) == C - 1;
      if (sm.last) a.arrive[unit] = 0;
      __threadfence();
    }
    __syncthreads();
    if (!sm.last) continue;
    join_segments<D>(sm, a, unit, c0, C, tail, tid);
  }
  if (!waited) pdl_wait();
  if (!ok) {  // a wait ran out: let the copies in flight land before the CTA's memory goes
#pragma unroll 1
    for (int k = 0; k < SLOTS; ++k) mbar_drain_bounded(&sm.full[warp][k]);
  }
  // rows of sequences without tokens
#pragma unroll 1
  for (int u = blockIdx.x; u < a.B * a.Hkv; u += gridDim.x) {
    if (sm.stages[u / a.Hkv]) continue;
    for (int i = tid; i < a.G * D / 4; i += T)
      put_out<D>(a, u, i / (D / 4), 4 * (i % (D / 4)), make_float4(0.f, 0.f, 0.f, 0.f), 0.f);
  }
}

template <int D, int KV, bool SPARSE>
cudaError_t attend8_as(const Attend8Args& a, cudaStream_t st) {
  Attend8Args args = a;
  void* argv[] = {&args};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.P);
  cfg.blockDim = dim3(Smem8<D, SPARSE>::kThreads);
  cfg.dynamicSmemBytes = sizeof(Smem8<D, SPARSE>) + 1024;
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
template <int D, int KV, bool SPARSE>
cudaError_t prepare_as() {
  static_assert(sizeof(Smem8<D, SPARSE>) + 1024 <= 232448, "shared memory of a CTA");
  return raise_smem_limit(reinterpret_cast<const void*>(&attend8_kernel<D, KV, SPARSE>),
                          (int)sizeof(Smem8<D, SPARSE>) + 1024);
}
template <int D>
cudaError_t prepare_d() {
  cudaError_t e = prepare_as<D, kKvInt8, true>();
  if (e == cudaSuccess) e = prepare_as<D, kKvInt8, false>();
  if (e == cudaSuccess) e = prepare_as<D, kKvE4m3, true>();
  return e == cudaSuccess ? prepare_as<D, kKvE4m3, false>() : e;
}

}  // namespace

cudaError_t prepare_attend8(int d) { return d == 128 ? prepare_d<128>() : prepare_d<64>(); }
cudaError_t launch_attend8(const Attend8Args& a, cudaStream_t st) {
  return a.d == 128 ? attend8_d<128>(a, st) : attend8_d<64>(a, st);
}

}  // namespace compkv
