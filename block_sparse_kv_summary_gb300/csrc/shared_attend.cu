// Exact attention of every sequence over a prefix that one sequence of the
// cache holds for all and over its own tokens, under one softmax:
//   out = sum_j e^(z_j) v_j / sum_j e^(z_j),   z_j = q . k_j / sqrt(d),
// j over the prefix's tokens and the sequence's own.
//
// A prefix is read once for up to 256 query rows (sequences x query heads of a
// KV head; 128 in fp32); a sequence's own tokens are one more item with G
// rows.  Items are walked in tiles of 128 keys.  One persistent CTA per
// multiprocessor takes an equal run of the tiles of all items, so that a long
// prefix and few rows still fill the chip; each piece of an item leaves its
// rows' reference, sum and unnormalised output in the workspace, and when all
// CTAs have left theirs (a cooperative launch) their warps join the pieces of
// a row each.  A second kernel for the join took 0.5 to 3 us more on the GPU
// and 5 us more to launch.
//
// Within a CTA (tcgen05; a step is one K/V tile times 128 rows, one or two
// steps a tile, one step in flight behind the other):
//   warp 16  copies K and V tiles by tensor maps into a ring of stages,
//   warp 17  issues S = Q K^T into one of two TMEM buffers,
//   warp 18  issues O += P V,
//   warps 0-15 load Q, take the weights and their sum (thread = row and quarter
//            of the keys), and write the weights P over S in TMEM.  Eight warps
//            with half the keys each took as long for a step and longer for the
//            queries and outputs of many rows (512 rows behind 64K: 43 us, 35
//            with sixteen).
// Measured behind a long prefix, d 128: a tile with one step takes 1.3 us, the
// time its K and V need from DRAM; with two, 1.8 us: their scores, weights and
// outputs wait for one another, and two steps are in flight.  In fp32 a step
// takes 1.9 to 2.1 us, most of it 48 products of 16 on the tensor cores.  d 64:
// 0.9 to 1.1, 1.7 and 1.4 us.
//
// Weights are e^(z - reference).  The reference is the row's maximum in the
// piece's first tile and stays while the weights of a tile add up to less than
// 2^30: floating point loses nothing by a common factor, and the join divides
// it out.  Only where they do not is the tile's maximum taken, O scaled and
// the tile done again, so that no other tile pays for a maximum.
//
// bf16 queries take one product each, and their weights are rounded to bf16,
// as the result is, which doubles the variance of its error (2.3e-3 of the
// result in the mean square against 1.7e-3 from its own rounding).  The weights'
// sum is that of the rounded ones.  Weights in two parts bring 1.7e-3 back and
// cost 28 % (64 sequences behind 128K: 187 us in place of 138), so whoever needs
// those bits passes fp32 queries.  O stays in TMEM over the tiles of a piece: its
// truncation (below) is far under a bf16 step.  fp32 queries and weights are split into three bf16 parts
// of 8 bits each and multiplied part by part (K and V are bf16 as they are),
// the smallest first: the accumulator truncates what each addition of 16
// products loses below its last bit, always towards zero, and only the last
// part's additions meet a large accumulator.  For the same reason O of a tile
// is added up over the tiles in registers, rounded to nearest: left in TMEM
// over 32K keys it came out 8e-6 too small.
#include "compkv_launch.h"

namespace compkv {

namespace {

constexpr int kTile = 128;                // keys of a tile, and query rows of an item at most
constexpr int kSoftmaxWarps = 16;
constexpr int kCols = kTile / (kSoftmaxWarps / 4);  // keys of a tile that a softmax thread has, for one row
constexpr int kThreads = 32 * (kSoftmaxWarps + 4);  // registers are dealt out by groups of four warps
constexpr float kMostWeight = 1073741824.f;  // 2^30: what a tile's weights of a row may add up to
constexpr size_t kSmemLimit = 232448;

// ---------------------------------------------------------------- the plan
// Work is dealt in units: a tile counts two, or three with more than 128 rows,
// and an item four more, and one for each 32 rows, for its queries and its
// outputs.  That is the proportion of bf16 and d 128 (1.3 and 1.8 us a tile, 2 to
// 3 us an item of a few rows, 7 us one of 256).  In fp32 a tile takes 2 us and in
// d 64 with few rows 0.9, so there an item counts too much or too little beside
// it, and CTAs with many short items end before or after the others.  CTA c of P
// takes the units [c T / P, (c + 1) T / P) of the T units of all entries and
// heads, in order, and the tiles that begin there.
struct Plan {
  int cum[kMaxSharedEntries + 1];         // units of all heads of the entries before e
  unsigned char last[kMaxSharedEntries];  // keys of its last tile
};

__device__ __forceinline__ int tile_units(const SharedArgs& a, int e) { return a.rows[e] > kTile ? 3 : 2; }
__device__ __forceinline__ int item_units(const SharedArgs& a, int e) { return 4 + a.rows[e] / 32; }
__device__ __forceinline__ int entry_units(const SharedArgs& a, const Plan& p, int e) {  // per head
  return (p.cum[e + 1] - p.cum[e]) / a.Hkv;
}
__device__ __forceinline__ int item_keys(const SharedArgs& a, const Plan& p, int e) {
  const int u = entry_units(a, p, e);
  return u ? ((u - item_units(a, e)) / tile_units(a, e) - 1) * kTile + p.last[e] : 0;
}
// By one warp; the caller synchronises.
__device__ void build_plan(const SharedArgs& a, Plan& p, int lane) {
  int base = 0;
  for (int e0 = 0; e0 < a.entries; e0 += 32) {
    const int e = e0 + lane;
    int u = 0;
    if (e < a.entries) {
      const int held = max(0, min(__ldcg(a.seq_len + a.holder[e]), a.cap[e])), most = a.most[e];
      const int len = max(0, min(held, most) - a.skip[e]);
      if (e < a.prefixes && held < most) set_error(a.status, kDevInvalidArg, a.holder[e], -1, 5);
      p.last[e] = (unsigned char)((len + kTile - 1) % kTile + 1);
      u = len ? ((len + kTile - 1) / kTile * tile_units(a, e) + item_units(a, e)) * a.Hkv : 0;
    }
    int x = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (e < a.entries) p.cum[e] = base + x - u;
    base += __shfl_sync(0xffffffffu, x, 31);
  }
  if (lane == 0) p.cum[a.entries] = base;
}

__device__ __forceinline__ int cta_unit(int c, int P, int total) { return (int)((int64_t)total * c / P); }

// The tiles [from, to) of an item that begin in the units [x, y) of the item.
struct Tiles {
  int from, to;
};
__device__ __forceinline__ Tiles tiles_between(const SharedArgs& a, int e, int x, int y) {
  const int w = tile_units(a, e), start = item_units(a, e);
  return {max(x - start + w - 1, 0) / w, max(y - start + w - 1, 0) / w};
}

// Walks the segments (pieces of items) of one CTA; every role walks alike.
struct Segment {
  int e, h, tile0, tile1;
  int tiles, last;  // of the whole item
  __device__ __forceinline__ int valid(int t) const { return t == tiles - 1 ? last : kTile; }
};
struct Walk {
  int u, end, e;
  __device__ __forceinline__ Walk(const SharedArgs& a, const Plan& p, int c) {
    const int total = p.cum[a.entries];
    u = cta_unit(c, a.P, total);
    end = cta_unit(c + 1, a.P, total);
    e = 0;
  }
  __device__ __forceinline__ bool next(const SharedArgs& a, const Plan& p, Segment& g) {
    while (u < end) {
      while (p.cum[e + 1] <= u) ++e;
      const int per = entry_units(a, p, e), at = u - p.cum[e];
      g.e = e;
      g.h = at / per;
      const int x = at - g.h * per, n = min(per - x, end - u);
      const Tiles t = tiles_between(a, e, x, x + n);
      u += n;
      g.tile0 = t.from;
      g.tile1 = t.to;
      g.tiles = (per - item_units(a, e)) / tile_units(a, e);
      g.last = p.last[e];
      if (g.tile1 > g.tile0) return true;
    }
    return false;
  }
};
// Workspace row of the first row of a segment of CTA c: segments follow one another by item or by CTA,
// and each step adds at least the rows of the segment before it (256 at most).
__device__ __forceinline__ int segment_row(const SharedArgs& a, int e, int h, int c) {
  return a.row0[e] + h * a.rows[e] + 256 * c;
}

// ---------------------------------------------------------------- tcgen05
__device__ __forceinline__ void tma_box(void* dst, const void* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
// Shared-memory operand with the 128-byte swizzle: `lead` and `stride` in bytes.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// kind::f16, bf16 x bf16 -> fp32, M = 128; the second operand is K-major, or N-major where `n_major`.
__device__ __forceinline__ constexpr uint32_t instruction(int n, bool n_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((n_major ? 1u : 0u) << 16) | ((uint32_t)(n / 8) << 17) |
         ((uint32_t)(kTile / 16) << 24);
}
// Issued by the warp's leader; the whole warp computes the operands, which then stand in uniform registers.
__device__ __forceinline__ uint32_t elect_leader() {
  uint32_t lead;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(lead));
  return lead;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}
// A value that all lanes hold, in a form that the compiler knows to be uniform: operands of tcgen05 stand in
// uniform registers, and moving each there anew costs as much as the product.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
// Registers of this warp from here on; every warp of its group of four says the same, and they have met between two
// changes.
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Loads of a lane's columns, complete when they return: the wait stands in the same statement, so that no use of
// the registers can move in front of it.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* f) {
  uint32_t* r = reinterpret_cast<uint32_t*>(f);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%2"
      "6,%27,%28,%29,%30,%31"
      "}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float* f) {
  uint32_t* r = reinterpret_cast<uint32_t*>(f);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15"
      "}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
      "%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16"
      "};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two floats rounded to bf16, `a` in the low half; what is left of them goes back into a and b.
__device__ __forceinline__ uint32_t split2(float& a, float& b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
  const float2 left = __ffma2_rn(make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)),
                                 make_float2(-1.f, -1.f), make_float2(a, b));
  a = left.x;
  b = left.y;
  return u;
}

// ---------------------------------------------------------------- the CTA
template <int D, int PARTS>
struct Shape {
  static constexpr int kHalf = kTile * 128;             // 64 coordinates of 128 rows, 128 bytes a row
  static constexpr int kStage = kHalf * (D / 64);       // a K or a V tile, or 128 rows of Q in one part
  static constexpr int kSub = PARTS == 1 ? 2 : 1;       // times 128 query rows of an item at most
  static constexpr int kQ = kStage * PARTS * kSub;
  static constexpr bool kTileO = PARTS == 3;            // O of one tile at a time; added up in registers
  // TMEM columns: two buffers of 128 scores and, over and behind them, up to three parts of weights; O
  static constexpr int kBuffer = PARTS == 3 ? 192 : 128;
  static constexpr int kO = 2 * kBuffer;
  static constexpr int kColumns = 512;
};
struct Control {
  Plan plan;
  unsigned char member[kMaxBatch];  // of the arguments: there a warp's lanes would read them one after another
  float row_max[kTile / kCols][kTile];  // [part of the keys][row]; sums at the end of a segment
  uint64_t full[8], empty[8], q_full, s_full[2], p_full[2], o_full[2];  // [tile & 1]
  uint32_t tmem;
  int abort;
};
template <int D, int PARTS>
__host__ __device__ constexpr int stages() {
  const size_t n = (kSmemLimit - sizeof(Control) - Shape<D, PARTS>::kQ) / Shape<D, PARTS>::kStage;
  return n > 8 ? 8 : (int)n;
}
template <int D, int PARTS>
__host__ __device__ constexpr size_t smem_bytes() {
  return Shape<D, PARTS>::kQ + (size_t)stages<D, PARTS>() * Shape<D, PARTS>::kStage + sizeof(Control);
}

// Bounded wait.  Once one wait of the CTA ran out, none waits any more: every
// role runs through its loops without touching memory, so all of them meet at
// the end.
__device__ __forceinline__ bool wait(Control* ctl, uint64_t* bar, uint32_t parity, int* status, int site) {
  if (mbar_try_wait(bar, parity)) return true;
  volatile int* abort = &ctl->abort;
  if (*abort) return false;
  if (mbar_wait_bounded(bar, parity, status, -1, -1, site)) return true;
  *abort = 1;
  return false;
}

// The same by a whole warp.
__device__ __forceinline__ bool warp_wait(Control* ctl, uint64_t* bar, uint32_t parity, int* status, int site) {
  const bool ok = wait(ctl, bar, parity, status, site);
  __syncwarp();
  return ok;
}

// Scores behind the last key.
__device__ __forceinline__ void mask(float* s, int valid) {
  if (valid < kCols) {
#pragma unroll
    for (int i = 0; i < kCols; ++i)
      if (i >= valid) s[i] = -INFINITY;
  }
}
// Weights 2^(scale s - ref) in the place of scores; their sum.  With one part they are rounded to bf16 here, two to a
// word in the first half of s, and the sum is that of the rounded ones: numerator and denominator then hold the same
// weights, and a value that all keys share comes out as it is.
template <int PARTS>
__device__ __forceinline__ float weights(float* s, float scale, float ref) {
  float2 sum[2] = {};
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) {
    const float2 x = __ffma2_rn(make_float2(s[2 * i], s[2 * i + 1]), make_float2(scale, scale), make_float2(-ref, -ref));
    float2 w = make_float2(exp2_approx(x.x), exp2_approx(x.y));
    if (PARTS == 1) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(w.x, w.y);
      const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
      s[i] = __uint_as_float(u);
      w = make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    } else {
      s[2 * i] = w.x;
      s[2 * i + 1] = w.y;
    }
    sum[i & 1] = __fadd2_rn(sum[i & 1], w);
  }
  return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}
// The warps of the same 32 rows meet at barrier `id`; whether `p` holds for one of their lanes.
constexpr int kRowThreads = kSoftmaxWarps / 4 * 32;
__device__ __forceinline__ void meet(int id) { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kRowThreads) : "memory"); }
__device__ __forceinline__ bool any_of(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %2, 0;\n\tbarrier.cta.red.or.pred b, %1, %3, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)p), "n"(kRowThreads)
      : "memory");
  return r != 0;
}

// A whole 32-byte sector: lanes write rows of their own, and half sectors would reach L2 one by one.
__device__ __forceinline__ void store_sector(float* p, const float* x) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]),
               "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}

// The queries of an item with few rows, a chunk of 8 coordinates a thread at
// most: fetched a segment ahead, put into shared memory when the segment
// before is through with its own.
template <int D, int PARTS>
struct NextQueries {
  static constexpr int CH = D / 8, W = PARTS == 1 ? 1 : 2;
  uint4 x[W];
  __device__ __forceinline__ static bool fits(const SharedArgs& a, const Segment& g) { return a.rows[g.e] * CH <= 32 * kSoftmaxWarps; }
  __device__ __forceinline__ void fetch(const SharedArgs& a, const Control* ctl, const Segment& g) {
    const int r = threadIdx.x / CH, gs = 31 - __clz(a.G);
    if (r >= a.rows[g.e]) return;
    const int s = g.e < a.prefixes ? ctl->member[a.member0[g.e] + (r >> gs)] : a.holder[g.e];
    const int64_t at = ((int64_t)s * a.Hkv * a.G + g.h * a.G + (r & (a.G - 1))) * D + 8 * (threadIdx.x % CH);
    const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(a.q) + at * (2 * W));
#pragma unroll
    for (int w = 0; w < W; ++w) x[w] = __ldg(src + w);
  }
  __device__ __forceinline__ void put(const SharedArgs& a, const Segment& g, char* q_smem) const {
    const int r = threadIdx.x / CH, c = threadIdx.x % CH;
    if (r >= a.rows[g.e]) return;
    char* to = q_smem + (c / 8) * Shape<D, PARTS>::kHalf + r * 128 + (((c % 8) ^ (r & 7)) << 4);
    if (PARTS == 1) {
      *reinterpret_cast<uint4*>(to) = x[0];
    } else {
      float4 u = *reinterpret_cast<const float4*>(&x[0]), v = *reinterpret_cast<const float4*>(&x[W - 1]);
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
        *reinterpret_cast<uint4*>(to + p * Shape<D, PARTS>::kStage) =
            make_uint4(split2(u.x, u.y), split2(u.z, u.w), split2(v.x, v.y), split2(v.z, v.w));
    }
  }
};

// Rows of the segment's queries into shared memory, swizzled, in PARTS parts; by
// the softmax warps.  A thread keeps its 16-byte column and goes down the
// rows.  Written for few instructions (they are fetched cold here) and with all
// loads in flight.
template <int D, int PARTS>
__device__ __forceinline__ void load_queries(const SharedArgs& a, const Control* ctl, const Segment& g, char* q_smem) {
  constexpr int CH = D / 8, STEP = 32 * kSoftmaxWarps / CH;  // chunks of 8 coordinates in a row; rows of a turn
  const int rows = a.rows[g.e], gs = 31 - __clz(a.G), c = threadIdx.x % CH;
  const bool prefix = g.e < a.prefixes;
  const unsigned char* member = ctl->member + (prefix ? a.member0[g.e] : 0);
  const int holder = a.holder[g.e], Hq = a.Hkv * a.G;
  int r = threadIdx.x / CH;
  char* to = q_smem + (c / 8) * Shape<D, PARTS>::kHalf + r * 128 + (((c % 8) ^ (r & 7)) << 4);  // STEP is a multiple of 8
  auto source = [&](int r) {
    const int s = prefix ? member[r >> gs] : holder;
    return ((int64_t)s * Hq + g.h * a.G + (r & (a.G - 1))) * D + 8 * c;
  };
  if constexpr (PARTS == 1) {
    for (; r < rows; r += STEP) {
      cp_async16(to, reinterpret_cast<const __nv_bfloat16*>(a.q) + source(r));
      to += STEP * 128;
      if (r % kTile + STEP >= kTile) to += Shape<D, PARTS>::kStage - kTile * 128;  // the next 128 rows
    }
    cp_async_wait_all();
  } else {
    // the 8 floats come into the places of the first two parts, and the thread that fetched them splits them
    for (int i = r; i < rows; i += STEP) {
      const float* src = reinterpret_cast<const float*>(a.q) + source(i);
      char* at = to + (i - r) * 128;
      cp_async16(at, src);
      cp_async16(at + Shape<D, PARTS>::kStage, src + 4);
    }
    cp_async_wait_all();
#pragma unroll 1
    for (; r < rows; r += STEP, to += STEP * 128) {
      float4 u = *reinterpret_cast<const float4*>(to), v = *reinterpret_cast<const float4*>(to + Shape<D, PARTS>::kStage);
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
        *reinterpret_cast<uint4*>(to + p * Shape<D, PARTS>::kStage) =
            make_uint4(split2(u.x, u.y), split2(u.z, u.w), split2(v.x, v.y), split2(v.z, v.w));
    }
  }
}

// Waits until every CTA of the grid has come here (the CTA's warps have: all
// that it wrote to the workspace is done).  The count runs on from call to
// call, a multiple of the CTAs between calls.  By the tiles' times above 280 GB of
// keys and values take some 60 ms, and four times that where 512 rows in fp32 go
// through them in four passes; a unit of the plan takes at most about twice as
// long in one CTA as in another, so the first waits for half of that, 0.12 s.
constexpr unsigned long long kArriveNs = 1000ull * 1000 * 1000;  // 1 s
__device__ __forceinline__ bool all_arrived(const SharedArgs& a, Control* ctl) {
  if (threadIdx.x == 0) {
    __threadfence();
    const unsigned long long ticket = atomicAdd(a.arrivals, 1ull), goal = (ticket / a.P + 1) * a.P;
    auto count = [&] {
      unsigned long long v;
      asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(a.arrivals) : "memory");
      return v;
    };
    bool ok = count() >= goal;
    const unsigned long long t0 = global_ns();
    for (uint32_t i = 1; !ok && i < kWaitPolls; ++i) {
      ok = count() >= goal;
      if ((i & 31) == 0 && global_ns() - t0 > kArriveNs) break;
    }
    if (!ok) {
      set_error(a.status, kDevTimeout, -1, -1, 59);
      ctl->abort = 1;
    }
  }
  __syncthreads();
  return ctl->abort == 0;
}

// One query row by `share` warps of a CTA: the pieces of its prefix and of its
// own tokens, 32 at a time: a lane's piece gives its reference and sum, then
// the warp adds up their outputs, several loads in flight.  Warp `part` takes
// every share-th piece; with share > 1 the CTA's warps come here together, and
// the first of each row adds up what the others leave in `left`.
// Returns whether a lane of the row has NaN.
template <int D>
__device__ __forceinline__ bool join_row(const SharedArgs& a, const Plan& plan, int item, int part, int share,
                                         float* left, int lane) {
  constexpr int V = D / 32;
  const int Hq = a.Hkv * a.G;
  const bool mine = item < a.B * Hq && a.part[item / Hq];
  if (!mine) item = 0;
  const int s = item / Hq, hq = item % Hq, h = hq / a.G;
  const int total = plan.cum[a.entries];
  int count[2] = {0, 0}, c0[2] = {0, 0}, row[2] = {0, 0}, entry[2] = {0, 0}, begin[2] = {0, 0};
#pragma unroll 1
  for (int side = 0; mine && side < 2; ++side) {
    if (side == 0 && a.prefix_entry[s] < 0) continue;
    const int e = side ? a.own_entry[s] : a.prefix_entry[s];
    const int units = entry_units(a, plan, e), b = plan.cum[e] + h * units;
    if (!units) continue;
    // the CTAs that hold its first and its last unit
    const int first = (int)(((int64_t)(b + 1) * a.P - 1) / total), last = (int)(((int64_t)(b + units) * a.P - 1) / total);
    const int r = segment_row(a, e, h, 0) + hq % a.G + (side ? 0 : a.prefix_row[s]);
    if (!side) count[0] = last - first + 1, c0[0] = first, row[0] = r, entry[0] = e, begin[0] = b;
    else count[1] = last - first + 1, c0[1] = first, row[1] = r, entry[1] = e, begin[1] = b;
  }
  float m = -INFINITY, l = 0.f, o[V] = {};
  const int pieces = count[0] + count[1];
#pragma unroll 1
  for (int x0 = part; x0 < pieces; x0 += 32 * share) {
    const int x = x0 + lane * share, side = x >= count[0];
    const int c = (side ? c0[1] - count[0] : c0[0]) + x;
    const int at = (side ? row[1] : row[0]) + 256 * c;
    // a CTA in which no tile begins holds no piece
    const int b = side ? begin[1] : begin[0], e = side ? entry[1] : entry[0], units = entry_units(a, plan, e);
    const Tiles t = tiles_between(a, e, max(cta_unit(c, a.P, total) - b, 0), min(cta_unit(c + 1, a.P, total) - b, units));
    const bool some = x < pieces && t.from < t.to;
    float2 w = some ? __ldcg(a.ml + at) : make_float2(-INFINITY, 0.f);
    // the largest weight is 1; without it (a first tile of scores of -infinity has no reference) nothing here counts
    if (some && !(w.y >= 0.5f)) w.y = NAN;
    const float top = fmaxf(m, warp_max(w.x));
    const float f0 = m == top ? 1.f : exp2_approx(m - top), f = !some ? 0.f : w.x == top ? 1.f : exp2_approx(w.x - top);
    l = l * f0 + warp_sum(w.y * f);
    m = top;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] *= f0;
    const unsigned have = __ballot_sync(0xffffffffu, some);
    const int n = min(32, (pieces - x0 + share - 1) / share);
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const float fj = __shfl_sync(0xffffffffu, f, j);
      const float* src = a.acc + (int64_t)__shfl_sync(0xffffffffu, at, j) * D + lane * V;
      float y[V] = {};
      if (have >> j & 1) {
        if (V == 4) {
          const float4 t = __ldcg(reinterpret_cast<const float4*>(src));
          y[0] = t.x; y[1] = t.y; y[V - 2] = t.z; y[V - 1] = t.w;
        } else {
          const float2 t = __ldcg(reinterpret_cast<const float2*>(src));
          y[0] = t.x; y[1] = t.y;
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = fmaf(y[i], fj, o[i]);
    }
  }
  if (share > 1) {  // [warp][D + 2]
    float* own = left + (threadIdx.x >> 5) * (D + 2);
#pragma unroll
    for (int i = 0; i < V; ++i) own[lane * V + i] = o[i];
    if (lane == 0) {
      own[D] = m;
      own[D + 1] = l;
    }
    __syncthreads();
    for (int w = 1; w < share && part == 0; ++w) {
      const float* x = own + w * (D + 2);
      const float top = fmaxf(m, x[D]);
      const float f0 = m == top ? 1.f : exp2_approx(m - top), f = x[D] == top ? 1.f : exp2_approx(x[D] - top);
      l = l * f0 + x[D + 1] * f;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = o[i] * f0 + x[lane * V + i] * f;
      m = top;
    }
    __syncthreads();
  }
  if (!mine || part) return false;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    o[i] = l > 0.f ? o[i] / l : l == 0.f ? 0.f : l;  // without a token: zero; NaN stays
    odd |= isnan(o[i]);
  }
  const int64_t at = (int64_t)item * D + lane * V;
  if (a.q_bf16) {
#pragma unroll
    for (int i = 0; i < V; i += 2)
      *reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<__nv_bfloat16*>(a.out) + at + i) = __floats2bfloat162_rn(o[i], o[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2)
      *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.out) + at + i) = make_float2(o[i], o[i + 1]);
  }
  return odd;
}

// A warp's rows that came out with NaN, once more, straight from the definition:
// the largest score, then weights and sums in fp32, a key at a time.  Infinities
// among the tokens bring them here: a value in parts has parts of either sign and
// of zero, which an infinite factor turns into NaN where the whole value gives an
// infinity or, as a score of -infinity, no weight at all.  Finite scores come here
// only past 2^23, where the rounding of a reference passes a power of two.  Bound
// by the loads' latency: four rows behind 128K keys take 12 ms a pass, 2048 rows
// 68 ms for both.
template <int D>
__device__ __noinline__ void plain_rows(const SharedArgs& a, const Plan& plan, int row, int step, int lane) {
  constexpr int V = D / 32, U = 8;  // coordinates of a lane; keys at a time
  struct alignas(2 * V) Coords {
    __nv_bfloat16 c[V];
  };
  const int Hq = a.Hkv * a.G;
  const float scale = 1.4426950408889634f / sqrtf((float)D);
  auto get = [&](const void* x, int64_t i) {
    return a.q_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(x)[i]) : reinterpret_cast<const float*>(x)[i];
  };
#pragma unroll 1
  for (; row < a.B * Hq; row += step) {
    const int s = row / Hq, h = row % Hq / a.G;
    const int64_t at = (int64_t)row * D + lane * V;
    if (!a.part[s]) continue;
    bool odd = false;
    float q[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      odd |= isnan(get(a.out, at + i));  // as this lane has left it
      q[i] = get(a.q, at + i);
    }
    if (!__any_sync(0xffffffffu, odd)) continue;
    float m = -INFINITY, l = 0.f, o[V] = {};
    bool lost = false;  // a score of NaN or infinity: the sum is no number
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass)
#pragma unroll 1
      for (int side = 0; side < 2; ++side) {
        if (!side && a.prefix_entry[s] < 0) continue;
        const int e = side ? a.own_entry[s] : a.prefix_entry[s], keys = item_keys(a, plan, e);
        const int64_t first = ((int64_t)a.token0[e] + (int64_t)h * a.cap[e]) * D + lane * V;
#pragma unroll 1
        for (int j0 = 0; j0 < keys && !lost; j0 += kTile) {
          float lt = 0.f, ot[V] = {};  // of a tile, so that long sums keep their bits
#pragma unroll 1
          for (int j = j0; j < min(j0 + kTile, keys); j += U) {
            Coords x[U];
#pragma unroll
            for (int u = 0; u < U; ++u)  // keys behind the last repeat it
              x[u] = *reinterpret_cast<const Coords*>(a.k + first + (int64_t)min(j + u, keys - 1) * D);
            float z[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              z[u] = 0.f;
#pragma unroll
              for (int i = 0; i < V; ++i) z[u] += q[i] * __bfloat162float(x[u].c[i]);
              z[u] = warp_sum(z[u]) * scale;
              m = pass ? m : fmaxf(m, z[u]);
              lost |= !(z[u] < INFINITY);
            }
            if (lost || !pass) continue;
#pragma unroll
            for (int u = 0; u < U; ++u)
              x[u] = *reinterpret_cast<const Coords*>(a.v + first + (int64_t)min(j + u, keys - 1) * D);
#pragma unroll
            for (int u = 0; u < U; ++u) {
              if (j + u >= keys) break;
              float w = exp2f(z[u] - m);
              if (w == 0.f && z[u] > -INFINITY) w = 1.4e-45f;  // as good as nothing, but an infinite value counts
              lt += w;
#pragma unroll
              for (int i = 0; i < V; ++i) ot[i] += w * __bfloat162float(x[u].c[i]);
            }
          }
          l += lt;
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] += ot[i];
        }
      }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float y = lost ? NAN : o[i] / l;
      if (a.q_bf16) reinterpret_cast<__nv_bfloat16*>(a.out)[at + i] = __float2bfloat16(y);
      else reinterpret_cast<float*>(a.out)[at + i] = y;
    }
  }
}

template <int D, int PARTS>
__global__ void __launch_bounds__(kThreads, 1) shared_attend_kernel(const __grid_constant__ SharedArgs a) {
  using S = Shape<D, PARTS>;
  constexpr int STAGES = stages<D, PARTS>();
  extern __shared__ __align__(1024) char smem[];
  char* q_smem = smem;
  char* ring = smem + S::kQ;
  Control* ctl = reinterpret_cast<Control*>(ring + STAGES * S::kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((smem_u32(smem) & 1023u) != 0u) {  // the swizzle counts on it
    if (threadIdx.x == 0) set_error(a.status, kDevInternal, -1, -1, 50);
    return;
  }

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl->tmem)),
                 "r"(S::kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == 1) {
    build_plan(a, ctl->plan, lane);
  } else if (warp == 2 && lane == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    mbar_init(&ctl->q_full, kSoftmaxWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], kSoftmaxWarps);
      mbar_init(&ctl->o_full[i], 1);
    }
    ctl->abort = 0;
    fence_mbar_init();
  } else if (warp == 3) {
    ctl->member[lane] = a.member[lane];
    ctl->member[lane + 32] = a.member[lane + 32];
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = ctl->tmem;
  const int c = blockIdx.x;
  Walk walk(a, ctl->plan, c);
  Segment g;

  if (warp >= kSoftmaxWarps) {
    fewer_registers<64>();  // 128 x 64 + 512 x 104: the 640 x 96 of the launch
    if (warp == kSoftmaxWarps) {
      // ---- copies: K and V of every tile in turn, 16-token boxes where the item ends inside the tile
      if (lane == 0) {
        int slot = 0, phase = 0;
        while (walk.next(a, ctl->plan, g)) {
          const int tok = a.token0[g.e] + g.h * a.cap[g.e];
          for (int t = g.tile0; t < g.tile1; ++t) {
            const int valid = g.valid(t), y = tok + t * kTile;
            for (int kv = 0; kv < 2; ++kv) {
              if (wait(ctl, &ctl->empty[slot], phase ^ 1, a.status, 51)) {
                char* dst = ring + slot * S::kStage;
                if (valid == kTile) {
                  mbar_arrive_expect_tx(&ctl->full[slot], S::kStage);
#pragma unroll
                  for (int x = 0; x < D / 64; ++x)
                    tma_box(dst + x * S::kHalf, kv ? a.v128 : a.k128, 64 * x, y, &ctl->full[slot]);
                } else {
                  const int nb = (valid + kBlock - 1) / kBlock;
                  mbar_arrive_expect_tx(&ctl->full[slot], nb * kBlock * D * 2);
                  for (int b = 0; b < nb; ++b)
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                      tma_box(dst + x * S::kHalf + b * kBlock * 128, kv ? a.v16 : a.k16, 64 * x, y + b * kBlock,
                              &ctl->full[slot]);
                }
              }
              if (++slot == STAGES) {
                slot = 0;
                phase ^= 1;
              }
            }
          }
        }
      }
    } else if (warp == kSoftmaxWarps + 1) {
      // ---- S = Q K^T of every step, into the buffer whose weights the step before last has used up
      const uint32_t q_addr = smem_u32(q_smem), ring_addr = smem_u32(ring), lead = elect_leader();
      int n = 0, segs = 0;      // steps and segments before this one
      int slot = 0, phase = 0;  // of the tile in the ring
      while (walk.next(a, ctl->plan, g)) {
        const int subs = (a.rows[g.e] + kTile - 1) / kTile;
        warp_wait(ctl, &ctl->q_full, segs & 1, a.status, 54);
        ++segs;
        for (int t = g.tile0; t < g.tile1; ++t) {
          bool ok = warp_wait(ctl, &ctl->full[slot], phase, a.status, 55);
          const uint64_t kd = operand(uniform(ring_addr + slot * S::kStage), 16, 1024);
          for (int sub = 0; sub < subs; ++sub, ++n) {
            const uint64_t qd = operand(uniform(q_addr + sub * (PARTS * S::kStage)), 16, 1024);
            const uint32_t d = uniform(tmem + (n & 1) * S::kBuffer);
            if (n >= 2) ok &= warp_wait(ctl, &ctl->o_full[n & 1], ((n >> 1) - 1) & 1, a.status, 53);
            fence_after();
            if (ok) {
#pragma unroll
              for (int part = PARTS - 1; part >= 0; --part)
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                  const uint32_t off = (i / 4) * S::kHalf + (i % 4) * 32;
                  mma_ss(d, qd + (part * S::kStage + off) / 16, kd + off / 16, instruction(kTile, false),
                         part < PARTS - 1 || i > 0, lead);
                }
              mma_commit(&ctl->s_full[n & 1], lead);
              if (sub == subs - 1) mma_commit(&ctl->empty[slot], lead);
            }
          }
          slot += 2;
          if (slot >= STAGES) {
            slot -= STAGES;
            phase ^= 1;
          }
        }
      }
    } else if (warp == kSoftmaxWarps + 2) {
      // ---- O += P V of every step; a warp of its own, so that waiting for weights holds up no scores
      const uint32_t ring_addr = smem_u32(ring), lead = elect_leader();
      int n = 0, slot = 1, phase = 0;
      while (walk.next(a, ctl->plan, g)) {
        const int subs = (a.rows[g.e] + kTile - 1) / kTile;
        for (int t = g.tile0; t < g.tile1; ++t) {
          bool ok = warp_wait(ctl, &ctl->full[slot], phase, a.status, 52);
          const int valid = g.valid(t);
          if (valid % kBlock) {  // weights behind the last key are zero, but 0 x NaN is not
            const int upto = (valid + kBlock - 1) / kBlock * kBlock;
            for (int i = lane; i < (upto - valid) * (D / 8); i += 32) {
              const int r = valid + i / (D / 8), ch = i % (D / 8);
              *reinterpret_cast<uint4*>(ring + slot * S::kStage + (ch / 8) * S::kHalf + r * 128 + (ch % 8) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            __syncwarp();
          }
          const uint64_t vd = operand(uniform(ring_addr + slot * S::kStage), S::kHalf, 1024);
          for (int sub = 0; sub < subs; ++sub, ++n) {
            const uint32_t p = uniform(tmem + (n & 1) * S::kBuffer), o = uniform(tmem + S::kO + sub * D);
            const bool add = !(t == g.tile0 || S::kTileO);
            ok &= warp_wait(ctl, &ctl->p_full[n & 1], (n >> 1) & 1, a.status, 53);
            fence_after();
            if (ok) {
              if (valid == kTile) {
#pragma unroll
                for (int part = PARTS - 1; part >= 0; --part)
#pragma unroll
                  for (int k = 0; k < kTile / 16; ++k)
                    mma_ts(o, p + part * 64 + k * 8, vd + k * (16 * 128 / 16), instruction(D, true),
                           part < PARTS - 1 || k > 0 || add, lead);
              } else {
                for (int part = PARTS - 1; part >= 0; --part)
                  for (int k = 0; k < (valid + 15) / 16; ++k)
                    mma_ts(o, p + part * 64 + k * 8, vd + k * (16 * 128 / 16), instruction(D, true),
                           part < PARTS - 1 || k > 0 || add, lead);
              }
              mma_commit(&ctl->o_full[n & 1], lead);
              if (sub == subs - 1) mma_commit(&ctl->empty[slot], lead);
            }
          }
          slot += 2;
          if (slot >= STAGES) {
            slot -= STAGES;
            phase ^= 1;
          }
        }
      }
    }
  } else {
    more_registers<104>();
    // ---- softmax: thread = row (its TMEM lane) and a quarter of the keys, and of O's coordinates
    constexpr int OC = D * kCols / kTile;
    const int quarter = warp >> 2, row = (warp & 3) * 32 + lane, bar = 1 + (warp & 3);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const float scale = 1.4426950408889634f / sqrtf((float)D);  // logits in powers of two
    int n = 0;
    bool more = walk.next(a, ctl->plan, g);
    if (more) {
      load_queries<D, PARTS>(a, ctl, g, q_smem);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_full);
    }
    while (more) {
      const Segment cur = g;
      more = walk.next(a, ctl->plan, g);
      NextQueries<D, PARTS> ahead;
      const bool few = more && ahead.fits(a, g);
      if (few) ahead.fetch(a, ctl, g);
      const int rows = a.rows[cur.e], subs = (rows + kTile - 1) / kTile;
      float m2[2] = {-INFINITY, -INFINITY}, l2[2] = {0.f, 0.f};  // per 128 rows: reference of the weights, their sum here
      float acc[S::kTileO ? OC : 1] = {};                        // kTileO: O so far, in units of the reference
      for (int t = cur.tile0; t < cur.tile1; ++t) {
        for (int sub = 0; sub < subs; ++sub, ++n) {
          warp_wait(ctl, &ctl->s_full[n & 1], (n >> 1) & 1, a.status, 56);
          fence_after();
          if (sub * kTile + (warp & 3) * 32 < rows) {  // the same for all warps of these rows
            const uint32_t buf = tmem + lanes + (n & 1) * S::kBuffer;
            const uint32_t o_at = tmem + lanes + S::kO + sub * D + quarter * OC;
            float s[kCols];
            tmem_ld32(buf + quarter * kCols, s);
            const int valid = cur.valid(t) - quarter * kCols;  // keys of this quarter
            mask(s, valid);
            float m = sub ? m2[1] : m2[0], l = sub ? l2[1] : l2[0], f = 1.f;
            float sum;
            bool raise = t == cur.tile0;
            if (!raise) {
              sum = weights<PARTS>(s, scale, m);
              // all have read S when they have passed, and P may take its place
              fence_before();
              raise = any_of(bar, sub * kTile + row < rows && !(sum < kMostWeight));
              fence_after();
              if (raise) {
                tmem_ld32(buf + quarter * kCols, s);
                mask(s, valid);
              }
            }
            if (raise) {
              float top = s[0];
#pragma unroll
              for (int i = 1; i < kCols; ++i) top = fmaxf(top, s[i]);
              ctl->row_max[quarter][row] = top * scale;
              fence_before();
              meet(bar);
              fence_after();
              top = m;
#pragma unroll
              for (int i = 0; i < kTile / kCols; ++i) top = fmaxf(top, ctl->row_max[i][row]);
              if (top == -INFINITY) top = 0.f;
              f = exp2_approx(m - top);  // 0 in the first tile: m = -inf
              m = top;
              l = t == cur.tile0 ? 0.f : l * f;
              sum = weights<PARTS>(s, scale, m);
              if (!S::kTileO && t > cur.tile0) {
                // O of the tile before is complete (with two steps a tile: S was issued behind its product),
                // and the next product into it waits for p_full
                if (subs == 1) warp_wait(ctl, &ctl->o_full[(n - 1) & 1], ((n - 1) >> 1) & 1, a.status, 57);
                fence_after();
#pragma unroll
                for (int x = 0; x < OC / 16; ++x) {
                  float o[16];
                  tmem_ld16(o_at + 16 * x, o);
#pragma unroll
                  for (int i = 0; i < 16; ++i) o[i] *= f;
                  tmem_st16(o_at + 16 * x, reinterpret_cast<const uint32_t*>(o));
                }
              }
              meet(bar);  // the maxima have been read
            }
            l += sum;
            if (sub) {
              m2[1] = m;
              l2[1] = l;
            } else {
              m2[0] = m;
              l2[0] = l;
            }
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
              uint32_t w[kCols / 2];
#pragma unroll
              for (int i = 0; i < kCols / 2; ++i) w[i] = PARTS == 1 ? __float_as_uint(s[i]) : split2(s[2 * i], s[2 * i + 1]);
              tmem_st16(buf + part * 64 + quarter * (kCols / 2), w);
            }
            if (S::kTileO && t > cur.tile0) {
              // O of the tile before, in the reference of its weights; the next product waits for p_full
              warp_wait(ctl, &ctl->o_full[(n - 1) & 1], ((n - 1) >> 1) & 1, a.status, 57);
              fence_after();
#pragma unroll
              for (int x = 0; x < OC / 16; ++x) {
                float o[16];
                tmem_ld16(o_at + 16 * x, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[(16 * x + i) % (S::kTileO ? OC : 1)] += o[i];
              }
              if (raise) {
#pragma unroll
                for (int i = 0; i < OC; ++i) acc[i % (S::kTileO ? OC : 1)] *= f;
              }
            }
            wait_st();
            fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->p_full[n & 1]);
        }
      }
      // every S of this segment has been computed: the next one's queries may overwrite these
      if (more) {
        if (few) ahead.put(a, g, q_smem);
        else load_queries<D, PARTS>(a, ctl, g, q_smem);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->q_full);
      }
      warp_wait(ctl, &ctl->o_full[(n - 1) & 1], ((n - 1) >> 1) & 1, a.status, 58);
      fence_after();
      for (int sub = 0; sub < subs; ++sub) {
        const int r = sub * kTile + row;
        if (sub * kTile + (warp & 3) * 32 >= rows) break;
        float l = sub ? l2[1] : l2[0];
        ctl->row_max[quarter][row] = l;
        meet(bar);
        if (!quarter) {
#pragma unroll
          for (int i = 1; i < kTile / kCols; ++i) l += ctl->row_max[i][row];
        }
        const int64_t at = segment_row(a, cur.e, cur.h, c) + r;
        float* dst = a.acc + at * D + quarter * OC;
#pragma unroll
        for (int x = 0; x < OC / 16; ++x) {
          float o[16];
          tmem_ld16(tmem + lanes + S::kO + sub * D + quarter * OC + 16 * x, o);
          if (S::kTileO) {
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] += acc[(16 * x + i) % (S::kTileO ? OC : 1)];
          }
          if (r < rows) {
            store_sector(dst + 16 * x, o);
            store_sector(dst + 16 * x + 8, o + 8);
          }
        }
        if (!quarter && r < rows) a.ml[at] = make_float2(sub ? m2[1] : m2[0], l);
        meet(bar);  // the sums have been read
      }
      fence_before();
    }
  }
  __syncwarp();
  if (ctl->abort) {  // copies and products in flight get a bounded time to end
    const unsigned long long t0 = global_ns();
    for (uint32_t i = 0; i < kWaitPolls && global_ns() - t0 < kWaitNs; ++i) __nanosleep(1000);
  }
  fence_before();
  __syncthreads();
  fence_after();
  // what follows is for all warps alike: each has the launch's registers again (the warps of a group must have met
  // since their last change, and the softmax warps give back what the others wait for)
  if (warp >= kSoftmaxWarps) more_registers<96>();
  else fewer_registers<96>();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kColumns) : "memory");
  if (!all_arrived(a, ctl)) return;
  // rows are dealt to the CTAs; few rows leave several warps for each
  constexpr int kWarps = kThreads / 32;
  const int rows = a.B * a.Hkv * a.G, share = rows <= a.P ? kWarps : rows * 4 <= a.P * kWarps ? 4 : 1;
  static_assert(kWarps % 4 == 0, "warps of a row");
  const int step = a.P * (kWarps / share);
  bool odd = false;
  for (int r0 = blockIdx.x * (kWarps / share); r0 < rows; r0 += step)
    odd |= join_row<D>(a, ctl->plan, r0 + warp / share, warp % share, share, reinterpret_cast<float*>(ring), lane);
  if (__any_sync(0xffffffffu, odd)) plain_rows<D>(a, ctl->plan, blockIdx.x * (kWarps / share) + warp / share, step, lane);
}

template <int D, int PARTS>
cudaError_t launch(const SharedArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = a.P;
  cfg.blockDim = kThreads;
  cfg.dynamicSmemBytes = smem_bytes<D, PARTS>();
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeCooperative;  // its CTAs wait for one another
  at[0].val.cooperative = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shared_attend_kernel<D, PARTS>, a);
}

}  // namespace

cudaError_t prepare_shared(int d) {
  cudaError_t e;
  if (d == 128) {
    e = raise_smem_limit((const void*)shared_attend_kernel<128, 1>, (int)smem_bytes<128, 1>());
    if (e == cudaSuccess) e = raise_smem_limit((const void*)shared_attend_kernel<128, 3>, (int)smem_bytes<128, 3>());
  } else {
    e = raise_smem_limit((const void*)shared_attend_kernel<64, 1>, (int)smem_bytes<64, 1>());
    if (e == cudaSuccess) e = raise_smem_limit((const void*)shared_attend_kernel<64, 3>, (int)smem_bytes<64, 3>());
  }
  return e;
}

cudaError_t launch_attend_shared(const SharedArgs& a, cudaStream_t st) {
  if (a.d == 128) return a.q_bf16 ? launch<128, 1>(a, st) : launch<128, 3>(a, st);
  return a.q_bf16 ? launch<64, 1>(a, st) : launch<64, 3>(a, st);
}

}  // namespace compkv
