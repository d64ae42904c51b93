// Exact attention of every sequence over a prefix that one sequence of the
// cache holds for all and over its own tokens, under one softmax:
//   out = sum_j e^(z_j) v_j / sum_j e^(z_j),   z_j = q . k_j / sqrt(d),
// j over the prefix's tokens and the sequence's own.
//
// A prefix is read once for up to 128 query rows (sequences x query heads of a
// KV head); a sequence's own tokens are one more item with G rows.  Items are
// walked in tiles of 128 keys.  One persistent CTA per multiprocessor takes an
// equal run of the tiles of all items, so that a long prefix and few rows
// still fill the chip; each piece of an item leaves its rows' maximum, sum and
// unnormalised output, and a second kernel joins the pieces.
//
// Within a CTA (tcgen05, one tile in flight behind the other):
//   warp 8   copies K and V tiles by tensor maps into a ring of stages,
//   warp 9   issues S = Q K^T into one of two TMEM buffers and O += P V,
//   warps 0-7 load Q, take the running maximum and sum (thread = row and half
//            of the keys), and write the weights P over S in TMEM.
// O stays in TMEM and is scaled only when a row's maximum rose by more than 8
// (in powers of two): the weights then stay below 2^8, and what the final
// division by their sum loses by that is nothing.
//
// fp32 queries and weights are split into three bf16 parts of 8 bits each and
// multiplied part by part (K and V are bf16 as they are), so the products hold
// 24 bits; bf16 queries take one product, and their weights are rounded to
// bf16, 2^-9 of each on average, as the result is.
#include "compkv_launch.h"

namespace compkv {

namespace {

constexpr int kTile = 128;                // keys of a tile, and query rows of an item at most
constexpr int kSoftmaxWarps = 8;
constexpr int kThreads = 32 * (kSoftmaxWarps + 2);
constexpr int kItemUnits = 1;             // what starting an item costs, in tiles
constexpr float kRescale = 8.f;           // log2 of the factor that a maximum may rise by before O is scaled
constexpr size_t kSmemLimit = 232448;

// ---------------------------------------------------------------- the plan
// Entry e has tiles + kItemUnits units per head (0 without tokens); CTA c of P
// takes the units [c T / P, (c + 1) T / P) of the T units of all entries and
// heads, in order.
struct Plan {
  int cum[kMaxSharedEntries + 1];         // units of all heads of the entries before e
  unsigned char last[kMaxSharedEntries];  // keys of its last tile
};

__device__ __forceinline__ int held_tokens(const SharedArgs& a, int s) {
  return max(0, min(__ldcg(a.seq_len + s), a.cap_blocks[s] * kBlock));
}
__device__ __forceinline__ int entry_units(const SharedArgs& a, const Plan& p, int e) {  // per head
  return (p.cum[e + 1] - p.cum[e]) / a.Hkv;
}
// First token of an entry in its sequence: a holder's own tokens begin behind its prefix.
__device__ __forceinline__ int entry_first(const SharedArgs& a, int e, int held) {
  const int s = a.holder[e];
  return e >= a.prefixes && a.prefix_seq[s] == s ? min(a.prefix_len[s], held) : 0;
}

// By one warp; the caller synchronises.
__device__ void build_plan(const SharedArgs& a, Plan& p, int lane) {
  int base = 0;
  for (int e0 = 0; e0 < a.entries; e0 += 32) {
    const int e = e0 + lane;
    int u = 0;
    if (e < a.entries) {
      const int s = a.holder[e], held = held_tokens(a, s);
      const int len = e < a.prefixes ? min(held, a.prefix_len[s]) : held - entry_first(a, e, held);
      if (e < a.prefixes && held < a.prefix_len[s]) set_error(a.status, kDevInvalidArg, s, -1, 5);
      p.last[e] = (unsigned char)((len + kTile - 1) % kTile + 1);
      u = len ? ((len + kTile - 1) / kTile + kItemUnits) * a.Hkv : 0;
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
      u += n;
      g.tile0 = max(x - kItemUnits, 0);
      g.tile1 = x + n - kItemUnits;
      g.tiles = per - kItemUnits;
      g.last = p.last[e];
      if (g.tile1 > g.tile0) return true;
    }
    return false;
  }
};
// Workspace row of the first row of a segment of CTA c: segments follow one another by item or by CTA,
// and each step adds at least the rows of the segment before it.
__device__ __forceinline__ int64_t segment_row(const SharedArgs& a, int e, int h, int c) {
  return a.row0[e] + h * a.rows[e] + (int64_t)kTile * c;
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
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
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
__device__ __forceinline__ void tmem_ld64(uint32_t addr, float* f) {
  uint32_t* r = reinterpret_cast<uint32_t*>(f);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%2"
      "6,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%5"
      "0,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63"
      "}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]),
        "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]),
        "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
        "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
        "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
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
  a -= __uint_as_float(u << 16);
  b -= __uint_as_float(u & 0xffff0000u);
  return u;
}

// ---------------------------------------------------------------- the CTA
template <int D, int PARTS>
struct Shape {
  static constexpr int kHalf = kTile * 128;             // 64 coordinates of 128 rows, 128 bytes a row
  static constexpr int kStage = kHalf * (D / 64);       // a K or a V tile
  static constexpr int kQ = kStage * PARTS;
  // TMEM columns: two buffers of 128 scores and, over and behind them, up to three parts of weights; O
  static constexpr int kBuffer = PARTS == 3 ? 192 : 128;
  static constexpr int kO = 2 * kBuffer;
  static constexpr int kColumns = 512;
};
struct Control {
  Plan plan;
  float row_max[2][2][kTile];  // [tile & 1][half of the keys][row]; sums at the end of a segment
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

// Rows of the segment's queries into shared memory, swizzled, in PARTS parts; by the softmax warps.
template <int D, int PARTS>
__device__ __forceinline__ void load_queries(const SharedArgs& a, const Segment& g, char* q_smem) {
  constexpr int CH = D / 8;  // 16-byte chunks of 8 coordinates
  const int rows = a.rows[g.e];
  for (int i = threadIdx.x; i < rows * CH; i += 32 * kSoftmaxWarps) {
    const int r = i / CH, c = i % CH;
    const int s = g.e < a.prefixes ? a.member[a.member0[g.e] + r / a.G] : a.holder[g.e];
    const int64_t at = (((int64_t)s * a.Hkv + g.h) * a.G + r % a.G) * D + 8 * c;
    const int to = (c / 8) * Shape<D, PARTS>::kHalf + r * 128 + (((c % 8) ^ (r & 7)) << 4);
    if (PARTS == 1) {
      *reinterpret_cast<uint4*>(q_smem + to) = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.q) + at));
    } else {
      const float4* src = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.q) + at);
      const float4 u = __ldg(src), v = __ldg(src + 1);
      float x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
      for (int p = 0; p < PARTS; ++p) {
        uint4 w;
        w.x = split2(x[0], x[1]);
        w.y = split2(x[2], x[3]);
        w.z = split2(x[4], x[5]);
        w.w = split2(x[6], x[7]);
        *reinterpret_cast<uint4*>(q_smem + p * Shape<D, PARTS>::kStage + to) = w;
      }
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
  }
  fence_before();
  __syncthreads();
  fence_after();
  pdl_trigger();
  const uint32_t tmem = ctl->tmem;
  const int c = blockIdx.x;
  Walk walk(a, ctl->plan, c);
  Segment g;

  if (warp == kSoftmaxWarps) {
    // ---- copies: K and V of every tile in turn, 16-token boxes where the item ends inside the tile
    if (lane == 0) {
      int slot = 0, phase = 0;
      while (walk.next(a, ctl->plan, g)) {
        const int s = a.holder[g.e];
        const int64_t tok = (a.layer_row0 + a.seq_row0[s] + (int64_t)g.h * a.cap_blocks[s]) * kBlock +
                            entry_first(a, g.e, held_tokens(a, s));
        for (int t = g.tile0; t < g.tile1; ++t) {
          const int valid = g.valid(t), y = (int)(tok + (int64_t)t * kTile);
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
    // ---- products: S of tile n + 1 is issued ahead of O += P V of tile n
    const uint32_t q_addr = smem_u32(q_smem), ring_addr = smem_u32(ring);
    int n = 0, segs = 0;       // tiles and segments before this one
    int slot = 0, phase = 0;   // of the next K tile in the ring
    int v_slot = 0, v_phase = 0, v_valid = 0;
    bool pending = false, first = false;  // a tile whose P V is still to come, and whether O starts with it
    auto issue_pv = [&] {
      // tile n - 1
      warp_wait(ctl, &ctl->full[v_slot], v_phase, a.status, 52);
      const uint32_t v = ring_addr + v_slot * S::kStage;
      if (v_valid % kBlock) {  // weights behind the last key are zero, but 0 x NaN is not
        const int upto = (v_valid + kBlock - 1) / kBlock * kBlock;
        for (int i = lane; i < (upto - v_valid) * (D / 8); i += 32) {
          const int r = v_valid + i / (D / 8), ch = i % (D / 8);
          *reinterpret_cast<uint4*>(ring + v_slot * S::kStage + (ch / 8) * S::kHalf + r * 128 + (ch % 8) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
        __syncwarp();
      }
      const bool ok = warp_wait(ctl, &ctl->p_full[(n - 1) & 1], ((n - 1) >> 1) & 1, a.status, 53);
      fence_after();
      if (lane == 0 && ok) {
        const uint32_t p = tmem + ((n - 1) & 1) * S::kBuffer;
        const int steps = (v_valid + 15) / 16;
        for (int part = 0; part < PARTS; ++part)
          for (int k = 0; k < steps; ++k)
            mma_ts(tmem + S::kO, p + part * 64 + k * 8, operand(v + k * 16 * 128, S::kHalf, 1024),
                   instruction(D, true), !(first && part == 0 && k == 0));
        mma_commit(&ctl->empty[v_slot]);
        mma_commit(&ctl->o_full[(n - 1) & 1]);
      }
      pending = false;
    };
    while (walk.next(a, ctl->plan, g)) {
      for (int t = g.tile0; t < g.tile1; ++t) {
        if (t == g.tile0) {
          if (pending) issue_pv();
          warp_wait(ctl, &ctl->q_full, segs & 1, a.status, 54);
          ++segs;
        }
        const bool ok = warp_wait(ctl, &ctl->full[slot], phase, a.status, 55);
        fence_after();
        if (lane == 0 && ok) {
          const uint32_t k = ring_addr + slot * S::kStage;
#pragma unroll
          for (int part = 0; part < PARTS; ++part)
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const uint32_t off = (i / 4) * S::kHalf + (i % 4) * 32;
              mma_ss(tmem + (n & 1) * S::kBuffer, operand(q_addr + part * S::kStage + off, 16, 1024),
                     operand(k + off, 16, 1024), instruction(kTile, false), part + i > 0);
            }
          mma_commit(&ctl->empty[slot]);
          mma_commit(&ctl->s_full[n & 1]);
        }
        if (pending) issue_pv();
        if (++slot == STAGES) {
          slot = 0;
          phase ^= 1;
        }
        v_slot = slot;
        v_phase = phase;
        v_valid = g.valid(t);
        first = t == g.tile0;
        pending = true;
        if (++slot == STAGES) {
          slot = 0;
          phase ^= 1;
        }
        ++n;
      }
    }
    if (pending) issue_pv();
  } else {
    // ---- softmax: thread = row (its TMEM lane) and half of the keys
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const float scale = 1.4426950408889634f / sqrtf((float)D);  // logits in powers of two
    int n = 0;
    bool more = walk.next(a, ctl->plan, g);
    if (more) {
      load_queries<D, PARTS>(a, g, q_smem);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_full);
    }
    while (more) {
      const Segment cur = g;
      const int rows = a.rows[cur.e];
      const bool live = (warp & 3) * 32 < rows;  // the same for both warps of these rows
      float m = -INFINITY, l = 0.f;              // maximum that the weights refer to, and their sum over this half
      for (int t = cur.tile0; t < cur.tile1; ++t, ++n) {
        warp_wait(ctl, &ctl->s_full[n & 1], (n >> 1) & 1, a.status, 56);
        fence_after();
        if (live) {
          const uint32_t buf = tmem + lanes + (n & 1) * S::kBuffer;
          float s[64];
          tmem_ld64(buf + half * 64, s);
          const int valid = cur.valid(t) - half * 64;  // keys of this half
          if (valid < 64) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i >= valid) s[i] = -INFINITY;
          }
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int i = 4; i < 64; ++i) mx[i & 3] = fmaxf(mx[i & 3], s[i]);
          const float mine = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
          ctl->row_max[n & 1][half][row] = mine;
          fence_before();
          asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory");  // both halves have read S, too
          fence_after();
          const float top = fmaxf(mine, ctl->row_max[n & 1][half ^ 1][row]);
          const bool raise = row < rows && top > m + kRescale;  // holds for a segment's first tile: m = -inf
          if (__any_sync(0xffffffffu, raise)) {
            const float next = raise ? top : m;
            if (t > cur.tile0) {
              // O of the tiles before is complete, and the next product waits for p_full
              warp_wait(ctl, &ctl->o_full[(n - 1) & 1], ((n - 1) >> 1) & 1, a.status, 57);
              fence_after();
              const float f = m == next ? 1.f : exp2_approx(m - next);
#pragma unroll
              for (int x = 0; x < D / 64; ++x) {
                float o[32];
                tmem_ld32(tmem + lanes + S::kO + half * (D / 2) + 32 * x, o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= f;
                tmem_st32(tmem + lanes + S::kO + half * (D / 2) + 32 * x, reinterpret_cast<const uint32_t*>(o));
              }
              l *= f;
            }
            m = next;
          }
          const float ref = m == -INFINITY ? 0.f : m;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            s[i] = exp2_approx(fmaf(s[i], scale, -ref));
            sum[i & 3] += s[i];
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
          for (int part = 0; part < PARTS; ++part) {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = split2(s[2 * i], s[2 * i + 1]);
            tmem_st32(buf + part * 64 + half * 32, w);
          }
          wait_st();
          fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->p_full[n & 1]);
      }
      // every S of this segment has been computed: the next one's queries may overwrite these
      more = walk.next(a, ctl->plan, g);
      if (more) {
        load_queries<D, PARTS>(a, g, q_smem);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->q_full);
      }
      warp_wait(ctl, &ctl->o_full[(n - 1) & 1], ((n - 1) >> 1) & 1, a.status, 58);
      fence_after();
      if (live) {
        if (half) ctl->row_max[n & 1][0][row] = l;
        asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory");
        if (!half) l += ctl->row_max[n & 1][0][row];
        const int64_t at = segment_row(a, cur.e, cur.h, c) + row;
        float* dst = a.acc + at * D + half * (D / 2);
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          float o[32];
          tmem_ld32(tmem + lanes + S::kO + half * (D / 2) + 32 * x, o);
          if (row < rows) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<float4*>(dst + 32 * x)[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        if (!half && row < rows) a.ml[at] = make_float2(m, l);
        asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory");  // the sums have been read
        fence_before();
      }
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
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kColumns) : "memory");
}

// ---------------------------------------------------------------- joining
// One warp per (sequence, query head): the pieces of its prefix and of its own tokens.
template <int D>
__global__ void __launch_bounds__(256) shared_join_kernel(const __grid_constant__ SharedArgs a) {
  __shared__ Plan plan;
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) build_plan(a, plan, lane);
  __syncthreads();
  pdl_wait();
  const int Hq = a.Hkv * a.G;
  const int item = blockIdx.x * 8 + (threadIdx.x >> 5), s = item / Hq, hq = item % Hq, h = hq / a.G;
  if (item >= a.B * Hq || !a.part[s]) return;
  const int total = plan.cum[a.entries];
  float m = -INFINITY, l = 0.f, o[V] = {};
  for (int side = 0; side < 2; ++side) {
    if (side == 0 && a.prefix_seq[s] < 0) continue;
    const int e = side ? a.tail_entry[s] : a.prefix_entry[s];
    const int r = hq % a.G + (side ? 0 : a.prefix_row[s]);
    const int units = entry_units(a, plan, e);
    if (!units) continue;
    const int64_t u0 = plan.cum[e] + h * units + kItemUnits, u1 = plan.cum[e] + (h + 1) * units - 1;  // first and last tile
    const int c1 = (int)(((u1 + 1) * a.P - 1) / total);
    for (int c = (int)(((u0 + 1) * a.P - 1) / total); c <= c1; ++c) {
      if (cta_unit(c, a.P, total) == cta_unit(c + 1, a.P, total)) continue;
      const int64_t at = segment_row(a, e, h, c) + r;
      const float2 w = __ldcg(a.ml + at);
      const float top = fmaxf(m, w.x);
      const float f = m == top ? 1.f : exp2_approx(m - top), f2 = w.x == top ? 1.f : exp2_approx(w.x - top);
      l = l * f + w.y * f2;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = o[i] * f + __ldcg(a.acc + at * D + i * 32 + lane) * f2;
      m = top;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float y = l > 0.f ? o[i] / l : l == 0.f ? 0.f : l;  // without a token: zero; NaN stays
    const int64_t at = (int64_t)item * D + i * 32 + lane;
    if (a.q_bf16) reinterpret_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
    else reinterpret_cast<float*>(a.out)[at] = y;
  }
}

template <int D, int PARTS>
cudaError_t launch(const SharedArgs& a, cudaStream_t st) {
  shared_attend_kernel<D, PARTS><<<a.P, kThreads, smem_bytes<D, PARTS>(), st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = (a.B * a.Hkv * a.G + 7) / 8;
  cfg.blockDim = 256;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shared_join_kernel<D>, a);
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
