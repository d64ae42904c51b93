// Pages of the cache: the tokens and summaries of a sequence copied to other
// sequences (or cut short in place), and listed blocks moved to the front of
// a sequence.  One row of the cache is one 16-token block of a (layer,
// sequence, head), so a sequence's blocks of one head are one contiguous run
// in each of the five arrays.
#include "block_summary.cuh"
#include "compkv_launch.h"

namespace compkv {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int64_t first_row(const PageArgs& a, int layer, int s, int h) {
  return a.rows_per_layer * layer + a.seq_row0[s] + (int64_t)h * a.cap_blocks[s];
}

// Copies `chunks` 16-byte chunks, kThreads threads, four loads in flight each.
__device__ __forceinline__ void copy16(void* dst, const void* src, int chunks) {
  uint4* d = reinterpret_cast<uint4*>(dst);
  const uint4* s = reinterpret_cast<const uint4*>(src);
  for (int i = threadIdx.x; i < chunks; i += 4 * kThreads) {
    uint4 t[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * kThreads < chunks) t[u] = s[i + u * kThreads];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * kThreads < chunks) d[i + u * kThreads] = t[u];
  }
}

// Tokens that pair i of this layer copies; -1 when it is refused.
__device__ __forceinline__ int pair_len(const PageArgs& a, int layer, int i, int held, bool report) {
  const int len = a.lens[i] < 0 ? held : a.lens[i];
  if (len > held || len > a.cap_blocks[a.dst[i]] * kBlock) {
    if (report) set_error(a.status, len > held ? kDevInvalidArg : kDevCapacity, a.dst[i], -1, 3);
    return -1;
  }
  return len;
}

// A work item of a copy: `chunk` blocks of a (group of pairs with one source, layer, head).
struct Item {
  int g, layer, h, b0;
};
__device__ __forceinline__ Item fork_item(const PageArgs& a, int it) {
  Item x;
  x.g = 0;
  while (x.g + 1 < a.groups && a.item0[x.g + 1] <= it) ++x.g;
  const int per = (a.item0[x.g + 1] - a.item0[x.g]) / (a.layers * a.Hkv);  // chunks of a (layer, head)
  it -= a.item0[x.g];
  x.b0 = it % per * a.chunk;
  it /= per;
  x.h = it % a.Hkv;
  x.layer = a.layer0 + it / a.Hkv;
  return x;
}
__device__ __forceinline__ int held_tokens(const PageArgs& a, int layer, int s) {
  return max(0, min(__ldcg(a.seq_len + (int64_t)layer * a.B + s), a.cap_blocks[s] * kBlock));
}

// What remains of an item beside the bulk of it, by one warp: lengths, grouped variances, the summary of a block
// that the copy leaves incomplete, cuts in place.
template <int D>
__device__ __forceinline__ void fork_rest(const PageArgs& a, const Item& x, int held, int lane) {
  const int s = a.src[a.pair0[x.g]];
  const bool first = !x.h && !x.b0;
  for (int i = a.pair0[x.g]; i < a.pair0[x.g + 1]; ++i) {
    const int to = a.dst[i];
    if (to == s && !first) continue;
    const int len = pair_len(a, x.layer, i, held, first && lane == 0);
    if (len < 0) continue;
    const int part = len % kBlock;
    if (to == s) {  // a cut in place: one warp for all heads, the length last
      for (int h = 0; part && len < held && h < a.Hkv; ++h) {
        const int64_t row = first_row(a, x.layer, s, h) + len / kBlock;
        warp_block_summary<D>(a.k + row * kBlock * D, a.v + row * kBlock * D, part, nullptr, nullptr, a.kbar + row * D,
                              a.vbar + row * D, a.dbar + row * a.r, a.r, lane);
      }
      if (lane == 0) a.seq_len[(int64_t)x.layer * a.B + to] = len;
      continue;
    }
    if (first && lane == 0) a.seq_len[(int64_t)x.layer * a.B + to] = len;
    const int tokens = min(len - x.b0 * kBlock, a.chunk * kBlock);
    if (tokens <= 0) continue;
    const int64_t rs = first_row(a, x.layer, s, x.h) + x.b0, rd = first_row(a, x.layer, to, x.h) + x.b0;
    const bool cut = part && len < held && tokens < a.chunk * kBlock;
    const int nb = tokens / kBlock + (tokens % kBlock && !cut);
    for (int c = lane; c < nb * a.r; c += 32) a.dbar[rd * a.r + c] = a.dbar[rs * a.r + c];
    if (cut)
      warp_block_summary<D>(a.k + (rs + nb) * kBlock * D, a.v + (rs + nb) * kBlock * D, part, nullptr, nullptr,
                            a.kbar + (rd + nb) * D, a.vbar + (rd + nb) * D, a.dbar + (rd + nb) * a.r, a.r, lane);
  }
}

// Persistent CTAs.  One thread moves the runs of K, V, kbar and vbar by bulk
// copies through a ring of stages in shared memory: each run is read once and
// written to every destination of the group; a warp does the rest of the items.
// Bound by DRAM with r 4: one copy of 64K tokens of 4 layers moves 2.42 GB in
// 381 us, 0.94 of the copy rate; 15 copies of 8K tokens, almost all of it writes,
// 2.42 GB in 409 to 424 us (plain loads and stores: 480).  With r 64 and 128 the one warp
// that copies Dbar, a word a lane at a time, sets the pace: 647 and 999 us for the
// one copy, 455 and 648 for the 15.
constexpr int kStageBytes = 32 * 1024, kForkStages = 3;
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
template <int D>
__global__ void __launch_bounds__(64) fork_bulk_kernel(const __grid_constant__ PageArgs a) {
  extern __shared__ __align__(128) char ring[];
  __shared__ __align__(8) uint64_t full[kForkStages];
  const int items = a.item0[a.groups];
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kForkStages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x >= 32) {
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
      const Item x = fork_item(a, it);
      fork_rest<D>(a, x, held_tokens(a, x.layer, a.src[a.pair0[x.g]]), lane);
    }
    return;
  }
  if (lane) return;

  struct Run {
    Item x;
    int held, kind, off, bytes;  // array, and bytes of the item's run in it
  };
  constexpr int kRow[4] = {kBlock * D * 2, kBlock * D * 2, D * 4, D * 4};  // bytes of a block
  char* base[4] = {reinterpret_cast<char*>(a.k), reinterpret_cast<char*>(a.v), reinterpret_cast<char*>(a.kbar),
                   reinterpret_cast<char*>(a.vbar)};
  // bytes of an item that `len` tokens give in an array; the summary of a block left incomplete is not copied
  auto extent = [&](const Run& r, int len, int kind) {
    const int tokens = max(0, min(len - r.x.b0 * kBlock, a.chunk * kBlock));
    if (kind < 2) return tokens * D * 2;
    return (tokens / kBlock + (tokens % kBlock && len == r.held)) * (D * 4);
  };
  Run run[kForkStages];
  int it = blockIdx.x;
  Run cur;
  int most = 0;  // tokens that the longest copy of the current item's group takes
  bool open = false;
  auto next = [&](Run& r) {  // the next run with bytes in it
    for (;;) {
      if (!open) {
        if (it >= items) return false;
        cur.x = fork_item(a, it);
        it += gridDim.x;
        const int s = a.src[a.pair0[cur.x.g]];
        cur.held = held_tokens(a, cur.x.layer, s);
        most = -1;
        for (int i = a.pair0[cur.x.g]; i < a.pair0[cur.x.g + 1]; ++i)
          if (a.dst[i] != s) most = max(most, pair_len(a, cur.x.layer, i, cur.held, false));
        if (most < 0) continue;
        cur.kind = cur.off = 0;
        open = true;
      }
      const int all = extent(cur, most, cur.kind);
      if (cur.off >= all) {
        cur.off = 0;
        open = ++cur.kind < 4;
        continue;
      }
      cur.bytes = min(all - cur.off, kStageBytes);
      r = cur;
      cur.off += cur.bytes;
      return true;
    }
  };
  int loads = 0, done = 0;
  bool more = true, lost = false;
  while (!lost) {
    while (more && loads < done + kForkStages - 1) {
      const int st = loads % kForkStages;
      // the stores out of this stage, kForkStages loads ago, have read it: all but the last group have
      if (loads >= kForkStages) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      if (!(more = next(run[st]))) break;
      const Run& r = run[st];
      const char* src = base[r.kind] + (first_row(a, r.x.layer, a.src[a.pair0[r.x.g]], r.x.h) + r.x.b0) * kRow[r.kind] + r.off;
      mbar_arrive_expect_tx(&full[st], r.bytes);
      bulk_g2s(ring + st * kStageBytes, src, r.bytes, &full[st]);
      ++loads;
    }
    if (done == loads) break;
    const int st = done % kForkStages;
    lost = !mbar_wait_bounded(&full[st], (done / kForkStages) & 1, a.status, -1, -1, 60);
    const Run& r = run[st];
    const int s = a.src[a.pair0[r.x.g]];
    for (int i = a.pair0[r.x.g]; !lost && i < a.pair0[r.x.g + 1]; ++i) {
      if (a.dst[i] == s) continue;
      const int len = pair_len(a, r.x.layer, i, r.held, false);
      const int n = len < 0 ? 0 : min(extent(r, len, r.kind) - r.off, r.bytes);
      if (n > 0)
        bulk_s2g(base[r.kind] + (first_row(a, r.x.layer, a.dst[i], r.x.h) + r.x.b0) * kRow[r.kind] + r.off, ring + st * kStageBytes, n);
    }
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    ++done;
  }
  if (lost)
    for (; done < loads; ++done) mbar_drain_bounded(&full[done % kForkStages]);
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the stages stay until they have been read
}

// The same with plain loads and stores, for K and V in host memory: one CTA
// per item.
template <int D>
__global__ void __launch_bounds__(kThreads) fork_kernel(const __grid_constant__ PageArgs a) {
  const Item x = fork_item(a, blockIdx.x);
  const int s = a.src[a.pair0[x.g]], held = held_tokens(a, x.layer, s);
  __syncthreads();  // every thread has read the length, which a cut in place changes
  if (threadIdx.x < 32) fork_rest<D>(a, x, held, threadIdx.x);
  for (int i = a.pair0[x.g]; i < a.pair0[x.g + 1]; ++i) {
    const int len = a.dst[i] == s ? -1 : pair_len(a, x.layer, i, held, false);
    const int tokens = min(len - x.b0 * kBlock, a.chunk * kBlock);
    if (tokens <= 0) continue;
    const int64_t rs = first_row(a, x.layer, s, x.h) + x.b0, rd = first_row(a, x.layer, a.dst[i], x.h) + x.b0;
    copy16(a.k + rd * kBlock * D, a.k + rs * kBlock * D, tokens * D / 8);
    copy16(a.v + rd * kBlock * D, a.v + rs * kBlock * D, tokens * D / 8);
    const int nb = tokens / kBlock + (tokens % kBlock && len == held);
    copy16(a.kbar + rd * D, a.kbar + rs * D, nb * D / 4);
    copy16(a.vbar + rd * D, a.vbar + rs * D, nb * D / 4);
  }
}

// By a CTA, for pair `x` = (layer, i) of the call: are the lists of all heads
// ascending block indices of the source, equally long, padded by -1, and does
// the source's last block stand in all of them or in none (it may hold fewer
// tokens)?  Kept blocks (-1: refused) and tokens.  `tell`: reports a refusal,
// or sets the destination's length.
__device__ int2 compact_verdict(const PageArgs& a, int x, bool tell) {
  __shared__ int s_count[32], s_last[32], s_bad;
  const int i = x % a.n, layer = a.layer0 + x / a.n;
  const int src = a.src[i], to = a.dst[i];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int held = held_tokens(a, layer, src);
  const int N = ceil_blocks(held);
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  for (int h = warp; h < a.Hkv; h += kThreads / 32) {
    const int* list = a.keep + ((int64_t)x * a.Hkv + h) * a.keep_blocks;
    int count = 0, last = 0, bad = 0;
    for (int j = lane; j < a.keep_blocks; j += 32) {
      const int b = __ldg(list + j), before = j ? __ldg(list + j - 1) : -1;
      if (b >= 0) {
        ++count;
        bad |= b >= N || before >= b || (j && before < 0);
        last |= b == N - 1;
      } else {
        bad |= b != -1;
      }
    }
    for (int o = 16; o > 0; o >>= 1) count += __shfl_xor_sync(0xffffffffu, count, o);
    last = __any_sync(0xffffffffu, last);
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&s_bad, 1);
    if (lane == 0) {
      s_count[h] = count;
      s_last[h] = last;
    }
  }
  __syncthreads();
  const int count = s_count[0];
  bool bad = s_bad != 0;
  for (int h = 1; h < a.Hkv; ++h) bad |= s_count[h] != count || s_last[h] != s_last[0];
  const bool full = count > a.cap_blocks[to];
  const int tokens = !count ? 0 : s_last[0] ? (count - 1) * kBlock + held - (N - 1) * kBlock : count * kBlock;
  if (tell && threadIdx.x == 0) {
    if (bad || full) set_error(a.status, bad ? kDevBadSelection : kDevCapacity, src, -1, 4);
    else a.seq_len[(int64_t)layer * a.B + to] = tokens;
  }
  return bad || full ? make_int2(-1, 0) : make_int2(count, tokens);
}

__global__ void __launch_bounds__(kThreads) compact_check_kernel(const __grid_constant__ PageArgs a) {
  const int2 v = compact_verdict(a, blockIdx.x, true);
  if (threadIdx.x == 0) a.verdict[blockIdx.x] = v;
}

// Out of place: one CTA per (layer, pair) and 8 blocks of its heads' lists, a
// warp a block.  AT_ONCE: it checks the lists itself; the source's length stays.  Bound by DRAM (8 sequences to
// 1024 blocks each, 2 layers: 2.42 GB in 368 us); 64 blocks of 8 heads take 5.7 us.
template <int D, bool AT_ONCE>
__global__ void __launch_bounds__(kThreads) compact_copy_kernel(const __grid_constant__ PageArgs a) {
  const int lane = threadIdx.x & 31, x = blockIdx.y, i = x % a.n, layer = a.layer0 + x / a.n;
  if (a.src[i] == a.dst[i]) return;
  const int2 v = AT_ONCE ? compact_verdict(a, x, blockIdx.x == 0) : __ldcg(a.verdict + x);
  const int it = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);  // (head, place in its list)
  const int h = it / a.keep_blocks, j = it % a.keep_blocks;
  if (h >= a.Hkv || j >= v.x) return;
  const int64_t rs = first_row(a, layer, a.src[i], h) + __ldg(a.keep + ((int64_t)x * a.Hkv + h) * a.keep_blocks + j);
  const int64_t rd = first_row(a, layer, a.dst[i], h) + j;
  const int chunks = min(v.y - j * kBlock, kBlock) * D / 8;
  const uint4* ks = reinterpret_cast<const uint4*>(a.k + rs * kBlock * D);
  const uint4* vs = reinterpret_cast<const uint4*>(a.v + rs * kBlock * D);
  uint4* kd = reinterpret_cast<uint4*>(a.k + rd * kBlock * D);
  uint4* vd = reinterpret_cast<uint4*>(a.v + rd * kBlock * D);
  constexpr int U = kBlock * D / 8 / 32;
  uint4 kt[U], vt[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u * 32 + lane < chunks) {
      kt[u] = ks[u * 32 + lane];
      vt[u] = vs[u * 32 + lane];
    }
  const int e = lane * (D / 32);
  float mk[D / 32], mv[D / 32];
#pragma unroll
  for (int u = 0; u < D / 32; ++u) {
    mk[u] = a.kbar[rs * D + e + u];
    mv[u] = a.vbar[rs * D + e + u];
  }
  for (int c = lane; c < a.r; c += 32) a.dbar[rd * a.r + c] = a.dbar[rs * a.r + c];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u * 32 + lane < chunks) {
      kd[u * 32 + lane] = kt[u];
      vd[u * 32 + lane] = vt[u];
    }
#pragma unroll
  for (int u = 0; u < D / 32; ++u) {
    a.kbar[rd * D + e + u] = mk[u];
    a.vbar[rd * D + e + u] = mv[u];
  }
}

// In place.  Block j comes from keep[j] >= j, so blocks have to be moved in
// ascending order, but the columns of a row are independent of one another: a
// CTA takes a 512-byte column slice of one array of one (layer, pair, head)
// and walks the list alone, kInBlocks blocks a turn (all loaded before any is
// stored; later turns read behind what this one wrote).  8 sequences of 8 heads
// and 2 layers, forked whole and then cut from 2048 blocks to 256, take 837 to 851
// us in different runs, 0.96 to 0.94 of the copy rate in all.
constexpr int kInBlocks = 32;
template <int D>
__global__ void __launch_bounds__(kThreads) compact_in_place_kernel(const __grid_constant__ PageArgs a) {
  constexpr int KS = kBlock * D * 2 / 512;  // slices of K, as many of V, then kbar, vbar, dbar
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = blockIdx.x;
  const int slice = (int)(x % (2 * KS + 3));
  x /= 2 * KS + 3;
  const int h = (int)(x % a.Hkv);
  x /= a.Hkv;
  const int i = (int)(x % a.n), layer = a.layer0 + (int)(x / a.n);
  if (a.src[i] != a.dst[i]) return;
  const int2 v = __ldcg(a.verdict + x);
  const int* list = a.keep + (x * a.Hkv + h) * a.keep_blocks;
  const int64_t r0 = first_row(a, layer, a.src[i], h);
  // this lane's bytes of a row: `base + row * pitch`, `step` floats or 16-byte chunks
  const bool tokens = slice < 2 * KS;
  constexpr int PER = kInBlocks / (kThreads / 32);
  if (tokens) {
    const int col = (slice % KS) * 32 + lane;  // 16-byte chunk of the row
    uint4* base = reinterpret_cast<uint4*>(slice < KS ? a.k : a.v) + r0 * (kBlock * D / 8) + col;
    for (int j0 = 0; j0 < v.x; j0 += kInBlocks) {
      uint4 t[PER];
      bool go[PER];
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int j = j0 + u * (kThreads / 32) + warp;
        const int b = j < v.x ? __ldg(list + j) : j;
        go[u] = b > j && col < min(v.y - j * kBlock, kBlock) * D / 8;
        if (go[u]) t[u] = base[(int64_t)b * (kBlock * D / 8)];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < PER; ++u)
        if (go[u]) base[(int64_t)(j0 + u * (kThreads / 32) + warp) * (kBlock * D / 8)] = t[u];
    }
  } else {
    const int w = slice == 2 * KS + 2 ? a.r : D;
    float* base = (slice == 2 * KS ? a.kbar : slice == 2 * KS + 1 ? a.vbar : a.dbar) + r0 * w;
    for (int j0 = 0; j0 < v.x; j0 += kInBlocks) {
      float t[PER][4];
      int b[PER];
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int j = j0 + u * (kThreads / 32) + warp;
        b[u] = j < v.x ? __ldg(list + j) : j;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (b[u] > j && c * 32 + lane < w) t[u][c] = base[(int64_t)b[u] * w + c * 32 + lane];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int j = j0 + u * (kThreads / 32) + warp;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (b[u] > j && c * 32 + lane < w) base[(int64_t)j * w + c * 32 + lane] = t[u][c];
      }
    }
  }
}

}  // namespace

cudaError_t launch_fork(const PageArgs& a, int sms, cudaStream_t st) {
  const int items = a.item0[a.groups];
  if (a.kv_host) {
    if (a.d == 128) fork_kernel<128><<<(unsigned)items, kThreads, 0, st>>>(a);
    else fork_kernel<64><<<(unsigned)items, kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  const unsigned grid = (unsigned)(items < 2 * sms ? items : 2 * sms);
  const int smem = kForkStages * kStageBytes;
  if (a.d == 128) fork_bulk_kernel<128><<<grid, 64, smem, st>>>(a);
  else fork_bulk_kernel<64><<<grid, 64, smem, st>>>(a);
  return cudaGetLastError();
}

cudaError_t prepare_pages(int d) {
  return raise_smem_limit(d == 128 ? (const void*)fork_bulk_kernel<128> : (const void*)fork_bulk_kernel<64>,
                          kForkStages * kStageBytes);
}

cudaError_t launch_compact(const PageArgs& a, int in, cudaStream_t st) {
  const int pairs = a.layers * a.n;
  const dim3 grid((unsigned)(((int64_t)a.Hkv * a.keep_blocks + kThreads / 32 - 1) / (kThreads / 32)), pairs);
  if (compact_at_once(a, in)) {
    if (a.d == 128) compact_copy_kernel<128, true><<<grid, kThreads, 0, st>>>(a);
    else compact_copy_kernel<64, true><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  compact_check_kernel<<<pairs, kThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && in < a.n) {
    if (a.d == 128) compact_copy_kernel<128, false><<<grid, kThreads, 0, st>>>(a);
    else compact_copy_kernel<64, false><<<grid, kThreads, 0, st>>>(a);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && in) {
    const unsigned ctas = (unsigned)(pairs * a.Hkv) * (2 * kBlock * a.d * 2 / 512 + 3);
    if (a.d == 128) compact_in_place_kernel<128><<<ctas, kThreads, 0, st>>>(a);
    else compact_in_place_kernel<64><<<ctas, kThreads, 0, st>>>(a);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace compkv
