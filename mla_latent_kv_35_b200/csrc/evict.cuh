// evict.cuh -- eviction from the paged cache by gathered attention weight.
//
// What it computes, for a sequence of L cached tokens and a budget: the
// n_out = min(max(L - budget, 0), free) free slots with the smallest
// (weight, slot) leave, where a slot is free when its token's position is
// neither among the first n_sink nor among the last n_recent positions.  The
// survivors end in slots [0, L - n_out): the k-th survivor behind that end
// moves into the k-th slot that was vacated before it.  Attention sums over
// the cached tokens in any order (a RoPE key carries its position), so the
// order of slots need not follow positions, and this moves the fewest rows
// there can be: sources lie behind the new end and destinations before it,
// so every row moves on its own, in place.
//
// evict_plan_kernel: a cluster of 1 to 8 blocks per sequence.
//   * Weights are compared as 32-bit keys that order like the floats (-0 as
//     0; NaN behind +inf, so a NaN weight is kept longest).  Three passes of
//     11, 11 and 10 bits find the n_out-th smallest key: a histogram of the
//     digit in shared memory, summed over the cluster's blocks through
//     distributed shared memory, then a scan for the digit that holds the
//     rank.  Nothing is sorted.
//   * Among equal keys the lowest slots leave.  Every warp owns one run of
//     consecutive slots and walks it with ballots, so ranks within a run need
//     no barrier; the runs' counts meet in two scans per block and one
//     exchange per cluster.
//   * It writes the pairs (vacated slot, moving slot), the survivors' weights
//     and positions that stay where they are, and the new length.
// evict_move_kernel: a warp per pair copies the row, its weight and its
// position.
//
// Bound: the plan by latency (six walks over a block's part of the weights,
// the later ones from L1, and four cluster barriers), the move by memory
// bandwidth.
#pragma once

#include "common.cuh"

namespace mla {

constexpr int kEvictThreads = 1024;
constexpr int kEvictMaxCluster = 8;
constexpr int kEvictBins = 2048;
// slots per block from which a sequence gets another block
constexpr int kEvictSlotsPerBlock = 4096;

struct EvictArgs {
  const int32_t* seq_lens;
  const int32_t* budget;
  const float* weights;       // [B][stride]
  const int32_t* slot_pos;    // [B][stride], or nullptr: position = slot
  float* new_weights;         // [B][stride], may be weights
  int32_t* new_pos;           // [B][stride], may be slot_pos; nullptr: not kept
  int32_t* new_lens;          // [B], may be seq_lens
  int2* pairs;                // [B][stride]: (to, from)
  int32_t* n_pairs;           // [B]
  long long stride;
  int max_tokens;             // max_pages * page_size
  int n_sink, n_recent;
};

// key order: -inf < ... < -0 = 0 < ... < +inf < NaN
__device__ __forceinline__ uint32_t evict_key(float w) {
  uint32_t u = __float_as_uint(w);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  if ((u & 0x7FFFFFFFu) == 0) u = 0;
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ uint32_t cluster_nctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}

__device__ __forceinline__ int ld_cluster(uint32_t addr, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(addr, rank)) : "memory");
  return v;
}

__device__ __forceinline__ int warp_inclusive(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Exclusive prefix over the warps of the cluster's blocks, in slot order, of
// one count per warp; *total receives the sum.  Every thread of the cluster
// calls it; cell is a shared word that no other call of the kernel uses.
struct EvictScan {
  int warp_sum[32];
  int block_sum;
};
__device__ __forceinline__ int evict_scan(EvictScan* sc, int count, int warp, int lane,
                                          uint32_t rank, uint32_t n, int* total) {
  if (lane == 0) sc->warp_sum[warp] = count;
  __syncthreads();
  const int mine = sc->warp_sum[lane];
  const int inc = warp_inclusive(mine, lane);
  const int before = __shfl_sync(0xffffffffu, inc - mine, warp);
  const int all = __shfl_sync(0xffffffffu, inc, 31);
  if (n == 1) {
    *total = all;
    return before;
  }
  if (threadIdx.x == 0) sc->block_sum = all;
  cluster_sync();
  int base = 0, sum = 0;
  for (uint32_t r = 0; r < n; ++r) {
    const int v = ld_cluster(smem_u32(&sc->block_sum), r);
    base += r < rank ? v : 0;
    sum += v;
  }
  *total = sum;
  return base + before;
}

__global__ void __launch_bounds__(kEvictThreads) evict_plan_kernel(const EvictArgs a) {
  __shared__ int hist[3][kEvictBins];        // one per pass: no barrier to reuse it
  __shared__ EvictScan scan_free, scan_eq, scan_hole, scan_move;
  __shared__ int digit_sh, below_sh, max_sh;
  const uint32_t n = cluster_nctas(), rank = cluster_ctarank();
  const int b = blockIdx.x / n;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int L = a.seq_lens[b];
  const bool bad = L < 0 || L > a.max_tokens || L > a.stride;
  const float* w = a.weights + b * a.stride;
  const int32_t* sp = a.slot_pos != nullptr ? a.slot_pos + b * a.stride : nullptr;
  const int Lc = bad ? 0 : L;
  // this warp's run of slots: a multiple of 32 for every warp
  const int run = ((Lc + (int)n * 1024 - 1) / ((int)n * 1024)) * 32;
  const int s0 = min(Lc, ((int)rank * 32 + warp) * run), s1 = min(Lc, s0 + run);
  for (int i = threadIdx.x; i < 3 * kEvictBins; i += kEvictThreads) (&hist[0][0])[i] = 0;
  if (threadIdx.x == 0) max_sh = -1;
  __syncthreads();

  // ---- the end of the positions, and how many slots are free ----
  int end = Lc;
  if (sp != nullptr) {
    int mx = -1;
    for (int t = s0 + lane; t < s1; t += 32) mx = max(mx, sp[t]);
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (lane == 0) atomicMax(&max_sh, mx);
    if (n > 1) {
      cluster_sync();
      mx = -1;
      for (uint32_t r = 0; r < n; ++r) mx = max(mx, ld_cluster(smem_u32(&max_sh), r));
    } else {
      __syncthreads();
      mx = max_sh;
    }
    end = mx + 1;
  }
  const int p1 = end - a.n_recent;   // free positions: [n_sink, p1)
  auto is_free = [&](int t) {
    const int p = sp != nullptr ? sp[t] : t;
    return p >= a.n_sink && p < p1;
  };
  int n_free = 0;
  if (sp != nullptr) {
    int c = 0;
    for (int t = s0; t < s1; t += 32)
      c += __popc(__ballot_sync(0xffffffffu, t + lane < s1 && is_free(t + lane)));
    evict_scan(&scan_free, c, warp, lane, rank, n, &n_free);
  } else {
    n_free = max(0, p1 - a.n_sink);
  }
  const int n_out = min(max(Lc - max(a.budget[b], 0), 0), n_free);
  const int new_len = Lc - n_out;

  // ---- the n_out-th smallest key, digit by digit ----
  uint32_t prefix = 0;      // digits found so far
  int need = n_out;         // rank among the keys with that prefix, from 1
  if (n_out > 0) {
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bits = pass == 2 ? 10 : 11;
      const uint32_t known = pass == 0 ? 0u : pass == 1 ? 0xFFE00000u : 0xFFFFFC00u;
      for (int t = s0 + lane; t < s1; t += 32) {
        const uint32_t k = evict_key(w[t]);
        if ((k & known) == prefix && is_free(t))
          atomicAdd(&hist[pass][(k >> shift) & ((1u << bits) - 1)], 1);
      }
      if (n > 1) cluster_sync(); else __syncthreads();
      // thread i owns bins 2i, 2i + 1
      int c0 = 0, c1 = 0;
      const uint32_t cell = smem_u32(&hist[pass][2 * threadIdx.x]);
      if (n == 1) {
        c0 = hist[pass][2 * threadIdx.x];
        c1 = hist[pass][2 * threadIdx.x + 1];
      } else {
        for (uint32_t r = 0; r < n; ++r) {
          c0 += ld_cluster(cell, r);
          c1 += ld_cluster(cell + 4, r);
        }
      }
      const int inc = warp_inclusive(c0 + c1, lane);
      if (lane == 31) scan_move.warp_sum[warp] = inc;
      __syncthreads();
      const int ws = scan_move.warp_sum[lane];
      const int wi = warp_inclusive(ws, lane);
      const int before = __shfl_sync(0xffffffffu, wi - ws, warp) + inc - c0 - c1;
      if (before < need && need <= before + c0 + c1) {
        const bool second = need > before + c0;
        digit_sh = 2 * threadIdx.x + (second ? 1 : 0);
        below_sh = before + (second ? c0 : 0);
      }
      __syncthreads();
      prefix |= (uint32_t)digit_sh << shift;
      need -= below_sh;
    }
  }
  const uint32_t kth = prefix;   // `need` of the slots with this key leave, the lowest ones
  __syncthreads();

  // ---- ranks of the equal keys, then of the vacated and the moving slots ----
  int eq0 = 0, n_eq = 0;
  if (n_out > 0) {
    int c = 0;
    for (int t = s0; t < s1; t += 32) {
      const int u = t + lane;
      c += __popc(__ballot_sync(0xffffffffu, u < s1 && evict_key(w[u]) == kth && is_free(u)));
    }
    eq0 = evict_scan(&scan_eq, c, warp, lane, rank, n, &n_eq);
  }
  // one bit per slot of 32: leaves; eq counts the equal keys before the slots
  auto leaving = [&](int t, int& eq) {
    const int u = t + lane;
    const uint32_t k = u < s1 ? evict_key(w[u]) : 0u;
    const bool fr = u < s1 && is_free(u);
    const uint32_t e = __ballot_sync(0xffffffffu, fr && k == kth);
    const int r = eq + __popc(e & ((1u << lane) - 1));
    eq += __popc(e);
    return __ballot_sync(0xffffffffu, fr && (k < kth || (k == kth && r < need)));
  };
  const int live_end = s1;
  int n_hole = 0;
  if (n_out > 0) {
    int eq = eq0, holes = 0, moves = 0;
    for (int t = s0; t < s1; t += 32) {
      const uint32_t out = leaving(t, eq);
      const uint32_t live = live_end - t >= 32 ? 0xffffffffu : (1u << (live_end - t)) - 1;
      const uint32_t front = new_len - t >= 32 ? 0xffffffffu
                             : new_len > t     ? (1u << (new_len - t)) - 1 : 0u;
      holes += __popc(out & front);
      moves += __popc(live & ~out & ~front);
    }
    int n_move;
    int hole = evict_scan(&scan_hole, holes, warp, lane, rank, n, &n_hole);
    int move = evict_scan(&scan_move, moves, warp, lane, rank, n, &n_move);
    int2* pairs = a.pairs + b * a.stride;
    const uint32_t lower = (1u << lane) - 1;
    eq = eq0;
    for (int t = s0; t < s1; t += 32) {
      const uint32_t out = leaving(t, eq);
      const uint32_t live = live_end - t >= 32 ? 0xffffffffu : (1u << (live_end - t)) - 1;
      const uint32_t front = new_len - t >= 32 ? 0xffffffffu
                             : new_len > t     ? (1u << (new_len - t)) - 1 : 0u;
      const uint32_t h = out & front, m = live & ~out & ~front;
      if (h >> lane & 1) pairs[hole + __popc(h & lower)].x = t + lane;
      if (m >> lane & 1) pairs[move + __popc(m & lower)].y = t + lane;
      hole += __popc(h);
      move += __popc(m);
      if ((live & front & ~out) >> lane & 1) {
        if (a.new_weights != a.weights) a.new_weights[b * a.stride + t + lane] = w[t + lane];
        if (a.new_pos != nullptr && a.new_pos != a.slot_pos)
          a.new_pos[b * a.stride + t + lane] = sp != nullptr ? sp[t + lane] : t + lane;
      }
    }
  } else {
    for (int t = s0 + lane; t < s1; t += 32) {
      if (a.new_weights != a.weights) a.new_weights[b * a.stride + t] = w[t];
      if (a.new_pos != nullptr && a.new_pos != a.slot_pos)
        a.new_pos[b * a.stride + t] = sp != nullptr ? sp[t] : t;
    }
  }
  // every block of the cluster has read seq_lens[b] and its peers' shared
  // memory: the length may be overwritten, and the blocks may end
  if (n > 1) cluster_sync(); else __syncthreads();
  if (rank == 0 && threadIdx.x == 0) {
    if (bad) raise_flag(kFlagBounds);
    a.n_pairs[b] = n_hole;
    a.new_lens[b] = bad ? L : new_len;
  }
}

// Copies the rows of all pairs: a warp per pair, block (x, b) takes pairs
// 8x, 8x + 1, .. of sequence b and every 8 gridDim.x-th after them.  U is the
// widest unit that divides a row (16 or 2 bytes).
template <typename U>
__global__ void __launch_bounds__(256) evict_move_kernel(
    U* pool, int units, int n_pages, int page_size, const int32_t* page_table, int max_pages,
    const float* weights, const int32_t* slot_pos, float* new_weights, int32_t* new_pos,
    const int2* pairs, const int32_t* n_pairs, long long stride) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int n = n_pairs[b];
  const int32_t* pages = page_table + (long long)b * max_pages;
  for (int i = blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += gridDim.x * 8) {
    const int2 p = pairs[b * stride + i];
    const int pt = pages[p.x / page_size], pf = pages[p.y / page_size];
    if (pt < 0 || pt >= n_pages || pf < 0 || pf >= n_pages) {
      if (lane == 0) raise_flag(kFlagBounds);
    } else {
      U* to = pool + ((long long)pt * page_size + p.x % page_size) * units;
      const U* from = pool + ((long long)pf * page_size + p.y % page_size) * units;
#pragma unroll 4
      for (int u = lane; u < units; u += 32) to[u] = from[u];
    }
    if (lane == 0) {
      new_weights[b * stride + p.x] = weights[b * stride + p.y];
      if (new_pos != nullptr)
        new_pos[b * stride + p.x] = slot_pos != nullptr ? slot_pos[b * stride + p.y] : p.y;
    }
  }
}

}  // namespace mla
