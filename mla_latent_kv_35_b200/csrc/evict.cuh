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
//     digit in shared memory, then one warp finds the digit that holds the
//     rank, first among sums of 64 bins, then among the 64, each summed over
//     the cluster's blocks through distributed shared memory (32 + 64 words of
//     every block; reading all 2048 bins took 4000 clocks a pass against 1600
//     with eight blocks).  Nothing is sorted.  The first pass's sum is the number of free
//     slots, so it needs no count of its own.  Where all keys that share the
//     digits found so far leave, the remaining passes are left out.
//   * Every warp owns one run of consecutive slots, 32 at a time, and keeps
//     their keys in registers (up to 16 per thread; each pass reads the
//     weights of a longer run's rest again).  Ranks
//     within a run come from ballots; the runs' counts meet in one scan per
//     block and one exchange per cluster.
//   * Where at most three leave, the least (key, slot) is found that many
//     times instead, each by a minimum over registers, warps and blocks.
//   * Among equal keys the lowest slots leave.  Their ranks take another
//     exchange, made only where some of the equal ones stay.
//   * It writes the vacated and the moving slots, the weights and positions
//     before the new end, and the new length.  Those of a vacated slot are
//     written too, while they are at hand, since the move overwrites them.
// evict_move_kernel: every warp takes an even share of all sequences' pairs
// and copies row, weight and position, two rows in flight; pairs and page ids
// are looked up 32 at a time, a lane each (two rows at a time, three trips to
// memory for each: 55 against 52 us for the ragged batch).  (A grid of blocks
// per sequence left the SMs of the short ones idle: 116 us against 33 for 64
// ragged sequences.)
//
// Bound: the plan by latency (loads, then three to six cluster barriers) and by
// instruction issue (32 warps on one SM), the move by memory bandwidth.
// Measured in a graph: one token of 16 x 4097 8.2 us (8.8 with positions), 64
// sequences of 129 to 32769 tokens to 30 % 53 us (plan 18.5), 4 x 131072 halved
// 76 to 79 us (plan 21).
#pragma once

#include "common.cuh"

namespace mla {

constexpr int kEvictThreads = 1024;
constexpr int kEvictMaxCluster = 8;    // (16, beyond the portable size: 42 against 35 us)
constexpr int kEvictMaxStride = 1 << 30;   // slots are counted in 32 bits, with room
constexpr int kEvictBins = 2048;
// Keys a thread can hold: 8 where that is enough (fewer instructions per
// thread: with 1024 threads the plan is bound by instruction issue), else 16.
constexpr int kEvictFewKeys = 8, kEvictKeys = 16;
// Up to so many tokens of a sequence leave one after the other, as when every
// decode step adds a few to a full budget: 1.3 to 1.6 us each for 4097 tokens
// (one token: 8.2 us with its move, 8.8 with positions, against 12.3 by the
// histograms; four take 12.2 either way), 3 us for 131072 (one: 13.5, 15.4 with
// positions, against 23.3; four 21.5 against 23.5).
constexpr int kEvictPicks = 3;
constexpr int kEvictGroups = 2048;                          // sequence groups of the move

struct EvictArgs {
  const int32_t* seq_lens;
  const int32_t* budget;
  const float* weights;       // [B][stride]
  const int32_t* slot_pos;    // [B][stride], or nullptr: position = slot
  float* new_weights;         // [B][stride], may be weights
  int32_t* new_pos;           // [B][stride], may be slot_pos; nullptr: not kept
  int32_t* new_lens;          // [B], may be seq_lens
  int32_t* pairs;             // [B][2][stride]: vacated slots, moving slots
  int32_t* n_pairs;           // [B]
  long long stride;
  int max_tokens;             // max_pages * page_size
  int n_sink, n_recent;
};

// key order: -inf < ... < -0 = 0 < ... < +inf < NaN < a slot that is not free
constexpr uint32_t kEvictKept = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t evict_key(float w) {
  uint32_t u = __float_as_uint(w);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return kEvictKept - 1;
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

// Sum of the words at `p` over the cluster's n blocks, all remote reads in
// flight at once: one takes about 600 clocks.
__device__ __forceinline__ int cluster_sum(const int* p, uint32_t n) {
  if (n == 1) return *p;
  int sum = 0, v[kEvictMaxCluster];
#pragma unroll
  for (uint32_t r = 0; r < kEvictMaxCluster; ++r) {
    v[r] = 0;
    if (r < n)
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v[r]) : "r"(mapa_shared(smem_u32(p), r)));
  }
#pragma unroll
  for (uint32_t r = 0; r < kEvictMaxCluster; ++r) sum += v[r];
  return sum;
}

// The pair of words at `addr` in every block of the cluster (zeros past the
// n-th).
__device__ __forceinline__ void ld_cluster_all(uint32_t addr, uint32_t n,
                                               int2 (&v)[kEvictMaxCluster]) {
#pragma unroll
  for (uint32_t r = 0; r < kEvictMaxCluster; ++r) {
    v[r] = make_int2(0, 0);
    if (r < n)
      asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];"
                   : "=r"(v[r].x), "=r"(v[r].y)
                   : "r"(mapa_shared(addr, r)));
  }
}
__device__ __forceinline__ int2 cluster_sum(const int2* p, uint32_t n) {
  if (n == 1) return *p;
  int2 sum = make_int2(0, 0), v[kEvictMaxCluster];
  ld_cluster_all(smem_u32(p), n, v);
#pragma unroll
  for (uint32_t r = 0; r < kEvictMaxCluster; ++r) {
    sum.x += v[r].x;
    sum.y += v[r].y;
  }
  return sum;
}

__device__ __forceinline__ int warp_inclusive(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

__device__ __forceinline__ unsigned long long warp_least(unsigned long long x) {
  const uint32_t hi = (uint32_t)(x >> 32);
  const uint32_t h = __reduce_min_sync(0xffffffffu, hi);
  const uint32_t l = __reduce_min_sync(0xffffffffu, hi == h ? (uint32_t)x : 0xffffffffu);
  return (unsigned long long)h << 32 | l;
}

// Exclusive prefix over the warps of the cluster's blocks, in slot order, of
// one pair of counts per warp; *total receives the sums.  Every thread of the
// cluster calls it, each call with a cell of its own.
struct EvictScan {
  int2 warp_sum[32];
  __align__(8) int2 block_sum;
};
__device__ __forceinline__ int2 evict_scan(EvictScan* sc, int2 count, int warp, int lane,
                                           uint32_t rank, uint32_t n, int2* total) {
  if (lane == 0) sc->warp_sum[warp] = count;
  __syncthreads();
  const int2 mine = sc->warp_sum[lane];
  const int ix = warp_inclusive(mine.x, lane), iy = warp_inclusive(mine.y, lane);
  int2 before = make_int2(__shfl_sync(0xffffffffu, ix - mine.x, warp),
                          __shfl_sync(0xffffffffu, iy - mine.y, warp));
  *total = make_int2(__shfl_sync(0xffffffffu, ix, 31), __shfl_sync(0xffffffffu, iy, 31));
  if (n == 1) return before;
  if (threadIdx.x == 0) sc->block_sum = *total;
  cluster_sync();
  int2 sum = make_int2(0, 0), v[kEvictMaxCluster];
  ld_cluster_all(smem_u32(&sc->block_sum), n, v);
#pragma unroll
  for (uint32_t r = 0; r < kEvictMaxCluster; ++r) {
    before.x += r < rank ? v[r].x : 0;
    before.y += r < rank ? v[r].y : 0;
    sum.x += v[r].x;
    sum.y += v[r].y;
  }
  *total = sum;
  return before;
}

// kKeys: keys that a thread holds; kRest: a run may be longer than that.
template <int kKeys, bool kRest>
__global__ void __launch_bounds__(kEvictThreads) evict_plan_kernel(const EvictArgs a) {
  __shared__ __align__(16) int hist[3][kEvictBins];   // one per pass: no barrier to reuse it
  __shared__ EvictScan scan_eq, scan_out;
  __shared__ int coarse[3][32];                      // sums of a warp's 64 bins
  __shared__ int4 lists[32][32];                     // per warp: what its groups list
  __shared__ int4 pick_sh;                           // digit, keys below it, keys with it, sum
  __shared__ int max_sh;
  __shared__ __align__(8) unsigned long long picks[kEvictPicks][32], block_pick[kEvictPicks];
  __shared__ int picked[kEvictPicks];                // slots that leave, where few do
  const uint32_t n = cluster_nctas(), rank = cluster_ctarank();
  const int b = blockIdx.x / n;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // (uniform to the compiler)
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < 3 * kEvictBins / 4; i += kEvictThreads)
    reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
  if (threadIdx.x == 0) max_sh = -1;
  pdl_wait();
  pdl_launch();
  const int L = a.seq_lens[b];
  const int cut = a.budget[b];
  const bool bad = L < 0 || L > a.max_tokens || L > a.stride;
  const float* w = a.weights + b * a.stride;
  const int32_t* sp = a.slot_pos != nullptr ? a.slot_pos + b * a.stride : nullptr;
  const int Lc = bad ? 0 : L;
  const int over = max(Lc - max(cut, 0), 0);     // slots above the budget
  // this warp's run of slots: a multiple of 32 for every warp
  const int run = ((Lc + (int)n * kEvictThreads - 1) / ((int)n * kEvictThreads)) * 32;
  const int s0 = min(Lc, ((int)rank * 32 + warp) * run), s1 = min(Lc, s0 + run);
  const int groups = (s1 - s0 + 31) / 32;                // of 32 slots

  // keys of this thread's slots s0 + 32 i + lane
  uint32_t key[kKeys];
  int last = Lc - 1 - a.n_recent;        // free positions: [n_sink, last]
  auto key_of = [&](float x, int p) {
    return p >= a.n_sink && p <= last ? evict_key(x) : kEvictKept;
  };
  // f(i, key) over this thread's groups
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i)
      if (i < groups) f(i, key[i]);
    for (int i = kKeys; kRest && i < groups; ++i) {
      const int t = s0 + 32 * i + lane;
      f(i, t < s1 ? key_of(w[t], sp != nullptr ? sp[t] : t) : kEvictKept);
    }
  };
  // Weight and position of a slot that stays.  A vacated slot before the new
  // end may be written too: the move fills it.
  float* nw = a.new_weights != a.weights ? a.new_weights + b * a.stride : nullptr;
  int32_t* np = a.new_pos != nullptr && a.new_pos != a.slot_pos ? a.new_pos + b * a.stride : nullptr;
  int copied = s0;                       // this warp's slots before it are written

  int n_out = 0, need = 0, n_hole = 0;
  uint32_t kth = 0;       // key of the last slot to leave; `need` slots with it leave
  bool all_leave = false; // all slots up to kth leave
  if (over > 0) {
    int mx = -1;
    // all loads first (a slot past the run reads the run's last one), so that
    // they are in flight together
    int pos[kKeys];
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      key[i] = 0;
      if (i < groups) key[i] = __float_as_uint(w[min(s0 + 32 * i + lane, s1 - 1)]);
    }
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int t = min(s0 + 32 * i + lane, s1 - 1);
      pos[i] = t;
      if (sp != nullptr && i < groups) pos[i] = sp[t];
    }
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int t = s0 + 32 * i + lane;
      if (t < s1) mx = max(mx, pos[i]);
      // the new end lies at Lc - over or behind it
      if (t < min(s1, Lc - over)) {
        if (nw != nullptr) nw[t] = __uint_as_float(key[i]);
        if (np != nullptr) np[t] = pos[i];
      }
    }
    copied = max(s0, min(Lc - over, s0 + 32 * kKeys));
    if (kRest && sp != nullptr)
      for (int t = s0 + 32 * kKeys + lane; t < s1; t += 32) mx = max(mx, sp[t]);
    __syncthreads();
    if (sp != nullptr) {
      mx = __reduce_max_sync(0xffffffffu, mx);
      if (lane == 0) atomicMax(&max_sh, mx);
      if (n > 1) cluster_sync(); else __syncthreads();
      mx = max_sh;
      if (n > 1)
        for (uint32_t r = 0; r < n; ++r) mx = max(mx, ld_cluster(smem_u32(&max_sh), r));
      last = mx - a.n_recent;
    }
#pragma unroll
    for (int i = 0; i < kKeys; ++i)
      key[i] = s0 + 32 * i + lane < s1 ? key_of(__uint_as_float(key[i]), pos[i]) : kEvictKept;

    if (over <= kEvictPicks) {
      // ---- few leave: the least (key, slot), one after the other ----
      unsigned long long least = 0;          // the next one to leave is this or above it
      for (; n_out < over; ++n_out) {
        unsigned long long m = ~0ull;
        each([&](int i, uint32_t k) {
          const unsigned long long x =
              (unsigned long long)k << 32 | (uint32_t)(s0 + 32 * i + lane);
          if (k != kEvictKept && x >= least && x < m) m = x;
        });
        m = warp_least(m);
        if (lane == 0) picks[n_out][warp] = m;
        __syncthreads();
        m = warp_least(picks[n_out][lane]);
        if (n > 1) {
          if (threadIdx.x == 0) block_pick[n_out] = m;
          cluster_sync();
          unsigned long long x = ~0ull;
          if (lane < n)
            asm volatile("ld.shared::cluster.u64 %0, [%1];"
                         : "=l"(x)
                         : "r"(mapa_shared(smem_u32(&block_pick[n_out]), lane)));
          m = warp_least(x);
        }
        if (m == ~0ull) break;               // (uniform: nothing is free)
        if (threadIdx.x == 0) picked[n_out] = (int)(uint32_t)m;
        least = m + 1;
      }
    }
    // ---- the n_out-th smallest key, digit by digit ----
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      if (over <= kEvictPicks) break;
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t mask = pass == 2 ? 0x3FFu : 0x7FFu;
      const uint32_t known = pass == 0 ? 0u : pass == 1 ? 0xFFE00000u : 0xFFFFFC00u;
      each([&](int, uint32_t k) {
        if (k != kEvictKept && (k & known) == kth) atomicAdd(&hist[pass][(k >> shift) & mask], 1);
      });
      __syncthreads();
      {
        const int2 c = reinterpret_cast<const int2*>(hist[pass])[threadIdx.x];
        const int sum = __reduce_add_sync(0xffffffffu, c.x + c.y);
        if (lane == 0) coarse[pass][warp] = sum;
      }
      if (n > 1) cluster_sync(); else __syncthreads();
      if (warp == 0) {
        // the 64 bins that hold the rank, then the bin
        const int c = cluster_sum(&coarse[pass][lane], n);
        const int inc = warp_inclusive(c, lane), all = __shfl_sync(0xffffffffu, inc, 31);
        const int want = pass == 0 ? min(over, all) : need;
        if (want > 0) {
          const int g = __ffs(__ballot_sync(0xffffffffu, inc >= want)) - 1;
          const int front = __shfl_sync(0xffffffffu, inc - c, g);
          const int2 v = cluster_sum(reinterpret_cast<const int2*>(&hist[pass][64 * g]) + lane, n);
          const int before = front + warp_inclusive(v.x + v.y, lane) - v.x - v.y;
          if (before < want && want <= before + v.x + v.y) {
            const bool second = want > before + v.x;
            pick_sh = make_int4(64 * g + 2 * lane + (second ? 1 : 0),
                                before + (second ? v.x : 0), second ? v.y : v.x, all);
          }
        } else if (lane == 0) {
          pick_sh = make_int4(0, 0, 0, all);
        }
      }
      __syncthreads();
      const int4 pick = pick_sh;
      if (pass == 0) {
        n_out = min(over, pick.w);        // the sum: every free slot
        need = n_out;
      }
      if (n_out == 0) break;              // (uniform: nothing is free)
      kth |= (uint32_t)pick.x << shift;
      need -= pick.y;
      all_leave = need == pick.z;
      if (all_leave) {                    // uniform: every key with these digits leaves
        kth = min(kth | ((1u << shift) - 1), kEvictKept - 1);
        break;
      }
    }
  }
  const int new_len = Lc - n_out;
  const uint32_t lower = (1u << lane) - 1;
  if (over <= kEvictPicks) {
    // the vacated slots in order, and the slots behind the new end that stay
    if (rank == 0 && threadIdx.x == 0) {
      int32_t* holes = a.pairs + 2 * b * a.stride;
      int n_move = 0;
      for (int at = -1;;) {
        int hole = new_len;
        for (int i = 0; i < n_out; ++i)
          if (picked[i] > at) hole = min(hole, picked[i]);
        if (hole == new_len) break;
        holes[n_hole++] = at = hole;
      }
      for (int t = new_len; t < Lc; ++t) {
        bool out = false;
        for (int i = 0; i < n_out; ++i) out |= picked[i] == t;
        if (!out) holes[a.stride + n_move++] = t;
      }
    }
  } else if (n_out > 0) {
    // ---- ranks of the equal keys, where some of them stay ----
    int eq0 = 0;
    if (!all_leave) {
      int c = 0;
      each([&](int, uint32_t k) { c += __popc(__ballot_sync(0xffffffffu, k == kth)); });
      int2 sum;
      eq0 = evict_scan(&scan_eq, make_int2(c, 0), warp, lane, rank, n, &sum).x;
    }
    // the slots of a group that leave, as a mask of lanes; eq counts the
    // equal keys of the groups before it
    auto leaving = [&](uint32_t k, int& eq) {
      if (all_leave) return __ballot_sync(0xffffffffu, k <= kth);
      const uint32_t e = __ballot_sync(0xffffffffu, k == kth);
      const int r = eq + __popc(e & lower);
      eq += __popc(e);
      return __ballot_sync(0xffffffffu, k < kth || (k == kth && r < need));
    };
    // slots of group i before the new end, and slots of the run, as masks of
    // lanes
    const int gf = max(new_len - s0, 0) / 32;
    const uint32_t edge = new_len > s0 ? (1u << ((new_len - s0) & 31)) - 1 : 0u;
    const uint32_t tail = s1 - s0 == 32 * groups ? 0xffffffffu : (1u << ((s1 - s0) & 31)) - 1;
    auto front_of = [&](int i) { return i < gf ? 0xffffffffu : i == gf ? edge : 0u; };
    auto run_of = [&](int i) { return i == groups - 1 ? tail : 0xffffffffu; };
    // ---- ranks of the vacated and the moving slots ----
    // Lane i keeps the leaving slots of group i0 + i as a mask, so that a warp
    // scans 32 groups at once; the masks of the first 32 serve both passes.
    auto masks = [&](int i0, int& eq) {
      uint32_t mine = 0;
      if (i0 == 0) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i)
          if (i < groups) {
            const uint32_t out = leaving(key[i], eq);
            mine = lane == i ? out : mine;
          }
      }
      for (int i = max(i0, kKeys); kRest && i < min(groups, i0 + 32); ++i) {
        const int t = s0 + 32 * i + lane;
        const uint32_t out =
            leaving(t < s1 ? key_of(w[t], sp != nullptr ? sp[t] : t) : kEvictKept, eq);
        mine = lane == i - i0 ? out : mine;
      }
      return mine;
    };
    int eq = eq0, eq_first = 0;
    uint32_t first_masks = 0;
    int2 c = make_int2(0, 0);
    for (int i0 = 0; i0 < groups; i0 += 32) {
      const uint32_t out = masks(i0, eq), front = front_of(i0 + lane);
      const uint32_t in = i0 + lane < groups ? run_of(i0 + lane) : 0u;
      if (i0 == 0) {
        first_masks = out;
        eq_first = eq;
      }
      c.x += __popc(out & front);
      c.y += __popc(in & ~out & ~front);
    }
    c.x = __reduce_add_sync(0xffffffffu, c.x);
    c.y = __reduce_add_sync(0xffffffffu, c.y);
    int2 sum, at = evict_scan(&scan_out, c, warp, lane, rank, n, &sum);
    n_hole = sum.x;
    int32_t* holes = a.pairs + 2 * b * a.stride;
    eq = eq_first;
    for (int i0 = 0; i0 < groups; i0 += 32) {
      const uint32_t out = i0 == 0 ? first_masks : masks(i0, eq), front = front_of(i0 + lane);
      const uint32_t in = i0 + lane < groups ? run_of(i0 + lane) : 0u;
      const uint32_t hole = out & front, move = in & ~out & ~front;
      const int nh = __popc(hole), nm = __popc(move);
      const int ih = warp_inclusive(nh, lane), im = warp_inclusive(nm, lane);
      // A slot before the new end is listed as vacated, one behind it as
      // moving; in the group that the end cuts, vacated slots come first.
      __syncwarp();
      lists[warp][lane] = make_int4((int)(hole | move), at.x + ih - nh, at.y + im - nm - nh, 0);
      __syncwarp();
      auto list = [&](int i) {
        const int4 g = lists[warp][i];
        const int t = s0 + 32 * (i0 + i) + lane;
        const bool behind = t >= new_len;
        if ((uint32_t)g.x >> lane & 1)
          (behind ? holes + a.stride : holes)[(behind ? g.z : g.y) + __popc((uint32_t)g.x & lower)] = t;
      };
      if (i0 == 0) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i)
          if (i < groups) list(i);
      }
      for (int i = i0 == 0 ? kKeys : 0; kRest && i < min(32, groups - i0); ++i) list(i);
      at.x += __shfl_sync(0xffffffffu, ih, 31);
      at.y += __shfl_sync(0xffffffffu, im, 31);
    }
  }
  for (int t = copied + lane; t < min(new_len, s1); t += 32) {
    if (nw != nullptr) nw[t] = w[t];
    if (np != nullptr) np[t] = sp != nullptr ? sp[t] : t;
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

// Moves the rows of all pairs.  The pairs of all sequences laid end to end are
// cut evenly over the grid's warps.  U is the widest unit that divides a row
// (16 or 2 bytes).
template <typename U>
__global__ void __launch_bounds__(256) evict_move_kernel(
    U* pool, int units, int n_pages, int page_size, const int32_t* page_table, int max_pages,
    const float* weights, const int32_t* slot_pos, float* new_weights, int32_t* new_pos,
    const int32_t* pairs, const int32_t* n_pairs, int B, long long stride) {
  __shared__ long long before[kEvictGroups + 1];   // pairs before each group of sequences
  __shared__ long long sums[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch();
  const long long warps = (long long)gridDim.x * 8, me = (long long)blockIdx.x * 8 + warp;
  long long lo, hi;          // this warp's pairs
  int b, i, n;               // sequence of pair lo, the pair within it, its pairs
  if (B <= 32) {
    // every warp scans for itself
    const int mine = lane < B ? n_pairs[lane] : 0;
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const long long all = __shfl_sync(0xffffffffu, inc, 31);
    lo = all * me / warps;
    hi = all * (me + 1) / warps;
    if (lo >= hi) return;
    b = __ffs(__ballot_sync(0xffffffffu, inc > lo)) - 1;
    n = __shfl_sync(0xffffffffu, mine, b);
    i = (int)(lo - (__shfl_sync(0xffffffffu, inc, b) - n));
  } else {
    const int per = (B + kEvictGroups - 1) / kEvictGroups, n_groups = (B + per - 1) / per;
    long long base = 0;
    for (int g0 = 0; g0 < n_groups; g0 += 256) {
      const int g = g0 + threadIdx.x;
      long long c = 0;
      for (int s = g * per; g < n_groups && s < min(B, (g + 1) * per); ++s) c += n_pairs[s];
      long long inc = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) sums[warp] = inc;
      __syncthreads();
      long long all = 0, front = 0;
      for (int w = 0; w < 8; ++w) {
        front += w < warp ? sums[w] : 0;
        all += sums[w];
      }
      if (g < n_groups) before[g] = base + front + inc - c;
      base += all;
      __syncthreads();
    }
    if (threadIdx.x == 0) before[n_groups] = base;
    __syncthreads();
    lo = base * me / warps;
    hi = base * (me + 1) / warps;
    if (lo >= hi) return;
    int ga = 0, gb = n_groups - 1;
    while (ga < gb) {
      const int mid = (ga + gb) >> 1;
      if (before[mid + 1] > lo) gb = mid; else ga = mid + 1;
    }
    b = ga * per;
    i = (int)(lo - before[ga]);
    n = n_pairs[b];
    while (i >= n) {
      i -= n;
      n = n_pairs[++b];
    }
  }
  // A lane looks up one pair (slots, pages, rows) and moves its weight and
  // position; then the warp copies the 32 pairs' rows.
  constexpr int kRows = 2;                 // rows in flight (3 or 4 leave fewer warps: no faster)
  for (long long g = lo; g < hi; g += 32) {
    const int count = (int)min(32ll, hi - g);
    int lb = b, li = i + min(lane, count - 1), ln = n;     // (a lane past the end: the last pair)
    while (li >= ln) {
      li -= ln;
      ln = n_pairs[++lb];
    }
    const int to = pairs[2 * lb * stride + li], from = pairs[(2 * lb + 1) * stride + li];
    const int32_t* pages = page_table + (long long)lb * max_pages;
    const int pt = pages[to / page_size], pf = pages[from / page_size];
    long long row_to = (long long)pt * page_size + to % page_size;
    const long long row_from = (long long)pf * page_size + from % page_size;
    if (pt < 0 || pt >= n_pages || pf < 0 || pf >= n_pages) {
      raise_flag(kFlagBounds);
      row_to = -1;
    }
    // weight and position go with the row, or stay with it
    if (lane < count && row_to >= 0) {
      const long long d = lb * stride;
      new_weights[d + to] = weights[d + from];
      if (new_pos != nullptr) new_pos[d + to] = slot_pos != nullptr ? slot_pos[d + from] : from;
    }
    for (int q0 = 0; q0 < count; q0 += kRows) {
      U* dst[kRows];
      const U* src[kRows];
#pragma unroll
      for (int q = 0; q < kRows; ++q) {
        const long long rt = __shfl_sync(0xffffffffu, row_to, q0 + q);
        const long long rf = __shfl_sync(0xffffffffu, row_from, q0 + q);
        dst[q] = q0 + q < count && rt >= 0 ? pool + rt * units : nullptr;
        src[q] = pool + rf * units;
      }
      for (int u0 = 0; u0 < units; u0 += 96) {
        U v[kRows][3];
#pragma unroll
        for (int q = 0; q < kRows; ++q)
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const int u = u0 + 32 * k + lane;
            if (dst[q] != nullptr && u < units) v[q][k] = src[q][u];
          }
#pragma unroll
        for (int q = 0; q < kRows; ++q)
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const int u = u0 + 32 * k + lane;
            if (dst[q] != nullptr && u < units) dst[q][u] = v[q][k];
          }
      }
    }
    // the pair after the last lane's
    b = __shfl_sync(0xffffffffu, lb, 31);
    i = __shfl_sync(0xffffffffu, li, 31) + 1;
    n = __shfl_sync(0xffffffffu, ln, 31);
  }
}

}  // namespace mla
