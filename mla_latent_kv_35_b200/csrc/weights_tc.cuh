// weights_tc.cuh -- the attention weight that every cached token receives from
// the queries of a chunk (tcgen05 pair MMAs, TMEM accumulators, TMA).
//
// What it computes: with s = scale * q . row the scores of mla_decode or
// mla_chunk_attention, and lse what that call returned,
//   w_out[b, t] = keep * w_in[b, t] + sum over the queries j and heads i of
//                 sequence b that see t of exp(s_{j,i,t} - lse_{j,i})
// (w_in read for the tokens cached before the chunk).  The softmax's
// denominators are known, so one pass without running maxima does it: a
// product of the cache rows with the queries, exponentials, and a sum over
// the queries.
//
// Scores are formed with the tokens as the M dimension: S[token, query row]
// lands in TMEM with one token per lane, so the sum over query rows is a sum
// over a thread's own columns, and nothing is exchanged between lanes.  A
// pair of SMs takes 256 tokens (cta_group::2, M = 256): CTA r holds tokens
// [128 r, 128 r + 128) of them (two pages) as its half of A and half of the
// query rows as its half of B.
//
// Two forms, by which operand stays in shared memory:
//   kQStat: all query rows of a sequence (at most kN = 128 or 256: decode
//     and speculative steps) stay, and the cache streams past them, 16 KB
//     stages of 128 tokens x 64 columns.  Every cache row is read once from
//     HBM: bound by memory.
//   otherwise: 256 tokens stay (147 KB per SM) and the query rows stream past
//     them, 256 at a time, from L2: bound by the tensor pipe.  A token tile
//     belongs to one pair for all its rows, so the sum needs no second pass
//     and its order is fixed.
// Work: all sequences' tokens laid end to end, cut into one contiguous run per
// pair: in pages where the queries stay (a run's tiles start at any page, so
// that runs differ by one page, not by one tile), in whole tiles otherwise,
// each weighing the row blocks it meets.  Every CTA finds its run itself (a
// scan over the sequences), so there is no planning launch and no workspace.
//
// Measured: 64 ragged sequences of 129 to 65537 tokens (991 MB) 157 to 166 us
// in a graph, 6.0 to 6.3 TB/s, boxes of three 64-column chunks (one: 203, two:
// 190, three: 182 us with the cache flushed); 16 x 4096 tokens 18.5 to 19 us,
// the start of a sequence counted as three pages in the split (none: 32.0,
// three: 28.7 us with the launch).  4 x 32 queries over 8 K tokens 126 us in a
// graph: 693 clocks per 64-column stage against 512 of MMA, about 64 KB of
// shared memory traffic each, and two tiles for most pairs against 1.73 on
// average.
//
// Row sums: four chains per thread over 32 columns at a time, fp32.  Rows
// whose lse is -inf (a query that saw nothing) or +inf give nothing; one whose
// lse is NaN gives NaN to the tokens it sees.
// Tokens past a sequence's end compute on whatever the page holds there and
// are not stored.
//
// Every mbarrier wait is bounded as in the decode kernel.
#pragma once

#include "common.cuh"
#include "decode_tc.cuh"
#include "chunk_tc.cuh"

namespace mla {

namespace wtc {
constexpr int kD = 576;
constexpr int kPage = 64;
constexpr int kTile = 256;                      // tokens per pair
constexpr int kTileBytes = 9 * 128 * 128;       // this CTA's 128 tokens x 576 columns (147 KB)
constexpr int kThreads = 384;
constexpr int kEpiWarp0 = 4;
constexpr int kEpiThreads = 256;
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxStages = 9;
// Pages that the start of a sequence counts for in the split of resident
// queries: its queries are loaded and one more partial tile is worked.
constexpr int kOpenPages = 3;
template <bool kQStat, int kN>
struct Shape {
  static constexpr int kStat = kQStat ? 9 * (kN / 2) * 128 : kTileBytes;       // stationary bytes
  // A stage: kCps 64-column chunks of 128 tokens, or one of kN / 2 query rows.
  static constexpr int kCps = kQStat && kN == 128 ? 3 : 1;
  static constexpr int kStage = kQStat ? kCps * 128 * 128 : (kN / 2) * 128;
  static constexpr int kSteps = 9 / kCps;                                       // per tile or row block
  static constexpr int kRing = kStat > 100 * 1024 ? 64 * 1024 : 144 * 1024;
  static constexpr int kStages = kRing / kStage;
  static constexpr int kBufs = (int)kTmemCols / kN;                             // S buffers
  static constexpr uint32_t kSmem = kStat + kStages * kStage + 1024;
};
}  // namespace wtc

struct WeightsParams {
  const float* lse;            // [total_q][H]
  const int32_t* cu_q;         // [B + 1]
  const int32_t* page_table;
  const int32_t* seq_lens;
  const float* w_in;           // [B][stride], or nullptr
  float* w_out;                // [B][stride]
  long long stride;
  int total_q, max_q, max_tokens, max_pages, n_pages, B, H;
  float scale_log2, keep;
};

// Units of work of sequence b (0 where its length is impossible): pages where
// the queries stay, else tiles; returns what a unit weighs: 1, or the row
// blocks that a tile meets.
template <bool kQStat, int kN>
__device__ __forceinline__ int weights_units(const WeightsParams& P, int b, int& units) {
  const int T = P.cu_q[b + 1] - P.cu_q[b], L = P.seq_lens[b];
  const bool ok = T >= 0 && L >= T && L <= P.max_tokens && L <= P.stride;
  constexpr int kUnit = kQStat ? wtc::kPage : wtc::kTile;
  units = ok ? (L + kUnit - 1) / kUnit : 0;
  return kQStat ? 1 : max(1, (int)(((long long)T * P.H + kN - 1) / kN));
}

template <bool kQStat, int kN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(wtc::kThreads, 1)
    attn_weights_kernel(const __grid_constant__ CUtensorMap tmQ,
                        const __grid_constant__ CUtensorMap tmK, const WeightsParams P) {
  using namespace wtc;
  using S = Shape<kQStat, kN>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages];
  __shared__ __align__(8) uint64_t stat_full[9], stat_empty[9];   // per 64-column chunk
  __shared__ __align__(8) uint64_t s_full[4], s_free[4], drain;
  __shared__ __align__(16) float lse2_sh[2][kN];
  __shared__ __align__(16) int lim_sh[2][kN];
  __shared__ float red[2][128];
  __shared__ uint32_t odd_sh[2];           // refresh (from 1) whose rows were not all finite
  __shared__ long long sums[kThreads / 32], run_sh[3];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sStat = base, sRing = base + S::kStat;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);      // the leader's arrive with both CTAs' bytes
      mbar_init(smem_u32(&empty[s]), 1);     // MMA commit (both CTAs)
    }
    for (int c = 0; c < 9; ++c) {
      mbar_init(smem_u32(&stat_full[c]), 1);
      mbar_init(smem_u32(&stat_empty[c]), 1);
    }
    for (int b = 0; b < S::kBufs; ++b) {
      mbar_init(smem_u32(&s_full[b]), 1);    // MMA commit (both CTAs)
      mbar_init(smem_u32(&s_free[b]), 16);   // 8 epilogue warps x 2 CTAs
    }
    mbar_init(smem_u32(&drain), 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    odd_sh[0] = odd_sh[1] = 0;
    run_sh[0] = P.B;
    run_sh[1] = 0;
    run_sh[2] = 0;
  }
  if (warp == 1) {
    tmem_alloc<2>(smem_u32(&tmem_base_sh), kTmemCols);
    tmem_relinquish<2>();
  }

  pdl_wait();
  pdl_launch();

  // ---- this pair's run: first sequence, first tile, cost at its end ----
  constexpr int kOpen = kQStat ? kOpenPages : 0;
  bool wrong = false;
  long long mine = 0;
  int u_first = 0, c_first = 1;          // of the thread's first sequence
  for (int b = threadIdx.x; b < P.B; b += kThreads) {
    wrong |= chunk_bad(P.cu_q, b, P.total_q, P.max_q);
    int units;
    const int c = weights_units<kQStat, kN>(P, b, units);
    mine += (long long)units * c + (units > 0 ? kOpen : 0);
    if (b < kThreads) {
      u_first = units;
      c_first = c;
    }
    if (blockIdx.x == 0 && (P.seq_lens[b] < P.cu_q[b + 1] - P.cu_q[b] ||
                            P.seq_lens[b] > P.max_tokens || P.seq_lens[b] > P.stride))
      raise_flag(kFlagBounds);
  }
  if (__syncthreads_or(wrong)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_flag(kFlagBounds);
    mine = 0;
    wrong = true;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) sums[warp] = mine;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) total += sums[w];
  const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
  const long long lo = total * pair / pairs, hi = total * (pair + 1) / pairs;
  // units whose place in the whole lies in [lo, hi)
  if (hi > lo) {
    long long before = 0;
    for (int b0 = 0; b0 < P.B; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      int units = u_first, c = c_first;
      if (b0 > 0) {
        units = 0;
        if (b < P.B) c = weights_units<kQStat, kN>(P, b, units);
      }
      const long long x = (long long)units * c + (units > 0 ? kOpen : 0);
      long long inc = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      __syncthreads();
      if (lane == 31) sums[warp] = inc;
      __syncthreads();
      long long at = before + inc - x, all = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        at += w < warp ? sums[w] : 0;
        all += sums[w];
      }
      // the first unit at or past lo: in this sequence, or at the start of a
      // later one
      if (x > 0 && at <= lo && lo < at + x) {
        const long long t = (max(lo - at - kOpen, 0ll) + c - 1) / c;
        run_sh[0] = t < units ? b : b + 1;
        run_sh[1] = t < units ? t : 0;
        run_sh[2] = t < units ? at + kOpen + t * c : at + x;
      }
      before += all;
    }
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  volatile int* abort_p = &abort_flag;

  // Every role walks the same tiles: sequences from run_sh on, tiles in
  // order, until the cost reaches hi.
  struct Walk {
    int b, x, units;         // sequence, next unit, its units
    int T, L, q0, blocks;    // its queries, length, first query token, row blocks (0: no queries)
    int page, pages;         // this tile: first page, pages (1 .. 4)
    bool last;               // the last tile of this sequence in the run
    bool first;              // the run's first sequence: its start is in cost
    long long cost, hi;
  };
  // the next tile; false at the end of the run
  auto walk_next = [&](Walk& w) {
    while (w.cost < w.hi && w.b < P.B) {
      if (w.units < 0) {                       // a new sequence
        w.blocks = weights_units<kQStat, kN>(P, w.b, w.units);
        w.q0 = P.cu_q[w.b];
        w.T = P.cu_q[w.b + 1] - w.q0;
        w.L = P.seq_lens[w.b];
        if (w.T == 0) w.blocks = 0;
        if (!w.first && w.units > 0) w.cost += kOpen;
        w.first = false;
        if (w.cost >= w.hi) return false;
      }
      if (w.x < w.units) {
        if constexpr (kQStat) {
          w.page = w.x;
          w.pages = (int)min((long long)min(4, w.units - w.x), w.hi - w.cost);
          w.x += w.pages;
          w.cost += w.pages;
        } else {
          w.page = 4 * w.x;
          w.pages = min(4, (w.L + kPage - 1) / kPage - w.page);
          ++w.x;
          w.cost += max(1, w.blocks);
        }
        w.last = w.x >= w.units;
        return true;
      }
      ++w.b;
      w.x = 0;
      w.units = -1;
    }
    return false;
  };
  Walk w0;
  w0.b = (int)run_sh[0];
  w0.x = (int)run_sh[1];
  w0.units = -1;
  w0.cost = run_sh[2];
  w0.first = true;
  w0.hi = hi > lo ? hi : 0;
  // pool page of page i (0, 1) of this CTA's half of the tile; -1: the tile
  // ends before it, n_pages: its id lies outside the pool (the box reads zeros)
  auto page_at = [&](const Walk& w, int i) {
    const int k = 2 * (int)rank + i;
    if (k >= w.pages) return -1;
    const int pg = P.page_table[(long long)w.b * P.max_pages + w.page + k];
    if (pg < 0 || pg >= P.n_pages) {
      raise_flag(kFlagBounds);
      return P.n_pages;
    }
    return pg;
  };

  // this CTA's pages of a tile: kCps chunks from chunk c on.  The leader arms a
  // barrier with both CTAs' bytes; a page past the tile is not loaded (its
  // rows compute on what the buffer held).
  auto load_tile = [&](uint32_t dst, int c, int pg0, int pg1, uint32_t bar) {
    if (pg0 >= 0) tma_load_5d_pair(dst, &tmK, 0, 0, c, 0, pg0, bar);
    if (pg1 >= 0) tma_load_5d_pair(dst + S::kCps * 8192, &tmK, 0, 0, c, 0, pg1, bar);
  };

  if (warp == 0 && lane == 0) {
    // ==============  producer of the ring (both CTAs)  ==============
    const uint32_t lead_full0 = mapa_shared(smem_u32(&full[0]), 0);
    uint32_t it = 0;
    bool ok = true;
    // the next tile is looked up while this one loads: page ids take as long
    // as a box
    Walk next = w0;
    int npg0 = 0, npg1 = 0;
    bool more = walk_next(next);
    auto look = [&]() {
      if (kQStat && more && next.blocks > 0) {
        npg0 = page_at(next, 0);
        npg1 = page_at(next, 1);
      }
    };
    look();
    while (ok && more) {
      const Walk w = next;
      const int pg0 = npg0, pg1 = npg1;
      more = walk_next(next);
      look();
      const int steps = kQStat ? min(1, w.blocks) : w.blocks;
      for (int rb = 0; rb < steps && ok; ++rb)
        for (int c = 0; c < S::kSteps; ++c, ++it) {
          const int s = it % S::kStages;
          if (!mbar_wait(smem_u32(&empty[s]), ((it / S::kStages) & 1) ^ 1, abort_p, 41, it)) {
            ok = false;
            break;
          }
          const uint32_t fb = lead_full0 + 8 * s;
          if (rank == 0)
            mbar_expect_tx(smem_u32(&full[s]),
                           kQStat ? (uint32_t)w.pages * S::kCps * 8192 : 2 * S::kStage);
          if constexpr (kQStat)
            load_tile(sRing + s * S::kStage, S::kCps * c, pg0, pg1, fb);
          else
            tma_load_2d_pair(sRing + s * S::kStage, &tmQ, 64 * c,
                             w.q0 * P.H + rb * kN + (kN / 2) * (int)rank, fb);
        }
    }
    if (!ok && rank == 0)
      // leaving early: wait (bounded) for the copies already armed
      for (uint32_t i = it > (uint32_t)S::kStages ? it - S::kStages : 0u; i < it; ++i)
        mbar_wait_bounded(smem_u32(&full[i % S::kStages]), (i / S::kStages) & 1, kDrainNs);
  } else if (warp == 2 && lane == 0) {
    // =====  producer of the resident operand (both CTAs), chunk by chunk  =====
    // A chunk is reloaded once the last MMA on it completed, while the later
    // chunks are still in use.
    const uint32_t lead_stat0 = mapa_shared(smem_u32(&stat_full[0]), 0);
    uint32_t stats = 0;
    int armed = 0;                         // chunks of load `stats` under way
    bool ok = true;
    int loaded = -1;                       // sequence whose rows are resident
    Walk w = w0;
    while (ok && walk_next(w)) {
      if (w.blocks == 0 || (kQStat && loaded == w.b)) continue;
      int pg0 = 0, pg1 = 0;
      if constexpr (!kQStat) {
        pg0 = page_at(w, 0);
        pg1 = page_at(w, 1);
      }
      for (int c = 0; c < 9; ++c) {
        if (stats > 0 &&
            !mbar_wait(smem_u32(&stat_empty[c]), (stats - 1) & 1, abort_p, 40, stats)) {
          ok = false;
          break;
        }
        const uint32_t fb = lead_stat0 + 8 * c;
        if (rank == 0)
          mbar_expect_tx(smem_u32(&stat_full[c]),
                         kQStat ? 2 * (S::kStat / 9) : (uint32_t)w.pages * 8192);
        if constexpr (kQStat)
          tma_load_2d_pair(sStat + c * (S::kStat / 9), &tmQ, 64 * c,
                           w.q0 * P.H + (kN / 2) * (int)rank, fb);
        else
          load_tile(sStat + c * 16384, c, pg0, pg1, fb);
        ++armed;
      }
      if (ok) {
        ++stats;
        armed = 0;
      }
      loaded = w.b;
    }
    if (rank == 0 && *abort_p)
      for (int c = 0; c < 9; ++c)
        if (c < armed || stats > 0)
          mbar_wait_bounded(smem_u32(&stat_full[c]), (c < armed ? stats : stats - 1) & 1, kDrainNs);
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // =====================  MMA issuer (leader)  =====================
    const uint32_t idesc = idesc_bf16_f32(256, kN, false, false);
    const uint64_t stat_desc = sw128_desc(sStat, 16, 1024);
    // a page's box lands as [8 slot groups][kCps chunks][8 slots][128 B]
    const uint64_t ring_desc = sw128_desc(sRing, 16, 1024 * S::kCps);
    uint32_t it = 0, stats = 0, j = 0;
    bool ok = true;
    Walk w = w0;
    int loaded = -1;
    while (ok && walk_next(w)) {
      const int steps = kQStat ? min(1, w.blocks) : w.blocks;
      for (int rb = 0; rb < steps && ok; ++rb, ++j) {
        const bool fresh = kQStat ? loaded != w.b : rb == 0;       // just loaded
        const bool done = kQStat ? w.last : rb == steps - 1;       // reloaded next
        loaded = w.b;
        const int buf = j % S::kBufs;
        if (j >= (uint32_t)S::kBufs &&
            !mbar_wait(smem_u32(&s_free[buf]), (j / S::kBufs - 1) & 1, abort_p, 43, j)) {
          ok = false;
          break;
        }
        for (int k = 0; k < S::kSteps; ++k, ++it) {
          const int s = it % S::kStages;
          if (!mbar_wait(smem_u32(&full[s]), (it / S::kStages) & 1, abort_p, 44, it)) {
            ok = false;
            break;
          }
          auto issue = [&](int cc) {
            const int c = k * S::kCps + cc;
            const uint64_t st = stat_desc + (uint64_t)((c * (S::kStat / 9)) >> 4);
            const uint64_t ri = ring_desc + (uint64_t)((s * S::kStage + cc * 1024) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ss<2>(tmem + kN * buf, (kQStat ? ri : st) + 2 * kk,
                             (kQStat ? st : ri) + 2 * kk, idesc, (c | kk) ? 1u : 0u);
          };
          if (!fresh && !done) {
            tc_fence_after();
#pragma unroll
            for (int cc = 0; cc < S::kCps; ++cc) issue(cc);
          } else {
            for (int cc = 0; cc < S::kCps && ok; ++cc) {
              const int c = k * S::kCps + cc;
              ok = !fresh || mbar_wait(smem_u32(&stat_full[c]), stats & 1, abort_p, 42, stats);
              if (!ok) break;
              tc_fence_after();
              issue(cc);
              if (done) mma_commit_2_mc(smem_u32(&stat_empty[c]), 3);
            }
          }
          if (!ok) break;
          mma_commit_2_mc(smem_u32(&empty[s]), 3);
        }
        if (ok) mma_commit_2_mc(smem_u32(&s_full[buf]), 3);
        if (fresh) ++stats;
      }
    }
    if (!ok) {
      mma_commit_2_mc(smem_u32(&drain), 1);
      mbar_wait_bounded(smem_u32(&drain), 0, kDrainNs);
    }
  } else if (warp >= kEpiWarp0) {
    // =====================  epilogue (both CTAs)  =====================
    const int ew = warp - kEpiWarp0;
    const int quad = ew & 3, ch = ew >> 2;            // TMEM lane quadrant, column half
    const int tl = 32 * quad + lane;                  // token of this CTA = TMEM lane
    const int et = threadIdx.x - 32 * kEpiWarp0;      // 0 .. 255
    const uint32_t lane_addr = (uint32_t)(32 * quad) << 16;
    const uint32_t lead_free = mapa_shared(smem_u32(&s_free[0]), 0);
    uint32_t j = 0, refresh = 0, done = 0;
    int loaded = -1;
    // Every warp takes every barrier; a wait that gave up only marks the warp,
    // and the next barrier tells all of them to leave together.
    bool dead = false, leave = false;
    Walk w = w0;
    while (!leave && walk_next(w)) {
      const int k = 2 * (int)rank + (tl >> 6);           // page of the tile
      const int t = (w.page + k) * kPage + (tl & 63);
      const int steps = kQStat ? min(1, w.blocks) : w.blocks;
      const long long at = w.b * P.stride + t;
      const bool store = ch == 0 && k < w.pages && t < w.L;
      float acc = 0.f, old = 0.f;
      if (store && P.w_in != nullptr && P.keep != 0.f && t < w.L - w.T) old = P.w_in[at];
      // lse of row r = et (+ kEpiThreads) of a row block, in units of log2;
      // +inf for a row that gives nothing
      constexpr int kRowsMine = (kN + kEpiThreads - 1) / kEpiThreads;
      auto row_lse = [&](int rb, float (&v)[kRowsMine]) {
#pragma unroll
        for (int i = 0; i < kRowsMine; ++i) {
          const int r = rb * kN + et + i * kEpiThreads;
          v[i] = INFINITY;
          if (et + i * kEpiThreads < kN && r < w.T * P.H) {
            const float x = P.lse[(long long)w.q0 * P.H + r];
            if (x != -INFINITY) v[i] = x * 1.4426950408889634f;
          }
        }
      };
      float next[kRowsMine];
      if (steps > 0 && (!kQStat || loaded != w.b)) row_lse(0, next);
      for (int rb = 0; rb < steps; ++rb, ++j) {
        // the rows' lse and visible limits.  Two sets in turn: the barrier of
        // the next refresh keeps a set from being rewritten while it is read.
        // The next row block's are on their way meanwhile.
        if (!kQStat || loaded != w.b) {
#pragma unroll
          for (int i = 0; i < kRowsMine; ++i) {
            const int r = et + i * kEpiThreads;
            if (r >= kN) break;
            lse2_sh[refresh & 1][r] = next[i];
            lim_sh[refresh & 1][r] = w.L - w.T + (rb * kN + r) / P.H + 1;
            if (!(next[i] < INFINITY)) odd_sh[refresh & 1] = refresh + 1;
          }
          ++refresh;
          loaded = w.b;
          leave = named_bar_or(1, kEpiThreads, dead || *abort_p != 0);
          if (leave) break;
          if (rb + 1 < steps) row_lse(rb + 1, next);
        }
        const float* l2 = lse2_sh[(refresh - 1) & 1] + (kN / 2) * ch;
        const int* lim = lim_sh[(refresh - 1) & 1] + (kN / 2) * ch;
        // every row counts and sees the whole tile (the block's first row sees
        // the least)
        const bool plain = odd_sh[(refresh - 1) & 1] != refresh &&
                           (w.page + w.pages) * kPage <= w.L - w.T + rb * kN / P.H + 1;
        const int buf = j % S::kBufs;
        const bool got = mbar_wait(smem_u32(&s_full[buf]), (j / S::kBufs) & 1, abort_p, 45, j);
        if (!__all_sync(0xffffffffu, got)) {
          dead = true;
          continue;
        }
        tc_fence_after();
        const uint32_t sa = tmem + lane_addr + kN * buf + (kN / 2) * ch;
        float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int g = 0; g < kN / 64; ++g) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld32(sa + 32 * g, r);
          tmem_wait_ld();
          if (plain) {
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float4 l = *reinterpret_cast<const float4*>(l2 + 32 * g + c);
              s4[0] += ex2_approx(fmaf(__uint_as_float(r[c]), P.scale_log2, -l.x));
              s4[1] += ex2_approx(fmaf(__uint_as_float(r[c + 1]), P.scale_log2, -l.y));
              s4[2] += ex2_approx(fmaf(__uint_as_float(r[c + 2]), P.scale_log2, -l.z));
              s4[3] += ex2_approx(fmaf(__uint_as_float(r[c + 3]), P.scale_log2, -l.w));
            }
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const float l = l2[32 * g + c];
              const float p = ex2_approx(fmaf(__uint_as_float(r[c]), P.scale_log2, -l));
              s4[c & 3] += t < lim[32 * g + c] && l != INFINITY ? p : 0.f;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead_free + 8 * buf);
        acc += (s4[0] + s4[1]) + (s4[2] + s4[3]);
      }
      if (leave) break;
      // the two column halves meet; one thread per token stores
      if (ch == 1) red[done & 1][tl] = acc;
      leave = named_bar_or(2, kEpiThreads, dead || *abort_p != 0);
      if (leave) break;
      if (store) P.w_out[at] = fmaf(P.keep, old, acc + red[done & 1][tl]);
      ++done;
    }
  }

  // =====================  teardown  =====================
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) tmem_dealloc<2>(tmem, kTmemCols);
}

template <bool kQStat, int kN>
inline mla_status launch_weights(bool (*make_tmap)(CUtensorMap*, const void*, int, const uint64_t*,
                                                   const uint64_t*, const uint32_t*),
                                 const void* qbuf, long long rows, const void* pool,
                                 const WeightsParams& p, int pairs, cudaStream_t st) {
  using namespace wtc;
  CUtensorMap tQ, tK;
  {
    const uint64_t dims[2] = {(uint64_t)kD, (uint64_t)rows};
    const uint64_t strides[1] = {(uint64_t)kD * 2};
    const uint32_t box[2] = {64, kN / 2};
    if (!make_tmap(&tQ, qbuf, 2, dims, strides, box)) return MLA_ERR_CUDA;
  }
  // the pool as (64 columns, 8 slots, 9 chunks, 8 slot groups, pages), as the
  // decode reads it: a box is kCps chunks of one page
  {
    const uint64_t dims[5] = {64, 8, 9, 8, (uint64_t)p.n_pages};
    const uint64_t strides[4] = {(uint64_t)kD * 2, 128, (uint64_t)kD * 2 * 8,
                                 (uint64_t)kPage * kD * 2};
    const uint32_t box[5] = {64, 8, (uint32_t)Shape<kQStat, kN>::kCps, 8, 1};
    if (!make_tmap(&tK, pool, 5, dims, strides, box)) return MLA_ERR_CUDA;
  }
  auto kfn = attn_weights_kernel<kQStat, kN>;
  constexpr uint32_t smem = Shape<kQStat, kN>::kSmem;
  if (cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
      cudaSuccess)
    return MLA_ERR_CUDA;
  return launch_pdl(kfn, dim3(2 * pairs), kThreads, smem, st, tQ, tK, p) == cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}

}  // namespace mla
