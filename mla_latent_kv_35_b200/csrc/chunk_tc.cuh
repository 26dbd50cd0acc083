// chunk_tc.cuh -- attention of ragged chunks of new tokens over the paged
// latent cache, with the absorbed query.
//
// What it computes: mla_decode's attention (scores over the 576 cached
// numbers, values the first 512) for chunks of any length: sequence b brings
// T_b query tokens, the last T_b of its L_b cached tokens, and query j sees
// tokens t <= L_b - T_b + j.  One launch covers decode tokens, speculative
// tokens and prompt tails of a mixed batch.  Against rebuilt per-head keys
// (prefill_tc.cuh) a query-token-head costs 1088 instead of 320
// multiply-adds, but nothing is rebuilt: 512 x 256 multiply-adds per
// (token, head), repaid from about 170 queries per sequence on.
//
// The tensor-core kernel is the decode's (decode_tc.cuh: pair MMAs, 128 query
// rows per cluster, 256-token blocks), over another list of virtual
// sequences.  Each chunk's T_b H rows are cut into blocks of 128; a block
// visits only the token blocks that its last row sees.  One worker per pair of
// SMs takes a run of token blocks.  Opening a row block costs a worker about
// kOpen token blocks of time (the last one's O leaves, a new Q comes, the
// pipeline refills).
//   * All blocks of all row blocks are laid end to end, kOpen more before each
//     row block, and split evenly: one long chunk among many short ones keeps
//     every SM busy, and short row blocks count what they cost (13 mixed
//     chunks: the worker with five one-block row blocks took 67 us, the median
//     43, when only the blocks counted).
//   * With at least as many workers as row blocks, every worker may serve one
//     row block instead: t is the least number with sum_v ceil(blocks_v / t)
//     <= workers, and row block v is split over ceil(blocks_v / t) of them.
//     Fewer row blocks are cut; the merge of cut ones costs about 2 blocks, so
//     this is taken up to 2 above the even share (16 x 4 queries over 4096
//     tokens: 18 against 15.6, 104 -> 92 us).
//   * A worker's pieces that cover their virtual sequence whole are final:
//     the epilogue writes bf16 rows and the LSE.  Only a worker's first and
//     last piece can be partial, so 2 slots per worker hold all partial
//     results (fp32), whatever the batch, and the merge (chunk_combine_kernel)
//     reads the few virtual sequences that a worker boundary cuts.
//   * o is stored in bf16: it is the W_UV product's input, and P is bf16.
//
// Bound: the tensor pipe and the loads that feed it.  128 rows meet each
// 576-number row of the cache, which comes through L2 as a key (1152 bytes) and
// again as a value (1024): 128 operations per byte.
#pragma once

#include "decode_tc.cuh"

namespace mla {

// Virtual sequences a batch can have: full blocks of 128 rows, and a partial
// one per sequence.
inline long long chunk_max_v(long long total_q, int B, int H) { return total_q * H / 128 + B; }

constexpr int kPlanThreads = 256;

// Block-wide exclusive prefix sum of one value per thread (kPlanThreads).
__device__ __forceinline__ int block_exclusive(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_sums[w] = inc;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kPlanThreads / 32; ++i) {
    const int y = warp_sums[i];
    before += i < w ? y : 0;
    all += y;
  }
  *total = all;
  __syncthreads();
  return before + inc - x;
}

// Whether cu_q breaks its rules at sequence b: ascending from 0 to at most
// total_q, no chunk longer than max_q.
__device__ __forceinline__ bool chunk_bad(const int32_t* cu_q, int b, int total_q, int max_q) {
  const int a = cu_q[b], z = cu_q[b + 1];
  return a < 0 || (b == 0 && a != 0) || z < a || z > total_q || z - a > max_q;
}

// Virtual sequences of the batch, sequence by sequence, and the prefix sums
// of their token blocks.  A cu_q that breaks its rules anywhere gives no
// blocks at all: chunks could overlap.  A sequence whose length is impossible
// keeps its rows with nothing to see (one empty block), so that they come out
// as 0 and -inf.  first: [B + 1], scratch for B > kPlanSeqs.  lo[k], k
// <= G: worker k's first block; worker_v[k]: its virtual sequence.  cuts[k], k < G - 1: the virtual sequence that the boundary between workers k and k + 1
// cuts (-1: none), with its first and last worker.
constexpr int kPlanSeqs = 2048;
constexpr int kOpen = 2;
struct ChunkCut {
  int v, k0, k1, pad;
};
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const int32_t* cu_q,
                                                          const int32_t* seq_lens, int B, int H,
                                                          int total_q, int max_q, int max_tokens,
                                                          int V, int G, int32_t* first_global,
                                                          VSeq* vseq, int32_t* start,
                                                          ChunkCut* cuts, int32_t* worker_v,
                                                          int32_t* lo) {
  __shared__ int warp_sums[kPlanThreads / 32];
  __shared__ int start_sh[kPlanSeqs];  // start, where it fits
  __shared__ int aligned;              // t of the aligned split, or 0
  __shared__ int first_sh[kPlanSeqs + 1];
  __shared__ int len_sh[kPlanThreads];
  pdl_wait();
  pdl_launch();
  int32_t* first = B <= kPlanSeqs ? first_sh : first_global;
  for (int k = threadIdx.x; k < G; k += kPlanThreads) cuts[k].v = -1;
  // (lengths of the first sequences come along with cu_q: one trip to memory)
  const int L_mine = threadIdx.x < B ? seq_lens[threadIdx.x] : 0;
  bool wrong = false;
  for (int b = threadIdx.x; b < B; b += kPlanThreads) wrong |= chunk_bad(cu_q, b, total_q, max_q);
  len_sh[threadIdx.x] = L_mine;
  if (__syncthreads_or(wrong)) {
    for (int v = threadIdx.x; v <= V; v += kPlanThreads) start[v] = 0;
    for (int k = threadIdx.x; k <= G; k += kPlanThreads) lo[k] = 0;
    if (threadIdx.x == 0) raise_flag(kFlagBounds);
    return;
  }
  int base = 0;
  for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    const int T = b < B ? cu_q[b + 1] - cu_q[b] : 0;
    int sum;
    const int off = block_exclusive((int)(((long long)T * H + 127) / 128), warp_sums, &sum);
    if (b < B) first[b] = base + off;
    base += sum;
  }
  if (threadIdx.x == 0) first[B] = base;
  __syncthreads();
  const int live = base;    // <= V, as the chunks do not overlap
  int blocks = 0;
  for (int v0 = 0; v0 < V; v0 += kPlanThreads) {
    const int v = v0 + threadIdx.x;
    int nb = 0;
    if (v < live) {
      const int b = seq_of_block(first, B, v);
      VSeq s;
      s.b = b;
      s.row0 = (v - first[b]) * 128;
      s.q0 = cu_q[b];
      s.T = cu_q[b + 1] - s.q0;
      s.L = b < kPlanThreads ? len_sh[b] : seq_lens[b];
      if (s.L < s.T || s.L > max_tokens) {
        if (s.row0 == 0) raise_flag(kFlagBounds);
        s.L = 0;
        nb = 1;
      } else {
        const int last = min(s.T - 1, (s.row0 + 127) / H);      // last query of the block
        nb = (s.L - s.T + last + 1 + dtc::kBlk - 1) / dtc::kBlk;
      }
      vseq[v] = s;
    }
    int sum;
    const int off = block_exclusive(nb, warp_sums, &sum);
    if (v < V) {
      start[v] = blocks + off;
      if (v < kPlanSeqs) start_sh[v] = blocks + off;
    }
    blocks += sum;
  }
  if (threadIdx.x == 0) {
    start[V] = blocks;
    if (V < kPlanSeqs) start_sh[V] = blocks;
  }
  __syncthreads();
  const int32_t* first_block = V < kPlanSeqs ? start_sh : start;
  if (blocks == 0) {                   // no queries
    for (int k = threadIdx.x; k <= G; k += kPlanThreads) lo[k] = 0;
    return;
  }
  // cost of everything, kOpen before each row block
  const long long cost = (long long)blocks + (long long)kOpen * live;
  constexpr int kMine = 4;             // row blocks per lane of the aligned split
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int t = 0;
    if (live <= min(G, 32 * kMine)) {
      // consecutive row blocks per lane, in registers
      int nb[kMine], most = 0;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int v = kMine * lane + i;
        nb[i] = v < live ? first_block[v + 1] - first_block[v] : 0;
        most = max(most, nb[i]);
      }
      most = __reduce_max_sync(0xffffffffu, most);
      int a = (blocks + G - 1) / G, z = most;      // the least t lies in [a, z]
      while (a < z) {
        const int mid = (a + z) >> 1;
        int m = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) m += (nb[i] + mid - 1) / mid;
        if ((int)__reduce_add_sync(0xffffffffu, m) <= G) z = mid; else a = mid + 1;
      }
      if (a + kOpen <= (cost + G - 1) / G + 2) t = a;
    }
    if (lane == 0) aligned = t;
  }
  __syncthreads();
  // quotients of 64 bits take a third of a microsecond each
  const bool small = cost < (1 << 24) && G < 255;           // 32 bits hold k cost
  auto quotient = [&](long long x, long long y) {
    return small ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
  };
  if (aligned > 0) {
    const int v = threadIdx.x;                   // live <= 128
    const int v0 = v < live ? first_block[v] : 0;
    const int nb = v < live ? first_block[v + 1] - v0 : 0;
    const int n = (nb + aligned - 1) / aligned;
    int used;
    const int k = block_exclusive(n, warp_sums, &used);
    for (int j = 0; j < n; ++j) {
      lo[k + j] = v0 + (int)quotient((long long)nb * j, n);
      worker_v[k + j] = v;
      if (j + 1 < n) cuts[k + j] = ChunkCut{v, k, k + n - 1, 0};
    }
    for (int j = used + threadIdx.x; j <= G; j += kPlanThreads) lo[j] = blocks;
    return;
  }
  // boundary k lies at floor(k cost / workers): in row block v's part [c0, c1),
  // at its start or kOpen blocks less into it
  const long long workers = min(G, blocks);
  for (int k = (int)workers + threadIdx.x; k <= G; k += kPlanThreads) lo[k] = blocks;
  for (int v = threadIdx.x; v < live; v += kPlanThreads) {
    const int v0 = first_block[v];
    const long long c0 = v0 + (long long)kOpen * v;
    const long long c1 = first_block[v + 1] + (long long)kOpen * (v + 1);
    int k0 = -1, k1 = -1;              // first and last worker of a row block that is cut
    for (long long k = quotient(c0 * workers + cost - 1, cost); k < workers; ++k) {
      const long long at = quotient(k * cost, workers);
      if (at >= c1) break;
      const int x = (int)max(at - c0 - kOpen, 0ll);
      lo[k] = v0 + x;
      worker_v[k] = v;
      if (x > 0) {
        if (k0 < 0) k0 = (int)k - 1;
        k1 = (int)k;
      }
    }
    for (int k = k0; k < k1; ++k) cuts[k] = ChunkCut{v, k0, k1, 0};
  }
}

// Merges the virtual sequences that worker boundaries cut, by log-sum-exp.  A
// virtual sequence cut into n pieces has n - 1 boundaries, each with 16
// blocks; its 128 rows go 8, 4, 2 or 1 to a block, so that few pieces use few
// blocks and many pieces (a long context with few queries) all of them.  The
// 8 / rows warps of a row take its pieces in turn and meet in shared memory;
// a lane owns four float4 columns.
__global__ void __launch_bounds__(256) chunk_combine_kernel(const float* ws_lse, const float* ws_o,
                                                            const ChunkCut* cuts, const VSeq* vseq,
                                                            int H, __nv_bfloat16* o, float* lse) {
  __shared__ float4 part[8][128];
  pdl_wait();
  pdl_launch();
  const ChunkCut c = cuts[blockIdx.x];
  if (c.v < 0) return;
  const int n = c.k1 - c.k0 + 1;
  const int blocks = 16 * (n - 1);
  const int rows = blocks >= 128 ? 1 : blocks >= 64 ? 2 : blocks >= 32 ? 4 : 8;
  const int first = ((int)(blockIdx.x - c.k0) * 16 + (int)blockIdx.y) * rows;
  if (first >= 128) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int wpr = 8 / rows, u = w % wpr;
  const int r = first + w / wpr;
  const VSeq s = vseq[c.v];
  const bool live = s.row0 + r < s.T * H;
  // piece i: worker k0 + i; the first opens the virtual sequence
  auto slot = [&](int i) { return (long long)(2 * (c.k0 + i) + (i == 0 ? 1 : 0)) * 128 + r; };
  float mx = -INFINITY;
  for (int i = lane; i < n; i += 32) mx = fmaxf(mx, ws_lse[slot(i)]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  // z: 0 where no piece saw anything, NaN where one had a NaN (which the
  // maximum passes over)
  const float m0 = mx == -INFINITY ? 0.f : mx;
  float z = 0.f;
  float4 acc[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = lane; i < n; i += 32) z += __expf(ws_lse[slot(i)] - m0);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
  if (z != 0.f && live) {
#pragma unroll 2
    for (int i = u; i < n; i += wpr) {
      const float e = __expf(ws_lse[slot(i)] - m0);
      const float4* src = reinterpret_cast<const float4*>(ws_o + slot(i) * dtc::kDC);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 x = src[32 * q + lane];
        acc[q].x = fmaf(e, x.x, acc[q].x);
        acc[q].y = fmaf(e, x.y, acc[q].y);
        acc[q].z = fmaf(e, x.z, acc[q].z);
        acc[q].w = fmaf(e, x.w, acc[q].w);
      }
    }
  }
  if (wpr > 1) {
    if (u != 0)
#pragma unroll
      for (int q = 0; q < 4; ++q) part[w][32 * q + lane] = acc[q];
    __syncthreads();
    if (u != 0) return;
    for (int t = 1; t < wpr; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 y = part[w + t][32 * q + lane];
        acc[q].x += y.x; acc[q].y += y.y; acc[q].z += y.z; acc[q].w += y.w;
      }
  }
  if (!live) return;
  const float inv = z != 0.f ? 1.f / z : 0.f;
  const long long row = (long long)s.q0 * H + s.row0 + r;
  uint2* dst = reinterpret_cast<uint2*>(o + row * dtc::kDC);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    dst[32 * q + lane] = make_uint2(pack_bf16x2(acc[q].x * inv, acc[q].y * inv),
                                    pack_bf16x2(acc[q].z * inv, acc[q].w * inv));
  if (lane == 0) lse[row] = z != 0.f ? m0 + logf(z) : -INFINITY;
}

struct ChunkLayout {
  long long V;
  int G;
  size_t off_first, off_vseq, off_cuts, off_wv, off_lo, off_lse, off_o, total;
};

inline ChunkLayout chunk_layout(long long total_q, int B, int H, int G) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  ChunkLayout c;
  c.V = chunk_max_v(total_q, B, H);
  c.G = G;
  c.off_first = up(sizeof(int32_t) * (c.V + 1));
  c.off_vseq = c.off_first + up(sizeof(int32_t) * ((size_t)B + 1));
  c.off_cuts = c.off_vseq + up(sizeof(VSeq) * c.V);
  c.off_wv = c.off_cuts + up(sizeof(ChunkCut) * G);
  c.off_lo = c.off_wv + up(sizeof(int32_t) * G);
  c.off_lse = c.off_lo + up(sizeof(int32_t) * (G + 1));
  c.off_o = c.off_lse + up(sizeof(float) * 2 * G * 128);
  c.total = c.off_o + sizeof(float) * 2 * G * 128 * dtc::kDC;
  return c;
}

inline mla_status launch_chunk_tc_impl(
    bool (*make_tmap)(CUtensorMap*, const void*, int, const uint64_t*, const uint64_t*,
                      const uint32_t*),
    const void* qbuf, const int32_t* cu_q, int total_q, int max_q, const void* pool, int n_pages,
    const int32_t* page_table, int max_pages, const int32_t* seq_lens, int B, int H, float scale,
    char* ws, const ChunkLayout& c, __nv_bfloat16* o, float* lse, cudaStream_t st) {
  using namespace dtc;
  int32_t* start = reinterpret_cast<int32_t*>(ws);
  int32_t* first = reinterpret_cast<int32_t*>(ws + c.off_first);
  VSeq* vseq = reinterpret_cast<VSeq*>(ws + c.off_vseq);
  ChunkCut* cuts = reinterpret_cast<ChunkCut*>(ws + c.off_cuts);
  int32_t* worker_v = reinterpret_cast<int32_t*>(ws + c.off_wv);
  int32_t* lo = reinterpret_cast<int32_t*>(ws + c.off_lo);
  float* ws_lse = reinterpret_cast<float*>(ws + c.off_lse);
  float* ws_o = reinterpret_cast<float*>(ws + c.off_o);
  CUtensorMap tQ, tQK, tPV;
  if (!decode_tc_tmaps(make_tmap, qbuf, (long long)total_q * H, pool, n_pages, tQ, tQK, tPV))
    return MLA_ERR_CUDA;
  if (cudaFuncSetAttribute(decode_tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kSmemBytes) != cudaSuccess)
    return MLA_ERR_CUDA;
  if (launch_pdl(chunk_plan_kernel, dim3(1), kPlanThreads, 0, st, cu_q, seq_lens, B, H, total_q,
                 max_q, max_pages * kPage, (int)c.V, c.G, first, vseq, start, cuts, worker_v,
                 lo) != cudaSuccess)
    return MLA_ERR_CUDA;
  DecodeTcParams p{};
  p.pool = static_cast<const uint8_t*>(pool);
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.start = start;
  p.ws_lse = ws_lse;
  p.ws_o = ws_o;
  p.n_pages = n_pages;
  p.max_pages = max_pages;
  p.B = B;
  p.H = H;
  p.G = c.G;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.vseq = vseq;
  p.worker_v = worker_v;
  p.worker_lo = lo;
  p.V = (int)c.V;
  p.o = o;
  p.lse = lse;
  if (launch_pdl(decode_tc_kernel<true>, dim3(2 * c.G), kThreads, kSmemBytes, st, tQ, tQK, tPV,
                 p) != cudaSuccess ||
      launch_pdl(chunk_combine_kernel, dim3(c.G, 16), 256, 0, st, ws_lse, ws_o, cuts, vseq, H, o,
                 lse) != cudaSuccess)
    return MLA_ERR_CUDA;
  return MLA_OK;
}

}  // namespace mla
