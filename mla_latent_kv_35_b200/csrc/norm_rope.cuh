// norm_rope.cuh -- RMS norms of the query heads, the latent and the shared
// RoPE key, the position rotation and the cache append in one pass over the
// A0 rows.
//
// What it computes.  A row y[t] = [q_1 .. q_H | c | k_rope] as mla_project
// writes it holds H + 2 vectors that are normed each on its own,
//   n(x) = x / sqrt(mean_e x_e^2 + eps) * w        (w of the vector's width)
// over the d_nope + d_rope numbers of a head, the d_latent numbers of the
// latent and the d_rope numbers of the RoPE key; the last d_rope numbers of
// a head and the RoPE key are then turned by the position's angles.  The
// absorbed form scores against what is cached, so the key's norms are those
// of the cached parts: a norm of W_UK c would not commute with the
// absorption.  Sums of squares, the norm and the rotation are fp32; a value
// is rounded once, when it is stored.
//
// Bound: memory.  A row is read once and written once, ~6 operations per
// number; 4096 tokens of 128 heads (412 MB) take 66 us, 6.2 TB/s.  At DeepSeek-V2's widths (norm_rope_kernel):
//   * Eight lanes share a query head, so a warp holds four heads and a block
//     of eight warps 32; a lane keeps its 24 numbers in registers between the
//     sum and the store (16-byte pieces 8j + l of the head for lane l: every
//     load of the warp covers whole 128-byte lines).
//   * A block per (token, 32 heads): at one token 128 heads still spread over
//     four SMs; at many tokens 8 blocks per SM keep 96 KB in flight.
//   * The 32 angles of the token are formed one per lane while the loads are
//     in flight, from frequencies that the host passes in fp64: angle and
//     reduction to [-pi, pi] in fp64 (positions of 128K keep their phase),
//     then one fp32 sincos of the reduced angle (error 2^-23, below the
//     rounding of the products).  Lanes fetch the pairs they need by shuffle.
//   * Latent and RoPE key go one warp per token, in blocks of their own.
// Other widths, strides or alignments take norm_rope_any_kernel, a warp per
// vector that reads it twice.
#pragma once

#include "common.cuh"
#include "pre_attn.cuh"

namespace mla {

constexpr int kNormThreads = 256;
constexpr int kNormHeads = 32;       // query heads per block (8 warps x 4)
constexpr int kNormDN = 128, kNormDR = 64, kNormDC = 512;

struct NormRopeArgs {
  const void* y;          // [T][ys_tok]
  long long ys_tok;
  const void* w_q;        // [d_nope + d_rope], or nullptr: heads are not normed
  const void* w_c;        // [d_latent], or nullptr
  const void* w_kr;       // [d_rope], or nullptr
  const int32_t* pos;
  const int32_t* batch_idx;
  const int32_t* slot;
  const int32_t* page_table;
  void* pool;             // nullptr: no append
  void* q;                // [T][qs_tok], head i at i * (d_nope + d_rope)
  long long qs_tok;
  void* qbuf;             // [T][H][d_latent + d_rope], or nullptr: RoPE part stays with q
  void* ckr;              // [T][cs_tok], or nullptr
  long long cs_tok;
  int H, d_nope, d_rope, d_latent, n_seqs, max_pages, n_pages, page_size, T;
  float eps;
  double base;
  double freq[kNormDR / 2];   // base^(-2k/64), for norm_rope_kernel
};

// cos and sin of p * freq: angle and reduction in fp64, sincos in fp32 of an
// argument within [-pi, pi]
__device__ __forceinline__ void norm_cos_sin(double freq, int p, float& c, float& s) {
  const double ang = (double)p * freq;
  const double red = ang - 6.283185307179586476925286766559 *
                               rint(ang * 0.15915494309189533576888376337251);
  sincosf((float)red, &s, &c);
}

// Pool row of token t's slot, or nullptr (raising MLA_ERR_BOUNDS) when its
// sequence, slot or page lies outside the page table or pool.
template <typename T>
__device__ __forceinline__ T* norm_pool_row(const NormRopeArgs& a, int t, bool report) {
  if (a.batch_idx[t] >= a.n_seqs) {
    if (report) raise_flag(kFlagBounds);
    return nullptr;
  }
  return append_row(a.batch_idx, a.slot, t, a.page_table, a.max_pages, static_cast<T*>(a.pool),
                    a.n_pages, a.page_size, a.d_latent + a.d_rope, report);
}

template <typename T>
struct Piece;   // 16 bytes of T as floats
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[8]) {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Piece<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const __grid_constant__
                                                                 NormRopeArgs a) {
  constexpr int E = Piece<T>::E;
  constexpr int dqk = kNormDN + kNormDR, D = kNormDC + kNormDR;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (a.H + kNormHeads - 1) / kNormHeads;
  pdl_wait();
  pdl_launch();
  const long long q_blocks = (long long)a.T * groups;
  if ((long long)blockIdx.x < q_blocks) {
    // ---------------- query heads ----------------
    constexpr int NP = dqk / E / 8;          // pieces per lane
    constexpr int NN = kNormDN / E / 8;      // of which without rotation
    const int t = blockIdx.x / groups;
    const int head = (blockIdx.x % groups) * kNormHeads + 4 * warp + (lane >> 3);
    const int l = lane & 7;
    const bool live = head < a.H;
    uint4 v[NP];
    if (live) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(a.y) +
                                                        t * a.ys_tok + (long long)head * dqk);
#pragma unroll
      for (int j = 0; j < NP; ++j) v[j] = src[8 * j + l];
    } else {
#pragma unroll
      for (int j = 0; j < NP; ++j) v[j] = make_uint4(0, 0, 0, 0);
    }
    float c, s;
    norm_cos_sin(a.freq[lane], a.pos[t], c, s);
    float x[NP][E];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      Piece<T>::get(v[j], x[j]);
#pragma unroll
      for (int e = 0; e < E; ++e) ss = fmaf(x[j][e], x[j][e], ss);
    }
    ss += __shfl_xor_sync(0xffffffffu, ss, 1);
    ss += __shfl_xor_sync(0xffffffffu, ss, 2);
    ss += __shfl_xor_sync(0xffffffffu, ss, 4);
    if (a.w_q != nullptr) {
      const float r = rsqrtf(ss * (1.0f / dqk) + a.eps);
      const uint4* wp = static_cast<const uint4*>(a.w_q);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        float w[E];
        Piece<T>::get(wp[8 * j + l], w);
#pragma unroll
        for (int e = 0; e < E; ++e) x[j][e] = x[j][e] * r * w[e];
      }
    }
#pragma unroll
    for (int j = NN; j < NP; ++j)
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        // numbers (8(j - NN) + l) E + e, + 1 of the RoPE part: their pair
        const int k = ((8 * (j - NN) + l) * E + e) / 2;
        const float ck = __shfl_sync(0xffffffffu, c, k), sk = __shfl_sync(0xffffffffu, s, k);
        rope_rotate(x[j][e], x[j][e + 1], ck, sk, x[j][e], x[j][e + 1]);
      }
    if (!live) return;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.q) + t * a.qs_tok +
                                          (long long)head * dqk);
    uint4* rot = a.qbuf == nullptr
                     ? dst + kNormDN / E
                     : reinterpret_cast<uint4*>(static_cast<T*>(a.qbuf) +
                                                ((long long)t * a.H + head) * D + kNormDC);
#pragma unroll
    for (int j = 0; j < NN; ++j) dst[8 * j + l] = Piece<T>::put(x[j]);
#pragma unroll
    for (int j = NN; j < NP; ++j) rot[8 * (j - NN) + l] = Piece<T>::put(x[j]);
  } else {
    // ---------------- latent and RoPE key: a warp per token ----------------
    constexpr int NC = kNormDC / E / 32;
    const long long t = ((long long)blockIdx.x - q_blocks) * (kNormThreads / 32) + warp;
    if (t >= a.T) return;
    const T* row = static_cast<const T*>(a.y) + t * a.ys_tok + (long long)a.H * dqk;
    const uint4* src = reinterpret_cast<const uint4*>(row);
    uint4 v[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) v[j] = src[32 * j + lane];
    float k0 = to_f32(row[kNormDC + 2 * lane]), k1 = to_f32(row[kNormDC + 2 * lane + 1]);
    float c, s;
    norm_cos_sin(a.freq[lane], a.pos[t], c, s);
    float x[NC][E];
    float sc = 0.f, sk = fmaf(k0, k0, k1 * k1);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      Piece<T>::get(v[j], x[j]);
#pragma unroll
      for (int e = 0; e < E; ++e) sc = fmaf(x[j][e], x[j][e], sc);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sc += __shfl_xor_sync(0xffffffffu, sc, o);
      sk += __shfl_xor_sync(0xffffffffu, sk, o);
    }
    if (a.w_c != nullptr) {
      const float r = rsqrtf(sc * (1.0f / kNormDC) + a.eps);
      const uint4* wp = static_cast<const uint4*>(a.w_c);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        float w[E];
        Piece<T>::get(wp[32 * j + lane], w);
#pragma unroll
        for (int e = 0; e < E; ++e) x[j][e] = x[j][e] * r * w[e];
      }
    }
    if (a.w_kr != nullptr) {
      const float r = rsqrtf(sk * (1.0f / kNormDR) + a.eps);
      const T* wp = static_cast<const T*>(a.w_kr) + 2 * lane;
      k0 = k0 * r * to_f32(wp[0]);
      k1 = k1 * r * to_f32(wp[1]);
    }
    rope_rotate(k0, k1, c, s, k0, k1);
    T* out[2] = {nullptr, nullptr};
    if (a.pool != nullptr) out[0] = norm_pool_row<T>(a, (int)t, lane == 0);
    if (a.ckr != nullptr) out[1] = static_cast<T*>(a.ckr) + t * a.cs_tok;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (out[i] == nullptr) continue;
#pragma unroll
      for (int j = 0; j < NC; ++j)
        reinterpret_cast<uint4*>(out[i])[32 * j + lane] = Piece<T>::put(x[j]);
      if constexpr (E == 8)
        reinterpret_cast<uint32_t*>(out[i] + kNormDC)[lane] = pack_bf16x2(k0, k1);
      else
        reinterpret_cast<float2*>(out[i] + kNormDC)[lane] = make_float2(k0, k1);
    }
  }
}

// Any widths, strides and alignments: a warp per vector, which it reads
// twice.  Vectors 0 .. H - 1 of a token are its heads, H the latent, H + 1 the
// RoPE key.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_rope_any_kernel(const __grid_constant__
                                                                     NormRopeArgs a) {
  const int lane = threadIdx.x & 31;
  const long long i = (long long)blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5);
  const long long t = i / (a.H + 2);
  const int h = (int)(i % (a.H + 2));
  pdl_wait();
  pdl_launch();
  if (t >= a.T) return;
  const int dqk = a.d_nope + a.d_rope, D = a.d_latent + a.d_rope;
  const T* row = static_cast<const T*>(a.y) + t * a.ys_tok;
  const long long off = h <= a.H ? (long long)h * dqk : (long long)a.H * dqk + a.d_latent;
  const int plain = h < a.H ? a.d_nope : h == a.H ? a.d_latent : 0;
  const int turned = h == a.H ? 0 : a.d_rope;
  const T* x = row + off;
  const T* w = static_cast<const T*>(h < a.H ? a.w_q : h == a.H ? a.w_c : a.w_kr);
  float r = 1.f;
  if (w != nullptr) {
    float ss = 0.f;
    for (int e = lane; e < plain + turned; e += 32) ss = fmaf(to_f32(x[e]), to_f32(x[e]), ss);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    r = rsqrtf(ss / (float)(plain + turned) + a.eps);
  }
  auto normed = [&](int e) { return w != nullptr ? to_f32(x[e]) * r * to_f32(w[e]) : to_f32(x[e]); };
  T* out[2] = {nullptr, nullptr};   // places of the vector
  T* rot[2] = {nullptr, nullptr};   // places of its turned part
  if (h < a.H) {
    out[0] = static_cast<T*>(a.q) + t * a.qs_tok + (long long)h * dqk;
    rot[0] = a.qbuf == nullptr
                 ? out[0] + a.d_nope
                 : static_cast<T*>(a.qbuf) + (t * a.H + h) * (long long)D + a.d_latent;
  } else {
    const int o = h == a.H ? 0 : a.d_latent;
    if (a.pool != nullptr) {
      out[0] = norm_pool_row<T>(a, (int)t, lane == 0 && h == a.H);
      if (out[0] != nullptr) out[0] += o;
    }
    if (a.ckr != nullptr) out[1] = static_cast<T*>(a.ckr) + t * a.cs_tok + o;
    rot[0] = out[0];
    rot[1] = out[1];
  }
  // a number is read and written by one lane, so q and ckr may be y itself
  for (int e = lane; e < plain; e += 32) {
    const T v = from_f32<T>(normed(e));
    if (out[0] != nullptr) out[0][e] = v;
    if (out[1] != nullptr) out[1][e] = v;
  }
  for (int k = lane; k < turned / 2; k += 32) {
    float c, s, y0, y1;
    rope_cos_sin(k, a.pos[t], a.d_rope, a.base, c, s);
    rope_rotate(normed(plain + 2 * k), normed(plain + 2 * k + 1), c, s, y0, y1);
    for (int i2 = 0; i2 < 2; ++i2)
      if (rot[i2] != nullptr) {
        rot[i2][2 * k] = from_f32<T>(y0);
        rot[i2][2 * k + 1] = from_f32<T>(y1);
      }
  }
}

}  // namespace mla
