// kd_swa.cu -- sliding-window attention with first tokens kept, on CUDA cores
// for fp32 tensors, and the passes around the products that the tensor-core
// path for bf16 (kd_swa_tc.cu) shares.
//
// Query t sees key j when j <= t and (t - j < W or j < S).
//   forward   x = scale q k^T over the visible keys, one pass with the running
//             maximum and sum; o = sum p v, lse = max + log sum
//   backward  p = exp(x - lse), delta = dO.o, dS = p (dO v^T - delta):
//             dq = scale dS k,  dk = scale dS^T q,  dv = p^T dO
//
// 64 queries x 64 keys at a time from shared memory, 256 threads with 4 x 4
// tiles of the products; bound by shared-memory loads and fp32 FMA (at d = 128
// 65 and 69% of the L1's rate, 56 and 57% of the issue slots, with one CTA per SM
// that does not load while it computes).  B2 T4096 H8 window 512, in ms: forward
// 0.65, 0.35, 0.22 and backward 2.0, 0.98, 0.58 for d = 128, 64, 32 (25 and 29
// TFLOP/s at d = 128).  Tiles with no visible pair
// are not visited.  The gradients recompute p from lse, dk and dv by key tile
// and dq by query tile, so that
// every sum has a fixed order and needs no atomics.
#include "kd_hybrid.h"
#include "kd_rows.cuh"

namespace kd {

namespace {

constexpr int kB = 64;  // queries and keys of a tile
constexpr int kThreads = 256;
constexpr int kPitch = kB + 4;  // of a row of weights: 16-byte aligned
constexpr float kLog2e = 1.44269504088896f;

__device__ __forceinline__ float* floats(char* ws, size_t off) { return reinterpret_cast<float*>(ws + off); }

__device__ __forceinline__ bool visible(int t, int j, int W, int S) { return j <= t && (t - j < W || j < S); }

// Queries whose only key is their own: p = 1 whatever the scores, so dS is
// exactly 0 (computed, it would be the difference of two equal roundings).
__device__ __forceinline__ bool single_key(int t, int W, int S) { return t == 0 || (W == 1 && S == 0); }

// Rows t0 .. t0 + 63 of head h of a [B,T,H,D] tensor into [64][D + 4] fp32;
// rows at or behind T become zero.
template <int D>
__device__ __forceinline__ void load_tile(float* dst, const float* src, int t0, int T_, int H, int h, size_t b) {
  for (int i = threadIdx.x; i < kB * (D / 4); i += kThreads) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4, t = t0 + r;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < T_) v = *reinterpret_cast<const float4*>(src + ((b * T_ + t) * (size_t)H + h) * D + c);
    *reinterpret_cast<float4*>(dst + r * (D + 4) + c) = v;
  }
}

// acc[i][j] = A[ra + 16 i] . B[rb + 16 j]
template <int D>
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int ra, int rb, float (&acc)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(A + (ra + 16 * i) * (D + 4) + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(B + (rb + 16 * j) * (D + 4) + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = fmaf(a[i].x, b[j].x, acc[i][j]);
        acc[i][j] = fmaf(a[i].y, b[j].y, acc[i][j]);
        acc[i][j] = fmaf(a[i].z, b[j].z, acc[i][j]);
        acc[i][j] = fmaf(a[i].w, b[j].w, acc[i][j]);
      }
  }
}

// The D / 16 columns of thread tx: vectors of E consecutive ones, 16 E apart.
template <int D>
struct Cols {
  static constexpr int N = D / 16, E = N < 4 ? N : 4;
  static __device__ __forceinline__ int at(int tx, int n) { return n / E * 16 * E + tx * E + n % E; }
};

// acc[i][n] += sum_r Wt[ra + 16 i][r] X[r][column n of tx], four r at a time:
// a row of weights and a row of X are one vector access each.
template <int D>
__device__ __forceinline__ void mix_tile(const float* Wt, const float* X, int ra, int tx, float (&acc)[4][D / 16]) {
  using C = Cols<D>;
  using V = Pack<float, C::E>;
#pragma unroll 2
  for (int r = 0; r < kB; r += 4) {
    float4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(Wt + (ra + 16 * i) * kPitch + r);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int n = 0; n < C::N; n += C::E) {
        const V x = *reinterpret_cast<const V*>(X + (r + k) * (D + 4) + C::at(tx, n));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = k == 0 ? w[i].x : k == 1 ? w[i].y : k == 2 ? w[i].z : w[i].w;
#pragma unroll
          for (int e = 0; e < C::E; ++e) acc[i][n + e] = fmaf(f, x.x[e], acc[i][n + e]);
        }
      }
  }
}

// This thread's columns of a row.
template <int D>
__device__ __forceinline__ void store_cols(float* row, int tx, const float (&v)[D / 16]) {
  using C = Cols<D>;
#pragma unroll
  for (int n = 0; n < C::N; n += C::E) {
    float p[C::E];
#pragma unroll
    for (int e = 0; e < C::E; ++e) p[e] = v[n + e];
    store_row<float, C::E>(row + C::at(tx, n), p);
  }
}

__device__ __forceinline__ float max16(float x) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// The key tiles of query rows q0 .. q1 - 1: those of the first tokens, then
// those of the band.  tile(i) for i in [0, count).
struct KeyTiles {
  int first, band, count;
  __device__ KeyTiles(int q0, int q1, int W, int S, int B) {
    const int lo = q0 - W + 1 > 0 ? q0 - W + 1 : 0;
    band = lo / B;
    const int s = (S + B - 1) / B;
    first = s < band ? s : band;
    count = first + (q1 - 1) / B - band + 1;
  }
  __device__ int tile(int i) const { return i < first ? i : band + i - first; }
};

template <int D>
__global__ void __launch_bounds__(kThreads) swa_fwd_kernel(SwaArgs a) {
  extern __shared__ __align__(16) float sm[];
  float *Q = sm, *K = Q + kB * (D + 4), *V = K + kB * (D + 4), *Pt = V + kB * (D + 4);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int q0 = blockIdx.x * kB, h = blockIdx.y, hk = h / (a.H / a.Hk);
  const size_t b = blockIdx.z;
  const int q1 = q0 + kB < a.T ? q0 + kB : a.T;
  load_tile<D>(Q, static_cast<const float*>(a.q), q0, a.T, a.H, h, b);
  float o[4][D / 16], top[4], sum[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    top[i] = -INFINITY;
    sum[i] = 0.f;
#pragma unroll
    for (int jj = 0; jj < D / 16; ++jj) o[i][jj] = 0.f;
  }
  const float s2 = a.scale * kLog2e;
  const KeyTiles kt(q0, q1, a.window, a.sinks, kB);
  for (int n = 0; n < kt.count; ++n) {
    const int k0 = kt.tile(n) * kB;
    __syncthreads();
    load_tile<D>(K, static_cast<const float*>(a.k), k0, a.T, a.Hk, hk, b);
    load_tile<D>(V, static_cast<const float*>(a.v), k0, a.T, a.Hk, hk, b);
    __syncthreads();
    float x[4][4];
    dot_tile<D>(Q, K, ty, tx, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = q0 + ty + 16 * i;
      float m = top[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[i][j] = visible(t, k0 + tx + 16 * j, a.window, a.sinks) ? x[i][j] * s2 : -INFINITY;
        m = fmaxf(m, x[i][j]);
      }
      m = max16(m);
      // a row that has seen no key yet keeps m = -inf; its factors are 0, not NaN
      const float ms = m == -INFINITY ? 0.f : m;
      const float f = exp2f(top[i] - ms);
      float p = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = exp2f(x[i][j] - ms);
        Pt[(ty + 16 * i) * kPitch + tx + 16 * j] = e;
        p += e;
      }
      top[i] = m;
      sum[i] = fmaf(sum[i], f, p);
#pragma unroll
      for (int jj = 0; jj < D / 16; ++jj) o[i][jj] *= f;
    }
    __syncwarp();  // a row of Pt is written and read by the 16 lanes of one ty
    mix_tile<D>(Pt, V, ty, tx, o);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = q0 + ty + 16 * i;
    const float l = group_sum<16>(sum[i]);
    if (t >= a.T) continue;
    const size_t row = (b * a.T + t) * (size_t)a.H + h;
    const float r = 1.f / l;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) o[i][n] *= r;
    store_cols<D>(static_cast<float*>(a.out) + row * D, tx, o[i]);
    if (tx == 0) a.lse[row] = (top[i] + log2f(l)) * 0.693147180559945f;
  }
}

// p and dS of a 64 x 64 tile of queries q0.. (index r of the score tile along
// `kt` = keys or queries) in shared memory, row-major by the tile's rows.
// kKeyRows: rows are keys, columns queries.
template <bool kKeyRows>
__device__ __forceinline__ void weights(float (&x)[4][4], float (&dp)[4][4], const float* lse2, const float* delta,
                                        int q0, int k0, int T_, int W, int S, float s2, float* Pt, float* Dt) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int qi = kKeyRows ? tx + 16 * j : ty + 16 * i, t = q0 + qi;
      const int key = k0 + (kKeyRows ? ty + 16 * i : tx + 16 * j);
      const bool see = t < T_ && visible(t, key, W, S);
      const float p = see ? exp2f(fmaf(x[i][j], s2, -lse2[qi])) : 0.f;
      const float ds = single_key(t, W, S) ? 0.f : p * (dp[i][j] - delta[qi]);
      const int at = (ty + 16 * i) * kPitch + tx + 16 * j;
      if (Pt) Pt[at] = p;
      Dt[at] = ds;
    }
}

// dk, dv of key tile `tile` from its band's queries, all query heads of key
// head h0 / group (piece < 0); or of a tile of first tokens from piece `piece`
// of the queries beyond its band, query head h0.
template <int D>
__device__ __forceinline__ void dkv_item(const SwaArgs& a, const SwaBwdLayout& L, float* sm, int tile, int piece, int h0,
                                         size_t b, bool has_far) {
  float *Q = sm, *K = Q + kB * (D + 4), *V = K + kB * (D + 4), *G = V + kB * (D + 4);
  float *Pt = G + kB * (D + 4), *Dt = Pt + kB * kPitch, *lse2 = Dt + kB * kPitch, *delta = lse2 + kB;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, group = a.H / a.Hk;
  const bool far = piece >= 0;
  const int k0 = tile * kB, h1 = far ? h0 + 1 : h0 + group;
  const int band_end = (long long)k0 + kB - 1 + a.window < a.T ? k0 + kB - 1 + a.window : a.T;
  int q_lo = k0, q_hi = band_end;
  if (far) {
    q_lo = piece * kSwaPiece > band_end ? piece * kSwaPiece : band_end;
    q_hi = (piece + 1) * kSwaPiece < a.T ? (piece + 1) * kSwaPiece : a.T;
    if (q_lo >= q_hi) return;  // the sum skips it too
  }
  const int hk = h0 / group;
  load_tile<D>(K, static_cast<const float*>(a.k), k0, a.T, a.Hk, hk, b);
  load_tile<D>(V, static_cast<const float*>(a.v), k0, a.T, a.Hk, hk, b);
  float dk[4][D / 16], dv[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int jj = 0; jj < D / 16; ++jj) dk[i][jj] = dv[i][jj] = 0.f;
  for (int h = h0; h < h1; ++h) {
    const float* gl = floats(a.ws, L.lse2) + (b * a.H + h) * L.Tp;
    const float* gd = floats(a.ws, L.delta) + (b * a.H + h) * L.Tp;
    for (int q0 = q_lo / kB * kB; q0 < q_hi; q0 += kB) {
      __syncthreads();
      load_tile<D>(Q, static_cast<const float*>(a.q), q0, a.T, a.H, h, b);
      load_tile<D>(G, static_cast<const float*>(a.dO), q0, a.T, a.H, h, b);
      if (threadIdx.x < kB) {
        // queries outside [q_lo, q_hi) belong to another item: p = 0
        const int t = q0 + threadIdx.x;
        lse2[threadIdx.x] = t >= q_lo && t < q_hi ? gl[t] : INFINITY;
        delta[threadIdx.x] = gd[t];
      }
      __syncthreads();
      float x[4][4], dp[4][4];
      dot_tile<D>(K, Q, ty, tx, x);
      dot_tile<D>(V, G, ty, tx, dp);
      weights<true>(x, dp, lse2, delta, q0, k0, a.T, a.window, a.sinks, a.scale * kLog2e, Pt, Dt);
      __syncwarp();
      mix_tile<D>(Pt, G, ty, tx, dv);
      mix_tile<D>(Dt, Q, ty, tx, dk);
    }
  }
  const size_t part = (size_t)L.pieces * a.B * a.H * a.sinks * D, band = (size_t)a.B * a.Hk * a.sinks * D;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = k0 + ty + 16 * i;
    if (j >= a.T) continue;
    float *pk = nullptr, *pv = nullptr;
    if (far) {
      if (j >= a.sinks) continue;
      pk = floats(a.ws, L.part) + ((((size_t)piece * a.B + b) * a.H + h0) * a.sinks + j) * D;
      pv = pk + part;
    } else if (has_far && j < a.sinks) {
      pk = floats(a.ws, L.band) + ((b * a.Hk + hk) * a.sinks + j) * D;
      pv = pk + band;
    }
    const size_t row = ((b * a.T + j) * (size_t)a.Hk + hk) * D;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) dk[i][n] *= a.scale;
    if (pk) {
      store_cols<D>(pk, tx, dk[i]);
      store_cols<D>(pv, tx, dv[i]);
    } else {
      store_cols<D>(static_cast<float*>(a.dk) + row, tx, dk[i]);
      store_cols<D>(static_cast<float*>(a.dv) + row, tx, dv[i]);
    }
  }
}

// dq of query tile `tile`, head h.
template <int D>
__device__ __forceinline__ void dq_item(const SwaArgs& a, const SwaBwdLayout& L, float* sm, int tile, int h, size_t b) {
  float *Q = sm, *K = Q + kB * (D + 4), *V = K + kB * (D + 4), *G = V + kB * (D + 4);
  float *Dt = G + kB * (D + 4), *lse2 = Dt + kB * kPitch, *delta = lse2 + kB;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int q0 = tile * kB, hk = h / (a.H / a.Hk);
  const int q1 = q0 + kB < a.T ? q0 + kB : a.T;
  load_tile<D>(Q, static_cast<const float*>(a.q), q0, a.T, a.H, h, b);
  load_tile<D>(G, static_cast<const float*>(a.dO), q0, a.T, a.H, h, b);
  if (threadIdx.x < kB) {
    const size_t at = (b * a.H + h) * L.Tp + q0 + threadIdx.x;
    lse2[threadIdx.x] = floats(a.ws, L.lse2)[at];
    delta[threadIdx.x] = floats(a.ws, L.delta)[at];
  }
  float dq[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int jj = 0; jj < D / 16; ++jj) dq[i][jj] = 0.f;
  const KeyTiles kt(q0, q1, a.window, a.sinks, kB);
  for (int n = 0; n < kt.count; ++n) {
    const int k0 = kt.tile(n) * kB;
    __syncthreads();
    load_tile<D>(K, static_cast<const float*>(a.k), k0, a.T, a.Hk, hk, b);
    load_tile<D>(V, static_cast<const float*>(a.v), k0, a.T, a.Hk, hk, b);
    __syncthreads();
    float x[4][4], dp[4][4];
    dot_tile<D>(Q, K, ty, tx, x);
    dot_tile<D>(G, V, ty, tx, dp);
    weights<false>(x, dp, lse2, delta, q0, k0, a.T, a.window, a.sinks, a.scale * kLog2e, nullptr, Dt);
    __syncwarp();
    mix_tile<D>(Dt, K, ty, tx, dq);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = q0 + ty + 16 * i;
    if (t >= a.T) continue;
    const size_t row = ((b * a.T + t) * (size_t)a.H + h) * D;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) dq[i][n] *= a.scale;
    store_cols<D>(static_cast<float*>(a.dq) + row, tx, dq[i]);
  }
}

// One launch for all of them: the key tiles, the first tokens' far pieces (far
// items of `far_tiles` tiles) and the query tiles.
template <int D>
__global__ void __launch_bounds__(kThreads) swa_bwd_kernel(SwaArgs a, SwaBwdLayout L, int tiles, int far_tiles,
                                                           int key_items, int far_items) {
  extern __shared__ __align__(16) float sm[];
  int i = blockIdx.x;
  if (i < key_items) {
    const int kb = i / tiles;
    dkv_item<D>(a, L, sm, i % tiles, -1, kb % a.Hk * (a.H / a.Hk), kb / a.Hk, far_tiles > 0);
    return;
  }
  i -= key_items;
  if (i < far_items) {
    const int per = L.pieces * far_tiles, hb = i / per;
    dkv_item<D>(a, L, sm, i % far_tiles, i % per / far_tiles, hb % a.H, hb / a.H, true);
    return;
  }
  i -= far_items;
  const int hb = i / tiles;
  dq_item<D>(a, L, sm, i % tiles, hb % a.H, hb / a.H);
}

// HBM-bound: 39 us at T16384 H16 d128 bf16 (201 MB, 5.2 TB/s).
// delta = dO . o (o with its rounding added back) and lse in base 2, by head:
// 32 tokens of one head per CTA, four per warp.
template <typename T, int D>
__global__ void __launch_bounds__(256) swa_delta_kernel(SwaArgs a, SwaBwdLayout L) {
  constexpr int E = D / 32;
  __shared__ float sd[32], sl[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y;
  const size_t b = blockIdx.z;
  const int t0 = blockIdx.x * 32;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + warp * 4 + i;
    float dot = 0.f, l = INFINITY;
    if (t < a.T) {
      const size_t row = (b * a.T + t) * (size_t)a.H + h, at = row * D + lane * E;
      float g[E], o[E];
      load_stream<T, E>(static_cast<const T*>(a.dO) + at, g);
      load_stream<T, E>(static_cast<const T*>(a.o) + at, o);
      if (a.olo_in) {
        float lo[E];
        load_stream<T, E>(static_cast<const T*>(a.olo_in) + at, lo);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += lo[e];
      }
#pragma unroll
      for (int e = 0; e < E; ++e) dot = fmaf(g[e], o[e], dot);
      l = a.lse_in[row] * kLog2e;
    }
    dot = warp_sum(dot);
    if (lane == 0) {
      sd[warp * 4 + i] = dot;
      sl[warp * 4 + i] = l;
    }
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const size_t at = (b * a.H + h) * L.Tp + t0 + threadIdx.x;
    floats(a.ws, L.delta)[at] = sd[threadIdx.x];
    floats(a.ws, L.lse2)[at] = sl[threadIdx.x];
  }
}

// dk, dv of the first tokens: the band's part and the far pieces of every
// query head of the group, in that order, eight loads in flight.  Latency: 12 us
// for 4 first tokens at T16384 H16 Hk4 (25 with one load at a time).
template <typename T>
__global__ void __launch_bounds__(128) swa_sink_sum_kernel(SwaArgs a, SwaBwdLayout L, int tile) {
  const int c = threadIdx.x, j = blockIdx.x >> 1, which = blockIdx.x & 1, hk = blockIdx.y, b = blockIdx.z;
  const int group = a.H / a.Hk;
  if (c >= a.d || j >= a.T) return;
  const int band_end = j / tile * tile + tile - 1 + a.window;  // far queries start here (below 2^31: window <= T)
  const int first = band_end < a.T ? band_end / kSwaPiece : L.pieces;  // the pieces before it are empty
  const int far = L.pieces - first, n = group * far;
  const float* band = floats(a.ws, L.band) + (size_t)which * a.B * a.Hk * a.sinks * a.d;
  const float* part = floats(a.ws, L.part) + (size_t)which * L.pieces * a.B * a.H * a.sinks * a.d;
  float t = band[((size_t)(b * a.Hk + hk) * a.sinks + j) * a.d + c];
  for (int i = 0; i < n; i += 8) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int g = (i + u) / far, p = first + (i + u) - g * far;
      v[u] = i + u < n ? part[((((size_t)p * a.B + b) * a.H + hk * group + g) * a.sinks + j) * a.d + c] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) t += v[u];
  }
  T* dst = static_cast<T*>(which ? a.dv : a.dk);
  dst[(((size_t)b * a.T + j) * a.Hk + hk) * a.d + c] = from_f<T>(t);
}

template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int D>
cudaError_t fwd_go(const SwaArgs& a, cudaStream_t st) {
  const size_t smem = (3 * kB * (D + 4) + kB * kPitch) * sizeof(float);
  cudaError_t e = allow_smem(swa_fwd_kernel<D>, smem);
  if (e != cudaSuccess) return e;
  prof_begin(st, "swa_fwd_simt");
  swa_fwd_kernel<D><<<dim3((a.T + kB - 1) / kB, a.H, a.B), kThreads, smem, st>>>(a);
  prof_end(st);
  return cudaGetLastError();
}

template <int D>
cudaError_t bwd_go(const SwaArgs& a, cudaStream_t st) {
  const SwaBwdLayout L = swa_bwd_layout(a.B, a.T, a.H, a.Hk, a.d, a.window, a.sinks);
  const size_t smem = (4 * kB * (D + 4) + 2 * kB * kPitch + 2 * kB) * sizeof(float);
  cudaError_t e = allow_smem(swa_bwd_kernel<D>, smem);
  if (e == cudaSuccess) e = launch_swa_delta(a, L, st);
  if (e != cudaSuccess) return e;
  const int tiles = (a.T + kB - 1) / kB;
  const bool has_far = a.sinks > 0 && kB - 1 + a.window < a.T;
  const int far_tiles = has_far ? (a.sinks + kB - 1) / kB : 0;  // sinks <= T
  const long long key_items = (long long)tiles * a.Hk * a.B, far_items = (long long)L.pieces * far_tiles * a.H * a.B;
  const long long items = key_items + far_items + (long long)tiles * a.H * a.B;
  if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
  prof_begin(st, "swa_bwd_simt");
  swa_bwd_kernel<D><<<(unsigned)items, kThreads, smem, st>>>(a, L, tiles, far_tiles, (int)key_items, (int)far_items);
  prof_end(st);
  e = cudaGetLastError();
  if (e == cudaSuccess && has_far) e = launch_swa_sink_sum(a, L, kB, st);
  return e;
}

}  // namespace

SwaBwdLayout swa_bwd_layout(int B, int T, int H, int Hk, int d, int window, int sinks) {
  SwaBwdLayout L;
  size_t off = 0;
  auto take = [&](size_t floats) {
    const size_t o = off;
    off = (off + floats * 4 + 255) & ~size_t(255);
    return o;
  };
  L.Tp = (T + 127) / 128 * 128;
  L.pieces = (T + kSwaPiece - 1) / kSwaPiece;
  L.lse2 = take((size_t)B * H * L.Tp);
  L.delta = take((size_t)B * H * L.Tp);
  if (sinks > 0 && window < T) {
    L.part = take((size_t)2 * L.pieces * B * H * sinks * d);
    L.band = take((size_t)2 * B * Hk * sinks * d);
  }
  L.bytes = off;
  return L;
}

cudaError_t launch_swa_fwd_simt(const SwaArgs& a, cudaStream_t st) {
  return a.d == 32 ? fwd_go<32>(a, st) : a.d == 64 ? fwd_go<64>(a, st) : fwd_go<128>(a, st);
}

cudaError_t launch_swa_bwd_simt(const SwaArgs& a, cudaStream_t st) {
  return a.d == 32 ? bwd_go<32>(a, st) : a.d == 64 ? bwd_go<64>(a, st) : bwd_go<128>(a, st);
}

template <typename T>
static void delta_go(const SwaArgs& a, const SwaBwdLayout& L, cudaStream_t st) {
  const dim3 grid(L.Tp / 32, a.H, a.B);
  if (a.d == 32) swa_delta_kernel<T, 32><<<grid, 256, 0, st>>>(a, L);
  else if (a.d == 64) swa_delta_kernel<T, 64><<<grid, 256, 0, st>>>(a, L);
  else swa_delta_kernel<T, 128><<<grid, 256, 0, st>>>(a, L);
}

cudaError_t launch_swa_delta(const SwaArgs& a, const SwaBwdLayout& L, cudaStream_t st) {
  prof_begin(st, "swa_delta");
  if (a.dtype == 1) delta_go<__nv_bfloat16>(a, L, st);
  else delta_go<float>(a, L, st);
  prof_end(st);
  return cudaGetLastError();
}

cudaError_t launch_swa_sink_sum(const SwaArgs& a, const SwaBwdLayout& L, int tile, cudaStream_t st) {
  const dim3 grid(2 * a.sinks, a.Hk, a.B);
  prof_begin(st, "swa_sink_sum");
  if (a.dtype == 1) swa_sink_sum_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(a, L, tile);
  else swa_sink_sum_kernel<float><<<grid, 128, 0, st>>>(a, L, tile);
  prof_end(st);
  return cudaGetLastError();
}

}  // namespace kd
