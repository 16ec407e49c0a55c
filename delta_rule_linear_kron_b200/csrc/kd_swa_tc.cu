// kd_swa_tc.cu -- sliding-window attention with first tokens kept, on tcgen05
// (bf16).  The formulas are in kd_swa.cu.  Kernels are made for d = 64 and 128;
// d = 32 is d = 64 whose tiles' second half lies outside the tensors: loaded as
// zeros, never stored (B2 T4096 H8 window 512: forward 44 and backward 99 us;
// on CUDA cores, which have no use for the zeros, 228 and 626).
//
// Times are at H16 Hk16 T16384 d128 window 2048, in us, of single calls at the
// full 1.965 GHz.  Calls back to back reach the power limit (1.67 GHz), where a
// training step with 4 first tokens takes 1,450 in place of 1,309: forward 363
// (317), delta 42 (39), backward 1,026 (899), first tokens' sums 9, and gaps.
//
// Every kernel has 19 warps: four groups of four (thread = TMEM lane = tile row,
// a part of its columns) for the elementwise work, which bounds these kernels
// (with half as many warps of twice the columns: dk and dv 685 in place of 530,
// dq 505 in place of 400, the forward 370 in place of 315), one thread that
// loads tiles by TMA into a ring, and two warps that issue MMAs, each the
// products of one chain (scores, then what is made of them), so that one chain's
// waits lie beside the other's products.  A whole warp issues, one lane elected:
// from a single thread, whose descriptors are no values of the warp, eight MMAs
// take up to 1,000 cycles to issue (backward 992 in place of 909). Tiles are 128
// x 128: an MMA of 128 x 64 x 16 takes 50 cycles where one of 128 x 128 x 16
// takes 68.  B operands of the second products (v, k, dO, q) are read MN-major
// from the same shared-memory tile that the score product reads K-major, so no
// tile is stored twice or transposed.
//
// Forward: 295, 0.87 PFLOP/s over the visible pairs.  256 queries of one head
// per CTA, a group to each 128.  Scores are read into registers at once and
// their TMEM columns given back for the next tile's, p goes to shared memory as
// the next product's A operand; per tile pair 32 MMAs (2,200 cycles) stand
// against 2,050 cycles of the hardware exponential, and 384 KB go through shared
// memory (3,070 cycles at 128 bytes), which is what bounds the 3,600 cycles that
// a pair takes.  The weights are made in registers before the wait for the
// product that still reads the last ones (319 where they follow it).  With p
// over the scores in TMEM, where a group waits for both products between two
// tiles, it took 410. The output stays in TMEM and is rescaled only when a row's
// maximum has grown by more than 2^8 over the one its sums refer to (then p <=
// 2^8, still exact enough in bf16, whose precision does not depend on the size).
//
// Backward: 852, 1.06 PFLOP/s over the visible pairs' seven products; bound by
// each tile's chain of waits, exponential and conversions (2,600 cycles for dq,
// 3,600 for dk, dv, against 1,750 and 2,500 of shared-memory traffic), and by 5
// us of start and end of each CTA.  p is recomputed from the saved lse.  dk, dv:
// 128 keys per CTA (rows are keys: S^T = k q^T, dP^T = v dO^T), 128 queries at a
// time; dv += P^T dO, dk += dS^T q. dq: 128 queries per CTA; dq += dS k.  The
// groups take the columns of each tile in parts; p is formed while dP is still
// being multiplied.  dS goes over dP (dq: over the scores, of which it has two
// buffers) in TMEM; dkv's p goes to shared memory, so that the next scores need
// not wait for dv.  (64-column tiles, two at a time, a group to each: dk and dv
// 880, dq 750.)  Seven products in place of the five of one joint pass, but no
// atomics and no fp32 copy of dq: every sum has one order.
#include "kd_hybrid.h"
#include "kd_rows.cuh"
#include "kd_tc.cuh"
#include "kd_tmap.h"

namespace kd {

namespace {

constexpr int kTcThreads = 608;
constexpr int kLoadWarp = 16, kMmaWarp = 17;  // and 18; 0-15 are the groups'
constexpr float kLog2e = 1.44269504088896f;
constexpr float kLn2 = 0.693147180559945f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ bool single_key(int t, int W, int S) { return t == 0 || (W == 1 && S == 0); }

// A wait that a whole warp gives up together (its TMEM loads need all lanes).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* err, int code, volatile int* ab) {
  return __all_sync(0xffffffffu, tc::mbar_wait<false>(bar, parity, err, code, ab));
}

__device__ __forceinline__ float bf16_pair(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return __uint_as_float(*reinterpret_cast<const uint32_t*>(&v));
}

// The key tiles of B keys that query rows q0 .. q1 - 1 see: those of the band,
// then those of the first tokens.  (With the first tokens first, the forward's
// two groups would both begin with them and go on in step: 350 in place of
// 310 us with 4 first tokens.)
struct KeyRange {
  int first, band, end, count;
  __device__ KeyRange(int q0, int q1, int W, int S, int B) {
    if (q0 >= q1) {
      first = count = 0;
      band = 1;
      end = 0;
      return;
    }
    band = (q0 - W + 1 > 0 ? q0 - W + 1 : 0) / B;
    end = (q1 - 1) / B;
    const int s = (S + B - 1) / B;
    first = s < band ? s : band;
    count = first + end - band + 1;
  }
  __device__ int tile(int i) const { return i < count - first ? band + i : i - (count - first); }
  __device__ bool has(int kt) const { return kt < first || (kt >= band && kt <= end); }
};

// Scores of N columns from column 0 on: visible are those below `end` that are
// at `begin` or later, or below `first` (first tokens).  `upper`, `lower`: which
// bounds the tile needs at all (one for the whole warp).
template <int N>
__device__ __forceinline__ void hide(float (&x)[N], bool upper, bool lower, int end, int begin, int first) {
  if (upper) {
#pragma unroll
    for (int c = 0; c < N; ++c) x[c] = c < end ? x[c] : -INFINITY;
  }
  if (lower) {
#pragma unroll
    for (int c = 0; c < N; ++c) x[c] = c >= begin || c < first ? x[c] : -INFINITY;
  }
}

// N fp32 values of this thread's TMEM lane, scaled, as bf16 into row r of a
// swizzled tile (column c0 on) for a TMA store; the rounding that is left over
// into the same place of `lo` where it is given.
template <int N>
__device__ __forceinline__ void stage_lane(uint32_t lanes, float scale, unsigned char* tile, unsigned char* lo, int r,
                                           int c0) {
#pragma unroll
  for (int c = 0; c < N; c += 16) {
    float v[16];
    tc::tmem_ld16(lanes + c, v);
    tc::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
      const int k = (c0 + c + i) / 8;  // 16-byte chunk of the row
      const uint32_t at = k / 8 * 16384 + r * 128 + ((k % 8) ^ (r & 7)) * 16;
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = v[i + e] * scale;
      store_row<__nv_bfloat16, 8>(reinterpret_cast<__nv_bfloat16*>(tile + at), w);
      if (lo) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] -= __bfloat162float(__float2bfloat16_rn(w[e]));
        store_row<__nv_bfloat16, 8>(reinterpret_cast<__nv_bfloat16*>(lo + at), w);
      }
    }
  }
}

// Tile of rows x 64-channel blocks by TMA (D / 64 boxes).
template <int D>
__device__ __forceinline__ void load_tile(unsigned char* dst, const CUtensorMap* m, int h, int t0, int b, uint64_t* bar) {
#pragma unroll
  for (int c = 0; c < D; c += 64) tc::tma_load_4d(dst + c * 256, m, c, h, t0, b, bar);
}

// The same the other way; rows behind T are not written.
template <int D>
__device__ __forceinline__ void store_tile(const unsigned char* src, const CUtensorMap* m, int h, int t0, int b) {
#pragma unroll
  for (int c = 0; c < D; c += 64) tc::tma_store_4d(m, src + c * 256, c, h, t0, b);
}

// D = A B^T of 128 x 128, K = d: both tiles of 128 rows, K-major.
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t id = tc::idesc(128, 128, 1);
  const uint64_t da = tc::desc_sw128(a), db = tc::desc_sw128(b);
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    const uint32_t o = s / 4 * 16384 + s % 4 * 32;
    tc::warp_mma_bf16_ss(d, tc::desc_at(da, o), tc::desc_at(db, o), id, s > 0);
  }
}

// D (+)= W X of 128 x d, K = 128: W in TMEM, group g's 32 weights in 16 columns
// at w + 32 g (their low parts in the 16 behind), X a tile of 128 rows read
// MN-major.
template <int D>
__device__ __forceinline__ void mma_mix(uint32_t d, uint32_t w, uint32_t x, bool acc) {
  constexpr uint32_t id = tc::idesc(128, D, 1) | tc::kMajorB;
  const uint64_t dx = tc::desc_sw128_mn(x, 16384u);
#pragma unroll
  for (int s = 0; s < 8; ++s)
    tc::warp_mma_bf16_ts(d, w + s / 2 * 32 + s % 2 * 8, tc::desc_at(dx, s * 2048), id, acc || s > 0);
}

// ---- forward -----------------------------------------------------------------

template <int D>
struct FwdCfg {
  static constexpr uint32_t TILE = 128 * D * 2;
  static constexpr int SLOTS = D == 128 ? 3 : 6;  // ring of key and value tiles
  static constexpr uint32_t P = 2 * TILE;         // behind the two query tiles: weights, 32 KB per group
  static constexpr uint32_t RING = P + 65536;
  static constexpr uint32_t HALF = RING + SLOTS * TILE;  // fp32 [query tile][half of the columns][row]
  static constexpr uint32_t BARS = HALF + 2048;
  static constexpr uint32_t BYTES = BARS + 256;   // no static shared memory: all 227 KB at d = 128
  static constexpr int S_COL = 0, O_COL = 256;    // 128 columns per query tile: scores; the output
};

struct FwdBars {
  uint64_t q_full[2], full[6], empty[6], s_full[2], s_free[2], p_full[2], o_full[2];
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(FwdBars) <= 256, "barriers fit behind the tiles");

// The kernels' tiles need the dynamic shared memory to start on 1024 bytes,
// which it does where there is no static one; checked, since the swizzle
// depends on it.
__device__ __forceinline__ bool tiles_aligned(const unsigned char* sm, int* err) {
  if (!(tc::smem_u32(sm) & 1023u)) return true;
  if (threadIdx.x == 0) atomicOr(err, tc::kErrTimeoutLoad);
  return false;
}

// Order of the ring's loads: k0 k1 v0 k2 v1 k3 .. (count tiles of each).
__device__ __forceinline__ int load_of_k(int n) { return n < 2 ? n : 2 * n - 1; }
__device__ __forceinline__ int load_of_v(int n, int count) { return (n + 2 < count ? n + 2 : count) + n; }

template <int D, bool kFine>
__global__ void __launch_bounds__(kTcThreads, 1) swa_fwd_tc_kernel(
    const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
    const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to,
    const __grid_constant__ CUtensorMap tl, SwaArgs a) {
  using Cf = FwdCfg<D>;
  extern __shared__ __align__(1024) unsigned char sm[];
  FwdBars& s = *reinterpret_cast<FwdBars*>(sm + Cf::BARS);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // heavy CTAs (late rows: full windows) first
  const int q0 = ((int)gridDim.x - 1 - (int)blockIdx.x) * 256, h = blockIdx.y, b = blockIdx.z;
  const int hk = h / (a.H / a.Hk), W = a.window, S = a.sinks;
  const auto upto = [&](int x) { return x < a.T ? x : a.T; };
  const KeyRange all(q0, upto(q0 + 256), W, S, 128);

  if (!tiles_aligned(sm, a.err)) return;
  const int loads = 2 * all.count;
  volatile int* ab = &s.abort_flag;
  int kn = 0, vn = 0;
  const auto load = [&](int n) {  // the ring's n-th tile
    const bool is_k = kn < all.count && load_of_k(kn) == n;
    const int slot = n % Cf::SLOTS, tile = is_k ? kn++ : vn++;
    tc::mbar_expect_tx(&s.full[slot], Cf::TILE);
    load_tile<D>(sm + Cf::RING + slot * Cf::TILE, is_k ? &tk : &tv, hk, all.tile(tile) * 128, b, &s.full[slot]);
  };
  const auto load_q = [&](int i) {
    tc::mbar_expect_tx(&s.q_full[i], Cf::TILE);
    load_tile<D>(sm + i * Cf::TILE, &tq, h, q0 + 128 * i, b, &s.q_full[i]);
  };
  if (warp == kLoadWarp && lane == 0) {  // what the first scores want flies while the CTA sets up
    tc::mbar_init(&s.q_full[0], 1);
    tc::mbar_init(&s.q_full[1], 1);
    for (int i = 0; i < Cf::SLOTS; ++i) {
      tc::mbar_init(&s.full[i], 1);
      tc::mbar_init(&s.empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s.s_full[i], 1);
      tc::mbar_init(&s.s_free[i], 256);
      tc::mbar_init(&s.p_full[i], 256);
      tc::mbar_init(&s.o_full[i], 1);
    }
    tc::mbar_init_fence();
    s.abort_flag = 0;
    load_q(0);
    load(0);
  }
  if (warp == 0) tc::tmem_alloc(&s.tmem, 512);
  tc::tc_before_sync();
  __syncthreads();
  tc::tc_after_sync();
  const uint32_t tmem = s.tmem;

  if (warp == kLoadWarp) {
    if (lane == 0) {
      if (q0 + 128 < a.T) load_q(1);
      for (int n = 1; n < loads; ++n) {
        if (n >= Cf::SLOTS &&
            !tc::mbar_wait<false>(&s.empty[n % Cf::SLOTS], (n / Cf::SLOTS - 1) & 1, a.err, tc::kErrTimeoutLoad, ab)) break;
        load(n);
      }
    }
  } else if (warp >= kMmaWarp) {
    const int i = warp - kMmaWarp;
    const KeyRange mine(upto(q0 + 128 * i), upto(q0 + 128 * i + 128), W, S, 128);
    const uint32_t base = tc::smem_u32(sm);
    const uint32_t q = base + i * Cf::TILE, p = base + Cf::P + i * 32768;
    const uint32_t sc = tmem + Cf::S_COL + i * 128, o = tmem + Cf::O_COL + i * 128;
    // (all lanes run every tile, also when a wait gave up and the later ones
    // return at once: elect.sync wants the whole warp)
    const auto wait = [&](uint64_t* bar, uint32_t parity, int code) { tc::mbar_wait<false>(bar, parity, a.err, code, ab); };
    int s_done = 0, p_done = 0;  // tiles whose scores, whose products are issued
    const auto landed = [&](int load) {
      wait(&s.full[load % Cf::SLOTS], (load / Cf::SLOTS) & 1, tc::kErrTimeoutLoad);
      return base + Cf::RING + load % Cf::SLOTS * Cf::TILE;
    };
    const auto release = [&](int load, bool used) {  // only where the slot is loaded again: every commit is waited for
      if (load + Cf::SLOTS >= loads) return;
      if (used)
        tc::warp_mma_commit(&s.empty[load % Cf::SLOTS]);
      else if (lane == 0)
        tc::mbar_arrive(&s.empty[load % Cf::SLOTS]);
    };
    // S = q k^T of tile n, when the group has read the scores before
    const auto scores = [&](int n) {
      const bool has = mine.has(all.tile(n));
      // a tile that this group skips is waited for as well, so that its slot's
      // barrier counts one arrival of each chain per load
      const uint32_t k = landed(load_of_k(n));
      if (has) {
        const int m = s_done++;
        if (m > 0) wait(&s.s_free[i], (m - 1) & 1, tc::kErrTimeoutMma);
        tc::tc_after_sync();
        mma_scores<D>(sc, q, k);
        tc::warp_mma_commit(&s.s_full[i]);
      }
      release(load_of_k(n), has);
    };
    // O += P v of tile n
    const auto mix = [&](int n) {
      const bool has = mine.has(all.tile(n));
      const int load = load_of_v(n, all.count);
      const uint32_t v = landed(load);
      if (has) {
        constexpr uint32_t id = tc::idesc(128, D, 1) | tc::kMajorB;
        const int m = p_done++;
        wait(&s.p_full[i], m & 1, tc::kErrTimeoutMma);
        tc::tc_after_sync();
        const uint64_t dp = tc::desc_sw128(p), dv = tc::desc_sw128_mn(v, 16384u);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          tc::warp_mma_bf16_ss(o, tc::desc_at(dp, c / 4 * 16384 + c % 4 * 32), tc::desc_at(dv, c * 2048), id, m > 0 || c > 0);
        if (kFine) {  // the low parts, over the scores
#pragma unroll
          for (int c = 0; c < 8; ++c)
            tc::warp_mma_bf16_ts(o, sc + c / 4 * 64 + c % 4 * 8, tc::desc_at(dv, c * 2048), id, 1);
        }
        tc::warp_mma_commit(&s.o_full[i]);
      }
      release(load, has);
    };
    if (mine.count) wait(&s.q_full[i], 0, tc::kErrTimeoutLoad);
    scores(0);
    for (int n = 0; n < all.count; ++n) {
      const bool more = n + 1 < all.count;
      if (more && !kFine) scores(n + 1);
      mix(n);
      if (more && kFine) scores(n + 1);
    }
  } else {
    // query tile i, columns 64 g .. 64 g + 63 of row r
    const int i = warp >> 3, g = (warp >> 2) & 1, r = tid & 127, r0 = upto(q0 + 128 * i), t = q0 + 128 * i + r;
    const KeyRange mine(r0, upto(q0 + 128 * i + 128), W, S, 128);
    const uint32_t s_lane = tc::tmem_lane_addr(tmem, warp, Cf::S_COL + i * 128 + g * 64);
    const uint32_t o_lane = tc::tmem_lane_addr(tmem, warp, Cf::O_COL + i * 128 + g * (D / 2));
    // this row of the group's weights: 16-byte chunk c of a block at (c ^ (row & 7)) * 16
    unsigned char* prow = sm + Cf::P + i * 32768 + g * 16384 + r * 128;
    const float s2 = a.scale * kLog2e;
    // the two warps that share 32 rows meet to exchange a value per row: the
    // maximum of their columns (both have read it before the next scores can
    // come: s_free follows), at the end the sum (the last product waited for
    // both)
    const auto meet = [&] { asm volatile("bar.sync %0, 64;" ::"r"(1 + i * 4 + (warp & 3)) : "memory"); };
    float* half = reinterpret_cast<float*>(sm + Cf::HALF) + i * 256 + r;
    float top = -INFINITY, sum = 0.f;  // sums refer to 2^(s2 top)
    for (int j = 0, n = -1; j < all.count; ++j) {  // in the order of the loads
      const int k0 = all.tile(j) * 128;
      if (!mine.has(all.tile(j))) continue;
      ++n;
      if (!warp_wait(&s.s_full[i], n & 1, a.err, tc::kErrTimeoutMma, ab)) *ab = 1;  // both warps of the rows go on
      tc::tc_after_sync();
      float x[64];
      tc::tmem_ld32(s_lane, x);
      tc::tmem_ld32(s_lane + 32, x + 32);
      tc::tmem_ld_wait();
      const int end = t - k0 - g * 64 + 1;
      hide(x, k0 + 127 > r0, r0 + 127 - k0 >= W && k0 + 127 >= S, end, end - W, S - k0 - g * 64);
      float m0 = x[0], m1 = x[1], m2 = x[2], m3 = x[3];
#pragma unroll
      for (int c = 4; c < 64; c += 4) {
        m0 = fmaxf(m0, x[c]);
        m1 = fmaxf(m1, x[c + 1]);
        m2 = fmaxf(m2, x[c + 2]);
        m3 = fmaxf(m3, x[c + 3]);
      }
      float m = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
      half[g * 128] = m;
      meet();
      m = fmaxf(m, half[(g ^ 1) * 128]);
      if (!kFine) {
        tc::tc_before_sync();
        tc::mbar_arrive(&s.s_free[i]);
      }
      const bool grow = n == 0 ? m > top : (m - top) * s2 > 8.f;  // false while a row has seen no key
      const float f = n > 0 && grow ? ex2((top - m) * s2) : 1.f;
      if (grow) top = m;
      const float ref = top == -INFINITY ? 0.f : top * s2;
      // the product before has read the weights, and the output is complete
      const auto before = [&] {
        if (n == 0) return;
        warp_wait(&s.o_full[i], (n - 1) & 1, a.err, tc::kErrTimeoutMma, ab);
        if (!__any_sync(0xffffffffu, grow)) return;
        tc::tc_after_sync();  // each warp its half of the channels
#pragma unroll
        for (int c = 0; c < D / 2; c += 16) {
          float o[16];
          tc::tmem_ld16(o_lane + c, o);
          tc::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] *= f;
          tc::tmem_st16(o_lane + c, o);
        }
        tc::tmem_st_wait();
      };
      if (kFine) before();
      float a0 = 0.f, a1 = 0.f;
      uint4 w[kFine ? 1 : 8];
#pragma unroll
      for (int c = 0; c < 64; c += 8) {
        uint4& wc = w[kFine ? 0 : c / 8];
        uint32_t* wp = reinterpret_cast<uint32_t*>(&wc);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          x[c + e] = ex2(fmaf(x[c + e], s2, -ref));
          x[c + e + 1] = ex2(fmaf(x[c + e + 1], s2, -ref));
          wp[e / 2] = __float_as_uint(bf16_pair(x[c + e], x[c + e + 1]));
          a0 += x[c + e];
          a1 += x[c + e + 1];
        }
        if (kFine) {  // and what the rounding left
          *reinterpret_cast<uint4*>(prow + ((c / 8) ^ (r & 7)) * 16) = wc;
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            x[c + e] -= __uint_as_float(wp[e / 2] << 16);
            x[c + e + 1] -= __uint_as_float(wp[e / 2] & 0xffff0000u);
          }
        }
      }
      sum = fmaf(sum, f, a0 + a1);
      if (!kFine) {
        before();
#pragma unroll
        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(prow + (c ^ (r & 7)) * 16) = w[c];
      }
      if (kFine) {
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          float l[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) l[e / 2] = bf16_pair(x[c + e], x[c + e + 1]);
          tc::tmem_st16(s_lane + c / 2, l);
        }
        tc::tmem_st_wait();
      }
      tc::fence_proxy_async();
      tc::tc_before_sync();
      tc::mbar_arrive(&s.p_full[i]);
      if (kFine) tc::mbar_arrive(&s.s_free[i]);  // the next scores follow this tile's product
    }
    if (mine.count) {
      warp_wait(&s.o_full[i], (mine.count - 1) & 1, a.err, tc::kErrTimeoutMma, ab);
      tc::tc_after_sync();
      half[g * 128] = sum;
      meet();
      sum += half[(g ^ 1) * 128];
      // out over the queries, its rounding over the weights: nothing reads them any more
      unsigned char *out = sm + i * Cf::TILE, *lo = sm + Cf::P + i * 32768;
      stage_lane<D / 2>(o_lane, 1.f / sum, out, a.olo ? lo : nullptr, r, g * (D / 2));
      if (t < a.T && g == 0) a.lse[((size_t)b * a.T + t) * a.H + h] = fmaf(top, s2, log2f(sum)) * kLn2;
      tc::fence_proxy_async();
      asm volatile("bar.sync %0, 256;" ::"r"(9 + i) : "memory");
      if ((tid & 255) == 0) {
        store_tile<D>(out, &to, h, r0, b);
        if (a.olo) store_tile<D>(lo, &tl, h, r0, b);
        tc::bulk_commit();
        tc::bulk_wait_read();
      }
    }
  }
  tc::tc_before_sync();
  __syncthreads();
  tc::tc_after_sync();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// ---- backward ----------------------------------------------------------------

// The CTA's own two tiles, a ring of tiles, and for dkv (which has one slot
// less) the weights p.
template <int D, bool kDkv>
struct BwdCfg {
  static constexpr uint32_t TILE = 128 * D * 2;
  static constexpr int SLOTS = kDkv ? 4 : 5;
  static constexpr uint32_t RING = 2 * TILE;
  static constexpr uint32_t P = RING + SLOTS * TILE;
  static constexpr uint32_t ROWS = P + (kDkv ? 32768 : 0);  // dkv: lse2, delta of two query tiles
  static constexpr uint32_t BARS = ROWS + 2 * 1024;
  static constexpr uint32_t BYTES = BARS + 256;            // no static shared memory: all 227 KB at d = 128
};

struct BwdBars {
  uint64_t own[2], full[5], empty[5], s_full[2], s_free, dp_full, p_ready, p_read, ds_ready[2], done;
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(BwdBars) <= 256, "barriers fit behind the tiles");

// `chains`: MMA chains that a slot's tile and an accumulator's end wait for.
template <typename F>
__device__ __forceinline__ bool bwd_setup(unsigned char* sm, BwdBars& s, int chains, int* err, F first_loads) {
  if (!tiles_aligned(sm, err)) return false;
  if (threadIdx.x == kLoadWarp * 32) {  // what the first scores want flies while the CTA sets up
    tc::mbar_init(&s.own[0], 1);
    tc::mbar_init(&s.own[1], 1);
    for (int i = 0; i < 5; ++i) {
      tc::mbar_init(&s.full[i], 1);
      tc::mbar_init(&s.empty[i], chains);
    }
    tc::mbar_init(&s.s_full[0], 1);
    tc::mbar_init(&s.s_full[1], 1);
    tc::mbar_init(&s.s_free, 512);
    tc::mbar_init(&s.dp_full, 1);
    tc::mbar_init(&s.p_ready, 512);
    tc::mbar_init(&s.p_read, 1);
    tc::mbar_init(&s.ds_ready[0], 512);
    tc::mbar_init(&s.ds_ready[1], 512);
    tc::mbar_init(&s.done, chains);
    tc::mbar_init_fence();
    s.abort_flag = 0;
    first_loads();
  }
  if (threadIdx.x < 32) tc::tmem_alloc(&s.tmem, 512);
  tc::tc_before_sync();
  __syncthreads();
  tc::tc_after_sync();
  return true;
}

__device__ __forceinline__ void bwd_finish(uint32_t tmem) {
  tc::tc_before_sync();
  __syncthreads();
  tc::tc_after_sync();
  if (threadIdx.x < 32) tc::tmem_dealloc(tmem, 512);
}

// The ring of a backward item as its MMA warps see it.  (All lanes run every
// tile, also when a wait gave up and the later ones return at once: elect.sync
// wants the whole warp.)
template <typename Cf>
struct BwdRing {
  BwdBars& s;
  uint32_t base;
  int loads;
  int* err;
  struct At {  // every second load
    int load, slot;
    uint32_t parity;
    __device__ explicit At(int first) : load(first), slot(first % Cf::SLOTS), parity(first / Cf::SLOTS & 1) {}
    __device__ void next() {
      load += 2;
      slot += 2;
      if (slot >= Cf::SLOTS) {
        slot -= Cf::SLOTS;
        parity ^= 1;
      }
    }
  };
  __device__ uint32_t tile(const At& x) const { return base + Cf::RING + x.slot * Cf::TILE; }
  __device__ uint32_t landed(const At& x) const {
    tc::mbar_wait<false>(&s.full[x.slot], x.parity, err, tc::kErrTimeoutLoad, &s.abort_flag);
    tc::tc_after_sync();
    return tile(x);
  }
  __device__ void release(const At& x) const {  // only where the slot is loaded again
    if (x.load + Cf::SLOTS < loads) tc::warp_mma_commit(&s.empty[x.slot]);
  }
  __device__ void ready(uint64_t* bar, int use) const {
    tc::mbar_wait<false>(bar, use & 1, err, tc::kErrTimeoutMma, &s.abort_flag);
    tc::tc_after_sync();
  }
};

// 32 weights of this thread's row, rounded, as the A operand at `dst`, and with
// kFine what the rounding leaves in the 16 columns behind.
template <bool kFine>
__device__ __forceinline__ void store_weights(uint32_t dst, const float (&x)[32]) {
  float w[16];
#pragma unroll
  for (int e = 0; e < 32; e += 2) w[e / 2] = bf16_pair(x[e], x[e + 1]);
  tc::tmem_st16(dst, w);
  if (kFine) {
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const uint32_t hi = __float_as_uint(w[e / 2]);
      w[e / 2] = bf16_pair(x[e] - __uint_as_float(hi << 16), x[e + 1] - __uint_as_float(hi & 0xffff0000u));
    }
    tc::tmem_st16(dst + 16, w);
  }
  tc::tmem_st_wait();
  tc::tc_before_sync();
}

struct BwdMaps {  // tiles of 128 rows
  CUtensorMap q, g, dq, k, v, dk, dv;  // g: dO
};

// dq of query tile `tile`, head h, batch entry b.
template <int D, bool kFine>
__device__ __forceinline__ void dq_item(const BwdMaps& m, const SwaArgs& a, const SwaBwdLayout& L, unsigned char* sm,
                                        int tile, int h, int b) {
  using Cf = BwdCfg<D, false>;
  constexpr int DP = 256, DQ = 384;  // TMEM: two buffers of scores, dP, dq
  BwdBars& s = *reinterpret_cast<BwdBars*>(sm + Cf::BARS);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q0 = tile * 128, hk = h / (a.H / a.Hk), W = a.window, S = a.sinks;
  const KeyRange keys(q0, q0 + 128 < a.T ? q0 + 128 : a.T, W, S, 128);
  const int count = keys.count;
  const auto load = [&](int n) {  // k0 v0 k1 v1 ..
    const int slot = n % Cf::SLOTS;
    tc::mbar_expect_tx(&s.full[slot], Cf::TILE);
    load_tile<D>(sm + Cf::RING + slot * Cf::TILE, n & 1 ? &m.v : &m.k, hk, keys.tile(n / 2) * 128, b, &s.full[slot]);
  };
  if (!bwd_setup(sm, s, 1, a.err, [&] {
        tc::mbar_expect_tx(&s.own[0], Cf::TILE);
        load_tile<D>(sm, &m.q, h, q0, b, &s.own[0]);
        load(0);
      }))
    return;
  const uint32_t tmem = s.tmem;
  volatile int* ab = &s.abort_flag;
  if (warp == kLoadWarp) {
    if (lane == 0) {
      tc::mbar_expect_tx(&s.own[1], Cf::TILE);
      load_tile<D>(sm + Cf::TILE, &m.g, h, q0, b, &s.own[1]);
      for (int n = 1; n < 2 * count; ++n) {
        if (n >= Cf::SLOTS &&
            !tc::mbar_wait<false>(&s.empty[n % Cf::SLOTS], (n / Cf::SLOTS - 1) & 1, a.err, tc::kErrTimeoutLoad, ab)) break;
        load(n);
      }
    }
  } else if (warp == kMmaWarp) {  // scores and dq
    const BwdRing<Cf> ring{s, tc::smem_u32(sm), 2 * count, a.err};
    typename BwdRing<Cf>::At at(0), ahead(2);
    ring.ready(&s.own[0], 0);
    mma_scores<D>(tmem, ring.base, ring.landed(at));
    tc::warp_mma_commit(&s.s_full[0]);
    for (int n = 0; n < count; ++n, at.next(), ahead.next()) {
      if (n + 1 < count) {  // the next scores, while the groups work on dS
        mma_scores<D>(tmem + (n + 1) % 2 * 128, ring.base, ring.landed(ahead));
        tc::warp_mma_commit(&s.s_full[(n + 1) % 2]);
      }
      ring.ready(&s.ds_ready[n % 2], n >> 1);
      mma_mix<D>(tmem + DQ, tmem + n % 2 * 128, ring.tile(at), n > 0);
      if (kFine) mma_mix<D>(tmem + DQ, tmem + n % 2 * 128 + 16, ring.tile(at), true);
      ring.release(at);
    }
    tc::warp_mma_commit(&s.done);
  } else if (warp == kMmaWarp + 1) {  // dP, when the groups have read the one before
    const BwdRing<Cf> ring{s, tc::smem_u32(sm), 2 * count, a.err};
    typename BwdRing<Cf>::At at(1);
    ring.ready(&s.own[1], 0);
    for (int n = 0; n < count; ++n, at.next()) {
      const uint32_t v = ring.landed(at);
      if (n > 0) ring.ready(&s.ds_ready[(n - 1) % 2], (n - 1) >> 1);
      mma_scores<D>(tmem + DP, ring.base + Cf::TILE, v);
      tc::warp_mma_commit(&s.dp_full);
      ring.release(at);
    }
  } else {
    const int g = warp >> 2, t = q0 + (tid & 127);  // columns 32 g .. 32 g + 31
    const uint32_t lanes = tc::tmem_lane_addr(tmem, warp, g * 32);
    const size_t at = ((size_t)b * a.H + h) * L.Tp + t;
    const float lse2 = reinterpret_cast<const float*>(a.ws + L.lse2)[at];
    const float delta = reinterpret_cast<const float*>(a.ws + L.delta)[at];
    const float s2 = a.scale * kLog2e;
    const bool lone = single_key(t, W, S);  // dS is exactly 0; its one key is in the tile with an upper bound
    for (int n = 0; n < count; ++n) {
      const int k0 = keys.tile(n) * 128;
      const uint32_t buf = lanes + n % 2 * 128;
      if (!warp_wait(&s.s_full[n % 2], (n >> 1) & 1, a.err, tc::kErrTimeoutMma, ab)) break;
      tc::tc_after_sync();
      float x[32], dp[32];
      tc::tmem_ld32(buf, x);
      tc::tmem_ld_wait();
      const int end = t - k0 - g * 32 + 1;
      hide(x, k0 + 127 > q0, q0 + 127 - k0 >= W && k0 + 127 >= S, lone ? 0 : end, end - W, S - k0 - g * 32);
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = ex2(fmaf(x[e], s2, -lse2));
      if (!warp_wait(&s.dp_full, n & 1, a.err, tc::kErrTimeoutMma, ab)) break;
      tc::tc_after_sync();
      tc::tmem_ld32(lanes + DP, dp);
      tc::tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] *= dp[e] - delta;
      store_weights<kFine>(buf, x);
      tc::mbar_arrive(&s.ds_ready[n % 2]);
    }
    warp_wait(&s.done, 0, a.err, tc::kErrTimeoutMma, ab);
    tc::tc_after_sync();
    stage_lane<D / 4>(tc::tmem_lane_addr(tmem, warp, DQ + g * (D / 4)), a.scale, sm, nullptr, tid & 127, g * (D / 4));
    tc::fence_proxy_async();
    asm volatile("bar.sync 1, 512;" ::: "memory");
    if (tid == 0) {  // over q, which nothing reads any more
      store_tile<D>(sm, &m.dq, h, q0, b);
      tc::bulk_commit();
      tc::bulk_wait_read();
    }
  }
  bwd_finish(tmem);
}

// dk, dv of key tile `tile` from its band's queries, all query heads of key
// head h0 / group (piece < 0); or the first tokens' part from piece `piece` of the
// queries beyond their tile's band, query head h0.
template <int D, bool kFine>
__device__ __forceinline__ void dkv_item(const BwdMaps& m, const SwaArgs& a, const SwaBwdLayout& L, unsigned char* sm,
                                         int tile, int piece, int h0, int b, bool has_far) {
  using Cf = BwdCfg<D, true>;
  constexpr int DP = 128, DV = 256, DK = 384;  // TMEM: scores, dP, dv, dk
  BwdBars& s = *reinterpret_cast<BwdBars*>(sm + Cf::BARS);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.H / a.Hk, W = a.window, S = a.sinks, k0 = tile * 128;
  const bool far = piece >= 0;
  const int band_end = k0 + 127 + W < a.T ? k0 + 127 + W : a.T;
  const int heads = far ? 1 : group;
  int q_lo = k0, q_hi = band_end;
  if (far) {
    q_lo = piece * kSwaPiece > band_end ? piece * kSwaPiece : band_end;
    q_hi = (piece + 1) * kSwaPiece < a.T ? (piece + 1) * kSwaPiece : a.T;
    if (q_lo >= q_hi) return;  // the sum skips it too
  }
  const int hk = h0 / group, qt0 = q_lo / 128, per = (q_hi - 1) / 128 - qt0 + 1, count = per * heads;
  const auto load = [&](int n) {  // q0 dO0 q1 dO1 ..; lse2 and delta with q
    const int slot = n % Cf::SLOTS, i = n / 2, h = h0 + i / per, t0 = (qt0 + i % per) * 128;
    unsigned char* st = sm + Cf::RING + slot * Cf::TILE;
    if (n & 1) {
      tc::mbar_expect_tx(&s.full[slot], Cf::TILE);
      load_tile<D>(st, &m.g, h, t0, b, &s.full[slot]);
    } else {
      // the rows of two tiles ago were in this place, and that tile's q in
      // this slot: the groups were through with them when it was released
      static_assert(Cf::SLOTS == 4, "rows and q of a tile are replaced together");
      float* rows = reinterpret_cast<float*>(sm + Cf::ROWS + i % 2 * 1024);
      const size_t at = ((size_t)b * a.H + h) * L.Tp + t0;
      tc::mbar_expect_tx(&s.full[slot], Cf::TILE + 1024);
      load_tile<D>(st, &m.q, h, t0, b, &s.full[slot]);
      tc::bulk_g2s(rows, reinterpret_cast<const float*>(a.ws + L.lse2) + at, 512, &s.full[slot]);
      tc::bulk_g2s(rows + 128, reinterpret_cast<const float*>(a.ws + L.delta) + at, 512, &s.full[slot]);
    }
  };
  if (!bwd_setup(sm, s, 2, a.err, [&] {
        tc::mbar_expect_tx(&s.own[0], Cf::TILE);
        load_tile<D>(sm, &m.k, hk, k0, b, &s.own[0]);
        load(0);
      }))
    return;
  const uint32_t tmem = s.tmem;
  volatile int* ab = &s.abort_flag;
  if (warp == kLoadWarp) {
    if (lane == 0) {
      tc::mbar_expect_tx(&s.own[1], Cf::TILE);
      load_tile<D>(sm + Cf::TILE, &m.v, hk, k0, b, &s.own[1]);
      for (int n = 1; n < 2 * count; ++n) {
        if (n >= Cf::SLOTS &&
            !tc::mbar_wait<false>(&s.empty[n % Cf::SLOTS], (n / Cf::SLOTS - 1) & 1, a.err, tc::kErrTimeoutLoad, ab)) break;
        load(n);
      }
    }
  } else if (warp == kMmaWarp) {  // scores and dv
    const BwdRing<Cf> ring{s, tc::smem_u32(sm), 2 * count, a.err};
    typename BwdRing<Cf>::At q_at(0), g_at(1);
    ring.ready(&s.own[0], 0);
    const auto scores = [&](int n) {
      const uint32_t q = ring.landed(q_at);
      if (n > 0) ring.ready(&s.s_free, n - 1);
      mma_scores<D>(tmem, ring.base, q);
      tc::warp_mma_commit(&s.s_full[0]);
      ring.release(q_at);
      q_at.next();
    };
    scores(0);
    for (int n = 0; n < count; ++n, g_at.next()) {
      if (!kFine && n + 1 < count) scores(n + 1);  // while the groups work on p
      const uint32_t g = ring.landed(g_at), p = ring.base + Cf::P;
      ring.ready(&s.p_ready, n);
      constexpr uint32_t id = tc::idesc(128, D, 1) | tc::kMajorB;
      const uint64_t dp = tc::desc_sw128(p), dg = tc::desc_sw128_mn(g, 16384u);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        tc::warp_mma_bf16_ss(tmem + DV, tc::desc_at(dp, i / 4 * 16384 + i % 4 * 32), tc::desc_at(dg, i * 2048), id,
                             n > 0 || i > 0);
      if (kFine) mma_mix<D>(tmem + DV, tmem, g, true);  // p's low parts, over the scores
      tc::warp_mma_commit(&s.p_read);
      ring.release(g_at);
      if (kFine && n + 1 < count) scores(n + 1);
    }
    tc::warp_mma_commit(&s.done);
  } else if (warp == kMmaWarp + 1) {  // dP and dk
    const BwdRing<Cf> ring{s, tc::smem_u32(sm), 2 * count, a.err};
    typename BwdRing<Cf>::At q_at(0), g_at(1);
    ring.ready(&s.own[1], 0);
    for (int n = 0; n < count; ++n, q_at.next(), g_at.next()) {
      mma_scores<D>(tmem + DP, ring.base + Cf::TILE, ring.landed(g_at));
      tc::warp_mma_commit(&s.dp_full);
      ring.release(g_at);
      const uint32_t q = ring.landed(q_at);
      ring.ready(&s.ds_ready[0], n);
      mma_mix<D>(tmem + DK, tmem + DP, q, n > 0);
      if (kFine) mma_mix<D>(tmem + DK, tmem + DP + 16, q, true);
      ring.release(q_at);
    }
    tc::warp_mma_commit(&s.done);
  } else {
    const int g = warp >> 2, key = k0 + (tid & 127);  // columns 32 g .. 32 g + 31
    const uint32_t buf = tc::tmem_lane_addr(tmem, warp, g * 32);
    const float s2 = a.scale * kLog2e;
    // this key's row of the weights, the group's 32 columns: 16-byte chunk c of a
    // block of 64 at (c ^ (row & 7)) * 16
    unsigned char* prow = sm + Cf::P + g / 2 * 16384 + (tid & 127) * 128;
    typename BwdRing<Cf>::At at(0);
    for (int n = 0, i = 0; n < count; ++n, at.next()) {
      const int q0 = (qt0 + i) * 128;  // query tile i of this head
      if (++i == per) i = 0;
      const float4* rows = reinterpret_cast<const float4*>(sm + Cf::ROWS + n % 2 * 1024) + g * 8;
      // the scores' commit follows the arrival of q and its rows, but only this
      // wait lets this thread read what the copy wrote
      if (!warp_wait(&s.full[at.slot], at.parity, a.err, tc::kErrTimeoutLoad, ab)) break;
      if (!warp_wait(&s.s_full[0], n & 1, a.err, tc::kErrTimeoutMma, ab)) break;
      tc::tc_after_sync();
      float x[32], dp[32];
      tc::tmem_ld32(buf, x);
      tc::tmem_ld_wait();
      if (!kFine) {
        tc::tc_before_sync();
        tc::mbar_arrive(&s.s_free);
      }
      // queries from the key on, up to the window's end (a first token: any)
      const int c0 = q0 + g * 32, from = (key > q_lo ? key : q_lo) - c0;
      const int end = (key >= S && key + W < q_hi ? key + W : q_hi) - c0;
      hide(x, q0 + 127 >= q_hi || (k0 + 127 >= S && q0 + 127 - k0 >= W), q0 < q_lo || q0 < k0 + 127, end, from, 0);
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const float4 l = rows[e / 4];
        x[e] = ex2(fmaf(x[e], s2, -l.x));
        x[e + 1] = ex2(fmaf(x[e + 1], s2, -l.y));
        x[e + 2] = ex2(fmaf(x[e + 2], s2, -l.z));
        x[e + 3] = ex2(fmaf(x[e + 3], s2, -l.w));
      }
      if (n > 0 && !warp_wait(&s.p_read, (n - 1) & 1, a.err, tc::kErrTimeoutMma, ab)) break;
      float lo[16];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint4 w;
        uint32_t* wp = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          wp[e] = __float_as_uint(bf16_pair(x[c * 8 + 2 * e], x[c * 8 + 2 * e + 1]));
          if (kFine)
            lo[c * 4 + e] = bf16_pair(x[c * 8 + 2 * e] - __uint_as_float(wp[e] << 16),
                                      x[c * 8 + 2 * e + 1] - __uint_as_float(wp[e] & 0xffff0000u));
        }
        *reinterpret_cast<uint4*>(prow + ((g % 2 * 4 + c) ^ (tid & 7)) * 16) = w;
      }
      tc::fence_proxy_async();
      if (kFine) {
        tc::tmem_st16(buf, lo);
        tc::tmem_st_wait();
        tc::tc_before_sync();
        tc::mbar_arrive(&s.s_free);  // the next scores follow this tile's product
      }
      tc::mbar_arrive(&s.p_ready);
      if (!warp_wait(&s.dp_full, n & 1, a.err, tc::kErrTimeoutMma, ab)) break;
      tc::tc_after_sync();
      tc::tmem_ld32(buf + DP, dp);
      tc::tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const float4 d = rows[32 + e / 4];
        x[e] *= dp[e] - d.x;
        x[e + 1] *= dp[e + 1] - d.y;
        x[e + 2] *= dp[e + 2] - d.z;
        x[e + 3] *= dp[e + 3] - d.w;
      }
      if (c0 == 0) x[0] = 0.f;  // the first query has one key: dS is exactly 0
      if (W == 1 && S == 0) {   // and so has every query of a window of one
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = 0.f;
      }
      store_weights<kFine>(buf + DP, x);
      tc::mbar_arrive(&s.ds_ready[0]);
    }
    warp_wait(&s.done, 0, a.err, tc::kErrTimeoutMma, ab);
    tc::tc_after_sync();
    // groups 0 and 1 write the halves of dv, 2 and 3 of dk
    const bool is_k = g >= 2;
    const int c0 = g % 2 * (D / 2);
    const uint32_t lanes = tc::tmem_lane_addr(tmem, warp, (is_k ? DK : DV) + c0);
    const float f = is_k ? a.scale : 1.f;
    const bool mine = key < a.T && c0 < a.d;
    const bool first = key < S && mine && has_far;  // rows that other items add to: fp32 parts
    float* part = nullptr;
    if (first && far)
      part = reinterpret_cast<float*>(a.ws + L.part) +
             (((((size_t)(is_k ? 0 : 1) * L.pieces + piece) * a.B + b) * a.H + h0) * S + key) * a.d + c0;
    else if (first)
      part = reinterpret_cast<float*>(a.ws + L.band) +
             ((((size_t)(is_k ? 0 : 1) * a.B + b) * a.Hk + hk) * S + key) * a.d + c0;
    if (k0 < S && has_far) {  // the tile of the first tokens: row by row
      __nv_bfloat16* dst =
          static_cast<__nv_bfloat16*>(is_k ? a.dk : a.dv) + (((size_t)b * a.T + key) * a.Hk + hk) * a.d + c0;
      const bool plain = !far && !first && mine;
#pragma unroll
      for (int c = 0; c < D / 2; c += 16) {
        float v[16];
        __syncwarp();
        tc::tmem_ld16(lanes + c, v);
        tc::tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] *= f;
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          if (part) *reinterpret_cast<float4*>(part + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
#pragma unroll
        for (int e = 0; e < 16; e += 8) {  // 16 bytes at a time: what dk and dv are aligned to
          float w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = v[e + i];
          if (plain) store_row<__nv_bfloat16, 8>(dst + c + e, w);
        }
      }
    } else {  // dk over k, dv over v, which nothing reads any more
      stage_lane<D / 2>(lanes, f, sm + (is_k ? 0 : Cf::TILE), nullptr, tid & 127, c0);
      tc::fence_proxy_async();
      asm volatile("bar.sync 1, 512;" ::: "memory");
      if (tid == 0) {
        store_tile<D>(sm, &m.dk, hk, k0, b);
        store_tile<D>(sm + Cf::TILE, &m.dv, hk, k0, b);
        tc::bulk_commit();
        tc::bulk_wait_read();
      }
    }
  }
  bwd_finish(tmem);
}

// One launch for all of them: the key tiles, the first tokens' far pieces and
// the query tiles.  One launch and two, delta pass included: 61 and 77 us (T1024
// H16 Hk4 window 512), 485 and 500 (T16384), 330 and 400 (T4096 Hk1 window
// 1024), the same where every SM has many tiles of each kind.
template <int D, bool kFine>
__global__ void __launch_bounds__(kTcThreads, 1) swa_bwd_tc_kernel(const __grid_constant__ BwdMaps m, SwaArgs a,
                                                                   SwaBwdLayout L, int tiles, int far_items,
                                                                   int key_items) {
  extern __shared__ __align__(1024) unsigned char sm[];
  int i = blockIdx.x;
  if (i < key_items) {
    const int group = a.H / a.Hk, kb = i / tiles;
    dkv_item<D, kFine>(m, a, L, sm, i % tiles, -1, kb % a.Hk * group, kb / a.Hk, far_items > 0);
    return;
  }
  i -= key_items;
  if (i < far_items) {
    const int hb = i / L.pieces;
    dkv_item<D, kFine>(m, a, L, sm, 0, i % L.pieces, hb % a.H, hb / a.H, true);
    return;
  }
  i -= far_items;
  const int hb = i / tiles;
  dq_item<D, kFine>(m, a, L, sm, tiles - 1 - i % tiles, hb % a.H, hb / a.H);
}

template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// Rows of at most this many keys take the finer weights.  Errors of dq against
// its own rounding to bf16, with one bf16 weight: 1.72 at 1 to 2 keys (the
// forward's rounding of p reaches it through delta), 1.52 at 9, 1.45 at 129,
// and by chance up to 1.84 where a batch has only some ten rows; from some
// hundred keys on 1.43, which is what rounding dS alone costs.  With the finer
// ones 1.00 throughout.  They cost 112 -> 137 us forward and 271 -> 346 backward
// at T16384 H16 Hk4 d128 window 252, 11 -> 13 and 13 -> 15 at T200 Hk16.
constexpr int kFineKeys = 256;
bool fine(const SwaArgs& a) {
  return (a.window + a.sinks < a.T ? a.window + a.sinks : a.T) <= kFineKeys;  // window, sinks <= T
}

template <int D, bool kFine>
cudaError_t fwd_go(const SwaArgs& a, cudaStream_t st) {
  using Cf = FwdCfg<D>;
  CUtensorMap tq, tk, tv, to, tl;
  if (!make_tmap_bthd(&to, a.out, 2, a.B, a.T, a.H, a.d, 64, true, 128) ||
      !make_tmap_bthd(&tl, a.olo ? a.olo : a.out, 2, a.B, a.T, a.H, a.d, 64, true, 128) ||
      !make_tmap_bthd(&tq, a.q, 2, a.B, a.T, a.H, a.d, 64, true, 128) ||
      !make_tmap_bthd(&tk, a.k, 2, a.B, a.T, a.Hk, a.d, 64, true, 128) ||
      !make_tmap_bthd(&tv, a.v, 2, a.B, a.T, a.Hk, a.d, 64, true, 128))
    return cudaErrorInvalidValue;
  cudaError_t e = allow_smem(swa_fwd_tc_kernel<D, kFine>, Cf::BYTES);
  if (e != cudaSuccess) return e;
  prof_begin(st, "swa_fwd_tc");
  swa_fwd_tc_kernel<D, kFine><<<dim3((a.T + 255) / 256, a.H, a.B), kTcThreads, Cf::BYTES, st>>>(tq, tk, tv, to, tl, a);
  prof_end(st);
  return cudaGetLastError();
}

template <int D, bool kFine>
cudaError_t bwd_go(const SwaArgs& a, cudaStream_t st) {
  constexpr uint32_t kBytes = BwdCfg<D, true>::BYTES > BwdCfg<D, false>::BYTES ? BwdCfg<D, true>::BYTES
                                                                               : BwdCfg<D, false>::BYTES;
  const SwaBwdLayout L = swa_bwd_layout(a.B, a.T, a.H, a.Hk, a.d, a.window, a.sinks);
  BwdMaps m;
  CUtensorMap* maps[7] = {&m.q, &m.g, &m.dq, &m.k, &m.v, &m.dk, &m.dv};
  const void* src[7] = {a.q, a.dO, a.dq, a.k, a.v, a.dk, a.dv};
  for (int i = 0; i < 7; ++i)
    if (!make_tmap_bthd(maps[i], src[i], 2, a.B, a.T, i < 3 ? a.H : a.Hk, a.d, 64, true, 128)) return cudaErrorInvalidValue;
  cudaError_t e = allow_smem(swa_bwd_tc_kernel<D, kFine>, kBytes);
  if (e == cudaSuccess) e = launch_swa_delta(a, L, st);
  if (e != cudaSuccess) return e;
  const int tiles = (a.T + 127) / 128;
  const bool has_far = a.sinks > 0 && 127 + a.window < a.T;
  const long long key_items = (long long)tiles * a.Hk * a.B, far_items = has_far ? (long long)L.pieces * a.H * a.B : 0;
  const long long items = key_items + far_items + (long long)tiles * a.H * a.B;
  if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
  prof_begin(st, "swa_bwd_tc");
  swa_bwd_tc_kernel<D, kFine><<<(unsigned)items, kTcThreads, kBytes, st>>>(m, a, L, tiles, (int)far_items, (int)key_items);
  prof_end(st);
  e = cudaGetLastError();
  if (e == cudaSuccess && has_far) e = launch_swa_sink_sum(a, L, 128, st);
  return e;
}

}  // namespace

bool swa_tc_supported(int dtype) { return dtype == 1; }
cudaError_t launch_swa_fwd_tc(const SwaArgs& a, cudaStream_t st) {
  if (fine(a)) return a.d <= 64 ? fwd_go<64, true>(a, st) : fwd_go<128, true>(a, st);
  return a.d <= 64 ? fwd_go<64, false>(a, st) : fwd_go<128, false>(a, st);
}
cudaError_t launch_swa_bwd_tc(const SwaArgs& a, cudaStream_t st) {
  if (fine(a)) return a.d <= 64 ? bwd_go<64, true>(a, st) : bwd_go<128, true>(a, st);
  return a.d <= 64 ? bwd_go<64, false>(a, st) : bwd_go<128, false>(a, st);
}

}  // namespace kd
