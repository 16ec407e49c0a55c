// kd_swa_tc.cu -- sliding-window attention with first tokens kept, on tcgen05
// (bf16, d = 64 and 128).  The formulas are in kd_swa.cu.
//
// Every kernel has ten warps: two groups of four (thread = TMEM lane = tile
// row) for the elementwise work, one thread that loads tiles by TMA into a
// ring, one that issues the MMAs.  The groups work on separate tiles, so that
// the tensor core multiplies one group's operands while the other group turns
// its scores into weights.  The weights (p, dS) are rounded to bf16 and go
// back to TMEM over the scores they came from, as the next product's A
// operand; the B operand of those products (v, k, dO, q) is read MN-major from
// the same shared-memory tile that the score product reads K-major, so no tile
// is stored twice or transposed.
//
// Forward: 256 queries of one head per CTA, a group to each 128; keys in tiles
// of 128.  Bound by the hardware exponential as much as by the MMAs (128 x 128
// exponentials take as long as the two products of that tile at d = 128).  The
// output stays in TMEM; it is rescaled only when a row's maximum has grown by
// more than 2^8 over the one its sums refer to (then p <= 2^8, still exact
// enough in bf16, whose precision does not depend on the size).  Short rows
// (kFine) take the weights as bf16 high and low parts: over a few keys the
// roundings of p do not average out, and the backward's delta = dO.o would
// pass them on to every gradient.
//
// Backward: p is recomputed from the saved lse.  dk, dv: 128 keys per CTA
// (rows are keys: S^T = k q^T, dP^T = v dO^T), 64 queries at a time, the two
// groups alternating; dv += P^T dO, dk += dS^T q.  dq: 128 queries per CTA, 64
// keys at a time; dq += dS k.  Seven products in place of the five of one
// joint pass, but no atomics and no fp32 copy of dq: every sum has one order.
#include "kd_hybrid.h"
#include "kd_rows.cuh"
#include "kd_tc.cuh"
#include "kd_tmap.h"

namespace kd {

namespace {

constexpr int kTcThreads = 320;
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr float kLog2e = 1.44269504088896f;
constexpr float kLn2 = 0.693147180559945f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ bool visible(int t, int j, int W, int S) { return j <= t && (t - j < W || j < S); }
__device__ __forceinline__ bool single_key(int t, int W, int S) { return t == 0 || (W == 1 && S == 0); }

// A wait that a whole warp gives up together (its TMEM loads need all lanes).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* err, int code, volatile int* ab) {
  return __all_sync(0xffffffffu, tc::mbar_wait<false>(bar, parity, err, code, ab));
}

__device__ __forceinline__ float bf16_pair(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return __uint_as_float(*reinterpret_cast<const uint32_t*>(&v));
}

// The key tiles of B keys that query rows q0 .. q1 - 1 see: those of the first
// tokens, then those of the band.
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
  __device__ int tile(int i) const { return i < first ? i : band + i - first; }
  __device__ bool has(int kt) const { return kt < first || (kt >= band && kt <= end); }
};

// Row of D fp32 values of this thread's TMEM lane, scaled, to global bf16; the
// rounding that is left over goes to `lo` where it is given.
template <int D>
__device__ __forceinline__ void store_lane(uint32_t lanes, float scale, __nv_bfloat16* dst, __nv_bfloat16* lo) {
#pragma unroll
  for (int c = 0; c < D; c += 32) {
    float v[32];
    __syncwarp();  // rows without a destination skip the stores, not the warp's loads
    tc::tmem_ld32(lanes + c, v);
    tc::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32 && dst; i += 8) {
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = v[i + e] * scale;
      store_row<__nv_bfloat16, 8>(dst + c + i, w);
      if (lo) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] -= __bfloat162float(__float2bfloat16_rn(w[e]));
        store_row<__nv_bfloat16, 8>(lo + c + i, w);
      }
    }
  }
}

// ---- forward -----------------------------------------------------------------

template <int D>
struct FwdCfg {
  static constexpr uint32_t TILE = 128 * D * 2;
  static constexpr int SLOTS = D == 128 ? 5 : 8;  // ring of key and value tiles
  static constexpr uint32_t RING = 2 * TILE;      // behind the two query tiles
  static constexpr uint32_t BYTES = (2 + SLOTS) * TILE + 1024;
  static constexpr int S_COL = 0, O_COL = 256;    // 128 columns per group each
};

template <int D, bool kFine>
__global__ void __launch_bounds__(kTcThreads, 1) swa_fwd_tc_kernel(
    const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
    const __grid_constant__ CUtensorMap tv, SwaArgs a) {
  using Cf = FwdCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t q_full, full[Cf::SLOTS], empty[Cf::SLOTS], s_full[2], p_full[2], o_full[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // heavy CTAs (late rows: full windows) first
  const int q0 = ((int)gridDim.x - 1 - (int)blockIdx.x) * 256, h = blockIdx.y, b = blockIdx.z;
  const int hk = h / (a.H / a.Hk), W = a.window, S = a.sinks;
  const auto upto = [&](int x) { return x < a.T ? x : a.T; };
  const KeyRange all(q0, upto(q0 + 256), W, S, 128);

  if (tid == 0) {
    tc::mbar_init(&q_full, 1);
    for (int i = 0; i < Cf::SLOTS; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s_full[i], 1);
      tc::mbar_init(&p_full[i], 128);
      tc::mbar_init(&o_full[i], 1);
    }
    tc::mbar_init_fence();
    abort_flag = 0;
  }
  if (warp == 0) tc::tmem_alloc(&tmem_slot, 512);
  tc::tc_before_sync();
  __syncthreads();
  tc::tc_after_sync();
  const uint32_t tmem = tmem_slot;
  volatile int* ab = &abort_flag;

  if (warp == kLoadWarp) {
    if (lane == 0) {
      const bool two = q0 + 128 < a.T;
      tc::mbar_expect_tx(&q_full, (two ? 2 : 1) * Cf::TILE);
      for (int i = 0; i < (two ? 2 : 1); ++i)
        for (int c = 0; c < D; c += 64) tc::tma_load_4d(sm + i * Cf::TILE + c * 256, &tq, c, h, q0 + 128 * i, b, &q_full);
      for (int n = 0; n < 2 * all.count; ++n) {  // keys, values of one tile after the other
        const int slot = n % Cf::SLOTS, use = n / Cf::SLOTS;
        if (use && !tc::mbar_wait<false>(&empty[slot], (use - 1) & 1, a.err, tc::kErrTimeoutLoad, ab)) break;
        tc::mbar_expect_tx(&full[slot], Cf::TILE);
        for (int c = 0; c < D; c += 64)
          tc::tma_load_4d(sm + Cf::RING + slot * Cf::TILE + c * 256, n & 1 ? &tv : &tk, c, hk, all.tile(n / 2) * 128, b,
                          &full[slot]);
      }
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      const uint32_t ID_S = tc::idesc(128, 128, 1), ID_O = tc::idesc(128, D, 1) | tc::kMajorB;
      const KeyRange mine[2] = {KeyRange(q0, upto(q0 + 128), W, S, 128),
                                KeyRange(upto(q0 + 128), upto(q0 + 256), W, S, 128)};
      const uint32_t base = tc::smem_u32(sm);
      bool started[2] = {false, false};
      int p_use[2] = {0, 0};
      const auto landed = [&](int n) {
        return tc::mbar_wait<false>(&full[n % Cf::SLOTS], (n / Cf::SLOTS) & 1, a.err, tc::kErrTimeoutLoad, ab);
      };
      const auto scores = [&](int i, int n) {  // S_i = q_i k_n^T
        const uint32_t k = base + Cf::RING + (2 * n) % Cf::SLOTS * Cf::TILE, q = base + i * Cf::TILE;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t o = s / 4 * 16384 + s % 4 * 32;
          tc::mma_bf16_ss(tmem + Cf::S_COL + i * 128, tc::desc_sw128(q + o), tc::desc_sw128(k + o), ID_S, s > 0);
        }
        tc::mma_commit(&s_full[i]);
      };
      const auto release = [&](int n) {  // only where the slot is loaded again: every commit is waited for
        if (n + Cf::SLOTS < 2 * all.count) tc::mma_commit(&empty[n % Cf::SLOTS]);
      };
      tc::mbar_wait<false>(&q_full, 0, a.err, tc::kErrTimeoutLoad, ab);
      landed(0);
      tc::tc_after_sync();
      for (int i = 0; i < 2; ++i)
        if (mine[i].has(all.tile(0))) scores(i, 0);
      release(0);
      for (int n = 0; n < all.count && !*ab; ++n) {
        const int kt = all.tile(n);
        const bool more = n + 1 < all.count;
        landed(2 * n + 1);
        if (more) landed(2 * n + 2);
        const uint32_t v = base + Cf::RING + (2 * n + 1) % Cf::SLOTS * Cf::TILE;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (mine[i].has(kt)) {
            tc::mbar_wait<false>(&p_full[i], p_use[i]++ & 1, a.err, tc::kErrTimeoutMma, ab);
            tc::tc_after_sync();
#pragma unroll
            for (int s = 0; s < (kFine ? 16 : 8); ++s)  // O_i += P_i v
              tc::mma_bf16_ts(tmem + Cf::O_COL + i * 128, tmem + Cf::S_COL + i * 128 + s * 8,
                              tc::desc_sw128_mn(v + s % 8 * 2048, 16384u), ID_O, started[i] || s > 0);
            started[i] = true;
            if (kt == mine[i].end) tc::mma_commit(&o_full[i]);
          }
          if (more && mine[i].has(all.tile(n + 1))) scores(i, n + 1);
        }
        release(2 * n + 1);
        if (more) release(2 * n + 2);
      }
    }
  } else {
    const int i = warp >> 2, r0 = upto(q0 + 128 * i), t = q0 + tid;
    const KeyRange mine(r0, upto(q0 + 128 * i + 128), W, S, 128);
    const uint32_t s_lane = tc::tmem_lane_addr(tmem, warp, Cf::S_COL + i * 128);
    const uint32_t o_lane = tc::tmem_lane_addr(tmem, warp, Cf::O_COL + i * 128);
    const float s2 = a.scale * kLog2e;
    float top = -INFINITY, sum = 0.f;  // sums refer to 2^(s2 top)
    for (int n = 0; n < mine.count; ++n) {
      const int k0 = mine.tile(n) * 128;
      if (!warp_wait(&s_full[i], n & 1, a.err, tc::kErrTimeoutMma, ab)) break;
      tc::tc_after_sync();
      float x[128];
#pragma unroll
      for (int c = 0; c < 128; c += 32) tc::tmem_ld32(s_lane + c, x + c);
      tc::tmem_ld_wait();
      if (!(k0 + 127 <= r0 && (r0 + 127 - k0 < W || k0 + 127 < S))) {
        const int hi = t - k0, lo = hi - W, sk = S - k0;
#pragma unroll
        for (int c = 0; c < 128; ++c) x[c] = c <= hi && (c > lo || c < sk) ? x[c] : -INFINITY;
      }
      float m0 = x[0], m1 = x[1], m2 = x[2], m3 = x[3];
#pragma unroll
      for (int c = 4; c < 128; c += 4) {
        m0 = fmaxf(m0, x[c]);
        m1 = fmaxf(m1, x[c + 1]);
        m2 = fmaxf(m2, x[c + 2]);
        m3 = fmaxf(m3, x[c + 3]);
      }
      const float m = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
      const bool grow = n == 0 ? m > top : (m - top) * s2 > 8.f;  // false while a row has seen no key
      if (n > 0 && __any_sync(0xffffffffu, grow)) {
        // the commit of these scores covered the product before: O is complete
        const float f = grow ? ex2((top - m) * s2) : 1.f;
        sum *= f;
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          float o[16];
          tc::tmem_ld16(o_lane + c, o);
          tc::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] *= f;
          tc::tmem_st16(o_lane + c, o);
        }
      }
      if (grow) top = m;
      const float ref = top == -INFINITY ? 0.f : top * s2;
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        float w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          x[c + e] = ex2(fmaf(x[c + e], s2, -ref));
          x[c + e + 1] = ex2(fmaf(x[c + e + 1], s2, -ref));
          w[e / 2] = bf16_pair(x[c + e], x[c + e + 1]);
        }
        tc::tmem_st16(s_lane + c / 2, w);
        if (kFine) {  // what the rounding left, behind the 64 columns of the high parts
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint32_t hi = __float_as_uint(w[e / 2]);
            w[e / 2] = bf16_pair(x[c + e] - __uint_as_float(hi << 16), x[c + e + 1] - __uint_as_float(hi & 0xffff0000u));
          }
          tc::tmem_st16(s_lane + 64 + c / 2, w);
        }
      }
      tc::tmem_st_wait();
      tc::tc_before_sync();
      tc::mbar_arrive(&p_full[i]);
      float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
      for (int c = 0; c < 128; c += 4) {
        a0 += x[c];
        a1 += x[c + 1];
        a2 += x[c + 2];
        a3 += x[c + 3];
      }
      sum += (a0 + a1) + (a2 + a3);
    }
    if (mine.count) {
      warp_wait(&o_full[i], 0, a.err, tc::kErrTimeoutMma, ab);
      tc::tc_after_sync();
      const bool live = t < a.T;
      const size_t row = ((size_t)b * a.T + t) * a.H + h;
      store_lane<D>(o_lane, 1.f / sum, live ? static_cast<__nv_bfloat16*>(a.out) + row * D : nullptr,
                    live && a.olo ? static_cast<__nv_bfloat16*>(a.olo) + row * D : nullptr);
      if (live) a.lse[row] = fmaf(top, s2, log2f(sum)) * kLn2;
    }
  }
  tc::tc_before_sync();
  __syncthreads();
  tc::tc_after_sync();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// ---- backward ----------------------------------------------------------------

template <int D>
struct BwdCfg {
  static constexpr uint32_t BIG = 128 * D * 2;    // the CTA's own two tiles of 128 rows
  static constexpr uint32_t SMALL = 64 * D * 2;   // a ring stage holds two tiles of 64 rows
  static constexpr int STAGES = 4;
  static constexpr uint32_t RING = 2 * BIG, STAGE = 2 * SMALL;
  static constexpr uint32_t ROWS = RING + STAGES * STAGE;  // lse2, delta of a stage's 64 queries
  static constexpr uint32_t BYTES = ROWS + STAGES * 512 + 1024;
  static constexpr int S_COL = 0, P_COL = 128;    // scores and dP, 64 columns per group each
  static constexpr int A_COL = 256, B_COL = 384;  // accumulators
};

struct BwdBars {
  uint64_t own, full[4], empty[4], s_full[2], w_full[2], done;
  uint32_t tmem;
  int abort_flag;
};

__device__ __forceinline__ uint32_t bwd_setup(BwdBars& s) {
  if (threadIdx.x == 0) {
    tc::mbar_init(&s.own, 1);
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&s.full[i], 1);
      tc::mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s.s_full[i], 1);
      tc::mbar_init(&s.w_full[i], 128);
    }
    tc::mbar_init(&s.done, 1);
    tc::mbar_init_fence();
    s.abort_flag = 0;
  }
  if (threadIdx.x < 32) tc::tmem_alloc(&s.tmem, 512);
  tc::tc_before_sync();
  __syncthreads();
  tc::tc_after_sync();
  return s.tmem;
}

__device__ __forceinline__ void bwd_finish(uint32_t tmem) {
  tc::tc_before_sync();
  __syncthreads();
  tc::tc_after_sync();
  if (threadIdx.x < 32) tc::tmem_dealloc(tmem, 512);
}

// The products of both backward kernels over `count` stages: into group n & 1,
// S = own0 stage0^T and dP = own1 stage1^T (128 x 64, K = d); then, from the
// weights that the group put over them, acc_b += W_dP stage0 (dS with k or q)
// and, with kTwo, acc_a += W_S stage1 (P^T with dO).  Without kTwo dS lies over S.
template <int D, bool kTwo>
__device__ __forceinline__ void bwd_products(BwdBars& s, unsigned char* sm, uint32_t tmem, int count, int* err) {
  using Cf = BwdCfg<D>;
  volatile int* ab = &s.abort_flag;
  const uint32_t ID_S = tc::idesc(128, 64, 1), ID_A = tc::idesc(128, D, 1) | tc::kMajorB;
  const uint32_t base = tc::smem_u32(sm);
  const auto scores = [&](int n) {
    const uint32_t stage = base + Cf::RING + n % Cf::STAGES * Cf::STAGE;
    const int g = n & 1;
    tc::mbar_wait<false>(&s.full[n % Cf::STAGES], (n / Cf::STAGES) & 1, err, tc::kErrTimeoutLoad, ab);
    tc::tc_after_sync();
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t o = k / 4 * 16384 + k % 4 * 32, p = k / 4 * 8192 + k % 4 * 32;
      tc::mma_bf16_ss(tmem + Cf::S_COL + g * 64, tc::desc_sw128(base + o), tc::desc_sw128(stage + p), ID_S, k > 0);
    }
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t o = k / 4 * 16384 + k % 4 * 32, p = k / 4 * 8192 + k % 4 * 32;
      tc::mma_bf16_ss(tmem + Cf::P_COL + g * 64, tc::desc_sw128(base + Cf::BIG + o),
                      tc::desc_sw128(stage + Cf::SMALL + p), ID_S, k > 0);
    }
    tc::mma_commit(&s.s_full[g]);
  };
  tc::mbar_wait<false>(&s.own, 0, err, tc::kErrTimeoutLoad, ab);
  scores(0);
  if (count > 1) scores(1);
  for (int n = 0; n < count && !*ab; ++n) {
    const uint32_t stage = base + Cf::RING + n % Cf::STAGES * Cf::STAGE;
    const int g = n & 1;
    tc::mbar_wait<false>(&s.w_full[g], (n >> 1) & 1, err, tc::kErrTimeoutMma, ab);
    tc::tc_after_sync();
    if (kTwo) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        tc::mma_bf16_ts(tmem + Cf::A_COL, tmem + Cf::S_COL + g * 64 + k * 8,
                        tc::desc_sw128_mn(stage + Cf::SMALL + k * 2048, 8192u), ID_A, n > 0 || k > 0);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      tc::mma_bf16_ts(tmem + Cf::B_COL, tmem + (kTwo ? Cf::P_COL : Cf::S_COL) + g * 64 + k * 8,
                      tc::desc_sw128_mn(stage + k * 2048, 8192u), ID_A, n > 0 || k > 0);
    if (n + Cf::STAGES < count) tc::mma_commit(&s.empty[n % Cf::STAGES]);
    if (n + 1 == count) tc::mma_commit(&s.done);
    if (n + 2 < count) scores(n + 2);
  }
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) swa_dq_tc_kernel(
    const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tg,
    const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, SwaArgs a, SwaBwdLayout L) {
  using Cf = BwdCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ BwdBars s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q0 = ((int)gridDim.x - 1 - (int)blockIdx.x) * 128, h = blockIdx.y, b = blockIdx.z;
  const int hk = h / (a.H / a.Hk), W = a.window, S = a.sinks;
  const KeyRange keys(q0, q0 + 128 < a.T ? q0 + 128 : a.T, W, S, 64);
  const uint32_t tmem = bwd_setup(s);
  volatile int* ab = &s.abort_flag;
  if (warp == kLoadWarp) {
    if (lane == 0) {
      tc::mbar_expect_tx(&s.own, 2 * Cf::BIG);
      for (int c = 0; c < D; c += 64) {
        tc::tma_load_4d(sm + c * 256, &tq, c, h, q0, b, &s.own);
        tc::tma_load_4d(sm + Cf::BIG + c * 256, &tg, c, h, q0, b, &s.own);
      }
      for (int n = 0; n < keys.count; ++n) {
        const int slot = n % Cf::STAGES, use = n / Cf::STAGES, k0 = keys.tile(n) * 64;
        if (use && !tc::mbar_wait<false>(&s.empty[slot], (use - 1) & 1, a.err, tc::kErrTimeoutLoad, ab)) break;
        unsigned char* st = sm + Cf::RING + slot * Cf::STAGE;
        tc::mbar_expect_tx(&s.full[slot], Cf::STAGE);
        for (int c = 0; c < D; c += 64) {
          tc::tma_load_4d(st + c * 128, &tk, c, hk, k0, b, &s.full[slot]);
          tc::tma_load_4d(st + Cf::SMALL + c * 128, &tv, c, hk, k0, b, &s.full[slot]);
        }
      }
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) bwd_products<D, false>(s, sm, tmem, keys.count, a.err);
  } else {
    const int g = warp >> 2, t = q0 + (tid & 127);
    const uint32_t s_lane = tc::tmem_lane_addr(tmem, warp, Cf::S_COL + g * 64);
    const uint32_t p_lane = tc::tmem_lane_addr(tmem, warp, Cf::P_COL + g * 64);
    const size_t at = ((size_t)b * a.H + h) * L.Tp + t;
    const float lse2 = reinterpret_cast<const float*>(a.ws + L.lse2)[at];
    const float delta = reinterpret_cast<const float*>(a.ws + L.delta)[at];
    const float s2 = a.scale * kLog2e;
    for (int n = g; n < keys.count; n += 2) {
      const int k0 = keys.tile(n) * 64;
      if (!warp_wait(&s.s_full[g], (n >> 1) & 1, a.err, tc::kErrTimeoutMma, ab)) break;
      tc::tc_after_sync();
      const bool all = k0 + 63 <= q0 && (q0 + 127 - k0 < W || k0 + 63 < S);
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        float x[32], dp[32], w[16];
        tc::tmem_ld32(s_lane + c, x);
        tc::tmem_ld32(p_lane + c, dp);
        tc::tmem_ld_wait();
        if (!all) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            x[e] = visible(t, k0 + c + e, W, S) && !single_key(t, W, S) ? x[e] : -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = ex2(fmaf(x[e], s2, -lse2)) * (dp[e] - delta);
#pragma unroll
        for (int e = 0; e < 32; e += 2) w[e / 2] = bf16_pair(x[e], x[e + 1]);
        tc::tmem_st16(s_lane + c / 2, w);
      }
      tc::tmem_st_wait();
      tc::tc_before_sync();
      tc::mbar_arrive(&s.w_full[g]);
    }
    warp_wait(&s.done, 0, a.err, tc::kErrTimeoutMma, ab);
    tc::tc_after_sync();
    if (g == 0) {
      const size_t row = ((size_t)b * a.T + t) * a.H + h;
      store_lane<D>(tc::tmem_lane_addr(tmem, warp, Cf::B_COL), a.scale,
                    t < a.T ? static_cast<__nv_bfloat16*>(a.dq) + row * D : nullptr, nullptr);
    }
  }
  bwd_finish(tmem);
}

// blockIdx.x < tiles: a key tile's band, all query heads of its group (only
// blockIdx.y < Hk); beyond: a piece of the first tokens' far queries, one head.
template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) swa_dkv_tc_kernel(
    const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
    const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tg, SwaArgs a, SwaBwdLayout L,
    int tiles, int has_far) {
  using Cf = BwdCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ BwdBars s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.z, group = a.H / a.Hk, W = a.window, S = a.sinks;
  const bool far = (int)blockIdx.x >= tiles;
  const int piece = far ? (int)blockIdx.x - tiles : 0, k0 = far ? 0 : (int)blockIdx.x * 128;
  const int band_end = k0 + 127 + W < a.T ? k0 + 127 + W : a.T;
  int h0 = blockIdx.y, heads = 1, q_lo, q_hi;
  if (far) {
    q_lo = piece * kSwaPiece > band_end ? piece * kSwaPiece : band_end;
    q_hi = (piece + 1) * kSwaPiece < a.T ? (piece + 1) * kSwaPiece : a.T;
    if (q_lo >= q_hi) return;  // the sum skips it too
  } else {
    if ((int)blockIdx.y >= a.Hk) return;
    h0 = blockIdx.y * group;
    heads = group;
    q_lo = k0;
    q_hi = band_end;
  }
  const int hk = h0 / group, qt0 = q_lo / 64, per = (q_hi - 1) / 64 - qt0 + 1, count = per * heads;
  const uint32_t tmem = bwd_setup(s);
  volatile int* ab = &s.abort_flag;
  if (warp == kLoadWarp) {
    if (lane == 0) {
      tc::mbar_expect_tx(&s.own, 2 * Cf::BIG);
      for (int c = 0; c < D; c += 64) {
        tc::tma_load_4d(sm + c * 256, &tk, c, hk, k0, b, &s.own);
        tc::tma_load_4d(sm + Cf::BIG + c * 256, &tv, c, hk, k0, b, &s.own);
      }
      for (int n = 0; n < count; ++n) {
        const int slot = n % Cf::STAGES, use = n / Cf::STAGES, h = h0 + n / per, t0 = (qt0 + n % per) * 64;
        if (use && !tc::mbar_wait<false>(&s.empty[slot], (use - 1) & 1, a.err, tc::kErrTimeoutLoad, ab)) break;
        unsigned char* st = sm + Cf::RING + slot * Cf::STAGE;
        float* rows = reinterpret_cast<float*>(sm + Cf::ROWS + slot * 512);
        const size_t at = ((size_t)b * a.H + h) * L.Tp + t0;
        tc::mbar_expect_tx(&s.full[slot], Cf::STAGE + 512);
        for (int c = 0; c < D; c += 64) {
          tc::tma_load_4d(st + c * 128, &tq, c, h, t0, b, &s.full[slot]);
          tc::tma_load_4d(st + Cf::SMALL + c * 128, &tg, c, h, t0, b, &s.full[slot]);
        }
        tc::bulk_g2s(rows, reinterpret_cast<const float*>(a.ws + L.lse2) + at, 256, &s.full[slot]);
        tc::bulk_g2s(rows + 64, reinterpret_cast<const float*>(a.ws + L.delta) + at, 256, &s.full[slot]);
      }
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) bwd_products<D, true>(s, sm, tmem, count, a.err);
  } else {
    const int g = warp >> 2, key = k0 + (tid & 127);
    const uint32_t s_lane = tc::tmem_lane_addr(tmem, warp, Cf::S_COL + g * 64);
    const uint32_t p_lane = tc::tmem_lane_addr(tmem, warp, Cf::P_COL + g * 64);
    const float s2 = a.scale * kLog2e;
    for (int n = g; n < count; n += 2) {
      const int q0 = (qt0 + n % per) * 64, slot = n % Cf::STAGES;
      const float4* rows = reinterpret_cast<const float4*>(sm + Cf::ROWS + slot * 512);
      // the scores' commit follows the stage's arrival, but only this wait lets
      // this thread read what the copy wrote
      if (!warp_wait(&s.full[slot], (n / Cf::STAGES) & 1, a.err, tc::kErrTimeoutLoad, ab)) break;
      if (!warp_wait(&s.s_full[g], (n >> 1) & 1, a.err, tc::kErrTimeoutMma, ab)) break;
      tc::tc_after_sync();
      const bool all = k0 + 127 <= q0 && (q0 + 63 - k0 < W || k0 + 127 < S) && q0 >= q_lo && q0 + 63 < q_hi;
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        float x[32], dp[32], w[16];
        tc::tmem_ld32(s_lane + c, x);
        tc::tmem_ld32(p_lane + c, dp);
        tc::tmem_ld_wait();
        if (!all) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int t = q0 + c + e;
            x[e] = t >= q_lo && t < q_hi && visible(t, key, W, S) ? x[e] : -INFINITY;
            if (single_key(t, W, S)) dp[e] = INFINITY;  // marks dS = 0 below
          }
        }
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 l = rows[(c + e) / 4], d = rows[16 + (c + e) / 4];
          const float ls[4] = {l.x, l.y, l.z, l.w}, ds[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[e + k] = ex2(fmaf(x[e + k], s2, -ls[k]));
            dp[e + k] = !all && dp[e + k] == INFINITY ? 0.f : x[e + k] * (dp[e + k] - ds[k]);
          }
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) w[e / 2] = bf16_pair(x[e], x[e + 1]);
        tc::tmem_st16(s_lane + c / 2, w);
#pragma unroll
        for (int e = 0; e < 32; e += 2) w[e / 2] = bf16_pair(dp[e], dp[e + 1]);
        tc::tmem_st16(p_lane + c / 2, w);
      }
      tc::tmem_st_wait();
      tc::tc_before_sync();
      tc::mbar_arrive(&s.w_full[g]);
    }
    warp_wait(&s.done, 0, a.err, tc::kErrTimeoutMma, ab);
    tc::tc_after_sync();
    // group 0 writes dv, group 1 dk
    const uint32_t lanes = tc::tmem_lane_addr(tmem, warp, g ? Cf::B_COL : Cf::A_COL);
    const float f = g ? a.scale : 1.f;
    const bool first = key < S && key < a.T && has_far;  // rows that other items add to: fp32 parts
    float* part = nullptr;
    if (first && far)
      part = reinterpret_cast<float*>(a.ws + L.part) +
             (((((size_t)(g ? 0 : 1) * L.pieces + piece) * a.B + b) * a.H + h0) * S + key) * D;
    else if (first)
      part = reinterpret_cast<float*>(a.ws + L.band) + ((((size_t)(g ? 0 : 1) * a.B + b) * a.Hk + hk) * S + key) * D;
    const bool plain = !far && !first && key < a.T;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(g ? a.dk : a.dv) + (((size_t)b * a.T + key) * a.Hk + hk) * D;
    store_lane<D>(lanes, f, plain ? dst : nullptr, nullptr);
    if (k0 < S && has_far) {
#pragma unroll
      for (int c = 0; c < D; c += 16) {
        float v[16];
        __syncwarp();
        tc::tmem_ld16(lanes + c, v);
        tc::tmem_ld_wait();
        if (part) {
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(part + c + e) = make_float4(v[e] * f, v[e + 1] * f, v[e + 2] * f, v[e + 3] * f);
        }
      }
    }
  }
  bwd_finish(tmem);
}

template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// Rows of at most this many keys take the finer weights.  Measured with bf16
// gradients, relative to their own rounding (1.41 is what rounding dS alone
// costs): dq 1.72 at 1 to 2 keys, 1.52 at 9, 1.45 at 129 with one bf16 weight.
constexpr int kFineKeys = 256;

template <int D, bool kFine>
cudaError_t fwd_go(const SwaArgs& a, cudaStream_t st) {
  using Cf = FwdCfg<D>;
  CUtensorMap tq, tk, tv;
  if (!make_tmap_bthd(&tq, a.q, 2, a.B, a.T, a.H, D, 64, true, 128) ||
      !make_tmap_bthd(&tk, a.k, 2, a.B, a.T, a.Hk, D, 64, true, 128) ||
      !make_tmap_bthd(&tv, a.v, 2, a.B, a.T, a.Hk, D, 64, true, 128))
    return cudaErrorInvalidValue;
  cudaError_t e = allow_smem(swa_fwd_tc_kernel<D, kFine>, Cf::BYTES);
  if (e != cudaSuccess) return e;
  prof_begin(st, "swa_fwd_tc");
  swa_fwd_tc_kernel<D, kFine><<<dim3((a.T + 255) / 256, a.H, a.B), kTcThreads, Cf::BYTES, st>>>(tq, tk, tv, a);
  prof_end(st);
  return cudaGetLastError();
}

template <int D>
cudaError_t bwd_go(const SwaArgs& a, cudaStream_t st) {
  using Cf = BwdCfg<D>;
  const SwaBwdLayout L = swa_bwd_layout(a.B, a.T, a.H, a.Hk, a.d, a.window, a.sinks);
  CUtensorMap big[4], small[4];  // q, dO, k, v with 128 and 64 rows to a box
  const void* src[4] = {a.q, a.dO, a.k, a.v};
  for (int i = 0; i < 4; ++i)
    if (!make_tmap_bthd(&big[i], src[i], 2, a.B, a.T, i < 2 ? a.H : a.Hk, D, 64, true, 128) ||
        !make_tmap_bthd(&small[i], src[i], 2, a.B, a.T, i < 2 ? a.H : a.Hk, D, 64, true, 64))
      return cudaErrorInvalidValue;
  cudaError_t e = allow_smem(swa_dkv_tc_kernel<D>, Cf::BYTES);
  if (e == cudaSuccess) e = allow_smem(swa_dq_tc_kernel<D>, Cf::BYTES);
  if (e == cudaSuccess) e = launch_swa_delta(a, L, st);
  if (e != cudaSuccess) return e;
  const int tiles = (a.T + 127) / 128;
  const int has_far = a.sinks > 0 && 127 + a.window < a.T;
  prof_begin(st, "swa_dkv_tc");
  swa_dkv_tc_kernel<D><<<dim3(tiles + (has_far ? L.pieces : 0), has_far ? a.H : a.Hk, a.B), kTcThreads, Cf::BYTES, st>>>(
      big[2], big[3], small[0], small[1], a, L, tiles, has_far);
  prof_end(st);
  prof_begin(st, "swa_dq_tc");
  swa_dq_tc_kernel<D><<<dim3(tiles, a.H, a.B), kTcThreads, Cf::BYTES, st>>>(big[0], big[1], small[2], small[3], a, L);
  prof_end(st);
  e = cudaGetLastError();
  if (e == cudaSuccess && has_far) e = launch_swa_sink_sum(a, L, 128, st);
  return e;
}

}  // namespace

bool swa_tc_supported(int d, int dtype) { return dtype == 1 && (d == 64 || d == 128); }
cudaError_t launch_swa_fwd_tc(const SwaArgs& a, cudaStream_t st) {
  const int keys = a.window + a.sinks < a.T ? a.window + a.sinks : a.T;  // window, sinks <= T
  if (keys <= kFineKeys) return a.d == 64 ? fwd_go<64, true>(a, st) : fwd_go<128, true>(a, st);
  return a.d == 64 ? fwd_go<64, false>(a, st) : fwd_go<128, false>(a, st);
}
cudaError_t launch_swa_bwd_tc(const SwaArgs& a, cudaStream_t st) { return a.d == 64 ? bwd_go<64>(a, st) : bwd_go<128>(a, st); }

}  // namespace kd
