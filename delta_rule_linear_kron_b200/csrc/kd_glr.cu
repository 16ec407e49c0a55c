// kd_glr.cu -- element-wise gated linear recurrence: forward, backward, step.
//
// Per channel, with a = e^{a_log}:
//   l_t = a log sigma(f~_t),  f_t = e^{l_t},  m_t = sqrt(1 - f_t^2),  i_t = sigma(i~_t)
//   h_t = f_t h_{t-1} + m_t i_t x_t
// Backward for <dh, out> + <dhT, hT>, with u_t = f_t g_t:
//   g_t = dh_t + u_{t+1}  (u_T = dhT),   dh0 = u_0
//   dx = g m i,  di~ = g m x i (1 - i),  dl = g (f h_{t-1} - i x f^2 / m)
//   df~ = dl a sigma(-f~),  da_log = sum dl l
//
// By its bytes (8.06 per element forward and 14.06 backward with bf16, the saved
// states among them) a stream through HBM, but with enough arithmetic per element
// that nothing may be computed twice.  One pass: a cluster of C CTAs takes 64
// channels and C consecutive chunks of 64 tokens at a time.  TMA brings the
// chunks' tiles a step ahead.  A warp holds 8 tokens, a lane 2 channels (one
// f32x2 register pair, so that most of the arithmetic is two channels an
// instruction); each thread scans its 8 tokens from zero, the warps'
// (prod f, h) pairs combine through shared memory and the CTAs' through
// distributed shared memory, and the thread then adds its start state's part,
// from registers.  The chain along the sequence is only ceil(T / 64C) cluster
// exchanges long.  B1 T16384 D2048, with the states saved: bf16 forward 114 us
// (271 MB, 2.4 TB/s), backward 184 us (472 MB, 2.6 TB/s); fp32 114 us (539 MB,
// 4.7 TB/s) and 357 us (941 MB, 2.6 TB/s: its tiles leave room for one CTA per
// SM); one step of 256 x 2048 7.2 us.  No unit is at its rate: 110 and 188
// instructions per pair of channels and token take 53 and 52% of the issue slots
// (8 of them on the special function unit, 31 and 18%), HBM is at 26 and 28%.
// What bounds them is latency: 13 warps per SM (256 CTAs leave 40 of the 148 SMs
// with one CTA) of which a scheduler finds one ready per cycle, in chains of
// dependent arithmetic, of waits for tiles, states and the exchange.
//
// Accuracy: the state's error builds up over 1 / (1 - f) steps, so f must not
// carry a bias.  With L = log2 f = n + r, |r| <= 1/2, and q = 2^r - 1 by a
// polynomial, f = 2^n + 2^n q and f - 1 = (2^n - 1) + 2^n q; where n = 0 (every
// gate that keeps more than 0.7) f - 1 is q itself, and 1 - f^2 = -(f - 1)(1 + f)
// keeps its relative precision however close f is to 1.
#include "kd_hybrid.h"
#include "kd_rows.cuh"
#include "kd_tc.cuh"
#include "kd_tmap.h"

namespace kd {

namespace {

constexpr int kWarps = 8, kTok = 8;    // a chunk: 8 warps of 8 tokens
constexpr int kChans = 64;             // channels of a CTA, 2 per lane
static_assert(kWarps * kTok == kChunk, "a CTA takes one chunk at a time");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rsq(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// fminf and fmaxf return the other operand for a NaN; these return the NaN
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
constexpr float kLog2e = 1.44269504088896f;
constexpr float kLn2 = 0.693147180559945f;

// Two channels in one register pair.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 pk(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 pk(float a) { return pk(a, a); }
__device__ __forceinline__ float2 un(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// -e^{a_log} log2 e of two channels.  Finite where e^{a_log} leaves fp32, so
// that a gate without a logarithm (1, as for tokens behind the end) stays 1.
__device__ __forceinline__ F2 exponents(const float* a_log) {
  return pk(max_nan(-kLog2e * expf(a_log[0]), -3.402823466e38f), max_nan(-kLog2e * expf(a_log[1]), -3.402823466e38f));
}

struct Gates {
  F2 L;  // log2 f, with kBack
  F2 f;
  F2 w;  // 1 - f^2
  F2 i;  // sigma(i~)
  F2 s, j;  // with kBack: sigma(-f~), and sigma(-i~) = 2^k sigma(i~) (1 - i would cancel)
};

// na2: -a log2 e.  A NaN in zf or na2 makes f NaN, one in zi i: no bound below
// may take it for a number, or a run that has diverged would go on as if its
// gates were shut.
template <bool kBack>
__device__ __forceinline__ Gates gates(float2 zf, float2 zi, F2 na2) {
  Gates g;
  const float ex = ex2(-kLog2e * fabsf(zf.x)), ey = ex2(-kLog2e * fabsf(zf.y));
  const F2 e = pk(ex, ey);
  const F2 d = add2(e, pk(2.f));
  // sigma(i~) = 1 / (1 + 2^k); the bound (2e-37, 0 for every purpose) keeps the
  // product of reciprocals below in range.  That product is f's too, which the
  // forward may spoil with a NaN of i~ (h_t is NaN with i alone); the backward
  // may not, since f_t carries the gradients of earlier tokens, so it keeps the
  // NaN aside (k2n) and gives it to i.
  F2 k2, k2n;
  if (kBack) {
    const float kx = ex2(-kLog2e * zi.x), ky = ex2(-kLog2e * zi.y);
    k2 = pk(fminf(kx, 0x1p122f), fminf(ky, 0x1p122f));
    k2n = pk(min_nan(kx, 0x1p122f), min_nan(ky, 0x1p122f));
  } else {
    k2 = pk(ex2(min_nan(-kLog2e * zi.x, 122.f)), ex2(min_nan(-kLog2e * zi.y, 122.f)));
  }
  const F2 c = add2(k2, pk(1.f));
  // the reciprocals of 2 + e, 1 + 2^k (and 1 + e) from one of their product
  F2 dc = mul2(d, c), one = add2(e, pk(1.f));
  const float2 den = un(kBack ? mul2(dc, one) : dc);
  const F2 r = pk(rcp(den.x), rcp(den.y));
  F2 rd;
  if (kBack) {
    g.s = mul2(mul2(r, dc), pk(zf.x >= 0.f ? ex : 1.f, zf.y >= 0.f ? ey : 1.f));
    const F2 ro = mul2(r, one);
    g.i = fma2(k2n, pk(0.f), mul2(ro, d));
    g.j = mul2(k2, g.i);
    rd = mul2(ro, c);
  } else {
    g.i = mul2(r, d);
    rd = mul2(r, c);
  }
  // log(1 + e) = 2 artanh(u), u = e / (2 + e) <= 1/3: artanh(u) = u + u z p(z),
  // z = u^2, p of least error on [0, 1/9] (1.6e-8 of the sum)
  const F2 u = mul2(e, rd), z = mul2(u, u);
  F2 p = fma2(z, pk(1.34418249e-1f), pk(1.41156361e-1f));
  p = fma2(z, p, pk(2.00038910e-1f));
  p = fma2(z, p, pk(3.33333194e-1f));
  p = fma2(mul2(u, z), p, u);
  const F2 soft = fma2(p, pk(2.f), pk(fmaxf(-zf.x, 0.f), fmaxf(-zf.y, 0.f)));
  const float2 Lf = un(mul2(soft, na2));
  // the backward's dl L must be 0, not 0 * infinity, where f~ starts a new sequence
  if (kBack) g.L = pk(max_nan(Lf.x, -1e30f), max_nan(Lf.y, -1e30f));
  const F2 Lc = pk(max_nan(Lf.x, -127.f), max_nan(Lf.y, -127.f));
  const float kMagic = 12582912.f;  // 1.5 2^23: rounds to an integer, kept in the low bits
  const F2 t = add2(Lc, pk(kMagic));
  const F2 n = add2(t, pk(-kMagic)), x = fma2(n, pk(-1.f), Lc);
  // 2^n by its bits; n = -127 gives exactly 0
  const float2 t2 = un(t);
  const F2 s = pk(__uint_as_float((__float_as_uint(t2.x) << 23) + 0x3f800000u),
                  __uint_as_float((__float_as_uint(t2.y) << 23) + 0x3f800000u));
  // (2^x - 1) / x of least error on [-1/2, 1/2] (1.3e-8 of it)
  F2 q = fma2(x, pk(1.54697351e-4f), pk(1.33908668e-3f));
  q = fma2(x, q, pk(9.61803086e-3f));
  q = fma2(x, q, pk(5.55035695e-2f));
  q = fma2(x, q, pk(2.40226507e-1f));
  q = fma2(x, q, pk(6.93147182e-1f));
  q = mul2(q, x);
  g.f = fma2(s, q, s);
  const F2 y = fma2(s, q, add2(s, pk(-1.f)));  // f - 1; for n = 0 it is q
  g.w = mul2(y, fma2(g.f, pk(-1.f), pk(-1.f)));
  return g;
}

// 1 / m.  The bound only meets gates so close to 1 that w rounds to 0: w / m
// is 0 there, and d l vanishes faster than 1 / m is large.
__device__ __forceinline__ F2 inv_m(F2 w) {
  const float2 v = un(w);
  return pk(rsq(fmaxf(v.x, 1e-30f)), rsq(fmaxf(v.y, 1e-30f)));
}

template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
  using type = __nv_bfloat162;
  static __device__ __forceinline__ float2 f(type v) { return __bfloat1622float2(v); }
  static __device__ __forceinline__ type of(F2 a) {
    const float2 v = un(a);
    return __floats2bfloat162_rn(v.x, v.y);
  }
};
template <> struct Pair<float> {
  using type = float2;
  static __device__ __forceinline__ float2 f(type v) { return v; }
  static __device__ __forceinline__ type of(F2 a) { return un(a); }
};

// (f products, states) of a run of tokens, two channels; `then` appends a later run.
struct Run {
  F2 f, h;
};
__device__ __forceinline__ Run then(Run a, Run b) { return {mul2(a.f, b.f), fma2(b.f, a.h, b.h)}; }

// This lane's run of CTA `rank` into CTA `to`, whose barrier counts the bytes.
// (A cluster barrier would do too, but its release waits for the outputs that
// the CTA has stored to global memory, on every step: 1.6 us of a 5 us step.)
__device__ __forceinline__ void send(Run* slot, uint64_t* bar, int to, Run v) {
  const float2 f = un(v.f), h = un(v.h);
  tc::st_async_v4(tc::mapa(tc::smem_u32(slot), to), make_float4(f.x, f.y, h.x, h.y), tc::mapa(tc::smem_u32(bar), to));
}

template <typename T, int kArrays>
struct GlrCfg {
  static constexpr uint32_t TILE = kChunk * kChans * sizeof(T);
  static constexpr uint32_t STAGE = kArrays * TILE;
  static constexpr uint32_t RUNS = 2 * STAGE;                                   // Run [2][kWarps][32]
  static constexpr uint32_t CRUNS = RUNS + 2 * kWarps * 32 * 16;                // Run [2][kGlrMaxCluster][32]
  static constexpr uint32_t U = CRUNS + 2 * kGlrMaxCluster * 32 * 16;           // backward: F2 [2][kWarps][32]
  static constexpr uint32_t KEEP = U + 2 * kWarps * 32 * 8;                     // backward: F2 [kTok][threads]
  static constexpr uint32_t BYTES = (kArrays == 3 ? U : KEEP + kTok * kWarps * 32 * 8) + 128;
};

// The tiles of one chunk (kArrays tensors) into a stage.
template <typename T, int kArrays>
__device__ __forceinline__ void load_stage(unsigned char* sm, int stage, const CUtensorMap* const (&maps)[kArrays], int c,
                                           int t0, int b, uint64_t* bar) {
  using Cf = GlrCfg<T, kArrays>;
  tc::mbar_expect_tx(bar, Cf::STAGE);
#pragma unroll
  for (int i = 0; i < kArrays; ++i) tc::tma_load_4d(sm + stage * Cf::STAGE + i * Cf::TILE, maps[i], c, 0, t0, b, bar);
}

// Tokens behind the sequence's end and channels behind D: this thread's words
// of a stage from token k on are set so that the gate keeps everything and
// writes nothing (f = 1 and m = 0 exactly), and the loops over the tokens need
// no branch.
template <typename T, int kArrays>
__device__ __forceinline__ void neutral_from(int k, unsigned char* st, int at) {
  using V = typename Pair<T>::type;
  for (int j = k; j < kTok; ++j)
#pragma unroll
    for (int i = 0; i < kArrays; ++i)
      reinterpret_cast<V*>(st + i * GlrCfg<T, kArrays>::TILE)[at + j * 32] = Pair<T>::of(pk(i == 2 ? 1e4f : 0.f));
  tc::fence_proxy_async();
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32, 2) glr_fwd_kernel(
    const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mi,
    const __grid_constant__ CUtensorMap mf, const float* __restrict__ a_log, const float* __restrict__ h0,
    T* __restrict__ out, float* __restrict__ hT, float* __restrict__ states, int T_, int D, int NC, int C, int* err) {
  using P = Pair<T>;
  using V = typename P::type;
  using Cf = GlrCfg<T, 3>;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((128u - (tc::smem_u32(smem_raw) & 127u)) & 127u);
  __shared__ uint64_t full[2], runs_in[2];
  __shared__ int abort_flag;
  Run(*runs)[kWarps][32] = reinterpret_cast<Run(*)[kWarps][32]>(sm + Cf::RUNS);
  Run(*cruns)[kGlrMaxCluster][32] = reinterpret_cast<Run(*)[kGlrMaxCluster][32]>(sm + Cf::CRUNS);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = C > 1 ? (int)tc::cluster_rank() : 0;
  const int b = blockIdx.y, c0 = (int)(blockIdx.x / C) * kChans, c = c0 + lane * 2;
  const bool live = c < D;
  const CUtensorMap* const maps[3] = {&mx, &mi, &mf};
  const int steps = (NC + C - 1) / C;
  if (threadIdx.x == 0) {
    tc::mbar_init(&full[0], 1);
    tc::mbar_init(&full[1], 1);
    tc::mbar_init(&runs_in[0], 1);
    tc::mbar_init(&runs_in[1], 1);
    tc::mbar_init_fence();
    abort_flag = 0;
    for (int s = 0; s < 2; ++s)
      if (s * C + rank < NC) load_stage<T, 3>(sm, s, maps, c0, (s * C + rank) * kChunk, b, &full[s]);
  }
  F2 na2 = pk(0.f), carry = pk(0.f);
  if (live) {
    na2 = exponents(a_log + c);
    if (h0) carry = *reinterpret_cast<const F2*>(h0 + (size_t)b * D + c);
  }
  __syncthreads();
  if (C > 1) tc::cluster_sync();  // every CTA of the cluster has started
  const size_t base = (size_t)b * T_ * D + c;
  // Tokens of this thread in chunk n.  (Asked for again where the outputs are
  // stored, as their address is: kept over the step it costs 4%.)
  const auto tokens = [&](int n) {
    const long long left = T_ - ((long long)n * kChunk + warp * kTok);
    return !live || left <= 0 ? 0 : left < kTok ? (int)left : kTok;
  };
  for (int s = 0; s < steps; ++s) {
    const int n = s * C + rank, par = s & 1;
    unsigned char* st = sm + par * Cf::STAGE;
    const int own = warp * kTok * 32 + lane;  // this thread's first word of a tile
    if (n < NC) tc::mbar_wait<false>(&full[par], (s >> 1) & 1, err, tc::kErrTimeoutLoad, &abort_flag);
    if (const int k = tokens(n); k < kTok) neutral_from<T, 3>(k, st, own);
    const V *xs = reinterpret_cast<const V*>(st) + own, *is = reinterpret_cast<const V*>(st + Cf::TILE) + own;
    const V* fs = reinterpret_cast<const V*>(st + 2 * Cf::TILE) + own;
    Run r[kTok], run = {pk(1.f), pk(0.f)};
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      const float2 x = P::f(xs[j * 32]);
      const Gates g = gates<false>(P::f(fs[j * 32]), P::f(is[j * 32]), na2);
      run = then(run, {g.f, mul2(mul2(mul2(g.w, inv_m(g.w)), g.i), pk(x.x, x.y))});
      r[j] = run;
    }
    if (C > 1 && threadIdx.x == 0) tc::mbar_expect_tx(&runs_in[par], (uint32_t)C * 32 * sizeof(Run));
    runs[par][warp][lane] = run;
    __syncthreads();  // and every thread is through with the stage
    if (threadIdx.x == 0 && n + 2 * C < NC)
      load_stage<T, 3>(sm, par, maps, c0, (n + 2 * C) * kChunk, b, &full[par]);
    Run pre = {pk(1.f), pk(0.f)};
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w)
      if (w < warp) pre = then(pre, runs[par][w][lane]);
    const Run all = then(pre, run);  // in the last warp: the whole chunk
    F2 mine = carry;  // state at the start of this CTA's chunk
    if (C > 1) {
      // the last warp hands the chunk's run to every CTA; the buffer's readers of
      // two steps ago are through: their CTA's runs of the step before have arrived here
      if (warp == kWarps - 1)
        for (int q = 0; q < C; ++q) send(&cruns[par][rank][lane], &runs_in[par], q, all);
      tc::mbar_wait<true>(&runs_in[par], (s >> 1) & 1, err, tc::kErrTimeoutCluster, &abort_flag);
#pragma unroll
      for (int q = 0; q < kGlrMaxCluster; ++q)
        if (q < C) {
          const Run v = cruns[par][q][lane];
          if (q == rank) mine = carry;
          carry = fma2(v.f, carry, v.h);
        }
    } else {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) carry = fma2(runs[par][w][lane].f, carry, runs[par][w][lane].h);
    }
    const F2 h = fma2(pre.f, mine, pre.h);
    if (states && warp == 0 && live && n < NC) *reinterpret_cast<F2*>(states + ((size_t)b * NC + n) * D + c) = mine;
    const int k = tokens(s * C + rank);
    T* o = out + base + ((size_t)(s * C + rank) * kChunk + warp * kTok) * D;
#pragma unroll
    for (int j = 0; j < kTok; ++j)
      if (j < k) __stcs(reinterpret_cast<V*>(o + (size_t)j * D), P::of(fma2(r[j].f, h, r[j].h)));
  }
  if (C > 1) tc::cluster_sync();  // no CTA leaves while another may still write to it
  if (hT && rank == 0 && warp == 0 && live) *reinterpret_cast<F2*>(hT + (size_t)b * D + c) = carry;
}

// The backward walks the chunks from the last.  The states h_{t-1} come from
// the chunk's saved start state, run forward again over the tokens in
// registers, so they are fp32 (the bf16 output would put its rounding into
// df~ and da_log).  What the last pass over the tokens needs and registers do
// not hold waits in shared memory: a sigma(-f~), and log2 f in place of the
// f~ and i~ that it came from; each thread reads back only what it wrote.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 2 ? 2 : 1) glr_bwd_kernel(
    const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mi,
    const __grid_constant__ CUtensorMap mf, const __grid_constant__ CUtensorMap mg, const float* __restrict__ a_log,
    const float* __restrict__ states, const float* __restrict__ dhT, T* __restrict__ dx, T* __restrict__ di,
    T* __restrict__ df, float* __restrict__ part, float* __restrict__ dh0, int T_, int D, int NC, int C, int* err) {
  using P = Pair<T>;
  using V = typename P::type;
  using Cf = GlrCfg<T, 4>;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((128u - (tc::smem_u32(smem_raw) & 127u)) & 127u);
  __shared__ uint64_t full[2], runs_in[2];
  __shared__ int abort_flag;
  Run(*runs)[kWarps][32] = reinterpret_cast<Run(*)[kWarps][32]>(sm + Cf::RUNS);
  Run(*cruns)[kGlrMaxCluster][32] = reinterpret_cast<Run(*)[kGlrMaxCluster][32]>(sm + Cf::CRUNS);
  F2(*us)[kWarps][32] = reinterpret_cast<F2(*)[kWarps][32]>(sm + Cf::U);
  F2* keep = reinterpret_cast<F2*>(sm + Cf::KEEP) + threadIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = C > 1 ? (int)tc::cluster_rank() : 0;
  const int b = blockIdx.y, c0 = (int)(blockIdx.x / C) * kChans, c = c0 + lane * 2;
  const bool live = c < D;
  const CUtensorMap* const maps[4] = {&mx, &mi, &mf, &mg};
  const int steps = (NC + C - 1) / C;
  // step s runs chunk ((steps - 1 - s) C + rank); a stage is loaded one step ahead
  const auto chunk = [&](int s) { return (steps - 1 - s) * C + rank; };
  int uses[2] = {0, 0};
  if (threadIdx.x == 0) {
    tc::mbar_init(&full[0], 1);
    tc::mbar_init(&full[1], 1);
    tc::mbar_init(&runs_in[0], 1);
    tc::mbar_init(&runs_in[1], 1);
    tc::mbar_init_fence();
    abort_flag = 0;
    for (int s = 0; s < 2 && s < steps; ++s)
      if (chunk(s) < NC) load_stage<T, 4>(sm, s, maps, c0, chunk(s) * kChunk, b, &full[s]);
  }
  F2 na2 = pk(0.f), carry = pk(0.f);
  if (live) {
    na2 = exponents(a_log + c);
    if (dhT) carry = *reinterpret_cast<const F2*>(dhT + (size_t)b * D + c);
  }
  const F2 a = mul2(na2, pk(-kLn2));
  F2 da = pk(0.f);
  __syncthreads();
  if (C > 1) tc::cluster_sync();  // every CTA of the cluster has started
  for (int s = 0; s < steps; ++s) {
    const int n = chunk(s), par = s & 1;
    const long long t0 = (long long)n * kChunk + warp * kTok, left = T_ - t0;
    const int k = !live || left <= 0 ? 0 : left < kTok ? (int)left : kTok;
    unsigned char* st = sm + par * Cf::STAGE;
    const int own = warp * kTok * 32 + lane;  // this thread's first word of a tile
    const V *xs = reinterpret_cast<const V*>(st) + own, *gs = reinterpret_cast<const V*>(st + 3 * Cf::TILE) + own;
    V *is = reinterpret_cast<V*>(st + Cf::TILE) + own, *fs = reinterpret_cast<V*>(st + 2 * Cf::TILE) + own;
    F2 start = pk(0.f);
    if (live && n < NC) start = *reinterpret_cast<const F2*>(states + ((size_t)b * NC + n) * D + c);
    if (n < NC) {
      tc::mbar_wait<false>(&full[par], uses[par] & 1, err, tc::kErrTimeoutLoad, &abort_flag);
      ++uses[par];
    }
    if (k < kTok) neutral_from<T, 4>(k, st, own);
    F2 F[kTok], M[kTok], Q[kTok], J[kTok];  // f, m i, f i x / m, sigma(-i~)
    Run run = {pk(1.f), pk(0.f)};
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      const float2 x = P::f(xs[j * 32]);
      const Gates g = gates<true>(P::f(fs[j * 32]), P::f(is[j * 32]), na2);
      const float2 L = un(g.L);
      *reinterpret_cast<float*>(&is[j * 32]) = L.x;
      *reinterpret_cast<float*>(&fs[j * 32]) = L.y;
      keep[j * kWarps * 32] = mul2(a, g.s);
      const F2 r = inv_m(g.w), x2 = pk(x.x, x.y);
      F[j] = g.f;
      J[j] = g.j;
      M[j] = mul2(mul2(g.w, r), g.i);
      Q[j] = mul2(mul2(g.f, x2), mul2(g.i, r));
      run = then(run, {g.f, mul2(M[j], x2)});
    }
    F2 u = pk(0.f);
#pragma unroll
    for (int j = kTok - 1; j >= 0; --j) {
      const float2 g = P::f(gs[j * 32]);
      u = mul2(F[j], add2(pk(g.x, g.y), u));
    }
    if (C > 1 && threadIdx.x == 0) tc::mbar_expect_tx(&runs_in[par], (uint32_t)C * 32 * sizeof(Run));
    runs[par][warp][lane] = run;
    us[par][warp][lane] = u;
    __syncthreads();
    // every thread is through with the other stage (the step before)
    if (threadIdx.x == 0 && s > 0 && s + 1 < steps && chunk(s + 1) < NC)
      load_stage<T, 4>(sm, par ^ 1, maps, c0, chunk(s + 1) * kChunk, b, &full[par ^ 1]);
    // what this warp's last token gets from the later ones: runs of (f products, u)
    Run post = {pk(1.f), pk(0.f)};
#pragma unroll
    for (int w = kWarps - 1; w > 0; --w)
      if (w > warp) post = then(post, {runs[par][w][lane].f, us[par][w][lane]});
    const Run all = then(post, {run.f, u});  // in the first warp: the whole chunk
    if (C > 1) {
      if (warp == 0)
        for (int q = 0; q < C; ++q) send(&cruns[par][rank][lane], &runs_in[par], q, all);
    }
    // state before this warp's first token, then before each of its tokens
    F2 h = start;
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w)
      if (w < warp) h = fma2(runs[par][w][lane].f, h, runs[par][w][lane].h);
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      const float2 x = P::f(xs[j * 32]);
      Q[j] = fma2(Q[j], pk(-1.f), h);  // h_{t-1} - f i x / m, whose product with u_t is dl
      h = fma2(F[j], h, mul2(M[j], pk(x.x, x.y)));
    }
    F2 mine = carry;
    if (C > 1) {
      tc::mbar_wait<true>(&runs_in[par], (s >> 1) & 1, err, tc::kErrTimeoutCluster, &abort_flag);
#pragma unroll
      for (int q = kGlrMaxCluster - 1; q >= 0; --q)
        if (q < C) {
          const Run v = cruns[par][q][lane];
          if (q == rank) mine = carry;
          carry = fma2(v.f, carry, v.h);
        }
    } else {
#pragma unroll
      for (int w = kWarps - 1; w >= 0; --w) carry = fma2(runs[par][w][lane].f, carry, us[par][w][lane]);
    }
    F2 v = fma2(post.f, mine, post.h);
    const size_t off = ((size_t)b * T_ + t0) * D + c;
#pragma unroll
    for (int j = kTok - 1; j >= 0; --j) {
      const float2 vg = P::f(gs[j * 32]), x = P::f(xs[j * 32]);
      const F2 g = add2(pk(vg.x, vg.y), v), gm = mul2(g, M[j]);
      v = mul2(F[j], g);
      const F2 dl = mul2(v, Q[j]);
      da = fma2(dl, pk(*reinterpret_cast<const float*>(&is[j * 32]), *reinterpret_cast<const float*>(&fs[j * 32])), da);
      if (j < k) {
        const size_t to = off + (size_t)j * D;
        __stcs(reinterpret_cast<V*>(dx + to), P::of(gm));
        __stcs(reinterpret_cast<V*>(di + to), P::of(mul2(mul2(gm, pk(x.x, x.y)), J[j])));
        __stcs(reinterpret_cast<V*>(df + to), P::of(mul2(dl, keep[j * kWarps * 32])));
      }
    }
    tc::fence_proxy_async();  // the words written over f~ and i~, before the stage is loaded again
  }
  if (C > 1) tc::cluster_sync();  // no CTA leaves while another may still write to it
  if (dh0 && rank == 0 && warp == 0 && live) *reinterpret_cast<F2*>(dh0 + (size_t)b * D + c) = carry;
  // da_log: the warps' sums in a fixed order, one row per CTA of the cluster
  __syncthreads();
  us[0][warp][lane] = da;
  __syncthreads();
  if (warp == 0 && live) {
    F2 t = pk(0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t = add2(t, us[0][w][lane]);
    *reinterpret_cast<F2*>(part + ((size_t)b * C + rank) * D + c) = mul2(t, pk(kLn2));
  }
}

// 32 channels x 8 shares of the rows; each share in order, then the shares.
__global__ void __launch_bounds__(256) glr_dalog_kernel(const float* __restrict__ part, int rows, int D,
                                                        float* __restrict__ da_log) {
  __shared__ float share[8][32];
  const int lane = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float t = 0.f;
  if (c < D) {
#pragma unroll 4
    for (int r = y; r < rows; r += 8) t += part[(size_t)r * D + c];
  }
  share[y][lane] = t;
  __syncthreads();
  if (y || c >= D) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) t += share[k][lane];
  da_log[c] = t;
}

template <typename T>
__global__ void __launch_bounds__(128) glr_decode_kernel(const T* __restrict__ x, const T* __restrict__ ip,
                                                         const T* __restrict__ fp, const float* __restrict__ a_log,
                                                         float* __restrict__ h, T* __restrict__ out, long long n,
                                                         int D) {
  using P = Pair<T>;
  using V = typename P::type;
  const long long at = ((long long)blockIdx.x * 128 + threadIdx.x) * 2;
  if (at >= n) return;
  const int c = (int)(at % D);
  const float2 vx = P::f(*reinterpret_cast<const V*>(x + at)), vi = P::f(*reinterpret_cast<const V*>(ip + at));
  const float2 vf = P::f(*reinterpret_cast<const V*>(fp + at));
  const F2 s = *reinterpret_cast<const F2*>(h + at);
  const Gates g = gates<false>(vf, vi, exponents(a_log + c));
  const F2 y = fma2(g.f, s, mul2(mul2(mul2(g.w, inv_m(g.w)), g.i), pk(vx.x, vx.y)));
  *reinterpret_cast<F2*>(h + at) = y;
  *reinterpret_cast<V*>(out + at) = P::of(y);
}

// CTAs of a cluster (chunks taken at a time): enough CTAs for all of 148 SMs,
// as far as the sequence has chunks, and at most the portable 8.  Forward and
// backward in us, clusters of 8 and of 1: 114 and 426, 184 and 826 (B1 T16384
// D2048: 256 CTAs and 32); where D and B make 256 CTAs by themselves, clusters
// of 1 and of 2: 175 and 187, 323 and 337 (B8 T4096 D2048).
int cluster_size(const GlrArgs& a, int NC) {
  const long long lanes = (long long)((a.D + kChans - 1) / kChans) * a.B;
  int C = 1;
  while (C < kGlrMaxCluster && C < NC && lanes * C < 148) C *= 2;
  return C;
}

template <typename K, typename... A>
cudaError_t launch_cluster(K kernel, dim3 grid, int C, size_t smem, cudaStream_t st, A... args) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = C;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// a chunk's tile of a [B,T,D] tensor: 64 channels of 64 tokens
template <typename T>
bool tile_map(CUtensorMap* m, const GlrArgs& a, const void* p) {
  return make_tmap_bthd(m, p, sizeof(T), a.B, a.T, 1, a.D, kChans, false, kChunk);
}

template <typename T>
cudaError_t glr_fwd_t(const GlrArgs& a, cudaStream_t st) {
  const int NC = (a.T + kChunk - 1) / kChunk, C = cluster_size(a, NC);
  const dim3 grid((unsigned)((a.D + kChans - 1) / kChans) * C, a.B);
  CUtensorMap mx, mi, mf;
  if (!tile_map<T>(&mx, a, a.x) || !tile_map<T>(&mi, a, a.i_pre) || !tile_map<T>(&mf, a, a.f_pre))
    return cudaErrorInvalidValue;
  prof_begin(st, "glr_fwd");
  const cudaError_t e = launch_cluster(glr_fwd_kernel<T>, grid, C, GlrCfg<T, 3>::BYTES, st, mx, mi, mf, a.a_log, a.h0,
                                       static_cast<T*>(a.out), a.hT, a.states, a.T, a.D, NC, C, a.err);
  prof_end(st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t glr_bwd_t(const GlrArgs& a, cudaStream_t st) {
  const int NC = (a.T + kChunk - 1) / kChunk, C = cluster_size(a, NC);
  const dim3 grid((unsigned)((a.D + kChans - 1) / kChans) * C, a.B);
  CUtensorMap mx, mi, mf, mg;
  if (!tile_map<T>(&mx, a, a.x) || !tile_map<T>(&mi, a, a.i_pre) || !tile_map<T>(&mf, a, a.f_pre) ||
      !tile_map<T>(&mg, a, a.dh))
    return cudaErrorInvalidValue;
  prof_begin(st, "glr_bwd");
  cudaError_t e = launch_cluster(glr_bwd_kernel<T>, grid, C, GlrCfg<T, 4>::BYTES, st, mx, mi, mf, mg, a.a_log,
                                 a.states_in, a.dhT, static_cast<T*>(a.dx), static_cast<T*>(a.di_pre),
                                 static_cast<T*>(a.df_pre), a.part, a.dh0, a.T, a.D, NC, C, a.err);
  prof_end(st);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  prof_begin(st, "glr_dalog");
  glr_dalog_kernel<<<(a.D + 31) / 32, 256, 0, st>>>(a.part, a.B * C, a.D, a.da_log);
  prof_end(st);
  return cudaGetLastError();
}

template <typename T>
cudaError_t glr_decode_t(const GlrArgs& a, cudaStream_t st) {
  const long long n = (long long)a.B * a.D;
  prof_begin(st, "glr_decode");
  glr_decode_kernel<T><<<(unsigned)((n / 2 + 127) / 128), 128, 0, st>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.i_pre), static_cast<const T*>(a.f_pre), a.a_log, a.hT,
      static_cast<T*>(a.out), n, a.D);
  prof_end(st);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_glr_fwd(const GlrArgs& a, cudaStream_t st) {
  return a.dtype == 1 ? glr_fwd_t<__nv_bfloat16>(a, st) : glr_fwd_t<float>(a, st);
}
cudaError_t launch_glr_bwd(const GlrArgs& a, cudaStream_t st) {
  return a.dtype == 1 ? glr_bwd_t<__nv_bfloat16>(a, st) : glr_bwd_t<float>(a, st);
}
cudaError_t launch_glr_decode(const GlrArgs& a, cudaStream_t st) {
  return a.dtype == 1 ? glr_decode_t<__nv_bfloat16>(a, st) : glr_decode_t<float>(a, st);
}

}  // namespace kd
